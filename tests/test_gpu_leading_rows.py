"""Packed sequences whose first offset is above 0, and offsets that are wrong: the rows ahead of the first sequence
belong to no sequence (a serving batch with its single tokens ahead of its prompts), and nothing outside the arrays
is read or written whatever the offsets say.

Bounds as for the convolution of rows that start at 0 (16 fp32 roundings of its magnitude, twice that for its gradient,
one rounding per add of a sum over tokens): where a sequence lies does not change its arithmetic."""
import math

import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OPS = 16
GAPS = [1, 8, 10, 33, 64]  # multiples of a tile of tokens and others, below and above W - 1 behind one
LENS = [5, 0, 41, 1, 30]


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


def offsets(gap, lens):
    return (gap + torch.tensor([0] + lens).cumsum(0)).to(device=DEV, dtype=torch.int32)


def make_conv(tokens, dim, W, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(tokens, dim, device=DEV, generator=g).to(TYPES[dtype])
    w = torch.randn(dim, W, device=DEV, generator=g) / W ** 0.5
    return g, x, w, torch.randn(dim, device=DEV, generator=g) * 0.1


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("dtype,W,dim", [("bf16", 4, 72), ("f32", 3, 20), ("f16", 2, 37)])
def test_convolution_and_gradient(gap, dtype, W, dim):
    tokens = gap + sum(LENS) + 3
    g, x, w, bias = make_conv(tokens, dim, W, dtype, 300 + gap)
    cu = offsets(gap, LENS)
    dy = [torch.randn(tokens, dim, device=DEV, generator=g).to(x.dtype)]
    x[:gap], x[-3:] = float("nan"), float("nan")  # rows of no sequence are not used
    out = (torch.full((tokens, dim), 7.0, device=DEV, dtype=x.dtype),)
    ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu, out=out)
    r = ref.conv(x, w, bias, cu=cu, dy=dy[0])
    k = r["covered"]
    ref.assert_within(out[0].cpu()[k], r["y"][k], r["mag"][k], x.dtype, "y", OPS)
    assert (out[0].cpu()[~k] == 7).all(), "rows of no sequence were written"
    b = ops.conv1d_tm_bwd(x, w, dy, bias, cu_seqlens=cu)
    ref.assert_within(b["dx"].cpu()[k], r["dx"][k], r["mag_dx"][k], x.dtype, "dx", 2 * OPS)
    assert (b["dx"].cpu()[~k] == 0).all()
    adds = max(32, math.ceil(tokens / 256)) + 256 + 2 * OPS
    ref.assert_within(b["dw"], r["dw"], r["mag_dw"], torch.float32, "dw", adds)
    ref.assert_within(b["dbias"], r["db"], r["mag_db"], torch.float32, "dbias", adds)


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("dtype,W,dim", [("bf16", 4, 72), ("f32", 4, 20), ("f16", 3, 37)])
def test_convolution_on_a_cache(gap, dtype, W, dim):
    tokens = gap + sum(LENS)
    g, x, w, bias = make_conv(tokens, dim, W, dtype, 400 + gap)
    state = torch.randn(8, dim, W - 1, device=DEV, generator=g)
    slots = torch.tensor([3, 7, -1, 0, 5], dtype=torch.int32, device=DEV)
    fresh = torch.tensor([0, 0, 0, 1, 0], dtype=torch.bool, device=DEV)
    cu = offsets(gap, LENS)
    r = ref.conv(x, w, bias, cu=cu, state=state, slots=slots, fresh=fresh)
    out = (torch.full((tokens, dim), 7.0, device=DEV, dtype=x.dtype),)
    ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu, state=state, slots=slots, fresh=fresh, out=out)
    k = r["covered"]
    ref.assert_within(out[0].cpu()[k], r["y"][k], r["mag"][k], x.dtype, "y", OPS)
    assert (out[0].cpu()[~k] == 7).all(), "rows of no sequence, or of padding, were written"
    assert torch.equal(state.cpu().double(), r["state"])


@pytest.mark.parametrize("gap", [8, 10, 64])
def test_autograd_leaves_leading_rows_zero(gap):
    g, x, w, bias = make_conv(gap + sum(LENS), 48, 4, "f32", 500 + gap)
    cu = offsets(gap, LENS)
    for t in (x, w, bias):
        t.requires_grad_(True)
    a, b = ops.causal_conv1d_tm_fn(x, w, bias, splits=(32, 16), cu_seqlens=cu)
    assert (a[:gap] == 0).all() and (b[:gap] == 0).all()
    dy = torch.randn(x.shape, device=DEV, generator=g)
    (torch.cat([a, b], 1) * dy).sum().backward()
    r = ref.conv(x, w, bias, cu=cu, dy=dy)
    ref.assert_within(x.grad, r["dx"], r["mag_dx"], torch.float32, "dx", 2 * OPS)
    assert (x.grad[:gap] == 0).all()
    ref.assert_within(w.grad, r["dw"], r["mag_dw"], torch.float32, "dw", 32 + 256 + 2 * OPS)


def test_many_rows_ahead():
    """Enough rows for the longest tiles; an element's arithmetic does not depend on where its sequence lies."""
    gap, lens = 1003, [2000, 1, 1996]
    g, x, w, bias = make_conv(gap + sum(lens), 4096, 4, "bf16", 600)
    out = (torch.full(x.shape, 7.0, device=DEV, dtype=x.dtype),)
    ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=offsets(gap, lens), out=out)
    (want,) = ops.conv1d_tm_fwd(x[gap:], w, bias, cu_seqlens=offsets(0, lens))
    assert (out[0][:gap] == 7).all() and torch.equal(out[0][gap:], want)


BAD = [[0, 10, 5, 30], [0, 10, 20, 99], [-4, 10, 20, 30], [25, 10, 20, 30], [64, 70, 80, 90], [30, 0, 0, 30],
       [17, -9, 30, 2], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dtype,dim", [("bf16", 16), ("f32", 9)])
@pytest.mark.parametrize("cache", [False, True])
def test_bad_offsets_stay_inside_the_arrays(bad, dtype, dim, cache):
    """Guard rows of NaN around x (one that is read shows in y) and of a sentinel around the outputs."""
    n, guard = 30, 40
    g, wide, w, bias = make_conv(n + 2 * guard, dim, 4, dtype, 800)
    wide[:guard], wide[-guard:] = float("nan"), float("nan")
    x = wide[guard:guard + n]
    room = torch.full((n + 2 * guard, dim), 7.0, device=DEV, dtype=x.dtype)
    out = (room[guard:guard + n],)
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    states = torch.full((5, dim, 3), 7.0, device=DEV)
    kw = dict(state=states[1:4]) if cache else {}
    ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu, out=out, **kw)
    assert ops.lib().ss_device_fault(1) == 8
    assert torch.isfinite(room).all() and torch.isfinite(states).all()
    assert (room[:guard] == 7).all() and (room[-guard:] == 7).all()
    assert (states[0] == 7).all() and (states[4] == 7).all()
    droom = torch.full((n + 2 * guard, dim), 7.0, device=DEV, dtype=x.dtype)
    dy = torch.full((n + 2 * guard, dim), float("nan"), device=DEV, dtype=x.dtype)
    dy[guard:guard + n] = 1.0
    b = ops.conv1d_tm_bwd(x, w, [dy[guard:guard + n]], bias, cu_seqlens=cu, dx=droom[guard:guard + n])
    assert ops.lib().ss_device_fault(1) == 8
    assert torch.isfinite(droom).all() and torch.isfinite(b["dw"]).all() and torch.isfinite(b["dbias"]).all()
    assert (droom[:guard] == 7).all() and (droom[-guard:] == 7).all()
