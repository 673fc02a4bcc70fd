"""Time-major causal conv1d over packed rows against its plain 64-bit form:
ragged sequences, window caches, padding, strided rows, gradients.

Counted in fp32 roundings: a pre-activation is W fused products and a bias
(W + 1 of its magnitude), the SiLU adds one exponential, one reciprocal and two
products (ex2 and rcp are within 2 ulp, the exponent's scaling adds |pre| 2^-24
of the result; |silu'| <= 1.1): 16 of the magnitude cover both."""
import math

import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OPS = 16


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


def make(lead, dim, W, dtype, seed, pad=0, off=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = torch.randn(*lead, dim + pad, device=DEV, generator=g).to(TYPES[dtype])
    x = rows[..., off:off + dim]
    w = torch.randn(dim, W, device=DEV, generator=g) / W ** 0.5
    bias = torch.randn(dim, device=DEV, generator=g) * 0.1
    return g, x, w, bias


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def check_fwd(out, r, dtype):
    y = torch.cat([o.reshape(-1, o.shape[-1]) for o in out], dim=1)
    k = r["covered"]
    ref.assert_within(y.cpu()[k], r["y"][k], r["mag"][k], dtype, "y", OPS)


@pytest.mark.parametrize("dtype,W,dim,splits,pad,off", [
    ("bf16", 4, 320, (192, 64, 64), 72, 64), ("f16", 4, 1056, (1024, 16, 16), 0, 0), ("f32", 3, 76, (60, 8, 8), 4, 4),
    ("bf16", 2, 37, (30, 7), 3, 1), ("f16", 1, 24, None, 0, 0), ("f32", 4, 5, (2, 2, 1), 0, 0)])
@pytest.mark.parametrize("lens", [[1], [70, 0, 1, 2, 3, 129, 64, 5], [0, 0], [4097]])
def test_ragged_forward_and_backward(dtype, W, dim, splits, pad, off, lens):
    tokens = sum(lens) + 3  # three rows behind the last sequence
    g, x, w, bias = make((tokens,), dim, W, dtype, 11 + W, pad, off)
    cu = cu_of(lens)
    widths = splits or (dim,)
    out = tuple(torch.full((tokens, s), 7.0, device=DEV, dtype=x.dtype) for s in widths)
    got = ops.conv1d_tm_fwd(x, w, bias, splits=splits, cu_seqlens=cu, out=out)
    dy = [torch.randn(tokens, s, device=DEV, generator=g).to(x.dtype) for s in widths]
    r = ref.conv(x, w, bias, cu=cu, dy=torch.cat(dy, 1))
    check_fwd(got, r, x.dtype)
    assert all((o[sum(lens):] == 7).all() for o in got), "rows behind the last sequence were written"
    b = ops.conv1d_tm_bwd(x, w, dy, bias, cu_seqlens=cu)
    ref.assert_within(b["dx"], r["dx"], r["mag_dx"], x.dtype, "dx", 2 * OPS)
    # a sum over n tokens in strips of at least 32 and at most 256 strips: each add is one rounding of the magnitude
    adds = max(32, math.ceil(tokens / 256)) + 256 + 2 * OPS
    ref.assert_within(b["dw"], r["dw"], r["mag_dw"], torch.float32, "dw", adds)
    ref.assert_within(b["dbias"], r["db"], r["mag_db"], torch.float32, "dbias", adds)


@pytest.mark.parametrize("dtype,W", [("bf16", 4), ("f32", 2), ("f16", 3), ("bf16", 1)])
def test_windows_in_a_cache(dtype, W):
    lens = [5, 0, 1, 2, 40, 0, 9]
    dim, room = 136, 12
    g, x, w, bias = make((sum(lens),), dim, W, dtype, 21)
    state = torch.randn(room, dim, W - 1, device=DEV, generator=g)
    slots = torch.tensor([3, 11, 0, -1, 7, 5, 2], dtype=torch.int32, device=DEV)
    fresh = torch.tensor([0, 0, 0, 0, 1, 1, 0], dtype=torch.bool, device=DEV)
    r = ref.conv(x, w, bias, cu=cu_of(lens), state=state, slots=slots, fresh=fresh)
    out = (torch.full((sum(lens), dim), 7.0, device=DEV, dtype=x.dtype),)
    got = ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu_of(lens), state=state, slots=slots, fresh=fresh, out=out)
    check_fwd(got, r, x.dtype)
    assert (got[0].cpu()[~r["covered"]] == 7).all(), "a padded sequence's rows were written"
    assert torch.equal(state.cpu().double(), r["state"]), "windows hold stored inputs exactly, others stay"


def test_pieces_through_the_cache_equal_one_call():
    g, x, w, bias = make((300,), 64, 4, "bf16", 31)
    (whole,) = ops.conv1d_tm_fwd(x, w, bias)
    state = torch.full((1, 64, 3), 5.0, device=DEV)
    at, parts = 0, []
    for i, n in enumerate([1, 1, 2, 0, 130, 166]):
        fresh = torch.tensor([i == 0], device=DEV)
        parts.append(ops.conv1d_tm_fwd(x[at:at + n], w, bias, state=state, fresh=fresh)[0])
        at += n
    assert torch.equal(torch.cat(parts), whole)


def test_dense_batch_equals_offsets():
    g, x, w, bias = make((3, 50), 72, 4, "bf16", 41, pad=8, off=8)
    a = ops.conv1d_tm_fwd(x, w, bias, splits=(40, 16, 16))
    b = ops.conv1d_tm_fwd(x.reshape(150, -1), w, bias, splits=(40, 16, 16), cu_seqlens=cu_of([50] * 3))
    for p, q in zip(a, b):
        assert p.shape[:2] == (3, 50) and torch.equal(p.reshape(150, -1), q)


def test_no_bias_no_silu_and_gradients_by_differences():
    """The loss is linear in y, and y is linear in x, w without the SiLU: the difference quotient is exact up to
    rounding.  With the SiLU, central differences of step h err by h^2 |y'''| / 6."""
    g, x, w, bias = make((40,), 8, 4, "f32", 51)
    cu = cu_of([17, 23])
    dy = torch.randn(40, 8, device=DEV, generator=g)
    b = ops.conv1d_tm_bwd(x, w, [dy], bias, cu_seqlens=cu)
    loss = lambda x, w, bias: float((ref.conv(x, w, bias, cu=cu)["y"] * dy.cpu().double()).sum())
    h = 1e-4
    for name, t, grad in (("x", x, b["dx"]), ("w", w, b["dw"]), ("bias", bias, b["dbias"])):
        for k in (0, 7, t.numel() // 2 + 1 if t.numel() > 8 else 3, t.numel() - 1):
            v = []
            for sgn in (1, -1):
                args = {"x": x.double().cpu(), "w": w.double().cpu(), "bias": bias.double().cpu()}
                args[name] = args[name].clone()
                args[name].reshape(-1)[k] += sgn * h
                v.append(loss(**args))
            want = (v[0] - v[1]) / (2 * h)
            # fp32 gradient: <= 64 roundings of a sum of at most 40 terms of size ~10; differences: h^2
            assert abs(float(grad.reshape(-1)[k]) - want) <= 64 * 2 ** -24 * 400 + 1e-6, (name, k)
    (y,) = ops.conv1d_tm_fwd(x, w, cu_seqlens=cu, silu=False)
    r = ref.conv(x, w, None, cu=cu, silu=False, dy=dy)
    ref.assert_within(y, r["y"], r["mag"], torch.float32, "y without SiLU", OPS)
    b = ops.conv1d_tm_bwd(x, w, [dy], cu_seqlens=cu, silu=False)
    ref.assert_within(b["dx"], r["dx"], r["mag_dx"], torch.float32, "dx without SiLU", OPS)


def test_gradient_into_a_column_slice():
    g, x, w, bias = make((90,), 64, 4, "bf16", 61, pad=32, off=16)
    dy = [torch.randn(90, 64, device=DEV, generator=g).to(x.dtype)]
    wide = torch.full((90, 96), 3.0, device=DEV, dtype=x.dtype)
    ops.conv1d_tm_bwd(x, w, dy, bias, dx=wide[:, 16:80])
    b = ops.conv1d_tm_bwd(x, w, dy, bias)
    assert torch.equal(wide[:, 16:80], b["dx"])
    assert (wide[:, :16] == 3).all() and (wide[:, 80:] == 3).all()


def test_autograd():
    g, x, w, bias = make((2, 33), 48, 4, "f32", 71)
    for t in (x, w, bias):
        t.requires_grad_(True)
    a, b = ops.causal_conv1d_tm_fn(x, w, bias, splits=(32, 16))
    da = torch.randn(2, 33, 32, device=DEV, generator=g)
    (a * da).sum().backward()  # the second piece is unused: its gradient is zero
    r = ref.conv(x, w, bias, dy=torch.cat([da, torch.zeros(2, 33, 16, device=DEV)], 2))
    ref.assert_within(x.grad.reshape(66, 48), r["dx"], r["mag_dx"], torch.float32, "dx", 2 * OPS)
    ref.assert_within(w.grad, r["dw"], r["mag_dw"], torch.float32, "dw", 300 + 2 * OPS)
    ref.assert_within(bias.grad, r["db"], r["mag_db"], torch.float32, "dbias", 300 + 2 * OPS)


def test_repeatable():
    g, x, w, bias = make((5000,), 200, 4, "bf16", 81)
    dy = [torch.randn(5000, 200, device=DEV, generator=g).to(x.dtype)]
    a, b = (ops.conv1d_tm_bwd(x, w, dy, bias) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_masked_rows_do_not_leak():
    """NaN and infinity behind the last sequence, in a neighbour and in a skipped slot's window stay there."""
    g, x, w, bias = make((64,), 64, 4, "bf16", 91)
    clean = x.clone()
    x[10:20], x[50:] = float("nan"), float("inf")
    cu = torch.tensor([0, 10, 20, 50], dtype=torch.int32, device=DEV)
    state = torch.zeros(4, 64, 3, device=DEV)
    state[3] = float("nan")
    fresh = torch.tensor([0, 0, 1], dtype=torch.bool, device=DEV)
    slots = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)  # the last one starts afresh on a slot of NaN
    (y,) = ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu, state=state, slots=slots, fresh=fresh)
    (want,) = ops.conv1d_tm_fwd(clean, w, bias, cu_seqlens=cu)
    for a, b in ((0, 10), (20, 50)):
        assert torch.equal(y[a:b], want[a:b])
    assert torch.isfinite(state[[0, 2, 3]]).all()
    dy = [torch.randn(64, 64, device=DEV, generator=g).to(x.dtype)]
    keep = dy[0].clone()
    dy[0][50:] = float("nan")
    b = ops.conv1d_tm_bwd(clean, w, dy, bias, cu_seqlens=cu)
    want = ops.conv1d_tm_bwd(clean[:50], w, [keep[:50].contiguous()], bias, cu_seqlens=cu)
    assert torch.equal(b["dx"][:50], want["dx"]) and (b["dx"][50:] == 0).all()
    assert torch.isfinite(b["dw"]).all() and torch.isfinite(b["dbias"]).all()


def test_bad_slots_and_offsets_are_reported_and_stay_in_bounds():
    g, x, w, bias = make((30,), 16, 4, "bf16", 101)
    state = torch.randn(3, 16, 3, device=DEV, generator=g)
    before = state.clone()
    cu = cu_of([10, 10, 10])
    out = (torch.full((30, 16), 7.0, device=DEV, dtype=x.dtype),)
    slots = torch.tensor([1, 1, 9], dtype=torch.int32, device=DEV)  # the second is taken, the third does not exist
    ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu, state=state, slots=slots, out=out)
    assert ops.lib().ss_device_fault(1) == 8
    r = ref.conv(x, w, bias, cu=cu, state=before, slots=[1, -1, -1])
    check_fwd(out, r, x.dtype)
    assert (out[0][10:] == 7).all() and torch.equal(state.cpu().double(), r["state"])
    for bad in ([0, 10, 5, 30], [0, 10, 20, 99], [-4, 10, 20, 30]):
        ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device=DEV))
        assert ops.lib().ss_device_fault(1) == 8


def test_captured_call_follows_offsets_and_slots():
    g, x, w, bias = make((64,), 32, 4, "bf16", 111)
    cu, slots = cu_of([20, 44]), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    fresh = torch.zeros(2, dtype=torch.bool, device=DEV)
    state = torch.zeros(4, 32, 3, device=DEV)
    out = (torch.empty(64, 32, device=DEV, dtype=x.dtype),)
    call = lambda: ops.conv1d_tm_fwd(x, w, bias, cu_seqlens=cu, state=state, slots=slots, fresh=fresh, out=out)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    cu.copy_(cu_of([50, 14]))
    slots.copy_(torch.tensor([3, 2], dtype=torch.int32))
    fresh.fill_(True)
    graph.replay()
    r = ref.conv(x, w, bias, cu=cu, state=state, slots=slots, fresh=fresh)
    check_fwd(out, r, x.dtype)
