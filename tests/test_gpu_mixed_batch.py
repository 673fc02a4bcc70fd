"""A serving batch with its single tokens ahead of its prompts: one projection, one output, the tokens' rows by the
step, the others by the prompts' operators with offsets that start behind them.  The projection's rows are as long as
its columns, not padded: their slices start on no 16-byte boundary."""
import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops
from test_gpu_mixer_run import EPS, Layer, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


class Unpadded(Layer):
    def __init__(self, *a, **k):
        super().__init__(*a, **k)
        self.width = self.d + self.dim + self.nh


@pytest.mark.parametrize("nh,ng,N,group,dtype", [
    (10, 1, 128, 640, torch.bfloat16), (6, 2, 64, 64, torch.float16), (5, 1, 64, 320, torch.bfloat16)])
@pytest.mark.parametrize("singles", [1, 9, 40])
def test_tokens_ahead_of_prompts(nh, ng, N, group, dtype, singles):
    m = Unpadded(nh, ng, N, group, 900 + nh + singles, dtype)
    lens = [130, 3, 200]
    tokens = singles + sum(lens)
    offsets = [singles, singles + 130, singles + 133, tokens]
    row = m.rows(tokens)
    win, state = m.caches(singles + 5)
    win0, state0 = win.clone(), state.clone()
    at, to = torch.arange(singles, dtype=torch.int32, device=DEV) + 4, i32(2, 0, 3)
    fresh = torch.tensor([True, False, False], device=DEV)
    z, xbc, dt = m.cut(row)

    y = torch.full((tokens, nh, 64), 7.0, device=DEV, dtype=dtype)
    ops.ssd_step(xbc[:singles], dt[:singles], m.w, m.A, win, state, conv_bias=m.bias, D=m.D, dt_bias=m.dt_bias, slots=at,
                 ngroups=ng, out=y[:singles])
    one = y[:singles].clone()
    pieces = tuple(torch.full((tokens, s), 7.0, device=DEV, dtype=dtype) for s in m.splits)
    ops.conv1d_tm_fwd(xbc, m.w, m.bias, splits=m.splits, cu_seqlens=i32(*offsets), state=win, slots=to, fresh=fresh,
                      out=pieces)
    x, B, C = (p.unflatten(1, s) for p, s in zip(pieces, ((nh, 64), (ng, N), (ng, N))))
    ops.ssd_prefill(x, dt, m.A, B, C, state=state, D=m.D, dt_bias=m.dt_bias, cu_seqlens=i32(*offsets), slots=to,
                    fresh=fresh, out=y)
    out, _ = ops.gated_norm_fwd(y.flatten(1), z, m.norm_w, group=group, eps=EPS, want_rstd=False)
    assert torch.equal(y[:singles], one), "the prompts' call wrote the rows of the single tokens"
    assert all((p[:singles] == 7).all() for p in pieces)

    # the prompts, against their 64-bit forms
    cu = i32(*offsets)
    c = ref.conv(xbc, m.w, m.bias, cu=cu, state=win0, slots=to, fresh=fresh)
    k = c["covered"]
    assert int(k.sum()) == sum(lens)
    got = torch.cat(pieces, 1).cpu()[k]
    ref.assert_within(got, c["y"][k], c["mag"][k], dtype, "convolution", 16)
    used = [2, 0, 3]
    assert torch.equal(win[used].cpu().double(), c["state"][used])
    r = ref.ssd(x, dt, m.A, B, C, D=m.D, dt_bias=m.dt_bias, cu=cu, state=state0, slots=to, fresh=fresh)
    extra = ref.half_step(dtype) * r["mag"][k]
    if dtype == torch.float16:  # its smallest half step, of the operands M and state copy
        extra = extra + 2.0 ** -25 * (ref.f64(x).abs().amax() * 128 + ref.f64(C).abs().sum(2).amax())
    ref.assert_within(y.cpu()[k], r["y"][k], r["mag"][k], dtype, "scan", 1024, extra=extra)
    ref.assert_within(state[used], r["state"][used], r["mag_state"][used], torch.float32, "state", 1024)

    # the single tokens, against the step of one more token
    w = torch.arange(singles + 1, dtype=torch.int32)
    c1 = ref.conv(xbc[:singles], m.w, m.bias, cu=w, state=win0, slots=at)
    cut = lambda v: (v[:, :m.d].reshape(-1, nh, 64), v[:, m.d:m.d + m.gn].reshape(-1, ng, N),
                     v[:, m.d + m.gn:].reshape(-1, ng, N))
    s1, q1 = (ref.ssd(a, dt[:singles], m.A, b, e, D=m.D, dt_bias=m.dt_bias, cu=w, state=s, slots=at)
              for (a, b, e), s in ((cut(c1["y"]), state0), (cut(c1["mag"]), state0.abs())))
    ref.assert_within(one, s1["y"], q1["mag"], dtype, "step", 128)
    used = list(range(4, 4 + singles))
    assert torch.equal(win[used].cpu().double(), c1["state"][used])
    ref.assert_within(state[used], s1["state"][used], q1["mag_state"][used], torch.float32, "state after the step", 128)
    assert torch.equal(win[1], win0[1]) and torch.equal(state[1], state0[1])
    n = ref.norm(y.flatten(1), z, m.norm_w, group, EPS)
    ref.assert_within(out, n["y"], n["y"].abs(), dtype, "norm", 64)
