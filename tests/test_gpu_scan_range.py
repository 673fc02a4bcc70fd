"""The range of the prompts' scan in the cached state: growing states, tokens that a later one makes the state forget,
and infinities, in both 16-bit types.

Bounds: 1024 fp32 roundings of the recurrence's magnitude, as for other prompts: Delta A sums of at most 128 terms make
an exponent of at most 14 here, each sum's roundings at most 12 of it, so exp adds under 200 to the 384 products of a
chunk.  In fp16 a product w x of the state's update is held in two pieces: within 2^-22 of itself (4 of those roundings)
or 2^-39 of the largest of its chunk and head, whichever is more."""
import math

import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SHAPES = [("f16", 2, 64), ("f16", 3, 128), ("bf16", 3, 64), ("bf16", 2, 128)]


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


def make(tokens, nh, N, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    q = dict(x=r(tokens, nh, 64), dt=torch.full((tokens, nh), 2.0 ** -5, device=DEV), B=r(tokens, 1, N) * N ** -0.5,
             C=r(tokens, 1, N) * N ** -0.5)
    q = {k: v.to(TYPES[dtype]) for k, v in q.items()}
    return g, q, r(1, nh, 64, N)


def run(q, A, state, dtype, what, finite=None):
    """Scan without softplus against the recurrence; state rows (heads, p) that `finite` leaves out are not compared."""
    r = ref.ssd(**q, A=A, softplus=False, state=state)
    y = ops.ssd_prefill(**q, A=A, dt_softplus=False, state=state)
    delta, B = ref.f64(q["dt"]), ref.f64(q["B"])[:, 0].abs()
    extra = torch.zeros(r["state"].shape, dtype=torch.float64)
    if dtype == "f16":  # 2^-39 of a chunk's largest product, |B| of its tokens, carried to the end
        left = torch.zeros_like(delta)
        left[:-1] = (delta * ref.f64(A)).flip(0).cumsum(0).flip(0)[1:]
        x = torch.nan_to_num(ref.f64(q["x"]), 0.0, 0.0, 0.0).abs().amax(2)
        for a in range(0, delta.shape[0], 128):
            b = min(a + 128, delta.shape[0])
            w = delta[a:b].abs() * torch.exp(left[a:b] - left[b - 1])
            top = (w * x[a:b]).amax(0) * torch.exp(left[b - 1])
            extra += 2.0 ** -39 * top[None, :, None, None] * B[a:b].sum(0)
    keep = torch.ones(r["state"].shape[:3], dtype=torch.bool) if finite is None else finite
    ref.assert_within(state.cpu()[keep], r["state"][keep], r["mag_state"][keep], torch.float32, what, 1024,
                      extra=extra[keep])
    return y, r


@pytest.mark.parametrize("dtype,nh,N", SHAPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("doublings,tokens", [(3, 128), (10, 128), (10, 300), (20, 100)])
def test_growing_state(dtype, nh, N, sign, doublings, tokens):
    """2^doublings in 128 tokens: A above 0, or Delta below 0."""
    g, q, state = make(tokens, nh, N, dtype, 31)
    A = torch.full((nh,), sign * doublings * math.log(2.0) / 128 / 2.0 ** -5, device=DEV)
    q["dt"] *= sign
    y, r = run(q, A, state, dtype, "state")
    k = (r["mag"].amax((1, 2)) < 2.0 ** 12)  # y itself is a 16-bit number of 16-bit operands
    half = ref.half_step(TYPES[dtype])
    sub = 2.0 ** -25 * 2.0 ** doublings * (ref.f64(q["x"]).abs().amax() * 128 + ref.f64(q["C"]).abs().sum(2).amax())
    extra = half * r["mag"][k] + (sub if dtype == "f16" else 0.0)
    ref.assert_within(y.cpu()[k], r["y"][k], r["mag"][k], TYPES[dtype], "y", 1024, extra=extra)


@pytest.mark.parametrize("dtype,nh,N", SHAPES)
@pytest.mark.parametrize("where", [3, 40, 100])
def test_what_a_reset_forgets_does_not_set_the_scale(dtype, nh, N, where):
    """A token of large |x| Delta, one that decays it (and the state before) by e^-100, and small tokens behind."""
    g, q, state = make(128, nh, N, dtype, 41)
    q["x"] *= 2.0 ** -9
    q["dt"][:] = 2.0 ** -10
    q["x"][where], q["dt"][where] = 1000.0, 8.0
    q["x"][where + 1], q["dt"][where + 1] = 0.0, 100.0
    run(q, torch.full((nh,), -1.0, device=DEV), state, dtype, "state")


@pytest.mark.parametrize("dtype,nh,N", SHAPES)
def test_infinity_stays_in_its_row_of_the_state(dtype, nh, N):
    """An infinity beside large values, in a chunk of small ones: it neither spoils nor scales the other rows."""
    g, q, state = make(200, nh, N, dtype, 51)
    q["x"] *= 2.0 ** -6
    q["x"][60] = 1000.0
    q["x"][60, 1, 17] = float("inf")
    keep = torch.ones(1, nh, 64, dtype=torch.bool)
    keep[0, 1, 17] = False
    run(q, torch.full((nh,), -1.0, device=DEV), state, dtype, "state", finite=keep)
    assert not torch.isfinite(state[0, 1, 17]).any()


@pytest.mark.parametrize("dtype,nh,N", SHAPES)
@pytest.mark.parametrize("dexp,xexp", [(-24, -10), (-24, 0), (-10, -14), (12, 0), (14, 6)])
def test_sums_of_every_size(dtype, nh, N, dexp, xexp):
    """A = 0: the state is a plain sum of products of 2^(dexp + xexp).  A token of zeros with the largest Delta there
    is takes no part in it."""
    g, q, state = make(150, nh, N, dtype, 61)
    q["x"] *= 2.0 ** xexp
    q["dt"][:] = 2.0 ** dexp
    q["x"][70], q["dt"][70] = 0.0, 2.0 ** 15
    run(q, torch.zeros(nh, device=DEV), state * 2.0 ** (dexp + xexp), dtype, "state")


@pytest.mark.parametrize("dtype,nh,N", SHAPES)
@pytest.mark.parametrize("big", [10.0, 500.0, 1e4, 6e4])
@pytest.mark.parametrize("where", [(0,), (35,), (62, 63), (64, 100, 127, 128)])
def test_y_behind_a_reset(dtype, nh, N, big, where):
    """Tokens that decay the state by e^-20 to e^-240000 between ordinary ones.  A block of 32 tokens holds at most two,
    which count for at most 160 each in its sums of log2 decays: below 512, where a rounding is off by at most 2^-16.
    An exponent is the difference of two sums of at most 8 such roundings each: 16 x 2^-16 x ln 2 < 2900 x 2^-24 of its
    exponential, beside the 1024 of the recurrence."""
    g, q, state = make(150, nh, N, dtype, 71)
    q["dt"][list(where)] = big
    A = -2.0 * (1.0 + torch.arange(nh, device=DEV))
    r = ref.ssd(**q, A=A, softplus=False, state=state)
    y = ops.ssd_prefill(**q, A=A, dt_softplus=False, state=state)
    extra = ref.half_step(TYPES[dtype]) * r["mag"]
    if dtype == "f16":  # the smallest half step, of M and of the state's copy
        extra = extra + 2.0 ** -25 * (ref.f64(q["x"]).abs().amax() * 128 + ref.f64(q["C"]).abs().sum(2).amax())
    ref.assert_within(y, r["y"], r["mag"], TYPES[dtype], "y", 4 * 1024, extra=extra)
