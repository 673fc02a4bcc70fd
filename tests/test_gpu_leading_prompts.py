"""Prompts on a state cache where the packed rows do not start at the first sequence, and where the offsets are
wrong: rows of no sequence are neither used nor written, and nothing outside the arrays is touched.

Bounds: 1024 fp32 roundings of the recurrence's magnitude (Delta, weights and up to 384 products a chunk), and for y a
half step of the storage type on the magnitude for the 16-bit operands M and state copy.  In fp16 a half step is never
below 2^-25, the subnormals': an element of M is off by that times |x_j|, for the token's chunk up to itself, and one
of the state copy by that times |C_n| (the decays on both are at most 1)."""
import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
BAD = [[0, 10, 5, 30], [0, 10, 20, 99], [-4, 10, 20, 30], [25, 10, 20, 30], [64, 70, 80, 90], [30, 0, 0, 30],
       [17, -9, 30, 2], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]]


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


def offsets(gap, lens):
    return (gap + torch.tensor([0] + lens).cumsum(0)).to(device=DEV, dtype=torch.int32)


def make_scan(tokens, nh, N, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    u = lambda lo, hi: lo + (hi - lo) * torch.rand(nh, device=DEV, generator=g)
    q = dict(x=r(tokens, nh, 64), dt=r(tokens, nh), A=-torch.exp(u(0.0, 2.77)), B=r(tokens, 1, N) * N ** -0.5,
             C=r(tokens, 1, N) * N ** -0.5)
    return g, {k: v if k == "A" else v.to(TYPES[dtype]) for k, v in q.items()}


def subnormals(q, gap, lens):
    """What fp16's smallest half step, 2^-25, of the operands M and state copy adds up to in y."""
    x, C = q["x"].double().abs().cpu(), q["C"].double().abs().sum(2, keepdim=True).cpu()
    total = torch.zeros_like(x)
    a = gap
    for n in lens:
        for c in range(a, a + n, 128):
            total[c:min(c + 128, a + n)] = x[c:min(c + 128, a + n)].cumsum(0)
        a += n
    return 2.0 ** -25 * (total + C)


@pytest.mark.parametrize("gap", [1, 64, 128, 200])
@pytest.mark.parametrize("dtype,nh,N", [("bf16", 3, 128), ("f16", 2, 64)])
def test_prompts(gap, dtype, nh, N):
    lens = [130, 0, 1, 257]
    tokens = gap + sum(lens) + 2
    g, q = make_scan(tokens, nh, N, dtype, 700 + gap)
    cu, state = offsets(gap, lens), torch.randn(5, nh, 64, N, device=DEV, generator=g)
    slots = torch.tensor([4, 0, 2, 1], dtype=torch.int32, device=DEV)
    for k in ("x", "B", "C"):
        q[k][:gap], q[k][-2:] = float("nan"), float("nan")
    r = ref.ssd(**q, cu=cu, state=state, slots=slots)
    out = torch.full((tokens, nh, 64), 7.0, device=DEV, dtype=TYPES[dtype])
    ops.ssd_prefill(**q, cu_seqlens=cu, state=state, slots=slots, out=out)
    k = r["covered"]
    extra = ref.half_step(TYPES[dtype]) * r["mag"][k]
    if dtype == "f16":
        extra = extra + subnormals(q, gap, lens)[k]
    ref.assert_within(out.cpu()[k], r["y"][k], r["mag"][k], TYPES[dtype], "y", 1024, extra=extra)
    assert (out.cpu()[~k] == 7).all(), "rows of no sequence were written"
    ref.assert_within(state, r["state"], r["mag_state"], torch.float32, "state", 1024)




@pytest.mark.parametrize("bad", BAD)
def test_bad_offsets_of_prompts_stay_inside_the_arrays(bad):
    n, guard, nh, N = 30, 130, 2, 64
    g, q = make_scan(n + 2 * guard, nh, N, "bf16", 900)
    for k in ("x", "B", "C", "dt"):
        q[k][:guard], q[k][-guard:] = float("nan"), float("nan")
        q[k] = q[k][guard:guard + n]
    room = torch.full((n + 2 * guard, nh, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    states = torch.full((5, nh, 64, N), 0.5, device=DEV)
    ops.ssd_prefill(**q, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device=DEV), state=states[1:4],
                    out=room[guard:guard + n])
    assert ops.lib().ss_device_fault(1) == 8
    assert torch.isfinite(room).all() and torch.isfinite(states).all()
    assert (room[:guard] == 7).all() and (room[-guard:] == 7).all()
    assert (states[0] == 0.5).all() and (states[4] == 0.5).all()
