"""A wait inside the prompts' scan that runs out: reported, drained, and without trace in the next call."""
import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dtype,nh,N,lens", [
    ("bf16", 1, 64, [40]),  # one block: a chunk that is not whole
    ("bf16", 2, 128, [256]),  # whole chunks, stored by TMA
    ("f16", 3, 64, [700]),  # more chunks than buffers, two pairs of heads
    ("f16", 4, 128, [130, 5, 300])])  # sequences of several blocks
def test_wait_that_runs_out_is_reported_and_the_context_recovers(dtype, nh, N, lens, monkeypatch):
    """SS_INJECT_WAIT_TIMEOUT makes the warp that issues the products of y give up in each block's first chunk, with
    copies and products in flight.  The other roles' waits run out one after the other, a second each at most; the block drains, frees its
    TMEM and ends: bit 1 of the fault word alone, guard rows around the outputs as they were, the next call right."""
    tokens, guard = sum(lens), 130
    g = torch.Generator(device=DEV).manual_seed(81)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    q = dict(x=r(tokens, nh, 64), dt=r(tokens, nh), B=r(tokens, 1, N) * N ** -0.5, C=r(tokens, 1, N) * N ** -0.5)
    q = {k: v.to(TYPES[dtype]) for k, v in q.items()}
    q["A"] = -torch.arange(1.0, nh + 1, device=DEV)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    first = r(len(lens), nh, 64, N)
    states = torch.full((len(lens) + 2, nh, 64, N), 7.0, device=DEV)
    rows = torch.full((tokens + 2 * guard, nh, 64), 7.0, device=DEV, dtype=TYPES[dtype])
    state, out = states[1:-1], rows[guard:-guard]
    ops.lib().ss_device_fault(1)
    for inject in (True, False):
        state.copy_(first)
        if inject:
            monkeypatch.setenv("SS_INJECT_WAIT_TIMEOUT", "1")
        ops.ssd_prefill(**q, cu_seqlens=cu, state=state, out=out)
        monkeypatch.delenv("SS_INJECT_WAIT_TIMEOUT", raising=False)
        assert ops.lib().ss_device_fault(1) == (2 if inject else 0)  # -1 would mean a CUDA error
        assert (rows[:guard] == 7).all() and (rows[-guard:] == 7).all()
        assert (states[0] == 7).all() and (states[-1] == 7).all()
    want = ref.ssd(**q, cu=cu, state=first)
    extra = ref.half_step(TYPES[dtype]) * want["mag"]
    if dtype == "f16":  # the smallest half step, of M and of the state's copy
        extra = extra + 2.0 ** -25 * (ref.f64(q["x"]).abs().amax() * 128 + ref.f64(q["C"]).abs().sum(2).amax())
    ref.assert_within(out, want["y"], want["mag"], TYPES[dtype], "y", 1024, extra=extra)
    ref.assert_within(state, want["state"], want["mag_state"], torch.float32, "state", 1024)
