"""Refusals of the time-major (Mamba-2) entry points: bad arguments come back as a
status, with the reason in ss_last_error, before anything touches a GPU; and the
binding refuses tensors that it cannot take.  The pointer values given to the C
calls are never dereferenced."""
import ctypes

import pytest
import torch

from selective_state_space_11_b200 import build as ssbuild
from selective_state_space_11_b200 import ops

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
F32, F16, BF16 = ops._DTYPE[torch.float32], ops._DTYPE[torch.float16], ops._DTYPE[torch.bfloat16]
P = 4096        # a well-aligned address
TOP = (1 << 31) - (1 << 16)

# every call with arguments that pass the checks, in the order of the C declaration
CALLS = {
    "ss_conv1d_tm_fwd": dict(
        tokens=8, nseq=2, dim=24, width=4, dtype=BF16, x=P, ldx=24, w=P, bias=P, cu=P, state=P, nslots=2, slots=P,
        fresh=P, silu=1, dim0=8, dim1=8, dim2=8, y0=P, y1=P, y2=P, stream=None),
    "ss_conv1d_tm_bwd": dict(
        tokens=8, nseq=2, dim=24, width=4, dtype=BF16, x=P, ldx=24, w=P, bias=P, cu=P, silu=1, dim0=8, dim1=8, dim2=8,
        dy0=P, dy1=P, dy2=P, dx=P, lddx=24, dw=P, dbias=P, ws=P, wsb=1 << 20, stream=None),
    "ss_ssd_prefill": dict(
        tokens=8, nseq=2, nheads=4, headdim=64, ngroups=2, dstate=64, dtype=BF16, x=P, ldx=256, dt=P, lddt=4, A=P, B=P,
        ldb=128, C=P, ldc=128, D=P, z=P, ldz=256, dt_bias=P, softplus=1, cu=P, state=P, nslots=2, slots=P, fresh=P,
        y=P, ws=P, wsb=1 << 30, stream=None),
    "ss_ssd_step": dict(
        batch=3, nheads=4, headdim=64, ngroups=2, dstate=64, width=4, dtype=BF16, xbc=P, ldx=512, dt=P, lddt=4, w=P,
        conv_bias=P, silu=1, A=P, D=P, z=P, ldz=256, dt_bias=P, softplus=1, conv_state=P, state=P, nslots=3, slots=P,
        y=P, ws=P, wsb=1 << 20, stream=None),
    "ss_gated_norm_fwd": dict(
        rows=4, dim=32, group=16, dtype=BF16, x=P, ldx=32, z=P, ldz=32, w=P, eps=1e-5, gate_last=0, y=P, rstd=P,
        stream=None),
    "ss_gated_norm_bwd": dict(
        rows=4, dim=32, group=16, dtype=BF16, x=P, ldx=32, z=P, ldz=32, w=P, rstd=P, dy=P, gate_last=0, dx=P, lddx=32,
        dz=P, lddz=32, dw=P, ws=P, wsb=1 << 20, stream=None),
}

BAD = [
    # sizes
    ("ss_conv1d_tm_fwd", dict(tokens=-1), INVALID),
    ("ss_conv1d_tm_fwd", dict(nseq=-1), INVALID),
    ("ss_conv1d_tm_fwd", dict(dim=0), INVALID),
    ("ss_conv1d_tm_fwd", dict(tokens=TOP), UNSUPPORTED),
    ("ss_conv1d_tm_fwd", dict(nseq=65537), UNSUPPORTED),
    ("ss_conv1d_tm_fwd", dict(cu=None, tokens=9), INVALID),            # 9 tokens in 2 equal sequences
    ("ss_conv1d_tm_fwd", dict(width=5), UNSUPPORTED),
    ("ss_conv1d_tm_fwd", dict(width=0), UNSUPPORTED),
    ("ss_conv1d_tm_fwd", dict(dim2=7), INVALID),                       # pieces do not sum to dim
    ("ss_conv1d_tm_fwd", dict(dim0=0, dim1=16), INVALID),
    ("ss_conv1d_tm_fwd", dict(dim1=-8, dim2=24), INVALID),
    ("ss_conv1d_tm_fwd", dict(dim0=8 + (1 << 63) - 16, dim1=8, dim2=8), INVALID),
    ("ss_conv1d_tm_fwd", dict(ldx=23), INVALID),
    ("ss_conv1d_tm_fwd", dict(dtype=9), INVALID),
    # pointers
    ("ss_conv1d_tm_fwd", dict(x=None), INVALID),
    ("ss_conv1d_tm_fwd", dict(w=None), INVALID),
    ("ss_conv1d_tm_fwd", dict(y1=None), INVALID),
    ("ss_conv1d_tm_fwd", dict(state=None), INVALID),
    ("ss_conv1d_tm_fwd", dict(slots=None, nslots=1), INVALID),         # 2 sequences on slots 0 and 1
    ("ss_conv1d_tm_fwd", dict(nslots=-1), INVALID),
    ("ss_conv1d_tm_fwd", dict(x=P + 1), ALIGNMENT),
    ("ss_conv1d_tm_fwd", dict(y2=P + 1), ALIGNMENT),
    ("ss_conv1d_tm_fwd", dict(bias=P + 2), ALIGNMENT),
    ("ss_conv1d_tm_fwd", dict(cu=P + 2), ALIGNMENT),
    ("ss_conv1d_tm_fwd", dict(nslots=0), INVALID),                     # slots without a cache
    ("ss_conv1d_tm_fwd", dict(nslots=0, slots=None, fresh=None), INVALID),
    ("ss_conv1d_tm_fwd", dict(nslots=0, slots=None, state=None), INVALID),
    ("ss_ssd_prefill", dict(state=None), INVALID),
    ("ss_ssd_prefill", dict(state=None, slots=None, nslots=0), INVALID),
    ("ss_ssd_prefill", dict(state=None, slots=None, fresh=None), INVALID),
    ("ss_conv1d_tm_bwd", dict(ldx=8), INVALID),
    ("ss_conv1d_tm_bwd", dict(lddx=8), INVALID),
    ("ss_conv1d_tm_bwd", dict(dy0=None), INVALID),
    ("ss_conv1d_tm_bwd", dict(dw=None), INVALID),
    ("ss_conv1d_tm_bwd", dict(dx=None), INVALID),
    ("ss_conv1d_tm_bwd", dict(dw=P + 2), ALIGNMENT),
    ("ss_conv1d_tm_bwd", dict(ws=P + 8), ALIGNMENT),
    ("ss_conv1d_tm_bwd", dict(wsb=24 * 5 * 4 - 1), WORKSPACE),
    ("ss_conv1d_tm_bwd", dict(ws=None), WORKSPACE),
    ("ss_ssd_prefill", dict(headdim=32), UNSUPPORTED),
    ("ss_ssd_prefill", dict(dstate=32), UNSUPPORTED),
    ("ss_ssd_prefill", dict(dtype=F32), UNSUPPORTED),
    ("ss_ssd_prefill", dict(ngroups=3), INVALID),
    ("ss_ssd_prefill", dict(nheads=0), INVALID),
    ("ss_ssd_prefill", dict(tokens=TOP), UNSUPPORTED),
    ("ss_ssd_prefill", dict(nseq=65537), UNSUPPORTED),
    ("ss_ssd_prefill", dict(cu=None, tokens=9), INVALID),
    ("ss_ssd_prefill", dict(A=None), INVALID),
    ("ss_ssd_prefill", dict(y=None), INVALID),
    ("ss_ssd_prefill", dict(dt=None), INVALID),
    ("ss_ssd_prefill", dict(slots=None, nslots=1), INVALID),
    ("ss_ssd_prefill", dict(ldz=255), INVALID),
    ("ss_ssd_prefill", dict(ldx=260), ALIGNMENT),                      # rows off 16-byte boundaries
    ("ss_ssd_prefill", dict(ldb=132), ALIGNMENT),
    ("ss_ssd_prefill", dict(C=P + 8), ALIGNMENT),
    ("ss_ssd_prefill", dict(y=P + 8), ALIGNMENT),
    ("ss_ssd_prefill", dict(state=P + 16), ALIGNMENT),
    ("ss_ssd_prefill", dict(A=P + 2), ALIGNMENT),
    ("ss_ssd_step", dict(batch=-1), UNSUPPORTED),
    ("ss_ssd_step", dict(batch=65536), UNSUPPORTED),
    ("ss_ssd_step", dict(headdim=128), UNSUPPORTED),
    ("ss_ssd_step", dict(dstate=16), UNSUPPORTED),
    ("ss_ssd_step", dict(width=5), UNSUPPORTED),
    ("ss_ssd_step", dict(ldx=511), INVALID),
    ("ss_ssd_step", dict(conv_state=None), INVALID),
    ("ss_ssd_step", dict(state=None), INVALID),
    ("ss_ssd_step", dict(slots=None, nslots=2), INVALID),
    ("ss_ssd_step", dict(y=None), INVALID),
    ("ss_ssd_step", dict(state=P + 8), ALIGNMENT),
    ("ss_ssd_step", dict(ws=P + 8), ALIGNMENT),
    ("ss_ssd_step", dict(wsb=3 * 512 * 4 - 1), WORKSPACE),
    ("ss_gated_norm_fwd", dict(group=12), INVALID),
    ("ss_gated_norm_fwd", dict(rows=-1), INVALID),
    ("ss_gated_norm_fwd", dict(dim=16384, group=16384, ldx=16384, ldz=16384), UNSUPPORTED),
    ("ss_gated_norm_fwd", dict(dtype=-1), INVALID),
    ("ss_gated_norm_fwd", dict(ldz=31), INVALID),
    ("ss_gated_norm_fwd", dict(w=None), INVALID),
    ("ss_gated_norm_fwd", dict(eps=-1.0), INVALID),
    ("ss_gated_norm_fwd", dict(eps=float("nan")), INVALID),
    ("ss_gated_norm_fwd", dict(y=P + 1), ALIGNMENT),
    ("ss_gated_norm_fwd", dict(rstd=P + 2), ALIGNMENT),
    ("ss_gated_norm_bwd", dict(group=0), INVALID),
    ("ss_gated_norm_bwd", dict(z=None), INVALID),                      # dz without z
    ("ss_gated_norm_bwd", dict(dz=None), INVALID),
    ("ss_gated_norm_bwd", dict(rstd=None), INVALID),
    ("ss_gated_norm_bwd", dict(dw=None), INVALID),
    ("ss_gated_norm_bwd", dict(lddz=31), INVALID),
    ("ss_gated_norm_bwd", dict(dy=P + 1), ALIGNMENT),
    ("ss_gated_norm_bwd", dict(wsb=127), WORKSPACE),
]


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return ops.lib()


def call(lib, name, change):
    args = {**CALLS[name], **change}
    assert len(args) == len(CALLS[name]), "a changed argument has no such name"
    return getattr(lib, name)(*args.values())


@pytest.mark.parametrize("name,change,status", BAD, ids=[f"{n[3:]}-{'-'.join(c)}-{i}" for i, (n, c, _) in enumerate(BAD)])
def test_bad_arguments_are_refused(lib, name, change, status):
    assert call(lib, name, change) == status, lib.ss_last_error()
    assert lib.ss_last_error(), "a refusal names its reason"


def test_the_argument_lists_above_match_the_binding(lib):
    for name, args in CALLS.items():
        assert len(ops.SIGNATURES[name][0]) == len(args), name


@pytest.mark.parametrize("name,change", [
    ("ss_conv1d_tm_fwd", dict(tokens=0, nseq=0)), ("ss_ssd_prefill", dict(tokens=0, nseq=0)),
    ("ss_ssd_step", dict(batch=0)), ("ss_gated_norm_fwd", dict(rows=0))])
def test_empty_calls_do_nothing(lib, name, change):
    """No token, no sequence, no row: fine, with nothing to launch (no GPU is needed to say so)."""
    assert call(lib, name, change) == 0


def test_workspace_sizes(lib):
    none = ctypes.c_size_t(-1).value
    assert lib.ss_conv1d_tm_bwd_workspace_size(0, 24, 4) == 0
    assert lib.ss_conv1d_tm_bwd_workspace_size(1, 24, 4) >= 24 * 5 * 4
    assert lib.ss_conv1d_tm_bwd_workspace_size(-1, 24, 4) == none
    assert lib.ss_conv1d_tm_bwd_workspace_size(8, 24, 5) == none
    assert lib.ss_ssd_step_workspace_size(3, 4, 64, 2, 64) >= 3 * 512 * 4
    assert lib.ss_ssd_step_workspace_size(0, 4, 64, 2, 64) == 0
    assert lib.ss_ssd_step_workspace_size(65536, 4, 64, 2, 64) == none
    assert lib.ss_ssd_step_workspace_size(3, 4, 64, 3, 64) == none
    assert lib.ss_ssd_prefill_workspace_size(8, 2, 4, 64, 2, 96) == none
    assert lib.ss_ssd_prefill_workspace_size(TOP, 2, 4, 64, 2, 64) == none
    assert lib.ss_gated_norm_bwd_workspace_size(4, 32, 16) >= 32 * 4
    assert lib.ss_gated_norm_bwd_workspace_size(4, 32, 12) == none


def test_the_binding_takes_cuda_tensors_only():
    f32, x = torch.float32, torch.zeros(4, 24)
    w = torch.zeros(24, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ops.conv1d_tm_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.conv1d_tm_bwd(x, w, [x])
    with pytest.raises(ValueError, match="CUDA"):
        ops.causal_conv1d_tm_fn(x, w)
    h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.ssd_prefill(h, h[..., 0], torch.zeros(2), h, h)
    with pytest.raises(ValueError, match="CUDA"):
        ops.ssd_step(torch.zeros(1, 64 + 128), torch.zeros(1, 1), torch.zeros(192, 4), torch.zeros(1),
                     torch.zeros(1, 192, 3), torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        ops.gated_norm_fwd(x, x, torch.zeros(24))
    with pytest.raises(ValueError, match="CUDA"):
        ops.gated_norm_fn(x, None, torch.zeros(24))


@pytest.mark.parametrize("call,match", [
    (lambda: ops.conv1d_tm_fwd(torch.zeros(4, 24, dtype=torch.int32), torch.zeros(24, 4)), "dtype"),
    (lambda: ops.conv1d_tm_fwd(torch.zeros(24), torch.zeros(24, 4)), "x is"),
    (lambda: ops.ssd_prefill(torch.zeros(4, 2, 64), torch.zeros(4, 2), torch.zeros(2), torch.zeros(4, 1, 64),
                             torch.zeros(4, 1, 64)), "dtype"),
    (lambda: ops.ssd_step(torch.zeros(1, 192), torch.zeros(1, 1), torch.zeros(192, 4), torch.zeros(1),
                          torch.zeros(1, 192, 3), torch.zeros(1, 64, 64)), "state is"),
    (lambda: ops.gated_norm_fwd(torch.zeros(24), None, torch.zeros(24)), "x is"),
], ids=["dtype", "rank", "prefill-dtype", "step-rank", "norm-rank"])
def test_the_binding_names_what_is_wrong(call, match):
    with pytest.raises(ValueError, match=match):
        call()
