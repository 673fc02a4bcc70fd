"""Gated group RMS norm against its plain 64-bit form, forward and backward.

Counted in fp32 roundings: v, the gate (8: exponential, reciprocal, products),
the sum of squares (pairwise over at most 8192 columns: 32 register adds at
most, 5 shuffles, 8 warps, halved by the root), rstd (4), two products: 64 cover
an output.  The backward's second sum over the group is of the same kind and its
magnitude is counted separately: 128 of the magnitudes."""
import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def make(lead, dim, dtype, seed, pad=0, off=0, gate=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[dtype]
    x = torch.randn(*lead, dim + pad, device=DEV, generator=g).to(dt)[..., off:off + dim]
    z = torch.randn(*lead, dim + pad, device=DEV, generator=g).to(dt)[..., off:off + dim] if gate else None
    dy = torch.randn(*lead, dim, device=DEV, generator=g).to(dt)
    w = 1 + 0.2 * torch.randn(dim, device=DEV, generator=g)
    return x, z, w, dy


def check(x, z, w, dy, group, gate_last):
    dim = x.shape[-1]
    y, rstd = ops.gated_norm_fwd(x, z, w, group=group, eps=EPS, gate_last=gate_last)
    b = ops.gated_norm_bwd(x, z, w, dy, rstd, group=group, gate_last=gate_last)
    r = ref.norm(x, z, w, group, EPS, gate_last, dy=dy)
    flat = lambda t: t.reshape(-1, t.shape[-1])
    ref.assert_within(flat(y), r["y"], r["y"].abs(), x.dtype, "y", 64)
    ref.assert_within(flat(rstd), r["rstd"], r["rstd"], torch.float32, "rstd", 64)
    ref.assert_within(flat(b["dx"]), r["dx"], r["mag_dx"], x.dtype, "dx", 128)
    if z is None:
        assert b["dz"] is None
    else:
        ref.assert_within(flat(b["dz"]), r["dz"], r["mag_dz"], x.dtype, "dz", 128)
    # one add per row of a walker, then one per walker
    rows = flat(x).shape[0]
    ref.assert_within(b["dw"], r["dw"], r["mag_dw"], torch.float32, "dw", 64 + rows)


@pytest.mark.parametrize("gate_last", [False, True])
@pytest.mark.parametrize("dtype,dim,group,pad,off,rows", [
    ("bf16", 1536, 1536, 24, 8, 50), ("bf16", 5120, 5120, 0, 0, 7), ("f16", 1024, 256, 8, 0, 33),
    ("f32", 384, 64, 0, 0, 129), ("bf16", 37, 37, 5, 3, 20), ("f16", 30, 10, 0, 0, 65), ("f32", 1, 1, 0, 0, 9),
    ("bf16", 8192, 8192, 0, 0, 3), ("f32", 8191, 8191, 0, 0, 2), ("f16", 1200, 600, 1, 0, 5), ("bf16", 6000, 2000, 0, 0, 1),
    ("bf16", 512, 512, 0, 0, 2000)])
def test_forward_and_backward(dtype, dim, group, pad, off, rows, gate_last):
    check(*make((rows,), dim, dtype, 5 + dim, pad, off), group, gate_last)


def test_without_gate_and_three_axes():
    check(*make((3, 11), 96, "bf16", 1, gate=False), 32, False)
    check(*make((3, 11), 96, "f32", 2, pad=8), 96, False)


def test_zero_and_huge_rows():
    x, z, w, dy = make((4,), 256, "f32", 3)
    x[1] = 0          # rstd = eps^-1/2
    x[2] *= 1e15      # squares reach 1e30, inside fp32
    z[3] = -200.0     # the gate underflows to zero
    check(x, z, w, dy, 128, False)
    y, _ = ops.gated_norm_fwd(x, z, w, eps=EPS)
    assert torch.isfinite(y).all()


def test_a_bad_row_stays_in_its_row():
    x, z, w, dy = make((6,), 512, "bf16", 4)
    want, _ = ops.gated_norm_fwd(x, z, w)
    x[2, 5], z[4, 7] = float("nan"), float("inf")
    y, _ = ops.gated_norm_fwd(x, z, w)
    for i in (0, 1, 3, 5):
        assert torch.equal(y[i], want[i])


def test_empty_and_rstd_left_out():
    x, z, w, dy = make((0,), 64, "bf16", 5)
    y, rstd = ops.gated_norm_fwd(x, z, w)
    b = ops.gated_norm_bwd(x, z, w, dy, rstd)
    assert y.shape == (0, 64) and (b["dw"] == 0).all()
    x, z, w, dy = make((3,), 64, "bf16", 6)
    y, rstd = ops.gated_norm_fwd(x, z, w, want_rstd=False)
    assert rstd is None and torch.equal(y, ops.gated_norm_fwd(x, z, w)[0])


def test_gradients_into_column_slices_and_repeatable():
    x, z, w, dy = make((300,), 128, "bf16", 7, pad=16, off=8)
    y, rstd = ops.gated_norm_fwd(x, z, w, group=64)
    wide = torch.full((300, 320), 3.0, device=DEV, dtype=x.dtype)
    a = ops.gated_norm_bwd(x, z, w, dy, rstd, group=64, dx=wide[:, :128], dz=wide[:, 160:288])
    b = ops.gated_norm_bwd(x, z, w, dy, rstd, group=64)
    assert torch.equal(wide[:, :128], b["dx"]) and torch.equal(wide[:, 160:288], b["dz"]) and torch.equal(a["dw"], b["dw"])
    assert (wide[:, 128:160] == 3).all() and (wide[:, 288:] == 3).all()


@pytest.mark.parametrize("gate_last", [False, True])
def test_autograd_against_differences(gate_last):
    x, z, w, dy = make((5,), 12, "f32", 8)
    for t in (x, z, w):
        t.requires_grad_(True)
    (ops.gated_norm_fn(x, z, w, group=6, gate_last=gate_last) * dy).sum().backward()
    h = 1e-5
    for name, t in (("x", x), ("z", z), ("w", w)):
        for k in range(0, t.numel(), 5):
            v = []
            for s in (h, -h):
                a = {"x": ref.f64(x), "z": ref.f64(z), "w": ref.f64(w)}
                a[name] = a[name].clone()
                a[name].reshape(-1)[k] += s
                v.append(float((ref.norm(a["x"], a["z"], a["w"], 6, EPS, gate_last)["y"] * ref.f64(dy)).sum()))
            # 128 fp32 roundings of terms below 100; central differences of step 1e-5 in 64 bits: below 1e-6
            assert abs(float(t.grad.reshape(-1)[k]) - (v[0] - v[1]) / (2 * h)) <= 128 * 2 ** -24 * 100 + 1e-6, (name, k)
