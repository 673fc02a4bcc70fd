"""Plain 64-bit forms of the time-major (Mamba-2) operators, sequence by
sequence on the CPU, each with the sums of absolute values that its rounding
bounds are counted in.  Test infrastructure only."""
import torch

F = torch.float64


def f64(t):
    return None if t is None else t.detach().cpu().to(F)


def half_step(dtype):
    """A rounding to `dtype` is off by at most this much of the value."""
    return torch.finfo(dtype).eps / 2


def spans(lead, cu):
    """(first, last + 1) token of every sequence of a token axis."""
    if cu is not None:
        c = cu.tolist()
        return list(zip(c[:-1], c[1:]))
    if len(lead) == 2:
        return [(i * lead[1], (i + 1) * lead[1]) for i in range(lead[0])]
    return [(0, lead[0])]


def assert_within(got, ref, mag, dtype, what, ops32, roundings=1.0, extra=0.0):
    """|got - ref| <= half a step of the output type on ref (times `roundings`, for results that were
    rounded on the way too) + ops32 fp32 roundings of the magnitude + extra."""
    got, ref, mag = f64(got), f64(ref), f64(mag)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    tol = ops32 * 2.0 ** -24 * mag + extra + 1e-37
    if dtype != torch.float32:
        tol = tol + roundings * half_step(dtype) * (ref.abs() + tol)
        if dtype == torch.float16:
            tol = tol + 2.0 ** -25  # half a step of the subnormals
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: "
                             f"{got[i].item()!r} for {ref[i].item()!r}, allowed {tol[i].item():.3e}")


def conv(x, w, bias, cu=None, state=None, slots=None, fresh=None, silu=True, dy=None):
    """Forward (and with dy, the gradient) of the packed convolution.  x (tokens, dim) or (batch, L, dim)."""
    lead = tuple(x.shape[:-1])
    x, w, bias = f64(x).reshape(-1, x.shape[-1]), f64(w), f64(bias)
    bias = torch.zeros(w.shape[0], dtype=F) if bias is None else bias
    W, state = w.shape[1], f64(state)
    out = dict(y=torch.full_like(x, float("nan")), mag=torch.zeros_like(x), covered=torch.zeros(x.shape[0], dtype=bool),
               state=None if state is None else state.clone())
    if dy is not None:
        dy = f64(dy).reshape(x.shape)
        out.update(dx=torch.zeros_like(x), mag_dx=torch.zeros_like(x), dw=torch.zeros_like(w), mag_dw=torch.zeros_like(w),
                   db=torch.zeros_like(bias), mag_db=torch.zeros_like(bias))
    for i, (a, b) in enumerate(spans(lead, cu)):
        slot = i if slots is None else int(slots[i])
        if slot < 0:
            continue
        before = torch.zeros(W - 1, x.shape[1], dtype=F)
        if state is not None and not (fresh is not None and bool(fresh[i])):
            before = state[slot].t()
        line = torch.cat([before, x[a:b]])
        n = b - a
        pre = bias + sum(line[k:k + n] * w[:, k] for k in range(W))
        mag = bias.abs() + sum((line[k:k + n] * w[:, k]).abs() for k in range(W))
        sig = torch.sigmoid(pre)
        out["y"][a:b] = pre * sig if silu else pre
        out["mag"][a:b] = mag
        out["covered"][a:b] = True
        if state is not None:
            out["state"][slot] = line[line.shape[0] - (W - 1):].t()
        if dy is not None:
            dpre = dy[a:b] * (sig * (1 + pre * (1 - sig)) if silu else torch.ones_like(pre))
            # silu' has slope at most 1/2 and value at most 1.1
            err = dy[a:b].abs() * (1.1 + 0.5 * mag)
            dl, ml = torch.zeros_like(line), torch.zeros_like(line)
            for k in range(W):
                dl[k:k + n] += dpre * w[:, k]
                ml[k:k + n] += err * w[:, k].abs()
                out["dw"][:, k] += (dpre * line[k:k + n]).sum(0)
                out["mag_dw"][:, k] += (err * line[k:k + n].abs()).sum(0)
            out["dx"][a:b], out["mag_dx"][a:b] = dl[W - 1:], ml[W - 1:]
            out["db"] += dpre.sum(0)
            out["mag_db"] += err.sum(0)
    return out


def ssd(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, cu=None, state=None, slots=None, fresh=None):
    """The recurrence, token by token; magnitudes from the same recurrence on absolute values."""
    lead = tuple(x.shape[:-2])
    nh, P = x.shape[-2:]
    ng, N = B.shape[-2:]
    x = f64(x).reshape(-1, nh, P)
    dt = f64(dt).reshape(-1, nh)
    B = f64(B).reshape(-1, ng, N).repeat_interleave(nh // ng, dim=1)
    C = f64(C).reshape(-1, ng, N).repeat_interleave(nh // ng, dim=1)
    z = None if z is None else f64(z).reshape(-1, nh, P)
    A, D, dt_bias, state = f64(A), f64(D), f64(dt_bias), f64(state)
    delta = dt + (0 if dt_bias is None else dt_bias)
    if softplus:
        delta = torch.nn.functional.softplus(delta, threshold=200)
    y, mag = torch.full_like(x, float("nan")), torch.zeros_like(x)
    covered = torch.zeros(x.shape[0], dtype=bool)
    out_state, mag_state = (None, None) if state is None else (state.clone(), torch.zeros_like(state))
    for i, (a, b) in enumerate(spans(lead, cu)):
        slot = i if slots is None else int(slots[i])
        if slot < 0:
            continue
        H = torch.zeros(nh, P, N, dtype=F)
        if state is not None and not (fresh is not None and bool(fresh[i])):
            H = state[slot].clone()
        Ha = H.abs()
        for t in range(a, b):
            dec = torch.exp(delta[t] * A)[:, None, None]
            add = (delta[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            H, Ha = dec * H + add, dec * Ha + add.abs()
            y[t] = (H * C[t][:, None, :]).sum(2)
            mag[t] = (Ha * C[t][:, None, :].abs()).sum(2)
            if D is not None:
                y[t] += D[:, None] * x[t]
                mag[t] += (D[:, None] * x[t]).abs()
        if z is not None:
            gate = z[a:b] * torch.sigmoid(z[a:b])
            y[a:b] *= gate
            mag[a:b] *= gate.abs()
        covered[a:b] = True
        if state is not None:
            out_state[slot], mag_state[slot] = H, Ha
    return dict(y=y, mag=mag, covered=covered, state=out_state, mag_state=mag_state)


def norm(x, z, w, group, eps, gate_last=False, dy=None):
    d = x.shape[-1]
    x, w = f64(x).reshape(-1, d), f64(w)
    z = None if z is None else f64(z).reshape(-1, d)
    sig = None if z is None else torch.sigmoid(z)
    gate = torch.ones_like(x) if z is None else z * sig
    dgate = None if z is None else sig * (1 + z * (1 - sig))
    v = x if gate_last else x * gate
    g = lambda t: t.reshape(t.shape[0], d // group, group)
    rstd = 1 / torch.sqrt((g(v) ** 2).mean(2, keepdim=True) + eps)
    n = (g(v) * rstd).reshape(x.shape)
    out = dict(y=n * w * (gate if gate_last else 1), rstd=rstd[:, :, 0])
    if dy is not None:
        dy = f64(dy).reshape(-1, d)
        q = dy * gate if gate_last else dy
        dn = q * w
        c = (g(dn) * g(n)).mean(2, keepdim=True)
        ca = (g(dn) * g(n)).abs().mean(2, keepdim=True)
        dv = ((g(dn) - g(n) * c) * rstd).reshape(x.shape)
        mv = ((g(dn).abs() + g(n).abs() * ca) * rstd).reshape(x.shape)
        out.update(dw=(q * n).sum(0), mag_dw=(q * n).abs().sum(0), dx=dv if gate_last else dv * gate,
                   mag_dx=mv if gate_last else mv * gate.abs())
        if z is not None:
            out["dz"] = dy * n * w * dgate if gate_last else dv * x * dgate
            # sigmoid' terms: values up to 1.1, formed from sums up to 1 + |z|
            spread = sig * (1 + z.abs())
            out["mag_dz"] = (dy * n * w).abs() * spread if gate_last else mv * x.abs() * spread
    return out
