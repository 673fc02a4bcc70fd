"""Cases of the Mamba-2 mixer's operators between its two projections: the time-major causal convolution
(`conv1d_tm_fwd`, `conv1d_tm_bwd`), the scan of ragged prompts on a state cache (`ssd_prefill`), the step of
one token per request (`ssd_step`) and the gated group norm (`gated_norm_fwd`, `gated_norm_bwd`).

Every case stands for one call of a model's layer.  The input projection writes one row per token, columns
[z | x B C | dt]; the operators read column slices of it, so their rows are as wide as the projection.
"""
import math
import random

import torch

own = False

HEADDIM = 64
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases -----
def listed():
    return [
        # the convolution of a serving batch: prompts of every length beside continued ones, windows in a cache
        dict(name="conv ragged prompts", op="conv", mode="serve", dtype="bf16", seqs=24, tokens=8192, spread=4.0,
             heads=80, groups=1, dstate=128, width=4),
        # one layer of a training step at the 2.7b shape, forward and backward
        dict(name="conv train layer", op="conv", mode="train", dtype="bf16", seqs=4, tokens=16384, spread=0.0,
             heads=80, groups=1, dstate=128, width=4),
        # a small fp32 model on packed documents, three taps, lengths that divide nothing
        dict(name="conv train small", op="conv", mode="train", dtype="f32", seqs=7, tokens=667, spread=2.0,
             heads=5, groups=1, dstate=64, width=3),
        # the first prompt of a quiet server: one short sequence of a 130m layer
        dict(name="prefill one short", op="prefill", dtype="bf16", seqs=1, tokens=37, spread=0.0, heads=24,
             groups=1, dstate=128),
        # a serving batch at the 2.7b shape: fresh prompts of every length beside continued ones
        dict(name="prefill ragged", op="prefill", dtype="bf16", seqs=24, tokens=8192, spread=4.0, heads=80,
             groups=1, dstate=128),
        # four long prompts at the 2.7b shape
        dict(name="prefill batch", op="prefill", dtype="bf16", seqs=4, tokens=16384, spread=0.0, heads=80,
             groups=1, dstate=128),
        # one long document of a 130m layer: few heads, so the work has to be split along the sequence
        dict(name="prefill long", op="prefill", dtype="f16", seqs=1, tokens=32768, spread=0.0, heads=24,
             groups=2, dstate=64),
        # decoding one request: latency
        dict(name="step single", op="step", dtype="bf16", seqs=1, heads=24, groups=1, dstate=128, width=4),
        # decoding a batch at the 2.7b shape: the state's bytes
        dict(name="step batch", op="step", dtype="bf16", seqs=64, heads=80, groups=1, dstate=128, width=4),
        # an odd large batch of a small fp16 model with grouped B and C
        dict(name="step odd batch", op="step", dtype="f16", seqs=243, heads=24, groups=2, dstate=64, width=4),
        # the norm of the training layer above, forward and backward
        dict(name="norm train layer", op="norm", mode="train", dtype="bf16", tokens=16384, heads=80, groups=1),
        # the norm of a decode batch, two groups
        dict(name="norm decode", op="norm", mode="serve", dtype="f16", tokens=64, heads=24, groups=2),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["conv", "prefill", "step", "norm"])
    groups = rng.choice([1, 1, 2, 4])
    heads = groups * max(1, log_int(2, 80) // groups)
    case = dict(op=op, dtype=rng.choice(["bf16", "f16"]), heads=heads, groups=groups)
    most = 16384 * 80 // heads  # tokens x heads of the largest listed layer
    if op == "norm":
        case.update(mode=rng.choice(["train", "serve"]), tokens=log_int(1, min(most, 65536)))
        if rng.random() < 0.3:
            case["dtype"] = "f32"
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    case["dstate"] = rng.choice([64, 128])
    if op == "step":
        case.update(seqs=log_int(1, max(1, min(1024, 64 * 80 // heads))), width=rng.choice([2, 3, 4, 4]))
        return case
    case["tokens"] = log_int(1, min(most // 2 if op == "conv" else most, 32768))
    case["seqs"] = min(log_int(1, 48), case["tokens"])
    case["spread"] = rng.choice([0.0, 2.0, 4.0])
    if op == "prefill":  # the plain form pads every sequence to the longest: keep that within the largest case
        if case["seqs"] * max(lengths(case)) * heads > 4 * 16384 * 80:
            case["spread"] = 0.0
    else:
        case.update(mode=rng.choice(["serve", "train"]), width=rng.choice([2, 3, 4, 4]))
        if rng.random() < 0.3:
            case["dtype"] = "f32"
            case["tokens"] = max(case["seqs"], case["tokens"] // 2)
    return case


def lengths(case):
    """The sequences' lengths: equal ones, or spread over a factor of e^spread."""
    n, total = case["seqs"], case["tokens"]
    if not case["spread"]:
        return [total // n + (1 if i < total % n else 0) for i in range(n)]
    rng = random.Random(1000003 * n + total)
    share = [math.exp(rng.uniform(0.0, case["spread"])) for _ in range(n)]
    got = [int(total * s / sum(share)) for s in share]
    got[share.index(max(share))] += total - sum(got)
    return got


def widths(case):
    """(columns of z and of x, of B and of C, of x|B|C, of the whole projection row)."""
    d = case["heads"] * HEADDIM
    bc = case["groups"] * case.get("dstate", 0)
    return d, bc, d + 2 * bc, 2 * d + 2 * bc + case["heads"]


# ------------------------------------------------------------------ inputs -----
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = dict(device="cuda", generator=gen)
    dtype = TYPES[case["dtype"]]
    d, bc, conv, row = widths(case)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, **dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, **dev)

    def caches(seqs):
        """Slots of a cache with room for more requests, in no order; some requests start afresh."""
        room = seqs + max(1, seqs // 4)
        s["slots"] = torch.randperm(room, **dev)[:seqs].to(torch.int32)
        s["fresh"] = torch.rand(seqs, **dev) < 0.5
        return room

    if case["op"] in ("conv", "prefill"):
        lens = lengths(case)
        s["longest"] = max(lens)
        s["cu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    if case["op"] in ("conv", "step"):
        s["w"] = normal(conv, case["width"]) / case["width"] ** 0.5
        s["bias"] = normal(conv) * 0.1
    if case["op"] in ("prefill", "step"):
        heads = case["heads"]
        s["A"] = -torch.exp(uniform(0.0, math.log(16.0), heads))
        s["D"] = uniform(0.0, 1.0, heads)
        s["dt_bias"] = torch.log(torch.expm1(uniform(1e-3, 0.1, heads)))

    if case["op"] == "conv":
        zx = normal(case["tokens"], row).to(dtype)
        s["x"] = zx[:, d:d + conv]
        s["splits"] = (d, bc, bc)
        if case["mode"] == "serve":
            s["window"] = normal(caches(case["seqs"]), conv, case["width"] - 1).to(dtype).float()
        else:
            s["dy"] = tuple(normal(case["tokens"], c).to(dtype) for c in s["splits"])
    elif case["op"] == "prefill":
        t, heads = case["tokens"], case["heads"]
        zx = normal(t, row).to(dtype)
        s["dt"] = zx[:, row - heads:]

        def convolved(*shape):  # what the convolution and its SiLU leave
            v = normal(*shape)
            return (v * torch.sigmoid(v)).to(dtype)

        s["x"] = convolved(t, heads, HEADDIM)
        s["B"] = convolved(t, case["groups"], case["dstate"])
        s["C"] = convolved(t, case["groups"], case["dstate"])
        s["state"] = normal(caches(case["seqs"]), heads, HEADDIM, case["dstate"]) * 0.3
    elif case["op"] == "step":
        n, heads = case["seqs"], case["heads"]
        zx = normal(n, row).to(dtype)
        s["xbc"], s["dt"] = zx[:, d:d + conv], zx[:, row - heads:]
        room = caches(n)
        s["window"] = normal(room, conv, case["width"] - 1).to(dtype).float()
        s["state"] = normal(room, heads, HEADDIM, case["dstate"]) * 0.3
    else:
        t = case["tokens"]
        zx = normal(t, 2 * d + case["heads"]).to(dtype)
        s["z"] = zx[:, :d]
        s["x"] = normal(t, d).to(dtype)
        s["w"] = 1.0 + 0.1 * normal(d)
        s["group"] = d // case["groups"]
        if case["mode"] == "train":
            s["dy"] = normal(t, d).to(dtype)
    return s


# ------------------------------------------------------------------ one pass -----
def run(s):
    return {"conv": run_conv, "prefill": run_prefill, "step": run_step, "norm": run_norm}[s["case"]["op"]](s)


def run_conv(s):
    if s["case"]["mode"] == "serve":
        if own:
            from selective_state_space_11_b200 import ops
            x, B, C = ops.conv1d_tm_fwd(s["x"], s["w"], s["bias"], splits=s["splits"], cu_seqlens=s["cu"],
                                        state=s["window"], slots=s["slots"], fresh=s["fresh"])
        else:
            x, B, C = plain_conv(s, s["window"])
        return {"x": x, "B": B, "C": C, "window": s["window"]}
    if own:
        from selective_state_space_11_b200 import ops
        x, B, C = ops.conv1d_tm_fwd(s["x"], s["w"], s["bias"], splits=s["splits"], cu_seqlens=s["cu"])
        g = ops.conv1d_tm_bwd(s["x"], s["w"], s["dy"], s["bias"], cu_seqlens=s["cu"])
        return {"x": x, "B": B, "C": C, "dx": g["dx"], "dw": g["dw"], "dbias": g["dbias"]}
    x, B, C = plain_conv(s, None)
    dx, dw, dbias = plain_conv_bwd(s)
    return {"x": x, "B": B, "C": C, "dx": dx, "dw": dw, "dbias": dbias}


def run_prefill(s):
    if own:
        from selective_state_space_11_b200 import ops
        y = ops.ssd_prefill(s["x"], s["dt"], s["A"], s["B"], s["C"], state=s["state"], D=s["D"],
                            dt_bias=s["dt_bias"], cu_seqlens=s["cu"], slots=s["slots"], fresh=s["fresh"])
    else:
        y = plain_prefill(s)
    return {"y": y, "state": s["state"]}


def run_step(s):
    if own:
        from selective_state_space_11_b200 import ops
        y = ops.ssd_step(s["xbc"], s["dt"], s["w"], s["A"], s["window"], s["state"], conv_bias=s["bias"], D=s["D"],
                         dt_bias=s["dt_bias"], slots=s["slots"], ngroups=s["case"]["groups"])
    else:
        y = plain_step(s)
    return {"y": y, "window": s["window"], "state": s["state"]}


def run_norm(s):
    if own:
        from selective_state_space_11_b200 import ops
        y, rstd = ops.gated_norm_fwd(s["x"], s["z"], s["w"], group=s["group"], eps=EPS)
        if "dy" not in s:
            return y
        g = ops.gated_norm_bwd(s["x"], s["z"], s["w"], s["dy"], rstd, group=s["group"])
        return {"y": y, "dx": g["dx"], "dz": g["dz"], "dw": g["dw"]}
    return plain_norm(s)


# ------------------------------------------------------------------ plain forms, fp32 -----
def silu(v):
    return v / (1.0 + torch.exp(-v))


def softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def places(cu, tokens):
    """The sequence and the position in it of every token."""
    t = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(cu.long(), t, right=True) - 1
    return t, seq, t - cu.long()[seq]


def history(s, window):
    """The windows that the sequences enter with, (sequences, channels, taps - 1)."""
    h = window[s["slots"].long()]
    return torch.where(s["fresh"][:, None, None], torch.zeros_like(h), h)


def taps_of(s, window):
    """The inputs under the taps of every token, (tokens, taps, channels)."""
    x, width = s["x"].float(), s["w"].shape[1]
    t, seq, pos = places(s["cu"], x.shape[0])
    back = torch.arange(width, device="cuda") - (width - 1)
    inside = (pos[:, None] + back >= 0)[:, :, None]
    under = x[(t[:, None] + back).clamp(min=0)]
    if window is None:
        return torch.where(inside, under, torch.zeros_like(under))
    old = history(s, window)
    at = (width - 1 + pos[:, None] + back).clamp(0, width - 2)
    return torch.where(inside, under, old.transpose(1, 2)[seq[:, None], at])


def plain_conv(s, window):
    v = silu((taps_of(s, window) * s["w"].t()).sum(1) + s["bias"])
    if window is not None:
        width, cu = s["w"].shape[1], s["cu"].long()
        last = (cu[1:] - cu[:-1])[:, None] - (width - 1) + torch.arange(width - 1, device="cuda")  # positions
        old = history(s, window).transpose(1, 2)
        new = s["x"].float()[(cu[:-1, None] + last).clamp(0, s["x"].shape[0] - 1)]
        keep = old.gather(1, (width - 1 + last).clamp(0, width - 2)[:, :, None].expand_as(old))
        window[s["slots"].long()] = torch.where((last >= 0)[:, :, None], new, keep).transpose(1, 2)
    return tuple(p.contiguous() for p in v.to(s["x"].dtype).split(s["splits"], dim=1))


def plain_conv_bwd(s):
    x, width, tokens = s["x"].float(), s["w"].shape[1], s["x"].shape[0]
    under = taps_of(s, None)
    pre = (under * s["w"].t()).sum(1) + s["bias"]
    sig = 1.0 / (1.0 + torch.exp(-pre))
    dpre = torch.cat([d.float() for d in s["dy"]], dim=1) * sig * (1.0 + pre * (1.0 - sig))
    t, seq, _ = places(s["cu"], tokens)
    ahead = (width - 1) - torch.arange(width, device="cuda")
    to = t[:, None] + ahead
    inside = (to < s["cu"].long()[seq + 1][:, None])[:, :, None]
    later = dpre[to.clamp(max=tokens - 1)]
    dx = (torch.where(inside, later, torch.zeros_like(later)) * s["w"].t()).sum(1)
    dw = (under * dpre[:, None]).sum(0).t().contiguous()
    return dx.to(s["x"].dtype), dw, dpre.sum(0)


def plain_prefill(s):
    case, chunk = s["case"], 64
    n, heads, groups, dstate = case["seqs"], case["heads"], case["groups"], case["dstate"]
    per, nc = heads // groups, -(-s["longest"] // chunk)
    cu = s["cu"].long()
    j = torch.arange(nc * chunk, device="cuda")
    valid = j < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(valid, cu[:-1, None] + j, torch.zeros_like(j))

    def chunks(v, *last):  # (tokens, ...) -> (sequences, chunks, steps, ...), zero behind each sequence
        v = v.float()[at] * valid.reshape(n, nc * chunk, *([1] * (v.dim() - 1)))
        return v.reshape(n, nc, chunk, *last)

    x = chunks(s["x"], groups, per, HEADDIM)
    B, C = chunks(s["B"], groups, dstate), chunks(s["C"], groups, dstate)
    dt = softplus(s["dt"].double() + s["dt_bias"].double())[at] * valid[:, :, None]
    dt = dt.reshape(n, nc, chunk, groups, per)
    cs = (dt * s["A"].double().reshape(groups, per)).cumsum(2)  # log decays since the chunk's start
    dt32 = dt.float()
    # inside a chunk: the masked, decayed products
    i = torch.arange(chunk, device="cuda")
    cst = cs.permute(0, 1, 3, 4, 2)
    decay = torch.where(i[:, None] >= i, cst[..., :, None] - cst[..., None, :], -torch.inf).exp().float()
    M = torch.einsum("bcigm,bcjgm->bcgij", C, B)[:, :, :, None] * decay
    M = M * dt32.permute(0, 1, 3, 4, 2)[..., None, :]
    y = torch.einsum("bcgrij,bcjgrp->bcigrp", M, x)
    # each chunk's own state, and the states entering the chunks and leaving the sequence
    left = (cs[:, :, -1:] - cs).exp().float() * dt32
    S = torch.einsum("bcjgrp,bcjgm->bcgrpm", x * left[..., None], B)
    old = s["state"][s["slots"].long()]
    old = torch.where(s["fresh"][:, None, None, None], torch.zeros_like(old), old)
    S = torch.cat([old.reshape(n, 1, groups, per, HEADDIM, dstate), S], dim=1)
    upto = torch.cat([torch.zeros_like(cs[:, :1, -1]), cs[:, :, -1].cumsum(1)], dim=1)  # (n, nc + 1, g, r)
    ends = upto.permute(0, 2, 3, 1)
    k = torch.arange(nc + 1, device="cuda")
    pass_on = torch.where(k[:, None] >= k, ends[..., :, None] - ends[..., None, :], -torch.inf).exp().float()
    H = torch.matmul(pass_on, S.permute(0, 2, 3, 1, 4, 5).reshape(n, groups, per, nc + 1, HEADDIM * dstate))
    s["state"][s["slots"].long()] = H[:, :, :, nc].reshape(n, heads, HEADDIM, dstate)
    H = H[:, :, :, :nc].reshape(n, groups, per, nc, HEADDIM, dstate)
    y = y + torch.einsum("bcigm,bgrcpm->bcigrp", C, H) * cs.exp().float()[..., None]
    y = y + x * s["D"].reshape(groups, per, 1)
    return y.reshape(n, nc * chunk, heads, HEADDIM)[valid].to(s["x"].dtype)


def plain_step(s):
    case, slots = s["case"], s["slots"].long()
    n, heads, groups, dstate = case["seqs"], case["heads"], case["groups"], case["dstate"]
    d, bc, _, _ = widths(case)
    full = torch.cat([s["window"][slots], s["xbc"].float()[:, :, None]], dim=2)
    v = silu((full * s["w"]).sum(2) + s["bias"])
    s["window"][slots] = full[:, :, 1:]
    x = v[:, :d].reshape(n, heads, HEADDIM)
    B = v[:, d:d + bc].reshape(n, groups, 1, dstate).expand(-1, -1, heads // groups, -1).reshape(n, heads, dstate)
    C = v[:, d + bc:].reshape(n, groups, 1, dstate).expand(-1, -1, heads // groups, -1).reshape(n, heads, dstate)
    dt = softplus(s["dt"].float() + s["dt_bias"])
    H = s["state"][slots] * torch.exp(dt * s["A"])[:, :, None, None]
    H = H + (dt[:, :, None] * x)[..., None] * B[:, :, None]
    s["state"][slots] = H
    y = (H * C[:, :, None]).sum(3) + s["D"][:, None] * x
    return y.to(s["xbc"].dtype)


def plain_norm(s):
    t, d = s["x"].shape
    x, z, w = s["x"].float(), s["z"].float(), s["w"]
    sig = 1.0 / (1.0 + torch.exp(-z))
    v = (x * (z * sig)).reshape(t, d // s["group"], s["group"])
    rstd = 1.0 / torch.sqrt((v * v).mean(2, keepdim=True) + EPS)
    n = v * rstd
    y = (n.reshape(t, d) * w).to(s["x"].dtype)
    if "dy" not in s:
        return y
    dy = s["dy"].float()
    dn = (dy * w).reshape(n.shape)
    dv = ((dn - n * (dn * n).mean(2, keepdim=True)) * rstd).reshape(t, d)
    dx = dv * (z * sig)
    dz = dv * x * sig * (1.0 + z * (1.0 - sig))
    return {"y": y, "dx": dx.to(y.dtype), "dz": dz.to(y.dtype), "dw": (dy * n.reshape(t, d)).sum(0)}


# ------------------------------------------------------------------ definitions, fp64 -----
def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": exact_conv, "prefill": exact_prefill, "step": exact_step, "norm": exact_norm}[case["op"]](s)


def exact_conv(s):
    """Sequence by sequence, tap by tap."""
    serve, cu = s["case"]["mode"] == "serve", s["cu"].tolist()
    x, w, bias = s["x"].double(), s["w"].double(), s["bias"].double()
    width = w.shape[1]
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(bias)
    dy = None if serve else torch.cat(s["dy"], dim=1).double()
    window = s["window"].double() if serve else None
    for i in range(len(cu) - 1):
        a, b = cu[i], cu[i + 1]
        before = x.new_zeros(width - 1, x.shape[1])
        if serve and not bool(s["fresh"][i]):
            before = window[s["slots"][i].long()].t()
        line = torch.cat([before, x[a:b]])
        pre = bias + sum(line[k:k + b - a] * w[:, k] for k in range(width))
        sig = torch.sigmoid(pre)
        y[a:b] = pre * sig
        if serve:
            window[s["slots"][i].long()] = line[line.shape[0] - (width - 1):].t()
            continue
        dpre = dy[a:b] * (sig + pre * sig * (1 - sig))
        dline = torch.zeros_like(line)
        for k in range(width):
            dline[k:k + b - a] += dpre * w[:, k]
            dw[:, k] += (dpre * line[k:k + b - a]).sum(0)
        db += dpre.sum(0)
        dx[a:b] = dline[width - 1:]
    parts = dict(zip("xBC", y.split(s["splits"], dim=1)))
    return {**parts, "window": window} if serve else {**parts, "dx": dx, "dw": dw, "dbias": db}


def exact_prefill(s):
    """The recurrence, one token after the other, all sequences side by side."""
    case, cu = s["case"], s["cu"].tolist()
    per = case["heads"] // case["groups"]
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=100)
    decay = torch.exp(dt * s["A"].double())
    x, B, C = s["x"].double(), s["B"].double(), s["C"].double()
    start = s["cu"][:-1].long()
    lens = s["cu"][1:].long() - start
    H = s["state"].double()[s["slots"].long()]
    H[s["fresh"]] = 0
    y = torch.empty_like(x)
    order = sorted(range(len(cu) - 1), key=lambda i: cu[i] - cu[i + 1])  # longest first
    order_t = torch.tensor(order, device="cuda")
    start, lens, H = start[order_t], lens[order_t], H[order_t]
    counts = sorted((cu[i + 1] - cu[i] for i in order), reverse=True)
    live = len(counts)
    for t in range(counts[0]):
        while counts[live - 1] <= t:
            live -= 1
        at = start[:live] + t
        Bt, Ct = (v[at].repeat_interleave(per, dim=1) for v in (B, C))
        part = H[:live]
        part.mul_(decay[at][:, :, None, None])
        part.add_((dt[at][:, :, None] * x[at])[..., None] * Bt[:, :, None])
        y[at] = torch.matmul(part, Ct[..., None])[..., 0]
    y += s["D"].double()[:, None] * x
    state = s["state"].double()
    state[s["slots"].long()[order_t]] = H
    return {"y": y, "state": state}


def exact_step(s):
    case = s["case"]
    d, bc, _, _ = widths(case)
    n, heads, groups, dstate = case["seqs"], case["heads"], case["groups"], case["dstate"]
    window, state, slots = s["window"].double(), s["state"].double(), s["slots"].long()
    x = s["xbc"].double()
    pre = s["bias"].double() + x * s["w"][:, -1].double()
    for k in range(case["width"] - 1):
        pre = pre + window[slots][:, :, k] * s["w"][:, k].double()
    v = pre * torch.sigmoid(pre)
    window[slots] = torch.cat([window[slots][:, :, 1:], x[:, :, None]], dim=2)
    u = v[:, :d].reshape(n, heads, HEADDIM)
    B = v[:, d:d + bc].reshape(n, groups, dstate).repeat_interleave(heads // groups, dim=1)
    C = v[:, d + bc:].reshape(n, groups, dstate).repeat_interleave(heads // groups, dim=1)
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=100)
    H = torch.exp(dt * s["A"].double())[..., None, None] * state[slots] + torch.einsum("bh,bhp,bhn->bhpn", dt, u, B)
    state[slots] = H
    y = torch.einsum("bhpn,bhn->bhp", H, C) + s["D"].double()[:, None] * u
    return {"y": y, "window": window, "state": state}


def exact_norm(s):
    x, z, w = s["x"].double(), s["z"].double(), s["w"].double()
    group = s["group"]
    sig = torch.sigmoid(z)
    v = (x * z * sig).unflatten(1, (-1, group))
    rstd = (v.square().sum(2, keepdim=True) / group + EPS).rsqrt()
    y = (v * rstd).flatten(1) * w
    if "dy" not in s:
        return y
    dy = s["dy"].double()
    dn = (dy * w).unflatten(1, (-1, group))
    dv = (rstd * dn - v * rstd ** 3 * (dn * v).sum(2, keepdim=True) / group).flatten(1)
    return {"y": y, "dx": dv * z * sig, "dz": dv * x * (sig + z * sig * (1 - sig)),
            "dw": (dy * (v * rstd).flatten(1)).sum(0)}


# ------------------------------------------------------------------ work -----
def work(case):
    d, bc, conv, _ = widths(case)
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "conv":
        t, taps = case["tokens"], case["width"]
        if case["mode"] == "serve":  # rows in and out, windows in and out, weights
            return {"bytes": 2 * t * conv * es + 2 * case["seqs"] * conv * (taps - 1) * 4 + conv * (taps + 1) * 4,
                    "flops": t * conv * (2 * taps + 4)}
        return {"bytes": 5 * t * conv * es + 2 * conv * (taps + 1) * 4,  # x, y; x, dy, dx
                "flops": t * conv * (8 * taps + 12)}
    if case["op"] == "prefill":
        t, heads = case["tokens"], case["heads"]
        state = case["seqs"] * d * case["dstate"] * 4
        return {"bytes": 2 * t * d * es + 2 * t * bc * es + t * heads * es + 2 * state,
                "flops": t * d * (4 * case["dstate"] + 2)}  # the recurrence's update and read-out
    if case["op"] == "step":
        n = case["seqs"]
        state = n * d * case["dstate"] * 4
        return {"bytes": 2 * state + 2 * n * conv * (case["width"] - 1) * 4 + n * (conv + d + case["heads"]) * es,
                "flops": n * d * 5 * case["dstate"]}
    t = case["tokens"]
    if case["mode"] == "serve":
        return {"bytes": 3 * t * d * es + d * 4, "flops": t * d * 9}
    return {"bytes": 8 * t * d * es + 2 * d * 4, "flops": t * d * 34}  # x, z, y; x, z, dy, dx, dz
