"""The time-major operators in a row, as a Mamba-2 layer calls them between its two
projections: prompts into the caches, token by token from there on, and a training
step.  Every stage is compared with the 64-bit form of that stage on the values that
entered it, in the bounds of the operators' own tests."""
import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


class Layer:
    """The weights of a layer, and its work on rows [z | x B C | dt] of the input projection."""

    def __init__(self, nh, ng, N, group, seed, dtype=torch.bfloat16):
        self.nh, self.ng, self.N, self.group, self.dtype = nh, ng, N, group, dtype
        self.d, self.gn = nh * 64, ng * N
        self.dim = self.d + 2 * self.gn
        self.splits = (self.d, self.gn, self.gn)
        # rows of a projection are padded to 16 bytes, as the tensor-core tiles of the scan need them
        self.width = (self.d + self.dim + nh + 7) // 8 * 8
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, device=DEV, generator=self.g)
        u = lambda lo, hi: lo + (hi - lo) * torch.rand(nh, device=DEV, generator=self.g)
        self.w, self.bias = r(self.dim, 4) / 2, r(self.dim) / 10
        self.A, self.D = -torch.exp(u(0.0, 2.77)), u(0.0, 1.0)
        self.dt_bias = torch.log(torch.expm1(u(1e-3, 0.1)))
        self.norm_w = 1 + r(self.d) / 5

    def rows(self, *lead):
        return torch.randn(*lead, self.width, device=DEV, generator=self.g).to(self.dtype)

    def cut(self, row):
        d, dim = self.d, self.dim
        return row[..., :d], row[..., d:d + dim], row[..., d + dim:d + dim + self.nh]

    def caches(self, slots):
        return (torch.randn(slots, self.dim, 3, device=DEV, generator=self.g),
                torch.randn(slots, self.nh, 64, self.N, device=DEV, generator=self.g))

    def prompts(self, row, cu, win, state, slots, fresh):
        z, xbc, dt = self.cut(row)
        x, B, C = ops.conv1d_tm_fwd(xbc, self.w, self.bias, splits=self.splits, cu_seqlens=cu, state=win, slots=slots,
                                    fresh=fresh)
        x, B, C = x.unflatten(1, (self.nh, 64)), B.unflatten(1, (self.ng, self.N)), C.unflatten(1, (self.ng, self.N))
        y = ops.ssd_prefill(x, dt, self.A, B, C, state=state, D=self.D, dt_bias=self.dt_bias, cu_seqlens=cu,
                            slots=slots, fresh=fresh)
        out, _ = ops.gated_norm_fwd(y.flatten(1), z, self.norm_w, group=self.group, eps=EPS, want_rstd=False)
        return dict(x=x, B=B, C=C, y=y, out=out)

    def token(self, row, win, state, slots):
        z, xbc, dt = self.cut(row)
        y = ops.ssd_step(xbc, dt, self.w, self.A, win, state, conv_bias=self.bias, D=self.D, dt_bias=self.dt_bias,
                         slots=slots, ngroups=self.ng)
        out, _ = ops.gated_norm_fwd(y.flatten(1), z, self.norm_w, group=self.group, eps=EPS, want_rstd=False)
        return dict(y=y, out=out)

    def check_norm(self, got, z):
        r = ref.norm(got["y"].flatten(1), z, self.norm_w, self.group, EPS)
        ref.assert_within(got["out"], r["y"], r["y"].abs(), self.dtype, "norm", 64)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("nh,ng,N,group", [(4, 1, 128, 256), (6, 2, 64, 64)])
def test_prompts_then_tokens(nh, ng, N, group):
    """Three prompts, one of them continuing a cached sequence, then 4 tokens of two requests; and the
    windows and states at the end are those of the whole sequences run as prompts."""
    m = Layer(nh, ng, N, group, 100 + nh)
    lens, more = [130, 3, 300], 4
    cu, slots = i32(0, 130, 133, 433), i32(4, 0, 2)
    fresh = torch.tensor([True, False, True], device=DEV)
    win, state = m.caches(5)
    win0, state0 = win.clone(), state.clone()
    row = m.rows(433)
    z, xbc, dt = m.cut(row)
    got = m.prompts(row, cu, win, state, slots, fresh)
    c = ref.conv(xbc, m.w, m.bias, cu=cu, state=win0, slots=slots, fresh=fresh)
    pieces = torch.cat([got["x"].flatten(1), got["B"].flatten(1), got["C"].flatten(1)], 1)
    ref.assert_within(pieces, c["y"], c["mag"], m.dtype, "convolution", 16)
    assert torch.equal(win.cpu().double(), c["state"])
    r = ref.ssd(got["x"], dt, m.A, got["B"], got["C"], D=m.D, dt_bias=m.dt_bias, cu=cu, state=state0, slots=slots,
                fresh=fresh)
    half = ref.half_step(m.dtype)
    ref.assert_within(got["y"], r["y"], r["mag"], m.dtype, "scan", 1024, extra=half * r["mag"])
    ref.assert_within(state, r["state"], r["mag_state"], torch.float32, "state", 1024)
    m.check_norm(got, z)

    going = i32(2, 4)          # the requests of slots 2 and 4 go on; slot 0 rests
    rest_win, rest_state = win[0].clone(), state[0].clone()
    tokens = m.rows(more, 2)
    for k in range(more):
        before_w, before_s = win.clone(), state.clone()
        zk, xk, dk = m.cut(tokens[k])
        one = m.token(tokens[k], win, state, going)
        at = torch.arange(3, dtype=torch.int32)
        c = ref.conv(xk, m.w, m.bias, cu=at, state=before_w, slots=going)
        heads = lambda v: (v[:, :m.d].reshape(2, nh, 64), v[:, m.d:m.d + m.gn].reshape(2, ng, N),
                           v[:, m.d + m.gn:].reshape(2, ng, N))
        for name, v, s in (("y", c["y"], before_s), ("mag", c["mag"], before_s.abs())):
            x, B, C = heads(v)
            q = ref.ssd(x, dk, m.A, B, C, D=m.D, dt_bias=m.dt_bias, cu=at, state=s, slots=going)
            if name == "y":
                want = q
        ref.assert_within(one["y"], want["y"], q["mag"], m.dtype, "step", 128)
        ref.assert_within(state, want["state"], q["mag_state"], torch.float32, "state after a step", 128)
        assert torch.equal(win.cpu().double(), c["state"])
        m.check_norm(one, zk)
    assert torch.equal(win[0], rest_win) and torch.equal(state[0], rest_state)

    # the same sequences as prompts: the window exactly; the state up to what rounding x, B and C to 16 bits in
    # front of the scan, where the step keeps them in fp32, leaves in the last tokens: each product of x and B
    # has two such roundings, of half a step each
    whole = torch.cat([row[133:433], tokens[:, 0], row[:130], tokens[:, 1]])
    cu2 = i32(0, 300 + more, 430 + 2 * more)
    win2, state2 = m.caches(5)
    yes = torch.ones(2, dtype=torch.bool, device=DEV)
    again = m.prompts(whole, cu2, win2, state2, going, yes)
    assert torch.equal(win2[[2, 4]], win[[2, 4]])
    _, xw, dw = m.cut(whole)
    c = ref.conv(xw, m.w, m.bias, cu=cu2)["mag"]
    x, B, C = c[:, :m.d].reshape(-1, nh, 64), c[:, m.d:m.d + m.gn].reshape(-1, ng, N), c[:, m.d + m.gn:].reshape(-1, ng, N)
    mag = ref.ssd(x, dw, m.A, B, C, dt_bias=m.dt_bias, cu=cu2, state=torch.zeros(2, nh, 64, N))["mag_state"]
    tol = (2 * half * (1 + half) + 2 * 1024 * 2.0 ** -24) * mag
    assert ((state2[[2, 4]].cpu().double() - state[[2, 4]].cpu().double()).abs() <= tol).all()
    assert torch.isfinite(again["out"]).all()


def test_a_captured_token_follows_its_slots_and_caches():
    """One captured decode step of padded batch 4, replayed for other requests and with padding, on a stream of
    its own: the results of the calls made one by one."""
    m = Layer(4, 1, 64, 128, 7)
    win, state = m.caches(6)
    w2, s2 = win.clone(), state.clone()
    row, slots = m.rows(4), i32(0, 1, 2, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.token(row, win.clone(), state.clone(), slots)     # warm
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = m.token(row, win, state, slots)
    torch.cuda.current_stream().wait_stream(side)
    for ids in ([0, 1, 2, 3], [5, 2, -1, 0], [3, -1, -1, -1], [-1, -1, -1, -1], [5, 4, 3, 2]):
        row.copy_(m.rows(4))
        slots.copy_(i32(*ids))
        live = [i for i, s in enumerate(ids) if s >= 0]
        graph.replay()
        want = m.token(row, w2, s2, slots)
        assert torch.equal(win, w2) and torch.equal(state, s2)
        for name in ("y", "out"):
            assert torch.equal(got[name][live], want[name][live])


@pytest.mark.parametrize("ragged", [False, True])
def test_training_step(ragged):
    """Convolution, scan and norm under autograd: each operator's gradient against the formula on what reached it.
    Ragged: the convolution over packed documents that leave 5 rows unused, ahead of the norm alone."""
    m = Layer(4, 2, 64, 128, 11)
    b, L = 2, 161
    row = m.rows(b * L).requires_grad_() if ragged else m.rows(b, L).requires_grad_()
    p = [t.clone().requires_grad_() for t in (m.w, m.bias, m.norm_w)]
    cu = i32(0, 1, 1, 200, b * L - 5) if ragged else None
    z, xbc, dt = m.cut(row)
    for t in (z, xbc):
        t.retain_grad()
    pieces = ops.causal_conv1d_tm_fn(xbc, p[0], p[1], splits=m.splits, cu_seqlens=cu)
    if ragged:
        assert all((t[b * L - 5:] == 0).all() for t in pieces)
        y = pieces[0] + pieces[1].repeat(1, m.d // m.gn) * pieces[2].repeat(1, m.d // m.gn)
    else:
        x, B, C = pieces
        y = ops.ssd_fn(x.unflatten(2, (m.nh, 64)), dt.contiguous(), m.A, B.unflatten(2, (m.ng, m.N)),
                       C.unflatten(2, (m.ng, m.N)), D=m.D, dt_bias=m.dt_bias).flatten(2)
    for t in pieces + (y,):
        t.retain_grad()
    out = ops.gated_norm_fn(y, z, p[2], group=m.group, eps=EPS)
    dout = torch.randn(out.shape, device=DEV, generator=m.g).to(m.dtype)
    out.backward(dout)

    r = ref.norm(y, z, p[2], m.group, EPS, dy=dout)
    flat = lambda t: t.reshape(-1, t.shape[-1])
    ref.assert_within(flat(out), r["y"], r["y"].abs(), m.dtype, "norm", 64)
    ref.assert_within(flat(y.grad), r["dx"], r["mag_dx"], m.dtype, "norm dx", 128)
    ref.assert_within(flat(z.grad), r["dz"], r["mag_dz"], m.dtype, "norm dz", 128)
    ref.assert_within(p[2].grad, r["dw"], r["mag_dw"], torch.float32, "norm dw", 64 + b * L)
    dy = torch.cat([t.grad for t in pieces], -1)
    r = ref.conv(xbc, p[0], p[1], cu=cu, dy=dy)
    k = r["covered"]
    ref.assert_within(flat(torch.cat(pieces, -1)).cpu()[k], r["y"][k], r["mag"][k], m.dtype, "convolution", 16)
    ref.assert_within(flat(xbc.grad), r["dx"], r["mag_dx"], m.dtype, "convolution dx", 32)
    ref.assert_within(p[0].grad, r["dw"], r["mag_dw"], torch.float32, "convolution dw", b * L + 32)
    ref.assert_within(p[1].grad, r["db"], r["mag_db"], torch.float32, "convolution dbias", b * L + 32)
    # the columns that the layer does not read have no gradient, the others are finite
    assert (row.grad[..., m.d + m.dim + m.nh:] == 0).all() and torch.isfinite(row.grad).all()


def test_a_captured_training_step():
    """Forward and backward of convolution and norm captured together through the explicit calls."""
    m = Layer(2, 1, 64, 128, 13)
    row, dout = m.rows(300), torch.randn(300, m.d, device=DEV, generator=m.g).to(m.dtype)
    grad = torch.zeros_like(row)

    def step():
        z, xbc, _ = m.cut(row)
        gz, gx, _ = m.cut(grad)
        x, B, C = ops.conv1d_tm_fwd(xbc, m.w, m.bias, splits=m.splits)
        out, rstd = ops.gated_norm_fwd(x, z, m.norm_w, group=m.group, eps=EPS)
        n = ops.gated_norm_bwd(x, z, m.norm_w, dout, rstd, group=m.group, dz=gz)
        c = ops.conv1d_tm_bwd(xbc, m.w, [n["dx"], B, C], m.bias, dx=gx)
        return out, n["dw"], c["dw"], c["dbias"]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        row.copy_(m.rows(300))
        dout.copy_(torch.randn(300, m.d, device=DEV, generator=m.g).to(m.dtype))
        graph.replay()
        seen = [t.clone() for t in (*got, grad)]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(seen, (*want, grad)))


@pytest.mark.parametrize("name", ["conv", "conv_bwd", "prefill", "step", "norm", "norm_bwd"])
def test_an_injected_launch_failure_is_reported_and_enqueues_nothing(name, monkeypatch):
    """The failure is made on the host; no GPU fault is involved."""
    m = Layer(2, 1, 64, 128, 17)
    row = m.rows(40)
    z, xbc, dt = m.cut(row)
    win, state = m.caches(40)
    win0, state0 = win.clone(), state.clone()
    x, B, C = ops.conv1d_tm_fwd(xbc, m.w, m.bias, splits=m.splits)
    _, rstd = ops.gated_norm_fwd(x, z, m.norm_w, group=m.group)
    out = torch.full_like(x, 7.0)
    calls = dict(
        conv=lambda: ops.conv1d_tm_fwd(xbc, m.w, m.bias, splits=m.splits, state=win, out=(out, B, C)),
        conv_bwd=lambda: ops.conv1d_tm_bwd(xbc, m.w, [x, B, C], m.bias),
        prefill=lambda: ops.ssd_prefill(x.unflatten(1, (2, 64)), dt, m.A, B.unflatten(1, (1, 64)), C.unflatten(1, (1, 64)),
                                        state=state, out=out.unflatten(1, (2, 64))),
        step=lambda: ops.ssd_step(xbc, dt, m.w, m.A, win, state, out=out.unflatten(1, (2, 64))),
        norm=lambda: ops.gated_norm_fwd(x, z, m.norm_w, group=m.group, out=out),
        norm_bwd=lambda: ops.gated_norm_bwd(x, z, m.norm_w, x, rstd, group=m.group, dx=out))
    monkeypatch.setenv("SS_FAIL_LAUNCH", "1")
    with pytest.raises(ops.SSError) as e:
        calls[name]()
    assert e.value.status == 5 and "SS_FAIL_LAUNCH" in str(e.value)
    torch.cuda.synchronize()
    assert (out == 7).all() and torch.equal(win, win0) and torch.equal(state, state0)
    monkeypatch.delenv("SS_FAIL_LAUNCH")
    calls[name]()
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits():
    """Rows a million elements apart and slots far into a cache of states, so that both pass 2^31 elements: the
    results of dense rows and a small cache."""
    m = Layer(4, 1, 128, 256, 23)
    tokens, far = 2200, (1 << 31) // (4 * 64 * 128) + 3
    dense = m.rows(tokens)
    wide = torch.empty(tokens, 1 << 20, device=DEV, dtype=m.dtype)[:, :m.width]
    wide.copy_(dense)
    grads = torch.empty(tokens, 1 << 20, device=DEV, dtype=m.dtype)[:, :m.width]
    cu = i32(0, 1500, tokens)
    win, state = m.caches(2)
    big_state = torch.empty(far, 4, 64, 128, device=DEV)
    big_win = torch.empty(far, m.dim, 3, device=DEV)
    big_state[-2:], big_win[-2:] = state, win
    here, there = i32(0, 1), i32(far - 2, far - 1)

    def run(row, w, s, slots, gz, gx):
        got = m.prompts(row, cu, w, s, slots, None)
        one = m.token(row[:2], w, s, slots)
        z, xbc, _ = m.cut(row)
        y = got["y"].flatten(1)
        out, rstd = ops.gated_norm_fwd(y, z, m.norm_w, group=m.group)
        n = ops.gated_norm_bwd(y, z, m.norm_w, out, rstd, group=m.group, dz=gz)
        c = ops.conv1d_tm_bwd(xbc, m.w, [n["dx"], got["B"].flatten(1), got["C"].flatten(1)], m.bias, cu_seqlens=cu, dx=gx)
        return [got["y"], got["out"], one["y"], one["out"], out, n["dx"], n["dw"], c["dw"], c["dbias"]]

    small = torch.empty_like(dense)
    a = run(dense, win, state, here, m.cut(small)[0], m.cut(small)[1])
    b = run(wide, big_win, big_state, there, m.cut(grads)[0], m.cut(grads)[1])
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert torch.equal(big_state[-2:], state) and torch.equal(big_win[-2:], win)
    assert all(torch.equal(u, v) for u, v in zip(m.cut(small)[:2], m.cut(grads)[:2]))
