"""The SSD scan of ragged prompts and the one-token step, on caches, against the
token-by-token recurrence in 64 bits.

Bounds.  State: Delta (8 fp32 roundings), the weights exp(sum of Delta A) (the
exponent is a sum of at most 128 terms, and w |exponent| stays below 1 where it
matters), up to 384 accumulated products per 128-token chunk: 1024 fp32
roundings of the recurrence on absolute values.  y: the same, plus where the
scan forms its matrix operands in 16 bits, one rounding each of the masked
products M and of the state copy: one half step of the type on the magnitude."""
import pytest
import torch

import time_major_ref as ref
from selective_state_space_11_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OPS = 1024


@pytest.fixture(autouse=True)
def no_fault():
    ops.lib().ss_device_fault(1)
    yield
    assert ops.lib().ss_device_fault(1) == 0


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def make(tokens, nh, ng, N, dtype, seed, slice_rows=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt_ = TYPES[dtype]

    def rows(*tail, scale=1.0):
        n = 1
        for t in tail:
            n *= t
        wide = (torch.randn(tokens, n + 16, device=DEV, generator=g) * scale).to(dt_)
        v = wide[:, 8:8 + n] if slice_rows else wide[:, :n].contiguous()
        return v.unflatten(1, tail) if len(tail) > 1 else v

    u = lambda lo, hi: lo + (hi - lo) * torch.rand(nh, device=DEV, generator=g)
    q = dict(x=rows(nh, 64), dt=rows(nh), A=-torch.exp(u(0.0, 2.77)), B=rows(ng, N, scale=N ** -0.5),
             C=rows(ng, N, scale=N ** -0.5))
    kw = dict(D=u(0, 1), z=rows(nh, 64), dt_bias=torch.log(torch.expm1(u(1e-3, 0.1))))
    return g, q, kw


def check(y, state, r, dtype, exact=False):
    k = r["covered"]
    y = y.reshape(-1, *y.shape[-2:]).cpu()
    extra = 0.0 if exact else ref.half_step(dtype) * r["mag"][k]
    ref.assert_within(y[k], r["y"][k], r["mag"][k], dtype, "y", OPS, extra=extra)
    if state is not None:
        ref.assert_within(state, r["state"], r["mag_state"], torch.float32, "state", OPS)


@pytest.mark.parametrize("dtype,nh,ng,N,strided", [
    ("bf16", 4, 1, 128, False), ("f16", 6, 2, 64, True), ("bf16", 3, 1, 64, False), ("f16", 2, 2, 128, False),
    ("bf16", 5, 5, 128, True), ("bf16", 1, 1, 64, False)])
@pytest.mark.parametrize("lens", [[1], [3, 0, 130, 64, 1, 128, 257], [127, 129], [700], [0]])
def test_ragged_prompts_on_a_cache(dtype, nh, ng, N, strided, lens):
    tokens = sum(lens) + 2
    g, q, kw = make(tokens, nh, ng, N, dtype, 7 + N + nh, strided)
    cu = cu_of(lens)
    room = len(lens) + 2
    state = torch.randn(room, nh, 64, N, device=DEV, generator=g)
    slots = torch.randperm(room, device=DEV, generator=g)[:len(lens)].to(torch.int32)
    fresh = torch.rand(len(lens), device=DEV, generator=g) < 0.4
    r = ref.ssd(**q, **kw, cu=cu, state=state, slots=slots, fresh=fresh)
    out = torch.full((tokens, nh, 64), 7.0, device=DEV, dtype=TYPES[dtype])
    y = ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=state, slots=slots, fresh=fresh, out=out)
    check(y, state, r, TYPES[dtype])
    assert (y[sum(lens):] == 7).all(), "rows behind the last sequence were written"


@pytest.mark.parametrize("dtype,nh,N", [("bf16", 3, 128), ("f16", 2, 64)])
def test_long_sequences_split_over_blocks(dtype, nh, N):
    """Sequences that many blocks share: states handed over at the cuts, ranges inside one sequence."""
    lens = [3001, 5, 0, 1500, 260]
    g, q, kw = make(sum(lens), nh, 1, N, dtype, 67)
    state = torch.randn(5, nh, 64, N, device=DEV, generator=g)
    fresh = torch.tensor([0, 0, 1, 1, 0], dtype=torch.bool, device=DEV)
    slots = torch.tensor([4, 0, 3, 1, 2], dtype=torch.int32, device=DEV)
    q["dt"][::3] = -6.0  # long memories: the state that is handed over matters far behind the cut
    r = ref.ssd(**q, **kw, cu=cu_of(lens), state=state, slots=slots, fresh=fresh)
    y = ops.ssd_prefill(**q, **kw, cu_seqlens=cu_of(lens), state=state, slots=slots, fresh=fresh)
    check(y, state, r, TYPES[dtype])


def test_bare_call_dense_batch_and_flags():
    g, q, _ = make(2 * 90, 4, 2, 128, "bf16", 17)
    q4 = {k: v if k == "A" else v.reshape(2, 90, *v.shape[1:]) for k, v in q.items()}
    q4["dt"] = q4["dt"].abs() * 0.1
    y = ops.ssd_prefill(**q4, dt_softplus=False)
    r = ref.ssd(**q4, softplus=False)
    check(y, None, r, torch.bfloat16)
    assert y.shape == (2, 90, 4, 64)


def test_pieces_through_the_cache_equal_one_call():
    """Within the bound of the recurrence: pieces fall on other chunk borders."""
    g, q, kw = make(500, 4, 1, 128, "bf16", 27)
    state = torch.zeros(1, 4, 64, 128, device=DEV)
    r = ref.ssd(**q, **kw, state=state)
    at, ys = 0, []
    for i, n in enumerate([1, 200, 0, 1, 298]):
        cut = {k: v if k == "A" else v[at:at + n] for k, v in q.items()}
        ys.append(ops.ssd_prefill(**cut, **{**kw, "z": kw["z"][at:at + n]}, state=state,
                                  fresh=torch.tensor([i == 0], device=DEV)))
        at += n
    check(torch.cat(ys), state, r, torch.bfloat16)


def test_padding_bad_slots_and_leaks():
    g, q, kw = make(400, 2, 1, 64, "bf16", 37)
    cu = cu_of([100, 100, 50, 70, 80])
    state = torch.randn(6, 2, 64, 64, device=DEV, generator=g)
    state[5] = float("nan")
    slots = [2, -1, 2, 9, 5]  # one of padding, one taken, one that does not exist, a fresh one on a slot of NaN
    fresh = torch.tensor([0, 0, 0, 0, 1], dtype=torch.bool, device=DEV)
    before = state.clone()
    q["x"][100:200], q["B"][210:320] = float("nan"), float("inf")
    r = ref.ssd(**q, **kw, cu=cu, state=before, slots=[2, -1, -1, -1, 5], fresh=fresh)
    out = torch.full((400, 2, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=state, slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                    fresh=fresh, out=out)
    assert ops.lib().ss_device_fault(1) == 8
    assert (out[100:320] == 7).all()
    check(out, state, r, torch.bfloat16)
    assert torch.equal(state[[0, 1, 3, 4]], before[[0, 1, 3, 4]])
    for bad in ([0, 100, 50, 400], [0, 100, 900], [-9, 400]):
        ops.ssd_prefill(**q, **kw, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device=DEV))
        assert ops.lib().ss_device_fault(1) == 8


def test_prefill_repeatable_and_captured():
    g, q, kw = make(600, 4, 1, 128, "bf16", 47)
    cu, slots = cu_of([250, 350]), torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    start = torch.randn(3, 4, 64, 128, device=DEV, generator=g)
    state, out = start.clone(), torch.empty(600, 4, 64, device=DEV, dtype=torch.bfloat16)
    call = lambda: ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=state, slots=slots, out=out)
    call()
    first = (out.clone(), state.clone())
    state.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    state.copy_(start)
    graph.replay()
    assert torch.equal(out, first[0]) and torch.equal(state, first[1])
    cu.copy_(cu_of([599, 1]))
    slots.copy_(torch.tensor([2, 1], dtype=torch.int32))
    state.copy_(start)
    r = ref.ssd(**q, **kw, cu=cu, state=start, slots=slots)
    graph.replay()
    check(out, state, r, torch.bfloat16)


@pytest.mark.parametrize("dtype,nh,ng,N,W,bsz", [
    ("bf16", 4, 1, 128, 4, 1), ("f16", 6, 2, 64, 3, 5), ("f32", 2, 2, 128, 2, 3), ("bf16", 3, 1, 64, 1, 40),
    ("f32", 1, 1, 64, 4, 2)])
def test_step(dtype, nh, ng, N, W, bsz):
    g = torch.Generator(device=DEV).manual_seed(3 + bsz)
    t = TYPES[dtype]
    d = nh * 64
    dim = d + 2 * ng * N
    row = torch.randn(bsz, d + dim + nh + 3, device=DEV, generator=g).to(t)  # odd rows: no 16-byte alignment
    z, xbc, dt = row[:, :d], row[:, d:d + dim], row[:, d + dim:d + dim + nh]
    w = torch.randn(dim, W, device=DEV, generator=g) / W ** 0.5
    bias = torch.randn(dim, device=DEV, generator=g) * 0.1
    u = lambda lo, hi: lo + (hi - lo) * torch.rand(nh, device=DEV, generator=g)
    A, D, dt_bias = -torch.exp(u(0.0, 2.77)), u(0, 1), torch.log(torch.expm1(u(1e-3, 0.1)))
    room = bsz + 3
    win = torch.randn(room, dim, W - 1, device=DEV, generator=g)
    state = torch.randn(room, nh, 64, N, device=DEV, generator=g)
    slots = torch.randperm(room, device=DEV, generator=g)[:bsz].to(torch.int32)
    if bsz > 2:
        slots[1] = -1
    cu = torch.arange(bsz + 1, dtype=torch.int32)
    c = ref.conv(xbc, w, bias, cu=cu, state=win, slots=slots)
    v = torch.where(c["covered"][:, None], c["y"], torch.zeros_like(c["y"]))
    r = ref.ssd(v[:, :d].reshape(bsz, nh, 64), dt, A, v[:, d:d + ng * N].reshape(bsz, ng, N),
                v[:, d + ng * N:].reshape(bsz, ng, N), D=D, z=z.reshape(bsz, nh, 64), dt_bias=dt_bias, cu=cu,
                state=state, slots=slots)
    # the convolution's own roundings (16 of its magnitude) pass through x, B and C: as products of sums, they are
    # bounded by 3 * 16 roundings of the recurrence on the magnitudes of the convolution
    m = c["mag"]
    wide = ref.ssd(m[:, :d].reshape(bsz, nh, 64), dt, A, m[:, d:d + ng * N].reshape(bsz, ng, N),
                   m[:, d + ng * N:].reshape(bsz, ng, N), D=D, z=z.reshape(bsz, nh, 64).abs(), dt_bias=dt_bias, cu=cu,
                   state=state.abs(), slots=slots)
    out = torch.full((bsz, nh, 64), 7.0, device=DEV, dtype=t)
    y = ops.ssd_step(xbc, dt, w, A, win, state, conv_bias=bias, D=D, z=z, dt_bias=dt_bias, slots=slots, ngroups=ng, out=out)
    k = r["covered"]
    # one step: Delta and the decay (16), the update (3) and N / 4 + 7 adds per lane of the read-out, the gate (8)
    ref.assert_within(y.cpu()[k], r["y"][k], wide["mag"][k].abs(), t, "y", 128)
    ref.assert_within(state, r["state"], wide["mag_state"], torch.float32, "state", 128)
    assert torch.equal(win.cpu().double(), c["state"])
    assert (y.cpu()[~k] == 7).all()


def test_step_bad_slots():
    g = torch.Generator(device=DEV).manual_seed(9)
    bsz, nh, N = 4, 2, 64
    dim = nh * 64 + 2 * N
    xbc, dt = torch.randn(bsz, dim, device=DEV, generator=g), torch.randn(bsz, nh, device=DEV, generator=g)
    w, A = torch.randn(dim, 4, device=DEV, generator=g), -torch.ones(nh, device=DEV)
    win, state = torch.randn(3, dim, 3, device=DEV, generator=g), torch.randn(3, nh, 64, N, device=DEV, generator=g)
    a, b = (win.clone(), state.clone()), (win.clone(), state.clone())
    slots = torch.tensor([2, 3, 2, 0], dtype=torch.int32, device=DEV)
    out = torch.full((bsz, nh, 64), 7.0, device=DEV)
    ops.ssd_step(xbc, dt, w, A, *a, slots=slots, out=out)
    assert ops.lib().ss_device_fault(1) == 8
    y = ops.ssd_step(xbc, dt, w, A, *b, slots=torch.tensor([2, -1, -1, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(out[[0, 3]], y[[0, 3]]) and (out[1:3] == 7).all()


def test_two_streams_with_their_own_workspaces():
    g, q, kw = make(300, 4, 1, 64, "bf16", 57)
    want = ops.ssd_prefill(**q, **kw)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(ops.ssd_prefill(**q, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


@pytest.mark.parametrize("dtype,nh,ng,N,gate", [("bf16", 5, 1, 128, True), ("f16", 6, 2, 64, False), ("bf16", 12, 4, 64, True)])
def test_many_prompts_per_block(dtype, nh, ng, N, gate):
    """More (sequence, head pair) units than blocks, so that a block goes through several of every kind: whole
    ones of one chunk or more, parts, empty ones, skipped ones, pairs that hold one head."""
    g = torch.Generator().manual_seed(nh)
    lens = torch.randint(0, 260, (130,), generator=g)
    lens[torch.randperm(130, generator=g)[:25]] = 0
    lens[17] = 1500
    cu = cu_of(lens.tolist())
    tokens = int(lens.sum())
    gd, q, kw = make(tokens + 9, nh, ng, N, dtype, 71 + nh, slice_rows=True)
    if not gate:
        kw["z"] = None
    slots = torch.randperm(140, generator=g)[:130].to(torch.int32)
    slots[torch.randperm(130, generator=g)[:12]] = -1
    fresh = torch.rand(130, generator=g) < 0.5
    slots, fresh = slots.to(DEV), fresh.to(DEV)
    state = torch.randn(140, nh, 64, N, device=DEV, generator=gd)
    r = ref.ssd(**q, **kw, cu=cu, state=state, slots=slots, fresh=fresh)
    out = torch.full((tokens + 9, nh, 64), 7.0, device=DEV, dtype=q["x"].dtype)
    start = state.clone()
    y = ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=state, slots=slots, fresh=fresh, out=out)
    check(y, state, r, q["x"].dtype)
    assert (y.cpu()[~r["covered"]] == 7).all()
    again = start.clone()
    y2 = ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=again, slots=slots, fresh=fresh)
    k = r["covered"]
    assert torch.equal(y.cpu()[k], y2.cpu()[k]) and torch.equal(state, again)


@pytest.mark.parametrize("dtype,nh,N", [("bf16", 2, 128), ("f16", 1, 64)])
def test_a_long_prompt_among_short_ones(dtype, nh, N):
    """The long one's chunks go to some twenty blocks, most of which hold nothing else: each sums the states of
    all before it."""
    lens = [40] * 15 + [6000] + [40] * 15
    cu = cu_of(lens)
    g, q, kw = make(sum(lens), nh, 1, N, dtype, 91)
    q["A"] = q["A"] * 1e-3      # slow decay: what the first blocks publish reaches the last
    state = torch.randn(len(lens), nh, 64, N, device=DEV, generator=g)
    r = ref.ssd(**q, **kw, cu=cu, state=state)
    start = state.clone()
    y = ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=state)
    check(y, state, r, q["x"].dtype)
    again = start.clone()
    y2 = ops.ssd_prefill(**q, **kw, cu_seqlens=cu, state=again)
    assert torch.equal(y, y2) and torch.equal(state, again)
