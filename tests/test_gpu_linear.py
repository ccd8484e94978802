"""Linear attention with a decay per head and its state pages, on the GPU,
against the 64-bit recurrence (tests/linear_ref.py has the bounds)."""
import random

import pytest
import torch

import gated_delta_rule_forward_b200 as gdr
import linear_ref as ref
from gated_delta_rule_forward_b200.inputs import make_decode_inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DECAYS = (-0.3, -1e-3, 0.0, -2.0, float("-inf"), -20.0, -0.05, -1e-6)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def decays(H, first=0):
    return torch.tensor([DECAYS[(first + i) % len(DECAYS)] for i in range(H)], device="cuda")


def tensors(seed, B, T, Hk, H, dk, dv, dtype):
    g = gen(seed)
    return (randn(g, B, T, Hk, dk, dtype=dtype), randn(g, B, T, Hk, dk, dtype=dtype),
            randn(g, B, T, H, dv, dtype=dtype), g)


def fine():
    torch.cuda.synchronize()
    gdr.device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,state", [
    (1, 1, 1, 1, 64, 64, True), (2, 2, 1, 2, 128, 128, False), (1, 63, 2, 2, 64, 128, True),
    (3, 64, 1, 3, 128, 64, True), (1, 65, 2, 4, 128, 128, True), (2, 127, 1, 1, 64, 64, False),
    (1, 130, 3, 6, 128, 64, True), (2, 200, 2, 2, 128, 128, True), (1, 321, 1, 1, 64, 128, False),
])
def test_forward(dtype, B, T, Hk, H, dk, dv, state):
    q, k, v, g = tensors(T, B, T, Hk, H, dk, dv, dtype)
    S0 = randn(g, B, H, dk, dv) if state else None
    ld = decays(H, T)
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, scale=dk ** -0.5)
    fine()
    for b in range(B):
        ref.check_forward(q[b], k[b], v[b], ld, S0[b] if state else None, dk ** -0.5, o[b], S[b], f"row {b}")


@pytest.mark.parametrize("dtype,T,H,dk,dv", [(BF16, 1500, 2, 128, 128), (BF16, 1345, 3, 64, 64), (F32, 700, 1, 128, 64),
                                            (BF16, 901, 1, 64, 128)])
def test_forward_segments(dtype, T, H, dk, dv):
    """Few long sequences, cut into segments; states kept and resumed from."""
    q, k, v, g = tensors(T, 1, T, H, H, dk, dv, dtype)
    S0 = randn(g, 1, H, dk, dv)
    ld = torch.tensor([-1e-3, -0.2, 0.0][:H], device="cuda")
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, scale=0.1)
    fine()
    ref.check_forward(q[0], k[0], v[0], ld, S0[0], 0.1, o[0], S[0])
    cut = 457
    o1, S1 = gdr.linear_forward(q[:, :cut], k[:, :cut], v[:, :cut], log_decay=ld, initial_state=S0, scale=0.1)
    o2, S2 = gdr.linear_forward(q[:, cut:], k[:, cut:], v[:, cut:], log_decay=ld, initial_state=S1, final_state=S1,
                                scale=0.1)
    assert S2.data_ptr() == S1.data_ptr()
    ref.check_forward(q[0], k[0], v[0], ld, S0[0], 0.1, torch.cat([o1, o2], 1)[0], S2[0], "resumed")


LENS = [0, 1, 64, 65, 0, 130, 3, 63, 200, 0]


@pytest.mark.parametrize("dtype,Hk,H,dk,dv,lens", [
    (BF16, 2, 2, 128, 128, LENS), (BF16, 1, 2, 128, 64, LENS), (BF16, 2, 4, 64, 128, LENS), (F32, 1, 2, 128, 64, LENS),
    (BF16, 1, 1, 128, 128, [1]), (F32, 1, 1, 64, 64, [0]), (BF16, 1, 2, 64, 64, [1000, 0, 1, 777]),
    (BF16, 1, 1, 128, 128, [1] * 70 + [0] * 5 + [66])])
def test_forward_packed(dtype, Hk, H, dk, dv, lens):
    """Packed sequences, with NaN in the rows that belong to none and pages by slot."""
    T, N = sum(lens) + 5, len(lens)
    q, k, v, g = tensors(N, 1, T, Hk, H, dk, dv, dtype)
    for x in (q, k, v):
        x[:, sum(lens):] = float("nan")
    ld = decays(H, 1)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    pages = N + 3
    slots = torch.randperm(pages, generator=g, device="cuda")[:N].to(torch.int32)
    pool = randn(g, pages, H, dk, dv)
    before = pool.clone()
    out = torch.full((1, T, H, dv), 7.0, device="cuda", dtype=dtype)
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=pool, final_state=pool, cu_seqlens=cu,
                              state_slots=slots, scale=0.2, out=out)
    fine()
    assert o.data_ptr() == out.data_ptr() and S.data_ptr() == pool.data_ptr()
    assert (out[:, sum(lens):] == 7.0).all()
    t = 0
    for n, L in enumerate(lens):
        page = int(slots[n])
        s = slice(t, t + L)
        ref.check_forward(q[0, s], k[0, s], v[0, s], ld, before[page], 0.2, o[0, s], pool[page], f"sequence {n}")
        t += L
    unused = [p for p in range(pages) if p not in slots.tolist()]
    assert torch.equal(pool[unused], before[unused])
    # without slots, fresh outputs: the same values, zeros behind the last sequence
    o2, S2 = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=before[slots.long()].contiguous(), cu_seqlens=cu,
                                scale=0.2)
    fine()
    assert torch.equal(o2[:, :t], o[:, :t]) and (o2[:, t:] == 0).all()
    assert torch.equal(S2, pool[slots.long()])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_tail_neighbours(dtype):
    """Non-finite tokens of the next sequence do not reach the one before it."""
    lens = [70, 30]
    q, k, v, _ = tensors(3, 1, 100, 1, 1, 128, 128, dtype)
    ld = torch.tensor([-0.1], device="cuda")
    cu = torch.tensor([0, 70, 100], device="cuda", dtype=torch.int32)
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, cu_seqlens=cu)
    for x in (q, k, v):
        x[:, 70:] = float("inf")
    o2, S2 = gdr.linear_forward(q, k, v, log_decay=ld, cu_seqlens=cu)
    fine()
    assert torch.equal(o[:, :70], o2[:, :70]) and torch.equal(S[0], S2[0])
    assert not torch.isfinite(S2[1]).all()


def test_forward_slots_outside_the_pool():
    lens, H = [5, 70, 9], 2
    q, k, v, g = tensors(4, 1, 84, H, H, 128, 128, BF16)
    ld = decays(H)
    cu = torch.tensor([0, 5, 75, 84], device="cuda", dtype=torch.int32)
    pool = randn(g, 2, H, 128, 128)
    before = pool.clone()
    slots = torch.tensor([-1, 1, 2], device="cuda", dtype=torch.int32)
    o, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=pool, final_state=pool, cu_seqlens=cu,
                              state_slots=slots)
    fine()
    assert torch.equal(pool[0], before[0])
    ref.check_forward(q[0, :5], k[0, :5], v[0, :5], ld, None, 1.0, o[0, :5], None)
    ref.check_forward(q[0, 5:75], k[0, 5:75], v[0, 5:75], ld, before[1], 1.0, o[0, 5:75], pool[1])
    ref.check_forward(q[0, 75:], k[0, 75:], v[0, 75:], ld, None, 1.0, o[0, 75:], None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_inputs(dtype):
    """q, k and v as slices of one projection, and the gradients from a strided d_o: bitwise the dense call's."""
    B, T, H, d = 2, 150, 3, 64
    g = gen(5)
    qkv = randn(g, B, T, 3 * H, d, dtype=dtype)
    q, k, v = qkv.split(H, 2)
    wide = randn(g, B, H, T, 2 * d, dtype=dtype)
    do = wide[..., d:].transpose(1, 2)
    ld = decays(H)
    a = gdr.linear_forward(q, k, v, log_decay=ld)
    b = gdr.linear_forward(q.contiguous(), k.contiguous(), v.contiguous(), log_decay=ld)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = gdr.linear_backward(q, k, v, do, log_decay=ld)
    y = gdr.linear_backward(q.contiguous(), k.contiguous(), v.contiguous(), do.contiguous(), log_decay=ld)
    fine()
    assert all(torch.equal(x[n], y[n]) for n in x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,state", [
    (1, 1, 1, 1, 128, 128, True), (2, 2, 1, 2, 64, 64, True), (1, 63, 2, 2, 64, 128, True),
    (2, 64, 1, 3, 128, 64, False), (1, 65, 1, 4, 128, 128, True), (3, 130, 2, 2, 64, 64, False),
    (1, 333, 1, 2, 128, 128, True),
])
def test_backward(dtype, B, T, Hk, H, dk, dv, state):
    q, k, v, g = tensors(T + 1, B, T, Hk, H, dk, dv, dtype)
    do = randn(g, B, T, H, dv, dtype=dtype)
    S0 = randn(g, B, H, dk, dv) if state else None
    dS = randn(g, B, H, dk, dv) if state else None
    ld = decays(H, T)
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, scale=0.3)
    fine()
    for b in range(B):
        ref.check_grads(q[b], k[b], v[b], do[b], ld, S0[b] if state else None, dS[b] if state else None, 0.3,
                        (x["q"][b], x["k"][b], x["v"][b], x["initial_state"][b]), f"row {b}")


@pytest.mark.parametrize("dtype,Hk,H,dk,dv,lens", [
    (BF16, 1, 1, 128, 128, LENS), (BF16, 1, 2, 64, 128, LENS), (F32, 1, 2, 128, 64, LENS),
    (BF16, 1, 1, 64, 64, [900, 0, 1, 411])])
def test_backward_packed(dtype, Hk, H, dk, dv, lens):
    T, N = sum(lens) + 4, len(lens)
    q, k, v, g = tensors(N + 1, 1, T, Hk, H, dk, dv, dtype)
    do = randn(g, 1, T, H, dv, dtype=dtype)
    for x in (q, k, v, do):
        x[:, sum(lens):] = float("nan")
    S0, dS = randn(g, N, H, dk, dv), randn(g, N, H, dk, dv)
    ld = decays(H, 6)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, cu_seqlens=cu, scale=0.3)
    fine()
    t = 0
    for n, L in enumerate(lens):
        s = slice(t, t + L)
        ref.check_grads(q[0, s], k[0, s], v[0, s], do[0, s], ld, S0[n], dS[n], 0.3,
                        (x["q"][0, s], x["k"][0, s], x["v"][0, s], x["initial_state"][n]), f"sequence {n}")
        t += L
    assert all((x[n][:, t:] == 0).all() for n in "qkv")


def test_backward_against_differences():
    """The forward is linear in each input, so <grad, d> is f(x + d) - f(x) without a truncation error (fp32)."""
    B, T, Hk, H, dk, dv, scale = 1, 150, 1, 2, 64, 64, 0.5
    q, k, v, g = tensors(8, B, T, Hk, H, dk, dv, F32)
    do, S0, dS = randn(g, B, T, H, dv), randn(g, B, H, dk, dv), randn(g, B, H, dk, dv)
    ld = torch.tensor([-0.05, -0.5], device="cuda")
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, scale=scale)

    def loss(q, k, v, S0):
        o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, scale=scale)
        return (do.double() * o.double()).sum() + (dS.double() * S.double()).sum()

    args = {"q": q, "k": k, "v": v, "initial_state": S0}
    at = loss(*args.values())
    # fp32_bound per element, summed over the products with d_o and d_final_state
    a_o, a_S = ref.run(q[0].abs(), k[0].abs(), v[0].abs(), ld, S0[0].abs(), scale)
    tol = 8 * (ref.fp32_bound(a_o, T, dk) * do[0].abs().double().cpu()).sum()
    tol = tol + 8 * (ref.fp32_bound(a_S, T, dk) * dS[0].abs().double().cpu()).sum()
    for name in args:
        d = randn(g, *args[name].shape)
        new = loss(*[a + d if n == name else a for n, a in args.items()])
        slope = (x[name].double() * d.double()).sum()
        assert abs((new - at - slope).item()) <= tol.item(), name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Hk,H,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 4, 128, 128), (5, 3, 3, 64, 128), (7, 1, 2, 128, 64),
                                         (80, 4, 8, 64, 64), (300, 1, 1, 128, 128)])
def test_decode(dtype, N, Hk, H, dk, dv):
    g = gen(N)
    pages = N + 4
    q, k, v = randn(g, N, Hk, dk, dtype=dtype), randn(g, N, Hk, dk, dtype=dtype), randn(g, N, H, dv, dtype=dtype)
    state = randn(g, pages, H, dk, dv)
    before = state.clone()
    slots = torch.randperm(pages, generator=g, device="cuda")[:N].to(torch.int32)
    if N > 2:
        slots[1], slots[2] = -1, pages
    ld = decays(H)
    o = gdr.linear_decode_step(q, k, v, state, log_decay=ld, state_slots=slots, scale=0.25)
    fine()
    touched = set()
    for n in range(N):
        page = int(slots[n])
        if not 0 <= page < pages:
            assert (o[n] == 0).all()
            continue
        touched.add(page)
        S, (r, rS) = before[page], ref.run(q[n:n + 1], k[n:n + 1], v[n:n + 1], ld, before[page], 0.25)
        a, aS = ref.run(q[n:n + 1].abs(), k[n:n + 1].abs(), v[n:n + 1].abs(), ld, S.abs(), 0.25)
        e = ref.fp32_bound(a, 1, dk)
        ref.check(o[n:n + 1], r, e + ref.HALF[dtype] * (r.abs() + e), f"row {n} o")   # fp32 inside for both types
        ref.check(state[page], rS, ref.fp32_bound(aS, 1, dk), f"row {n} state")
    rest = [p for p in range(pages) if p not in touched]
    assert torch.equal(state[rest], before[rest])


def test_decode_continues_the_forward():
    N, H, dk, dv, T = 3, 2, 128, 128, 70
    q, k, v, g = tensors(11, N, T + 5, H, H, dk, dv, F32)
    ld = torch.tensor([-0.01, -0.4], device="cuda")
    _, S = gdr.linear_forward(q[:, :T], k[:, :T], v[:, :T], log_decay=ld)
    o = [gdr.linear_decode_step(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(), S, log_decay=ld)
         for t in range(T, T + 5)]
    fine()
    for n in range(N):
        r, rS = ref.run(q[n], k[n], v[n], ld)
        a, aS = ref.run(q[n].abs(), k[n].abs(), v[n].abs(), ld)
        ref.check(torch.stack([x[n] for x in o]), r[T:], ref.out_bound(a, r, T + 5, dk, F32)[T:], f"sequence {n}")
        ref.check(S[n], rS, ref.fp32_bound(aS, T + 5, dk), f"state {n}")


@pytest.mark.parametrize("shape,n", [((5, 1, 64, 64), 12), ((3, 9, 2, 128, 64), 30), ((2, 700, 1, 64, 64), 1200),
                                     ((1, 3, 3, 128, 128), 1)])
def test_copy_states(shape, n):
    """Any list of pairs acts as one pair after another, dependent ones too."""
    pool = randn(gen(n), *shape)
    pages = shape[-4]
    rng = random.Random(n)
    src = [rng.randint(-1, pages - 1) for _ in range(n)]
    dst = [rng.randrange(pages) for _ in range(n)]
    want = pool.clone()
    for a, b in zip(src, dst):
        page = want.select(-4, b)
        page.copy_(want.select(-4, a) if a >= 0 else torch.zeros_like(page))
    gdr.copy_states(pool, src, dst)
    fine()
    assert torch.equal(pool, want)
    gdr.copy_states(pool, [], [])
    assert torch.equal(pool, want)


def test_serving_run():
    """Prefill into pages, fork, decode, free and compact, as a server does; then the delta-rule decode on the
    compacted front."""
    H, dk, dv = 2, 128, 128
    ld = [torch.tensor([-0.02, -0.3], device="cuda"), torch.tensor([-0.1, 0.0], device="cuda")]
    cache = gdr.StateCache(8, 2, H, dk, dv)
    g = gen(21)
    lens = [70, 1, 130]
    pages = cache.alloc(3)
    cu = torch.tensor([0, 70, 71, 201], device="cuda", dtype=torch.int32)
    history = {}    # page -> per layer (q, k, v) of all its tokens
    for l in range(2):
        q, k, v = (randn(g, 1, 201, H, d, dtype=BF16) for d in (dk, dk, dv))
        pool = cache.layer(l)
        o, _ = gdr.linear_forward(q, k, v, log_decay=ld[l], initial_state=pool, final_state=pool, cu_seqlens=cu,
                                  state_slots=torch.tensor(pages, device="cuda", dtype=torch.int32), scale=0.1)
        for n, p in enumerate(pages):
            s = slice(int(cu[n]), int(cu[n + 1]))
            history[l, p] = [x[0, s] for x in (q, k, v)]
            ref.check_forward(*history[l, p], ld[l], None, 0.1, o[0, s], pool[p], f"layer {l} page {p}")
    forks = cache.fork(pages[2], 2)
    for l in range(2):
        for p in forks:
            history[l, p] = history[l, pages[2]]
    cache.free([pages[0]])
    live = cache.live_pages
    rows = live + [-1]                       # one padding row

    def decode():
        slots = torch.tensor(rows, device="cuda", dtype=torch.int32)
        for l in range(2):
            q, k, v = (randn(g, len(rows), H, d, dtype=BF16) for d in (dk, dk, dv))
            gdr.linear_decode_step(q, k, v, cache.layer(l), log_decay=ld[l], state_slots=slots, scale=0.1)
            for i, p in enumerate(rows):
                if p >= 0:
                    history[l, p] = [torch.cat([a, b[i:i + 1]]) for a, b in zip(history[l, p], (q, k, v))]

    decode()
    cache.free([live[0]])
    moved = cache.compact()
    for old, new in moved.items():
        for l in range(2):
            history[l, new] = history.pop((l, old))
    live = cache.live_pages
    assert live == list(range(len(live)))
    rows = live + [-1]
    decode()
    fine()
    for l in range(2):
        for p in live:
            q, k, v = history[l, p]
            r, aS = ref.run(q, k, v, ld[l])[1], ref.run(q.abs(), k.abs(), v.abs(), ld[l])[1]
            ref.check(cache.layer(l)[p], r, ref.fp32_bound(aS, len(q), dk), f"layer {l} page {p}")
    d = {n: None if x is None else x.cuda() for n, x in make_decode_inputs("gdn", len(live), H, 5).items()}
    front = cache.layer(0)[:len(live)]
    want = front.clone()
    gates = {n: d[n] for n in ("beta", "log_g", "erase_b", "write_w")}
    a = gdr.decode_step(d["q"], d["k"], d["v"], want, variant="gdn", **gates)
    b = gdr.decode_step(d["q"], d["k"], d["v"], front, variant="gdn", **gates)
    fine()
    assert torch.equal(a, b) and torch.equal(front, want)


def test_repeatable_captured_and_on_streams():
    """The same inputs give the same bits: again, in a replayed graph (new inputs in the same buffers too), and on
    two side streams at once."""
    B, T, H, dk, dv = 1, 1100, 2, 128, 128
    q, k, v, g = tensors(13, B, T, H, H, dk, dv, BF16)
    do, S0 = randn(g, B, T, H, dv, dtype=BF16), randn(g, B, H, dk, dv)
    ld = torch.tensor([-0.01, -0.2], device="cuda")
    pool = randn(g, 6, H, dk, dv)

    def call(q=q, k=k, v=v, stream=None):
        o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, stream=stream)
        x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=S, stream=stream)
        return [o, S, x["q"], x["k"], x["v"], x["initial_state"]]

    want = call()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
        gdr.copy_states(pool, [0, 1, -1], [1, 2, 0])
    before = pool.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(pool[1], before[0]) and torch.equal(pool[2], before[0]) and (pool[0] == 0).all()
    q2, k2, v2, _ = tensors(14, B, T, H, H, dk, dv, BF16)
    want2 = call(q2, k2, v2)
    for a, b in zip((q, k, v), (q2, k2, v2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want2))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = [call(stream=s) for s in (s1, s2, s1, s2)]
    fine()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(r, want2))


def test_decode_captured():
    """A replayed decode step reads the slots and tokens of its buffers as they are at the replay."""
    N, H, dk, dv = 5, 2, 128, 64
    g, ld = gen(31), torch.tensor([-0.05, -1.0], device="cuda")
    q, k, v = (randn(g, N, H, d, dtype=BF16) for d in (dk, dk, dv))
    slots = torch.tensor([4, 0, -1, 6, 2], device="cuda", dtype=torch.int32)
    start = randn(g, 7, H, dk, dv)
    state, o = start.clone(), torch.empty(N, H, dv, device="cuda", dtype=BF16)
    gdr.linear_decode_step(q, k, v, state, log_decay=ld, state_slots=slots, scale=0.1, out=o)    # before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.linear_decode_step(q, k, v, state, log_decay=ld, state_slots=slots, scale=0.1, out=o)
    for turn, rows in enumerate(([4, 0, -1, 6, 2], [1, 9, 3, 0, -1])):
        for x in (q, k, v):
            x.copy_(randn(g, *x.shape, dtype=BF16))
        slots.copy_(torch.tensor(rows, dtype=torch.int32))
        state.copy_(start)
        want_state = start.clone()
        graph.replay()
        want = gdr.linear_decode_step(q, k, v, want_state, log_decay=ld, state_slots=slots, scale=0.1)
        fine()
        assert torch.equal(o, want) and torch.equal(state, want_state), turn
        assert (o[[i for i, r in enumerate(rows) if not 0 <= r < 7]] == 0).all()


def test_two_graphs_at_once():
    """Two captured calls in segments, replayed on two streams at the same time: each has its own workspace."""
    ld = torch.tensor([-0.01, -0.2], device="cuda")
    inputs, graphs, got, want = [], [], [], []
    for seed in (41, 42):
        q, k, v, g = tensors(seed, 1, 3000, 1, 2, 128, 64, BF16)
        do = randn(g, 1, 3000, 2, 64, dtype=BF16)
        inputs.append((q, k, v, do))      # they live as long as the graphs

        def call():
            o, S = gdr.linear_forward(q, k, v, log_decay=ld)
            x = gdr.linear_backward(q, k, v, do, log_decay=ld, d_final_state=S)
            return [o, S, x["q"], x["k"], x["v"], x["initial_state"]]

        want.append(call())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(call())
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
    fine()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_empty_calls():
    ld = decays(2)
    e = lambda *s, dt=BF16: torch.zeros(*s, device="cuda", dtype=dt)
    S0 = randn(gen(1), 1, 2, 64, 64)
    o, S = gdr.linear_forward(e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2, 64), log_decay=ld, initial_state=S0)
    assert o.shape == (1, 0, 2, 64) and torch.equal(S, S0)
    o, S = gdr.linear_forward(e(0, 5, 2, 64), e(0, 5, 2, 64), e(0, 5, 2, 64), log_decay=ld)
    assert S.shape == (0, 2, 64, 64)
    x = gdr.linear_backward(e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2, 64), log_decay=ld, d_final_state=S0)
    assert torch.equal(x["initial_state"], S0)
    x = gdr.linear_backward(e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2, 64), log_decay=ld)
    assert (x["initial_state"] == 0).all()
    assert gdr.linear_decode_step(e(0, 2, 64), e(0, 2, 64), e(0, 2, 64), e(3, 2, 64, 64, dt=F32), log_decay=ld,
                                  state_slots=e(0, dt=torch.int32)).shape == (0, 2, 64)
    fine()


def test_backward_without_value_heads():
    for shape, cu in (((2, 5), None), ((1, 5), torch.tensor([0, 4], dtype=torch.int32, device="cuda"))):
        q = randn(gen(2), *shape, 2, 64, dtype=BF16)
        v = torch.empty(*shape, 0, 64, dtype=BF16, device="cuda")
        torch.full((64, 64), 7.0, device="cuda")                   # freed: what a fresh tensor may hold
        x = gdr.linear_backward(q, q, v, v, log_decay=decays(0), cu_seqlens=cu)
        assert (x["q"] == 0).all() and (x["k"] == 0).all() and x["v"].shape == v.shape
        assert x["q"].shape == q.shape and x["initial_state"].numel() == 0
    fine()


# (the plan takes 2, 3, 4 and, from the fourth on, many segments on 148 SMs)
@pytest.mark.parametrize("dtype,T,Hk,H,dk,dv", [(BF16, 2048, 25, 50, 64, 64), (BF16, 1150, 24, 48, 64, 64),
                                               (BF16, 1400, 18, 36, 64, 64),
                                               (BF16, 901, 1, 2, 128, 128), (BF16, 705, 2, 4, 64, 128),
                                               (BF16, 1700, 1, 3, 128, 64), (F32, 901, 1, 2, 128, 128)])
def test_segments(dtype, T, Hk, H, dk, dv):
    """Segments chained by themselves and by the kernel between: decays that forget and that do not, shared heads,
    states both ways, the end state in the place of the start state."""
    q, k, v, g = tensors(T + 3, 1, T, Hk, H, dk, dv, dtype)
    S0 = randn(g, 1, H, dk, dv)
    ld = decays(H, T)
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, scale=0.1)
    state = S0.clone()
    o2, S2 = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=state, final_state=state, scale=0.1)
    o3, none = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, output_final_state=False, scale=0.1)
    fine()
    assert none is None and torch.equal(o, o3) and S2.data_ptr() == state.data_ptr()
    ref.check_forward(q[0], k[0], v[0], ld, S0[0], 0.1, o[0], S[0])
    ref.check_forward(q[0], k[0], v[0], ld, S0[0], 0.1, o2[0], S2[0], "in place")


@pytest.mark.parametrize("dtype,T,Hk,H,dk,dv,state", [(BF16, 2048, 6, 18, 64, 64, True), (BF16, 1150, 16, 16, 64, 64, True),
                                                     (BF16, 1400, 6, 12, 64, 64, True), (BF16, 901, 1, 2, 128, 64, True),
                                                     (F32, 1500, 2, 16, 64, 64, True),
                                                     (BF16, 1100, 3, 3, 64, 128, False), (F32, 500, 1, 2, 64, 128, True)])
def test_backward_segments(dtype, T, Hk, H, dk, dv, state):
    q, k, v, g = tensors(T + 4, 1, T, Hk, H, dk, dv, dtype)
    do = randn(g, 1, T, H, dv, dtype=dtype)
    S0, dS = (randn(g, 1, H, dk, dv), randn(g, 1, H, dk, dv)) if state else (None, None)
    ld = decays(H, T)
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, scale=0.3)
    fine()
    ref.check_grads(q[0], k[0], v[0], do[0], ld, S0[0] if state else None, dS[0] if state else None, 0.3,
                    (x["q"][0], x["k"][0], x["v"][0], x["initial_state"][0]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_short_sequences(dtype):
    N, H, d = 2000, 1, 64
    rng = random.Random(1)
    lens = [rng.choice([0, 0, 1, 1, 2, 3]) for _ in range(N)]
    T = sum(lens)
    q, k, v, g = tensors(31, 1, T, H, H, d, d, dtype)
    S0 = randn(g, N, H, d, d)
    ld = torch.tensor([-0.3], device="cuda")
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, cu_seqlens=cu)
    fine()
    q, k, v, S0, o, S = (x.cpu() for x in (q, k, v, S0, o, S))
    t = 0
    for n, L in enumerate(lens):
        s = slice(t, t + L)
        ref.check_forward(q[0, s], k[0, s], v[0, s], ld, S0[n], 1.0, o[0, s], S[n], f"sequence {n}")
        t += L


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_beyond_32_bits(dtype):
    """Tokens 2^27 elements apart: the last ones start past element 2^32 of their buffer."""
    T, d, far = 34, 64, 1 << 27
    flat = torch.empty((T - 1) * far + d, device="cuda", dtype=dtype)
    wide = flat.as_strided((1, T, 1, d), (d, far, d, 1))
    q, k, v, _ = tensors(41, 1, T, 1, 1, d, d, dtype)
    ld = torch.tensor([-0.1], device="cuda")
    want = gdr.linear_forward(q, k, v, log_decay=ld)
    grads = gdr.linear_backward(q, k, v, v, log_decay=ld)
    wide.copy_(v)
    got = gdr.linear_forward(q, k, wide, log_decay=ld)
    back = gdr.linear_backward(q, k, wide, wide, log_decay=ld)
    fine()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(back[n], grads[n]) for n in grads)


def test_pool_beyond_32_bits():
    """A pool of more than 2^31 elements: the pages behind that."""
    H, d, pages = 2, 128, 66000
    pool = torch.empty(pages, H, d, d, device="cuda")
    last = [pages - 1, pages - 2, 65536, 0]
    start = randn(gen(42), 4, H, d, d)
    gdr.copy_states(pool, [-1] * 4, last)
    for p, s in zip(last, start):
        pool[p] = s
    small = start.clone()
    g = gen(43)
    slots = torch.tensor(last, device="cuda", dtype=torch.int32)
    ld = torch.tensor([-0.1, -0.01], device="cuda")
    q, k, v = (randn(g, 4, H, d, dtype=BF16) for _ in range(3))
    a = gdr.linear_decode_step(q, k, v, pool, log_decay=ld, state_slots=slots)
    b = gdr.linear_decode_step(q, k, v, small, log_decay=ld)
    assert torch.equal(a, b)
    q, k, v = (randn(g, 1, 100, H, d, dtype=BF16) for _ in range(3))
    cu = torch.tensor([0, 10, 40, 90, 100], device="cuda", dtype=torch.int32)
    a = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=pool, final_state=pool, cu_seqlens=cu, state_slots=slots)
    b = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=small, final_state=small, cu_seqlens=cu)
    assert torch.equal(a[0], b[0]) and all(torch.equal(pool[p], s) for p, s in zip(last, small))
    gdr.copy_states(pool, last[:2], [7, pages - 3])
    fine()
    assert torch.equal(pool[7], small[0]) and torch.equal(pool[pages - 3], small[1])


def test_padding_rows_with_any_contents():
    """A decode row without a page may hold anything, and equal padding slots are fine."""
    q, k, v = (torch.full((3, 2, 64), float("nan"), device="cuda", dtype=BF16) for _ in range(3))
    g = gen(44)
    for x in (q, k, v):
        x[1] = randn(g, 2, 64, dtype=BF16)
    pool = randn(g, 2, 2, 64, 64)
    before, one = pool.clone(), pool[1:].clone()
    ld = torch.tensor([-0.1, 0.0], device="cuda")
    o = gdr.linear_decode_step(q, k, v, pool, log_decay=ld,
                               state_slots=torch.tensor([-1, 1, -1], device="cuda", dtype=torch.int32))
    o1 = gdr.linear_decode_step(q[1:2].contiguous(), k[1:2].contiguous(), v[1:2].contiguous(), one, log_decay=ld)
    fine()
    assert (o[0] == 0).all() and (o[2] == 0).all() and torch.equal(o[1:2], o1)
    assert torch.equal(pool[0], before[0]) and torch.equal(pool[1:], one)


# (256 tokens a segment: up to six of them in a sequence, at most 10 and 12 in a batch of 12 sequences)
@pytest.mark.parametrize("Hk,H,dk,dv,state", [(1, 2, 128, 64, True), (1, 1, 64, 128, True), (2, 2, 64, 64, False),
                                              (1, 1, 128, 128, True)])
@pytest.mark.parametrize("lens", [[3, 1500, 0, 1, 70, 256, 0, 64, 2, 130, 513, 9], [0] * 11 + [1281], [1024, 1025] + [40] * 10,
                                  [3, 700, 130], [513]])
def test_packed_long_among_short(Hk, H, dk, dv, state, lens):
    N, T = len(lens), sum(lens) + 5
    q, k, v, g = tensors(61, 1, T, Hk, H, dk, dv, BF16)
    pages, ld = N + 2, torch.tensor([-0.004, -0.5], device="cuda")[:H].contiguous()
    slots = torch.randperm(pages, generator=g, device="cuda")[:N].to(torch.int32)
    S0 = randn(g, pages, H, dk, dv) if state else None
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    S, place = torch.full((pages, H, dk, dv), 7.0, device="cuda"), torch.zeros(pages, H, dk, dv, device="cuda")
    if state:
        place.copy_(S0)
    o, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, final_state=S, state_slots=slots, cu_seqlens=cu)
    none, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, state_slots=slots if state else None, cu_seqlens=cu,
                                 output_final_state=False)
    there, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=place, final_state=place, state_slots=slots,
                                  cu_seqlens=cu)
    # the longest sequence without a page: zeros at its start, and no state of it kept
    longest = lens.index(max(lens))
    outside, pool = slots.clone(), randn(g, pages, H, dk, dv)
    outside[longest] = pages
    before = pool.clone()
    lost, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=pool, final_state=pool, state_slots=outside,
                                 cu_seqlens=cu)
    fine()
    assert torch.equal(pool[slots[longest]], before[slots[longest]])
    s = slice(sum(lens[:longest]), sum(lens[:longest + 1]))
    ref.check_forward(q[0, s], k[0, s], v[0, s], ld, None, 1.0, lost[0, s], None, "without a page")
    assert (S[[p for p in range(pages) if p not in slots.tolist()]] == 7).all()
    at = slots.tolist()
    assert torch.equal(o, there) and torch.equal(S[at], place[at])
    for n, p in enumerate(at):
        s = slice(sum(lens[:n]), sum(lens[:n + 1]))
        ref.check_forward(q[0, s], k[0, s], v[0, s], ld, S0[p] if state else None, 1.0, o[0, s], S[p], f"sequence {n}")
        # (a state that is not kept takes two bf16 terms of w c instead of three: other bits, the same bound)
        ref.check_forward(q[0, s], k[0, s], v[0, s], ld, S0[p] if state else None, 1.0, none[0, s], None, f"no state {n}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hk,H,dk,dv", [(2, 2, 128, 64), (1, 3, 64, 128), (1, 1, 64, 64)])
@pytest.mark.parametrize("T,lens", [(400, [70, 0, 130]), (400, [0, 0]), (2500, [1400, 3, 0]), (700, [1]), (90, [64, 26])])
def test_rows_of_no_sequence(dtype, Hk, H, dk, dv, T, lens):
    """They are zeros in fresh outputs, whatever the memory held, and left as they were in a given one."""
    q, k, v, g = tensors(51, 1, T, Hk, H, dk, dv, dtype)
    do, ld = randn(g, 1, T, H, dv, dtype=dtype), decays(H)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    used = sum(lens)
    for x in (q, k, v, do):
        x[:, used:] = float("nan")
    held = [torch.full((T * H * d * 4,), float("nan"), device="cuda") for d in (64, 128, 64, 128)]
    del held                                           # what the fresh outputs are made of
    o, S = gdr.linear_forward(q, k, v, log_decay=ld, cu_seqlens=cu)
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, cu_seqlens=cu, d_final_state=torch.ones_like(S))
    given = torch.full_like(v, 5.0)
    gdr.linear_forward(q, k, v, log_decay=ld, cu_seqlens=cu, out=given)
    fine()
    assert torch.equal(given[:, :used], o[:, :used]) and (given[:, used:] == 5).all()
    for name, y in (("o", o), ("q", x["q"]), ("k", x["k"]), ("v", x["v"])):
        assert (y[:, used:] == 0).all() and torch.isfinite(y).all(), name
    for n, L in enumerate(lens):
        s = slice(sum(lens[:n]), sum(lens[:n]) + L)
        if L <= 130:
            ref.check_forward(q[0, s], k[0, s], v[0, s], ld, None, 1.0, o[0, s], S[n], f"sequence {n}")
            ref.check_grads(q[0, s], k[0, s], v[0, s], do[0, s], ld, None, torch.ones_like(S[n]), 1.0,
                            [x["q"][0, s], x["k"][0, s], x["v"][0, s], x["initial_state"][n]], f"sequence {n}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_changing_decays_and_offsets(dtype):
    """Decays, offsets and slots overwritten on the stream between two calls are the second call's."""
    lens = [[300, 1, 600], [2, 800, 99]]
    H, d = 2, 128
    g = gen(51)
    q, k, v, do = (randn(g, 1, 901, H, d, dtype=dtype) for _ in range(4))
    lds = [torch.tensor([-0.1, -1.0], device="cuda"), torch.tensor([-2.0, -0.01], device="cuda")]
    cus = [torch.tensor([0] + x, device="cuda").cumsum(0).to(torch.int32) for x in lens]
    slots = [torch.tensor(x, device="cuda", dtype=torch.int32) for x in ([2, 0, 1], [0, 1, 2])]
    start = randn(g, 3, H, d, d)

    def call(ld, cu, slot):
        pool = start.clone()
        o, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=pool, final_state=pool, cu_seqlens=cu,
                                  state_slots=slot)
        x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=start, cu_seqlens=cu)
        dense = gdr.linear_forward(q, k, v, log_decay=ld)
        return [o, pool, *dense, *x.values()]

    want = [call(lds[i], cus[i], slots[i]) for i in range(2)]
    torch.cuda.synchronize()
    args = [lds[0].clone(), cus[0].clone(), slots[0].clone()]
    got = []
    for i in (0, 1, 0):
        for a, b in zip(args, (lds[i], cus[i], slots[i])):
            a.copy_(b)
        got.append((i, call(*args)))
    fine()
    for i, x in got:
        assert all(torch.equal(a, b) for a, b in zip(x, want[i]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_empty_sequences_of_narrow_values(dtype):
    """Batches of nothing but empty sequences, each ending at once, right before one that computes."""
    N, H, dk, dv = 700, 2, 128, 64
    q, k, v, g = tensors(71, 1, 130, H, H, dk, dv, dtype)
    S0, ld = randn(g, N, H, dk, dv), torch.tensor([-0.1, -0.01], device="cuda")
    nothing = torch.zeros(N + 1, device="cuda", dtype=torch.int32)
    dense = [gdr.linear_forward(q, k, v, log_decay=ld) for _ in range(2)]
    for _ in range(5):
        o, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, cu_seqlens=nothing)
        dense.append(gdr.linear_forward(q, k, v, log_decay=ld))
        x = gdr.linear_backward(q, k, v, v, log_decay=ld, d_final_state=S0, cu_seqlens=nothing)
        assert torch.equal(S, S0) and (o == 0).all() and torch.equal(x["initial_state"], S0)
        assert all((x[n] == 0).all() for n in "qkv")
    fine()
    assert all(torch.equal(a, b) for d in dense for a, b in zip(d, dense[0]))
    ref.check_forward(q[0], k[0], v[0], ld, None, 1.0, dense[-1][0][0], dense[-1][1][0])


@pytest.mark.parametrize("dtype,Hk,H,dk,dv,lens", [(BF16, 2, 2, 128, 64, [1500]), (BF16, 1, 3, 64, 128, [900, 0, 1, 411]),
                                                   (BF16, 1, 2, 128, 128, [1100]), (BF16, 1, 2, 64, 64, [40, 1000, 3]),
                                                   (F32, 1, 2, 64, 128, [700]), (F32, 2, 2, 128, 64, [30, 600, 0, 5])])
def test_backward_in_segments_again_and_again(dtype, Hk, H, dk, dv, lens):
    """Runs of different shapes and output types in one call, every call's segment states in memory that held NaN
    before: the same bits each time."""
    T, N = sum(lens), len(lens)
    q, k, v, g = tensors(81, 1, T, Hk, H, dk, dv, dtype)
    do, S0, dS = randn(g, 1, T, H, dv, dtype=dtype), randn(g, N, H, dk, dv), randn(g, N, H, dk, dv)
    ld = decays(H)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32) if N > 1 else None
    want = None
    for _ in range(20):
        held = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 18, 1 << 20, 1 << 22, 1 << 22)]
        del held
        x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, cu_seqlens=cu, scale=0.3)
        want = want or x
        assert all(torch.equal(x[n], want[n]) for n in x)
    fine()
    t = 0
    for n, L in enumerate(lens):
        s, t = slice(t, t + L), t + L
        ref.check_grads(q[0, s], k[0, s], v[0, s], do[0, s], ld, S0[n], dS[n], 0.3,
                        (want["q"][0, s], want["k"][0, s], want["v"][0, s], want["initial_state"][n]), f"sequence {n}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_captured(dtype):
    """A replayed prefill into a pool and a replayed packed backward take the offsets, slots, decays and tokens that
    their buffers hold at the replay: other lengths, empty sequences and rows of no sequence among them."""
    T, N, Hk, H, dk, dv, pages = 1600, 3, 1, 2, 128, 64, 5
    g = gen(91)
    q, k = (randn(g, 1, T, Hk, dk, dtype=dtype) for _ in range(2))
    v, do = (randn(g, 1, T, H, dv, dtype=dtype) for _ in range(2))
    ld = torch.empty(H, device="cuda")
    cu, slots = torch.empty(N + 1, device="cuda", dtype=torch.int32), torch.empty(N, device="cuda", dtype=torch.int32)
    start, S0 = randn(g, pages, H, dk, dv), randn(g, N, H, dk, dv)
    pool = start.clone()

    def call(pool):
        o, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=pool, final_state=pool, cu_seqlens=cu,
                                  state_slots=slots, scale=0.1)
        x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, cu_seqlens=cu, scale=0.1)
        return [o, *x.values()]

    def fill(lens, rows, decay):
        cu.copy_(torch.tensor([0] + lens).cumsum(0))
        slots.copy_(torch.tensor(rows))
        ld.copy_(torch.tensor(decay))
        pool.copy_(start)

    fill([1600, 0, 0], [0, 1, 2], [-0.1, -0.1])
    call(pool)                                            # before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(pool)
    for lens, rows, decay in (([3, 1500, 7], [2, 0, 4], [-0.01, 0.0]), ([0, 0, 0], [1, 2, 3], [-0.3, -2.0]),
                              ([700, 0, 800], [4, -1, 9], [-1e-3, float("-inf")])):
        fill(lens, rows, decay)
        graph.replay()
        mine = start.clone()
        want = call(mine)
        fine()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(pool, mine), lens
        assert all((x[:, sum(lens):] == 0).all() for x in got[:4])
