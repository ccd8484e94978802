"""Measured cases of the decayed linear attention and its state cache.

The operators: the forward over whole prompts (dense batches and packed ragged
ones), the single-token decode step on a pool of states, the backward, and the
page copies of the pool.  With ``own`` false ``run`` computes them from
elementary torch operations in 32 bits; with ``own`` true it makes the
framework's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # forward ------------------------------------------------------------------------------------------------
        # one short chat turn of one user on a small layer: latency
        dict(name="forward_short", op="forward", B=1, T=77, H=4, Hk=4, dk=64, dv=64, dtype="bf16", state=True),
        # a training or scoring batch of the 350M layer
        dict(name="forward_350m", op="forward", B=8, T=2048, H=8, Hk=8, dk=128, dv=128, dtype="bf16", state=False),
        # one long document on the 1.3B layer's heads
        dict(name="forward_64k", op="forward", B=1, T=65536, H=16, Hk=16, dk=128, dv=128, dtype="bf16", state=False),
        # a serving step that prefills ragged prompts in one packed batch, key heads shared by two value heads,
        # continued from earlier states; empty and one-token prompts among them, padding rows at the end
        dict(name="forward_packed", op="forward", B=1, T=9200, H=16, Hk=8, dk=128, dv=64, dtype="bf16", state=True,
             lens="1000,1,0,333,64,2048,7,129,4001,63,640,65,500,200,100,40"),
        # fp32 activations (evaluation)
        dict(name="forward_fp32", op="forward", B=2, T=500, H=4, Hk=4, dk=128, dv=128, dtype="fp32", state=True),
        # decode -------------------------------------------------------------------------------------------------
        # a few users on a small deployment: latency
        dict(name="decode_3x8", op="decode", N=3, pages=8, H=8, Hk=8, dk=128, dv=128, dtype="bf16"),
        # a full serving batch on a larger pool, padded rows among it
        dict(name="decode_256x16", op="decode", N=256, pages=320, H=16, Hk=16, dk=128, dv=128, dtype="bf16"),
        # backward -----------------------------------------------------------------------------------------------
        # a short ragged fine-tuning batch with shared key heads
        dict(name="backward_odd", op="backward", B=3, T=333, H=6, Hk=3, dk=64, dv=128, dtype="bf16", state=True),
        # the 350M layer's training step
        dict(name="backward_350m", op="backward", B=8, T=2048, H=8, Hk=8, dk=128, dv=128, dtype="bf16", state=False),
        # the 1.3B layer's training step
        dict(name="backward_1p3b", op="backward", B=4, T=4096, H=16, Hk=16, dk=128, dv=128, dtype="bf16", state=False),
        # pages --------------------------------------------------------------------------------------------------
        # one prompt's state forked to eight samples, a small model
        dict(name="pages_fork", op="pages", L=4, pages=24, H=8, dk=128, dv=128, kind="fork", n=8),
        # a serving pool compacted after many sequences ended, 24 layers
        dict(name="pages_compact", op="pages", L=24, pages=96, H=16, dk=128, dv=128, kind="compact", n=24),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "decode", "backward", "pages"])
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "pages":
        L, H = _log_int(rng, 1, 24), _log_int(rng, 1, 16)
        n = _log_int(rng, 1, 24)
        return dict(op=op, L=L, pages=4 * n + rng.randint(0, 5), H=H, dk=dk, dv=dv, n=n,
                    kind=rng.choice(["fork", "compact", "clear"]))
    Hk = _log_int(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 1, 2, 4])
    if op == "decode":
        N = _log_int(rng, 1, max(1, 4096 // H))
        return dict(op=op, N=N, pages=N + rng.randint(0, 64), H=H, Hk=Hk, dk=dk, dv=dv,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    most = 262144 if op == "backward" else 1048576       # token-heads of the largest listed cases
    dtype = "bf16"
    if op == "forward" and rng.random() < 0.2:
        dtype, most = "fp32", 16384
    case = dict(op=op, B=1, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, state=rng.random() < 0.5)
    if dtype == "bf16" and rng.random() < 0.4:
        lens, left = [], max(1, min(most // 4 // H, 16384))
        for _ in range(rng.randint(1, 32)):
            x = rng.choice([0, 1]) if rng.random() < 0.15 else _log_int(rng, 1, max(1, left // 3))
            lens.append(min(x, left))
            left -= lens[-1]
        case["lens"] = ",".join(map(str, lens))
        case["T"] = max(1, sum(lens) + rng.randint(0, 9))
    else:
        case["T"] = _log_int(rng, 1, max(1, min(most // H, 2048 if dtype == "fp32" else 65536)))
        case["B"] = _log_int(rng, 1, max(1, min(16, most // (H * case["T"]))))
    return case


def _lens(case):
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    return [case["T"]] * case["B"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    s = {"case": case}
    if case["op"] == "pages":
        s["pool"] = randn(case["L"], case["pages"], case["H"], case["dk"], case["dv"])
        rng = random.Random(int(seed))
        ids = rng.sample(range(case["pages"]), 2 * case["n"])
        if case["kind"] == "compact":          # live pages at the back move into holes at the front
            ids = sorted(ids)
            s["dst"], s["src"] = ids[:case["n"]], ids[case["n"]:]
        elif case["kind"] == "fork":           # one page to all the others
            s["dst"], s["src"] = ids[:case["n"]], [ids[-1]] * case["n"]
        else:                                  # pages of ended sequences cleared
            s["dst"], s["src"] = ids[:case["n"]], [-1] * case["n"]
        return s
    H, Hk, dk, dv, dt = case["H"], case["Hk"], case["dk"], case["dv"], DTYPES[case["dtype"]]
    # decays from nearly none to a few tokens' memory
    s["log_decay"] = -torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(1e4) - math.log(1e4))
    s["scale"] = dk ** -0.5
    if case["op"] == "decode":
        N, P = case["N"], case["pages"]
        s["q"], s["k"], s["v"] = randn(N, Hk, dk, dtype=dt), randn(N, Hk, dk, dtype=dt), randn(N, H, dv, dtype=dt)
        s["state"] = randn(P, H, dk, dv)
        slots = torch.randperm(P, generator=g, device="cuda")[:N].to(torch.int32)
        if N > 16:
            slots[-3:] = -1                    # the padded rows of a batch of fixed size
        s["slots"] = slots
        return s
    B, T = case["B"], case["T"]
    s["q"], s["k"], s["v"] = randn(B, T, Hk, dk, dtype=dt), randn(B, T, Hk, dk, dtype=dt), randn(B, T, H, dv, dtype=dt)
    lens = _lens(case)
    N = len(lens)
    s["s0"] = randn(N, H, dk, dv) if case["state"] else None
    s["lens"], s["cu"] = lens, None
    if "lens" in case:
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    if case["op"] == "backward":
        s["do"] = randn(B, T, H, dv, dtype=dt)
        s["ds"] = randn(N, H, dk, dv) if case["state"] else None
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------
CHUNK = 128


def _pad_index(s, T, device):
    """[N, Tmax] positions of every sequence's tokens among the T rows, and which of them exist."""
    lens = torch.tensor(s["lens"], device=device)
    at = torch.arange(max(1, max(s["lens"])), device=device)
    start = lens.cumsum(0) - lens
    return (start[:, None] + at).clamp(max=max(T - 1, 0)), at < lens[:, None], lens


def _plain_padded(q, k, v, log_decay, s0, lens, scale):
    """q, k [N,T,H,dk], v [N,T,H,dv] fp32 with zeros behind each sequence's end -> o [N,T,H,dv], S [N,H,dk,dv]."""
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    nc = -(-T // CHUNK)
    pad = nc * CHUNK - T

    def chunks(x):
        return torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(N, nc, CHUNK, H, -1).permute(0, 3, 1, 2, 4)

    q, k, v = chunks(q), chunks(k), chunks(v)                     # [N,H,nc,C,d]
    ld = log_decay.double()
    at = torch.arange(CHUNK, device=q.device, dtype=torch.float64)
    gap = at[:, None] - at
    D = torch.where(gap >= 0, torch.exp(ld[:, None, None] * gap.clamp(min=0)), 0.0).float()      # [H,C,C]
    o = ((q @ k.transpose(-1, -2)) * D[:, None]) @ v
    w = torch.exp(ld[:, None] * (CHUNK - 1 - at)).float()                                         # [H,C]
    own_part = (k * w[:, None, :, None]).transpose(-1, -2) @ v                                    # [N,H,nc,dk,dv]
    ci = torch.arange(nc, device=q.device, dtype=torch.float64)
    cgap = ci[:, None] - ci - 1
    M = torch.where(cgap >= 0, torch.exp(ld[:, None, None] * CHUNK * cgap.clamp(min=0)), 0.0).float()   # [H,nc,nc]
    start = (M @ own_part.reshape(N, H, nc, dk * dv)).view(N, H, nc, dk, dv)
    if s0 is not None:
        start = start + torch.exp(ld[:, None] * CHUNK * ci).float()[..., None, None] * s0[:, :, None]
    gamma = torch.exp(ld[:, None] * (at + 1)).float()
    o = scale * (o + (q * gamma[:, None, :, None]) @ start)
    # final state: every token's weight counted from its own sequence's end
    t = torch.arange(nc * CHUNK, device=q.device, dtype=torch.float64)
    left = lens[:, None] - 1 - t                                                                  # [N,T']
    wl = torch.exp(ld[None, :, None] * left.clamp(min=0)[:, None]).float() * (left >= 0)[:, None]  # [N,H,T']
    kf, vf = k.reshape(N, H, nc * CHUNK, dk), v.reshape(N, H, nc * CHUNK, dv)
    S = (kf * wl[..., None]).transpose(-1, -2) @ vf
    if s0 is not None:
        S = S + torch.exp(ld[None, :] * lens[:, None]).float()[..., None, None] * s0
    return o.permute(0, 2, 3, 1, 4).reshape(N, nc * CHUNK, H, dv)[:, :T], S


def _plain_sequences(s, q, k, v, s0):
    """q, k, v as given, in fp32 -> o [B,T,H,dv] (zeros in rows of no sequence), S."""
    H, G = s["case"]["H"], s["case"]["H"] // s["case"]["Hk"]
    q, k = q.repeat_interleave(G, 2), k.repeat_interleave(G, 2)
    B, T = q.shape[:2]
    if s["cu"] is None:
        lens = torch.tensor(s["lens"], device=q.device)
        return _plain_padded(q, k, v, s["log_decay"], s0, lens, s["scale"])
    at, there, lens = _pad_index(s, T, q.device)
    m = there[..., None, None]
    o, S = _plain_padded(q[0][at] * m, k[0][at] * m, v[0][at] * m, s["log_decay"], s0, lens, s["scale"])
    out = torch.zeros(B, T, H, v.shape[-1], device=q.device)
    out[0, at[there]] = o[there]
    return out, S


def _plain_forward(s):
    o, S = _plain_sequences(s, s["q"].float(), s["k"].float(), s["v"].float(), s["s0"])
    return {"o": o.to(s["q"].dtype), "state": S}


def _plain_backward(s):
    x = [s[n].float().requires_grad_() for n in "qkv"]
    s0 = s["s0"].detach().clone() if s["s0"] is not None else torch.zeros(
        len(s["lens"]), s["case"]["H"], s["case"]["dk"], s["case"]["dv"], device=x[0].device)
    s0.requires_grad_()
    o, S = _plain_sequences(s, *x, s0)
    up = [s["do"].float(), torch.zeros_like(S) if s["ds"] is None else s["ds"]]
    dq, dk, dv, d0 = torch.autograd.grad([o, S], x + [s0], up)
    t = s["q"].dtype
    return {"q": dq.to(t), "k": dk.to(t), "v": dv.to(t), "state": d0}


def _plain_decode(s):
    slots = s["slots"].long()
    live = slots >= 0
    G = s["case"]["H"] // s["case"]["Hk"]
    q = s["q"].float().repeat_interleave(G, 1)[live]
    k = s["k"].float().repeat_interleave(G, 1)[live]
    v = s["v"].float()[live]
    at = slots[live]
    S = torch.exp(s["log_decay"])[None, :, None, None] * s["state"][at] + k[..., None] * v[..., None, :]
    s["state"][at] = S
    o = torch.zeros(s["v"].shape, device=v.device)
    o[live] = s["scale"] * (q[..., None] * S).sum(-2)
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_pages(s):
    pool = s["pool"]
    src = torch.tensor(s["src"], device=pool.device)
    dst = torch.tensor(s["dst"], device=pool.device)
    pool[:, dst] = torch.where((src >= 0)[None, :, None, None, None], pool[:, src.clamp(min=0)], 0.0)
    return {"pool": pool}


def run(s):
    op = s["case"]["op"]
    if own:
        import gated_delta_rule_forward_b200 as gdr
        if op == "forward":
            o, S = gdr.linear_forward(s["q"], s["k"], s["v"], log_decay=s["log_decay"], initial_state=s["s0"],
                                      cu_seqlens=s["cu"], scale=s["scale"])
            return {"o": o, "state": S}
        if op == "backward":
            g = gdr.linear_backward(s["q"], s["k"], s["v"], s["do"], log_decay=s["log_decay"], initial_state=s["s0"],
                                    d_final_state=s["ds"], cu_seqlens=s["cu"], scale=s["scale"])
            return {"q": g["q"], "k": g["k"], "v": g["v"], "state": g["initial_state"]}
        if op == "decode":
            o = gdr.linear_decode_step(s["q"], s["k"], s["v"], s["state"], log_decay=s["log_decay"],
                                       state_slots=s["slots"], scale=s["scale"])
            return {"o": o, "state": s["state"]}
        gdr.copy_states(s["pool"], s["src"], s["dst"])
        return {"pool": s["pool"]}
    return {"forward": _plain_forward, "backward": _plain_backward, "decode": _plain_decode,
            "pages": _plain_pages}[op](s)


# ---- what a pass cannot do without --------------------------------------------------------------------------------
def work(case):
    if case["op"] == "pages":
        page = 4.0 * case["L"] * case["H"] * case["dk"] * case["dv"]
        read = {"fork": 1, "compact": case["n"], "clear": 0}[case["kind"]]
        return {"bytes": (read + case["n"]) * page, "flops": 0.0}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    e = 2 if case["dtype"] == "bf16" else 4
    page = 4.0 * H * dk * dv
    if case["op"] == "decode":
        live = case["N"] - (3 if case["N"] > 16 else 0)
        return {"bytes": live * (2 * page + e * (2 * Hk * dk + 2 * H * dv)), "flops": 5.0 * live * H * dk * dv}
    tokens, N = sum(_lens(case)), len(_lens(case))
    io = float(e * tokens)
    if case["op"] == "forward":
        states = N * page * (2 if case["state"] else 1)
        return {"bytes": io * (2 * Hk * dk + 2 * H * dv) + states, "flops": 4.0 * tokens * H * dk * dv}
    states = N * page * (3 if case["state"] else 1)
    return {"bytes": io * (4 * Hk * dk + 3 * H * dv) + states, "flops": 10.0 * tokens * H * dk * dv}


# ---- from the definition, token by token in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        pool = s["pool"].double()
        for a, b in zip(s["src"], s["dst"]):
            pool[:, b] = pool[:, a] if a >= 0 else 0.0
        return {"pool": pool}
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    H, Hk = case["H"], case["Hk"]
    head = torch.arange(H, device="cuda") // (H // Hk)
    if case["op"] == "decode":
        state, o = s["state"].double(), torch.zeros(s["v"].shape, device="cuda", dtype=torch.float64)
        at = s["slots"].long()
        rows = (at >= 0).nonzero()[:, 0]
        for i in range(0, len(rows), 64):
            r = rows[i:i + 64]
            S = lam * state[at[r]] + torch.einsum("nhi,nhj->nhij", s["k"].double()[r][:, head], s["v"].double()[r])
            state[at[r]] = S
            o[r] = s["scale"] * torch.einsum("nhij,nhi->nhj", S, s["q"].double()[r][:, head])
        return {"o": o, "state": state}
    dk, dv, lens = case["dk"], case["dv"], s["lens"]
    N, most = len(lens), max(lens)
    q, k, v = (s[n].double().flatten(0, 1) for n in "qkv")
    if q.shape[0] * H * N > 2 ** 31:
        return None
    length = torch.tensor(lens, device="cuda")
    first = length.cumsum(0) - length
    zeros = torch.zeros(N, H, dk, dv, device="cuda", dtype=torch.float64)
    S0 = zeros if s["s0"] is None else s["s0"].double()

    def step(t):
        if min(lens) == most:                  # every sequence has this token
            return (first + t >= 0)[:, None, None, None], first + t, first + t, slice(None)
        there = length > t
        at = (first + t).clamp(max=q.shape[0] - 1)
        return there[:, None, None, None], at, at[there], there

    if case["op"] == "forward":
        o = torch.zeros(q.shape[0], H, dv, device="cuda", dtype=torch.float64)
        S = S0
        for t in range(most):
            m, at, rows, there = step(t)
            S = torch.where(m, lam * S + k[at][:, head, :, None] * v[at][:, :, None, :], S)
            y = s["scale"] * (q[at][:, head, None, :] @ S)[:, :, 0]
            o[rows] = y[there]
        return {"o": o.view(case["B"], case["T"], H, dv), "state": S}
    do = s["do"].double().flatten(0, 1)
    gq, gk, gv = (torch.zeros_like(x) for x in (q, k, v))
    S = S0
    for t in range(most):
        m, at, rows, there = step(t)
        S = torch.where(m, lam * S + k[at][:, head, :, None] * v[at][:, :, None, :], S)
        y = s["scale"] * (S @ do[at][..., None])[..., 0]
        gq[rows] = y.view(N, Hk, H // Hk, dk).sum(2)[there]
    dS = zeros if s["ds"] is None else s["ds"].double()
    for t in reversed(range(most)):
        m, at, rows, there = step(t)
        dS = torch.where(m, dS + s["scale"] * q[at][:, head, :, None] * do[at][:, :, None, :], dS)
        gv[rows] = (k[at][:, head, None, :] @ dS)[:, :, 0][there]
        gk[rows] = (dS @ v[at][..., None])[..., 0].view(N, Hk, H // Hk, dk).sum(2)[there]
        dS = torch.where(m, lam * dS, dS)
    return {"q": gq.view(s["q"].shape), "k": gk.view(s["k"].shape), "v": gv.view(s["v"].shape), "state": dS}
