"""64-bit reference of the linear attention with a decay per head, token by
token from the recurrence, and the error bounds of its kernels.

Bounds.  Every output is a sum of products of the inputs; let `abs` be the same
sum over the absolute values.  A kernel that computes in fp32 takes at most
n = T + dk + dv + 16 roundings along any chain of operations (T state updates,
one dot product over dk or dv, a few scalings), each at most 2^-23 relative (a
tensor-core accumulator may truncate), so
    |err| <= n 2^-23 abs.
The bf16 kernels round, besides, the attention products and the state once to
bf16 before the product that makes an output (at most half a step, 2^-8 each, on
disjoint parts of the sum: tokens of the own block, and the state), and the
output itself:
    |err| <= (2^-8 + n 2^-23) abs + 2^-8 (|ref| + that).
The states are fp32 in both cases.
"""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def lam(log_decay):
    return torch.exp(log_decay.double()).cpu()[:, None, None]


def run(q, k, v, log_decay, S0=None, scale=1.0):
    """One sequence: q, k [T,Hk,dk], v [T,H,dv] -> o [T,H,dv], S [H,dk,dv], all fp64 on the CPU."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    T, H, dv = v.shape
    G = H // q.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    S = torch.zeros(H, q.shape[2], dv, dtype=torch.float64) if S0 is None else S0.double().cpu().clone()
    L = lam(log_decay)
    o = torch.zeros(T, H, dv, dtype=torch.float64)
    for t in range(T):
        S = L * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * torch.einsum("hij,hi->hj", S, q[t])
    return o, S


def grads(q, k, v, do, log_decay, S0=None, dS=None, scale=1.0):
    """One sequence's gradients: dq, dk [T,Hk,dk], dv [T,H,dv], dS0 [H,dk,dv]."""
    q, k, v, do = (x.double().cpu() for x in (q, k, v, do))
    T, H, dv = v.shape
    Hk = q.shape[1]
    G = H // Hk
    qh, kh = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    zero = torch.zeros(H, q.shape[2], dv, dtype=torch.float64)
    S = zero if S0 is None else S0.double().cpu()
    L = lam(log_decay)
    gq, gk, gv = torch.zeros_like(qh), torch.zeros_like(kh), torch.zeros_like(v)
    for t in range(T):
        S = L * S + kh[t][:, :, None] * v[t][:, None, :]
        gq[t] = scale * torch.einsum("hij,hj->hi", S, do[t])
    X = zero if dS is None else dS.double().cpu()
    for t in reversed(range(T)):
        X = X + scale * qh[t][:, :, None] * do[t][:, None, :]
        gv[t] = torch.einsum("hij,hi->hj", X, kh[t])
        gk[t] = torch.einsum("hij,hj->hi", X, v[t])
        X = L * X
    dk = q.shape[2]
    return gq.view(T, Hk, G, dk).sum(2), gk.view(T, Hk, G, dk).sum(2), gv, X


def _abs(*xs):
    return [None if x is None else x.abs() for x in xs]


def fp32_bound(abs_sum, T, d):
    return (T + d + 16) * 2.0 ** -23 * abs_sum


def out_bound(abs_sum, ref, T, d, dtype, shared=1):
    """Bound of an output in the I/O type (`shared`: value heads summed into it, one more rounding each)."""
    e = fp32_bound(abs_sum, T + shared, d)
    if dtype == torch.bfloat16:
        e = e + 2.0 ** -8 * abs_sum
    return e + HALF[dtype] * (ref.abs() + e)


def check(got, ref, bound, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} for {tuple(ref.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    worst = over.argmax() if over.numel() else None
    assert over.numel() == 0 or over.max() <= 0, (
        f"{what}: |err| {(got - ref).abs().flatten()[worst]:.3e} over its bound {bound.flatten()[worst]:.3e} "
        f"(value {ref.flatten()[worst]:.3e})")


def check_forward(q, k, v, log_decay, S0, scale, o, S, what=""):
    """One sequence of linear_forward: o [T,H,dv] and S [H,dk,dv] or None."""
    T, d = q.shape[0], q.shape[2]
    ref_o, ref_S = run(q, k, v, log_decay, S0, scale)
    a_o, a_S = run(*_abs(q, k, v), log_decay, *_abs(S0), abs(scale))
    check(o, ref_o, out_bound(a_o, ref_o, T, d, q.dtype), what + " o")
    if S is not None:
        check(S, ref_S, fp32_bound(a_S, T, d), what + " state")


def check_grads(q, k, v, do, log_decay, S0, dS, scale, g, what=""):
    """One sequence of linear_backward: g = (dq, dk, dv, dS0)."""
    T, d = q.shape[0], max(q.shape[2], v.shape[2])
    shared = v.shape[1] // q.shape[1]
    ref = grads(q, k, v, do, log_decay, S0, dS, scale)
    ab = grads(*_abs(q, k, v, do), log_decay, *_abs(S0, dS), abs(scale))
    for name, x, r, a in zip(("q", "k", "v"), g, ref, ab):
        check(x, r, out_bound(a, r, T, d, q.dtype, shared), f"{what} d{name}")
    if g[3] is not None:
        check(g[3], ref[3], fp32_bound(ab[3], T, d), what + " d_initial_state")
