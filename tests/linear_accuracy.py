"""What the linear attention's kernels may lose, counted from what they round,
and an emulation of their arithmetic in which single mistakes can be made.

A run (forward or reverse, of one head) computes, over tensors a, b [T,da] and
c [T,dc] with lambda = exp(log_decay),
    forward:  S <- lambda S + bscale b c^T,  y = yscale S^T a
    reverse:  S <- S + bscale b c^T,         y = yscale S^T a,   S <- lambda S
in blocks of 64 tokens counted from the sequence's start (bf16) or token by
token (fp32).

States, as a relative RMS per head.  An update of the state rounds once, by at
most 2^-24 of it, and updates further back than the state's memory are
forgotten, so that M = min(updates, 1 / (2 (1 - decay))) of them, independent,
give sqrt(M) 0.41 2^-24 (2^-24 / sqrt(3), times 0.72 for values spread over a binade); half of 2^-24 is taken.  A block's sum goes
through 12 accumulations of the tensor cores (four steps of 16 tokens, three terms of the
weighted values), which may drop up to 2^-23 of the sum each: half of it on average,
12 2^-24 = 0.75 2^-20 altogether.  So
    limit = 2^-20 + 0.5 sqrt(M) 2^-24        (bf16, an update a block)
    limit = 2 (2 + sqrt(M)) 2^-24            (fp32 and decode, an update a token; three roundings each)
Two bf16 terms in place of three lose 2.6e-6 of each weighted value; one fp32 value of
lambda (of lambda^64, or of the power that a segment's state is chained with) up to 2^-25 an update, all the same way.

Outputs (bf16), element by element.  P with its decays and the state operand are
rounded to bf16 (2^-8 of each value, on disjoint parts of the sum), everything else in
fp32 (2^-15 of the absolute sum for all of it: 64 + 128 + 64 roundings of 2^-23), then the output:
    |err| <= e + 2^-8 (|y| + e),   e = (2^-8 + 2^-15) yscale (sum_s |P_ts| |c_s| + Gamma_t sum_i |S_i| |a_ti|).
As a relative RMS: a rounding to bf16 is 1.63e-3 (2^-8 / sqrt(3), times 0.72 for values spread over a
binade), the two inner ones together weigh as much as the output's own, so 2.3e-3; the limit is 3.5e-3.
"""
import math

import torch

C = 64
OUT_RMS = 3.5e-3


def fp32(log_decay):
    return torch.as_tensor(log_decay).to(torch.float32).item()


def state_limit(updates, decay, dtype):
    memory = min(float(updates), 0.5 / (1.0 - decay)) if decay < 1.0 else float(updates)
    if dtype == torch.bfloat16:
        return 2.0 ** -20 + 0.5 * math.sqrt(memory) * 2.0 ** -24
    return 2.0 * (2.0 + math.sqrt(memory)) * 2.0 ** -24


def rms_error(got, ref):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), "not finite"
    return ((got - ref).pow(2).mean().sqrt() / ref.pow(2).mean().sqrt()).item()


def check_state(got, ref, T, log_decay, dtype, what):
    """One head's state against the 64-bit one; updates are blocks (bf16) or tokens."""
    step = C if dtype == torch.bfloat16 else 1
    limit = state_limit(-(-T // step), math.exp(fp32(log_decay) * step), dtype)
    err = rms_error(got, ref)
    assert err <= limit, f"{what}: relative RMS {err:.2e} over {limit:.2e}"


def blocks(T, reverse):
    at = [(t, min(T, t + C)) for t in range(0, T, C)]
    return at[::-1] if reverse else at


def exact_run(a, b, c, log_decay, S0=None, reverse=False, bscale=1.0, yscale=1.0):
    """64 bits: y [T,dc], the state left, and the bound of y's error (bf16)."""
    a, b, c = a.double().cpu(), b.double().cpu(), c.double().cpu()
    T, ld = a.shape[0], fp32(log_decay)
    S = torch.zeros(a.shape[1], c.shape[1], dtype=torch.float64) if S0 is None else S0.double().cpu()
    y, bound = torch.zeros(T, c.shape[1], dtype=torch.float64), torch.zeros(T, c.shape[1], dtype=torch.float64)
    power = lambda n: torch.where(n > 0, torch.exp(ld * n.clamp(min=1).double()), (n == 0).double())
    for t0, t1 in blocks(T, reverse):
        n, at = t1 - t0, torch.arange(t1 - t0)
        gap = at[None, :] - at[:, None] if reverse else at[:, None] - at[None, :]      # [t, s]
        D = torch.where(gap >= 0, power(gap.clamp(min=0)), 0.0)
        gamma, w = (power(n - 1 - at), power(at + 1)) if reverse else (power(at + 1), power(n - 1 - at))
        x, z, u = a[t0:t1], bscale * b[t0:t1], c[t0:t1]
        P = (x @ z.T) * D
        y[t0:t1] = yscale * (P @ u + gamma[:, None] * (x @ S))
        e = (2.0 ** -8 + 2.0 ** -15) * abs(yscale) * (P.abs() @ u.abs() + gamma[:, None] * (x.abs() @ S.abs()))
        bound[t0:t1] = e + 2.0 ** -8 * (y[t0:t1].abs() + e)
        S = power(torch.tensor(n)) * S + z.T @ (w[:, None] * u)
    return y, S, bound


def check_output(got, y, bound, what, rms=OUT_RMS):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    over = ((got - y).abs() / bound.clamp(min=1e-300)).max().item() if got.numel() else 0.0
    assert over <= 1.0, f"{what}: an element {over:.2f} times its bound off"
    if rms is not None:
        err = rms_error(got, y)
        assert err <= rms, f"{what}: relative RMS {err:.2e} over {rms:.2e}"


class Alternating:
    """A decay in 64 bits as one of the two fp32 values beside it, update by update (or always the nearest)."""

    def __init__(self, value, fixed=False):
        self.near = torch.tensor(value, dtype=torch.float64).float()
        off = value - self.near.double().item()
        self.other = self.near if off == 0 or fixed else torch.nextafter(
            self.near, torch.tensor(math.inf if off > 0 else -math.inf))
        step = self.other.double().item() - self.near.double().item()
        self.share, self.owed = (off / step if step else 0.0), 0.0

    def next(self):
        self.owed += self.share
        if self.owed > 0.5:
            self.owed -= 1.0
            return self.other
        return self.near


def emulated_run(a, b, c, log_decay, S0=None, reverse=False, bscale=1.0, yscale=1.0, terms=3, fixed=False,
                 start=1.0):
    """The block form in fp32 and bf16 as the kernels compute it: y in bf16 and the state.  Mistakes: fewer
    `terms` of the weighted values, a `fixed` decay, a carried state `start` times what it is in the outputs."""
    a, b, c = a.float(), b.float(), c.float()
    T, ld = a.shape[0], fp32(log_decay)
    half = lambda x: x.to(torch.bfloat16).float()
    pw = torch.tensor([math.exp(ld * m) if m else 1.0 for m in range(C + 1)], dtype=torch.float64).float()
    S = torch.zeros(a.shape[1], c.shape[1]) if S0 is None else S0.float().clone()
    y = torch.zeros(T, c.shape[1])
    decay = Alternating(math.exp(ld * C), fixed)
    for t0, t1 in blocks(T, reverse):
        n, at = t1 - t0, torch.arange(t1 - t0)
        gap = at[None, :] - at[:, None] if reverse else at[:, None] - at[None, :]
        D = torch.where(gap >= 0, pw[gap.clamp(min=0)], torch.tensor(0.0))
        gamma, w = (pw[n - 1 - at], pw[at + 1]) if reverse else (pw[at + 1], pw[n - 1 - at])
        x, z, u = a[t0:t1], b[t0:t1], c[t0:t1]
        P = half((x @ z.T) * (bscale * yscale * D))
        y[t0:t1] = yscale * gamma[:, None] * (x @ half(start * S)) + P @ u
        rest = (bscale * w)[:, None] * u
        dS = torch.zeros_like(S)
        for _ in range(terms):
            term = half(rest)
            dS, rest = dS + z.T @ term, rest - term
        S = (decay.next() if n == C else pw[n]) * S + dS
    return y.to(torch.bfloat16), S


def emulated_chain(b, c, log_decay, seg, parts=2):
    """The state after T tokens as the chain of its segments' states, which are right, with the power of lambda that
    joins them in `parts` fp32 values."""
    x = math.exp(fp32(log_decay) * seg)
    hi = torch.tensor(x, dtype=torch.float64).float()
    lo = torch.tensor((x - hi.double().item()) if parts == 2 else 0.0).float()
    fma = lambda f, s, y: (f.double() * s.double() + y.double()).float()
    S = torch.zeros(b.shape[1], c.shape[1])
    for t in range(0, b.shape[0], seg):
        X = decode_states(b[t:t + seg], c[t:t + seg], log_decay, torch.zeros_like(S)).float()
        S = fma(hi, S, fma(lo, S, X))
    return S


def decode_states(k, v, log_decay, S0):
    """The state after the tokens k [T,dk], v [T,dv] of one head, in 64 bits."""
    k, v, T, ld = k.double().cpu(), v.double().cpu(), k.shape[0], fp32(log_decay)
    left = torch.arange(T - 1, -1, -1, dtype=torch.float64)
    w = torch.where(left > 0, torch.exp(ld * left.clamp(min=1.0)), 1.0)
    return math.exp(ld * T) * S0.double().cpu() + k.T @ (w[:, None] * v)


def worst_decay(near, step, tries=400):
    """A log decay close to `near` (fp32) whose lambda^step lies about half way between two fp32 values."""
    best, at = 0.0, near
    for i in range(tries):
        ld = torch.tensor(near * (1 + 1e-3 * i), dtype=torch.float32).item()
        x = math.exp(ld * step)
        f = torch.tensor(x, dtype=torch.float64).float().double().item()
        if abs(f - x) > best:
            best, at = abs(f - x), ld
    return at
