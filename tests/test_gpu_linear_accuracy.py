"""Linear attention with a decay per head, on the GPU: what its kernels may lose of the 64-bit recurrence
(tests/linear_accuracy.py has the limits and says what they tell apart)."""
import math

import pytest
import torch

import gated_delta_rule_forward_b200 as gdr
from gated_delta_rule_forward_b200 import _lib
import linear_accuracy as acc

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
C = acc.C


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, positive=False):
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x.abs() if positive else x).to(dtype)


def fine():
    torch.cuda.synchronize()
    gdr.device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,dk,dv", [(2, 64, 64), (30, 128, 64)])
def test_decode_over_thousands_of_steps(dtype, N, dk, dv):
    """4000 tokens of one state, decays that forget within a step and within a million."""
    T, decays = 4000, [-1e-4, -1e-5, -1e-6, -0.3, -0.6, -0.8, -20.0, 0.0, -math.inf]
    H, g = len(decays), gen(N)
    ld = torch.tensor(decays, device="cuda")
    q = randn(g, T, 2, 1, dk, dtype=dtype, positive=True)
    k, v = randn(g, T, 2, 1, dk, dtype=dtype, positive=True), randn(g, T, 2, H, dv, dtype=dtype, positive=True)
    rows = torch.arange(N, device="cuda") % 2        # the same two sequences over and over
    S0 = randn(g, 2, H, dk, dv, positive=True)
    state = S0[rows].contiguous()
    for t in range(T):
        o = gdr.linear_decode_step(q[t][rows], k[t][rows], v[t][rows], state, log_decay=ld, scale=0.1)
    fine()
    assert torch.equal(state, state[:2][rows]) and torch.equal(o, o[:2][rows])
    for n in range(2):
        for h, x in enumerate(decays):
            S = acc.decode_states(k[:, n, 0], v[:, n, h], x, S0[n, h])
            acc.check_state(state[n, h], S, T, ld[h], F32, f"row {n}, decay {x}")
            # the sum over dk of positive products: at most dk roundings of 2^-24, and o's own
            y = 0.1 * (q[-1, n, 0].double().cpu() @ S)
            err = acc.rms_error(o[n, h], y)
            limit = acc.state_limit(T, math.exp(x), F32) + dk * 2.0 ** -24 + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24)
            assert err <= limit, f"row {n}, decay {x}: o {err:.2e} over {limit:.2e}"


def test_decode_of_an_infinite_state():
    """lambda times an infinity is one, whatever the token adds (and NaN at lambda = 0)."""
    ld = torch.tensor([-1e-4, -0.3, -2.0, 0.0, -math.inf], device="cuda")
    H, d = 5, 64
    state = torch.ones(1, H, d, d, device="cuda")
    state[..., 0, 0], state[..., 1, 1], state[..., 2, 2] = math.inf, -math.inf, 3e38
    q = torch.ones(1, H, d, device="cuda")
    gdr.linear_decode_step(q, q, q, state, log_decay=ld)
    fine()
    assert (state[0, :4, 0, 0] == math.inf).all() and (state[0, :4, 1, 1] == -math.inf).all()
    assert torch.isfinite(state[0, :, 2, 2]).all() and state[0, 4, :2, :2].isnan().sum() == 2


def sequences(seed, N, T, Hk, H, dk, dv, dtype=BF16, positive=False):
    g = gen(seed)
    q, k = (randn(g, N, T, Hk, dk, dtype=dtype, positive=positive) for _ in range(2))
    v, do = (randn(g, N, T, H, dv, dtype=dtype, positive=positive) for _ in range(2))
    return q, k, v, do, randn(g, N, H, dk, dv, positive=positive), randn(g, N, H, dk, dv, positive=positive)


# (80 rows of 2 heads fill the card: whole sequences; 1345 tokens of two heads: segments)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,T,dk,dv", [(1, 63, 128, 128), (2, 200, 64, 128), (1, 1345, 128, 64), (80, 1345, 64, 64),
                                       (3, 600, 128, 128)])
def test_states_are_kept_in_32_bits(dtype, N, T, dk, dv):
    """The end state and the gradient of the initial state, which two bf16 terms of w c would not make."""
    H, scale = 2, 0.125
    q, k, v, do, S0, dS = sequences(N + T, N, T, H, H, dk, dv, dtype)
    ld = torch.tensor([-1e-3, -0.04], device="cuda")
    _, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0)
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, scale=scale)
    fine()
    for n in {0, N - 1}:
        for h in range(H):
            _, want, _ = acc.exact_run(q[n, :, h], k[n, :, h], v[n, :, h], ld[h].item(), S0[n, h])
            acc.check_state(S[n, h], want, T, ld[h], dtype, f"row {n} head {h} state")
            _, want, _ = acc.exact_run(k[n, :, h], q[n, :, h], do[n, :, h], ld[h].item(), dS[n, h], True, scale)
            acc.check_state(x["initial_state"][n, h], want, T, ld[h], dtype, f"row {n} head {h} d_initial_state")


@pytest.mark.parametrize("dtype,T,H,heads", [(BF16, 16384, 150, (0, 77, 149)), (BF16, 65536, 1, (0,)), (BF16, 16384, 2, (0, 1)),
                                             (F32, 8192, 300, (0, 299)), (F32, 16384, 1, (0,))])
def test_states_of_long_memory(dtype, T, H, heads):
    """Values of one sign and decays whose power over a chunk, a token or a segment lies half way between two fp32
    values: one of them, used over and over, would be off by more than all roundings together."""
    d = 64
    size = _lib.lib().gdr_linear_workspace_size(int(dtype == BF16), 1, T, 1, H, d, d, 1, 0, 0)
    step, segments = (C if dtype == BF16 else 16), size // (4 * H * d * d)
    seg = step * -(-(T // step) // segments) if segments else 0
    near, power = (-5e-6, seg) if T > 60000 else (-2e-5, C if dtype == BF16 else 1)
    assert (segments > 16) == (H < 100)
    ld = torch.full((H,), acc.worst_decay(near, power), device="cuda")
    q, k, v, _, S0, _ = sequences(T + H, 1, T, 1, H, d, d, dtype, positive=True)
    _, S = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0)
    x = gdr.linear_backward(k, q, v, v, log_decay=ld, d_final_state=S0) if H <= 2 else None
    fine()
    for h in heads:
        want = acc.decode_states(k[0, :, 0], v[0, :, h], ld[h], S0[0, h])
        acc.check_state(S[0, h], want, T, ld[h], dtype, f"head {h} state")
        if x is not None:     # the same sum from the other end: token t's share decayed by t + 1
            want = math.exp(ld[h].item()) * acc.decode_states(k[0, :, 0].flip(0), v[0, :, h].flip(0), ld[h],
                                                              S0[0, h].double() / math.exp(ld[h].item()))
            acc.check_state(x["initial_state"][0, h], want, T, ld[h], dtype, f"head {h} d_initial_state")


# (300 tokens packed behind others; 1100 of one head run in segments)
@pytest.mark.parametrize("Hk,H,dk,dv,lens,packed", [(2, 2, 128, 128, [333], False), (1, 1, 64, 128, [1100], False),
                                                    (2, 2, 128, 64, [70, 0, 300, 1, 64], True), (1, 3, 64, 64, [200], False),
                                                    (1, 2, 128, 128, [1100], False)])
def test_outputs_are_off_by_their_roundings(Hk, H, dk, dv, lens, packed):
    """o, dq, dk and dv in bf16, element by element and in all: P, the state operand and the output rounded once."""
    T, N, scale = sum(lens), len(lens), dk ** -0.5
    g = gen(T + H)
    q, k = (randn(g, 1, T, Hk, dk, dtype=BF16) for _ in range(2))
    v, do = (randn(g, 1, T, H, dv, dtype=BF16) for _ in range(2))
    S0, dS = randn(g, N, H, dk, dv), randn(g, N, H, dk, dv)
    ld = torch.tensor([-0.01, -0.3, -1e-4][:H], device="cuda")
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32) if packed else None
    o, _ = gdr.linear_forward(q, k, v, log_decay=ld, initial_state=S0, cu_seqlens=cu, scale=scale)
    x = gdr.linear_backward(q, k, v, do, log_decay=ld, initial_state=S0, d_final_state=dS, cu_seqlens=cu, scale=scale)
    fine()
    G, t = H // Hk, 0
    for n, L in enumerate(lens):
        s, t = slice(t, t + L), t + L
        rms = acc.OUT_RMS if L >= 64 else None      # an average needs enough values
        sums = {"q": [0, 0], "k": [0, 0]}
        for h in range(H):
            c, j, what = ld[h].item(), h // G, f"sequence {n} head {h} "
            Q, K, V, D = q[0, s, j], k[0, s, j], v[0, s, h], do[0, s, h]
            y, _, e = acc.exact_run(Q, K, V, c, S0[n, h], yscale=scale)
            acc.check_output(o[0, s, h], y, e, what + "o", rms)
            y, _, e = acc.exact_run(K, Q, D, c, dS[n, h], True, scale)
            acc.check_output(x["v"][0, s, h], y, e, what + "dv", rms)
            for name, run in (("q", acc.exact_run(D, V, K, c, S0[n, h].T, yscale=scale)),
                              ("k", acc.exact_run(V, D, Q, c, dS[n, h].T, True, scale))):
                sums[name][0], sums[name][1] = sums[name][0] + run[0], sums[name][1] + run[2]
                if h % G == G - 1:
                    # (a shared head's sum is rounded once; each head's bound, with a rounding of its own, covers it:
                    # 2^-8 of the sum is at most the sum of 2^-8 of each)
                    acc.check_output(x[name][0, s, j], sums[name][0], sums[name][1], what + "d" + name, rms)
                    sums[name] = [0, 0]
