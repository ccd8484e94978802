"""Linear attention with a decay per head, on the GPU: what its kernels may lose of the 64-bit recurrence
(tests/linear_accuracy.py has the limits and says what they tell apart)."""
import math

import pytest
import torch

import gated_delta_rule_forward_b200 as gdr
import linear_accuracy as acc

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


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
