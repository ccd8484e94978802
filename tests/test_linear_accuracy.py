"""The limits of linear_accuracy.py tell the kernels' arithmetic from the same with a mistake in it (CPU, emulated)."""
import math

import pytest
import torch

import linear_accuracy as acc
import linear_ref as ref

BF16, F32 = torch.bfloat16, torch.float32


def tensors(seed, T, da, dc, positive=False):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(T, d, generator=g) for d in (da, da, dc)] + [torch.randn(da, dc, generator=g)]
    x = [t.abs() for t in x] if positive else x
    return [t.to(BF16) for t in x[:3]] + [x[3]]


@pytest.mark.parametrize("ld", [-0.3, -1e-3, 0.0, -20.0, -math.inf])
@pytest.mark.parametrize("reverse", [False, True])
def test_the_exact_run_is_the_recurrence(ld, reverse):
    a, b, c, S0 = tensors(1, 130, 8, 4)
    y, S, _ = acc.exact_run(a, b, c, ld, S0, reverse, 0.5, 0.25)
    lam = torch.tensor([ld])
    if reverse:
        _, _, dv, dS0 = ref.grads(b[:, None], a[:, None], c[:, None], c[:, None], lam, dS=S0[None], scale=0.5)
        assert torch.allclose(y, 0.25 * dv[:, 0], rtol=1e-12, atol=1e-12)
        assert torch.allclose(S, dS0[0], rtol=1e-12, atol=1e-12)
    else:
        o, R = ref.run(a[:, None], 0.5 * b[:, None].double(), c[:, None], lam, S0[None], 0.25)
        assert torch.allclose(y, o[:, 0], rtol=1e-12, atol=1e-12) and torch.allclose(S, R[0], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("T", [63, 200, 1345])
@pytest.mark.parametrize("reverse", [False, True])
def test_states_need_three_terms(T, reverse):
    a, b, c, S0 = tensors(2, T, 64, 64)
    ld = -1e-3
    _, S, _ = acc.exact_run(a, b, c, ld, S0, reverse)
    acc.check_state(acc.emulated_run(a, b, c, ld, S0, reverse)[1], S, T, ld, BF16, "three terms")
    for terms in (1, 2):
        with pytest.raises(AssertionError, match="relative RMS"):
            acc.check_state(acc.emulated_run(a, b, c, ld, S0, reverse, terms=terms)[1], S, T, ld, BF16, "fewer")


def test_states_need_both_decays():
    T = 16384
    ld = acc.worst_decay(-2e-5, acc.C)
    a, b, c, S0 = tensors(3, T, 8, 16, positive=True)
    _, S, _ = acc.exact_run(a, b, c, ld, S0)
    acc.check_state(acc.emulated_run(a, b, c, ld, S0)[1], S, T, ld, BF16, "both")
    with pytest.raises(AssertionError, match="relative RMS"):
        acc.check_state(acc.emulated_run(a, b, c, ld, S0, fixed=True)[1], S, T, ld, BF16, "one")


def test_chains_need_the_power_in_two_parts():
    seg, G = 448, 147
    ld = acc.worst_decay(-5e-6, seg)
    _, b, c, _ = tensors(6, seg * G, 8, 16, positive=True)
    S = acc.decode_states(b, c, ld, torch.zeros(8, 16))
    acc.check_state(acc.emulated_chain(b, c, ld, seg), S, seg * G, ld, BF16, "two parts")
    with pytest.raises(AssertionError, match="relative RMS"):
        acc.check_state(acc.emulated_chain(b, c, ld, seg, parts=1), S, seg * G, ld, BF16, "one part")


@pytest.mark.parametrize("reverse", [False, True])
def test_outputs_need_the_right_state(reverse):
    T, ld = 333, -0.01
    a, b, c, S0 = tensors(4, T, 128, 64)
    y, _, bound = acc.exact_run(a, b, c, ld, S0, reverse, yscale=0.1)
    acc.check_output(acc.emulated_run(a, b, c, ld, S0, reverse, yscale=0.1)[0], y, bound, "as it is")
    wrong = acc.emulated_run(a, b, c, ld, S0, reverse, yscale=0.1, start=1.03)[0]
    with pytest.raises(AssertionError, match="times its bound"):
        acc.check_output(wrong, y, bound, "3% off", rms=None)
    with pytest.raises(AssertionError, match="relative RMS"):
        acc.check_output(wrong, y, bound + 1e9, "3% off")


DECODE_DECAYS = (-1e-4, -1e-5, -1e-6)


@pytest.mark.parametrize("ld", DECODE_DECAYS + (-0.3, -0.6, -0.8, -20.0, 0.0, -math.inf))
def test_decode_steps_need_lambda_in_two_parts(ld):
    """S <- hi S + (lo S + k v) against S <- lambda S + k v with lambda in fp32, 4000 steps."""
    T = 4000
    g = torch.Generator().manual_seed(5)
    k, v = torch.randn(T, 32, generator=g).abs(), torch.randn(T, 32, generator=g).abs()
    S0 = torch.randn(32, 32, generator=g).abs()
    lam = torch.tensor(ld, dtype=F32)
    hi, lo = torch.exp(lam), torch.zeros(())
    if ld > -0.6931472:
        e = torch.expm1(lam)
        hi = 1 + e
        hi = torch.nextafter(hi, torch.zeros(())) if hi.double() > 1 + e.double() else hi     # rounded down
        lo = e - (hi - 1)
        assert lo >= 0 and hi.double() + lo.double() == 1 + e.double()
    two, one = S0.clone(), S0.clone()
    fma = lambda x, s, y: (x.double() * s.double() + y.double()).float()
    for t in range(T):
        kv = k[t][:, None] * v[t][None, :]
        two = fma(hi, two, fma(lo, two, kv))
        one = fma(torch.exp(lam), one, kv)
    S = acc.decode_states(k, v, ld, S0)
    acc.check_state(two, S, T, ld, F32, "two parts")
    if ld in DECODE_DECAYS:
        with pytest.raises(AssertionError, match="relative RMS"):
            acc.check_state(one, S, T, ld, F32, "one part")
