"""The bounded waits of the linear attention's bf16 kernels, run out without a fault of the GPU.

GDR_FAULT=wait (on the host) makes the first block of each launch leave out what its own waits wait for: the
copy of its first chunk in phase 1, the product P otherwise.  They give up after their limit (about a second),
the kernel ends, the status says GDR_ERR_TIMEOUT once, and the next call is right."""
import pytest
import torch

import gated_delta_rule_forward_b200 as gdr
import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def status():
    try:
        gdr.device_status()
        return 0
    except gdr.GdrError as e:
        return e.status


# (a short chunk alone, behind others and at the end of a ring; packed, with empty sequences; 1500 tokens of one head run
# in segments, with phase 1 before them)
@pytest.mark.parametrize("dv,lens,packed", [(128, [40], False), (64, [70], False), (128, [333], False), (64, [20, 0, 130], True),
                                            (128, [1500], False), (64, [1500, 0, 3], True)])
@pytest.mark.parametrize("backward", [False, True])
def test_timeout_is_reported_and_the_context_stays_usable(monkeypatch, dv, lens, packed, backward):
    g = torch.Generator(device="cuda").manual_seed(dv + sum(lens))
    T, H, dk = sum(lens), 1, 128
    q, k, v, do = (torch.randn(1, T, H, d, generator=g, device="cuda").to(BF16) for d in (dk, dk, dv, dv))
    ld = torch.tensor([-0.05], device="cuda")
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32) if packed else None

    def call():
        if backward:
            return gdr.linear_backward(q, k, v, do, log_decay=ld, cu_seqlens=cu)
        return gdr.linear_forward(q, k, v, log_decay=ld, cu_seqlens=cu)

    assert status() == 0                      # nothing stale
    monkeypatch.setenv("GDR_FAULT", "wait")
    call()
    monkeypatch.delenv("GDR_FAULT")
    assert status() == 5                      # GDR_ERR_TIMEOUT
    assert status() == 0                      # reported once
    x, t = call(), 0
    assert status() == 0
    for n, L in enumerate(lens):
        s, t = slice(t, t + L), t + L
        if backward:
            ref.check_grads(q[0, s], k[0, s], v[0, s], do[0, s], ld, None, None, 1.0,
                            (x["q"][0, s], x["k"][0, s], x["v"][0, s], x["initial_state"][n]), f"sequence {n}")
        else:
            ref.check_forward(q[0, s], k[0, s], v[0, s], ld, None, 1.0, x[0][0, s], x[1][n], f"sequence {n}")
