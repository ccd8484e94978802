"""Host-side checks of the linear-attention and state-page entry points (no GPU
work): refusals, and the page bookkeeping of StateCache."""
import ctypes

import pytest
import torch

import gated_delta_rule_forward_b200 as gdr
from gated_delta_rule_forward_b200 import _lib, linear

FAKE, MISALIGNED = 0x10000, 0x10008      # never dereferenced: every valid call stops at the injected launch failure


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    monkeypatch.setenv("GDR_FAULT", "launch")


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def args(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, log_decay=FAKE, final_state=FAKE, o=FAKE)
    a.update(over)
    return _lib.LinearArgs(**a)


def grads(**over):
    g = dict(d_o=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, d_initial_state=FAKE)
    g.update(over)
    return _lib.LinearGrads(**g)


def dims(dtype=1, B=2, T=70, Hk=2, H=4, dk=128, dv=128, N=2):
    return dtype, B, T, Hk, H, dk, dv, N


def fwd(L, a=None, ws=FAKE, ws_bytes=1 << 40, **d):
    return L.gdr_linear_forward(*dims(**d), ctypes.byref(a or args()), 1.0, ws, ws_bytes, None)


def bwd(L, a=None, g=None, ws=FAKE, ws_bytes=1 << 40, **d):
    return L.gdr_linear_backward(*dims(**d), ctypes.byref(a or args(o=None, final_state=None)),
                                 ctypes.byref(g or grads()), 1.0, ws, ws_bytes, None)


BAD_DIMS = [(dict(dtype=2), 1), (dict(dk=96), 2), (dict(dv=256), 2), (dict(B=-1, N=-1), 1), (dict(T=-1), 1),
            (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(N=3), 1), (dict(H=1 << 15, Hk=1), 2),
            (dict(T=(1 << 30) + 1, B=1, N=1), 2)]


@pytest.mark.parametrize("call", [fwd, bwd])
def test_valid_calls_reach_the_launch(L, call):
    for dt in (0, 1):
        for dk in (64, 128):
            for dv in (64, 128):
                assert call(L, dtype=dt, dk=dk, dv=dv) == 4
                assert "injected" in L.gdr_last_error().decode()
    assert call(L, Hk=4, T=1) == 4


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("over,code", BAD_DIMS)
def test_bad_dims(L, call, over, code):
    assert call(L, **over) == code
    assert L.gdr_last_error().decode()
    assert L.gdr_linear_workspace_size(*dims(**over), 0, 0) == 0


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("field", ["q", "k", "v", "log_decay"])
def test_missing_tensors(L, call, field):
    assert call(L, a=args(**{field: None})) == 1


@pytest.mark.parametrize("field", ["q", "k", "v", "o", "final_state", "initial_state"])
def test_forward_misaligned(L, field):
    assert fwd(L, a=args(**{field: MISALIGNED})) == 3


@pytest.mark.parametrize("field", ["d_o", "dq", "dk", "dv", "d_final_state", "d_initial_state"])
def test_backward_misaligned(L, field):
    assert bwd(L, g=grads(**{field: MISALIGNED})) == 3


@pytest.mark.parametrize("field", ["d_o", "dq", "dk", "dv"])
def test_backward_missing(L, field):
    assert bwd(L, g=grads(**{field: None})) == 1


def test_backward_state_written_over_one_it_reads(L):
    other = FAKE + 0x10000
    assert bwd(L, g=grads(d_final_state=FAKE)) == 1                    # d_initial_state itself
    assert bwd(L, a=args(initial_state=FAKE), g=grads(d_final_state=other)) == 1
    assert bwd(L, a=args(initial_state=other), g=grads(d_final_state=other)) == 4


def test_null_structs_and_slots(L):
    assert L.gdr_linear_forward(*dims(), None, 1.0, None, 0, None) == 1
    assert L.gdr_linear_backward(*dims(), ctypes.byref(args()), None, 1.0, None, 0, None) == 1
    assert bwd(L, a=args(state_slots=FAKE, pages=4)) == 2
    assert fwd(L, a=args(state_slots=FAKE, pages=-1)) == 1


@pytest.mark.parametrize("dtype,stride", [
    (1, (70 * 2 * 128, 2 * 128, 100)),     # heads closer than d
    (1, (70 * 2 * 128, 2 * 128 + 4, 128)),  # not a multiple of 16 bytes
    (0, (70 * 2 * 128, 2 * 128 + 2, 128)),
    (1, (0, 2 * 128, 128)), (1, (-70 * 2 * 128, 2 * 128, 128)), (1, (1 << 38, 2 * 128, 128))])
def test_bad_strides(L, dtype, stride):
    s = (ctypes.c_longlong * 3)(*stride)
    assert fwd(L, dtype=dtype, a=args(q_stride=s)) == 1
    assert "q: " in L.gdr_last_error().decode()
    assert bwd(L, dtype=dtype, Hk=2, H=2, g=grads(d_o_stride=s)) == 1


def test_good_strides(L):
    s = (ctypes.c_longlong * 3)(70 * 6 * 128, 6 * 128, 128)
    assert fwd(L, a=args(q_stride=s, k_stride=s)) == 4
    # the strides of single entries are never followed
    assert fwd(L, B=1, N=1, T=1, Hk=1, H=1, a=args(q_stride=(ctypes.c_longlong * 3)(3, 5, 7))) == 4


def test_packed(L):
    assert fwd(L, a=args(cu_seqlens=FAKE)) == 1                     # B = 2
    assert fwd(L, B=1, N=7, a=args(cu_seqlens=FAKE)) == 4
    assert fwd(L, B=1, N=0, a=args(cu_seqlens=FAKE)) == 0


def test_workspace(L):
    d = dims(B=1, N=1, T=65536, Hk=1, H=1)
    need = L.gdr_linear_workspace_size(*d, 0, 0)
    assert need > 0
    kw = dict(B=1, N=1, T=65536, Hk=1, H=1)
    assert fwd(L, ws_bytes=need - 1, **kw) == 1
    assert fwd(L, ws=None, **kw) == 1
    assert fwd(L, ws=MISALIGNED, **kw) == 3
    assert fwd(L, ws_bytes=need, **kw) == 4
    need = L.gdr_linear_workspace_size(*dims(), 0, 1)               # shared key heads: dq and dk per value head
    assert need >= 2 * 4 * 2 * 70 * 4 * 128
    assert bwd(L, ws_bytes=need - 1) == 1 and bwd(L, ws_bytes=need) == 4
    assert L.gdr_linear_workspace_size(*dims(T=0), 0, 1) == 0


def test_empty_calls_do_nothing(L):
    assert fwd(L, B=0, N=0) == 0
    assert fwd(L, H=0, Hk=0) == 0
    assert fwd(L, T=0, a=args(q=None, k=None, v=None, o=None, final_state=None)) == 0
    assert fwd(L, T=0, a=args(q=None, k=None, v=None, o=None)) == 4      # the state copy is a launch
    assert bwd(L, T=0, g=grads(d_o=None, dq=None, dk=None, dv=None, d_initial_state=None)) == 0


def decode(L, dtype=1, N=3, Hk=2, H=4, dk=128, dv=64, q=FAKE, k=FAKE, v=FAKE, ld=FAKE, state=FAKE, pages=3, slots=None,
           o=FAKE):
    return L.gdr_linear_decode_step(dtype, N, Hk, H, dk, dv, q, k, v, ld, state, pages, slots, o, 1.0, None)


@pytest.mark.parametrize("over,code", [
    (dict(), 4), (dict(slots=FAKE, pages=1), 4), (dict(dtype=7), 1), (dict(dk=32), 2), (dict(dv=0), 2),
    (dict(N=-1), 1), (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(pages=2), 1), (dict(pages=-1), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(ld=None), 1), (dict(o=None), 1), (dict(state=None), 1),
    (dict(state=None, pages=0, slots=FAKE), 4),          # a batch of padding rows
    (dict(q=MISALIGNED), 3), (dict(state=MISALIGNED), 3), (dict(o=MISALIGNED), 3), (dict(N=0), 0),
    (dict(N=1 << 30, pages=1 << 30), 2)])
def test_decode_refusals(L, over, code):
    assert decode(L, **over) == code


def copies(L, src, dst, pool=FAKE, layers=2, pages=4, H=2, dk=64, dv=64):
    ints = ctypes.c_int * len(src)
    return L.gdr_copy_states(pool, layers, pages, H, dk, dv, ints(*src), ints(*dst), len(src), None)


@pytest.mark.parametrize("src,dst,over,code", [
    ([0], [1], {}, 4), ([-1], [3], {}, 4), ([4], [0], {}, 1), ([-2], [0], {}, 1), ([0], [4], {}, 1), ([0], [-1], {}, 1),
    ([0, 1], [1, 9], {}, 1), ([], [], {}, 0), ([0], [1], dict(layers=0), 0), ([0], [1], dict(H=0), 0),
    ([0], [1], dict(pool=None), 1), ([0], [1], dict(pool=MISALIGNED), 3), ([0], [1], dict(dk=96), 2),
    ([0], [1], dict(pages=-1), 1), ([0], [1], dict(H=1 << 30), 2)])
def test_copy_refusals(L, src, dst, over, code):
    assert copies(L, src, dst, **over) == code


def test_binding_refuses_cpu_tensors():
    q, v, ld = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2, 64), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_forward(q, q, v, log_decay=ld)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_backward(q, q, v, v, log_decay=ld)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_decode_step(q[0], q[0], v[0], torch.zeros(4, 2, 64, 64), log_decay=ld)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.copy_states(torch.zeros(4, 2, 64, 64), [0], [1])
    with pytest.raises(ValueError, match="pool must be"):
        gdr.copy_states(torch.zeros(4, 64, 64), [0], [1])


def test_state_cache_pages(monkeypatch):
    def copy(pool, src, dst, *, stream=None):
        for a, b in zip(src, dst):
            pool[:, b] = pool[:, a] if a >= 0 else 0.0

    monkeypatch.setattr(linear, "copy_states", copy)
    c = gdr.StateCache(6, 2, 1, 64, 64, device="cpu")
    c.pool.fill_(9.0)
    a = c.alloc(4)
    assert a == [0, 1, 2, 3] and c.free_pages == 2 and (c.pool[:, a] == 0).all() and (c.pool[:, 4:] == 9).all()
    for p in a:
        c.pool[:, p] = float(p + 1)
    with pytest.raises(ValueError, match="2 are free"):
        c.alloc(3)
    f = c.fork(2, 1)
    assert f == [4] and (c.pool[:, 4] == 3).all()
    c.free([0, 3])
    for bad in ([0], [5], [6], [-1], [1, 1]):
        with pytest.raises(ValueError):
            c.free(bad)
    with pytest.raises(ValueError):
        c.fork(0)
    assert c.live_pages == [1, 2, 4]
    assert c.compact() == {4: 0}
    assert c.live_pages == [0, 1, 2] and (c.pool[:, 0] == 3).all() and c.free_pages == 3
    assert c.compact() == {}
    assert c.alloc(3) == [3, 4, 5] and c.free_pages == 0
    with pytest.raises(ValueError):
        c.fork(0)
    assert c.layer(1).data_ptr() == c.pool[1].data_ptr()


def test_state_cache_keeps_its_pages_when_a_copy_fails(monkeypatch):
    def fails(pool, src, dst, *, stream=None):
        raise _lib.GdrError(4, "injected")

    c = gdr.StateCache(3, 1, 1, 64, 64, device="cpu")
    monkeypatch.setattr(linear, "copy_states", lambda *a, **k: None)
    a = c.alloc(2)
    c.free(a[:1])
    monkeypatch.setattr(linear, "copy_states", fails)
    for call in (lambda: c.alloc(1), lambda: c.fork(a[1], 1), lambda: c.compact()):
        with pytest.raises(_lib.GdrError):
            call()
        assert c.live_pages == [a[1]] and c.free_pages == 2


def _fake_calls():
    """Keyword calls of the binding on stand-ins for CUDA tensors (no storage behind them)."""
    bf = dict(device="cuda", dtype=torch.bfloat16)
    q, k, v, d_o = (torch.empty(2, 5, 4, 64, **bf) for _ in range(4))
    ld = torch.empty(4, device="cuda")
    row = {n: torch.empty(2, 4, 64, **bf) for n in "qkv"}
    return [(gdr.linear_forward, dict(q=q, k=k, v=v, log_decay=ld)),
            (gdr.linear_backward, dict(q=q, k=k, v=v, d_o=d_o, log_decay=ld)),
            (gdr.linear_decode_step, dict(row, state=torch.empty(2, 4, 64, 64, device="cuda"), log_decay=ld))]


@pytest.mark.parametrize("which", range(3))
def test_binding_says_what_is_missing(which):
    """None, and tensors of another device, type or shape, are refused as arguments, before anything reads them."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        call, good = _fake_calls()[which]
        for name in good:
            with pytest.raises(ValueError, match=rf"\b{name}\b"):
                call(**dict(good, **{name: None}))
            if name == "q":                       # the others are compared with it
                continue
            with pytest.raises(ValueError, match=rf"\b{name}\b must be"):
                call(**dict(good, **{name: torch.empty(good[name].shape, dtype=good[name].dtype)}))
            with pytest.raises(ValueError, match=rf"\b{name}\b must be"):
                call(**dict(good, **{name: good[name].to(torch.float16)}))
            if name in ("k", "d_o", "log_decay"):
                with pytest.raises(ValueError, match=rf"\b{name}\b must have shape"):
                    call(**dict(good, **{name: good[name][:1]}))


def test_copies_need_a_pool():
    with pytest.raises(ValueError, match="pool must be"):
        gdr.copy_states(None, [0], [1])
