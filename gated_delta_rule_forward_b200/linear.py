"""Linear attention with a decay per head, and the pages of its states: the
binding of libgdr's gdr_linear_* and gdr_copy_states entry points (argument
marshalling only; the computation runs in the CUDA kernels, see
include/gdr.h).

    S_t = exp(log_decay) S_{t-1} + k_t v_t^T,    o_t = S_t^T (scale q_t)

``linear_forward`` runs whole prompts (dense or packed), ``linear_decode_step``
one token on a pool of states, ``linear_backward`` the gradients, and
``copy_states`` copies, forks, compacts and clears pages of a pool.  ``StateCache``
keeps the pages of a pool in hand: which are free, forks and compaction.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from ._lib import LinearArgs, LinearGrads, check, lib
from .ops import _DTYPES, _need

__all__ = ["linear_forward", "linear_decode_step", "linear_backward", "copy_states", "StateCache"]

_Stride3 = ctypes.c_longlong * 3


_here = contextlib.nullcontext()


def _on(device, stream):
    """The context a call allocates and launches in, and the handle of its
    stream.  Where they are not so already, the device is made current and
    `stream` (None: the device's current one) torch's current stream, so that
    what is allocated for a call belongs to the stream the call runs on."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)     # current_stream() without the object: 2 us less
        return _here if device.index == torch.cuda.current_device() else torch.cuda.device(device), handle
    if stream.device != device:
        raise ValueError(f"stream must be on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream      # makes its device current, too


def _dense(t, name, shape, dtype, device):
    """_need() with one test where it passes: these checks are half of a small call."""
    if not (t is not None and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _need(t, name, shape, dtype, device)


@functools.lru_cache(maxsize=1024)
def _workspace_size(device_index, *query):
    """gdr_linear_workspace_size on the (current) device, which it is a function of."""
    return lib().gdr_linear_workspace_size(*query)


def _strided(t, name, shape, dtype, device):
    """A [B,T,heads,d] input: unit stride along d; the other strides are the
    library's to check.  None for a dense one."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return None
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if any(n > 1 and s <= 0 for n, s in zip(t.shape[:3], t.stride()[:3])):
        raise ValueError(f"{name} must not be expanded along batch, tokens or heads")
    return _Stride3(*t.stride()[:3])


def _shape(q, k, v, log_decay, cu_seqlens):
    if q is None or v is None or q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B,T,Hk,dk] and v [B,T,H,dv]")
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise ValueError("q, k, v must be bf16 or fp32")
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"v's {H} heads must be a multiple of the {Hk} heads of q and k")
    strides = (_strided(q, "q", q.shape, dtype, dev), _strided(k, "k", q.shape, dtype, dev),
               _strided(v, "v", (B, T, H, dv), dtype, dev))
    _dense(log_decay, "log_decay", (H,), torch.float32, dev)
    a = LinearArgs(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), log_decay=log_decay.data_ptr())
    if strides != (None, None, None):
        for name, stride in zip(("q_stride", "k_stride", "v_stride"), strides):
            if stride is not None:
                setattr(a, name, stride)
    N = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed sequences (cu_seqlens) need B = 1")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() == 0:
            raise ValueError("cu_seqlens must hold N + 1 offsets")
        N = cu_seqlens.numel() - 1
        _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
        a.cu_seqlens = cu_seqlens.data_ptr()
    return a, (_DTYPES[dtype], B, T, Hk, H, dk, dv, N)


def linear_forward(q, k, v, *, log_decay, initial_state=None, output_final_state=True, cu_seqlens=None,
                   state_slots=None, scale=1.0, out=None, final_state=None, stream=None):
    """Linear attention with a decay per head over whole sequences.

    q, k: [B,T,Hk,dk]; v: [B,T,H,dv]; bf16 or fp32 (all the same), CUDA, H a
    multiple of Hk (value head h reads key head h // (H // Hk)); unit stride
    along the last dimension, the others multiples of 16 bytes (so slices of a
    fused projection need no copy).  log_decay: fp32 [H], <= 0.
    cu_seqlens: int32 [N+1] on the device; packs N sequences, empty ones allowed,
    into the T tokens of B = 1; rows of ``out`` behind the last one are left as
    they were (zeros in a fresh ``out``).  initial_state: fp32 [N,H,dk,dv] or
    None (N = B without cu_seqlens).  With state_slots (int32 [N], device)
    initial_state and final_state are pools [pages,H,dk,dv] and sequence n's
    states lie in page state_slots[n], which must differ from one another; a slot
    outside the pool reads zeros and writes nothing.  final_state may be
    initial_state; otherwise ``out`` and final_state overlap no input.  Returns
    (o [B,T,H,dv], final_state or None).

    bf16: products on the tensor cores with fp32 sums, fp32 states; the attention
    products and the state as a product's operand are rounded to bf16 once each, besides o
    (2.4e-3 relative RMS in all).  o's last bits may depend on whether a final state
    is wanted.  A NaN or an infinity in q, k or v reaches, besides the tokens after
    its own, at most the other tokens of its block of 64 in its own sequence (fp32:
    only those after it).
    """
    a, dims = _shape(q, k, v, log_decay, cu_seqlens)
    dt, B, T, Hk, H, dk, dv, N = dims
    dev, f32 = q.device, torch.float32
    pages = N
    if state_slots is not None:
        _dense(state_slots, "state_slots", (N,), torch.int32, dev)
        pool = final_state if final_state is not None else initial_state
        if pool is None:
            raise ValueError("state_slots needs initial_state or final_state")
        if final_state is None and output_final_state:
            raise ValueError("state_slots needs the pool to write as final_state (or output_final_state=False)")
        pages = pool.shape[0]
        a.state_slots, a.pages = state_slots.data_ptr(), pages
    if initial_state is not None:
        _dense(initial_state, "initial_state", (pages, H, dk, dv), f32, dev)
        a.initial_state = initial_state.data_ptr()
    if out is not None:
        _dense(out, "out", (B, T, H, dv), q.dtype, dev)
    if final_state is not None:
        _dense(final_state, "final_state", (pages, H, dk, dv), f32, dev)
    where, handle = _on(dev, stream)
    with where:
        if out is None:
            out = (torch.empty if N else torch.zeros)(B, T, H, dv, device=dev, dtype=q.dtype)
            a.zero_rest = 1
        if final_state is None and output_final_state:
            final_state = torch.empty(N, H, dk, dv, device=dev, dtype=f32)
        a.o = out.data_ptr()
        if final_state is not None:
            a.final_state = final_state.data_ptr()
        ws = _workspace_size(dev.index, *dims, cu_seqlens is not None, 0)
        workspace = torch.empty(ws, device=dev, dtype=torch.uint8) if ws else None
        check(lib().gdr_linear_forward(*dims, a, scale, workspace.data_ptr() if ws else None, ws, handle))
    return out, final_state


def linear_backward(q, k, v, d_o, *, log_decay, initial_state=None, d_final_state=None, cu_seqlens=None, scale=1.0,
                    stream=None):
    """Gradients of <d_o, o> + <d_final_state, S_T> for linear_forward over the
    same inputs.  d_o: [B,T,H,dv] in the I/O type, strided as q may be;
    d_final_state: fp32 [N,H,dk,dv] or None (zero).  Returns a dict: q, k
    [B,T,Hk,dk] (summed over the value heads that share a key head), v
    [B,T,H,dv] in the I/O type, and initial_state fp32 [N,H,dk,dv].  Rows behind
    the last packed sequence get zeros.  The decays are constants: they have no
    gradient.  Rounding and non-finite values as in linear_forward."""
    a, dims = _shape(q, k, v, log_decay, cu_seqlens)
    dt, B, T, Hk, H, dk, dv, N = dims
    dev, f32 = q.device, torch.float32
    stride = _strided(d_o, "d_o", v.shape, q.dtype, dev)
    g = LinearGrads(d_o=d_o.data_ptr())
    if stride is not None:
        g.d_o_stride = stride
    if initial_state is not None:
        _dense(initial_state, "initial_state", (N, H, dk, dv), f32, dev)
        a.initial_state = initial_state.data_ptr()
    if d_final_state is not None:
        _dense(d_final_state, "d_final_state", (N, H, dk, dv), f32, dev)
        g.d_final_state = d_final_state.data_ptr()
    where, handle = _on(dev, stream)
    with where:
        new = torch.empty if N and H else torch.zeros   # no value heads: sums of nothing
        a.zero_rest = 1
        grads = {"q": new(B, T, Hk, dk, device=dev, dtype=q.dtype), "k": new(B, T, Hk, dk, device=dev, dtype=q.dtype),
                 "v": new(B, T, H, dv, device=dev, dtype=q.dtype),
                 "initial_state": torch.empty(N, H, dk, dv, device=dev, dtype=f32)}
        g.dq, g.dk, g.dv = grads["q"].data_ptr(), grads["k"].data_ptr(), grads["v"].data_ptr()
        g.d_initial_state = grads["initial_state"].data_ptr()
        ws = _workspace_size(dev.index, *dims, cu_seqlens is not None, 1)
        workspace = torch.empty(ws, device=dev, dtype=torch.uint8) if ws else None
        check(lib().gdr_linear_backward(*dims, a, g, scale, workspace.data_ptr() if ws else None, ws, handle))
    return grads


def linear_decode_step(q, k, v, state, *, log_decay, state_slots=None, scale=1.0, out=None, stream=None):
    """One decode token for N sequences: q, k [N,Hk,dk]; v [N,H,dv] (contiguous,
    bf16 or fp32); state fp32 [pages,H,dk,dv], updated in place in page
    state_slots[n] (int32 [N], device; None: page n).  A row whose slot lies
    outside the pool is padding: its o is zeros and it touches no state.  The
    slots inside the pool must differ from one another.  Computed in fp32, lambda in two
    parts, so that thousands of steps stay within their roundings.  Returns o [N,H,dv]."""
    if q is None or v is None or state is None or q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q must be [N,Hk,dk], v [N,H,dv] and state [pages,H,dk,dv]")
    N, Hk, dk = q.shape
    H, dv = v.shape[1:]
    pages = state.shape[0]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    if q.dtype not in _DTYPES:
        raise ValueError("q, k, v must be bf16 or fp32")
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"v's {H} heads must be a multiple of the {Hk} heads of q and k")
    _dense(q, "q", (N, Hk, dk), q.dtype, dev)
    _dense(k, "k", (N, Hk, dk), q.dtype, dev)
    _dense(v, "v", (N, H, dv), q.dtype, dev)
    _dense(log_decay, "log_decay", (H,), torch.float32, dev)
    _dense(state, "state", (pages, H, dk, dv), torch.float32, dev)
    if state_slots is not None:
        _dense(state_slots, "state_slots", (N,), torch.int32, dev)
    elif pages != N:
        raise ValueError(f"without state_slots state must hold one page per row ({N}), got {pages}")
    if out is not None:
        _dense(out, "out", (N, H, dv), q.dtype, dev)
    where, handle = _on(dev, stream)
    with where:
        if out is None:
            out = torch.empty(N, H, dv, device=dev, dtype=q.dtype)
        check(lib().gdr_linear_decode_step(_DTYPES[q.dtype], N, Hk, H, dk, dv, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                           log_decay.data_ptr(), state.data_ptr(), pages,
                                           None if state_slots is None else state_slots.data_ptr(), out.data_ptr(), scale,
                                           handle))
    return out


def copy_states(pool, src, dst, *, stream=None):
    """Page copies of a state pool, [pages,H,dk,dv] or [layers,pages,H,dk,dv]
    (fp32, contiguous, CUDA; states of any variant): for each i in turn, page
    dst[i] of every layer becomes a copy of page src[i], or zeros where src[i] is
    -1.  src and dst are host sequences of ints."""
    if pool is None or pool.dim() not in (4, 5):
        raise ValueError("pool must be [pages,H,dk,dv] or [layers,pages,H,dk,dv]")
    if pool.device.type != "cuda":
        raise ValueError("pool must be a CUDA tensor (there is no CPU path)")
    _dense(pool, "pool", pool.shape, torch.float32, pool.device)
    n = len(src)
    if len(dst) != n:
        raise ValueError(f"src has {n} pages and dst {len(dst)}")
    layers = pool.shape[0] if pool.dim() == 5 else 1
    pages, H, dk, dv = pool.shape[-4:]
    if n and not (-1 <= min(src) and max(src) < pages and 0 <= min(dst) and max(dst) < pages):
        raise ValueError(f"pages must lie in [0, {pages}) (src: or be -1)")
    ints = ctypes.c_int * n
    where, handle = _on(pool.device, stream)
    with where:
        check(lib().gdr_copy_states(pool.data_ptr(), layers, pages, H, dk, dv, ints(*src), ints(*dst), n, handle))


class StateCache:
    """The recurrent states of the sequences being served: a pool
    [layers,pages,H,dk,dv] (fp32), a sequence's states of all layers in one page.

    ``layer(l)`` is layer l's pool, the ``state`` of linear_decode_step (with the
    pages as state_slots) and the state pool of linear_forward.  After
    ``compact`` the live pages are the first ones, so that ``layer(l)[:n]`` is the
    contiguous state that ``decode_step`` takes for the delta-rule variants.
    Page copies run on `stream` of each call (None: the current stream)."""

    def __init__(self, pages, layers, H, dk, dv, device="cuda"):
        if pages < 0 or layers < 0:
            raise ValueError("pages and layers must be >= 0")
        self.pool = torch.empty(layers, pages, H, dk, dv, device=device, dtype=torch.float32)
        self._live = [False] * pages
        self._free = list(range(pages - 1, -1, -1))     # the lowest page on top

    def layer(self, i):
        return self.pool[i]

    @property
    def free_pages(self):
        return len(self._free)

    @property
    def live_pages(self):
        return [p for p, live in enumerate(self._live) if live]

    def _check_live(self, pages):
        for p in pages:
            if not 0 <= p < len(self._live) or not self._live[p]:
                raise ValueError(f"page {p} is not in use")
        if len(set(pages)) != len(pages):
            raise ValueError("a page is named twice")

    def _new(self, source, n, stream):
        """n free pages with a copy of `source` (-1: zeros), lowest first; they are in use once the copy is made."""
        if n < 0 or n > len(self._free):
            raise ValueError(f"{n} pages asked for, {len(self._free)} are free")
        taken = self._free[len(self._free) - n:][::-1]
        copy_states(self.pool, [source] * n, taken, stream=stream)
        del self._free[len(self._free) - n:]
        for p in taken:
            self._live[p] = True
        return taken

    def alloc(self, n=1, stream=None):
        """n pages of zeros."""
        return self._new(-1, n, stream)

    def fork(self, page, n=1, stream=None):
        """n new pages with page's states."""
        self._check_live([page])
        return self._new(page, n, stream)

    def free(self, pages):
        """Gives pages back (their contents are cleared when they are allocated again)."""
        pages = list(pages)
        self._check_live(pages)
        for p in pages:
            self._live[p] = False
        self._free = sorted(self._free + pages, reverse=True)

    def compact(self, stream=None):
        """Moves the live pages to the front of the pool.  Returns {old page: new page} of those that moved."""
        live = self.live_pages
        n = len(live)
        holes = [p for p in range(n) if not self._live[p]]
        movers = [p for p in live if p >= n]            # as many as there are holes
        copy_states(self.pool, movers, holes, stream=stream)
        for old, new in zip(movers, holes):
            self._live[old], self._live[new] = False, True
        self._free = list(range(len(self._live) - 1, n - 1, -1))
        return dict(zip(movers, holes))
