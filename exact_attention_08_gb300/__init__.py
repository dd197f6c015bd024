"""Exact attention on GB300 (sm_103a): thin Python binding of libattn_gb300.so.

Every function here only marshals arguments (device pointers, sizes, the
current CUDA stream) and calls the C ABI declared in include/attn.h of the
same name; all attention arithmetic runs in the library's CUDA kernels.
PyTorch is used for device memory and streams only.  There is no fallback:
importing this package fails if the library cannot be built or loaded, and a
call fails if the library reports an error.

    o, lse = attn_fwd(q, k, v, causal=True)          # q [B,Sq,Hq,d], k/v [B,Skv,Hkv,d]
    o, lse = attn_fwd_ex(q, k, v, cu_q, cu_k, max_seqlen_q=..., causal=True)
    o, lse = attn_decode_paged(q, k_pages, v_pages, page_table, seqlens, num_splits=8)
    o, lse = attn_fwd_ex_sink(q, k, v, sink_logit, causal=True)   # sink_logit [Hq] fp32
    o, lse = attn_decode_paged_sink(q, k_pages, v_pages, page_table, seqlens, sink_logit)

Around the attention calls, rotary positions and the paged cache's upkeep:

    inv_freq = attn_rope_inv_freq(128, base=10000.0)              # fp64 [64]
    q, k = attn_rope(q, k, inv_freq)                              # attn_rope_bwd for gradients
    attn_pages_resize(page_table, seqlens, new_seqlens, refs, k_pages, v_pages)
    q = attn_append_paged(q, k, v, k_pages, v_pages, page_table, seqlens, inv_freq=inv_freq)
    attn_pages_fork(page_table, seqlens, refs, src, dst, k_pages, v_pages)
    new_index, num_live = attn_pages_compact(page_table, seqlens, refs, k_pages, v_pages)
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

from . import _build

__all__ = [
    "ATTN_OK", "ATTN_ERR_INVALID_ARG", "ATTN_ERR_UNSUPPORTED", "ATTN_ERR_CUDA", "ATTN_ERR_TIMEOUT",
    "ATTN_ERR_BAD_INPUT", "ATTN_ERR_NO_PAGES", "AttnError", "attn_fwd", "attn_fwd_ex", "attn_fwd_ex_sink",
    "attn_fwd_paged", "attn_fwd_strided", "attn_bwd", "attn_bwd_ex", "attn_bwd_ex_sink",
    "attn_bwd_workspace_size",
    "attn_decode_workspace_size", "attn_decode_paged", "attn_decode_paged_sink", "attn_device_status", "attn_check_wait_timeout", "attn_status_string",
    "attn_rope_inv_freq", "attn_rope", "attn_rope_bwd", "attn_append_paged",
    "attn_pages_workspace_size", "attn_pages_resize", "attn_pages_fork", "attn_pages_compact",
    "attn_last_error", "library_path", "lib",
]

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_BAD_INPUT = 5
ATTN_ERR_NO_PAGES = 6


def _load() -> ctypes.CDLL:
    path = _build.LIB
    if _build.needs_build():
        try:
            path = _build.build()
        except Exception as e:  # no silent fallback: the package is unusable without it
            raise ImportError(f"exact_attention_08_gb300: cannot build {_build.LIB}: {e}") from e
    if not os.path.exists(path):
        raise ImportError(f"exact_attention_08_gb300: {path} is missing")
    L = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
    L.attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, i, i, vp]
    L.attn_fwd_ex_sink.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, i, i,
                                   vp, vp]
    L.attn_fwd_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i,
                                 i, i, vp, vp]
    i64p = ctypes.POINTER(ctypes.c_longlong)
    L.attn_fwd_strided.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i64p, i64p, i64p, i64p, f,
                                   i, i, i, vp, vp]
    L.attn_bwd_workspace_size.argtypes = [i, i, i]
    L.attn_bwd_workspace_size.restype = sz
    L.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, sz, vp]
    L.attn_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f,
                              i, i, i, vp, sz, vp]
    L.attn_bwd_ex_sink.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                   i, f, i, i, i, vp, vp, vp, sz, vp]
    L.attn_decode_workspace_size.argtypes = [i, i, i, i]
    L.attn_decode_workspace_size.restype = sz
    L.attn_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, sz,
                                    vp]
    L.attn_decode_paged_sink.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp,
                                         vp, sz, vp]
    dbl = ctypes.c_double
    L.attn_rope_inv_freq.argtypes = [i, dbl, i, dbl, dbl, dbl, dbl, vp]
    L.attn_rope.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i64p, i64p, i64p, i64p,
                            vp]
    L.attn_rope_bwd.argtypes = L.attn_rope.argtypes
    L.attn_append_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f,
                                    i, i, i, i64p, i64p, i64p, i64p, vp]
    L.attn_pages_workspace_size.argtypes = [i, i]
    L.attn_pages_workspace_size.restype = sz
    L.attn_pages_resize.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    L.attn_pages_fork.argtypes = [vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    L.attn_pages_compact.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp]
    L.attn_device_status.argtypes = [vp]
    L.attn_check_wait_timeout.argtypes = [i, vp]
    L.attn_status_string.argtypes = [i]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_last_error.argtypes = []
    L.attn_last_error.restype = ctypes.c_char_p
    for fn in ("attn_fwd", "attn_fwd_ex", "attn_fwd_ex_sink", "attn_fwd_paged", "attn_fwd_strided",
               "attn_bwd", "attn_bwd_ex", "attn_bwd_ex_sink",
               "attn_decode_paged",
               "attn_decode_paged_sink", "attn_rope_inv_freq", "attn_rope", "attn_rope_bwd",
               "attn_append_paged", "attn_pages_resize", "attn_pages_fork", "attn_pages_compact",
               "attn_device_status", "attn_check_wait_timeout"):
        getattr(L, fn).restype = ctypes.c_int
    return L


lib = _load()
library_path = _build.LIB


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = lib.attn_last_error().decode()
        msg = f"{what}: {lib.attn_status_string(status).decode()}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


def attn_status_string(status: int) -> str:
    return lib.attn_status_string(int(status)).decode()


def attn_last_error() -> str:
    return lib.attn_last_error().decode()


def _check(rc: int, what: str) -> None:
    if rc != ATTN_OK:
        raise AttnError(rc, what)


_torch_module = _current_device = _raw_stream = None


def _torch():
    """torch, imported on first use, with the two calls of it that every launch around the
    attention makes: torch's own short forms where it has them, which a torch without
    CUDA does not, else the documented ones."""
    global _torch_module, _current_device, _raw_stream
    if _torch_module is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch_module = torch
    return _torch_module


def _stream(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def attn_fwd(q, k, v, o=None, lse=None, *, causal=False, window=0, scale=None, stream=None,
             want_lse=True):
    """Dense BSHD forward.  q [B,Sq,Hq,d], k/v [B,Skv,Hkv,d] bf16 -> o [B,Sq,Hq,d] bf16,
    lse [B,Hq,Sq] fp32 (None when want_lse is False and lse is not given)."""
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, q.device)
    B, Sq, Hq, d = q.shape
    Bk, Skv, Hkv, dk = k.shape
    if Bk != B or dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("q/k/v shapes disagree")
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", torch.bfloat16, q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv, d,
                      scale, int(bool(causal)), int(window), _stream(stream))
    _check(rc, "attn_fwd")
    return o, lse


def attn_fwd_ex(q, k, v, cu_seqlens_q=None, cu_seqlens_k=None, *, max_seqlen_q=None,
                max_seqlen_k=None, o=None, lse=None, causal=False, window=0, n_sink=0, scale=None,
                stream=None, want_lse=True):
    """Forward with sink keys and optional packing.  With cu_seqlens (int32 CUDA
    tensors [nseq+1]): q [Tq,Hq,d], k/v [Tk,Hkv,d], o [Tq,Hq,d], lse [Hq,Tq].
    Without: the dense layout of attn_fwd."""
    return _fwd_ex(q, k, v, cu_seqlens_q, cu_seqlens_k, None, max_seqlen_q, max_seqlen_k, o, lse,
                   causal, window, n_sink, scale, stream, want_lse)


def attn_fwd_ex_sink(q, k, v, sink_logit, cu_seqlens_q=None, cu_seqlens_k=None, *,
                     max_seqlen_q=None, max_seqlen_k=None, o=None, lse=None, causal=False,
                     window=0, n_sink=0, scale=None, stream=None, want_lse=True):
    """attn_fwd_ex with a logit sink per query head: sink_logit fp32 CUDA tensor [Hq]
    (-inf entries: no sink for that head)."""
    return _fwd_ex(q, k, v, cu_seqlens_q, cu_seqlens_k, sink_logit, max_seqlen_q, max_seqlen_k,
                   o, lse, causal, window, n_sink, scale, stream, want_lse)


def _fwd_ex(q, k, v, cu_seqlens_q, cu_seqlens_k, sink_logit, max_seqlen_q, max_seqlen_k, o, lse,
            causal, window, n_sink, scale, stream, want_lse):
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, q.device)
    varlen = cu_seqlens_q is not None
    if varlen:
        _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, q.device)
        _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, q.device)
        Tq, Hq, d = q.shape
        Tk, Hkv, _ = k.shape
        nseq = cu_seqlens_q.numel() - 1
        if max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("max_seqlen_q and max_seqlen_k are required with cu_seqlens")
        B, sq, sk = nseq, int(max_seqlen_q), int(max_seqlen_k)
        lse_shape = (Hq, Tq)
    else:
        B, sq, Hq, d = q.shape
        _, sk, Hkv, _ = k.shape
        Tq = Tk = 0
        lse_shape = (B, Hq, sq)
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", torch.bfloat16, q.device)
    if lse is None and want_lse:
        lse = torch.empty(*lse_shape, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if sink_logit is None:
        rc = lib.attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q),
                             _ptr(cu_seqlens_k), B, Hq, Hkv, sq, sk, Tq, Tk, d, scale,
                             int(bool(causal)), int(window), int(n_sink), _stream(stream))
        _check(rc, "attn_fwd_ex")
    else:
        _need(sink_logit, "sink_logit", torch.float32, q.device)
        if sink_logit.numel() != Hq:
            raise ValueError(f"sink_logit must hold Hq={Hq} values")
        rc = lib.attn_fwd_ex_sink(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                  _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, Hq, Hkv, sq, sk, Tq,
                                  Tk, d, scale, int(bool(causal)), int(window), int(n_sink),
                                  _ptr(sink_logit), _stream(stream))
        _check(rc, "attn_fwd_ex_sink")
    return o, lse


def attn_fwd_paged(q, k_pages, v_pages, page_table, cu_seqlens_q, seqlens_k, o=None, lse=None, *,
                   max_seqlen_q=None, causal=True, window=0, n_sink=0, sink_logit=None,
                   scale=None, stream=None, want_lse=True):
    """Packed queries q [Tq,Hq,d] bf16 against a paged cache k/v_pages [P,16,Hkv,d];
    page_table [B,maxP] int32, cu_seqlens_q [B+1] int32, seqlens_k [B] int32 ->
    o [Tq,Hq,d] bf16, lse [Hq,Tq] fp32.  Causal alignment is to the end of each
    sequence's keys."""
    torch = _torch()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(k_pages, "k_pages", torch.bfloat16, dev)
    _need(v_pages, "v_pages", torch.bfloat16, dev)
    _need(page_table, "page_table", torch.int32, dev)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev)
    _need(seqlens_k, "seqlens_k", torch.int32, dev)
    Tq, Hq, d = q.shape
    P, page, Hkv, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages shapes disagree with q")
    B = seqlens_k.numel()
    if page_table.dim() != 2 or page_table.shape[0] != B or cu_seqlens_q.numel() != B + 1:
        raise ValueError("page_table must be [B, max_pages], cu_seqlens_q [B+1], seqlens_k [B]")
    if max_seqlen_q is None:
        raise ValueError("max_seqlen_q is required")
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", torch.bfloat16, dev)
    if lse is None and want_lse:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if sink_logit is not None:
        _need(sink_logit, "sink_logit", torch.float32, dev)
        if sink_logit.numel() != Hq:
            raise ValueError(f"sink_logit must hold Hq={Hq} values")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib.attn_fwd_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                            _ptr(cu_seqlens_q), _ptr(seqlens_k), _ptr(o), _ptr(lse), B, Hq, Hkv,
                            int(max_seqlen_q), Tq, d, page, page_table.shape[1], P, scale,
                            int(bool(causal)), int(window), int(n_sink), _ptr(sink_logit),
                            _stream(stream))
    _check(rc, "attn_fwd_paged")
    return o, lse


def attn_fwd_strided(q, k, v, o=None, lse=None, *, causal=False, window=0, n_sink=0,
                     sink_logit=None, scale=None, stream=None, want_lse=True):
    """Dense forward on q [B,Sq,Hq,d], k/v [B,Skv,Hkv,d] of any strides with d
    contiguous (a BHSD tensor passed as ``t.transpose(1, 2)``, for instance).
    o defaults to ``empty_like(q)`` (same layout); lse is [B,Hq,Sq] contiguous."""
    torch = _torch()
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
            raise ValueError(f"{n} must be a bf16 CUDA tensor")
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{n} must be 4-D with a contiguous last dimension")
    B, Sq, Hq, d = q.shape
    Bk, Skv, Hkv, dk = k.shape
    if Bk != B or dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("q/k/v shapes disagree")
    if o is None:
        o = torch.empty_like(q)
    if o.dtype != torch.bfloat16 or tuple(o.shape) != tuple(q.shape) or o.stride(3) != 1:
        raise ValueError("o must be bf16, shaped like q, with a contiguous last dimension")
    if lse is None and want_lse:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if sink_logit is not None:
        _need(sink_logit, "sink_logit", torch.float32, dev)
        if sink_logit.numel() != Hq:
            raise ValueError(f"sink_logit must hold Hq={Hq} values")

    def strides(t):
        return (ctypes.c_longlong * 3)(t.stride(0), t.stride(1), t.stride(2))

    sq, sk, sv, so = strides(q), strides(k), strides(v), strides(o)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib.attn_fwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv,
                              d, sq, sk, sv, so, scale, int(bool(causal)), int(window),
                              int(n_sink), _ptr(sink_logit), _stream(stream))
    _check(rc, "attn_fwd_strided")
    return o, lse


def attn_bwd_workspace_size(B: int, Hq: int, Sq: int) -> int:
    return int(lib.attn_bwd_workspace_size(int(B), int(Hq), int(Sq)))


def attn_bwd(q, k, v, o, lse, dout, dq=None, dk=None, dv=None, *, causal=False, scale=None,
             workspace=None, stream=None):
    """Gradients of attn_fwd: q [B,Sq,Hq,d], k/v [B,Skv,Hkv,d], the forward's o and
    lse [B,Hq,Sq], dout like o (all contiguous, bf16 except lse) -> (dq, dk, dv) bf16."""
    torch = _torch()
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n, torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    B, Sq, Hq, d = q.shape
    Bk, Skv, Hkv, dk_ = k.shape
    if Bk != B or dk_ != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("q/k/v shapes disagree")
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("o and dout must be shaped like q")
    if tuple(lse.shape) != (B, Hq, Sq):
        raise ValueError("lse must be [B, Hq, Sq]")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, n, ref in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _need(t, n, torch.bfloat16, dev)
        if tuple(t.shape) != tuple(ref.shape):
            raise ValueError(f"{n} has the wrong shape")
    need = attn_bwd_workspace_size(B, Hq, Sq)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib.attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                      _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Skv, d, scale, int(bool(causal)),
                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                      _stream(stream))
    _check(rc, "attn_bwd")
    return dq, dk, dv


def attn_bwd_ex(q, k, v, o, lse, dout, cu_seqlens_q=None, cu_seqlens_k=None, dq=None, dk=None,
                dv=None, *, max_seqlen_q=None, max_seqlen_k=None, causal=False, window=0,
                n_sink=0, scale=None, workspace=None, stream=None):
    """Gradients of attn_fwd_ex (sink keys, sliding window, packed sequences).
    With cu_seqlens (int32 CUDA tensors [nseq+1]): q, o, dout [Tq,Hq,d], k/v
    [Tk,Hkv,d], lse [Hq,Tq]; without: the dense layout of attn_bwd."""
    return _bwd_ex(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, dq, dk, dv, None, None,
                   max_seqlen_q, max_seqlen_k, causal, window, n_sink, scale, workspace, stream)


def attn_bwd_ex_sink(q, k, v, o, lse, dout, sink_logit, cu_seqlens_q=None, cu_seqlens_k=None,
                     dq=None, dk=None, dv=None, dsink=None, *, max_seqlen_q=None,
                     max_seqlen_k=None, causal=False, window=0, n_sink=0, scale=None,
                     workspace=None, stream=None):
    """Gradients of attn_fwd_ex_sink: (dq, dk, dv, dsink), dsink fp32 [Hq]
    the gradient of the logit sink.  lse is the forward's (sink included)."""
    torch = _torch()
    _need(sink_logit, "sink_logit", torch.float32, q.device)
    Hq = q.shape[-2]
    if sink_logit.numel() != Hq:
        raise ValueError(f"sink_logit must hold Hq={Hq} values")
    dsink = torch.empty(Hq, dtype=torch.float32, device=q.device) if dsink is None else dsink
    _need(dsink, "dsink", torch.float32, q.device)
    if dsink.numel() != Hq:
        raise ValueError(f"dsink must hold Hq={Hq} values")
    return _bwd_ex(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, dq, dk, dv,
                   sink_logit.contiguous(), dsink, max_seqlen_q, max_seqlen_k, causal, window,
                   n_sink, scale, workspace, stream)


def _bwd_ex(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, dq, dk, dv, sink_logit, dsink,
            max_seqlen_q, max_seqlen_k, causal, window, n_sink, scale, workspace, stream):
    torch = _torch()
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n, torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    varlen = cu_seqlens_q is not None
    if varlen:
        _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev)
        _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev)
        Tq, Hq, d = q.shape
        Tk, Hkv, dk_ = k.shape
        if max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("max_seqlen_q and max_seqlen_k are required with cu_seqlens")
        B, sq, sk = cu_seqlens_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k)
        lse_shape = (Hq, Tq)
    else:
        B, sq, Hq, d = q.shape
        Bk, sk, Hkv, dk_ = k.shape
        if Bk != B:
            raise ValueError("q/k batch sizes disagree")
        Tq = Tk = 0
        lse_shape = (B, Hq, sq)
    if dk_ != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("q/k/v shapes disagree")
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("o and dout must be shaped like q")
    if tuple(lse.shape) != lse_shape:
        raise ValueError(f"lse must be {list(lse_shape)}")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, n, ref in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _need(t, n, torch.bfloat16, dev)
        if tuple(t.shape) != tuple(ref.shape):
            raise ValueError(f"{n} has the wrong shape")
    need = attn_bwd_workspace_size(B, Hq, sq)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
            _ptr(dv), _ptr(cu_seqlens_q) if varlen else None,
            _ptr(cu_seqlens_k) if varlen else None, B, Hq, Hkv, sq, sk, Tq, Tk, d, scale,
            int(bool(causal)), int(window), int(n_sink))
    tail = (_ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if sink_logit is None:
        _check(lib.attn_bwd_ex(*args, *tail), "attn_bwd_ex")
        return dq, dk, dv
    _check(lib.attn_bwd_ex_sink(*args, _ptr(sink_logit), _ptr(dsink), *tail), "attn_bwd_ex_sink")
    return dq, dk, dv, dsink


def attn_decode_workspace_size(B: int, Hq: int, d: int, num_splits: int) -> int:
    return int(lib.attn_decode_workspace_size(int(B), int(Hq), int(d), int(num_splits)))


def attn_decode_paged(q, k_pages, v_pages, page_table, seqlens, o=None, lse=None, *,
                      num_splits=8, scale=None, workspace=None, stream=None, want_lse=True):
    """One-token decode.  q [B,Hq,d] bf16, k/v_pages [P,16,Hkv,d] bf16, page_table
    [B,maxP] int32, seqlens [B] int32 -> o [B,Hq,d] bf16, lse [B,Hq] fp32."""
    return _decode(q, k_pages, v_pages, page_table, seqlens, None, o, lse, num_splits, scale,
                   workspace, stream, want_lse)


def attn_decode_paged_sink(q, k_pages, v_pages, page_table, seqlens, sink_logit, o=None,
                           lse=None, *, num_splits=8, scale=None, workspace=None, stream=None,
                           want_lse=True):
    """attn_decode_paged with a logit sink per query head: sink_logit fp32 CUDA tensor [Hq]."""
    return _decode(q, k_pages, v_pages, page_table, seqlens, sink_logit, o, lse, num_splits,
                   scale, workspace, stream, want_lse)


def _decode(q, k_pages, v_pages, page_table, seqlens, sink_logit, o, lse, num_splits, scale,
            workspace, stream, want_lse):
    torch = _torch()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(k_pages, "k_pages", torch.bfloat16, dev)
    _need(v_pages, "v_pages", torch.bfloat16, dev)
    _need(page_table, "page_table", torch.int32, dev)
    _need(seqlens, "seqlens", torch.int32, dev)
    B, Hq, d = q.shape
    P, page, Hkv, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages shapes disagree with q")
    if page_table.dim() != 2 or page_table.shape[0] != B or seqlens.numel() != B:
        raise ValueError("page_table must be [B, max_pages] and seqlens [B]")
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", torch.bfloat16, dev)
    if lse is None and want_lse:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    need = attn_decode_workspace_size(B, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    wbytes = workspace.numel() * workspace.element_size()
    if sink_logit is None:
        rc = lib.attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                   _ptr(seqlens), _ptr(o), _ptr(lse), B, Hq, Hkv, d, page,
                                   page_table.shape[1], P, int(num_splits), scale, _ptr(workspace),
                                   wbytes, _stream(stream))
        _check(rc, "attn_decode_paged")
    else:
        _need(sink_logit, "sink_logit", torch.float32, dev)
        if sink_logit.numel() != Hq:
            raise ValueError(f"sink_logit must hold Hq={Hq} values")
        rc = lib.attn_decode_paged_sink(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                        _ptr(seqlens), _ptr(o), _ptr(lse), B, Hq, Hkv, d, page,
                                        page_table.shape[1], P, int(num_splits), scale,
                                        _ptr(sink_logit), _ptr(workspace), wbytes, _stream(stream))
        _check(rc, "attn_decode_paged_sink")
    return o, lse


# ---------------------------------------------------------------- around the attention calls
# A decode step makes several of these calls a layer, each a few microseconds
# on the GPU, so their checks are kept to a few attribute reads; the text of a
# refusal is worked out only once one has failed.

class _Call:
    """Makes the tensors' device and the call's stream current (and with them where
    tensors made inside belong)."""
    __slots__ = ("_contexts",)

    def __init__(self, index, stream):
        torch = _torch()
        self._contexts = (torch.cuda.device(index),)
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                raw = int(getattr(stream, "cuda_stream", stream))
                stream = torch.cuda.ExternalStream(raw, device=index) if raw else \
                    torch.cuda.default_stream(index)
            elif stream.device_index != index:
                raise ValueError(f"stream is one of cuda:{stream.device_index}, the tensors are "
                                 f"on cuda:{index}")
            self._contexts += (torch.cuda.stream(stream),)

    def __enter__(self):
        for c in self._contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._contexts):
            c.__exit__(*exc)


def _rows_tensor(t, name, dims, index):
    """bf16 on device `index`, `dims` dimensions, the last one contiguous."""
    torch = _torch()
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.get_device() == index and \
            index >= 0 and t.dim() in dims and (t.is_contiguous() or t.stride(-1) == 1):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{name} must be a bf16 CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions")
    if t.shape[-1] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _int_tensor(t, name, index):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.int32 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on cuda:{index}")


def _int_vector(t, name, n, index):
    _int_tensor(t, name, index)
    if t.dim() != 1 or t.numel() != n:
        raise ValueError(f"{name} must be [{n}], got {list(t.shape)}")


_INT_MAX = 2 ** 31 - 1


def _c_int(n):
    """A size for the library's 32-bit arguments, into which ctypes would put the low bits of
    a larger one: both ends stand for what the library refuses."""
    return n if -1 <= n <= _INT_MAX else _INT_MAX if n > 0 else -1


def _frequencies(inv_freq, d, index):
    torch = _torch()
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype is not torch.float64 or \
            inv_freq.dim() != 1 or inv_freq.get_device() != index or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous float64 vector on cuda:{index}")
    rot = 2 * inv_freq.numel()
    if rot > d:
        raise ValueError(f"inv_freq holds {rot // 2} pairs, a head has {d // 2}")
    return rot


def _output(out, t, name):
    """`out` if it is a fit output for t, or a new one with t's layout."""
    if out is None:
        out = _torch_module.empty_like(t)
        # a broadcast t leaves the order of the new strides to torch
        if out.is_contiguous() or out.stride(-1) == 1:
            return out
        return _torch_module.empty(t.shape, dtype=t.dtype, device=t.device)
    _rows_tensor(out, name + "_out", (t.dim(),), t.get_device())
    if out.shape != t.shape:
        raise ValueError(f"{name}_out must be shaped like {name}")
    return out


def _strides(t, n):
    """{[batch,] row, head} strides as a C array of n, or None if t is contiguous.  Packed
    rows have no batch stride."""
    if t.is_contiguous():
        return None
    st = t.stride()[:-1]
    return (ctypes.c_longlong * n)(*(st if len(st) == n else (0, *st)))


_ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}


def attn_rope_inv_freq(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none",
                       factor: float = 1.0, original_length: float = 0.0, ramp=(1.0, 32.0),
                       device="cuda"):
    """Radians per position of each rotated pair, base^(-2i/rotary_dim), as the fp64
    tensor [rotary_dim / 2] that attn_rope and attn_append_paged take.  scaling
    stretches it for contexts longer than the trained one: "linear" (every
    frequency / factor), "base" (a larger base: the slowest pair / factor) or
    "ramp" (pairs that turn more than ramp[1] times over original_length are
    kept, those that turn less than ramp[0] times / factor, linear in the turns
    between; a model whose ramp is linear in the pair's index needs its own
    inv_freq)."""
    torch = _torch()
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}")
    rotary_dim = _c_int(int(rotary_dim))
    out = torch.empty(max(rotary_dim // 2, 0), dtype=torch.float64)
    _check(lib.attn_rope_inv_freq(rotary_dim, float(base), _ROPE_SCALINGS[scaling],
                                  float(factor), float(original_length), float(ramp[0]),
                                  float(ramp[1]), out.data_ptr()), "attn_rope_inv_freq")
    return out.to(device)


def attn_rope(q, k, inv_freq, positions=None, *, interleaved=False, amplitude=1.0, q_out=None,
              k_out=None, stream=None):
    """Rotary positions: q [B,S,Hq,d] and k [B,S,Hkv,d] (or packed [T,H,d]) bf16, any
    strides with d contiguous, turned by positions [B,S] ([T]) int32 (default: the
    row's index) times inv_freq fp64 [rotary_dim / 2] -> (q_out, k_out).  Either of q
    and k may be None.  In place: q_out=q, k_out=k."""
    return _rope(lib.attn_rope, "attn_rope", ("q", "k"), q, k, inv_freq, positions, interleaved,
                 amplitude, q_out, k_out, stream)


def attn_rope_bwd(dq, dk, inv_freq, positions=None, *, interleaved=False, amplitude=1.0,
                  dq_out=None, dk_out=None, stream=None):
    """Gradients of attn_rope: from dq, dk of its outputs those of its inputs, with the
    forward's inv_freq, positions, interleaved and amplitude -> (dq_out, dk_out)."""
    return _rope(lib.attn_rope_bwd, "attn_rope_bwd", ("dq", "dk"), dq, dk, inv_freq, positions,
                 interleaved, amplitude, dq_out, dk_out, stream)


def _rope(fn, what, names, q, k, inv_freq, positions, interleaved, amplitude, q_out, k_out,
          stream):
    torch = _torch()
    lead = k if q is None else q
    if lead is None:
        raise ValueError(f"{names[0]} or {names[1]} must be given")
    index = lead.get_device() if isinstance(lead, torch.Tensor) else -1
    _rows_tensor(lead, names[q is None], (3, 4), index)
    shape = lead.shape
    B, S, H, d = shape if len(shape) == 4 else (1, *shape)
    Hq, Hkv = (H, 0) if q is not None else (0, H)
    if q is not None and k is not None:
        _rows_tensor(k, names[1], (len(shape),), index)
        other = k.shape
        Hkv = other[-2]
        if other[0] != shape[0] or other[-1] != d or (len(shape) == 4 and other[1] != S):
            raise ValueError(f"{names[0]} and {names[1]} shapes disagree")
    rot = _frequencies(inv_freq, d, index)
    if positions is not None:
        _int_tensor(positions, "positions", index)
        if positions.numel() != B * S:
            raise ValueError(f"positions must hold {B * S} values")
    if stream is not None or index != _current_device():
        with _Call(index, stream):
            return _rope(fn, what, names, q, k, inv_freq, positions, interleaved, amplitude,
                         q_out, k_out, None)
    qp = kp = qo = ko = sq = sk = sqo = sko = None
    if q is not None:
        q_out = _output(q_out, q, names[0])
        qp, qo, sq, sqo = q.data_ptr(), q_out.data_ptr(), _strides(q, 3), _strides(q_out, 3)
    if k is not None:
        k_out = _output(k_out, k, names[1])
        kp, ko, sk, sko = k.data_ptr(), k_out.data_ptr(), _strides(k, 3), _strides(k_out, 3)
    rc = fn(qp, kp, qo, ko, None if positions is None else positions.data_ptr(),
            inv_freq.data_ptr(), B, S, Hq, Hkv, d, rot, 1 if interleaved else 0, amplitude, sq, sk,
            sqo, sko, _raw_stream(index))
    if rc != ATTN_OK:
        raise AttnError(rc, what)
    return q_out if q is not None else None, k_out if k is not None else None


def attn_append_paged(q, k, v, k_pages, v_pages, page_table, seqlens_k, cu_seqlens_q=None,
                      inv_freq=None, *, interleaved=False, amplitude=1.0, q_out=None, stream=None):
    """New tokens of a serving step: k, v [T,Hkv,d] written to their slots of the paged
    cache k_pages, v_pages [P,16,Hkv,d], k rotated on the way; returns q [T,Hq,d]
    rotated (None if q is None).  page_table [B,maxP], seqlens_k [B] (lengths WITH
    the new tokens) and cu_seqlens_q [B+1] int32; without cu_seqlens_q every
    sequence has one new token (T = B).  inv_freq None: nothing is rotated."""
    torch = _torch()
    index = k.get_device() if isinstance(k, torch.Tensor) else -1
    _rows_tensor(k, "k", (3,), index)
    _rows_tensor(v, "v", (3,), index)
    _rows_tensor(k_pages, "k_pages", (4,), index)
    _rows_tensor(v_pages, "v_pages", (4,), index)
    T, Hkv, d = k.shape
    P, page, Hp, dp = pool = k_pages.shape
    if v.shape != k.shape or Hp != Hkv or dp != d or v_pages.shape != pool:
        raise ValueError("k, v, k_pages and v_pages shapes disagree")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    _int_tensor(seqlens_k, "seqlens_k", index)
    B = seqlens_k.numel()
    _int_vector(seqlens_k, "seqlens_k", B, index)
    _int_tensor(page_table, "page_table", index)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages]")
    W = page_table.shape[1]
    if cu_seqlens_q is not None:
        _int_vector(cu_seqlens_q, "cu_seqlens_q", B + 1, index)
    elif T != B:
        raise ValueError("without cu_seqlens_q every sequence has one new token")
    Hq = 0
    if q is not None:
        _rows_tensor(q, "q", (3,), index)
        Tq, Hq, dq = q.shape
        if Tq != T or dq != d:
            raise ValueError("q and k shapes disagree")
    rot = 0 if inv_freq is None else _frequencies(inv_freq, d, index)
    if stream is not None or index != _current_device():
        with _Call(index, stream):
            return attn_append_paged(q, k, v, k_pages, v_pages, page_table, seqlens_k,
                                     cu_seqlens_q, inv_freq, interleaved=interleaved,
                                     amplitude=amplitude, q_out=q_out)
    if B > _INT_MAX or T > _INT_MAX or W > _INT_MAX:
        B, T, W = _c_int(B), _c_int(T), _c_int(W)
    qp = qo = sq = sqo = None
    if q is not None:
        q_out = _output(q_out, q, "q")
        qp, qo, sq, sqo = q.data_ptr(), q_out.data_ptr(), _strides(q, 2), _strides(q_out, 2)
    rc = lib.attn_append_paged(
        qp, k.data_ptr(), v.data_ptr(), qo, k_pages.data_ptr(), v_pages.data_ptr(),
        page_table.data_ptr(), _ptr(cu_seqlens_q), seqlens_k.data_ptr(), _ptr(inv_freq), B, Hq,
        Hkv, T, d, rot, 1 if interleaved else 0, amplitude, page, W, P, sq, _strides(k, 2),
        _strides(v, 2), sqo, _raw_stream(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_append_paged")
    return q_out if q is not None else None


@functools.lru_cache(maxsize=256)
def attn_pages_workspace_size(rows: int, num_pages: int) -> int:
    return int(lib.attn_pages_workspace_size(_c_int(int(rows)), _c_int(int(num_pages))))


def _cache_tables(page_table, seqlens, refs):
    """(device index, B, max_pages, P)"""
    torch = _torch()
    index = refs.get_device() if isinstance(refs, torch.Tensor) else -1
    if index < 0:
        raise ValueError("refs must be a CUDA tensor")
    _int_tensor(refs, "refs", index)
    _int_tensor(page_table, "page_table", index)
    if page_table.dim() != 2 or refs.dim() != 1:
        raise ValueError("page_table must be [B, max_pages], refs [P]")
    B, W = page_table.shape
    _int_vector(seqlens, "seqlens", B, index)
    P = refs.numel()
    if B > _INT_MAX or W > _INT_MAX or P > _INT_MAX:
        B, W, P = _c_int(B), _c_int(W), _c_int(P)
    return index, B, W, P


def _cache_pools(k_pages, v_pages, pages, index):
    """(layers, page size, Hkv, d) of pools [layers, P, 16, Hkv, d] or [P, 16, Hkv, d]."""
    _rows_tensor(k_pages, "k_pages", (4, 5), index)
    _rows_tensor(v_pages, "v_pages", (4, 5), index)
    shape = k_pages.shape
    layers, P, page, Hkv, d = shape if len(shape) == 5 else (1, *shape)
    if v_pages.shape != shape or P != pages:
        raise ValueError(f"k_pages and v_pages must hold the {pages} pages that refs counts")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    return layers, page, Hkv, d


@functools.lru_cache(maxsize=256)
def _vector_like(n, dtype, index):
    """A vector of n that holds no memory, only its shape: empty_like of it costs the host
    about a microsecond less than empty with a size, a type and a device.  The one element
    it is spread from goes back at once, so nothing stays allocated here, whatever pool
    (a capture's, say) it came from."""
    torch = _torch()
    t = torch.empty(1, dtype=dtype, device=torch.device("cuda", index)).expand(n)
    t.untyped_storage().resize_(0)
    return t


def _workspace(workspace, rows, pages, refs):
    torch = _torch()
    if workspace is None:
        return torch.empty_like(_vector_like(attn_pages_workspace_size(rows, pages), torch.uint8,
                                             refs.get_device()))
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or \
            workspace.get_device() != refs.get_device():
        raise ValueError(f"workspace must be a contiguous tensor on {refs.device}")
    return workspace


def attn_pages_resize(page_table, seqlens, new_seqlens, refs, k_pages=None, v_pages=None, *,
                      workspace=None, stream=None) -> None:
    """Sets every row's length, in place: pages past a shorter row's end are given back
    (0 frees the row), a longer row gets the lowest free pages; one that grows
    inside a last page it shares gets a copy of that page first.  page_table
    [B,maxP], seqlens, new_seqlens [B], refs [P] int32; k_pages, v_pages [P,16,Hkv,d]
    or [layers,P,16,Hkv,d], None for a cache that shares no pages.  A row that finds
    too few free pages keeps its length (ATTN_ERR_NO_PAGES)."""
    index, B, W, P = _cache_tables(page_table, seqlens, refs)
    _int_vector(new_seqlens, "new_seqlens", B, index)
    layers, page, Hkv, d = 1, 16, 1, 64
    if k_pages is not None or v_pages is not None:
        if k_pages is None or v_pages is None:
            raise ValueError("k_pages and v_pages must both be given, or neither")
        layers, page, Hkv, d = _cache_pools(k_pages, v_pages, P, index)
    if stream is not None or index != _current_device():
        with _Call(index, stream):
            return attn_pages_resize(page_table, seqlens, new_seqlens, refs, k_pages, v_pages,
                                     workspace=workspace)
    ws = _workspace(workspace, B, P, refs)
    rc = lib.attn_pages_resize(
        page_table.data_ptr(), seqlens.data_ptr(), new_seqlens.data_ptr(), refs.data_ptr(),
        _ptr(k_pages), _ptr(v_pages), B, layers, Hkv, d, page, W, P, ws.data_ptr(), ws.nbytes,
        _raw_stream(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_pages_resize")


def attn_pages_fork(page_table, seqlens, refs, src, dst, k_pages, v_pages, *, workspace=None,
                    stream=None) -> None:
    """Rows dst [n] become copies of rows src [n] (int32), in place: whole pages shared,
    a last page that is not full copied in every layer.  Rows dst must be empty
    (length 0).  Other arguments as attn_pages_resize's."""
    index, B, W, P = _cache_tables(page_table, seqlens, refs)
    _int_tensor(src, "src", index)
    n = src.numel()
    _int_vector(src, "src", n, index)
    _int_vector(dst, "dst", n, index)
    if n > _INT_MAX:
        n = _c_int(n)
    layers, page, Hkv, d = _cache_pools(k_pages, v_pages, P, index)
    if stream is not None or index != _current_device():
        with _Call(index, stream):
            return attn_pages_fork(page_table, seqlens, refs, src, dst, k_pages, v_pages,
                                   workspace=workspace)
    ws = _workspace(workspace, n, P, refs)
    rc = lib.attn_pages_fork(
        page_table.data_ptr(), seqlens.data_ptr(), refs.data_ptr(), src.data_ptr(),
        dst.data_ptr(), n, k_pages.data_ptr(), v_pages.data_ptr(), B, layers, Hkv, d, page, W, P,
        ws.data_ptr(), ws.nbytes, _raw_stream(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_pages_fork")


def attn_pages_compact(page_table, seqlens, refs, k_pages, v_pages, *, workspace=None,
                       stream=None):
    """Moves the live pages (refs > 0) to the front of the pool, in place, in every layer,
    and renames them in the table -> (new_index [P], num_live [1]) int32: where each
    page is now (-1: free) and how many are live."""
    index, B, W, P = _cache_tables(page_table, seqlens, refs)
    layers, page, Hkv, d = _cache_pools(k_pages, v_pages, P, index)
    if stream is not None or index != _current_device():
        with _Call(index, stream):
            return attn_pages_compact(page_table, seqlens, refs, k_pages, v_pages,
                                      workspace=workspace)
    torch = _torch()
    ws = _workspace(workspace, 0, P, refs)
    new_index = torch.empty_like(refs)
    num_live = torch.empty_like(_vector_like(1, torch.int32, index))
    rc = lib.attn_pages_compact(
        page_table.data_ptr(), seqlens.data_ptr(), refs.data_ptr(), new_index.data_ptr(),
        num_live.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), B, layers, Hkv, d, page, W,
        P, ws.data_ptr(), ws.nbytes, _raw_stream(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_pages_compact")
    return new_index, num_live


def attn_device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word."""
    return int(lib.attn_device_status(_stream(stream)))


def attn_check_wait_timeout(limit_us: int, stream=None) -> None:
    _check(lib.attn_check_wait_timeout(int(limit_us), _stream(stream)), "attn_check_wait_timeout")
