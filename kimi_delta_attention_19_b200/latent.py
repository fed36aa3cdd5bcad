"""Latent attention: the global-attention layer beside KDA layers, over the C ABI's
kda_latent_* calls (include/kda.h).

A token keeps one latent vector c (512) and a shared key part k_pe (64) for all heads.

    latent_attention            expanded form with gradients (training)
    latent_attn_fwd / _bwd      the same, as explicit calls
    latent_decode               absorbed form over the paged cache: a token or drafted tokens
                                of each sequence
    latent_cache                a paged cache, bf16 or with the latent in 8 bits
    latent_cache_write / _read  tokens into the cache and back
    latent_status               what calls without a `status` tensor have reported

Argument marshalling only: the computation runs in libkda.so's kernels, on the tensors'
device and on `stream` (default: that device's current stream).
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import kda
from .kda import KDA_BF16, KDA_ERR_DEVICE, KDA_ERR_INVALID_ARG, KDA_OK, KdaError, lib

D_NOPE, D_PE, D_V, D_C = 128, 64, 128, 512
CACHE_BF16, CACHE_E4M3 = 0, 1
E4M3_ROW_BYTES = 656


class LatentShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Tq", ctypes.c_int64),
                ("Tk", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("max_q", ctypes.c_int64),
                ("max_k", ctypes.c_int64), ("d_nope", ctypes.c_int32), ("d_pe", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("pe_token", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("causal", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float)]


class CacheShape(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("d_c", ctypes.c_int32), ("d_pe", ctypes.c_int32), ("format", ctypes.c_int32)]


class DecodeShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("L", ctypes.c_int32), ("H", ctypes.c_int32),
                ("table_pages", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float)]


def _declare(L: ctypes.CDLL) -> None:
    p, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
    shape, cache = ctypes.POINTER(LatentShape), ctypes.POINTER(CacheShape)
    dec = ctypes.POINTER(DecodeShape)
    L.kda_latent_attn_fwd.argtypes = [p] * 8 + [shape, p, p]
    L.kda_latent_attn_bwd_workspace_size.argtypes = [shape]
    L.kda_latent_attn_bwd_workspace_size.restype = sz
    L.kda_latent_attn_bwd.argtypes = [p] * 13 + [shape, p, sz, p, p]
    L.kda_latent_cache_write.argtypes = [p, i64, p, i64, p, i64, p, cache, p, p]
    L.kda_latent_cache_read.argtypes = [p, p, i64, p, p, i32, i64, p, cache, p, p]
    L.kda_latent_decode_workspace_size.argtypes = [dec, cache]
    L.kda_latent_decode_workspace_size.restype = sz
    L.kda_latent_decode.argtypes = [p] * 7 + [dec, cache, p, sz, p, p]
    L.kda_latent_status.argtypes = [p, ctypes.POINTER(i32)]
    for name in ("attn_fwd", "attn_bwd", "cache_write", "cache_read", "decode", "status"):
        getattr(L, "kda_latent_" + name).restype = ctypes.c_int


_declare(lib)

EXPORTED = ("kda_latent_attn_fwd", "kda_latent_attn_bwd_workspace_size", "kda_latent_attn_bwd",
            "kda_latent_cache_write", "kda_latent_cache_read",
            "kda_latent_decode_workspace_size", "kda_latent_decode", "kda_latent_status")


# The checks of a call are plain conditions (messages are formed only when one fails), pointers
# and streams go to the library as integers and structs are filled by position: a call that
# launches one small kernel costs the host more than the GPU otherwise.
def _typed(t: torch.Tensor | None, dtype: torch.dtype, shape, name: str, index: int) -> int | None:
    """Checks an optional contiguous tensor argument on GPU `index`; its address."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors are not")
    return t.data_ptr()


def _bf16(t: torch.Tensor, name: str, index: int) -> None:
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}: latent attention takes bfloat16")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors are not")


# The usual calls (current device and stream, results allocated here, no status word) go through
# an extension module; where that answers None, or is not built, the checks below run and say
# what is wrong.
try:
    from . import _latent_host as _host
    _host.bind(*(ctypes.cast(getattr(lib, "kda_latent_" + n), ctypes.c_void_p).value
                 for n in ("attn_fwd", "attn_bwd", "attn_bwd_workspace_size", "cache_write",
                           "cache_read", "decode", "decode_workspace_size")))
except ImportError:
    _host = None

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


def _elsewhere(index: int, stream) -> bool:
    """Whether a call on GPU `index` and `stream` has to make them current first."""
    if index < 0:
        raise ValueError("latent attention needs CUDA tensors")
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream is one of {stream.device}, the tensors are on cuda:{index}")
    return stream is not None or torch.cuda.current_device() != index


@contextlib.contextmanager
def _there(index: int, stream):
    with torch.cuda.device(index):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _scale(scale: float | None) -> float:
    """The library's scale, where 0 selects the default: None, and no number, stands for that."""
    if scale is None:
        return 0.0
    s = ctypes.c_float(scale).value
    if not 0.0 < s < math.inf:
        raise ValueError(f"scale must be positive and finite in fp32 ({scale})")
    return s


def _check(rc: int, what: str) -> None:
    if rc != KDA_OK:
        raise KdaError(rc, what)


# ------------------------------------------------------------------------ expanded form
def _strides(t: torch.Tensor, name: str, batched: bool):
    """(token, head) strides of [.., T, H, d], or (token, 0) of k_pe [.., T, d], in elements."""
    st, shape = t.stride(), t.shape
    if len(shape) == 3 and shape[0] > 1 and shape[1] > 1 and st[2] == 1 and name != "k_pe":
        return st[0], st[1]
    head = name != "k_pe"
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    token = st[-3] if head else st[-2]
    if batched and shape[1] == 1:    # one token of each sequence: they lie as the sequences do
        token = st[0]
    if batched and shape[0] != 1 and st[0] != token * shape[1] and t.numel() != 0:
        raise ValueError(f"{name}'s sequences must follow each other (strides {st})")
    # of a dimension of one the stride says nothing
    hs = (st[-2] if shape[-2] > 1 else shape[-1]) if head else 0
    if (shape[-3] if head else shape[-2]) <= 1 and not (batched and shape[0] > 1):
        token = max(hs * (shape[-2] if head else 0), shape[-1])
    return token, hs


def _attn_shape(q, k_nope, k_pe, v, cu_q, cu_k, max_q, max_k, causal, scale, index):
    qs, ks, vs, ps = q.shape, k_nope.shape, v.shape, k_pe.shape
    _bf16(q, "q", index)
    _bf16(k_nope, "k_nope", index)
    _bf16(k_pe, "k_pe", index)
    _bf16(v, "v", index)
    dim = len(qs)
    batched = dim == 4
    if dim not in (3, 4) or len(ks) != dim or len(vs) != dim or len(ps) != dim - 1:
        raise ValueError("q, k_nope, v must be [T, H, d] or [B, T, H, d] and k_pe [T, d] or "
                         "[B, T, d]")
    H, Tk = qs[-2], ks[-3]
    if ks[-2] != H or vs[-2] != H or vs[-3] != Tk or ps[-2] != Tk or \
            (batched and not qs[0] == ks[0] == vs[0] == ps[0]):
        raise ValueError(f"shapes do not agree: q {tuple(qs)}, k_nope {tuple(ks)}, "
                         f"k_pe {tuple(ps)}, v {tuple(vs)}")
    if qs[-1] != ks[-1] + ps[-1]:
        raise ValueError("q's channels must be k_nope's and k_pe's together")
    if (cu_q is None) != (cu_k is None) or (batched and cu_q is not None):
        raise ValueError("cu_seqlens takes packed [T, H, d] inputs, for queries and keys alike")
    n_seqs = 0
    if cu_q is not None:
        if cu_q.dim() != 1 or cu_q.numel() < 2:
            raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
        _typed(cu_q, torch.int32, None, "cu_seqlens", index)
        if cu_k is not cu_q:
            _typed(cu_k, torch.int32, cu_q.shape, "cu_seqlens_k", index)
        n_seqs = cu_q.numel() - 1
    qt, qh = _strides(q, "q", batched)
    kt, kh = _strides(k_nope, "k_nope", batched)
    vt, vh = _strides(v, "v", batched)
    pt, _ = _strides(k_pe, "k_pe", batched)
    return LatentShape(qs[0] if batched else 1, H, qs[-3], Tk, n_seqs, int(max_q), int(max_k),
                       ks[-1], ps[-1], vs[-1], qt, qh, kt, kh, pt, vt, vh, int(bool(causal)),
                       KDA_BF16, _scale(scale))


def latent_attn_fwd(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor,
                    *, cu_seqlens: torch.Tensor | None = None,
                    cu_seqlens_k: torch.Tensor | None = None, max_seqlen: int = 0,
                    max_seqlen_k: int = 0, causal: bool = True, scale: float | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream=None):
    """Expanded latent attention. q [T, H, 192] (or [B, T, H, 192]); k_nope [Tk, H, 128] and
    v [Tk, H, 128], possibly views of one [Tk, H, 256] projection; k_pe [Tk, 64], shared by
    the heads. Packed sequences come with cu_seqlens (int32 [n + 1]) and, where the keys'
    lengths differ (a cached prefix before the queries), cu_seqlens_k; max_seqlen and
    max_seqlen_k bound the lengths (0: the packed totals; a tight bound makes the launch
    smaller). scale: None is 1/sqrt(192). causal: query i sees keys up to its own position, the queries being the last
    tokens of their sequence.

    Returns (out [T, H, 128], lse [T, H] fp32, natural log). Rows that see no key have
    out = 0, lse = -inf; packed rows behind the last sequence are not written. Neither are those
    of a sequence that is malformed or longer than its bound: `status` (int32 device tensor)
    receives 1, or without it what latent_status() tells.
    """
    if cu_seqlens is not None and cu_seqlens_k is None:
        cu_seqlens_k, max_seqlen_k = cu_seqlens, max_seqlen_k or max_seqlen
    if _host is not None and stream is None and out is None and lse is None and status is None:
        r = _host.attn_fwd(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k, max_seqlen, max_seqlen_k,
                           causal, scale)
        if r is not None:
            return r
    at = q.get_device()
    if _elsewhere(at, stream):
        with _there(at, stream):
            return latent_attn_fwd(q, k_nope, k_pe, v, cu_seqlens=cu_seqlens,
                                   cu_seqlens_k=cu_seqlens_k, max_seqlen=max_seqlen,
                                   max_seqlen_k=max_seqlen_k, causal=causal, scale=scale, out=out,
                                   lse=lse, status=status)
    s = _attn_shape(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k, max_seqlen, max_seqlen_k,
                    causal, scale, at)
    lead = q.shape[:-1]
    if out is None:
        out = q.new_empty(lead + v.shape[-1:])
    else:
        _typed(out, torch.bfloat16, lead + v.shape[-1:], "out", at)
    if lse is None:
        lse = q.new_empty(lead, dtype=torch.float32)
    else:
        _typed(lse, torch.float32, lead, "lse", at)
    _check(lib.kda_latent_attn_fwd(
        q.data_ptr(), k_nope.data_ptr(), k_pe.data_ptr(), v.data_ptr(), _addr(cu_seqlens),
        _addr(cu_seqlens_k), out.data_ptr(), lse.data_ptr(), ctypes.byref(s),
        _typed(status, torch.int32, None, "status", at), _raw_stream(at)), "kda_latent_attn_fwd")
    return out, lse


def latent_attn_bwd(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor,
                    out: torch.Tensor, lse: torch.Tensor, d_out: torch.Tensor, *,
                    cu_seqlens: torch.Tensor | None = None,
                    cu_seqlens_k: torch.Tensor | None = None, max_seqlen: int = 0,
                    max_seqlen_k: int = 0, causal: bool = True, scale: float | None = None,
                    grads: tuple | None = None, workspace: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream=None):
    """Gradients of latent_attn_fwd from its inputs, its out and lse, and d_out (contiguous):
    (dq, dk_nope, dk_pe, dv), contiguous, dk_pe summed over the heads. `grads` gives the four
    tensors to write into. Packed rows behind the last sequence are not written. The same
    inputs give the same bits. To capture a training step in a CUDA graph, capture this call
    and latent_attn_fwd."""
    if cu_seqlens is not None and cu_seqlens_k is None:
        cu_seqlens_k, max_seqlen_k = cu_seqlens, max_seqlen_k or max_seqlen
    if _host is not None and stream is None and grads is None and workspace is None \
            and status is None:
        r = _host.attn_bwd(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k, max_seqlen, max_seqlen_k,
                           causal, scale, out, lse, d_out)
        if r is not None:
            return r
    at = q.get_device()
    if _elsewhere(at, stream):
        with _there(at, stream):
            return latent_attn_bwd(q, k_nope, k_pe, v, out, lse, d_out, cu_seqlens=cu_seqlens,
                                   cu_seqlens_k=cu_seqlens_k, max_seqlen=max_seqlen,
                                   max_seqlen_k=max_seqlen_k, causal=causal, scale=scale,
                                   grads=grads, workspace=workspace, status=status)
    s = _attn_shape(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k, max_seqlen, max_seqlen_k,
                    causal, scale, at)
    lead = q.shape[:-1]
    out_p = _typed(out, torch.bfloat16, lead + v.shape[-1:], "out", at)
    lse_p = _typed(lse, torch.float32, lead, "lse", at)
    d_out_p = _typed(d_out, torch.bfloat16, lead + v.shape[-1:], "d_out", at)
    status_p = _typed(status, torch.int32, None, "status", at)
    like = (q, k_nope, k_pe, v)
    if grads is None:
        grads = tuple(q.new_empty(t.shape) for t in like)
    else:
        if len(grads) != 4:
            raise ValueError("grads must be (dq, dk_nope, dk_pe, dv)")
        for g, t, name in zip(grads, like, ("dq", "dk_nope", "dk_pe", "dv")):
            _typed(g, torch.bfloat16, t.shape, name, at)
    if workspace is None:
        nbytes = lib.kda_latent_attn_bwd_workspace_size(ctypes.byref(s))
        if nbytes == 0:
            raise KdaError(KDA_ERR_INVALID_ARG, "kda_latent_attn_bwd_workspace_size")
        workspace = q.new_empty(nbytes, dtype=torch.uint8)
    else:
        _typed(workspace, torch.uint8, None, "workspace", at)
    _check(lib.kda_latent_attn_bwd(
        q.data_ptr(), k_nope.data_ptr(), k_pe.data_ptr(), v.data_ptr(), out_p, lse_p, d_out_p,
        _addr(cu_seqlens), _addr(cu_seqlens_k), *(g.data_ptr() for g in grads), ctypes.byref(s),
        workspace.data_ptr(), workspace.numel(), status_p, _raw_stream(at)),
        "kda_latent_attn_bwd")
    return tuple(grads)


class _LatentAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k_nope, k_pe, v, cu_q, cu_k, opts):
        # packed rows behind the last sequence: zero here, in out and in every gradient
        out = torch.zeros(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device) \
            if cu_q is not None else None
        out, lse = latent_attn_fwd(q, k_nope, k_pe, v, cu_seqlens=cu_q, cu_seqlens_k=cu_k,
                                   out=out, **opts)
        ctx.save_for_backward(q, k_nope, k_pe, v, out, lse, cu_q, cu_k)
        ctx.opts = opts
        return out

    @staticmethod
    def backward(ctx, d_out):
        saved = ctx.saved_tensors
        grads = _Gradients.apply(d_out, *saved, ctx.opts) if torch.is_grad_enabled() \
            else _gradients(d_out, *saved, ctx.opts)
        return grads + (None, None, None)


def _gradients(d_out, q, k_nope, k_pe, v, out, lse, cu_q, cu_k, opts):
    grads = tuple(torch.zeros(t.shape, dtype=t.dtype, device=t.device)
                  for t in (q, k_nope, k_pe, v)) if cu_q is not None else None
    d_out = d_out.contiguous()
    if d_out.data_ptr() % 16:     # a part of a larger gradient, which autograd hands on as a view
        d_out = d_out.clone()
    return latent_attn_bwd(q, k_nope, k_pe, v, out, lse, d_out, cu_seqlens=cu_q,
                           cu_seqlens_k=cu_k, grads=grads, **opts)


class _Gradients(torch.autograd.Function):
    """_gradients under create_graph=True: a later pass through them raises, where it would
    otherwise take them for constants."""
    @staticmethod
    def forward(ctx, *args):
        return _gradients(*args)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("latent_attention offers no gradients of its gradients")


def latent_attention(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor,
                     *, cu_seqlens: torch.Tensor | None = None,
                     cu_seqlens_k: torch.Tensor | None = None, max_seqlen: int = 0,
                     max_seqlen_k: int = 0, causal: bool = True, scale: float | None = None,
                     status: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable expanded latent attention: out as latent_attn_fwd returns it, with
    gradients for q, k_nope, k_pe and v (gradients of gradients are refused). Packed rows
    behind the last sequence come out as zeros, in out and in the gradients, and so do those
    of a sequence that is skipped because cu_seqlens is malformed there or max_seqlen too
    small: reported as 1 in `status` (int32 device tensor), by the forward and the backward
    pass, or without one to latent_status()."""
    if cu_seqlens is not None and cu_seqlens_k is None:
        cu_seqlens_k, max_seqlen_k = cu_seqlens, max_seqlen_k or max_seqlen
    return _LatentAttention.apply(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k,
                                  dict(max_seqlen=max_seqlen, max_seqlen_k=max_seqlen_k,
                                       causal=causal, scale=scale, status=status))


# -------------------------------------------------------------------------------- cache
def latent_cache(n_pages: int, page_size: int = 64, *, quantized: bool = False,
                 device="cuda") -> torch.Tensor:
    """A paged cache, zeros: bf16 [n_pages, page_size, 576], or with `quantized` 8-bit rows,
    uint8 [n_pages, page_size, 656]. page_size is 16, 32, 64 or 128."""
    if page_size not in (16, 32, 64, 128):
        raise ValueError(f"page_size must be 16, 32, 64 or 128 ({page_size})")
    if quantized:
        return torch.zeros(n_pages, page_size, E4M3_ROW_BYTES, dtype=torch.uint8, device=device)
    return torch.zeros(n_pages, page_size, D_C + D_PE, dtype=torch.bfloat16, device=device)


_FORMATS = {torch.bfloat16: (CACHE_BF16, D_C + D_PE), torch.uint8: (CACHE_E4M3, E4M3_ROW_BYTES)}


def _cache_shape(cache: torch.Tensor) -> CacheShape:
    shape = cache.shape
    if len(shape) != 3:
        raise ValueError(f"cache must be [n_pages, page_size, row] (got {tuple(shape)})")
    fmt = _FORMATS.get(cache.dtype)
    if fmt is None:
        raise TypeError(f"unsupported cache dtype {cache.dtype}: bfloat16 or uint8 rows")
    if shape[2] != fmt[1]:
        raise ValueError(f"a {cache.dtype} cache row has {fmt[1]} values (got {shape[2]})")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return CacheShape(shape[0], shape[1], D_C, D_PE, fmt[0])


def latent_cache_write(latent: torch.Tensor, k_pe: torch.Tensor, cache: torch.Tensor,
                       slots: torch.Tensor, *, status: torch.Tensor | None = None,
                       stream=None) -> None:
    """Writes tokens into the cache: latent [T, 512] and k_pe [T, 64] (bf16, rows possibly
    strided) to rows slots [T] (int64: page * page_size + offset). Negative slots are
    skipped (padding); one past the cache is skipped and reported as 3 in `status` (int32
    device tensor). Slots must be distinct."""
    if _host is not None and stream is None and status is None:
        if _host.cache_write(latent, k_pe, cache, slots):
            return
    at = cache.get_device()
    if _elsewhere(at, stream):
        with _there(at, stream):
            return latent_cache_write(latent, k_pe, cache, slots, status=status)
    cs, T = _cache_shape(cache), latent.shape[0]
    for t, name, d in ((latent, "latent", D_C), (k_pe, "k_pe", D_PE)):
        _bf16(t, name, at)
        if t.dim() != 2 or t.shape[1] != d or t.stride(1) != 1:
            raise ValueError(f"{name} must be [T, {d}] with contiguous channels")
    if k_pe.shape[0] != T:
        raise ValueError("latent and k_pe must have the same tokens")
    _check(lib.kda_latent_cache_write(
        latent.data_ptr(), latent.stride(0) if T > 1 else D_C, k_pe.data_ptr(),
        k_pe.stride(0) if T > 1 else D_PE, _typed(slots, torch.int64, (T,), "slots", at), T,
        cache.data_ptr(), ctypes.byref(cs), _typed(status, torch.int32, None, "status", at),
        _raw_stream(at)), "kda_latent_cache_write")


def latent_cache_read(cache: torch.Tensor, block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                      *, total: int | None = None, starts: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Reads cached tokens back, packed: sequence s's tokens from starts[s] (default 0) on go
    to rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 of the result [total, 576] bf16 (latent,
    then k_pe), for instance to expand a cached prefix in front of new queries. block_table
    is int32 [n, pages]. A token past its table or with a page out of range is NaN and
    reported as 3 in `status`; rows behind the last sequence are not written."""
    if _host is not None and stream is None and out is None and starts is None and status is None:
        r = _host.cache_read(cache, block_table, cu_seqlens, total)
        if r is not None:
            return r
    at = cache.get_device()
    if _elsewhere(at, stream):
        with _there(at, stream):
            return latent_cache_read(cache, block_table, cu_seqlens, total=total, starts=starts,
                                     out=out, status=status)
    cs = _cache_shape(cache)
    cu_p = _typed(cu_seqlens, torch.int32, None, "cu_seqlens", at)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
    n = cu_seqlens.numel() - 1
    table_p = _typed(block_table, torch.int32, None, "block_table", at)
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError(f"block_table must be [{n}, pages] (got {tuple(block_table.shape)})")
    if out is not None:
        _typed(out, torch.bfloat16, (out.shape[0] if total is None else total, D_C + D_PE),
               "out", at)
    elif total is None:
        raise ValueError("total (rows of the result) or out is needed")
    else:
        out = cache.new_empty((total, D_C + D_PE), dtype=torch.bfloat16)
    _check(lib.kda_latent_cache_read(
        cache.data_ptr(), table_p, block_table.shape[1], cu_p,
        _typed(starts, torch.int32, (n,), "starts", at), n, out.shape[0], out.data_ptr(),
        ctypes.byref(cs), _typed(status, torch.int32, None, "status", at), _raw_stream(at)),
        "kda_latent_cache_read")
    return out


# -------------------------------------------------------------------------- absorbed form
def latent_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, *, draft_mask: torch.Tensor | None = None,
                  scale: float | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Absorbed latent attention of each sequence's last tokens over the paged cache.

    q [N, H, 576] (one token a sequence) or [N, L, H, 576] (its L <= 64 last tokens, e.g.
    drafted ones): the query with the key projection folded in, then its k_pe part.
    block_table int32 [N, pages]; seq_lens int32 [N] counts the cached tokens, the query
    tokens included (write them first). Query i sees the cache up to its own token; with
    draft_mask (int64 [N, L]) it sees all before the L last tokens and, of those, token j
    where bit j of draft_mask[n, i] is set. scale: None is that of the expanded head,
    1/sqrt(192).

    Returns out like q with 512 channels (the value projection is the caller's); `lse`
    (fp32, q's leading shape) receives the natural log-sum-exp. A row that sees nothing has
    out = 0, lse = -inf. seq_lens past the table or a page out of range: NaN rows and 3 in
    `status`. `workspace` may be kept (latent_decode_workspace); it serves one call at a time.
    """
    if _host is not None and stream is None and out is None and lse is None \
            and workspace is None and status is None:
        r = _host.decode(q, cache, block_table, seq_lens, draft_mask, scale)
        if r is not None:
            return r
    at = cache.get_device()
    if _elsewhere(at, stream):
        with _there(at, stream):
            return latent_decode(q, cache, block_table, seq_lens, draft_mask=draft_mask,
                                 scale=scale, out=out, lse=lse, workspace=workspace,
                                 status=status)
    cs, qs = _cache_shape(cache), q.shape
    _bf16(q, "q", at)
    dim = len(qs)
    if dim not in (3, 4) or qs[-1] != D_C + D_PE:
        raise ValueError(f"q must be [N, H, {D_C + D_PE}] or [N, L, H, {D_C + D_PE}] "
                         f"(got {tuple(qs)})")
    N, L, H = qs[0], qs[1] if dim == 4 else 1, qs[-2]
    lead = qs[:-1]
    q_p = _typed(q, torch.bfloat16, None, "q", at)
    table_p = _typed(block_table, torch.int32, None, "block_table", at)
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError(f"block_table must be [{N}, pages] (got {tuple(block_table.shape)})")
    s = DecodeShape(N, L, H, block_table.shape[1], KDA_BF16, _scale(scale))
    if out is None:
        out = q.new_empty(lead + (D_C,))
    else:
        _typed(out, torch.bfloat16, lead + (D_C,), "out", at)
    if workspace is None:
        workspace = _decode_workspace(s, cs, cache)
    else:
        _typed(workspace, torch.uint8, None, "workspace", at)
    _check(lib.kda_latent_decode(
        q_p, cache.data_ptr(), table_p, _typed(seq_lens, torch.int32, (N,), "seq_lens", at),
        _typed(draft_mask, torch.int64, (N, L), "draft_mask", at), out.data_ptr(),
        _typed(lse, torch.float32, lead, "lse", at), ctypes.byref(s), ctypes.byref(cs),
        workspace.data_ptr(), workspace.numel(), _typed(status, torch.int32, None, "status", at),
        _raw_stream(at)), "kda_latent_decode")
    return out


def _decode_workspace(s: DecodeShape, cs: CacheShape, cache: torch.Tensor) -> torch.Tensor:
    n = lib.kda_latent_decode_workspace_size(ctypes.byref(s), ctypes.byref(cs))
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_latent_decode_workspace_size")
    return cache.new_empty(n, dtype=torch.uint8)


def latent_decode_workspace(N: int, H: int, cache: torch.Tensor, *, L: int = 1) -> torch.Tensor:
    """Scratch for latent_decode calls of N sequences, L query tokens and H heads."""
    with torch.cuda.device(cache.device):
        return _decode_workspace(DecodeShape(N=N, L=L, H=H, dtype=KDA_BF16),
                                 _cache_shape(cache), cache)


status_of = kda.workspace_status   # (status, device code) of a status word


def latent_status(device=None, stream=None) -> tuple[int, int]:
    """(status, device code) of the calls on `device` (default: the current one) that were given
    no `status` tensor, since this was last asked: KDA_ERR_DEVICE and 1 for a malformed or too
    long sequence (left as it was, or zeros from latent_attention), 2 for an expired bounded
    wait, 3 for a page or slot out of range. Synchronises `stream` (default: the device's
    current one); calls on other streams are covered once those are done."""
    code = ctypes.c_int32(0)
    with torch.cuda.device(device):
        s = torch.cuda.current_stream() if stream is None else stream
        rc = lib.kda_latent_status(s.cuda_stream, ctypes.byref(code))
    if rc not in (KDA_OK, KDA_ERR_DEVICE):
        raise KdaError(rc, "kda_latent_status")
    return rc, code.value
