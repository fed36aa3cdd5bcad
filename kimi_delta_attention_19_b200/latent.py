"""Latent attention: the global-attention layer beside KDA layers, over the C ABI's
kda_latent_* calls (include/kda.h).

A token keeps one latent vector c (512) and a shared key part k_pe (64) for all heads.

    latent_attention            expanded form with gradients (training)
    latent_attn_fwd / _bwd      the same, as explicit calls
    latent_decode               absorbed form over the paged cache: a token or drafted tokens
                                of each sequence
    latent_cache                a paged cache, bf16 or with the latent in 8 bits
    latent_cache_write / _read  tokens into the cache and back

Argument marshalling only: the computation runs in libkda.so's kernels, on the tensors'
device and on `stream` (default: that device's current stream).
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import kda
from .kda import KDA_BF16, KDA_ERR_INVALID_ARG, KDA_OK, KdaError, lib

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
    for name in ("attn_fwd", "attn_bwd", "cache_write", "cache_read", "decode"):
        getattr(L, "kda_latent_" + name).restype = ctypes.c_int


_declare(lib)

EXPORTED = ("kda_latent_attn_fwd", "kda_latent_attn_bwd_workspace_size", "kda_latent_attn_bwd",
            "kda_latent_cache_write", "kda_latent_cache_read",
            "kda_latent_decode_workspace_size", "kda_latent_decode")


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _bf16(t: torch.Tensor, name: str) -> None:
    if t.dtype != torch.bfloat16:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}: latent attention takes bfloat16")


def _typed(t: torch.Tensor | None, dtype: torch.dtype, shape, name: str, like: torch.Tensor):
    """Checks an optional contiguous tensor argument on `like`'s device."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if shape is not None:
        _need(tuple(t.shape) == tuple(shape),
              f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    _need(t.device == like.device, f"{name} is on {t.device}, not on {like.device}")


def _addr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@contextlib.contextmanager
def _on(t: torch.Tensor, stream):
    """The tensors' device and the stream of the call, current while scratch is allocated."""
    _need(t.is_cuda, f"latent attention needs CUDA tensors (got {t.device})")
    with torch.cuda.device(t.device):
        if stream is None:
            yield ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        else:
            with torch.cuda.stream(stream):
                yield ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, what: str) -> None:
    if rc != KDA_OK:
        raise KdaError(rc, what)


# ------------------------------------------------------------------------ expanded form
def _attn_shape(q, k_nope, k_pe, v, cu_q, cu_k, max_q, max_k, causal, scale):
    for t, name in ((q, "q"), (k_nope, "k_nope"), (k_pe, "k_pe"), (v, "v")):
        _bf16(t, name)
        _need(t.device == q.device, f"{name} is on {t.device}, not on {q.device}")
    batched = q.dim() == 4
    _need(q.dim() in (3, 4) and k_nope.dim() == q.dim() and v.dim() == q.dim()
          and k_pe.dim() == q.dim() - 1, "q, k_nope, v must be [T, H, d] or [B, T, H, d] and "
          "k_pe [T, d] or [B, T, d]")
    H = q.shape[-2]
    lead_k = tuple(k_nope.shape[:-2])
    _need(k_nope.shape[-2] == H and v.shape[-2] == H and tuple(v.shape[:-2]) == lead_k
          and tuple(k_pe.shape[:-1]) == lead_k
          and (not batched or q.shape[0] == k_nope.shape[0]),
          f"shapes do not agree: q {tuple(q.shape)}, k_nope {tuple(k_nope.shape)}, "
          f"k_pe {tuple(k_pe.shape)}, v {tuple(v.shape)}")
    _need(q.shape[-1] == k_nope.shape[-1] + k_pe.shape[-1],
          "q's channels must be k_nope's and k_pe's together")
    _need((cu_q is None) == (cu_k is None) and not (batched and cu_q is not None),
          "cu_seqlens takes packed [T, H, d] inputs, for queries and keys alike")
    if cu_q is not None:
        _typed(cu_q, torch.int32, None, "cu_seqlens", q)
        _typed(cu_k, torch.int32, cu_q.shape, "cu_seqlens_k", q)
        _need(cu_q.dim() == 1 and cu_q.numel() >= 2, "cu_seqlens must hold n_seqs + 1 offsets")

    def strides(t, name, head=True):
        s = t.stride()
        _need(s[-1] == 1 or t.shape[-1] == 1, f"{name}'s channels must be contiguous")
        token = s[-3] if head else s[-2]
        if batched:   # sequence after sequence
            _need(t.shape[0] == 1 or s[0] == token * t.shape[1] or t.numel() == 0,
                  f"{name}'s sequences must follow each other (strides {s})")
        # of a dimension of one the stride says nothing
        hs = (s[-2] if t.shape[-2] > 1 else t.shape[-1]) if head else 0
        n = t.shape[-3] if head else t.shape[-2]
        if n <= 1 and not (batched and t.shape[0] > 1):
            token = max(hs * (t.shape[-2] if head else 0), t.shape[-1])
        return token, hs

    qt, qh = strides(q, "q")
    kt, kh = strides(k_nope, "k_nope")
    vt, vh = strides(v, "v")
    pt, _ = strides(k_pe, "k_pe", head=False)
    return LatentShape(B=q.shape[0] if batched else 1, H=H, Tq=q.shape[-3], Tk=k_nope.shape[-3],
                       n_seqs=0 if cu_q is None else cu_q.numel() - 1, max_q=int(max_q),
                       max_k=int(max_k), d_nope=k_nope.shape[-1], d_pe=k_pe.shape[-1],
                       d_v=v.shape[-1], q_token=qt, q_head=qh, k_token=kt, k_head=kh,
                       pe_token=pt, v_token=vt, v_head=vh, causal=int(bool(causal)),
                       dtype=KDA_BF16, scale=0.0 if scale is None else float(scale))


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
    smaller). causal: query i sees keys up to its own position, the queries being the last
    tokens of their sequence.

    Returns (out [T, H, 128], lse [T, H] fp32, natural log). Rows that see no key have
    out = 0, lse = -inf; packed rows behind the last sequence are not written.
    """
    if cu_seqlens is not None and cu_seqlens_k is None:
        cu_seqlens_k, max_seqlen_k = cu_seqlens, max_seqlen_k or max_seqlen
    s = _attn_shape(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k, max_seqlen, max_seqlen_k,
                    causal, scale)
    lead = tuple(q.shape[:-1])
    _typed(out, torch.bfloat16, lead + (v.shape[-1],), "out", q)
    _typed(lse, torch.float32, lead, "lse", q)
    _typed(status, torch.int32, None, "status", q)
    with _on(q, stream) as st:
        if out is None:
            out = torch.empty(lead + (v.shape[-1],), dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty(lead, dtype=torch.float32, device=q.device)
        _check(lib.kda_latent_attn_fwd(_addr(q), _addr(k_nope), _addr(k_pe), _addr(v),
                                       _addr(cu_seqlens), _addr(cu_seqlens_k), _addr(out),
                                       _addr(lse), ctypes.byref(s), _addr(status), st),
               "kda_latent_attn_fwd")
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
    s = _attn_shape(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k, max_seqlen, max_seqlen_k,
                    causal, scale)
    lead = tuple(q.shape[:-1])
    _typed(out, torch.bfloat16, lead + (v.shape[-1],), "out", q)
    _typed(lse, torch.float32, lead, "lse", q)
    _typed(d_out, torch.bfloat16, lead + (v.shape[-1],), "d_out", q)
    _typed(status, torch.int32, None, "status", q)
    _typed(workspace, torch.uint8, None, "workspace", q)
    names = (("dq", q), ("dk_nope", k_nope), ("dk_pe", k_pe), ("dv", v))
    if grads is not None:
        _need(len(grads) == 4, "grads must be (dq, dk_nope, dk_pe, dv)")
        for g, (name, like) in zip(grads, names):
            _typed(g, torch.bfloat16, like.shape, name, q)
    with _on(q, stream) as st:
        if grads is None:
            grads = tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device)
                          for _, t in names)
        if workspace is None:
            nbytes = int(lib.kda_latent_attn_bwd_workspace_size(ctypes.byref(s)))
            if nbytes == 0:
                raise KdaError(KDA_ERR_INVALID_ARG, "kda_latent_attn_bwd_workspace_size")
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _check(lib.kda_latent_attn_bwd(_addr(q), _addr(k_nope), _addr(k_pe), _addr(v),
                                       _addr(out), _addr(lse), _addr(d_out), _addr(cu_seqlens),
                                       _addr(cu_seqlens_k), *(_addr(g) for g in grads),
                                       ctypes.byref(s), _addr(workspace), workspace.numel(),
                                       _addr(status), st), "kda_latent_attn_bwd")
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
        q, k_nope, k_pe, v, out, lse, cu_q, cu_k = ctx.saved_tensors
        grads = tuple(torch.zeros(t.shape, dtype=t.dtype, device=t.device)
                      for t in (q, k_nope, k_pe, v)) if cu_q is not None else None
        return latent_attn_bwd(q, k_nope, k_pe, v, out, lse, d_out.contiguous(),
                               cu_seqlens=cu_q, cu_seqlens_k=cu_k, grads=grads,
                               **ctx.opts) + (None, None, None)


def latent_attention(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor,
                     *, cu_seqlens: torch.Tensor | None = None,
                     cu_seqlens_k: torch.Tensor | None = None, max_seqlen: int = 0,
                     max_seqlen_k: int = 0, causal: bool = True,
                     scale: float | None = None) -> torch.Tensor:
    """Differentiable expanded latent attention: out as latent_attn_fwd returns it, with
    gradients for q, k_nope, k_pe and v. Packed rows behind the last sequence come out as
    zeros, in out and in the gradients."""
    if cu_seqlens is not None and cu_seqlens_k is None:
        cu_seqlens_k, max_seqlen_k = cu_seqlens, max_seqlen_k or max_seqlen
    return _LatentAttention.apply(q, k_nope, k_pe, v, cu_seqlens, cu_seqlens_k,
                                  dict(max_seqlen=max_seqlen, max_seqlen_k=max_seqlen_k,
                                       causal=causal, scale=scale))


# -------------------------------------------------------------------------------- cache
def latent_cache(n_pages: int, page_size: int = 64, *, quantized: bool = False,
                 device="cuda") -> torch.Tensor:
    """A paged cache, zeros: bf16 [n_pages, page_size, 576], or with `quantized` 8-bit rows,
    uint8 [n_pages, page_size, 656]. page_size is 16, 32, 64 or 128."""
    _need(page_size in (16, 32, 64, 128), f"page_size must be 16, 32, 64 or 128 ({page_size})")
    if quantized:
        return torch.zeros(n_pages, page_size, E4M3_ROW_BYTES, dtype=torch.uint8, device=device)
    return torch.zeros(n_pages, page_size, D_C + D_PE, dtype=torch.bfloat16, device=device)


def _cache_shape(cache: torch.Tensor) -> CacheShape:
    _need(cache.dim() == 3, f"cache must be [n_pages, page_size, row] (got {tuple(cache.shape)})")
    fmt, row = {torch.bfloat16: (CACHE_BF16, D_C + D_PE),
                torch.uint8: (CACHE_E4M3, E4M3_ROW_BYTES)}.get(cache.dtype, (None, 0))
    if fmt is None:
        raise TypeError(f"unsupported cache dtype {cache.dtype}: bfloat16 or uint8 rows")
    _need(cache.shape[2] == row, f"a {cache.dtype} cache row has {row} values "
          f"(got {cache.shape[2]})")
    _need(cache.is_contiguous(), "cache must be contiguous")
    return CacheShape(n_pages=cache.shape[0], page_size=cache.shape[1], d_c=D_C, d_pe=D_PE,
                      format=fmt)


def latent_cache_write(latent: torch.Tensor, k_pe: torch.Tensor, cache: torch.Tensor,
                       slots: torch.Tensor, *, status: torch.Tensor | None = None,
                       stream=None) -> None:
    """Writes tokens into the cache: latent [T, 512] and k_pe [T, 64] (bf16, rows possibly
    strided) to rows slots [T] (int64: page * page_size + offset). Negative slots are
    skipped (padding); one past the cache is skipped and reported as 3 in `status` (int32
    device tensor). Slots must be distinct."""
    cs = _cache_shape(cache)
    for t, name, d in ((latent, "latent", D_C), (k_pe, "k_pe", D_PE)):
        _bf16(t, name)
        _need(t.dim() == 2 and t.shape[1] == d and t.stride(1) == 1,
              f"{name} must be [T, {d}] with contiguous channels")
        _need(t.device == cache.device, f"{name} is on {t.device}, not on {cache.device}")
    T = latent.shape[0]
    _need(k_pe.shape[0] == T, "latent and k_pe must have the same tokens")
    _typed(slots, torch.int64, (T,), "slots", cache)
    _typed(status, torch.int32, None, "status", cache)
    strides = [t.stride(0) if T > 1 else t.shape[1] for t in (latent, k_pe)]
    with _on(cache, stream) as st:
        _check(lib.kda_latent_cache_write(_addr(latent), strides[0], _addr(k_pe), strides[1],
                                          _addr(slots), T, _addr(cache), ctypes.byref(cs),
                                          _addr(status), st), "kda_latent_cache_write")


def latent_cache_read(cache: torch.Tensor, block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                      *, total: int | None = None, starts: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Reads cached tokens back, packed: sequence s's tokens from starts[s] (default 0) on go
    to rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 of the result [total, 576] bf16 (latent,
    then k_pe), for instance to expand a cached prefix in front of new queries. block_table
    is int32 [n, pages]. A token past its table or with a page out of range is NaN and
    reported as 3 in `status`; rows behind the last sequence are not written."""
    cs = _cache_shape(cache)
    _typed(cu_seqlens, torch.int32, None, "cu_seqlens", cache)
    _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2,
          "cu_seqlens must hold n_seqs + 1 offsets")
    n = cu_seqlens.numel() - 1
    _typed(block_table, torch.int32, None, "block_table", cache)
    _need(block_table.dim() == 2 and block_table.shape[0] == n,
          f"block_table must be [{n}, pages] (got {tuple(block_table.shape)})")
    _typed(starts, torch.int32, (n,), "starts", cache)
    _typed(status, torch.int32, None, "status", cache)
    _need(total is not None or out is not None, "total (rows of the result) or out is needed")
    if out is not None:
        _typed(out, torch.bfloat16, (out.shape[0] if total is None else total, D_C + D_PE),
               "out", cache)
    with _on(cache, stream) as st:
        if out is None:
            out = torch.empty(total, D_C + D_PE, dtype=torch.bfloat16, device=cache.device)
        _check(lib.kda_latent_cache_read(_addr(cache), _addr(block_table), block_table.shape[1],
                                         _addr(cu_seqlens), _addr(starts), n, out.shape[0],
                                         _addr(out), ctypes.byref(cs), _addr(status), st),
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
    where bit j of draft_mask[n, i] is set.

    Returns out like q with 512 channels (the value projection is the caller's); `lse`
    (fp32, q's leading shape) receives the natural log-sum-exp. A row that sees nothing has
    out = 0, lse = -inf. seq_lens past the table or a page out of range: NaN rows and 3 in
    `status`. `workspace` may be kept (latent_decode_workspace); it serves one call at a time.
    """
    cs = _cache_shape(cache)
    _bf16(q, "q")
    _need(q.dim() in (3, 4) and q.shape[-1] == D_C + D_PE,
          f"q must be [N, H, {D_C + D_PE}] or [N, L, H, {D_C + D_PE}] (got {tuple(q.shape)})")
    N, L, H = q.shape[0], q.shape[1] if q.dim() == 4 else 1, q.shape[-2]
    lead = tuple(q.shape[:-1])
    _typed(q, torch.bfloat16, None, "q", cache)
    _typed(block_table, torch.int32, None, "block_table", cache)
    _need(block_table.dim() == 2 and block_table.shape[0] == N,
          f"block_table must be [{N}, pages] (got {tuple(block_table.shape)})")
    _typed(seq_lens, torch.int32, (N,), "seq_lens", cache)
    _typed(draft_mask, torch.int64, (N, L), "draft_mask", cache)
    _typed(out, torch.bfloat16, lead + (D_C,), "out", cache)
    _typed(lse, torch.float32, lead, "lse", cache)
    _typed(workspace, torch.uint8, None, "workspace", cache)
    _typed(status, torch.int32, None, "status", cache)
    s = DecodeShape(N=N, L=L, H=H, table_pages=block_table.shape[1], dtype=KDA_BF16,
                    scale=0.0 if scale is None else float(scale))
    with _on(cache, stream) as st:
        if out is None:
            out = torch.empty(lead + (D_C,), dtype=torch.bfloat16, device=q.device)
        if workspace is None:
            workspace = _decode_workspace(s, cs, q.device)
        _check(lib.kda_latent_decode(_addr(q), _addr(cache), _addr(block_table),
                                     _addr(seq_lens), _addr(draft_mask), _addr(out), _addr(lse),
                                     ctypes.byref(s), ctypes.byref(cs), _addr(workspace),
                                     workspace.numel(), _addr(status), st),
               "kda_latent_decode")
    return out


def _decode_workspace(s: DecodeShape, cs: CacheShape, device) -> torch.Tensor:
    n = int(lib.kda_latent_decode_workspace_size(ctypes.byref(s), ctypes.byref(cs)))
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_latent_decode_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def latent_decode_workspace(N: int, H: int, cache: torch.Tensor, *, L: int = 1) -> torch.Tensor:
    """Scratch for latent_decode calls of N sequences, L query tokens and H heads."""
    with torch.cuda.device(cache.device):
        return _decode_workspace(DecodeShape(N=N, L=L, H=H, dtype=KDA_BF16),
                                 _cache_shape(cache), cache.device)


status_of = kda.workspace_status   # (status, device code) of a status word
