"""CPU tests of the latent-attention part of the C ABI and its binding: bad arguments are
refused before anything is launched (no GPU needed; addresses are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = ctypes.c_void_p
A = 4096 * 16                                   # an aligned address


@pytest.fixture(scope="module")
def latent():
    from kimi_delta_attention_19_b200 import latent as m
    return m


def shape(latent, **kw):
    s = dict(B=1, H=4, Tq=100, Tk=100, n_seqs=0, max_q=0, max_k=0, d_nope=128, d_pe=64, d_v=128,
             q_token=4 * 192, q_head=192, k_token=4 * 256, k_head=256, pe_token=64,
             v_token=4 * 256, v_head=256, causal=1, dtype=1, scale=0.0)
    s.update(kw)
    return latent.LatentShape(**s)


def fwd(latent, s, q=A, kn=A, kp=A, v=A, cq=None, ck=None, out=A, lse=A, status=None):
    return latent.lib.kda_latent_attn_fwd(q, kn, kp, v, cq, ck, out, lse, ctypes.byref(s), status,
                                          None)


INVALID, UNSUPPORTED = 1, 2


def codes(latent):
    from kimi_delta_attention_19_b200 import kda
    return kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


BAD_SHAPES = [
    (dict(H=0), 0), (dict(B=0), 0), (dict(Tq=-1), 0), (dict(Tk=-1), 0), (dict(max_q=-1), 0),
    (dict(n_seqs=2, B=2), 0), (dict(causal=2), 0), (dict(scale=-1.0), 0),
    (dict(scale=float("nan")), 0), (dict(scale=float("inf")), 0), (dict(dtype=7), 0),
    (dict(q_head=191), 0), (dict(q_head=128), 0), (dict(k_token=124), 0), (dict(pe_token=60), 0),
    (dict(v_head=260), 0), (dict(k_head=120), 0),
    (dict(dtype=0), 1), (dict(d_nope=64), 1), (dict(d_pe=32), 1), (dict(d_v=192), 1),
    (dict(H=65536), 1), (dict(B=65536), 1), (dict(Tq=1 << 31), 1), (dict(B=40000, Tk=60000), 1),
]


@pytest.mark.parametrize("bad,kind", BAD_SHAPES)
def test_expanded_shapes_are_refused(latent, bad, kind):
    want = codes(latent)[kind]
    s = shape(latent, **bad)
    assert fwd(latent, s) == want
    assert latent.lib.kda_latent_attn_bwd_workspace_size(ctypes.byref(s)) == 0
    rc = latent.lib.kda_latent_attn_bwd(*[A] * 7, None, None, *[A] * 4, ctypes.byref(s), A, 1 << 40,
                                        None, None)
    assert rc == want


def test_expanded_pointers_are_refused(latent):
    inv = codes(latent)[0]
    s, packed = shape(latent), shape(latent, n_seqs=2)
    for name in ("q", "kn", "kp", "v", "out"):
        assert fwd(latent, s, **{name: None}) == inv, name
        assert fwd(latent, s, **{name: A + 8}) == inv, name
    assert fwd(latent, s, lse=A + 2) == inv
    assert fwd(latent, s, status=A + 2) == inv
    assert fwd(latent, s, cq=A, ck=A) == inv                    # n_seqs = 0
    assert fwd(latent, packed) == inv                           # neither of the two
    assert fwd(latent, packed, cq=A) == inv and fwd(latent, packed, ck=A) == inv
    assert fwd(latent, packed, cq=A + 1, ck=A) == inv
    assert latent.lib.kda_latent_attn_fwd(*[A] * 4, None, None, A, A, None, None, None) == inv
    n = latent.lib.kda_latent_attn_bwd_workspace_size(ctypes.byref(s))
    assert n > 0 and n % 256 == 0

    def bwd(ws=A, wsb=n, **kw):
        p = dict(q=A, kn=A, kp=A, v=A, out=A, lse=A, g=A, dq=A, dkn=A, dkp=A, dv=A)
        p.update(kw)
        return latent.lib.kda_latent_attn_bwd(p["q"], p["kn"], p["kp"], p["v"], p["out"], p["lse"],
                                              p["g"], None, None, p["dq"], p["dkn"], p["dkp"],
                                              p["dv"], ctypes.byref(s), ws, wsb, None, None)

    for name in ("q", "kn", "kp", "v", "out", "lse", "g", "dq", "dkn", "dkp", "dv"):
        assert bwd(**{name: None}) == inv, name
        assert bwd(**{name: A + 1}) == inv, name
    assert bwd(ws=None) == inv and bwd(ws=A + 128) == inv and bwd(wsb=n - 1) == inv


def test_nothing_to_do_is_not_an_error(latent):
    """Zero tokens launch nothing (and need no GPU)."""
    from kimi_delta_attention_19_b200 import kda
    assert fwd(latent, shape(latent, Tq=0), q=None, out=None, lse=None) == kda.KDA_OK
    cs = latent.CacheShape(4, 16, 512, 64, 0)
    assert latent.lib.kda_latent_cache_write(None, 512, None, 64, None, 0, None, ctypes.byref(cs),
                                             None, None) == kda.KDA_OK
    assert latent.lib.kda_latent_cache_read(None, None, 0, None, None, 1, 0, None, ctypes.byref(cs),
                                            None, None) == kda.KDA_OK


def test_cache_arguments_are_refused(latent):
    inv, uns = codes(latent)

    def write(c=A, ct=512, pe=A, pt=64, slots=A, T=5, cache=A, cs=None, **kw):
        d = dict(n_pages=4, page_size=16, d_c=512, d_pe=64, format=0)
        d.update(kw)
        return latent.lib.kda_latent_cache_write(c, ct, pe, pt, slots, T, cache,
                                                 ctypes.byref(latent.CacheShape(**d)), None, None)

    for kw, want in ((dict(T=-1), inv), (dict(ct=504), inv), (dict(ct=516), inv), (dict(pt=60), inv),
                     (dict(c=None), inv), (dict(c=A + 8), inv), (dict(pe=None), inv),
                     (dict(slots=None), inv), (dict(slots=A + 4), inv), (dict(cache=None), inv),
                     (dict(cache=A + 8), inv), (dict(n_pages=-1), inv), (dict(page_size=0), inv),
                     (dict(format=2), inv), (dict(page_size=24), uns), (dict(page_size=256), uns),
                     (dict(d_c=256), uns), (dict(d_pe=128), uns), (dict(n_pages=1 << 28), uns),
                     (dict(T=1 << 31), uns)):
        assert write(**kw) == want, kw

    def read(cache=A, table=A, pages=3, cu=A, starts=None, n=2, T=5, out=A, **kw):
        d = dict(n_pages=4, page_size=16, d_c=512, d_pe=64, format=1)
        d.update(kw)
        return latent.lib.kda_latent_cache_read(cache, table, pages, cu, starts, n, T, out,
                                                ctypes.byref(latent.CacheShape(**d)), None, None)

    for kw, want in ((dict(T=-1), inv), (dict(n=0), inv), (dict(pages=-1), inv), (dict(cu=None), inv),
                     (dict(cu=A + 2), inv), (dict(table=None), inv), (dict(starts=A + 2), inv),
                     (dict(out=None), inv), (dict(out=A + 4), inv), (dict(cache=None), inv),
                     (dict(page_size=8), uns), (dict(format=-1), inv)):
        assert read(**kw) == want, kw


def test_decode_arguments_are_refused(latent):
    inv, uns = codes(latent)
    good = dict(N=2, L=1, H=4, table_pages=3, dtype=1, scale=0.0)

    def decode(q=A, cache=A, table=A, lens=A, mask=None, out=A, lse=None, ws=A, wsb=1 << 40,
               status=None, cs=None, **kw):
        s = latent.DecodeShape(**{**good, **kw})
        c = latent.CacheShape(**{**dict(n_pages=4, page_size=16, d_c=512, d_pe=64, format=0),
                                 **(cs or {})})
        return latent.lib.kda_latent_decode(q, cache, table, lens, mask, out, lse, ctypes.byref(s),
                                            ctypes.byref(c), ws, wsb, status, None)

    for kw, want in ((dict(N=0), inv), (dict(L=0), inv), (dict(H=0), inv), (dict(table_pages=-1), inv),
                     (dict(scale=-0.5), inv), (dict(scale=float("nan")), inv), (dict(dtype=9), inv),
                     (dict(dtype=0), uns), (dict(L=65), uns), (dict(H=1025), uns),
                     (dict(N=65536), uns), (dict(table_pages=1 << 27), uns),
                     (dict(q=None), inv), (dict(q=A + 8), inv), (dict(cache=None), inv),
                     (dict(table=None), inv), (dict(lens=None), inv), (dict(lens=A + 2), inv),
                     (dict(mask=A + 4), inv), (dict(out=None), inv), (dict(lse=A + 2), inv),
                     (dict(ws=None), inv), (dict(ws=A + 16), inv), (dict(wsb=100), inv),
                     (dict(status=A + 2), inv), (dict(cs=dict(page_size=48)), uns),
                     (dict(cs=dict(format=5)), inv)):
        assert decode(**kw) == want, kw
    size = latent.lib.kda_latent_decode_workspace_size
    cs = latent.CacheShape(4, 16, 512, 64, 0)
    sizes = [size(ctypes.byref(latent.DecodeShape(**{**good, "H": h})), ctypes.byref(cs))
             for h in (1, 16, 17, 32, 33, 512)]
    assert all(n > 0 and n % 256 == 0 for n in sizes) and sizes == sorted(sizes)
    assert size(ctypes.byref(latent.DecodeShape(**{**good, "L": 65})), ctypes.byref(cs)) == 0


def test_binding_refuses_what_the_library_cannot_see(latent):
    """Types, shapes and devices are checked before the library is called; nothing here reaches
    a GPU (the tensors are on the CPU, so the last refusal is that)."""
    bf = torch.bfloat16
    q, kn, pe, v = (torch.zeros(8, 2, 192, dtype=bf), torch.zeros(8, 2, 128, dtype=bf),
                    torch.zeros(8, 64, dtype=bf), torch.zeros(8, 2, 128, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        latent.latent_attn_fwd(q, kn, pe, v)
    with pytest.raises(ValueError, match="CUDA"):
        latent.latent_attention(q, kn, pe, v)
    cache = latent.latent_cache(2, 16, device="cpu")
    assert cache.shape == (2, 16, 576) and cache.dtype == bf
    assert latent.latent_cache(2, 16, quantized=True, device="cpu").shape == (2, 16, 656)
    with pytest.raises(ValueError, match="page_size"):
        latent.latent_cache(2, 20)
    with pytest.raises(ValueError, match="CUDA"):
        latent.latent_cache_write(torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf), cache,
                                  torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError, match="cache dtype"):
        latent._cache_shape(torch.zeros(2, 16, 576))
    with pytest.raises(ValueError, match="row has"):
        latent._cache_shape(torch.zeros(2, 16, 575, dtype=bf))
    with pytest.raises(ValueError, match="contiguous"):
        latent._cache_shape(torch.zeros(2, 16, 1152, dtype=bf)[..., ::2])
    shape_of = lambda *a, **kw: latent._attn_shape(*a, kw.get("cq"), kw.get("ck"), 0, 0, True, None, -1)  # noqa: E731
    s = shape_of(q, kn, pe, v)
    assert (s.B, s.H, s.Tq, s.Tk, s.q_token, s.q_head, s.pe_token) == (1, 2, 8, 8, 384, 192, 64)
    with pytest.raises(TypeError, match="dtype"):
        shape_of(q.float(), kn, pe, v)
    with pytest.raises(ValueError, match="agree"):
        shape_of(q, kn[:7], pe, v)
    with pytest.raises(ValueError, match="agree"):
        shape_of(q, kn, pe, v[:, :1])
    with pytest.raises(ValueError, match="channels"):
        shape_of(q[..., :128], kn, pe, v)
    with pytest.raises(ValueError, match="contiguous"):
        shape_of(torch.zeros(8, 2, 384, dtype=bf)[..., ::2], kn, pe, v)
    with pytest.raises(ValueError, match="packed"):
        shape_of(q, kn, pe, v, cq=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="int32"):
        shape_of(q, kn, pe, v, cq=torch.zeros(2), ck=torch.zeros(2))
    four = [t.unsqueeze(0).expand(3, *t.shape) for t in (q, kn, pe, v)]   # sequence stride 0
    with pytest.raises(ValueError, match="follow"):
        shape_of(*four)


def test_heads_and_tokens_of_one(latent):
    """Of a dimension of one the stride says nothing: any view of it is taken."""
    bf = torch.bfloat16
    wide = torch.zeros(5, 640, dtype=bf)
    s = latent._attn_shape(wide[:, None, :192], wide[:, None, 192:320], wide[:, :64],
                           wide[:, None, 320:448], None, None, 0, 0, True, None, -1)
    assert (s.H, s.q_token, s.q_head, s.k_token, s.k_head, s.pe_token) == (1, 640, 192, 640, 128, 640)
    one = torch.zeros(1, 3, 640, dtype=bf)
    s = latent._attn_shape(one[..., :192], one[..., 192:320], one[:, 0, :64], one[..., 320:448], None,
                           None, 0, 0, True, None, -1)
    assert s.q_head == 640 and s.q_token >= 192 and s.q_token % 8 == 0 and s.pe_token == 64


def test_exported_names(latent):
    for name in latent.EXPORTED:
        assert hasattr(latent.lib, name)
