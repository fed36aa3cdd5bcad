"""Latent attention on the GPU at the ends of its ranges: offsets past 32 bits, scores that rise
all along a sequence, long sequences, values that are not finite, tensors made on other
streams. Against the fp64 references of tests/latent_ref.py."""
from __future__ import annotations

import math
import threading

import pytest
import torch

from tests import latent_ref as ref
from tests.test_latent_gpu import DEV, cu, decode_case, expanded_inputs, paged, rnd, slots_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def latent():
    from kimi_delta_attention_19_b200 import latent as m
    return m


@pytest.mark.parametrize("lq,lk,H,causal", [
    ([2300], [2300], 2, True),
    ([70], [3500], 3, True),                  # few queries behind a long prefix
    ([3000], [100], 1, True),                 # most rows see nothing
    ([1, 129], [4000, 5], 2, False),
    ([257] * 5, [257] * 5, 7, True),
])
def test_longer_sequences(latent, lq, lk, H, causal):
    q, kn, pe, v, g = expanded_inputs(lq, lk, H, seed=sum(lq))
    kw = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk), max_seqlen=max(lq), max_seqlen_k=max(lk),
              causal=causal)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    grads = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    want = ref.expanded(q, kn, pe, v, lq, lk, causal, d_out=g, out_used=out)
    ref.inside(out, want["out"], want["b_out"], "out")
    ref.lse_close(lse, want["lse"])
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), grads):
        ref.inside(got, want[name], want["b_" + name], name)


def test_loose_bounds_give_the_same(latent):
    """max_seqlen only sizes the launch."""
    lens = [100, 300, 0, 33]
    q, kn, pe, v, g = expanded_inputs(lens, lens, 2, seed=1)
    a = latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=cu(lens), max_seqlen=300)
    b = latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=cu(lens))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = latent.latent_attn_bwd(q, kn, pe, v, *a, g, cu_seqlens=cu(lens), max_seqlen=300)
    gb = latent.latent_attn_bwd(q, kn, pe, v, *a, g, cu_seqlens=cu(lens))
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_rising_scores(latent):
    """Scores that grow by some units every key tile: the softmax reference is raised again and
    again, and what came before fades to nothing. Scores reach some 200, so fp32 sums of 192
    products err by 192 * 2^-24 * (sum of magnitudes ~ 200) ~ 2e-3 at the very worst and by its
    root-sum some 2e-4: within the bound's room (2^-8 of p) for the keys that count."""
    n, H = 1200, 2
    gen = torch.Generator(device=DEV).manual_seed(2)
    dirn = torch.randn(192, generator=gen, device=DEV)
    dirn = dirn / dirn.norm()
    ramp = torch.linspace(0, 1, n, device=DEV)[:, None, None]
    q = (60 * dirn).expand(n, H, 192).to(torch.bfloat16).contiguous()
    k = (46 * ramp * dirn).expand(n, H, 192).to(torch.bfloat16)
    kn, pe = k[..., :128].contiguous(), k[:, 0, 128:].contiguous()
    v = rnd(gen, n, H, 128)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v)
    want = ref.expanded(q, kn, pe, v, [n], [n], True)
    assert float(want["lse"].max()) > 150
    ref.inside(out, want["out"], want["b_out"], "out")
    ref.lse_close(lse, want["lse"])
    # the same over a cache, whose rows and query carry the ramp in the latent part
    rows = torch.zeros(n, 576, dtype=torch.bfloat16, device=DEV)
    rows[:, :192] = k[:, 0]
    rows[:, 192:512] = rnd(gen, n, 320)
    table, pages = paged([n], 16, seed=3)
    cache = latent.latent_cache(pages, 16, device=DEV)
    latent.latent_cache_write(rows[:, :512], rows[:, 512:], cache, slots_of(table, [n], 16))
    qa = torch.zeros(1, 1, 20, 576, dtype=torch.bfloat16, device=DEV)
    qa[..., :192] = q[0, 0]
    o = latent.latent_decode(qa, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    want, bnd, _ = ref.absorbed(qa, cache, table, [n])
    ref.inside(o, want, bnd, "decode")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_query_stays_in_its_row(latent, bad):
    lens, H = [200, 90], 2
    q, kn, pe, v, g = expanded_inputs(lens, lens, H, seed=5)
    kw = dict(cu_seqlens=cu(lens), max_seqlen=200)
    clean, _ = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    q[77, 1] = bad
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    rest = torch.ones(q.shape[:2], dtype=torch.bool, device=DEV)
    rest[77, 1] = False
    assert torch.equal(out[rest], clean[rest])
    assert torch.isnan(out[77, 1].float()).all() and not torch.isfinite(lse[77, 1])
    x = decode_case(latent, [300, 5], 9, 1, 16, False, seed=6, garbage=False)
    clean = latent.latent_decode(*x)
    x[0][0, 0, 3] = bad
    o = latent.latent_decode(*x)
    rest = torch.ones(o.shape[:3], dtype=torch.bool, device=DEV)
    rest[0, 0, 3] = False
    assert torch.equal(o[rest], clean[rest]) and torch.isnan(o[0, 0, 3].float()).all()


def test_element_offsets_past_32_bits(latent):
    """Token strides of 32 M elements: rows more than 2^32 elements (and bytes) apart."""
    T, H, stride = 140, 2, 1 << 25
    gen = torch.Generator(device=DEV).manual_seed(7)
    base = torch.empty((T - 1) * stride + 4096, dtype=torch.bfloat16, device=DEV)
    view = lambda d, at, step: base.as_strided((T, H, d), (stride, step, 1), at)  # noqa: E731
    q, kn, v = view(192, 0, 192), view(128, 512, 256), view(128, 640, 256)
    pe = base.as_strided((T, 64), (stride, 1), 2048)
    for t in (q, kn, v, pe):
        t.copy_(rnd(gen, *t.shape))
    assert (T - 1) * stride > 1 << 32
    g = rnd(gen, T, H, 128)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v)
    grads = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g)
    near = [t.contiguous() for t in (q, kn, pe, v)]
    want = ref.expanded(*near, [T], [T], True, d_out=g, out_used=out)
    ref.inside(out, want["out"], want["b_out"], "out")
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), grads):
        ref.inside(got, want[name], want["b_" + name], name)


@pytest.mark.parametrize("quantized", [False, True])
def test_cache_offsets_past_32_bits(latent, quantized):
    """A cache of more than 4 GB, its last pages in use."""
    ps, lens = 128, [300, 129]
    n_pages = (56000 if quantized else 32000)                  # 4.7 GB
    cache = torch.empty(n_pages, ps, 656 if quantized else 576, device=DEV,
                        dtype=torch.uint8 if quantized else torch.bfloat16)
    assert cache.numel() * cache.element_size() > 1 << 32
    table = torch.tensor([[n_pages - 1, n_pages - 5, 3], [n_pages - 2, n_pages - 3, 0]],
                         dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(8)
    T = sum(lens)
    c, pe = rnd(gen, T, 512), rnd(gen, T, 64)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    latent.latent_cache_write(c, pe, cache, slots_of(table, lens, ps), status=st)
    back = latent.latent_cache_read(cache, table, cu(lens), total=T, status=st)
    want = ref.quantize(c)[0] if quantized else c.double()
    assert torch.equal(back[:, :512].double(), want) and torch.equal(back[:, 512:], pe)
    q = rnd(gen, 2, 1, 32, 576)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = latent.latent_decode(q, cache, table, sl, status=st)
    # the same rows in a small cache give the same bits
    small, pages = paged(lens, ps, seed=9)
    near = latent.latent_cache(pages, ps, quantized=quantized, device=DEV)
    latent.latent_cache_write(c, pe, near, slots_of(small, lens, ps))
    assert torch.equal(out, latent.latent_decode(q, near, small, sl))
    assert int(st) == 0


def test_padded_batch_of_queries_and_empty_sequences(latent):
    """A serving batch padded with length-0 sequences and skipped slots."""
    lens = [0, 700, 0, 0, 33, 0]
    q, cache, table, sl = decode_case(latent, lens, 32, 1, 64, True, seed=10)
    lse = torch.empty(q.shape[:3], device=DEV)
    out = latent.latent_decode(q, cache, table, sl, lse=lse)
    want, bnd, wl = ref.absorbed(q, cache, table, lens)
    ref.inside(out, want, bnd, "out")
    assert (out[[0, 2, 3, 5]] == 0).all() and (lse[[0, 2, 3, 5]] == -math.inf).all()
    # a table of no columns, a cache of no pages: every sequence of length 0 is empty
    none = latent.latent_cache(0, 16, device=DEV)
    zero = torch.zeros(6, dtype=torch.int32, device=DEV)
    out = latent.latent_decode(q, none, torch.zeros(6, 0, dtype=torch.int32, device=DEV), zero)
    assert (out == 0).all()


def test_inputs_made_on_another_stream(latent):
    """The call runs on the given stream, behind what that stream made."""
    lens = [500, 77]
    q, kn, pe, v, g = expanded_inputs(lens, lens, 2, seed=11)
    kw = dict(cu_seqlens=cu(lens), max_seqlen=500)
    want, _ = latent.latent_attn_fwd(q * 2, kn, pe, v, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):                                    # keeps the stream busy
            big = (big @ big).clamp(-1, 1)
        q2 = q * 2
    out, lse = latent.latent_attn_fwd(q2, kn, pe, v, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)


def test_two_captured_decodes_interleaved(latent):
    """Graphs with workspaces of their own, replayed in any order and beside eager calls."""
    cases = [decode_case(latent, [900, 40], 32, 1, 64, False, seed=12),
             decode_case(latent, [50, 3000], 8, 4, 16, True, seed=13)]
    want = [latent.latent_decode(*c) for c in cases]
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = latent.latent_decode(*c)
        graphs.append((g, o))
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for _, o in graphs:
            o.zero_()
        for i in order:
            graphs[i][0].replay()
        eager = latent.latent_decode(*cases[0])
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0])
        for i in set(order):
            assert torch.equal(graphs[i][1], want[i])


@pytest.mark.parametrize("quantized", [False, True])
def test_every_sequence_of_a_full_batch_has_a_bad_page(latent, quantized):
    """One-tile sequences, several a thread block: each is reported by itself, the good ones
    between them are not."""
    n = 700
    lens = [64] * n
    q, cache, table, sl = decode_case(latent, lens, 4, 1, 64, quantized, seed=14)
    good = latent.latent_decode(q, cache, table, sl)
    bad = torch.arange(n, device=DEV) % 7 != 3
    table[bad, 0] = cache.shape[0] + 5
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = latent.latent_decode(q, cache, table, sl, status=st)
    assert latent.status_of(st) == (4, 3)
    assert torch.isnan(out[bad].float()).all() and torch.equal(out[~bad], good[~bad])


@pytest.mark.parametrize("quantized", [False, True])
def test_a_nan_in_a_cached_row_reaches_its_sequence_only(latent, quantized):
    """Every one of the 512 channels, each in a sequence of its own: that sequence's rows are NaN
    in that channel (and in every channel where the score is NaN too, as it is), no other's."""
    n, ps = 512, 16
    lens = [20] * n
    gen = torch.Generator(device=DEV).manual_seed(15)
    table, pages = paged(lens, ps, seed=15)
    cache = latent.latent_cache(pages, ps, quantized=quantized, device=DEV)
    c, pe = rnd(gen, 20 * n, 512), rnd(gen, 20 * n, 64)
    pick = torch.arange(n, device=DEV)
    c[20 * pick[::2] + 7, pick[::2]] = math.nan           # every other sequence
    latent.latent_cache_write(c, pe, cache, slots_of(table, lens, ps))
    q = rnd(gen, n, 1, 5, 576)
    out = latent.latent_decode(q, cache, table, torch.full((n,), 20, dtype=torch.int32, device=DEV))
    assert torch.isnan(out[::2].float()).all() and torch.isfinite(out[1::2].float()).all()
    want, bnd, _ = ref.absorbed(q[1::2], cache, table[1::2], lens[1::2])
    ref.inside(out[1::2], want, bnd, "out")


def test_every_code_and_scale_of_a_row_in_8_bits(latent):
    """Rows put together by hand: all codes, scales the cache writes (bytes 7 to 247) and 2^-127 (0),
    which stands in rows nothing was written to. Read back exactly (a value below bf16's range
    rounds, one above it is infinite, as a conversion from 64 bits does), and attended to."""
    n, ps = 48, 16
    gen = torch.Generator(device=DEV).manual_seed(16)
    cache = latent.latent_cache(n // ps, ps, quantized=True, device=DEV)
    flat = cache.view(n, 656)
    codes = torch.arange(512, device=DEV) % 256
    flat[:, :512] = torch.stack([codes[torch.randperm(512, generator=gen, device=DEV)]
                                 for _ in range(n)]).to(torch.uint8)
    flat[:, 512:640] = rnd(gen, n, 64).view(torch.uint8)
    exps = torch.tensor([0, 7, 100, 119, 127, 134, 135, 200, 246, 247], device=DEV)
    flat[:, 640:644] = exps[torch.randint(len(exps), (n, 4), generator=gen, device=DEV)].to(torch.uint8)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    got = latent.latent_cache_read(cache, table, cu([n]), total=n)
    at = slots_of(table, [n], ps)
    torch.testing.assert_close(got, ref.rows_of(cache)[at].to(torch.bfloat16), rtol=0, atol=0,
                               equal_nan=True)

    flat[:, :512][flat[:, :512] & 127 == 127] = 5          # no NaN, and scores of ordinary size
    flat[:, 640:644] = exps[torch.randint(5, (n, 4), generator=gen, device=DEV)].to(torch.uint8)
    q = rnd(gen, 1, 3, 16, 576, std=0.02)
    lse = torch.empty(1, 3, 16, device=DEV)
    out = latent.latent_decode(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), lse=lse)
    want, bnd, want_lse = ref.absorbed(q, cache, table, [n])
    ref.inside(out, want, bnd, "out")
    ref.lse_close(lse, want_lse)


def test_gradients_of_gradients_are_refused(latent):
    q, kn, pe, v, g = expanded_inputs([9], [9], 2, seed=17)
    leaves = [t.detach().clone().requires_grad_() for t in (q, kn, pe, v)]
    out = latent.latent_attention(*leaves)
    grads = torch.autograd.grad(out, leaves, g, create_graph=True)
    plain = torch.autograd.grad(latent.latent_attention(*leaves), leaves, g)
    assert all(torch.equal(a, b) for a, b in zip(grads, plain))
    with pytest.raises(RuntimeError, match="no gradients of its gradients"):
        (out.float().sum() + sum(t.float().square().sum() for t in grads)).backward()


def test_threads_without_a_context(latent):
    """Each call as the first that a thread makes to the GPU (autograd's threads start like that)."""
    q, kn, pe, v, g = expanded_inputs([150], [150], 2, seed=18)
    dec = decode_case(latent, [150, 9], 5, 1, 16, False, seed=18)
    cache, table = dec[1], dec[2]
    off, slots = cu([9, 9]), torch.arange(18, device=DEV)
    c, c_pe = q[:18, 0].repeat(1, 3)[:, :512].contiguous(), pe[:18]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def results():
        n = dec[0].shape[:3]
        return {"out": torch.empty(150, 2, 128, dtype=torch.bfloat16, device=DEV),
                "lse": torch.empty(150, 2, device=DEV),
                "grads": tuple(torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in (q, kn, pe, v)),
                "decode": torch.empty(*n, 512, dtype=torch.bfloat16, device=DEV),
                "cache": torch.zeros_like(cache),
                "read": torch.empty(18, 576, dtype=torch.bfloat16, device=DEV)}

    def calls(r):
        return (lambda: latent.latent_attn_fwd(q, kn, pe, v, out=r["out"], lse=r["lse"]),
                lambda: latent.latent_attn_bwd(q, kn, pe, v, r["out"], r["lse"], g,
                                               grads=r["grads"], workspace=ws),
                lambda: latent.latent_decode(*dec, out=r["decode"], workspace=dws),
                lambda: latent.latent_cache_write(c, c_pe, r["cache"], slots),
                lambda: latent.latent_cache_read(cache, table, off, out=r["read"]))

    dws = latent.latent_decode_workspace(2, 5, cache)
    want, got, failed = results(), results(), []
    for call in calls(want):
        call()
    torch.cuda.synchronize()

    def run(call):
        try:
            call()
        except Exception as e:
            failed.append(e)

    for call in calls(got):
        t = threading.Thread(target=run, args=(call,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for k in want:
        for a, b in zip(want[k] if k == "grads" else (want[k],), got[k] if k == "grads" else (got[k],)):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("lq,lk,causal", [([1, 2, 3, 0, 5, 32], [1, 2, 3, 7, 5, 32], True),
                                          ([28], [28], True), ([9, 40], [20, 12], True),
                                          ([70, 3], [30, 1], False), ([1] * 100, [2] * 100, True)])
def test_gradients_of_short_sequences(latent, lq, lk, causal):
    """Rows of up to 32 keys: dS as exact as fp32 scores make it (two bf16 terms keep 2^-16 of it,
    dP and D are fp32 sums of 128 products), whatever out was rounded to."""
    q, kn, pe, v, g = expanded_inputs(lq, lk, 3, seed=19)
    kw = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk), max_seqlen=max(lq), max_seqlen_k=max(lk),
              causal=causal)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    dq, dkn, dpe, _ = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    a0 = b0 = 0
    for a, b in zip(lq, lk):
        sq, sk = slice(a0, a0 + a), slice(b0, b0 + b)
        a0, b0 = a0 + a, b0 + b
        Q, G, V = (t.double().transpose(0, 1) for t in (q[sq], g[sq], v[sk]))
        K = torch.cat((kn[sk].double(), pe[sk].double()[:, None].expand(-1, 3, -1)), -1).transpose(0, 1)
        x = Q @ K.transpose(1, 2) / math.sqrt(192)
        seen = torch.ones(a, b, dtype=torch.bool, device=DEV)
        if causal:
            seen = torch.arange(b, device=DEV)[None] <= torch.arange(a, device=DEV)[:, None] + b - a
        x = x.masked_fill(~seen, -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1))
        dp = G @ V.transpose(1, 2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(192)
        # p off by 2^-17 (scores of 192 products, the exponential), dP and D by as much of the
        # magnitudes they are summed from
        size = G.abs() @ V.abs().transpose(1, 2)
        e = 2.0 ** -15 * ds.abs() + \
            2.0 ** -16 * p * (size + (p * size).sum(-1, keepdim=True)) / math.sqrt(192)

        def check(got, val, err, name):
            ref.inside(got, val, 1.05 * ref.U * val.abs() + err + 1e-6, name)

        check(dq[sq].transpose(0, 1), ds @ K, e @ K.abs(), "dq")
        dk, ek = ds.transpose(1, 2) @ Q, e.transpose(1, 2) @ Q.abs()
        check(dkn[sk].transpose(0, 1), dk[..., :128], ek[..., :128], "dk_nope")
        check(dpe[sk], dk[..., 128:].sum(0), ek[..., 128:].sum(0), "dk_pe")
