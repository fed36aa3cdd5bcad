"""Latent attention on the GPU against fp64 references (tests/latent_ref.py)."""
from __future__ import annotations

import math

import pytest
import torch

from tests import latent_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def latent():
    from kimi_delta_attention_19_b200 import latent as m
    return m


def cu(lengths):
    c = [0]
    for n in lengths:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def rnd(gen, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=gen, device=DEV)).to(torch.bfloat16)


def expanded_inputs(lq, lk, H, seed=0, behind=0, std=1.5):
    """Packed inputs, k_nope and v views of one projection; `behind` rows of NaN follow."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    tq, tk = sum(lq) + behind, sum(lk) + behind
    q, kv, pe = rnd(gen, tq, H, 192, std=std), rnd(gen, tk, H, 256), rnd(gen, tk, 64)
    g = rnd(gen, tq, H, 128)
    if behind:
        for t in (q, kv, pe, g):
            t[-behind:] = math.nan
    return q, kv[..., :128], pe, kv[..., 128:], g


EXPANDED = [
    # lq, lk, H, causal
    ([1], [1], 1, True),
    ([1, 2, 3, 7], [1, 2, 3, 7], 3, True),
    ([63, 64, 65], [63, 64, 65], 2, True),
    ([127, 128, 129], [127, 128, 129], 2, True),
    ([255, 0, 257, 1], [255, 0, 257, 1], 2, True),
    ([513, 40], [513, 40], 2, False),
    ([1, 100, 130], [700, 101, 383], 4, True),      # cached prefixes before the queries
    ([5, 200], [0, 130], 2, True),                  # no keys; more queries than keys: empty rows
    ([33, 300], [129, 257], 1, False),
    ([1000], [1000], 5, True),
    ([90] * 17, [90] * 17, 1, True),
    ([385], [1025], 16, True),
]


@pytest.mark.parametrize("lq,lk,H,causal", EXPANDED)
def test_expanded_forward_and_backward(latent, lq, lk, H, causal):
    q, kn, pe, v, g = expanded_inputs(lq, lk, H, seed=len(lq) + H)
    kw = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk), max_seqlen=max(lq), max_seqlen_k=max(lk),
              causal=causal)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, status=st, **kw)
    grads = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, status=st, **kw)
    want = ref.expanded(q, kn, pe, v, lq, lk, causal, d_out=g, out_used=out)
    ref.inside(out, want["out"], want["b_out"], "out")
    ref.lse_close(lse, want["lse"])
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), grads):
        ref.inside(got, want[name], want["b_" + name], name)
    assert int(st) == 0


def test_batched_sequences_scale_and_contiguous_keys(latent):
    gen = torch.Generator(device=DEV).manual_seed(7)
    B, Tq, Tk, H = 3, 70, 150, 4
    q, kn, pe, v = (rnd(gen, B, Tq, H, 192), rnd(gen, B, Tk, H, 128), rnd(gen, B, Tk, 64),
                    rnd(gen, B, Tk, H, 128))
    g = rnd(gen, B, Tq, H, 128)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, scale=0.11)
    grads = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, scale=0.11)
    flat = [t.reshape(-1, *t.shape[2:]) for t in (q, kn, pe, v)]
    want = ref.expanded(*flat, [Tq] * B, [Tk] * B, True, scale=0.11, d_out=g.reshape(-1, H, 128),
                        out_used=out.reshape(-1, H, 128))
    ref.inside(out.reshape(-1, H, 128), want["out"], want["b_out"], "out")
    ref.lse_close(lse.reshape(-1, H), want["lse"])
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), grads):
        ref.inside(got.reshape(want[name].shape), want[name], want["b_" + name], name)


def test_strided_queries_and_permuted_heads(latent):
    """Token and head strides other than the packed ones: heads outermost, a slice of rows."""
    gen = torch.Generator(device=DEV).manual_seed(8)
    H, lq = 3, [130, 61]
    T = sum(lq)
    q = rnd(gen, H, T, 192).transpose(0, 1)                 # [T, H, 192], head stride largest
    kn = rnd(gen, T, 2 * H, 128)[:, ::2]
    v = rnd(gen, H, T, 256).transpose(0, 1)[..., 128:]
    pe = rnd(gen, T, 576)[:, 512:]
    kw = dict(cu_seqlens=cu(lq), max_seqlen=max(lq))
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    g = rnd(gen, T, H, 128)
    grads = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    want = ref.expanded(q, kn, pe, v, lq, lq, True, d_out=g, out_used=out)
    ref.inside(out, want["out"], want["b_out"], "out")
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), grads):
        ref.inside(got, want[name], want["b_" + name], name)


@pytest.mark.parametrize("lq,lk", [([100, 30], [100, 30]), ([64, 129], [200, 129])])
def test_rows_behind_the_last_sequence(latent, lq, lk):
    """NaN behind the last sequence reaches nothing, and its rows are left as they were."""
    behind, H = 70, 2
    q, kn, pe, v, g = expanded_inputs(lq, lk, H, seed=3, behind=behind)
    kw = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk), max_seqlen=max(lq), max_seqlen_k=max(lk))
    out = torch.full((q.shape[0], H, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    latent.latent_attn_fwd(q, kn, pe, v, out=out, lse=lse, **kw)
    grads = tuple(torch.full(t.shape, 5.0, dtype=torch.bfloat16, device=DEV)
                  for t in (q, kn, pe, v))
    latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, grads=grads, **kw)
    want = ref.expanded(q, kn, pe, v, lq, lk, True, d_out=g, out_used=out)
    for t in (out, lse) + grads:
        assert (t[-behind:] == 5).all()
    for name, got in zip(("out", "dq", "dk_nope", "dk_pe", "dv"), (out,) + grads):
        ref.inside(got, want[name], want["b_" + name], name)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_sequence_does_not_reach_its_neighbours(latent, bad):
    """Not finite values in one sequence stay in its rows, forward and backward."""
    lens, H = [70, 50, 90], 2
    q, kn, pe, v, g = expanded_inputs(lens, lens, H, seed=4)
    kw = dict(cu_seqlens=cu(lens), max_seqlen=90)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    clean = (out, lse) + latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    for t in (q, kn, pe, v, g):
        t[70:120] = bad
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    dirty = (out, lse) + latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    for a, b in zip(clean, dirty):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[120:], b[120:])
    assert torch.isnan(dirty[0][70:120].float()).any()


def test_far_scores(latent):
    """Scores of hundreds (and a key far above the rest late in the sequence) stay exact."""
    lens, H = [400], 2
    q, kn, pe, v, g = expanded_inputs(lens, lens, H, seed=5, std=12.0)
    kn[390] *= 8
    kw = dict(cu_seqlens=cu(lens), max_seqlen=400)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    want = ref.expanded(q, kn, pe, v, lens, lens, True)
    # scores of some hundreds carry fp32 errors of some 1e-5 into the probabilities
    ref.inside(out, want["out"], want["b_out"], "out")
    ref.lse_close(lse, want["lse"])


def test_malformed_sequences_are_reported(latent):
    lens = [40, 50]
    q, kn, pe, v, g = expanded_inputs(lens, lens, 1, seed=6)
    for offsets, most in (([0, 60, 40], 90), ([0, 40, 91], 90), ([3, 40, 90], 90),
                          ([0, 40, 90], 45), ([0, -5, 90], 90)):
        c = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=c, max_seqlen=most, status=st)
        assert latent.status_of(st) == (4, 1), offsets
        out.zero_(), lse.zero_()
        st.zero_()
        latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, cu_seqlens=c, max_seqlen=most, status=st)
        assert latent.status_of(st) == (4, 1), offsets


def test_same_bits_twice_and_without_lse_consumers(latent):
    lens = [700, 301]
    q, kn, pe, v, g = expanded_inputs(lens, lens, 4, seed=9)
    kw = dict(cu_seqlens=cu(lens), max_seqlen=700)
    runs = []
    for _ in range(2):
        out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
        runs.append((out, lse) + latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_gradients_against_differences(latent):
    """dL/dx . dx against L(x + dx) - L(x - dx) of the fp64 reference loss, for each input."""
    lens, H = [37, 20], 2
    q, kn, pe, v, g = expanded_inputs(lens, lens, H, seed=11)
    ins = [t.clone().requires_grad_() for t in (q, kn, pe, v)]
    out = latent.latent_attention(*ins, cu_seqlens=cu(lens), max_seqlen=37)
    out.backward(g)
    gen = torch.Generator(device=DEV).manual_seed(12)

    def loss(parts):
        o = ref.expanded(*parts, lens, lens, True)["out"]
        return float((o * g.double()).sum())

    base = [t.double() for t in (q, kn, pe, v)]
    for k in range(4):
        d = torch.randn(base[k].shape, generator=gen, device=DEV, dtype=torch.float64)
        eps = 1e-4
        hi, lo = list(base), list(base)
        hi[k], lo[k] = base[k] + eps * d, base[k] - eps * d
        num = (loss(hi) - loss(lo)) / (2 * eps)
        ana = float((ins[k].grad.double() * d).sum())
        # every gradient element is within 4u of sums of its terms: the products with d add up
        # like a random walk, so 4u * |grad|_2 * few is far above what is expected
        room = 8 * ref.U * float(ins[k].grad.double().norm())
        assert abs(num - ana) <= room, (k, num, ana, room)


def test_autograd_matches_the_explicit_calls_and_zeroes_padding(latent):
    lens, H, behind = [60, 33], 2, 9
    q, kn, pe, v, g = expanded_inputs(lens, lens, H, seed=13, behind=behind)
    g = g.nan_to_num(0)
    ins = [t.clone().requires_grad_() for t in (q, kn, pe, v)]
    out = latent.latent_attention(*ins, cu_seqlens=cu(lens), max_seqlen=60)
    out.backward(g)
    o2, lse = latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=cu(lens), max_seqlen=60)
    grads = latent.latent_attn_bwd(q, kn, pe, v, o2, lse, g, cu_seqlens=cu(lens), max_seqlen=60)
    n = sum(lens)
    assert torch.equal(out[:n], o2[:n]) and (out[n:] == 0).all()
    for t, want in zip(ins, grads):
        assert torch.equal(t.grad[:n], want[:n]) and (t.grad[n:] == 0).all()


# ------------------------------------------------------------------------------- the cache
def paged(lens, ps, seed, extra=2):
    """A shuffled block table for sequences of these lengths, and the number of pages."""
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + extra
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = perm[at:at + k]
        at += k
    return table.to(DEV), pages


def slots_of(table, lens, ps, starts=None):
    s = []
    for i, n in enumerate(lens):
        pos = torch.arange(n, device=DEV) + (starts[i] if starts else 0)
        s.append(table[i].long()[pos // ps] * ps + pos % ps)
    return torch.cat(s)


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("lens,ps", [([1], 16), ([5, 0, 33, 16], 16), ([130, 64, 65], 64),
                                     ([300], 128), ([31] * 9, 32)])
def test_cache_write_and_read(latent, lens, ps, quantized):
    gen = torch.Generator(device=DEV).manual_seed(sum(lens))
    T = sum(lens)
    c = rnd(gen, T, 512) * torch.exp2(torch.randint(-30, 30, (T, 1), generator=gen, device=DEV))
    c = c.to(torch.bfloat16)
    c[0, :128] = 0
    c[0, 130] = 448.0
    if T > 4:
        c[3, 256:384] = 2.0 ** -133                # subnormal bf16
        c[4, 5] = 3.0e38
    wide = rnd(gen, T, 640)                        # k_pe as a strided view
    pe = wide[:, 512:576]
    table, pages = paged(lens, ps, seed=T)
    cache = latent.latent_cache(pages, ps, quantized=quantized, device=DEV)
    before = cache.clone()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = slots_of(table, lens, ps)
    latent.latent_cache_write(c, pe, cache, slots, status=st)
    back = latent.latent_cache_read(cache, table, cu(lens), total=T, status=st)
    want = ref.quantize(c)[0] if quantized else c.double()
    assert torch.equal(back[:, :512].double(), want)
    assert torch.equal(back[:, 512:], pe)
    assert torch.equal(ref.rows_of(cache)[slots], torch.cat((want, pe.double()), 1))
    rest = torch.ones(pages * ps, dtype=torch.bool, device=DEV)
    rest[slots] = False
    assert torch.equal(cache.view(pages * ps, -1)[rest], before.view(pages * ps, -1)[rest])
    assert int(st) == 0


def test_cache_read_of_a_part_and_rows_behind(latent):
    ps, lens = 16, [100, 50]
    gen = torch.Generator(device=DEV).manual_seed(1)
    table, pages = paged(lens, ps, seed=1)
    cache = latent.latent_cache(pages, ps, device=DEV)
    cache.copy_(rnd(gen, pages, ps, 576))
    out = torch.full((40, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    latent.latent_cache_read(cache, table, cu([20, 11]), out=out,
                             starts=torch.tensor([77, 0], dtype=torch.int32, device=DEV))
    flat = cache.view(-1, 576)
    assert torch.equal(out[:20], flat[slots_of(table, [20], ps, starts=[77])])
    assert torch.equal(out[20:31], flat[slots_of(table[1:], [11], ps)])
    assert (out[31:] == 3).all()


def test_cache_bad_slots_pages_and_values(latent):
    ps = 16
    for quantized in (False, True):
        cache = latent.latent_cache(2, ps, quantized=quantized, device=DEV)
        gen = torch.Generator(device=DEV).manual_seed(2)
        c, pe = rnd(gen, 4, 512), rnd(gen, 4, 64)
        c[3, 7], c[3, 8], c[3, 200] = math.inf, -math.inf, math.nan
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        slots = torch.tensor([-1, 32, 5, 6], device=DEV)
        latent.latent_cache_write(c, pe, cache, slots, status=st)
        assert latent.status_of(st) == (4, 3)
        rows = ref.rows_of(cache)
        assert (rows[[i for i in range(32) if i not in (5, 6)]] == 0).all()
        if quantized:
            assert torch.equal(rows[5, :512], ref.quantize(c[2:3])[0][0])
            want = ref.quantize(c[3:4])[0][0]
            assert torch.isnan(want[[7, 8, 200]]).all() and int(torch.isnan(want).sum()) == 3
            assert torch.equal(rows[6, :512].nan_to_num(nan=9e9), want.nan_to_num(nan=9e9))
        st.zero_()
        table = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32, device=DEV)
        back = latent.latent_cache_read(cache, table, cu([18, 40]), total=58, status=st)
        assert latent.status_of(st) == (4, 3)
        bad = torch.isnan(back.float()).all(1)
        assert bad[16:18].all() and bad[18 + 16:].all()
        assert not bad[:16].any() and not bad[18:34].any()


# --------------------------------------------------------------------------------- decode
def decode_case(latent, lens, H, L, ps, quantized, seed, garbage=True, std=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    table, pages = paged(lens, ps, seed)
    rows = rnd(gen, pages * ps, 576)
    cache = latent.latent_cache(pages, ps, quantized=quantized, device=DEV)
    every = torch.arange(pages * ps, device=DEV)
    latent.latent_cache_write(rows[:, :512], rows[:, 512:], cache, every)
    if garbage:        # what no sequence owns is NaN: the ends of last pages, spare pages
        used = torch.zeros(pages * ps, dtype=torch.bool, device=DEV)
        if sum(lens):
            used[slots_of(table, lens, ps)] = True
        flat = cache.view(pages * ps, -1)
        if quantized:
            flat[~used] = 0x7f
            flat[~used, 640:644] = 255
            flat[~used, 512:640] = 255
        else:
            flat[~used] = math.nan
    q = rnd(gen, len(lens), L, H, 576, std=std)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return q, cache, table, sl


DECODE = [
    # lens, H, L, page
    ([1], 1, 1, 16),
    ([0, 1, 2], 3, 1, 16),
    ([15, 16, 17, 127, 128, 129], 16, 1, 16),
    ([1003], 32, 1, 64),
    ([255, 256, 257], 17, 1, 128),
    ([5000, 1, 300], 32, 1, 32),
    ([20000], 16, 1, 128),
    ([700, 64], 64, 1, 64),
    ([333], 100, 1, 32),
    ([40, 8, 500], 8, 5, 16),
    ([130, 2000], 32, 8, 64),
    ([64, 70], 3, 64, 16),
    ([3, 2, 1, 0], 4, 4, 16),                      # fewer cached tokens than query tokens
    ([37 * i % 211 for i in range(300)], 4, 1, 16),
]


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("lens,H,L,ps", DECODE)
def test_decode(latent, lens, H, L, ps, quantized):
    q, cache, table, sl = decode_case(latent, lens, H, L, ps, quantized, seed=sum(lens) + H)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.empty(q.shape[:3], device=DEV)
    out = latent.latent_decode(q, cache, table, sl, lse=lse, status=st)
    want, bnd, wl = ref.absorbed(q, cache, table, lens)
    ref.inside(out, want, bnd, "out")
    ref.lse_close(lse, wl)
    assert int(st) == 0


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("L,H,lens", [(4, 5, [4, 3, 60, 129, 700]), (64, 2, [64, 200, 10]),
                                      (8, 32, [8, 1000, 133])])
def test_decode_of_drafted_trees(latent, L, H, lens, quantized):
    q, cache, table, sl = decode_case(latent, lens, H, L, 16, quantized, seed=L)
    gen = torch.Generator(device=DEV).manual_seed(L)
    mask = torch.randint(-(1 << 63), (1 << 63) - 1, (len(lens), L), generator=gen, device=DEV)
    mask[0, 1] = 0          # of a sequence that is all drafts: sees nothing
    mask[1, 0] = -1
    lse = torch.empty(q.shape[:3], device=DEV)
    out = latent.latent_decode(q, cache, table, sl, draft_mask=mask, lse=lse, scale=0.05)
    want, bnd, wl = ref.absorbed(q, cache, table, lens, mask=mask, scale=0.05)
    assert (wl[0, 1] == -math.inf).all()
    ref.inside(out, want, bnd, "out")
    ref.lse_close(lse, wl)


def test_decode_far_scores(latent):
    lens = [900, 300]
    q, cache, table, sl = decode_case(latent, lens, 16, 1, 16, False, seed=5, std=12.0)
    out = latent.latent_decode(q, cache, table, sl)
    want, bnd, _ = ref.absorbed(q, cache, table, lens)
    # scores of some hundreds carry fp32 errors of some 1e-5 into the probabilities
    ref.inside(out, want, bnd, "out")


@pytest.mark.parametrize("quantized", [False, True])
def test_decode_bad_lengths_and_pages(latent, quantized):
    """Reported and NaN, for the sequence that has them only."""
    lens = [100, 3000, 60, 90, 5]
    q, cache, table, sl = decode_case(latent, lens, 16, 1, 16, quantized, seed=6)
    good = latent.latent_decode(q, cache, table, sl)
    table[0, 3], table[1, 100] = cache.shape[0], -1
    sl[2], sl[3] = -4, 16 * table.shape[1] + 1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.empty(q.shape[:3], device=DEV)
    out = latent.latent_decode(q, cache, table, sl, lse=lse, status=st)
    assert latent.status_of(st) == (4, 3)
    assert torch.isnan(out[:4].float()).all() and torch.isnan(lse[:4]).all()
    assert torch.equal(out[4], good[4])


def test_decode_graph_replays_on_new_lengths(latent):
    """A captured step serves other lengths, tables and queries; two graphs share a workspace
    on one stream; the same inputs give the same bits."""
    lens = [500, 900, 17]
    q, cache, table, sl = decode_case(latent, [1000] * 3, 16, 1, 64, True, seed=8, garbage=False)
    sl.copy_(torch.tensor(lens))
    ws = latent.latent_decode_workspace(3, 16, cache)
    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        latent.latent_decode(q, cache, table, sl, workspace=ws)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                o = latent.latent_decode(q, cache, table, sl, workspace=ws)
            graphs.append((g, o))
    stream.synchronize()
    for new in ([500, 900, 17], [1, 1000, 64], [0, 3, 999]):
        sl.copy_(torch.tensor(new))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for g, _ in graphs:
                g.replay()
        stream.synchronize()
        want, bnd, _ = ref.absorbed(q, cache, table, new)
        ref.inside(graphs[0][1], want, bnd, str(new))
        assert torch.equal(graphs[0][1], graphs[1][1])


def test_training_step_in_a_graph(latent):
    lens, H = [130, 70], 2
    q, kn, pe, v, g = expanded_inputs(lens, lens, H, seed=14)
    kw = dict(cu_seqlens=cu(lens), max_seqlen=130)

    def step():
        out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
        return (out,) + latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in (q, g):
        t.copy_(t.flip(0))
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_on_two_streams_at_once(latent):
    lens = [400, 222]
    ins = [expanded_inputs(lens, lens, 2, seed=20 + k) for k in range(2)]
    kw = dict(cu_seqlens=cu(lens), max_seqlen=400)
    alone = [latent.latent_attn_fwd(*x[:4], **kw)[0] for x in ins]
    dec = decode_case(latent, [3000, 100], 16, 1, 16, False, seed=21)
    d_alone = latent.latent_decode(*dec)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [latent.latent_attn_fwd(*x[:4], stream=s, **kw)[0] for x, s in zip(ins, streams)]
    d_got = latent.latent_decode(*dec, stream=streams[2])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, got)) and torch.equal(d_alone, d_got)


# ----------------------------------------------------------------- the operators together
@pytest.mark.parametrize("quantized", [False, True])
def test_prompt_then_cache_then_tokens(latent, quantized):
    """A layer as it is used: a prompt's latents are cached and attended in expanded form; its
    tail is then served a token at a time in absorbed form, and as a chunk behind the
    read-back prefix. The three agree."""
    gen = torch.Generator(device=DEV).manual_seed(30)
    H, ps, lens = 8, 32, [150, 77]
    T = sum(lens)
    c, pe = rnd(gen, T, 512), rnd(gen, T, 64)
    w_k, w_v = rnd(gen, H, 128, 512, std=512 ** -0.5), rnd(gen, H, 128, 512, std=512 ** -0.5)
    q = rnd(gen, T, H, 192)
    table, pages = paged(lens, ps, seed=30)
    cache = latent.latent_cache(pages, ps, quantized=quantized, device=DEV)
    latent.latent_cache_write(c, pe, cache, slots_of(table, lens, ps))
    back = latent.latent_cache_read(cache, table, cu(lens), total=T)
    x = back[:, :512]

    def project(w):
        return torch.einsum("tc,hdc->thd", x.float(), w.float()).to(torch.bfloat16)

    kn, v = project(w_k), project(w_v)
    full, _ = latent.latent_attn_fwd(q, kn, back[:, 512:], v, cu_seqlens=cu(lens),
                                     max_seqlen=150)
    # the last 5 tokens of each sequence, behind their prefixes
    ends = [sum(lens[:i + 1]) for i in range(len(lens))]
    last = torch.cat([torch.arange(e - 5, e) for e in ends]).to(DEV)
    chunk, _ = latent.latent_attn_fwd(q[last], kn, back[:, 512:], v, cu_seqlens=cu([5, 5]),
                                      cu_seqlens_k=cu(lens), max_seqlen=5, max_seqlen_k=150)
    # the same keys, but q rows land at other places of their tiles
    assert ((chunk.float() - full[last].float()).abs() <= 4 * ref.U * (0.2 + full[last].float().abs())).all()
    # absorbed: the same tokens as L = 5 query tokens
    qa = torch.cat((torch.einsum("thd,hdc->thc", q[last][..., :128].float(), w_k.float()),
                    q[last][..., 128:].float()), -1).to(torch.bfloat16).view(2, 5, H, 576)
    o = latent.latent_decode(qa, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    o = torch.einsum("nlhc,hdc->nlhd", o.float(), w_v.float()).reshape(10, H, 128)
    # k_nope, v, the absorbed query and out are each rounded to bf16 on one side only: errors of
    # u relative in sums of 512 and 192 terms, a few hundredths of the values' spread (~1)
    diff = (o - full[last].float()).norm() / full[last].float().norm()
    assert diff < 8 * ref.U, float(diff)
