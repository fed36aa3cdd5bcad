"""What the latent-attention operators are measured on, with their plain forms.

A layer of latent attention keeps ONE vector a token for all heads: a latent c (512 values,
from which every head's keys and values are projected) and a shared part k_pe (64 values).
  expanded form  (prompts, training): keys [k_nope | k_pe] of 128 + 64 and values of 128
                 channels a head; softmax(scale q k^T) v, causal, packed sequences;
  absorbed form  (single and drafted tokens): the projections are folded into the query, so
                 the cached vectors themselves are the keys (576) and the values (512);
  cache          paged rows written a token at a time, in bf16 or with the latent in 8 bits
                 (e4m3 and one power-of-two scale for 128 channels), and read back.

`run` computes a case in elementary torch operations, or with `own` set by the calls of
kimi_delta_attention_19_b200.latent.
"""
import math
import random

import torch

own = False

D_NOPE, D_PE, D_V, D_C = 128, 64, 128, 512
ROW8 = 656                 # bytes of an 8-bit cache row: 512 codes, 64 bf16, 4 exponents, 12 unused
SCALE = 1.0 / math.sqrt(D_NOPE + D_PE)


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a handful of short requests arriving together: launch latency counts
        _prompt("prompt_short", n=4, H=16, lo=3, hi=70, pre=0, lens=1),
        # one 8K prompt with 32 heads, as the 8K x 32-head prefill of this library
        _prompt("prompt_8k", n=1, H=32, lo=8192, hi=8192, pre=0, lens=2),
        # chunked prefill: odd pieces of prompts behind cached prefixes read back and expanded
        _prompt("prompt_behind_prefix", n=4, H=32, lo=301, hi=1100, pre=2900, lens=3),
        # a training step of one 4K sequence: the pass and all its gradients
        _prompt("train_4k", n=1, H=32, lo=4096, hi=4096, pre=0, lens=4, kind="train"),
        # packed training documents of odd lengths, 16 heads
        _prompt("train_packed", n=6, H=16, lo=97, hi=1500, pre=0, lens=5, kind="train"),
        # one request being answered: a token over a short cache (latency)
        _token("token_one", n=1, H=32, L=1, lo=1003, hi=1003, page=64, bits=16, lens=6),
        # serving 256 sequences, one token each, caches of mixed lengths
        _token("token_256", n=256, H=32, L=1, lo=1024, hi=8192, page=64, bits=16, lens=7),
        # the million-token context with 16 heads: one sequence over the whole GPU
        _token("token_1m", n=1, H=16, L=1, lo=1 << 20, hi=1 << 20, page=128, bits=16, lens=8),
        # the serving batch with the cache held in 8 bits
        _token("token_256_8bit", n=256, H=32, L=1, lo=1024, hi=8192, page=64, bits=8, lens=9),
        # a tree of 8 drafted tokens a sequence, checked in one pass
        _token("draft_tree", n=16, H=32, L=8, lo=501, hi=6000, page=32, bits=8, lens=10),
        # what 8 sequences add to their caches in a step of a few tokens, and its read-back
        _cache("cache_step", n=8, lo=1, hi=40, page=16, bits=8, lens=11),
        # prompts of 64K tokens in all entering an 8-bit cache, and a prefix read back
        _cache("cache_prompts", n=8, lo=4096, hi=12000, page=64, bits=8, lens=12),
    ]


def _prompt(name, n, H, lo, hi, pre, lens, kind="prompt", causal=True):
    return {"name": name, "kind": kind, "n": n, "H": H, "lo": lo, "hi": hi, "pre": pre,
            "causal": causal, "lens": lens}


def _token(name, n, H, L, lo, hi, page, bits, lens):
    return {"name": name, "kind": "token", "n": n, "H": H, "L": L, "lo": lo, "hi": hi,
            "page": page, "bits": bits, "lens": lens}


def _cache(name, n, lo, hi, page, bits, lens):
    return {"name": name, "kind": "cache", "n": n, "lo": lo, "hi": hi, "page": page,
            "bits": bits, "lens": lens}


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    kind = rng.choice(("prompt", "train", "token", "token", "cache"))
    lens = rng.randrange(1 << 20)
    if kind in ("prompt", "train"):
        n, H = log(1, 12), rng.choice((1, 4, 7, 16, 32))
        most = 4096 if kind == "prompt" else 2048
        hi = log(2, most)
        while n * H * hi * hi > 2.6e8:     # scores of the plain form, all heads
            n, hi = max(1, n // 2), hi if n > 1 else hi // 2
        lo = rng.randint(1, hi)
        pre = rng.choice((0, 0, rng.randint(0, max(1, hi // 2))))
        case = _prompt("", n, H, lo, hi, pre, lens, kind, rng.random() < 0.8)
    elif kind == "token":
        n, L = log(1, 256), rng.choice((1, 1, 1, 2, 5, 8))
        hi = log(16, 1 << 18)
        H = rng.choice((1, 8, 16, 32, 64))
        while n * hi > 1 << 20 or n * hi * L * H > 2.5e8:
            hi = max(16, hi // 2)
        case = _token("", n, H, L, rng.randint(L, hi), hi,
                      rng.choice((16, 32, 64, 128)), rng.choice((8, 16)), lens)
    else:
        n = log(1, 64)
        hi = log(1, 60000 // n)
        case = _cache("", n, rng.randint(1, hi), hi, rng.choice((16, 32, 64, 128)),
                      rng.choice((8, 16)), lens)
    del case["name"]
    return case


def _lengths(case):
    """([query lengths], [key lengths]) of a case, from the case alone."""
    r = random.Random(case["lens"])
    q = [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    pre = case.get("pre", 0)
    return q, [x + (r.randint(0, pre) if pre else 0) for x in q]


# --------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lq, lk = _lengths(case)
    s = dict(case)

    def randn(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=gen, device="cuda")).to(torch.bfloat16)

    if case["kind"] in ("prompt", "train"):
        H, tq, tk = case["H"], sum(lq), sum(lk)
        kv = randn(tk, H, D_NOPE + D_V)           # one projection makes both, as in a model
        s.update(q=randn(tq, H, D_NOPE + D_PE, std=1.5), k_nope=kv[..., :D_NOPE],
                 v=kv[..., D_NOPE:], k_pe=randn(tk, D_PE), cu_q=_cu(lq), cu_k=_cu(lk),
                 max_q=max(lq), max_k=max(lk))
        if case["kind"] == "train":
            s["d_out"] = randn(tq, H, D_V)
        return s
    ps = case["page"]
    need = [-(-x // ps) for x in lq]
    pages = sum(need) + 3
    table = torch.zeros(case["n"], max(need), dtype=torch.int32)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = perm[at:at + k]
        at += k
    s.update(table=table.cuda(), max_len=max(lq))
    if case["kind"] == "token":
        L = case["L"]
        rows = randn(pages * ps, D_C + D_PE)
        s["cache"] = (rows if case["bits"] == 16 else _pack8(rows)).view(pages, ps, -1)
        s["q"] = randn(case["n"], L, case["H"], D_C + D_PE)
        s["seq_lens"] = torch.tensor(lq, dtype=torch.int32, device="cuda")
        s["mask"] = None
        if L > 1:     # every drafted token hangs on one before it and sees its ancestors
            r, words = random.Random(seed), []
            for _ in range(case["n"]):
                seen = [1]
                for i in range(1, L):
                    seen.append(seen[r.randrange(i)] | 1 << i)
                words.append(seen)
            s["mask"] = torch.tensor(words, dtype=torch.int64, device="cuda")
        return s
    T = sum(lq)
    s["c"] = randn(T, D_C) * torch.exp(randn(T, 1, std=1.0))
    s["k_pe"] = randn(T, D_PE)
    s["cache"] = torch.zeros(pages, ps, D_C + D_PE, dtype=torch.bfloat16, device="cuda") \
        if case["bits"] == 16 else torch.zeros(pages, ps, ROW8, dtype=torch.uint8, device="cuda")
    pos = torch.cat([torch.arange(x) for x in lq])
    seq = torch.repeat_interleave(torch.arange(case["n"]), torch.tensor(lq))
    s["slots"] = (table[seq, pos // ps].long() * ps + pos % ps).cuda()
    s["cu_q"], s["total"] = _cu(lq), T
    return s


def _cu(lengths):
    c = [0]
    for x in lengths:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from kimi_delta_attention_19_b200 import latent
    if s["kind"] in ("prompt", "train"):
        seqs = dict(cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"], max_seqlen=s["max_q"],
                    max_seqlen_k=s["max_k"], causal=s["causal"])
        out, lse = latent.latent_attn_fwd(s["q"], s["k_nope"], s["k_pe"], s["v"], **seqs)
        if s["kind"] == "prompt":
            return out, lse
        return (out,) + latent.latent_attn_bwd(s["q"], s["k_nope"], s["k_pe"], s["v"], out, lse,
                                               s["d_out"], **seqs)
    if s["kind"] == "token":
        return latent.latent_decode(s["q"], s["cache"], s["table"], s["seq_lens"],
                                    draft_mask=s["mask"])
    latent.latent_cache_write(s["c"], s["k_pe"], s["cache"], s["slots"])
    return latent.latent_cache_read(s["cache"], s["table"], s["cu_q"], total=s["total"])


def _run_plain(s):
    if s["kind"] in ("prompt", "train"):
        return _plain_expanded(s)
    if s["kind"] == "token":
        return _plain_absorbed(s)
    rows = torch.cat((s["c"], s["k_pe"]), -1)
    s["cache"].view(-1, s["cache"].shape[-1])[s["slots"]] = \
        rows if s["bits"] == 16 else _pack8(rows)
    back = s["cache"].view(-1, s["cache"].shape[-1])[s["slots"]]
    return back if s["bits"] == 16 else _unpack8(back).to(torch.bfloat16)


def _padded(cu, most):
    """Packed positions [n, most] and whether there is a token."""
    at = torch.arange(most, device="cuda")
    there = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + at, 0).long(), there


def _plain_expanded(s):
    iq, oq = _padded(s["cu_q"], s["max_q"])
    ik, ok = _padded(s["cu_k"], s["max_k"])
    k = torch.cat((s["k_nope"], s["k_pe"][:, None].expand(-1, s["H"], -1)), -1)
    q = s["q"][iq].float().transpose(1, 2)                     # [n, H, mq, 192]
    k = k[ik].float().transpose(1, 2)
    v = s["v"][ik].float().transpose(1, 2)
    x = (q @ k.transpose(-1, -2)) * SCALE                      # [n, H, mq, mk]
    seen = oq[:, None, :, None] & ok[:, None, None, :]
    if s["causal"]:
        lag = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])
        i = torch.arange(s["max_q"], device="cuda")
        j = torch.arange(s["max_k"], device="cuda")
        seen = seen & (j <= i[:, None] + lag[:, None, None])[:, None]
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp_(x.sub_(torch.where(top == -math.inf, 0, top)))
    total = x.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]                     # -inf where nothing is seen
    p = x.div_(torch.where(total == 0, 1, total))
    o = p @ v
    out = o.transpose(1, 2)[oq].to(torch.bfloat16)             # packed again: [T, H, 128]
    if s["kind"] == "prompt":
        return out, lse.transpose(1, 2)[oq]
    d_out = torch.where(oq[..., None, None], s["d_out"][iq].float(), 0).transpose(1, 2)
    dv = p.transpose(-1, -2) @ d_out
    ds = d_out @ v.transpose(-1, -2)
    ds.sub_((d_out * o).sum(-1, keepdim=True)).mul_(p).mul_(SCALE)
    dq = ds @ k
    dk = ds.transpose(-1, -2) @ q
    dq, dk, dv = (t.transpose(1, 2)[o_].to(torch.float32)
                  for t, o_ in ((dq, oq), (dk, ok), (dv, ok)))
    return (out, dq.to(torch.bfloat16), dk[..., :D_NOPE].to(torch.bfloat16),
            dk[..., D_NOPE:].sum(1).to(torch.bfloat16), dv.to(torch.bfloat16))


def _plain_absorbed(s):
    L, ps, most = s["L"], s["page"], s["max_len"]
    at = torch.arange(most, device="cuda")
    there = at < s["seq_lens"][:, None]
    slot = torch.where(there, s["table"][:, at // ps].long() * ps + at % ps, 0)
    rows = s["cache"].view(-1, s["cache"].shape[-1])[slot]
    x = rows.float() if s["bits"] == 16 else _unpack8(rows)    # [n, most, 576]
    n = x.shape[0]
    q = s["q"].float().reshape(n, L * s["H"], -1)
    a = (q @ x.transpose(1, 2)).mul_(SCALE).view(n, L, s["H"], most)
    seen = there[:, None, :]
    if L > 1:         # position of a key among the drafted tokens; the cache before them is seen
        j = at - (s["seq_lens"][:, None] - L)
        bit = (s["mask"][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
        seen = seen & ((j < 0)[:, None, :] | (bit != 0))
    p = torch.softmax(a.masked_fill_(~seen[:, :, None, :], -math.inf), -1)
    o = p.view(n, -1, most) @ x[..., :D_C]
    return o.view(n, L, s["H"], D_C).to(torch.bfloat16)


def _pack8(rows):
    """8-bit cache rows [.., 656] of bf16 rows [.., 576]: the latent as e4m3 codes of x / 2^e,
    e the smallest exponent a 128-channel group's largest value fits with, biased by 127."""
    x = rows[:, :D_C].float().view(-1, 4, 128)
    m, e = torch.frexp(x.abs().amax(-1))               # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = (e - 9 + (m > 0.875)).clamp(-120, 120)
    y = x * _pow2(-e)[..., None]
    out = torch.zeros(rows.shape[0], ROW8, dtype=torch.uint8, device=rows.device)
    out[:, :D_C] = y.to(torch.float8_e4m3fn).view(torch.uint8).view(-1, D_C)
    out[:, D_C:D_C + 2 * D_PE] = rows[:, D_C:].contiguous().view(torch.uint8)
    out[:, D_C + 2 * D_PE:D_C + 2 * D_PE + 4] = (e + 127).to(torch.uint8)
    return out


def _unpack8(rows):
    """The fp32 values [.., 576] that 8-bit cache rows stand for."""
    lead = rows.shape[:-1]
    y = rows[..., :D_C].contiguous().view(torch.float8_e4m3fn).float().view(*lead, 4, 128)
    e = rows[..., D_C + 2 * D_PE:D_C + 2 * D_PE + 4].int()[..., None] - 127
    pe = rows[..., D_C:D_C + 2 * D_PE].contiguous().view(torch.bfloat16).float()
    return torch.cat(((y * _pow2(e)).view(*lead, D_C), pe), -1)


def _pow2(e):
    """2^e in fp32, exactly (a product with it rounds nothing), for -126 <= e <= 127."""
    return (e.to(torch.int32) + 127 << 23).view(torch.float32)


# ----------------------------------------------------------------------- work and 64 bits
def work(case):
    lq, lk = _lengths(case)
    if case["kind"] in ("prompt", "train"):
        H = case["H"]
        pairs = sum(a * b - a * (a - 1) // 2 if case["causal"] else a * b for a, b in zip(lq, lk))
        tq, tk = sum(lq), sum(lk)
        q, kv, pe, o = tq * H * 192 * 2, tk * H * 256 * 2, tk * 64 * 2, tq * H * 128 * 2
        if case["kind"] == "prompt":
            return {"bytes": q + kv + pe + o + tq * H * 4, "flops": 2 * 320 * H * pairs}
        # S and O; dV, dP, dQ, dK (scores and probabilities kept or not is the kernel's affair)
        return {"bytes": 2 * (q + kv + pe + o), "flops": 2 * 960 * H * pairs}
    row = 1152 if case["bits"] == 16 else 644
    if case["kind"] == "token":
        heads = case["n"] * case["L"] * case["H"]
        return {"bytes": sum(lq) * row + heads * (576 + 512) * 2,
                "flops": 2 * (576 + 512) * case["L"] * case["H"] * sum(lq)}
    return {"bytes": sum(lq) * (1152 + row + row + 1152), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    lq, lk = _lengths(case)
    if case["kind"] in ("prompt", "train"):
        return _exact_expanded(s, lq, lk)
    if case["kind"] == "cache":
        return _exact_cache(s)
    flat = s["cache"].view(-1, s["cache"].shape[-1])
    out = torch.empty(case["n"], case["L"], case["H"], D_C, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lq):
        pages = s["table"][i, :-(-n // s["page"])].long()
        x = flat.view(-1, s["page"], flat.shape[-1])[pages].reshape(-1, flat.shape[-1])[:n]
        if case["bits"] == 8:
            x = torch.cat((
                _values8(x[:, :D_C]) * _two(x[:, 640:644].long() - 127).repeat_interleave(128, 1),
                x[:, D_C:640].contiguous().view(torch.bfloat16).double()), 1)
        x = x.double()
        for t in range(case["L"]):
            a = s["q"][i, t].double() @ x.T / math.sqrt(192)
            if case["L"] > 1:
                word = int(s["mask"][i, t])
                for j in range(case["L"]):
                    if not word >> j & 1 and n - case["L"] + j >= 0:
                        a[:, n - case["L"] + j] = -math.inf
            a = torch.exp(a - a.max(1, keepdim=True).values)
            out[i, t] = (a @ x[:, :D_C]) / a.sum(1, keepdim=True)
    return out


def _values8(code):
    """e4m3 codes as 64-bit values, from the format: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    c = code.long()
    e, m = c >> 3 & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _two(e - 7))
    return torch.where(c >= 128, -mag, mag)


def _two(e):
    """2^e in 64 bits, from the exponent field."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _exact_cache(s):
    x = s["c"].double()
    if s["bits"] == 8:
        g = x.view(-1, 4, 128)
        top = g.abs().amax(-1, keepdim=True)
        e = torch.round(torch.log2(torch.where(top == 0, 2.0 ** -130, top) / 448)).long()
        e = (e + (top > 448 * _two(e)).long()).clamp(-120, 120)    # the least e that holds top
        y = g / _two(e)
        step = _two((y.abs().clamp_min(2.0 ** -6).view(torch.int64) >> 52) - 1023 - 3)
        x = (torch.round(y / step) * step * _two(e)).view(-1, D_C)
    return torch.cat((x, s["k_pe"].double()), 1)


def _exact_expanded(s, lq, lk):
    train, H = s["kind"] == "train", s["H"]
    new = lambda like: torch.zeros(like.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = torch.zeros(sum(lq), H, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(lq), H), -math.inf, dtype=torch.float64, device="cuda")
    dq, dkn, dpe, dv = new(s["q"]), new(s["k_nope"]), new(s["k_pe"]), new(s["v"])
    tq = tk = 0
    for a, b in zip(lq, lk):
        rq, rk = slice(tq, tq + a), slice(tk, tk + b)
        tq, tk = tq + a, tk + b
        hidden = torch.ones(a, b, dtype=torch.bool, device="cuda").triu(b - a + 1)
        for h in range(H):
            q, v = s["q"][rq, h].double(), s["v"][rk, h].double()
            k = torch.cat((s["k_nope"][rk, h], s["k_pe"][rk]), 1).double()
            x = q @ k.T / math.sqrt(192)
            if s["causal"]:
                x[hidden] = -math.inf
            lse[rq, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[rq, h, None].nan_to_num(neginf=0.0))
            out[rq, h] = p @ v
            if train:
                g = s["d_out"][rq, h].double()
                dv[rk, h] = p.T @ g
                ds = p * (g @ v.T - (g * out[rq, h]).sum(1, keepdim=True)) / math.sqrt(192)
                dq[rq, h] = ds @ k
                dk = ds.T @ q
                dkn[rk, h] = dk[:, :D_NOPE]
                dpe[rk] += dk[:, D_NOPE:]
    return (out, dq, dkn, dpe, dv) if train else (out, lse)
