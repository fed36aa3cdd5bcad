"""fp64 references of the latent-attention operators, from their formulas, with the error
bounds the kernels are held to.

Bounds count roundings to bf16 (half a step: u = 2^-8 relative): probabilities and score
gradients are rounded once before a product, results once at the end, so a sum of terms t
may be off by u * (sum |t| + |result|); the factor 1.05 leaves room for what fp32 adds
(scores of 192 or 576 products at 2^-24 each, the exponential's few ulps), `tiny` for
results that cancel to nothing."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8


def bound(result, sum_abs, tiny=1e-6):
    return 1.05 * U * (result.abs() + sum_abs) + tiny


def expanded(q, k_nope, k_pe, v, lq, lk, causal, scale=None, d_out=None, out_used=None):
    """Packed references: out, lse, bounds and (with d_out) gradients and their bounds, as a
    dict; a dict's "b_x" bounds "x". Rows of no sequence are NaN. out_used: the out the
    backward was given (D of rows that see more than 32 keys is formed from it)."""
    scale = scale if scale is not None else 1 / math.sqrt(q.shape[-1])
    H = q.shape[1]
    r = {}

    def nan(t, d=None):
        shape = t.shape if d is None else t.shape[:-1] + (d,)
        return torch.full(shape, math.nan, dtype=torch.float64, device=t.device)

    for n in ("out", "b_out"):
        r[n] = nan(q, v.shape[-1])
    r["lse"] = torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=q.device)
    for n, t in (("dq", q), ("dk_nope", k_nope), ("dk_pe", k_pe), ("dv", v)):
        r[n], r["b_" + n] = nan(t), nan(t)
    a0 = b0 = 0
    for a, b in zip(lq, lk):
        sq, sk = slice(a0, a0 + a), slice(b0, b0 + b)
        a0, b0 = a0 + a, b0 + b
        Q = q[sq].double().transpose(0, 1)
        K = torch.cat((k_nope[sk].double(), k_pe[sk].double()[:, None].expand(-1, H, -1)),
                      -1).transpose(0, 1)
        V = v[sk].double().transpose(0, 1)
        x = scale * Q @ K.transpose(1, 2)
        if causal:
            i = torch.arange(a, device=q.device)[:, None]
            j = torch.arange(b, device=q.device)[None]
            x = x.masked_fill(j > i + b - a, -math.inf)
        lse = torch.logsumexp(x, -1) if b else torch.full(x.shape[:2], -math.inf, device=q.device,
                                                          dtype=torch.float64)
        p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        o = p @ V
        r["out"][sq] = o.transpose(0, 1)
        r["b_out"][sq] = bound(o, p @ V.abs()).transpose(0, 1)
        r["lse"][sq] = lse.transpose(0, 1)
        if d_out is None:
            continue
        g = d_out[sq].double().transpose(0, 1)
        oo = out_used[sq].double().transpose(0, 1)
        dp = g @ V.transpose(1, 2)
        few = (x > -math.inf).sum(-1, keepdim=True) <= 32   # there D is the formula's own sum
        D = torch.where(few, (p * dp).sum(-1, keepdim=True), (g * oo).sum(-1, keepdim=True))
        ds = scale * p * (dp - D)
        # fp32 sums inside dP and D (128 terms at 2^-24 of their magnitudes) before the
        # difference, the exponential, and ds rounded to bf16
        slack = scale * p * ((g.abs() @ V.abs().transpose(1, 2))
                             + (g * oo).abs().sum(-1, keepdim=True)) * 2.0 ** -17
        e = U * ds.abs() + slack

        def put(name, s, val, err):
            r[name][s] = val.transpose(0, 1) if val.dim() == 3 else val
            bb = 1.05 * (U * val.abs() + err) + 1e-6
            r["b_" + name][s] = bb.transpose(0, 1) if bb.dim() == 3 else bb

        dk, ek = ds.transpose(1, 2) @ Q, e.transpose(1, 2) @ Q.abs()
        put("dq", sq, ds @ K, e @ K.abs())
        put("dk_nope", sk, dk[..., :128], ek[..., :128])
        put("dk_pe", sk, dk[..., 128:].sum(0), ek[..., 128:].sum(0))
        put("dv", sk, p.transpose(1, 2) @ g, U * (p.transpose(1, 2) @ g.abs()))
    return r


def quantize(c):
    """(values [T, 512], exponents [T, 4]) an 8-bit row holds of latents c [T, 512], in 64 bits."""
    x = c.double().view(-1, 4, 128)
    fin = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    e = torch.full(fin.shape, -120, dtype=torch.int64, device=c.device)
    for k in range(-119, 121):        # the least e in range with fin <= 448 * 2^e
        e = torch.where(fin > 448.0 * 2.0 ** (k - 1), k, e)
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), e.cpu().double()).to(c.device)[..., None]
    y = x / s
    m, ex = torch.frexp(y.abs().clamp_min(2.0 ** -6))
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), (ex - 4).cpu().double()).to(c.device)
    v = torch.round(y / step) * step * s
    return torch.where(torch.isfinite(x), v, math.nan).view(-1, 512), e


def rows_of(cache):
    """The fp64 vectors [rows, 576] a cache tensor stands for, from the row formats."""
    flat = cache.reshape(-1, cache.shape[-1])
    if cache.dtype == torch.bfloat16:
        return flat.double()
    code = flat[:, :512].long()
    e, m = code >> 3 & 15, (code & 7).double()
    table = torch.tensor([2.0 ** (i - 7) for i in range(16)], dtype=torch.float64,
                         device=cache.device)
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * table[e])
    v = torch.where(code & 127 == 127, math.nan, torch.where(code > 127, -v, v))
    ex = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64,
                      device=cache.device)[flat[:, 640:644].long()]
    pe = flat[:, 512:640].contiguous().view(torch.bfloat16).double()
    return torch.cat((v * ex.repeat_interleave(128, 1), pe), 1)


def absorbed(q, cache, table, lens, mask=None, scale=None):
    """(out, bound, lse) [N, L, H, ..] of absorbed attention, q [N, L, H, 576]."""
    scale = scale if scale is not None else 1 / math.sqrt(192)
    N, L, H, _ = q.shape
    ps = cache.shape[1]
    x_all = rows_of(cache)
    out = torch.zeros(N, L, H, 512, dtype=torch.float64, device=q.device)
    bnd, lse = torch.zeros_like(out), torch.full((N, L, H), -math.inf, dtype=torch.float64,
                                                 device=q.device)
    for n, ln in enumerate(lens):
        if ln == 0:
            continue
        pos = torch.arange(ln, device=q.device)
        x = x_all[table[n].long()[pos // ps] * ps + pos % ps]
        j = pos - (ln - L)
        for i in range(L):
            seen = j <= i if mask is None else \
                (j < 0) | ((int(mask[n, i]) >> j.clamp(0, 63)) & 1).bool()
            y = x[seen]
            if not len(y):
                continue
            s = scale * q[n, i].double() @ y.T
            lse[n, i] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[n, i][:, None])
            out[n, i] = p @ y[:, :512]
            bnd[n, i] = bound(out[n, i], p @ y[:, :512].abs())
    return out, bnd, lse


def inside(got, want, bnd, what=""):
    """Every element within its bound (and NaN of `want`, rows of no sequence, left out)."""
    there = ~torch.isnan(want)
    err = (got.double() - want).abs()
    err = torch.where(there, err, torch.zeros_like(err))
    bad = ~(err <= torch.where(there, bnd, torch.ones_like(bnd)))
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside their bound, first "
                             f"at {at}: got {float(got[at])}, want {float(want[at])} "
                             f"+- {float(bnd[at])}")


def lse_close(got, want):
    """lse: fp32 sums, and scores off by some 2^-24 of sums of up to 576 products."""
    there = ~torch.isnan(want)
    empty = want == -math.inf
    assert torch.equal((got == -math.inf)[there], empty[there])
    ok = there & ~empty
    assert ((got.double() - want)[ok].abs() <= 2e-5 * (1 + want[ok].abs())).all()
