"""Gradients of latent attention against the formula's own, all in 64 bits: D is the formula's sum,
not formed from the out that the kernels rounded.

The limit on each gradient's error, over all its elements together, is the sum of what the
kernels' roundings to bf16 may bring. A value m 2^e, 1 <= m < 2, is off by at most 2^-8 2^e, evenly
spread: its relative error's mean square is 2^-16 / 3 / m^2, and with m spread as the digits of
products and sums are (evenly in its logarithm) the mean of 1/m^2 is 3 / (8 ln 2) = 0.541. So a
rounding brings r^2 = 0.541 * 2^-16 / 3 of a value's square (r = 1.66e-3), and as roundings are
independent, their squares add:

    the result itself                      r^2 |value|^2
    p in dv, dS in dq and dk (the terms    r^2 sum p^2 dO^2,  r^2 sum dS^2 k^2,  r^2 sum dS^2 q^2
    of a sum are off independently)
    out, through D_i = dO_i . out_i        v_i = r^2 sum_c (dO out)^2, and from it
                                           v_i (scale sum_j p k)^2,  sum_i v_i (scale p q)^2

dS of sequences of at most 384 keys is documented to be kept in two bf16 terms (2^-16 of it is
lost): its line is left out there. What fp32 adds (scores of 192 products at 2^-24 of magnitudes of
some tens) is a thousandth of these. An eighth more is allowed: the squares of some thousand
independent errors come within some hundredths of what is expected, but a few rows of large
gradients count for most of a short sequence's."""
from __future__ import annotations

import math

import pytest
import torch

from tests.test_latent_gpu import cu, expanded_inputs

pytestmark = pytest.mark.gpu
R2 = 3 / (8 * math.log(2)) * 2.0 ** -16 / 3


def true_gradients(q, kn, pe, v, g, lq, lk, causal):
    """{name: (gradient, expected square of each element's error)} of packed sequences."""
    H, scale = q.shape[1], 1 / math.sqrt(192)
    acc = {n: ([], []) for n in ("dq", "dk_nope", "dk_pe", "dv")}
    a0 = b0 = 0
    for a, b in zip(lq, lk):
        sq, sk = slice(a0, a0 + a), slice(b0, b0 + b)
        a0, b0 = a0 + a, b0 + b
        Q, G, V = (t.double().transpose(0, 1) for t in (q[sq], g[sq], v[sk]))
        K = torch.cat((kn[sk].double(), pe[sk].double()[:, None].expand(-1, H, -1)), -1).transpose(0, 1)
        x = scale * Q @ K.transpose(1, 2)
        if causal:
            hide = torch.arange(b, device=q.device)[None] > torch.arange(a, device=q.device)[:, None] + b - a
            x = x.masked_fill(hide, -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1))
        dp = G @ V.transpose(1, 2)
        ds = scale * p * (dp - (p * dp).sum(-1, keepdim=True))
        r2 = R2 if b > 384 else 0.0                                     # of dS
        vd = R2 * ((G * (p @ V)) ** 2).sum(-1, keepdim=True)            # of D

        def put(name, val, var):
            acc[name][0].append(val)
            acc[name][1].append(var + R2 * val ** 2)

        put("dq", (ds @ K).transpose(0, 1),
            (r2 * ds ** 2 @ K ** 2 + vd * (scale * p @ K) ** 2).transpose(0, 1))
        dk = ds.transpose(1, 2) @ Q
        ek = r2 * (ds ** 2).transpose(1, 2) @ Q ** 2 + \
            (scale ** 2 * p ** 2 * vd).transpose(1, 2) @ Q ** 2
        put("dk_nope", dk[..., :128].transpose(0, 1), ek[..., :128].transpose(0, 1))
        put("dk_pe", dk[..., 128:].sum(0), ek[..., 128:].sum(0))
        put("dv", (p.transpose(1, 2) @ G).transpose(0, 1),
            (R2 * (p ** 2).transpose(1, 2) @ G ** 2).transpose(0, 1))
    return {n: (torch.cat(x), torch.cat(y)) for n, (x, y) in acc.items()}


@pytest.mark.parametrize("lq,lk,causal", [
    ([33], [33], True), ([33] * 40, [33] * 40, True), ([40, 50, 64] * 5, [40, 50, 64] * 5, True),
    ([245] * 4, [245] * 4, True), ([384] * 3, [384] * 3, True), ([385] * 3, [385] * 3, True),
    ([425] * 3, [425] * 3, True), ([1000], [1000], True), ([2100], [2100], True),
    ([125], [425], True), ([64] * 4, [320] * 4, True), ([300], [600], True), ([8] * 9, [1000] * 9, True),
    ([3] * 30, [36] * 30, True), ([200], [33], False), ([200], [384], False), ([200], [385], False),
    ([90], [1000], False),
])
def test_gradients_against_the_formulas_own(lq, lk, causal):
    from kimi_delta_attention_19_b200 import latent
    q, kn, pe, v, g = expanded_inputs(lq, lk, 4, seed=len(lq) + lk[0])
    kw = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk), max_seqlen=max(lq), max_seqlen_k=max(lk),
              causal=causal)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    grads = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    want = true_gradients(q, kn, pe, v, g, lq, lk, causal)
    for (name, (val, var)), got in zip(want.items(), grads):
        off = float((got.double() - val).norm() / val.norm())
        most = 1.125 * math.sqrt(float(var.sum())) / float(val.norm())
        assert off <= most, (name, off, most)
