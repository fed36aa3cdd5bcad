"""Query rows that see no key add nothing to any gradient, whatever they and their d_out hold (the
gradient of a norm of such a row's zeros is NaN, for instance)."""
from __future__ import annotations

import math

import pytest
import torch

from tests import latent_ref as ref
from tests.test_latent_gpu import cu, expanded_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("lq,lk", [([40], [10]), ([64], [1]), ([65], [64]), ([300], [172]), ([200, 90], [71, 89]),
                                   ([100, 33, 20], [36, 33, 0]), ([129], [65]), ([600], [7])])
def test_rows_that_see_nothing_may_hold_anything(lq, lk, bad):
    from kimi_delta_attention_19_b200 import latent
    H = 2
    q, kn, pe, v, g = expanded_inputs(lq, lk, H, seed=1)
    kw = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk), max_seqlen=max(lq), max_seqlen_k=max(lk))
    blind = torch.cat([torch.arange(a) < a - b for a, b in zip(lq, lk)]).to(q.device)

    def step():
        out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
        return (out, lse) + latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)

    clean = step()
    assert (clean[1][blind] == -math.inf).all() and torch.isfinite(clean[1][~blind]).all()
    want = ref.expanded(q, kn, pe, v, lq, lk, True, d_out=g, out_used=clean[0])
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), clean[2:]):
        ref.inside(got, want[name], want["b_" + name], name)
    q[blind], g[blind] = bad, bad
    dirty = step()
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
