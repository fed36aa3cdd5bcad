"""Calls of the latent binding that its documentation allows and that were once refused, or answered
for another call than the one made."""
from __future__ import annotations

import pytest
import torch

DEV = "cuda:0"


@pytest.fixture(scope="module")
def latent():
    from kimi_delta_attention_19_b200 import latent as m
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_gradient_at_any_address(latent, packed):
    """Autograd hands on parts of larger gradients as views; one may start at any element."""
    from tests.test_latent_gpu import cu, expanded_inputs
    lens = [33, 20]
    q, kn, pe, v, g = expanded_inputs(lens, lens, 2, seed=3)
    kw = dict(cu_seqlens=cu(lens), max_seqlen=33) if packed else {}
    ins = [t.clone().requires_grad_() for t in (q, kn, pe, v)]
    few = torch.zeros(3, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    both = torch.cat([few, latent.latent_attention(*ins, **kw).flatten()])
    both.backward(torch.cat([torch.zeros(3, dtype=torch.bfloat16, device=DEV), g.flatten()]))
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
    want = latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw)
    assert all(torch.equal(t.grad, w) for t, w in zip(ins, want))
