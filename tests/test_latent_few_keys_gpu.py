"""Many queries of a few keys, without causality: the backward's exact sums for such rows run all over
the GPU, not on a few thread blocks of each head."""
from __future__ import annotations

import pytest
import torch

from tests import latent_ref as ref
from tests.test_latent_gpu import expanded_inputs

pytestmark = pytest.mark.gpu


def step(n, keys, H=1, seed=1):
    from kimi_delta_attention_19_b200 import latent
    q, kn, pe, v, g = expanded_inputs([n], [keys], H, seed=seed)
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, causal=False)
    return (q, kn, pe, v, g, out), lambda: latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, causal=False)


@pytest.mark.parametrize("n,keys,H", [(5001, 32, 2), (3000, 1, 1), (9, 20, 3), (20011, 5, 1)])
def test_gradients_of_many_queries_of_few_keys(n, keys, H):
    (q, kn, pe, v, g, out), call = step(n, keys, H)
    want = ref.expanded(q, kn, pe, v, [n], [keys], False, d_out=g, out_used=out)
    for name, got in zip(("dq", "dk_nope", "dk_pe", "dv"), call()):
        ref.inside(got, want[name], want["b_" + name], name)


def test_few_keys_cost_about_what_more_keys_cost():
    """One head, 64 K queries: 32 keys against 33, whose rows take no such sums. The sums are 320
    products a pair, 0.7 G in all: a tenth of a millisecond on all of the GPU's multipliers, where
    the walk over 64 K queries takes over one; on four thread blocks they took five times that."""
    def time(keys):
        _, call = step(1 << 16, keys)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert time(32) < 2 * time(33)
