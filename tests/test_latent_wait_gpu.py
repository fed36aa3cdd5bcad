"""GPU test of the latent-attention kernels' bounded waits running out.

In the test-only libkda_shortwait.so every wait of these kernels gives up after 64 clocks, so
most do. A call through it must report device code 2 in the status word and return (copies and
products drained, tensor memory freed), and the regular library must then give the same bits
as before on the same device.
"""
from __future__ import annotations

import os

import pytest
import torch

from tests.test_latent_gpu import DEV, cu, decode_case, expanded_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def latent():
    from kimi_delta_attention_19_b200 import latent as m
    return m


@pytest.mark.timeout(300)
@pytest.mark.parametrize("what", ["decode", "decode 8 bit", "forward", "backward"])
def test_waits_running_out_are_reported(latent, monkeypatch, what):
    from kimi_delta_attention_19_b200 import build as kbuild
    from kimi_delta_attention_19_b200 import kda
    assert os.path.exists(kbuild.SHORTWAIT_LIB), "build() makes the short-wait variant"
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    if what.startswith("decode"):
        x = decode_case(latent, [900, 3000, 64], 32, 2, 64, what.endswith("bit"), seed=1)
        call = lambda: (latent.latent_decode(*x, status=st),)  # noqa: E731
    else:
        lens = [700, 300]
        q, kn, pe, v, g = expanded_inputs(lens, lens, 3, seed=2)
        kw = dict(cu_seqlens=cu(lens), max_seqlen=700, status=st)
        out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
        call = (lambda: latent.latent_attn_fwd(q, kn, pe, v, **kw)) if what == "forward" else \
            (lambda: latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw))
    good = call()
    assert int(st) == 0
    short = kda.load_library(kbuild.SHORTWAIT_LIB)
    latent._declare(short)
    with monkeypatch.context() as m:
        m.setattr(latent, "lib", short)
        call()
        assert latent.status_of(st) == (kda.KDA_ERR_DEVICE, 2)    # synchronises
    st.zero_()
    again = call()
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(a, b) for a, b in zip(good, again))
