"""The latent-attention kernels free tensor memory only once their products are done, also when the
last wait of all runs out.

On the CPU: every issuing role commits and waits for its last products without looking whether a
wait ran out before (a look there comes too early: the wait for the results may still run out).
On the GPU: in the test-only libkda_lastwait.so the wait for a unit's last products gives up at
once, so results are read, and the thread block ends, while products may be in flight. The call
must report device code 2, and the regular library must then give the bits it gave before.
"""
from __future__ import annotations

import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "kimi_delta_attention_19_b200", "csrc")
DEV = "cuda:0"


@pytest.mark.parametrize("name,roles", [("fwd", 1), ("bwd", 2), ("decode", 2)])
def test_products_are_waited_for_in_any_case(name, roles):
    with open(os.path.join(CSRC, f"kda_latent_{name}.cu")) as f:
        lines = [re.sub(r"//.*", "", line) for line in f]
    at = [i for i, line in enumerate(lines) if re.search(r"umma_commit\(drain", line)]
    assert len(at) == roles
    for i in at:
        assert "mbar_wait(drain" in lines[i + 1]
        assert "bail" not in lines[i - 1] and lines[i - 1].strip() in ("}", "umma_commit(o_full);")


@pytest.mark.gpu
@pytest.mark.timeout(300)
@pytest.mark.parametrize("what", ["decode", "decode 8 bit", "forward", "backward"])
def test_last_wait_running_out_is_reported(monkeypatch, what):
    from kimi_delta_attention_19_b200 import build as kbuild
    from kimi_delta_attention_19_b200 import kda, latent
    from tests.test_latent_gpu import cu, decode_case, expanded_inputs
    assert os.path.exists(kbuild.LASTWAIT_LIB), "build() makes the last-wait variant"
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    if what.startswith("decode"):
        x = decode_case(latent, [900, 3000, 64, 5], 32, 2, 64, what.endswith("bit"), seed=1)
        call = lambda: (latent.latent_decode(*x, status=st),)  # noqa: E731
    else:
        lens = [700, 300, 1]
        q, kn, pe, v, g = expanded_inputs(lens, lens, 3, seed=2)
        kw = dict(cu_seqlens=cu(lens), max_seqlen=700, status=st)
        out, lse = latent.latent_attn_fwd(q, kn, pe, v, **kw)
        call = (lambda: latent.latent_attn_fwd(q, kn, pe, v, **kw)) if what == "forward" else \
            (lambda: latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, **kw))
    good = call()
    assert int(st) == 0
    last = kda.load_library(kbuild.LASTWAIT_LIB)
    latent._declare(last)
    with monkeypatch.context() as m:
        m.setattr(latent, "lib", last)
        for _ in range(3):
            call()
        assert latent.status_of(st) == (kda.KDA_ERR_DEVICE, 2)    # synchronises
    st.zero_()
    again = call()
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(a, b) for a, b in zip(good, again))
