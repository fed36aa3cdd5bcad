"""What the latent-attention kernels find wrong on the device is never lost: calls without a
`status` tensor report in a word that the library keeps, and latent_attention takes one too."""
from __future__ import annotations

import inspect
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


@pytest.fixture(scope="module")
def latent():
    from kimi_delta_attention_19_b200 import latent as m
    return m


def test_every_call_takes_a_status_word(latent):
    for f in (latent.latent_attention, latent.latent_attn_fwd, latent.latent_attn_bwd,
              latent.latent_decode, latent.latent_cache_write, latent.latent_cache_read):
        assert inspect.signature(f).parameters["status"].default is None, f.__name__
    assert hasattr(latent.lib, "kda_latent_status") and "kda_latent_status" in latent.EXPORTED


@pytest.fixture
def case(latent):
    """(inputs, tight and too small bounds); the word is clear before and after."""
    from tests.test_latent_gpu import cu, expanded_inputs
    lens = [40, 90, 33]
    latent.latent_status()
    yield expanded_inputs(lens, lens, 2, seed=1), cu(lens)
    torch.cuda.synchronize()
    assert latent.latent_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_attention_reports_a_too_small_bound(latent, case, given):
    (q, kn, pe, v, g), off = case
    st = torch.zeros(1, dtype=torch.int32, device=DEV) if given else None

    def asked():
        if given:
            assert latent.latent_status() == (0, 0)
            r = latent.status_of(st)
            st.zero_()
            return r
        return latent.latent_status()

    ins = [t.clone().requires_grad_() for t in (q, kn, pe, v)]
    out = latent.latent_attention(*ins, cu_seqlens=off, max_seqlen=90, status=st)
    out.backward(g)
    assert asked() == (0, 0)
    good = [t.grad.clone() for t in ins]
    for t in ins:
        t.grad = None
    out = latent.latent_attention(*ins, cu_seqlens=off, max_seqlen=89, status=st)
    assert asked() == (4, 1)
    assert (out[40:130] == 0).all() and (out[130:] != 0).any()
    out.backward(g)
    assert asked() == (4, 1)
    assert asked() == (0, 0)                                     # asked once, then clear
    for t, w in zip(ins, good):
        assert (t.grad[40:130] == 0).all()
        assert torch.equal(t.grad[:40], w[:40]) and torch.equal(t.grad[130:], w[130:])


@pytest.mark.gpu
def test_calls_without_a_status_tensor_report(latent, case):
    (q, kn, pe, v, g), off = case
    out, lse = latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=off, max_seqlen=90)
    assert latent.latent_status() == (0, 0)
    latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=off, max_seqlen=89)
    assert latent.latent_status() == (4, 1)
    latent.latent_attn_bwd(q, kn, pe, v, out, lse, g, cu_seqlens=off, max_seqlen=89)
    assert latent.latent_status() == (4, 1)
    bad = off.clone()
    bad[1] = 91                                                  # then sequence 1 has -1 tokens
    bad[2] = 90
    latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=bad, out=out, lse=lse)   # not the usual call
    assert latent.latent_status(DEV) == (4, 1)

    from tests.test_latent_gpu import cu, decode_case
    for quantized in (False, True):
        x = decode_case(latent, [40, 9], 4, 1, 16, quantized, seed=2)
        latent.latent_decode(*x)
        assert latent.latent_status() == (0, 0)
        x[2][0, 1] = x[1].shape[0]
        latent.latent_decode(*x)
        assert latent.latent_status() == (4, 3)
        latent.latent_cache_read(x[1], x[2], cu([20, 5]), total=25)
        assert latent.latent_status() == (4, 3)
        latent.latent_cache_write(q[:2, 0].repeat(1, 3)[:, :512].contiguous(), pe[:2], x[1],
                                  torch.tensor([0, 1 << 40], device=DEV))
        assert latent.latent_status() == (4, 3)


@pytest.mark.gpu
def test_a_given_word_and_the_librarys_are_apart(latent, case):
    (q, kn, pe, v, g), off = case
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=off, max_seqlen=89, status=st)
    assert latent.latent_status() == (0, 0) and latent.status_of(st) == (4, 1)


@pytest.mark.gpu
def test_calls_on_a_stream_and_replays_report(latent, case):
    (q, kn, pe, v, g), off = case
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=off, max_seqlen=89, stream=side)
    assert latent.latent_status(stream=side) == (4, 1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        latent.latent_attn_fwd(q, kn, pe, v, cu_seqlens=off, max_seqlen=89)
    assert latent.latent_status() == (0, 0)
    for _ in range(2):
        graph.replay()
        assert latent.latent_status() == (4, 1)


@pytest.mark.gpu
def test_the_first_call_of_a_process_may_be_captured():
    """The library's word is looked up without anything that a capture does not allow."""
    code = """
import torch
from kimi_delta_attention_19_b200 import latent
x = [torch.zeros(9, 2, 192, device='cuda'), torch.zeros(9, 2, 128, device='cuda'),
     torch.zeros(9, 64, device='cuda'), torch.ones(9, 2, 128, device='cuda')]
x = [t.to(torch.bfloat16) for t in x]
off = torch.tensor([0, 4, 9], dtype=torch.int32, device='cuda')
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    with torch.no_grad():
        out = latent.latent_attention(*x, cu_seqlens=off, max_seqlen=4)
graph.replay()
assert latent.latent_status() == (4, 1)
assert (out[:4] == 1).all() and (out[4:] == 0).all()
print('fine')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
