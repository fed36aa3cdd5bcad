"""Calls of the latent binding that its documentation allows and that were once refused, or answered
for another call than the one made."""
from __future__ import annotations

import math
import types

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


def inputs(H=2, T=8):
    bf = torch.bfloat16
    return (torch.zeros(T, H, 192, dtype=bf), torch.zeros(T, H, 128, dtype=bf),
            torch.zeros(T, 64, dtype=bf), torch.zeros(T, H, 128, dtype=bf))


NO_SCALES = [0.0, 0, -0.0, 1e-60, -1.0, math.nan, math.inf, 1e60]


@pytest.mark.parametrize("scale", NO_SCALES)
def test_a_scale_of_zero_is_not_the_default(latent, scale):
    """The library's 0 selects 1/sqrt(192); a caller's 0 does not mean that, nor what becomes 0 in
    32 bits."""
    with pytest.raises(ValueError, match="scale"):
        latent._attn_shape(*inputs(), None, None, 0, 0, True, scale, -1)
    with pytest.raises(ValueError, match="scale"):
        latent._scale(scale)
    assert latent._scale(None) == 0.0 and latent._scale(0.125) == 0.125


@pytest.mark.gpu
@pytest.mark.parametrize("scale", NO_SCALES)
def test_a_scale_of_zero_is_refused_by_every_call(latent, scale):
    from tests.test_latent_gpu import decode_case
    x = [t.to(DEV) for t in inputs()]
    dec = decode_case(latent, [40, 9], 4, 1, 16, False, seed=2)
    out, lse = latent.latent_attn_fwd(*x)
    for call in (lambda: latent.latent_attn_fwd(*x, scale=scale),
                 lambda: latent.latent_attn_bwd(*x, out, lse, out, scale=scale),
                 lambda: latent.latent_attention(*x, scale=scale),
                 lambda: latent.latent_decode(*dec, scale=scale)):
        with pytest.raises(ValueError, match="scale"):
            call()


def test_a_stream_of_another_device_is_refused(latent):
    """Making it current makes its device current; the call then went to the tensors' device's
    current stream instead, unordered with what the caller had put on the given one."""
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    assert latent._elsewhere(1, stream)
    with pytest.raises(ValueError, match="stream"):
        latent._elsewhere(0, stream)


def last_tokens(B=3, T=5, H=2):
    """The last token of each sequence of a batch, its queries cut from longer ones."""
    q, kn, pe, v = (t.unsqueeze(0).repeat(B, *[1] * t.dim()) for t in inputs(H, T))
    return q[:, -1:], kn, pe, v


def test_one_token_of_each_sequence_of_a_batch(latent):
    """Of a dimension of one the stride says nothing, so the sequences' own stride is the tokens'."""
    q, kn, pe, v = last_tokens()
    s = latent._attn_shape(q, kn, pe, v, None, None, 0, 0, True, None, -1)
    assert (s.B, s.Tq, s.Tk, s.q_token, s.q_head, s.k_token) == (3, 1, 5, 5 * 2 * 192, 192, 2 * 128)
    s = latent._attn_shape(q, kn[:, :1], pe[:, :1], v[:, :1], None, None, 0, 0, True, None, -1)
    assert (s.k_token, s.pe_token, s.v_token) == (5 * 2 * 128, 5 * 64, 5 * 2 * 128)
    s = latent._attn_shape(q[:1], kn[:1], pe[:1], v[:1], None, None, 0, 0, True, None, -1)
    assert s.B == 1 and s.q_token >= 192 and s.q_token % 8 == 0


@pytest.mark.gpu
def test_one_token_of_each_sequence_of_a_batch_on_the_gpu(latent):
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = [torch.randn(t.shape, generator=gen, device=DEV).to(torch.bfloat16) for t in
         last_tokens(4, 150)]
    q = torch.randn(4, 9, 2, 192, generator=gen, device=DEV).to(torch.bfloat16)[:, -1:]
    got, near = latent.latent_attn_fwd(q, *x[1:]), latent.latent_attn_fwd(q.contiguous(), *x[1:])
    assert all(torch.equal(a, b) for a, b in zip(got, near))
    g = torch.ones_like(got[0])
    a = latent.latent_attn_bwd(q, *x[1:], *got, g)
    b = latent.latent_attn_bwd(q.contiguous(), *x[1:], *got, g)
    assert all(torch.equal(y, z) for y, z in zip(a, b))
