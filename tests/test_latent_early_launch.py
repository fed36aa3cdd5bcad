"""Kernels that start while the kernel ahead of them on the stream still runs: what they may not do
before griddepcontrol.wait returns, read from their source (both faults would be races that a GPU
shows rarely or as a hang), and the calls back to back on the GPU."""
from __future__ import annotations

import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "kimi_delta_attention_19_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def kernels(text):
    """(name, body) of every __global__ function, whose bodies end with a } in the first column."""
    return re.findall(r"__global__\s+void\s.*?(\w+_kernel)\((.*?)\n}\n", text, flags=re.S)


EARLY = {"kda_latent_fwd.cu": ["fwd_kernel"], "kda_latent_decode.cu": ["decode_kernel", "join_kernel"],
         "kda_latent_cache.cu": ["cache_write_kernel", "cache_read_kernel"]}


@pytest.mark.parametrize("name", EARLY)
def test_tensor_memory_is_not_held_while_waiting_for_the_kernel_ahead(name):
    """Columns taken before the wait would be held while this kernel waits for one whose CTAs may
    wait for columns."""
    found = dict(kernels(source(name)))
    assert sorted(found) == sorted(EARLY[name])
    for body in found.values():
        wait = body.rindex("griddep_wait()")        # (of all threads)
        alloc = body.find("tmem_alloc(")
        assert alloc < 0 or alloc > wait


@pytest.mark.parametrize("name", EARLY)
def test_early_kernels_read_by_ordinary_loads(name):
    """The read-only path (ld.global.nc) is for memory nobody writes while the kernel runs; the
    kernel ahead may still be writing when an early one starts."""
    text = source(name)
    assert "__ldg(" not in text and "global.nc" not in text
    assert "__restrict__" not in text            # with const it lets the compiler choose that path


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
def test_tokens_written_and_attended_to_back_to_back(quantized):
    """Sequences grow a token a step, each step a write and a decode with nothing in between: the
    same bits as with a synchronisation after every call. A row's 656 bytes share sectors and lines
    with rows that steps before have read, and the block table's next entry is set by a step too."""
    from kimi_delta_attention_19_b200 import latent
    dev, n, ps, H, steps = "cuda:0", 6, 16, 32, 70
    gen = torch.Generator(device=dev).manual_seed(1)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)

    c, pe, q = rnd(steps, n, 512), rnd(steps, n, 64), rnd(steps, n, H, 576)
    pages = torch.randperm(n * 5, generator=torch.Generator().manual_seed(2)).view(n, 5)
    full = pages.to(torch.int32).to(dev)
    slots = [(pages[:, t // ps] * ps + t % ps).to(dev) for t in range(steps)]

    def run(sync):
        cache = latent.latent_cache(n * 5, ps, quantized=quantized, device=dev)
        table = torch.full_like(full, -1)
        lens = torch.zeros(n, dtype=torch.int32, device=dev)
        outs = []
        for t in range(steps):
            if t % ps == 0:
                table[:, t // ps] = full[:, t // ps]
            lens.add_(1)
            latent.latent_cache_write(c[t], pe[t], cache, slots[t])
            if sync:
                torch.cuda.synchronize()
            outs.append(latent.latent_decode(q[t], cache, table, lens))
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, run(False)))
    assert all(torch.isfinite(o.float()).all() for o in want)
