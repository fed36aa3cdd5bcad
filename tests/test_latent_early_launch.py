"""Kernels that start while the kernel ahead of them on the stream still runs: what they may not do
before griddepcontrol.wait returns, read from their source (both faults would be races that a GPU
shows rarely or as a hang), and the calls back to back on the GPU."""
from __future__ import annotations

import os
import re

import pytest

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
