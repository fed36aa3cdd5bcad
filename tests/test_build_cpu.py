"""The build on the CPU: the library does not depend on the latent binding's extension module."""
from __future__ import annotations

import os

import pytest

from kimi_delta_attention_19_b200 import build as kbuild


@pytest.fixture
def dry(monkeypatch, tmp_path):
    """build() into tmp_path with compilers that only note what they are asked; its notes."""
    notes = {"linked": [], "host": 0}

    def compile_(src, obj, extra=None):
        with open(obj, "w"):
            return ""

    monkeypatch.setattr(kbuild, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(kbuild, "HOST_MODULE", str(tmp_path / "_latent_host.so"))
    monkeypatch.setattr(kbuild, "_compile", compile_)
    monkeypatch.setattr(kbuild, "_link", lambda lib, objs: notes["linked"].append(lib))
    return notes


def failing(src):
    raise RuntimeError("Python.h: No such file or directory")


def test_library_is_linked_though_the_extension_module_cannot_be_built(dry, monkeypatch):
    monkeypatch.setattr(kbuild, "_build_host", failing)
    with pytest.warns(UserWarning, match="Python.h"):
        assert kbuild.build() == kbuild.LIB
    assert dry["linked"][0] == kbuild.LIB


def test_a_stale_extension_module_is_not_left_behind(dry, monkeypatch):
    """One built against an older kda.h would pass structs the library reads differently."""
    with open(kbuild.HOST_MODULE, "w"):
        pass
    os.utime(kbuild.HOST_MODULE, (1, 1))
    monkeypatch.setattr(kbuild, "_build_host", failing)
    with pytest.warns(UserWarning):
        kbuild.build()
    assert not os.path.exists(kbuild.HOST_MODULE)


def test_a_failing_cuda_source_still_fails_the_build(dry, monkeypatch):
    def broken(src, obj, extra=None):
        raise RuntimeError("nvcc failed")

    monkeypatch.setattr(kbuild, "_compile", broken)
    monkeypatch.setattr(kbuild, "_build_host", lambda src: "")
    with pytest.raises(RuntimeError, match="nvcc"):
        kbuild.build()
    assert not dry["linked"]
