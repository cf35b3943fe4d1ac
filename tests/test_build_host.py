"""What build.build compiles, from recorded commands: the C library needs nvcc alone; the CPython module is built
against the torch that is there, and again when that changes."""

import os
import sys

import pytest
import torch

from top_sparse_attention_attn_b200 import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Runs build.build() into an empty folder, its commands recorded and their outputs made as empty files."""
    ran = []

    def run(cmd):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsparse_attn.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_kv8_ext.so"))

    def call():
        del ran[:]
        build.build()
        return [os.path.basename(c[c.index("-o") + 1]) for c in ran]
    return call


def test_the_library_is_linked_before_the_module_that_loads_it(commands):
    made = commands()
    assert made.index("libsparse_attn.so") < made.index("_kv8_ext.so") and "kv8_ext.o" in made
    assert commands() == []


@pytest.mark.parametrize("what", ["no_torch", "cpu_torch"])
def test_the_library_builds_without_a_torch_that_has_cuda(commands, monkeypatch, what):
    with monkeypatch.context() as m:
        if what == "no_torch":
            m.setitem(sys.modules, "torch", None)          # import torch raises ImportError
        else:
            m.setattr(torch.version, "cuda", None)
        made = commands()
        assert "libsparse_attn.so" in made and not any("kv8_ext" in x for x in made)
        assert commands() == []
    assert commands() == ["kv8_ext.o", "_kv8_ext.so"]


def test_the_module_is_built_again_for_another_torch(commands, monkeypatch):
    commands()
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert commands() == ["kv8_ext.o", "_kv8_ext.so"]
    assert commands() == []
