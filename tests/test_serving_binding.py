"""The Python side of the serving calls, as far as it needs no GPU."""

import importlib.util
import os
import shutil
import subprocess
import sys
import types

import pytest
import torch

import block_sparse_attention_48_b200 as fa


@pytest.mark.parametrize("name", ["rope_apply", "paged_append", "flex_decode_paged", "flex_decode_shared"])
def test_stream_of_another_device(name):
    """stream= looks at the first tensor, whether it is given by place or by name."""
    fn, first = getattr(fa, name), "k" if name == "paged_append" else "q"
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(x, stream=stream)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(**{first: x}, stream=stream)
    for bad in ({}, {first: None}, {first: [1.0]}):
        with pytest.raises(TypeError, match=first):
            fn(**bad, stream=stream)


# ------------------------------------------------------------------ the torch that it was built against

PKG = os.path.dirname(os.path.abspath(fa.__file__))


def test_another_torch_builds_the_binding_again(tmp_path, monkeypatch):
    """A built binding is reused for the torch it was built against only."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    for name in ("BINDING", "BUILD_DIR"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name: types.SimpleNamespace(submodule_search_locations=[str(torch_dir)]))
    compiled = []

    def compile_(cmd):
        compiled.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build.subprocess, "check_call", compile_)
    for version, builds in (("2.11.0+cu128", 1), ("2.11.0+cu128", 1), ("2.12.0", 2), ("2.12.0", 2), ("2.11.0+cu128", 3)):
        (torch_dir / "version.py").write_text(f"from typing import Optional\n__version__{': str' if builds > 1 else ''} = '{version}'\n")
        build.build_binding()
        assert len(compiled) == builds, version
    os.utime(build.BINDING, (0, 0))  # older than its source
    build.build_binding()
    assert len(compiled) == 4


def test_a_binding_for_another_torch_is_named_at_import(tmp_path):
    """The import says what to do when the binding is one for another torch, or no library
    that loads at all."""
    pkg = tmp_path / "block_sparse_attention_48_b200"
    pkg.mkdir()
    for name in ("__init__.py", "_binding.so"):
        shutil.copy(os.path.join(PKG, name), pkg / name)
    os.symlink(os.path.join(PKG, "libflexattn.so"), pkg / "libflexattn.so")

    def importing(first=""):
        code = f"import sys; sys.path.insert(0, {str(tmp_path)!r}); import torch; {first}import block_sparse_attention_48_b200"
        return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=tmp_path)
    assert importing().returncode == 0
    other = importing("torch.__version__ = '9.9.0'; ")
    assert "ImportError" in other.stderr and "this is 9.9.0" in other.stderr and "build.py" in other.stderr
    (pkg / "_binding.so").write_bytes(b"no library")
    broken = importing()
    assert "ImportError" in broken.stderr and "does not load" in broken.stderr and "build.py" in broken.stderr
