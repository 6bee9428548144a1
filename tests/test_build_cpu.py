"""The build and the import without the parts that only the cache's Python calls need."""
import os
import subprocess
import sys
import sysconfig
import types

import pytest

from context_parallelism_02_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of one small file and a binding of the caller's text."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    for name, at in (("CSRC", csrc), ("BUILD", tmp_path / "out"), ("LIB", tmp_path / "out" / "libcp.so"),
                     ("BINDING", tmp_path / "out" / "binding.so")):
        monkeypatch.setattr(build, name, str(at))
    return types.SimpleNamespace(binding=csrc / build.BINDING_SRC, lib=tmp_path / "out" / "libcp.so",
                                 so=tmp_path / "out" / "binding.so")


def test_library_is_linked_where_the_binding_does_not_compile(tree):
    tree.binding.write_text("#error not this one\n")
    with pytest.raises(RuntimeError, match=build.BINDING_SRC):
        build.build()
    assert tree.lib.exists() and not tree.so.exists()
    with pytest.raises(RuntimeError, match=build.BINDING_SRC):   # and again, with the library up to date
        build.build()


def test_library_without_python_headers(tree, tmp_path, monkeypatch):
    tree.binding.write_text("#error not compiled\n")
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == str(tree.lib)
    assert tree.lib.exists() and not tree.so.exists()


def test_library_without_torch(tree, monkeypatch):
    tree.binding.write_text("#error not compiled\n")
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="kv4 calls"):
        assert build.build() == str(tree.lib)
    assert tree.lib.exists() and not tree.so.exists()


def test_binding_is_compiled_beside_the_library(tree):
    tree.binding.write_text('#include <Python.h>\n#include <torch/csrc/Exceptions.h>\nextern "C" int two() { return 2; }\n')
    assert build.build() == str(tree.lib)
    assert tree.lib.exists() and tree.so.exists()


def test_binding_file_belongs_to_this_python():
    assert build.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_missing_binding_is_named(cplib, monkeypatch):
    monkeypatch.setattr(_lib, "_kv4_module", None)
    monkeypatch.setattr(_lib, "_kv4_tables", {})
    monkeypatch.setattr(build, "BINDING", build.BINDING + ".none")
    with pytest.raises(RuntimeError, match="needs the headers"):
        _lib.kv4()


def test_import_with_a_torch_without_cuda(cplib):
    """The host calls (shard maps, schedules) need no CUDA build of torch, and the cache's refuse host tensors there."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from context_parallelism_02_gb300 import api
assert api.cp_shard_map(16, 4, 1).shape == (4, 4)
assert api.cp_schedule_pairs(256, 2, 0, True)[0].sum() == 256 * 257 // 2
x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
i = torch.zeros(1, 1, dtype=torch.int32)
try:
    api.kv4_attn(x, torch.zeros(1, 1, 16, 80, dtype=torch.uint8), i, i[0])
except ValueError:
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
