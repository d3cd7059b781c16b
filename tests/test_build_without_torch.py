"""The C library needs nvcc and g++ alone: it builds, and the package imports, where torch is absent or has no CUDA."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BUILD = """
import importlib.util, os, sys
hide, out = sys.argv[1], sys.argv[2]
if hide == "absent":
    sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("_tq_build", os.path.join("turboquant_quantized_kv_tq_gb300", "_build.py"))
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
m.OBJ_DIR = m.LIB_DIR = out
m.LIB_PATH, m.EXT_PATH = os.path.join(out, "libtq.so"), os.path.join(out, "_tq_torch.so")
one = [s for s in m.sources() if s.endswith("tq_host_tables.cpp")]
assert len(one) == 1
m.sources = lambda: one          # (one host file stands for all: this is about what else build() asks for)
open(m.EXT_PATH, "w").write("of an earlier build")
if hide == "cpu":
    import types
    fake = types.ModuleType("torch")
    fake.__file__ = os.path.join(out, "torch", "__init__.py")
    sys.modules["torch"] = fake
m.build()
assert os.path.exists(m.LIB_PATH)
assert not os.path.exists(m.EXT_PATH), "an extension that this build did not make"
"""


@pytest.mark.parametrize("torch", ["absent", "cpu"])
def test_library_builds_without_torch(tmp_path, torch):
    res = subprocess.run([sys.executable, "-c", BUILD, torch, str(tmp_path)], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


UNBUILT = """
import importlib.util, sys
spec = importlib.util.spec_from_file_location("turboquant_quantized_kv_tq_gb300._build", "turboquant_quantized_kv_tq_gb300/_build.py")
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
m.EXT_PATH = "not/built"
sys.modules[spec.name] = m
"""


@pytest.mark.parametrize("first,names", [("import sys; sys.modules['torch'] = None\n", False), (UNBUILT, False), ("", True)],
                         ids=["no torch", "not built", "all"])
def test_star_import(first, names):
    """`import *` takes what is there: everything where the torch extension is built, the rest as ever without it."""
    if names:
        pytest.importorskip("torch")
    code = first + ("from turboquant_quantized_kv_tq_gb300 import *\n"
                    "assert QuantizedKVCache and PagedKVCache and TQError and binding\n"
                    f"assert all((n in globals()) == {names} for n in ('PagedByteCache', 'Rotary', 'norm_rotate'))\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_names_are_there_by_name():
    pytest.importorskip("torch")
    import turboquant_quantized_kv_tq_gb300 as tq
    assert {"PagedByteCache", "Rotary", "norm_rotate"} <= set(tq.__all__) and tq.PagedByteCache and tq.Rotary and tq.norm_rotate
    with pytest.raises(AttributeError):
        tq.no_such_name
