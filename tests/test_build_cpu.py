"""Building and loading the native module beside the library: it fits one version of torch and of Python, the library is
built whether or not it can be, and without it every call goes through ctypes.  No compiler runs here."""

import os
import subprocess
import sys

import pytest

from kronecker_hessian_gptq_gb300 import _lib, _projection, build
from test_layers_calls_cpu import bf16, entries as _entries_of_layers, f32  # noqa: F401
from test_projection_calls_cpu import codes, entries  # noqa: F401


@pytest.fixture
def folder(monkeypatch, tmp_path):
    """Build into a folder of its own, with compilers that write empty files; returns the commands that were run."""
    made, fails = [], set()

    class Process:
        def __init__(self, cmd, **kw):
            made.append(cmd)
            self.out = cmd[cmd.index("-o") + 1]
            self.returncode = int(any(f in " ".join(cmd) for f in fails))

        def communicate(self):
            if not self.returncode:
                open(self.out, "w").close()
            return "", None

    def run(cmd, check):
        Process(cmd).communicate()

    for name, file in (("LIB", "libbakron.so"), ("MARSHAL", "_marshal.so"), ("MARSHAL_TAG", "_marshal.tag"), ("BUILD", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    monkeypatch.setattr(build.subprocess, "Popen", Process)
    monkeypatch.setattr(build.subprocess, "run", run)
    return tmp_path, made, fails


def _modules(made):
    return [c for c in made if any(a.endswith("marshal.cpp") for a in c)]


def test_a_module_for_this_torch_and_python(folder):
    import torch

    at, made, _ = folder
    build.build()
    assert (at / "libbakron.so").exists() and (at / "_marshal.so").exists() and len(_modules(made)) == 1
    assert build.up_to_date() and build.marshal_fits(build.marshal_tag(torch.__version__))
    del made[:]
    build.build()
    assert made == []


def test_another_torch_or_python_makes_it_stale(folder, monkeypatch):
    at, made, _ = folder
    build.build()
    for stale in (build.marshal_tag("0.0.1"), "", None):
        (at / "_marshal.tag").unlink() if stale is None else (at / "_marshal.tag").write_text(stale)
        assert not build.up_to_date()
        del made[:]
        build.build()
        assert len(made) == 1 == len(_modules(made)) and build.up_to_date()  # the module alone
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-999")
    assert not build.up_to_date()


def test_the_library_is_built_without_torch(folder, monkeypatch):
    at, made, _ = folder
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == str(at / "libbakron.so") and (at / "libbakron.so").exists()
    assert not _modules(made) and not (at / "_marshal.so").exists() and build.up_to_date()


def test_the_library_is_linked_where_the_module_does_not_compile(folder):
    at, _, fails = folder
    fails.add("marshal.cpp")
    with pytest.raises(RuntimeError, match="_marshal.so"):
        build.build()
    assert (at / "libbakron.so").exists() and not (at / "_marshal.tag").exists()
    fails.clear()
    fails.add("adamw.cu")
    (at / "libbakron.so").unlink()
    with pytest.raises(RuntimeError, match="adamw.cu"):
        build.build()
    assert not (at / "libbakron.so").exists()


@pytest.mark.parametrize("stale", ["torch 0.0.1, Python cpython-39", None])
def test_a_module_of_another_version_is_not_loaded(monkeypatch, tmp_path, stale):
    monkeypatch.setattr(_lib, "_marshal", None)
    monkeypatch.setattr(build, "MARSHAL_TAG", str(tmp_path / "tag"))
    if stale is not None:
        (tmp_path / "tag").write_text(stale)
    assert _lib.load_marshal() is None


def test_calls_go_through_ctypes_without_the_module(entries, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_projection, "_native", None)
    monkeypatch.setattr(_lib, "load_marshal", lambda: None)
    made = []
    monkeypatch.setattr(_projection, "_call", lambda name, *args: made.append(name))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        _projection.fp8_matmul(bf16(40, 256), codes(130, 256), f32(2, 2))
    _projection.fp8_matmul_backward(bf16(40, 130), bf16(40, 256), codes(130, 256), f32(2, 2))  # warned once
    _projection.head_norm_rotary(bf16(6, 4, 64), None, None, None)
    _projection.head_norm_rotary_backward(bf16(6, 4, 64), None, bf16(6, 4, 64), None, None, None)
    _projection.adamw([f32(9)], [bf16(9)], {k: [f32(9)] for k in "mv"}, 1)
    assert made == ["bakron_fp8_matmul", "bakron_fp8_matmul_backward", "bakron_head_norm_rotary", "bakron_head_norm_rotary_backward",
                    "bakron_adamw"]


def test_the_build_imports_no_torch():
    code = "import sys; sys.path.insert(0, sys.argv[1]); from kronecker_hessian_gptq_gb300 import build as b; b.up_to_date(); " \
           "assert 'torch' not in sys.modules"
    subprocess.run([sys.executable, "-c", code, os.path.dirname(build.PKG)], check=True)
