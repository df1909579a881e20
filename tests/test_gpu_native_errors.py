"""An error of the library in a call made natively: it is raised, and the call is not made a second time (an AdamW step
would be two).  A library of stand-ins, which launch nothing, counts its calls and returns the status it is told."""

import ctypes
import shutil
import subprocess

import pytest

from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu

CALLS = ["bakron_fp8_matmul", "bakron_fp8_matmul_backward", "bakron_head_norm_rotary", "bakron_head_norm_rotary_backward", "bakron_adamw"]
SIZES = [name + "_workspace_size" for name in CALLS if name != "bakron_head_norm_rotary"]


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("stand_in")
    # Arguments lie where the caller put them and are not read.
    text = "extern \"C\" {\nint calls = 0, status = 0;\n"
    text += "".join(f"int {n}(...) {{ ++calls; return status; }}\n" for n in CALLS)
    text += "".join(f"unsigned long {n}(...) {{ return 256; }}\n" for n in SIZES)
    text += "const char* bakron_status_string(int) { return \"BAKRON_ERR_CUDA\"; }\n}\n"
    (at / "stand_in.cpp").write_text(text)
    subprocess.run([cxx, "-shared", "-fPIC", str(at / "stand_in.cpp"), "-o", str(at / "stand_in.so")], check=True)
    return str(at / "stand_in.so")


@pytest.fixture
def native(bk, stand_in, monkeypatch):  # noqa: F811
    """The native module over the stand-ins; calls through ctypes are counted, and made by none."""
    from kronecker_hessian_gptq_gb300 import _lib, _projection

    module = _lib.load_marshal()
    lib = ctypes.CDLL(stand_in)
    again = []
    monkeypatch.setattr(_projection, "_call", lambda name, *args: again.append(name))
    assert module.bind(stand_in)
    try:
        yield lib, again
    finally:
        assert module.bind(_lib.LIB_PATH)


def _run(bk, name):  # noqa: F811
    import torch

    x, q = torch.zeros((5, 256), device="cuda"), torch.zeros((5, 2, 64), device="cuda")
    v, s = torch.zeros((128, 256), dtype=torch.uint8, device="cuda"), torch.zeros((1, 2), device="cuda")
    if name == "bakron_fp8_matmul":
        return bk.fp8_matmul(x, v, s)
    if name == "bakron_fp8_matmul_backward":
        return bk.fp8_matmul_backward(x[:, :128].contiguous(), x, v, s)
    if name == "bakron_head_norm_rotary":
        return bk.head_norm_rotary(q, None, None, None)
    if name == "bakron_head_norm_rotary_backward":
        return bk.head_norm_rotary_backward(q, None, q, None, None, None)
    p = [torch.zeros(300, device="cuda")]
    return bk.adamw(p, [torch.zeros(300, device="cuda")], bk.adamw_states(p), 1)


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_call_is_raised_and_not_made_again(bk, native, name):  # noqa: F811
    lib, again = native
    calls, status = (ctypes.c_int.in_dll(lib, n) for n in ("calls", "status"))
    calls.value, status.value = 0, 3  # BAKRON_ERR_CUDA
    with pytest.raises(RuntimeError, match=f"{name} failed: BAKRON_ERR_CUDA"):
        _run(bk, name)
    assert calls.value == 1 and again == []


@pytest.mark.parametrize("code", [1, 4])  # an argument, the workspace: nothing was enqueued
@pytest.mark.parametrize("name", CALLS)
def test_a_refused_call_goes_through_the_checks(bk, native, name, code):  # noqa: F811
    lib, again = native
    calls, status = (ctypes.c_int.in_dll(lib, n) for n in ("calls", "status"))
    calls.value, status.value = 0, code
    _run(bk, name)
    assert calls.value == 1 and again == [name]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_that_succeeds_is_made_once(bk, native, name):  # noqa: F811
    lib, again = native
    calls, status = (ctypes.c_int.in_dll(lib, n) for n in ("calls", "status"))
    calls.value, status.value = 0, 0
    _run(bk, name)
    assert calls.value == 1 and again == []
