"""Building and importing without _fastcall.so, the host accelerator of the
Python binding: the C library and every call do without it. Needs no GPU."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "bit_nf4_quantized_03_amd", "build.py")
built = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "bit_nf4_quantized_03_amd", "libqlora_nf4.so")),
                           reason="the library is not built")


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


@built
def test_import_without_fastcall():
    r = _python("""
import sys
class Missing:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._fastcall"):
            raise ImportError(name)
sys.meta_path.insert(0, Missing())
import torch
import bit_nf4_quantized_03_amd as qb
from bit_nf4_quantized_03_amd import autograd
assert len(qb.qlora_nf4_codebook()) == 16 and qb.qlora_mx_scale_pitch(544) == 32
for call in (lambda: qb.qlora_mx_quantize(torch.zeros(4, 64)), lambda: qb.qlora_mx_dequantize(qb.MXMatrix.empty(4, 64, "cpu")),
             lambda: qb.qlora_rmsnorm_fwd(torch.zeros(4, 64).bfloat16(), torch.ones(64))):
    try:
        call()
    except TypeError as e:
        assert "CUDA (HIP) tensor" in str(e)
    else:
        raise AssertionError("not refused")
print("fine")
""")
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@built
def test_import_with_a_torch_for_the_cpu():
    """Sizes, levels and refusals need no GPU support in torch."""
    r = _python("""
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import bit_nf4_quantized_03_amd as qb
assert qb.qlora_nf4_storage_bytes(64, 64) > 0 and qb.qlora_mx_storage_bytes(3, 64, qb.QLORA_MX_FP8) == 240
try:
    qb.qlora_mx_quantize(torch.zeros(4, 64))
except TypeError as e:
    print("fine", e)
""")
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@built
def test_package_loaded_again():
    """After a reload, which a build does, the microscaled calls are declared and raise the package's error."""
    r = _python("""
import ctypes, importlib
import bit_nf4_quantized_03_amd as qb
qb = importlib.reload(qb)
assert qb.mx.lib is qb.lib and qb.mx.QloraError is qb.QloraError
assert qb.lib.qlora_mx_storage_bytes.restype is ctypes.c_size_t
qb.mx._stream, qb.mx._current = lambda index: None, lambda: 0   # no device here
try:
    qb.mx._entry("qlora_mx_dequantize")(qb.mx._current(), None, None, 0)
except qb.QloraError as e:
    print("fine", e)
""")
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def _build_in(tmp_path):
    spec = importlib.util.spec_from_file_location("_build_in", BUILD)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.BUILD_DIR, mod.PKG_DIR = str(tmp_path / "obj"), str(tmp_path)
    mod.LIB_PATH, mod.FASTCALL_PATH = str(tmp_path / mod.LIB_NAME), str(tmp_path / "_fastcall.so")
    mod.SOURCES = ["codebook.cpp"]
    try:
        mod._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    return mod


@pytest.mark.parametrize("where", ["compile", "link"])
def test_library_is_built_without_fastcall(tmp_path, monkeypatch, capsys, where):
    mod = _build_in(tmp_path)

    def fails(*_):
        raise RuntimeError("no headers here")
    monkeypatch.setattr(mod, f"_{where}_fastcall", fails)
    if where == "link":
        monkeypatch.setattr(mod, "_compile_fastcall", lambda: "unused.o")
    (tmp_path / "_fastcall.so").write_bytes(b"of an older library")
    assert mod.build() == mod.LIB_PATH and os.path.exists(mod.LIB_PATH)
    assert not os.path.exists(mod.FASTCALL_PATH)
    assert "no headers here" in capsys.readouterr().err


def test_library_that_does_not_compile_is_an_error(tmp_path, monkeypatch):
    mod = _build_in(tmp_path)
    mod.SOURCES = ["not_there.cpp"]
    monkeypatch.setattr(mod, "_compile_fastcall", lambda: "unused.o")
    with pytest.raises(RuntimeError, match="compile failed"):
        mod.build()


@built
@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_fastcall_is_built_where_it_can_be():
    assert os.path.exists(os.path.join(ROOT, "bit_nf4_quantized_03_amd", "_fastcall.so"))
    r = _python("import bit_nf4_quantized_03_amd.mx as m; assert m._fast is not None")
    assert r.returncode == 0, r.stderr
