"""The package without its C++ module, or with one built for another PyTorch: the operators of
libsp24.so over ctypes are all there, and the others say what is missing when they are called."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytest.importorskip("bf16_gemm_linear_amd", reason="libsp24.so not built")

NATIVE = ("quant_mxfp4", "dequant_mxfp4", "gemm_mxfp4", "gated_mxfp4", "rmsnorm", "ffn_mxfp4")
BEFORE = {
    "no module": "import sys; sys.modules['bf16_gemm_linear_amd._sp24'] = None",
    "another PyTorch": "import torch; torch.__version__ = '1.13.1+rocm5.2'",
    "PyTorch without GPU support": "import sys, torch; sys.modules['bf16_gemm_linear_amd._sp24'] = None\n"
                                   "del torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice",
}


@pytest.mark.parametrize("case", BEFORE)
def test_import_without_the_module(case):
    code = BEFORE[case] + """
import bf16_gemm_linear_amd as sp
assert sp.version() > 0 and sp.plan(sp.OP_GEMM, sp.FP8, 16, 4096, 4096)["tile_n"] > 0
assert sp.ffn_mxfp4_workspace_size(1, 128, 128) > 0
for name in %r:
    try:
        getattr(sp, name)()
    except ImportError as e:
        assert name in str(e) and "_sp24" in str(e), e
    else:
        raise AssertionError(name)
print("ok")
""" % (NATIVE,)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_module_is_of_this_pytorch():
    import torch

    from bf16_gemm_linear_amd import _sp24
    assert str(torch.__version__).startswith(_sp24.torch_version)
