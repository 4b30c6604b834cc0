"""The integer 4-bit operators, the router and the experts without the C++ module: the call says what is missing,
and what needs no module (workspace sizes, the codes' order) works."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytest.importorskip("bf16_gemm_linear_amd", reason="libsp24.so not built")

NATIVE = ("quant_int4", "dequant_int4", "gemm_int4", "route", "experts_int4")


def test_import_without_the_module():
    code = """
import sys
sys.modules['bf16_gemm_linear_amd._sp24'] = None
import torch
import bf16_gemm_linear_amd as sp
assert sp.experts_int4_workspace_size(1, 128, 128, 4, 2) > 0 and sp.gemm_int4_workspace_size(1, 128, 128) == 0
q = torch.arange(16, dtype=torch.uint8).reshape(1, 16)
assert torch.equal(sp.unpack_int4(sp.pack_int4(q)), q)
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
