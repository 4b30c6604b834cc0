"""Errors that PyTorch raises inside a call of the C++ module keep their types: a caller that frees
memory on torch.OutOfMemoryError and tries again does so for these operators too.  Host-only, on the
runtime of test_current_device."""
import json
import os
import subprocess
import sys

from test_current_device import HERE, runtime  # noqa: F401


def test_out_of_memory(runtime):  # noqa: F811
    r = subprocess.run([sys.executable, os.path.join(HERE, "two_gpus.py"), runtime, "out_of_memory"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    got = json.loads(r.stdout.strip().splitlines()[-1])
    assert set(got) == {"gemm_mxfp4", "gated_mxfp4", "gemm"}
    for name, types in got.items():
        assert types[0] == "OutOfMemoryError", (name, types)
