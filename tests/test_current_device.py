"""Tensors on a GPU that is not the current one: every launch goes to the tensors' device, and the
current device is the same afterwards.  Host-only: a stand-in for the HIP runtime writes the launches
down (two_gpus.c)."""
import json
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
HIP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")


@pytest.fixture(scope="module")
def runtime(tmp_path_factory):
    pytest.importorskip("bf16_gemm_linear_amd", reason="libsp24.so not built")
    import torch
    gcc = shutil.which("gcc")
    if gcc is None or torch.version.hip is None or not os.path.isdir(HIP) or os.path.exists("/dev/kfd"):
        pytest.skip("needs gcc, HIP's headers and a host without GPUs")
    out = str(tmp_path_factory.mktemp("runtime") / "two_gpus.so")
    subprocess.run([gcc, "-O1", "-shared", "-fPIC", "-w", "-I" + HIP, "-o", out, os.path.join(HERE, "two_gpus.c")],
                   check=True)
    return out


@pytest.mark.parametrize("group", ["mxfp4", "sparse"])
def test_launches_go_to_the_tensors_device(runtime, group):
    r = subprocess.run([sys.executable, os.path.join(HERE, "two_gpus.py"), runtime, group], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    got = json.loads(r.stdout.strip().splitlines()[-1])
    for name, g in got.items():
        assert g["devices"] and set(g["devices"]) == {1}, (name, g)
        assert g["current"] == 0, (name, g)
