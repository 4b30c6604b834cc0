"""Errors that PyTorch raises inside a call of the C++ module keep their types: a caller that frees
memory on torch.OutOfMemoryError and tries again does so for these operators too.  And grids that the
runtime would refuse are not asked for, nor is a configuration taken for another that SP24_MX4 names with
a "!".  Host-only, on the runtime of test_current_device."""
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


def test_grids_are_launchable(runtime):  # noqa: F811
    """HIP launches fewer than 2^32 threads along a dimension.  No outputs that fit 288 GB need more
    (bf16: 2^37, MXFP4 of the gated product: 2^39); past that a call returns an error."""
    r = subprocess.run([sys.executable, os.path.join(HERE, "two_gpus.py"), runtime, "grids"], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    got = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(got) == 8
    for outputs, status, threads in got:
        if outputs <= 1 << 38:
            assert status == 0 and len(threads) == 1 and threads[0] < 1 << 32, (outputs, status, threads)
        else:
            assert status != 0 and not threads, (outputs, status, threads)


def test_named_configuration_or_an_error(runtime):  # noqa: F811
    r = subprocess.run([sys.executable, os.path.join(HERE, "two_gpus.py"), runtime, "configurations"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    yes, no = [0, 1], [-6, 0]  # one launch; an error and none
    assert json.loads(r.stdout.strip().splitlines()[-1]) == {
        "stream,8 17": [yes, yes, yes],  # without the "!" the planner's
        "stream,8! 16": [yes, yes, yes], "stream,8! 17": [no, no, no], "stream,1! 8": [yes, no, no],
        "stream,2! 64": [yes, yes, no], "stream,2! 65": [no, no, no], "wave,4! 8": [yes, yes, yes],
        "wave,5! 8": [yes, no, no], "tiled,3! 8": [yes, yes, yes], "tiled,4! 8": [yes, no, no],
        "wave,9! 8": [no, no, no], "walk,1! 8": [no, no, no], "! 8": [no, no, no]}
