"""The integer 4-bit operators, the router and the experts with tensors on a GPU that is not the current
one, their refusals of tensors that do not fit, and the grids of their largest calls.  Host-only: a
stand-in for the HIP runtime writes the launches down (two_gpus.c)."""
import json
import os
import subprocess
import sys

import pytest

from test_current_device import HERE, runtime  # noqa: F401


def child(runtime, group):  # noqa: F811
    r = subprocess.run([sys.executable, os.path.join(HERE, "two_gpus_int4.py"), runtime, group], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_launches_go_to_the_tensors_device(runtime):  # noqa: F811
    for name, g in child(runtime, "devices").items():
        assert g["devices"] and set(g["devices"]) == {1}, (name, g)
        assert g["current"] == 0, (name, g)


def test_refusals(runtime):  # noqa: F811
    for name, (error, launches) in child(runtime, "refusals").items():
        assert error in ("ValueError", "TypeError", "Sp24Error"), (name, error)
        assert launches == 0, name


def test_grids(runtime):  # noqa: F811
    """A call launches what HIP counts in 32 bits, or returns an error."""
    for name, (status, least, most) in child(runtime, "grids").items():
        assert status in (0, -6), (name, status)
        assert most < 1 << 32, (name, most)
        if status == 0:
            assert least > 0, name
        if not name.startswith(("gemm 2097152 2097152",)):
            assert status == 0, (name, status)
