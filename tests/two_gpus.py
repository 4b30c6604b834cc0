"""Child process of test_current_device: the package on the two GPUs of two_gpus.c, which run nothing.

    python tests/two_gpus.py LIBRARY GROUP

Calls every function of the group with tensors on cuda:1 while cuda:0 is current, and prints one JSON
object: for each function the devices that its launches went to and the device current afterwards."""
import ctypes
import json
import os
import sys

runtime = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # before PyTorch: see two_gpus.c
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bf16_gemm_linear_amd as sp  # noqa: E402


class Launch(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("stream", ctypes.c_void_p), ("grid", ctypes.c_uint * 3),
                ("block", ctypes.c_uint * 3)]


runtime.fake_launches.restype = ctypes.POINTER(Launch)
M, N, K = 4, 512, 512


def new(shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda:1")


def mxfp4():
    x, w = new((M, K)), new(K)
    xq = new((M, K // 2), torch.uint8), new(M * K // 32, torch.uint8)
    wq = new((2 * N, K // 2), torch.uint8), new(2 * N * K // 32, torch.uint8)
    dn = new((K, N // 2), torch.uint8), new(K * N // 32, torch.uint8)
    return {
        "quant_mxfp4": lambda: sp.quant_mxfp4(x),
        "dequant_mxfp4": lambda: sp.dequant_mxfp4(*xq),
        "gemm_mxfp4": lambda: sp.gemm_mxfp4(*xq, *wq),
        "gated_mxfp4": lambda: sp.gated_mxfp4(*xq, *wq),
        "gated_mxfp4 quantise": lambda: sp.gated_mxfp4(*xq, *wq, quantise=True),
        "rmsnorm": lambda: sp.rmsnorm(x, w, sp.NORM_FP8_ROWS),
        "ffn_mxfp4": lambda: sp.ffn_mxfp4(x, w, *wq, *dn),
    }


def main():
    torch.cuda.set_device(0)
    got = {}
    for name, call in globals()[sys.argv[2]]().items():
        runtime.fake_clear()
        call()
        n = runtime.fake_count()
        got[name] = {"devices": [runtime.fake_launches()[i].device for i in range(n)],
                     "current": torch.cuda.current_device()}
    print(json.dumps(got))


if __name__ == "__main__":
    main()
