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


def sparse():
    x, w, u8, f32, i32 = new((M, K)), new((N, K)), torch.uint8, torch.float32, torch.int32
    v, meta, one = new((N, K // 2)), new(N * K // 32, i32), new(1, f32)
    q, qv, qw = new((M, K), u8), new((N, K // 2), u8), new((N, K), u8)
    xs, kp = new(M, f32), K // 8 * 12  # k of a 6:8 weight lifted to 2:4 windows
    sv, sm = new((N, kp // 2), u8), new(N * kp // 32, i32)
    pw = sp.PaletteWeight(N, K, new(16, u8), torch.empty(N, dtype=i32, device="cuda:1"), new(N * K, u8),
                          new(N * K // 8, i32), new(0, i32), new(0))
    big = new(1 << 20, u8)
    return {
        "prune_compress": lambda: sp.prune_compress(w),
        "decompress": lambda: sp.decompress(v, meta, K),
        "check_meta": lambda: sp.check_meta(meta, K, new(1, i32)),
        "quant_fp8": lambda: sp.quant_fp8(x),
        "quant_int8": lambda: sp.quant_int8(x),
        "gemm": lambda: sp.gemm(x, v, meta),
        "dense_gemm": lambda: sp.dense_gemm(x, w),
        "quant_fp8_rows": lambda: sp.quant_fp8_rows(x),
        "quant_int8_rows": lambda: sp.quant_int8_rows(x),
        "slide_prune_pack": lambda: sp.slide_prune_pack(w),
        "slide_quant_fp8_rows": lambda: sp.slide_quant_fp8_rows(x),
        "slide_quant_int8_rows": lambda: sp.slide_quant_int8_rows(x),
        "gemm_rows": lambda: sp.gemm_rows(q, qv, meta, xs, one),
        "gemm_qx": lambda: sp.gemm_qx(x, qv, meta, one),
        "gemm_qx_noalloc": lambda: sp.gemm_qx_noalloc(x, qv, meta, one, new(1, f32), new((M, N))),
        "quant_fp8_groups": lambda: sp.quant_fp8_groups(x, 128),
        "gemm_groups": lambda: sp.gemm_groups(q, new((M, K // 128), f32), qv, meta, new((N, K // 128), f32), 128),
        "gemm_rows_qx": lambda: sp.gemm_rows_qx(x, qv, meta, one),
        "slide_gemm_qx": lambda: sp.slide_gemm_qx(x, sv, sm, one),
        "palette_decode": lambda: sp.palette_decode(pw),
        "palette_gemm": lambda: sp.palette_gemm(x, pw),
        "probe_mfma_layout": lambda: sp.probe_mfma_layout(0, big, big, big, big, 1),
        "probe_mfma_rate": lambda: sp.probe_mfma_rate(0, 1, 1, 1, new(64, f32)),
        "probe_copy": lambda: sp.probe_copy(big, new(1 << 20, u8)),
        "probe_read": lambda: sp.probe_read(big, new(1 << 20, i32)),
        "probe_ring": lambda: sp.probe_ring(8, 16, 4, True, big, 8 << 10, big, 1, 1, new(1, i32)),
    }


def out_of_memory():
    """Outputs that no memory is left for: the exceptions of the C++ functions and of a ctypes one."""
    q = new((1 << 19, 64), torch.uint8), new(1 << 21, torch.uint8)
    x, v, meta = new((1 << 18, 64)), new((1 << 18, 32)), new(1 << 19, torch.int32)
    got = {}
    for name, call in {"gemm_mxfp4": lambda: sp.gemm_mxfp4(*q, *q),
                       "gated_mxfp4": lambda: sp.gated_mxfp4(*q, *q),
                       "gemm": lambda: sp.gemm(x, v, meta)}.items():
        try:
            call()
        except Exception as e:
            got[name] = [t.__name__ for t in type(e).__mro__]
    print(json.dumps(got))


def grids():
    """The largest products that the documented limits and the card's memory allow, and beyond: their
    status and the threads of the grid in x, from the C calls with addresses that nothing reads."""
    at = [ctypes.c_void_p((i + 1) << 44) for i in range(8)]
    got = []
    for m, f, k in ((1 << 21, 1 << 17, 128), (1 << 18, 1 << 20, 128), (1 << 20, 1 << 18, 4096), (1 << 21, 1 << 20, 128)):
        runtime.fake_clear()
        status = sp.lib.sp24_gated_mxfp4(m, f, k, *at[:4], None, at[4], at[5], None)
        got.append([m * f, status, [l.grid[0] * l.block[0] for l in runtime.fake_launches()[:runtime.fake_count()]]])
    for m, n, k in ((1 << 18, 1 << 19, 128), (1 << 21, 1 << 16, 128), (1 << 16, 1 << 21, 256), (1 << 21, 1 << 21, 128)):
        runtime.fake_clear()
        status = sp.lib.sp24_gemm_mxfp4(m, n, k, *at[:5], None)
        got.append([m * n, status, [l.grid[0] * l.block[0] for l in runtime.fake_launches()[:runtime.fake_count()]]])
    print(json.dumps(got))


def configurations():
    """SP24_MX4 by name: status and number of launches of a product, a gated product and one to MXFP4, of
    the tokens given, from the C calls with addresses that nothing reads."""
    at = [ctypes.c_void_p((i + 1) << 44) for i in range(8)]
    got = {}
    for config, m in (("stream,8", 17), ("stream,8!", 16), ("stream,8!", 17), ("stream,1!", 8), ("stream,2!", 64),
                      ("stream,2!", 65), ("wave,4!", 8), ("wave,5!", 8), ("tiled,3!", 8), ("tiled,4!", 8),
                      ("wave,9!", 8), ("walk,1!", 8), ("!", 8)):
        os.environ["SP24_MX4"] = config
        got["%s %d" % (config, m)] = calls = []
        for call in (lambda: sp.lib.sp24_gemm_mxfp4(m, 512, 256, *at[:5], None),
                     lambda: sp.lib.sp24_gated_mxfp4(m, 256, 256, *at[:5], None, None, None),
                     lambda: sp.lib.sp24_gated_mxfp4(m, 256, 256, *at[:4], None, at[4], at[5], None)):
            runtime.fake_clear()
            status = call()
            calls.append([status, runtime.fake_count()])
    print(json.dumps(got))


def main():
    torch.cuda.set_device(0)
    if sys.argv[2] == "out_of_memory":
        return out_of_memory()
    if sys.argv[2] == "grids":
        return grids()
    if sys.argv[2] == "configurations":
        return configurations()
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
