"""Child process of test_current_device_int4: the integer 4-bit operators, the router and the experts on
the two GPUs of two_gpus.c, which run nothing.

    python tests/two_gpus_int4.py LIBRARY GROUP

`devices`: every function with tensors on cuda:1 while cuda:0 is current; prints the devices that its
launches went to and the device current afterwards.  `refusals`: calls that must raise, and what they
raise.  `grids`: the C calls at the limits of their sizes, with addresses that nothing reads."""
import ctypes
import json
import sys

import two_gpus  # loads the runtime
from two_gpus import new, runtime, sp, torch

U8, F32, I32 = torch.uint8, torch.float32, torch.int32


def weight(n, k, group=64, experts=None, zeros=False):
    sh = (n,) if experts is None else (experts, n)
    return (new((*sh, k // 2), U8), new((*sh, k // group)), new((*sh, k // group), U8) if zeros else None)


def calls(tokens):
    E, d, f, top = 6, 256, 128, 2
    w, gu, dn = weight(512, 256, zeros=True), weight(2 * f, d, experts=E), weight(d, f, experts=E)
    x, ids, wt = new((tokens, d)), new((tokens, top), I32), new((tokens, top), F32)
    return {
        "quant_int4": lambda: sp.quant_int4(new((512, 256)), group=32, zeros=True),
        "dequant_int4": lambda: sp.dequant_int4(*w),
        "gemm_int4": lambda: sp.gemm_int4(x, *w),
        "route": lambda: sp.route(new((tokens, 64), F32), 4, bias=new(64, F32)),
        "experts_int4": lambda: sp.experts_int4(x, ids, wt, gu[0], gu[1], dn[0], dn[1]),
    }


def devices():
    got = {}
    for tokens in (1, 40, 3000):
        for name, call in calls(tokens).items():
            runtime.fake_clear()
            call()
            n = runtime.fake_count()
            got["%s %d" % (name, tokens)] = {"devices": [runtime.fake_launches()[i].device for i in range(n)],
                                             "current": torch.cuda.current_device()}
    return got


def refusals():
    E, d, f, top, m = 6, 256, 128, 2, 5
    w, gu, dn = weight(512, 256), weight(2 * f, d, experts=E), weight(d, f, experts=E)
    x, ids, wt = new((m, d)), new((m, top), I32), new((m, top), F32)
    l = new((m, 64), F32)
    ex = [x, ids, wt, gu[0], gu[1], dn[0], dn[1]]

    def experts(at, value, **kw):
        a = list(ex)
        a[at] = value
        return lambda: sp.experts_int4(*a, **kw)

    bad = {
        "quant group": lambda: sp.quant_int4(new((4, 96)), group=64),
        "quant group size": lambda: sp.quant_int4(new((4, 256)), group=256),
        "quant type": lambda: sp.quant_int4(new((4, 256), F32)),
        "quant zeros_out": lambda: sp.quant_int4(new((4, 256)), zeros_out=new((4, 2), U8)),
        "quant out": lambda: sp.quant_int4(new((4, 256)), out=new((4, 64), U8)),
        "quant strides": lambda: sp.quant_int4(new((256, 4)).t()),
        "dequant scales": lambda: sp.dequant_int4(w[0], new((512, 3))),
        "dequant scale type": lambda: sp.dequant_int4(w[0], new((512, 4), F32)),
        "dequant zeros": lambda: sp.dequant_int4(w[0], w[1], new((512, 2), U8)),
        "gemm columns": lambda: sp.gemm_int4(new((m, 128)), w[0], w[1]),
        "gemm scales rows": lambda: sp.gemm_int4(x, w[0], new((256, 4))),
        "gemm out": lambda: sp.gemm_int4(x, w[0], w[1], out=new((m, 256))),
        "gemm device": lambda: sp.gemm_int4(torch.empty((m, d), dtype=torch.bfloat16, device="cuda:0"), w[0], w[1]),
        "gemm workspace": lambda: sp.gemm_int4(x, w[0], w[1], ws=torch.empty(64, dtype=U8)),
        "route top": lambda: sp.route(l, 65),
        "route groups": lambda: sp.route(l, 4, groups=5),
        "route top of groups": lambda: sp.route(l, 5, groups=16, top_groups=1),
        "route kind": lambda: sp.route(l, 4, kind=2),
        "route best": lambda: sp.route(l, 4, group_best=3),
        "route bias": lambda: sp.route(l, 4, bias=new(63, F32)),
        "route bias type": lambda: sp.route(l, 4, bias=new(64)),
        "route type": lambda: sp.route(new((m, 64), torch.float16), 4),
        "route ids": lambda: sp.route(l, 4, ids=new((m, 4), torch.int64)),
        "route factor": lambda: sp.route(l, 4, factor=float("inf")),
        "experts ids": experts(1, new((m, top), torch.int64)),
        "experts ids rows": experts(1, new((m + 1, top), I32)),
        "experts weights": experts(2, new((m, top + 1), F32)),
        "experts down": experts(5, new((E, d, f), U8)),
        "experts count": experts(5, new((E + 1, d, f // 2), U8)),
        "experts gate": experts(3, new((E, f, d // 2), U8)),
        "experts scales": experts(4, new((E, 2 * f, 3))),
        "experts zeros": lambda: sp.experts_int4(*ex, gu_zeros=new((E, 2 * f, 2), U8)),
        "experts groups": lambda: sp.experts_int4(*ex[:5], dn[0], new((E, d, f // 32))),
    }
    got = {}
    for name, call in bad.items():
        runtime.fake_clear()
        try:
            call()
            got[name] = [None, runtime.fake_count()]
        except Exception as e:
            got[name] = [type(e).__name__, runtime.fake_count()]
    return got


def grids():
    """[status, least and most threads of the grids in x] of calls at the limits of their sizes."""
    at = [ctypes.c_void_p((i + 1) << 45) for i in range(12)]
    got = {}

    def run(name, call):
        runtime.fake_clear()
        status = call()
        t = [l.grid[0] * l.block[0] for l in runtime.fake_launches()[:runtime.fake_count()]]
        got[name] = [status, min(t), max(t)] if t else [status, 0, 0]

    for m, n, k in ((1, 1 << 21, 128), (2, 1 << 21, 1 << 20), (3, 1 << 21, 128), (1024, 1 << 21, 4096), (1 << 21, 1 << 17, 128),
                    (1 << 21, 1, 128), (1 << 21, 1 << 21, 128), (16, 1 << 16, 1 << 20), (1000, 8, 1 << 20)):
        run("gemm %d %d %d" % (m, n, k),
            lambda: sp.lib.sp24_gemm_int4(m, n, k, 128, *at[:5], at[5], 1 << 44, None))
    for tokens, count, top, d, f in ((4, 1024, 64, 32, 1 << 18), (1, 1, 1, 1 << 20, 1 << 20), (1 << 21, 1024, 1, 32, 32),
                                     (1 << 15, 8, 64, 4096, 4096), (1, 1024, 64, 4096, 4096), (64, 8, 2, 256, 1 << 20)):
        st = sp._ExpertsStruct(count, d, f, 32, *[a.value for a in at[:6]])
        run("experts %d %d %d %d %d" % (tokens, count, top, d, f),
            lambda: sp.lib.sp24_experts_int4(ctypes.byref(st), tokens, top, *at[6:10], at[10], 1 << 44, None))
    r = sp._RouterStruct(1, 1, 1024, 64, 64, 64, 2, 1, 1.0)
    run("route", lambda: sp.lib.sp24_route(ctypes.byref(r), 1 << 21, *at[:4], None))
    return got


if __name__ == "__main__":
    torch.cuda.set_device(0)
    print(json.dumps(globals()[sys.argv[2]]()))
