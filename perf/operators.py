"""Cases and plain forms of the microscaled 4-bit (MXFP4) operators and of the fused norms.

Five operators of a feed-forward block served in few bits, each at the sizes this
repository's workloads have (an 8B-class model's projections at decode and prefill, the
8192-token prefill) and at ragged ones:

  quant   bf16 -> E2M1 codes with one E8M0 scale per 32 values, and the values they stand for
  gemm    Y = X . W^T of two such operands, bf16 out
  gated   silu(X . Wg^T) * (X . Wu^T), bf16 out, W = [gate rows; up rows]
  norm    t = x + residual, v = t * rsqrt(mean(t^2) + eps) * weight, v in bf16, in E4M3 or INT8
          with a scale per token, or in E4M3 with a scale per group of the row
  ffn     norm -> MXFP4 -> gated -> MXFP4 -> down-projection, bf16 out

Storage: codes uint8 [rows, cols/2], value 2i of a row in the low half of byte i; scales
uint8, byte (r, b) of block b of row r, four bytes to a word, the cols/128 words of a row
cut into blocks of 4 words, block after block, in each every row's words row after row.
"""
import math

import torch

own = False

GATE_UP = 28672
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the activations of a 16-token decode step in front of a down-projection
        {"name": "quant_16x14336", "op": "quant", "m": 16, "k": 14336},
        # a whole gate+up weight quantised at load time
        {"name": "quant_28672x8192", "op": "quant", "m": GATE_UP, "k": 8192},
        # up-projection of one token: latency and the weight's bytes
        {"name": "gemm_1x14336x4096", "op": "gemm", "m": 1, "n": 14336, "k": 4096},
        # down-projection of a ragged decode batch: few rows of W, long K
        {"name": "gemm_77x4096x14336", "op": "gemm", "m": 77, "n": 4096, "k": 14336},
        # gate+up projection of an 8192-token prefill: matrix-core throughput
        {"name": "gemm_8192x28672x8192", "op": "gemm", "m": 8192, "n": GATE_UP, "k": 8192},
        # gated projection of one token
        {"name": "gated_1x14336x4096", "op": "gated", "m": 1, "n": 14336, "k": 4096},
        # gated projection of a 2047-token prompt
        {"name": "gated_2047x14336x4096", "op": "gated", "m": 2047, "n": 14336, "k": 4096},
        # the norm in front of a projection of one token: the smallest call
        {"name": "norm_fp8_1x4096", "op": "norm", "m": 1, "k": 4096, "kind": "fp8", "group": 0, "residual": True},
        # a 256-token batch in front of an INT8 projection, first layer (no residual yet)
        {"name": "norm_int8_256x4096", "op": "norm", "m": 256, "k": 4096, "kind": "int8", "group": 0,
         "residual": False},
        # a long prompt in front of a projection with a scale per 128 values
        {"name": "norm_groups_8191x8192", "op": "norm", "m": 8191, "k": 8192, "kind": "fp8_groups", "group": 128,
         "residual": True},
        # a feed-forward block at a 16-token decode step, and at a 1000-token prompt
        {"name": "ffn_16x4096x14336", "op": "ffn", "m": 16, "n": 14336, "k": 4096},
        {"name": "ffn_1000x4096x14336", "op": "ffn", "m": 1000, "n": 14336, "k": 4096},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = 8192 * GATE_UP * 8192
    while True:
        op = rng.choice(("quant", "gemm", "gemm", "gated", "norm", "norm", "ffn"))
        m, k = _log(rng, 1, 8192), 128 * _log(rng, 1, 112)
        if op == "quant":
            case = {"op": op, "m": _log(rng, 1, GATE_UP), "k": k}
        elif op == "norm":
            kind = rng.choice(("bf16", "fp8", "int8", "fp8_groups"))
            group = 0
            if kind == "fp8_groups":
                group = rng.choice([g for g in (32, 128, 256, 384, k) if k % g == 0])
            else:
                k = 8 * _log(rng, 1, 2048)
            case = {"op": op, "m": m, "k": k, "kind": kind, "group": group, "residual": rng.random() < 0.7}
        elif op == "gemm":
            case = {"op": op, "m": m, "n": _log(rng, 1, GATE_UP), "k": k}
        elif op == "gated":
            case = {"op": op, "m": m, "n": _log(rng, 1, 14336), "k": k}
        else:
            case = {"op": op, "m": m, "n": 128 * _log(rng, 1, 112), "k": 128 * _log(rng, 1, 64)}
        sizes = [case.get("m"), case.get("n", 1), case.get("k")]
        per = {"gated": 2, "ffn": 3}.get(op, 1)
        if per * sizes[0] * sizes[1] * sizes[2] <= most and not set(sizes) & {3072}:
            return case


def work(case):
    op, m, n, k = case["op"], case["m"], case.get("n", 0), case["k"]
    mx = 0.5 + 1 / 32  # bytes of a value in 4 bits with its share of a scale
    if op == "quant":
        return {"bytes": 4 * m * k, "flops": 4 * m * k}
    if op == "gemm":
        return {"bytes": mx * (m + n) * k + 2 * m * n, "flops": 2 * m * n * k}
    if op == "gated":
        return {"bytes": mx * (m + 2 * n) * k + 2 * m * n, "flops": 4 * m * n * k}
    if op == "norm":
        b = {"bf16": 2, "fp8": 1, "int8": 1, "fp8_groups": 1}[case["kind"]] * m * k + 2 * m * k + 2 * k
        b += 4 * m * (k // case["group"]) if case["group"] else 4 * m
        b += 4 * m * k if case["residual"] else 0
        return {"bytes": b, "flops": 8 * m * k}
    return {"bytes": mx * 3 * n * k + 2 * k + 8 * m * k, "flops": 6 * m * n * k}


# ---------------------------------------------------------------- inputs


def _store(nat):
    """Scales [rows, blocks] in storage order."""
    rows, c = nat.shape
    full = c // 16 * 16
    a = nat[:, :full].reshape(rows, full // 16, 16).transpose(0, 1).reshape(-1)
    return torch.cat((a, nat[:, full:].reshape(-1)))


def _quantise(v):
    """fp32 [rows, cols] -> (codes, scales in storage order): the scale 2^(floor(log2 amax) - 2)
    (1 for a block of zeros), the value to nearest even of E2M1, at most 6 in magnitude."""
    rows, cols = v.shape
    v = v.view(rows, cols // 32, 32)
    amax = v.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.zeros((), dtype=torch.int32, device=v.device))
    e = e.clamp(-127, 127)
    u = v * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)  # times 2^-e, exactly
    a = u.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5
    code += 8 * (u < 0).to(torch.uint8) * (code > 0)
    code = code.view(rows, cols)
    return code[:, 0::2] | (code[:, 1::2] << 4), _store((e + 127).to(torch.uint8))


def _randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _activations(m, k, g):
    """N(0, 1) with 1% of the channels 20 times as large, as a model's residual stream has."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x[:, torch.randperm(k, generator=g, device="cuda")[: max(1, round(0.01 * k))]] *= 20.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, m, n, k = case["op"], case["m"], case.get("n", 0), case["k"]
    st = {key: case[key] for key in case if key != "residual"}
    if op == "quant":
        st["x"] = _activations(m, k, g) if m < 8192 else _randn((m, k), g, 0.02)
        st["codes"] = torch.empty((m, k // 2), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(m * k // 32, dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty_like(st["x"])
        return st
    if op in ("gemm", "gated"):
        st["xq"], st["xs"] = _quantise(_activations(m, k, g).float())
        st["wq"], st["ws"] = _quantise(_randn((n if op == "gemm" else 2 * n, k), g, 0.02).float())
        st["y"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        return st
    st["x"] = _activations(m, k, g)
    if op == "ffn" or case["residual"]:
        st["residual"] = _activations(m, k, g)
        st["residual_out"] = torch.empty_like(st["x"])
    st["weight"] = (1 + 0.1 * torch.randn(k, generator=g, device="cuda")).to(torch.bfloat16)
    if op == "norm":
        kind = case["kind"]
        dt = {"bf16": torch.bfloat16, "int8": torch.int8}.get(kind, torch.float8_e4m3fn)
        st["q"] = torch.empty((m, k), dtype=dt, device="cuda")
        if kind != "bf16":
            st["s"] = torch.empty((m, k // case["group"]) if case["group"] else (m,), device="cuda")
        return st
    st["wq"], st["ws"] = _quantise(_randn((2 * n, k), g, 0.02).float())
    st["dq"], st["ds"] = _quantise(_randn((k, n), g, 0.02).float())
    st["y"] = torch.empty_like(st["x"])
    return st


# ---------------------------------------------------------------- the framework's operators


def _own(st):
    import bf16_gemm_linear_amd as sp

    op = st["op"]
    if op == "quant":
        sp.quant_mxfp4(st["x"], out=st["codes"], scales=st["scales"])
        return {"values": sp.dequant_mxfp4(st["codes"], st["scales"], out=st["out"])}
    if op == "gemm":
        return {"y": sp.gemm_mxfp4(st["xq"], st["xs"], st["wq"], st["ws"], out=st["y"])}
    if op == "gated":
        return {"h": sp.gated_mxfp4(st["xq"], st["xs"], st["wq"], st["ws"], out=st["y"])}
    if op == "ffn":
        y, r = sp.ffn_mxfp4(st["x"], st["weight"], st["wq"], st["ws"], st["dq"], st["ds"], residual=st["residual"],
                            eps=EPS, out=st["y"], residual_out=st["residual_out"])
        return {"y": y, "residual": r}
    kind = {"bf16": sp.NORM_BF16, "fp8": sp.NORM_FP8_ROWS, "int8": sp.NORM_INT8_ROWS,
            "fp8_groups": sp.NORM_FP8_GROUPS}[st["kind"]]
    q, s, r = sp.rmsnorm(st["x"], st["weight"], kind, residual=st.get("residual"), eps=EPS, group=st["group"],
                         out=st["q"], scales=st.get("s"), residual_out=st.get("residual_out"))
    # INT8 codes as the numbers they are, in a floating type (exact up to 2048)
    return {"q": q.to(torch.float16) if st["kind"] == "int8" else q, "s": s, "residual": r}


# ---------------------------------------------------------------- plain forms


def _values(codes, scales):
    """What codes and scales stand for, fp32 [rows, cols]."""
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    c = torch.stack((codes & 15, codes >> 4), -1).view(rows, cols)
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)[c.int()]
    nb = cols // 32
    full = nb // 16 * 16
    nat = torch.empty((rows, nb), dtype=torch.uint8, device=codes.device)
    nat[:, :full] = scales[: rows * full].view(full // 16, rows, 16).transpose(0, 1).reshape(rows, full)
    nat[:, full:] = scales[rows * full:].view(rows, nb - full)
    e = nat.int()
    s = torch.where(e > 0, e << 23, torch.full((), 1 << 22, dtype=torch.int32, device=codes.device))
    return (v.view(rows, nb, 32) * s.view(torch.float32).unsqueeze(-1)).view(rows, cols)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _norm(st):
    t = st["x"].float()
    r = None
    if st.get("residual") is not None:
        t = t + st["residual"].float()
        r = t.to(torch.bfloat16)
    return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * st["weight"].float(), r


def _gated(x, w):
    n = w.shape[0] // 2
    return _silu(x @ w[:n].t()) * (x @ w[n:].t())


def _plain(st):
    op = st["op"]
    if op == "quant":
        return {"values": _values(*_quantise(st["x"].float())).to(torch.bfloat16)}
    if op == "gemm":
        return {"y": (_values(st["xq"], st["xs"]) @ _values(st["wq"], st["ws"]).t()).to(torch.bfloat16)}
    if op == "gated":
        return {"h": _gated(_values(st["xq"], st["xs"]), _values(st["wq"], st["ws"])).to(torch.bfloat16)}
    v, r = _norm(st)
    if op == "ffn":
        h = _gated(_values(*_quantise(v)), _values(st["wq"], st["ws"]))
        y = _values(*_quantise(h)) @ _values(st["dq"], st["ds"]).t()
        return {"y": y.to(torch.bfloat16), "residual": r}
    kind, (m, k) = st["kind"], v.shape
    if kind == "bf16":
        return {"q": v.to(torch.bfloat16), "s": None, "residual": r}
    top = 127.0 if kind == "int8" else 448.0
    v = v.view(m, -1, st["group"] or k)
    amax = v.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    q = (v / s).clamp(-top, top).view(m, k)
    s = s.view(m, -1) if st["group"] else s.view(m)
    q = torch.round(q).to(torch.float16) if kind == "int8" else q.to(torch.float8_e4m3fn)
    return {"q": q, "s": s, "residual": r}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits


def _decode64(codes, scales):
    """Sign, exponent and mantissa of each code put together, with the scale's byte looked up at
    its place in storage."""
    rows, half = codes.shape
    cols = 2 * half
    col = torch.arange(cols, device=codes.device)
    c = (codes[:, col // 2].int() >> (4 * (col % 2))) & 15
    e, f = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e > 0, (1 + f / 2) * torch.exp2(e.double() - 1), f / 2)
    words, b = cols // 128, torch.arange(cols // 32, device=codes.device)
    w = b // 4
    width = torch.clamp(words - 4 * (w // 4), max=4)
    at = 4 * (4 * rows * (w // 4) + torch.arange(rows, device=codes.device)[:, None] * width + w % 4) + b % 4
    s = torch.exp2(scales[at].double() - 127)
    return torch.where(c >= 8, -mag, mag) * s.repeat_interleave(32, dim=1)


def _round_to(v, step):
    return torch.round(v / step) * step  # half to even


def _floor_log2(a):
    return torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))[1].double() - 1


def _mx64(v):
    """The values that the MXFP4 form of v stands for."""
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.exp2((_floor_log2(amax) - 2).clamp(-127, 127)), torch.ones_like(amax))
    u = b / s
    step = torch.exp2(_floor_log2(u.abs()).clamp(min=0) - 1)
    return (_round_to(u, step).clamp(-6, 6) * s).view_as(v)


def _e4m3_64(v):
    return _round_to(v, torch.exp2(_floor_log2(v.abs()).clamp(min=-6) - 3)).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return {"values": _mx64(st["x"].double())}
    if op in ("gemm", "gated"):
        x, w = _decode64(st["xq"], st["xs"]), _decode64(st["wq"], st["ws"])
        y = x @ w.t()
        if op == "gemm":
            return {"y": y}
        a, b = y[:, : case["n"]], y[:, case["n"]:]
        return {"h": a * torch.sigmoid(a) * b}
    t = st["x"].double()
    r = None
    if "residual" in st:
        t = r = t + st["residual"].double()
    v = t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS) * st["weight"].double()
    if op == "ffn":
        y = _mx64(v) @ _decode64(st["wq"], st["ws"]).t()
        a, b = y[:, : case["n"]], y[:, case["n"]:]
        h = _mx64(a * torch.sigmoid(a) * b)
        return {"y": h @ _decode64(st["dq"], st["ds"]).t(), "residual": r}
    kind, m, k = case["kind"], case["m"], case["k"]
    if kind == "bf16":
        return {"q": v, "s": None, "residual": r}
    top = 127 if kind == "int8" else 448
    v = v.view(m, -1, case["group"] or k)
    amax = v.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    q = (v / s).view(m, k)
    q = torch.round(q).clamp(-top, top) if kind == "int8" else _e4m3_64(q)
    return {"q": q, "s": s.view(m, -1) if case["group"] else s.view(m), "residual": r}
