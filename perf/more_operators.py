"""Cases and plain forms of the operators over integer 4-bit weights with group scales and of the
router to experts.

Four operators that a server of feed-forward blocks (dense or of experts) runs, each at the sizes
this repository's workloads have (an 8B-class model's projections at decode and prefill, its
4096 x 14336 block cut into experts of 1792) and at ragged ones:

  quant    bf16 W -> 4-bit codes with a bf16 scale (and a zero point) per group, and the values
           they stand for
  gemm     Y = X . W^T, X in bf16 and W in that form, bf16 out
  route    scores of a token's experts, limited to groups, the best few of them and their weights
  experts  sum over a token's experts of weight * down(silu(gate(x)) * up(x)), weights in that form

Storage: w = (q - z) s. Codes uint8 [rows, cols/2], eight values of a row to four bytes, value j of
them at bits 4 (j / 2) + 16 (j % 2) of the little-endian word; scales bf16 and zero points uint8
(absent: 8) [rows, cols/group].
"""
import math

import torch

own = False

GATE_UP = 28672


def listed():
    return [
        # a down-projection's weight prepared at load time
        {"name": "quant_4096x14336", "op": "quant", "n": 4096, "k": 14336, "group": 128, "zeros": False},
        # a whole gate+up weight, with zero points and small groups
        {"name": "quant_zeros_28672x8192", "op": "quant", "n": GATE_UP, "k": 8192, "group": 64, "zeros": True},
        # up-projection of one token: latency and the weight's bytes
        {"name": "gemm_1x14336x4096", "op": "gemm", "m": 1, "n": 14336, "k": 4096, "group": 128, "zeros": False},
        # down-projection of a decode batch: long rows, zero points
        {"name": "gemm_16x4096x14336", "op": "gemm", "m": 16, "n": 4096, "k": 14336, "group": 128, "zeros": True},
        # fused QKV projection of a ragged decode batch, the smallest groups
        {"name": "gemm_77x6144x4096", "op": "gemm", "m": 77, "n": 6144, "k": 4096, "group": 32, "zeros": False},
        # gate+up projection of a 2047-token prompt: matrix-core throughput
        {"name": "gemm_2047x28672x8192", "op": "gemm", "m": 2047, "n": GATE_UP, "k": 8192, "group": 128,
         "zeros": False},
        # the router of one token: the smallest call
        {"name": "route_1x64", "op": "route", "m": 1, "experts": 64, "top": 8, "kind": "softmax", "bf16": False,
         "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "renormalise": True},
        # a prompt's tokens over many experts in groups, with a bias that balances their load
        {"name": "route_groups_8191x256", "op": "route", "m": 8191, "experts": 256, "top": 8, "kind": "sigmoid",
         "bf16": False, "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "renormalise": True},
        # a prompt's tokens over 60 experts, bf16 logits, weights as the softmax gives them
        {"name": "route_4000x60", "op": "route", "m": 4000, "experts": 60, "top": 4, "kind": "softmax", "bf16": True,
         "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "renormalise": False},
        # the experts of one token
        {"name": "experts_1x4096x1792", "op": "experts", "m": 1, "d": 4096, "f": 1792, "experts": 64, "top": 8,
         "group": 128, "zeros": False},
        # a ragged decode batch: nearly every expert has a few tokens
        {"name": "experts_29x4096x1792", "op": "experts", "m": 29, "d": 4096, "f": 1792, "experts": 64, "top": 8,
         "group": 128, "zeros": True},
        # a prompt: experts with two hundred tokens on average
        {"name": "experts_1777x4096x1792", "op": "experts", "m": 1777, "d": 4096, "f": 1792, "experts": 64, "top": 8,
         "group": 128, "zeros": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("quant", "gemm", "gemm", "route", "route", "experts", "experts"))
        group, zeros = rng.choice((32, 64, 128)), rng.random() < 0.4
        if op == "route":
            e = _log(rng, 8, 512)
            groups = rng.choice([g for g in (1, 1, 2, 4, 8) if e % g == 0 and e // g >= 2])
            top_groups = rng.randint(1, groups)
            case = {"op": op, "m": _log(rng, 1, 8192), "experts": e,
                    "top": rng.randint(1, min(10, top_groups * (e // groups))),
                    "kind": rng.choice(("softmax", "sigmoid")), "bf16": rng.random() < 0.5, "bias": rng.random() < 0.5,
                    "groups": groups, "top_groups": top_groups, "group_best": rng.choice((1, 2)),
                    "renormalise": rng.random() < 0.6}
            if case["m"] * e <= 8191 * 256:
                return case
        elif op == "experts":
            e = _log(rng, 2, 128)
            case = {"op": op, "m": _log(rng, 1, 2048), "d": 128 * _log(rng, 1, 32), "f": 128 * _log(rng, 1, 32),
                    "experts": e, "top": rng.randint(1, min(8, e)), "group": group, "zeros": zeros}
            size = case["d"] * case["f"]
            if e * size <= 64 * 4096 * 1792 and case["m"] * case["top"] * size <= 1777 * 8 * 4096 * 1792:
                return case
        else:
            case = {"op": op, "n": _log(rng, 1, GATE_UP), "k": group * _log(rng, 1, 14336 // group), "group": group,
                    "zeros": zeros}
            if op == "gemm":
                case["m"] = _log(rng, 1, 4096)
            if case["n"] * case["k"] <= GATE_UP * 8192 and case.get("m", 1) * case["n"] * case["k"] <= 2047 * GATE_UP * 8192:
                return case


def work(case):
    op = case["op"]
    if op == "route":
        m, e, top = case["m"], case["experts"], case["top"]
        return {"bytes": (2 if case["bf16"] else 4) * m * e + 8 * m * top + (4 * e if case["bias"] else 0),
                "flops": 4 * m * e}
    per = 0.5 + (3 if case["zeros"] else 2) / case["group"]  # bytes of a value with its share of scale and zero
    if op == "quant":
        return {"bytes": 4 * case["n"] * case["k"], "flops": 4 * case["n"] * case["k"]}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": per * n * k + 2 * m * (n + k), "flops": 2 * m * n * k}
    m, d, f, e, top = case["m"], case["d"], case["f"], case["experts"], case["top"]
    used = e * (1 - (1 - top / e) ** m)  # experts that a token went to, were all alike
    return {"bytes": per * 3 * used * d * f + 4 * m * d + 8 * m * top, "flops": 6 * m * top * d * f}


# ---------------------------------------------------------------- inputs


_PLACES = (0, 2, 4, 6, 1, 3, 5, 7)  # the value that each four bits of a word hold, lowest first


def _pack(q):
    """Codes [rows, cols] as numbers 0..15 -> bytes [rows, cols/2]."""
    b = q.to(torch.uint8).view(q.shape[0], -1, 8)[:, :, list(_PLACES)]
    return (b[:, :, 0::2] | (b[:, :, 1::2] << 4)).reshape(q.shape[0], -1)


def _unpack(codes):
    c = codes.view(codes.shape[0], -1, 4)
    p = torch.stack((c & 15, c >> 4), -1).view(codes.shape[0], -1, 8)
    return p[:, :, [_PLACES.index(j) for j in range(8)]].reshape(codes.shape[0], -1)


def _quantise(w, group, zeros):
    """(codes, scales, zero points or None) of bf16 w."""
    v = w.float().view(w.shape[0], -1, group)
    one = torch.ones((), device=w.device)
    if not zeros:
        s = (v.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).float()
        s = torch.where(s > 0, s, one)
        q = torch.round(v / s).clamp(-8, 7) + 8
        z = None
    else:
        lo, hi = v.amin(-1, keepdim=True).clamp(max=0), v.amax(-1, keepdim=True).clamp(min=0)
        s = ((hi - lo) / 15).to(torch.bfloat16).float()
        s = torch.where(s > 0, s, one)
        z = torch.round(-lo / s).clamp(0, 15)
        q = (torch.round(v / s) + z).clamp(0, 15)
        z = z.squeeze(-1).to(torch.uint8)
    return _pack(q.view(w.shape)), s.squeeze(-1).to(torch.bfloat16), z


def _randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _activations(m, k, g):
    """N(0, 1) with 1% of the channels 20 times as large, as a model's residual stream has."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x[:, torch.randperm(k, generator=g, device="cuda")[: max(1, round(0.01 * k))]] *= 20.0
    return x.to(torch.bfloat16)


def _logits(m, e, g):
    """Experts differ in how often they are wanted."""
    return 1.5 * torch.randn((m, e), generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")


def _expert_weights(e, n, k, g, case):
    parts = [_quantise(_randn((n, k), g, 0.02), case["group"], case["zeros"]) for _ in range(e)]
    return [torch.stack(p) if p[0] is not None else None for p in zip(*parts)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case)
    if op == "quant":
        n, k, group = case["n"], case["k"], case["group"]
        st["w"] = _randn((n, k), g, 0.02)
        if case["zeros"]:
            st["w"] += 0.01 * torch.randn((n, 1), generator=g, device="cuda").to(torch.bfloat16)
            st["z"] = torch.empty((n, k // group), dtype=torch.uint8, device="cuda")
        st["codes"] = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty((n, k // group), dtype=torch.bfloat16, device="cuda")
        st["out"] = torch.empty_like(st["w"])
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = _activations(m, k, g)
        st["w"] = _quantise(_randn((n, k), g, 0.02), case["group"], case["zeros"])
        st["y"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    elif op == "route":
        m, e, top = case["m"], case["experts"], case["top"]
        st["logits"] = _logits(m, e, g).to(torch.bfloat16 if case["bf16"] else torch.float32)
        st["b"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        st["ids"] = torch.empty((m, top), dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty((m, top), device="cuda")
    else:
        m, d, f, e, top = case["m"], case["d"], case["f"], case["experts"], case["top"]
        st["x"] = _activations(m, d, g)
        l = _logits(m, e, g)
        order = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :top]
        st["ids"] = order.to(torch.int32)
        st["weights"] = torch.softmax(torch.gather(l, 1, order), 1)
        st["gu"] = _expert_weights(e, 2 * f, d, g, case)
        st["dn"] = _expert_weights(e, d, f, g, case)
        st["y"] = torch.empty((m, d), dtype=torch.bfloat16, device="cuda")
        if own:  # the workspace that a program keeps
            import bf16_gemm_linear_amd as sp

            st["ws"] = torch.empty(sp.experts_int4_workspace_size(m, d, f, e, top), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- the framework's operators


def _own(st):
    import bf16_gemm_linear_amd as sp

    op = st["op"]
    if op == "quant":
        c, s, z = sp.quant_int4(st["w"], group=st["group"], zeros=st["zeros"], out=st["codes"], scales_out=st["s"],
                                zeros_out=st.get("z"))
        return {"values": sp.dequant_int4(c, s, z, out=st["out"])}
    if op == "gemm":
        return {"y": sp.gemm_int4(st["x"], *st["w"], out=st["y"])}
    if op == "route":
        kind = sp.ROUTE_SOFTMAX if st["kind"] == "softmax" else sp.ROUTE_SIGMOID
        ids, w = sp.route(st["logits"], st["top"], kind=kind, bias=st["b"], groups=st["groups"],
                          top_groups=st["top_groups"], group_best=st["group_best"], renormalise=st["renormalise"],
                          ids=st["ids"], weights=st["weights"])
        return {"ids": ids, "weights": w}
    (gc, gs, gz), (dc, ds, dz) = st["gu"], st["dn"]
    return {"y": sp.experts_int4(st["x"], st["ids"], st["weights"], gc, gs, dc, ds, gu_zeros=gz, down_zeros=dz,
                                 out=st["y"], ws=st["ws"])}


# ---------------------------------------------------------------- plain forms


def _values(codes, scales, zeros):
    """What codes, scales and zero points stand for, fp32 [rows, cols]."""
    rows, groups = scales.shape
    q = _unpack(codes).float().view(rows, groups, -1)
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).view(rows, -1)


def _gated(y):
    gate, up = y.chunk(2, dim=1)
    return gate / (1 + torch.exp(-gate)) * up


def _best(c, count):
    """The indices of the `count` largest of each row, ties to the lowest index."""
    return torch.sort(c, dim=1, descending=True, stable=True)[1][:, :count]


def _route(st):
    l = st["logits"].double()  # the order of near scores
    m, e = l.shape
    if st["kind"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    c = l if st["b"] is None else p + st["b"].double()
    if st["groups"] > 1:
        n = e // st["groups"]
        if st["b"] is None and st["group_best"] > 1:
            v = torch.sort(p.view(m, -1, n), dim=2, descending=True)[0]
        else:
            v = torch.sort(c.view(m, -1, n), dim=2, descending=True)[0]
        keep = torch.zeros((m, st["groups"]), dtype=torch.bool, device=l.device)
        keep.scatter_(1, _best(v[:, :, : st["group_best"]].sum(2), st["top_groups"]), True)
        c = torch.where(keep.repeat_interleave(n, 1), c, torch.full((), -math.inf, dtype=c.dtype, device=c.device))
    ids = _best(c, st["top"])
    w = torch.gather(p, 1, ids)
    if st["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w.float()}


def _plain(st):
    op = st["op"]
    if op == "quant":
        return {"values": _values(*_quantise(st["w"], st["group"], st["zeros"])).to(torch.bfloat16)}
    if op == "gemm":
        return {"y": (st["x"].float() @ _values(*st["w"]).t()).to(torch.bfloat16)}
    if op == "route":
        return _route(st)
    x, ids, weights = st["x"].float(), st["ids"], st["weights"]
    y = torch.zeros_like(x)

    def expert(part, e):
        return _values(*(None if t is None else t[e] for t in part))

    for e in torch.unique(ids).tolist():
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        h = _gated(x[token] @ expert(st["gu"], e).t())
        y.index_add_(0, token, (h @ expert(st["dn"], e).t()) * weights[token, slot].unsqueeze(1))
    return {"y": y.to(torch.bfloat16)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits


def _decode64(codes, scales, zeros):
    """Each value's four bits looked up at their place in the row's words."""
    rows, half = codes.shape
    col = torch.arange(2 * half, device=codes.device)
    j = col % 8
    bit = 4 * (j // 2) + 16 * (j % 2)
    q = ((codes[:, 4 * (col // 8) + bit // 8].int() >> (bit % 8)) & 15).double()
    g = col // (2 * half // scales.shape[1])
    return (q - (8 if zeros is None else zeros.double()[:, g])) * scales.double()[:, g]


def _bf16_64(v):
    """v to the nearest of bf16's values (seven of the 52 bits stay), ties to even; still in 64."""
    bits = v.view(torch.int64)
    return ((bits + ((1 << 44) - 1) + ((bits >> 45) & 1)) & ~((1 << 45) - 1)).view(torch.float64)


def _quant64(w, group, zeros):
    v = w.double().view(w.shape[0], -1, group)
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    if zeros:
        lo, hi = lo.clamp(max=0), hi.clamp(min=0)
        s = _bf16_64((hi - lo) / 15)
        s = torch.where(s == 0, 1.0, s)
        z = torch.round(-lo / s).clamp(0, 15)
        return ((torch.round(v / s) + z).clamp(0, 15) - z).mul(s).view(w.shape)
    s = _bf16_64(torch.maximum(hi, -lo) / 7)
    s = torch.where(s == 0, 1.0, s)
    return torch.round(v / s).clamp(-8, 7).mul(s).view(w.shape)


def _route64(st):
    """Places counted: how many of a row come before each."""

    def places(c):
        i = torch.arange(c.shape[1], device=c.device)
        out = torch.empty(c.shape, dtype=torch.int64, device=c.device)
        for a in range(0, c.shape[0], 256):
            v = c[a : a + 256]
            over, same = v[:, None, :] > v[:, :, None], v[:, None, :] == v[:, :, None]
            out[a : a + 256] = (over | (same & (i[None, None, :] < i[None, :, None]))).sum(2)
        return out

    l = st["logits"].double()
    m, e = l.shape
    p = torch.softmax(l, 1) if st["kind"] == "softmax" else torch.sigmoid(l)
    c = l if st["b"] is None else p + st["b"].double()
    if st["groups"] > 1:
        of = p if st["b"] is None and st["group_best"] == 2 else c
        best = torch.topk(of.view(m, st["groups"], -1), st["group_best"], dim=2)[0].sum(2)
        out = places(best) >= st["top_groups"]
        c = c.masked_fill(out.repeat_interleave(e // st["groups"], 1), -math.inf)
    place = places(c)
    ids = torch.empty((m, st["top"]), dtype=torch.int64, device=l.device)
    row, col = torch.nonzero(place < st["top"], as_tuple=True)
    ids[row, place[row, col]] = col
    w = torch.gather(p, 1, ids)
    return {"ids": ids.to(torch.int32), "weights": w / w.sum(1, keepdim=True) if st["renormalise"] else w}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return {"values": _quant64(st["w"], case["group"], case["zeros"])}
    if op == "gemm":
        return {"y": st["x"].double() @ _decode64(*st["w"]).t()}
    if op == "route":
        return _route64(st)
    x, ids = st["x"].double(), st["ids"].long()
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        w = (st["weights"].double() * (ids == e)).sum(1)  # a token has an expert once
        at = torch.nonzero(w)[:, 0]
        if at.numel() == 0:
            continue
        gu, dn = (_decode64(*(None if t is None else t[e] for t in st[part])) for part in ("gu", "dn"))
        a = x[at] @ gu[: case["f"]].t()
        h = a * torch.sigmoid(a) * (x[at] @ gu[case["f"]:].t())
        y[at] += w[at, None] * (h @ dn.t())
    return {"y": y}
