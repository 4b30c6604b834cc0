"""CPU oracle of the integer 4-bit weights, the router and the experts' block, NumPy in 64 bits.

Written from the definitions alone; shares no code with the kernels or their binding.
"""
from __future__ import annotations

import numpy as np

from .sp24_ref import bf16_to_f32

BF16_MIN_EXP = -133  # 2^-133: bf16's least subnormal


def bf16_round(v):
    """float64 -> the nearest bf16 value (ties to even), as float64; finite."""
    v = np.asarray(v, dtype=np.float64)
    e = np.frexp(v)[1]  # v = m 2^e, 0.5 <= |m| < 1: a step is 2^(e - 8)
    step = np.exp2(np.maximum(e - 8, BF16_MIN_EXP).astype(np.float64))
    return np.where(v == 0, 0.0, np.rint(v / step) * step)


def bits_of(v):
    """bf16-valued float64 -> uint16 patterns (NaN: 0x7FC0)."""
    f = np.asarray(v, dtype=np.float64).astype(np.float32)
    return np.where(np.isnan(f), np.uint16(0x7FC0), (f.view(np.uint32) >> 16).astype(np.uint16))


def pack(q):
    """Numbers 0..15 [..., cols] -> bytes [..., cols/2]: value j of eight at bits 4 (j // 2) + 16 (j % 2)."""
    q = np.asarray(q, dtype=np.uint32).reshape(*np.shape(q)[:-1], -1, 8)
    word = np.zeros(q.shape[:-1], dtype=np.uint32)
    for j in range(8):
        word |= q[..., j] << np.uint32(4 * (j // 2) + 16 * (j % 2))
    return np.ascontiguousarray(word.astype("<u4")).view(np.uint8).reshape(*q.shape[:-2], -1)


def unpack(codes):
    word = np.ascontiguousarray(codes).view("<u4").astype(np.uint32)
    q = [(word >> np.uint32(4 * (j // 2) + 16 * (j % 2))) & np.uint32(15) for j in range(8)]
    return np.stack(q, -1).reshape(*codes.shape[:-1], -1).astype(np.uint8)


def quant(w_bits, group, zeros):
    """bf16 patterns [rows, cols] -> (numbers q [rows, cols], scales float64 [rows, groups], z or None)."""
    rows, cols = w_bits.shape
    w = bf16_to_f32(w_bits).astype(np.float64).reshape(rows, cols // group, group)
    bad = ~np.isfinite(w).all(-1, keepdims=True)
    w = np.where(bad, 0.0, w)
    if zeros:
        lo, hi = np.minimum(w.min(-1, keepdims=True), 0.0), np.maximum(w.max(-1, keepdims=True), 0.0)
        s = bf16_round((hi - lo) / 15.0)
        s = np.where(s == 0, 1.0, s)
        z = np.clip(np.rint(-lo / s), 0, 15)
        q = np.clip(np.rint(w / s) + z, 0, 15)
    else:
        s = bf16_round(np.abs(w).max(-1, keepdims=True) / 7.0)
        s = np.where(s == 0, 1.0, s)
        z = np.full_like(s, 8.0)
        q = np.clip(np.rint(w / s), -8, 7) + 8
    q, z, s = np.where(bad, 8.0, q), np.where(bad, 8.0, z), np.where(bad, np.nan, s)
    return (q.reshape(rows, cols).astype(np.uint8), s[..., 0], z[..., 0].astype(np.uint8) if zeros else None)


def dequant(q, scales, z=None):
    """(q - z) s in float64; q [..., cols] numbers, scales and z [..., groups]."""
    g = q.shape[-1] // scales.shape[-1]
    zz = 8.0 if z is None else np.repeat(z.astype(np.float64), g, -1)
    return (q.astype(np.float64) - zz) * np.repeat(np.asarray(scales, np.float64), g, -1)


def silu(x):
    return x / (1.0 + np.exp(-x))


def route(logits, top, sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1, renormalise=True, factor=1.0):
    """float64 logits [tokens, experts] -> (ids, weights), one row after the other."""
    l = np.asarray(logits, np.float64)
    tokens, experts = l.shape
    ids, weights = np.zeros((tokens, top), np.int32), np.zeros((tokens, top))
    for t in range(tokens):
        row = np.minimum(np.where(np.isnan(l[t]), -np.inf, l[t]), np.finfo(np.float32).max)
        masked = np.isneginf(row)
        with np.errstate(all="ignore"):
            if sigmoid:
                score = 1.0 / (1.0 + np.exp(-row))
            else:
                score = np.exp(row - (0.0 if masked.all() else row.max()))
                score = score / score.sum() if score.sum() != 0 else np.zeros(experts)
        score = np.where(masked, 0.0, score)
        choice = row if bias is None else score + np.asarray(bias, np.float64)
        choice = np.where(masked | np.isnan(choice), -np.inf, choice)
        allowed = np.ones(experts, bool)
        if groups > 1:
            n = experts // groups
            value = np.full(groups, -np.inf)
            for g in range(groups):
                of = score if bias is None and group_best == 2 else choice
                there = [v for v, c in zip(of[g * n:(g + 1) * n], choice[g * n:(g + 1) * n]) if c != -np.inf]
                if there:
                    value[g] = sum(sorted(there)[-group_best:])
            best = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            allowed = np.isin(np.arange(experts) // n, best)
        order = sorted(np.flatnonzero(allowed), key=lambda e: (-choice[e], e))[:top]
        w = score[order]
        if renormalise:
            with np.errstate(all="ignore"):
                if not sigmoid:  # the softmax over those chosen
                    at = row[order]
                    w = np.exp(at - (0.0 if np.isneginf(at).all() else at.max()))
                w = w / w.sum() if w.sum() != 0 else np.zeros(top)
        ids[t], weights[t] = order, w * factor
    return ids, weights
