"""MXFP4 operands, their products and the fused norms in NumPy, in float64.

Test infrastructure only; shares no code with the library.  bf16 tensors are
uint16 bit patterns, as in sp24_ref.  A block of 32 values of a row is stored as
E2M1 codes (sign, two exponent bits, one mantissa bit) and the byte e + 127 of
its scale 2^e, e = floor(log2 amax) - 2 held to [-127, 127] (0 for a block of
zeros); a block with an Inf or NaN has byte 255 and codes 0.
"""
from __future__ import annotations

import numpy as np

from oracle.sp24_ref import bf16_to_f64

# the sixteen E2M1 values, by the format's definition
E2M1 = np.array([(-1.0) ** (c >> 3) * ((c & 1) * 0.5 if not (c >> 1) & 3 else
                                       2.0 ** (((c >> 1) & 3) - 1) * (1 + 0.5 * (c & 1))) for c in range(16)])


def e2m1_encode(u):
    """Codes of float64 values: the nearest E2M1 value, ties to the even code, saturated at 6; the
    sign is kept where the code is not zero or the value is negative."""
    a = np.abs(u)
    mid = (E2M1[:7] + E2M1[1:8]) / 2
    pick = np.searchsorted(mid, a, side="left")  # a tie stays with the lower code ...
    tie = a == mid[np.minimum(pick, 6)]
    pick = np.where(tie & (pick % 2 == 1), pick + 1, pick)  # ... unless that one is odd
    return (pick + 8 * np.signbit(u)).astype(np.uint8)


def block_scale_bytes(v):
    """Scale bytes [rows, cols/32] of float64 values [rows, cols]."""
    b = np.abs(v.reshape(v.shape[0], -1, 32))
    finite = np.isfinite(b).all(-1)
    amax = np.where(finite, b.max(-1), 1.0)
    e = np.floor(np.log2(np.where(amax > 0, amax, 1.0)))
    # log2 can round up just below a power of two
    e = np.where(np.where(amax > 0, amax, 1.0) < 2.0 ** e, e - 1, e) - 2
    e = np.clip(np.where(amax > 0, e, 0), -127, 127)
    return np.where(finite, e + 127, 255).astype(np.uint8)


def quant(v):
    """float64 [rows, cols] -> (codes uint8 [rows, cols/2], scale bytes [rows, cols/32])."""
    rows, cols = v.shape
    s = block_scale_bytes(v)
    bad = (s == 255)[..., None]
    u = np.where(bad, 0.0, v.reshape(rows, -1, 32)) / 2.0 ** (s.astype(np.float64) - 127)[..., None]
    c = np.where(bad, 0, e2m1_encode(u)).reshape(rows, cols).astype(np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def quant_bits(x_bits):
    return quant(bf16_to_f64(x_bits))


def scale_values(s):
    return np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))


def dequant(codes, s):
    """float64 values of codes [rows, cols/2] and scale bytes [rows, cols/32]."""
    rows, half = codes.shape
    c = np.empty((rows, 2 * half), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    return E2M1[c] * np.repeat(scale_values(s), 32, axis=1)


def store_scales(s):
    """Scale bytes [rows, cols/32] in storage order: words of 4 blocks, blocks of 4 words."""
    rows, nb = s.shape
    out = []
    for b0 in range(0, nb, 16):
        out.append(s[:, b0:b0 + 16].reshape(-1))
    return np.concatenate(out)


def load_scales(stored, rows, cols):
    nb, out, at = cols // 32, np.empty((rows, cols // 32), np.uint8), 0
    for b0 in range(0, nb, 16):
        w = min(16, nb - b0)
        out[:, b0:b0 + w] = stored[at:at + rows * w].reshape(rows, w)
        at += rows * w
    return out


def gemm_ref(x, w):
    """(x w^T, |x| |w|^T) of float64 values."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def gated_ref(x, w):
    """(h, how far an h may be off when each product is off by up to d times its sum of
    magnitudes: returned for d = 1) of float64 values, w = [gate rows; up rows]."""
    f = w.shape[0] // 2
    g, gm = gemm_ref(x, w[:f])
    u, um = gemm_ref(x, w[f:])
    a = silu(g)
    return a * u, 1.1 * np.abs(u) * gm + np.abs(a) * um  # |silu'| < 1.1


def norm_ref(x_bits, res_bits, w_bits, eps):
    """(v, t): the normed rows and the sums with the residual, float64."""
    t = bf16_to_f64(x_bits)
    if res_bits is not None:
        t = t + bf16_to_f64(res_bits)
    return t / np.sqrt((t * t).mean(-1, keepdims=True) + eps) * bf16_to_f64(w_bits), t
