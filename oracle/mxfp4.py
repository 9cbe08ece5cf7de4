"""MXFP4 codec of the oracle and the expert MLP on it (float64, numpy).  Test
infrastructure only.

MXFP4 is MXFP8 ("Efficient MoE Training for Biological Foundation Models",
Challenge 2: one scaling factor per 32 consecutive values) with 4-bit elements:

* element type E2M1: sign, two exponent bits (bias 1), one mantissa bit; the
  magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; no NaN, no infinity;
* scale type E8M0, 2^(b-127), b = 0xFF is NaN;
* scale exponent s = the smallest integer with amax <= 6 * 2^s, clamped to
  [-127, 127]; an all-zero block gets -127, one holding a NaN or an infinity the
  NaN byte;
* element code = the nearest E2M1 value of v * 2^-s, ties to the even code.
  The smallest scale keeps every magnitude within 6, so nothing saturates.

The scale is found here by trying exponents, not from the amax's bits.
"""
from __future__ import annotations

import numpy as np

from . import moe

BLOCK = 32
MAGNITUDES = np.array([(1.0 + (c & 1) / 2.0) * 2.0 ** ((c >> 1) - 1) if c >> 1 else (c & 1) / 2.0 for c in range(8)])
SCALE_NAN = 0xFF


def scale_bytes(amax: np.ndarray) -> np.ndarray:
    """Block amax -> E8M0 byte, by search over the exponents."""
    amax = np.asarray(amax, np.float64)
    bounds = 6.0 * 2.0 ** np.arange(-127, 128, dtype=np.float64)   # largest amax of each exponent
    b = np.searchsorted(bounds, np.where(np.isfinite(amax), amax, 0.0), side="left")
    b = np.minimum(b, 254)
    return np.where(np.isfinite(amax), b, SCALE_NAN).astype(np.uint8)


def scale_values(b: np.ndarray) -> np.ndarray:
    b = np.asarray(b, np.int64)
    return np.where(b == SCALE_NAN, np.nan, np.ldexp(1.0, b - 127))


def encode(a: np.ndarray) -> np.ndarray:
    """Values (already divided by their scale) -> codes 0..15: all eight
    magnitudes tried, the nearest taken, of two the even code."""
    a = np.asarray(a, np.float64)
    mag = np.abs(a)
    best = np.zeros(a.shape, np.int64)
    err = np.full(a.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):      # even codes first: an odd one has to be strictly nearer
        d = np.abs(mag - MAGNITUDES[c])
        take = d < err
        best = np.where(take, c, best)
        err = np.where(take, d, err)
    return (best | (np.signbit(a).astype(np.int64) << 3)).astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    c = np.asarray(codes, np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def quantize_rows(x: np.ndarray):
    """[M, K] along K -> (codes uint8 [M, K] one per element, scale bytes
    uint8 [M, K/32]); the codes of a NaN block are left at 0."""
    x = np.asarray(x, np.float64)
    blk = x.reshape(x.shape[0], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        amax = np.abs(blk).max(axis=2)
    amax = np.where(np.isnan(blk).any(axis=2), np.nan, amax)
    b = scale_bytes(amax)
    s = np.where(b == SCALE_NAN, 1.0, scale_values(b))[:, :, None]
    fin = np.where(b[:, :, None] == SCALE_NAN, 0.0, blk)
    return encode(fin / s).reshape(x.shape), b


def dequantize_rows(codes: np.ndarray, b: np.ndarray) -> np.ndarray:
    v = decode(codes).reshape(codes.shape[0], -1, BLOCK)
    return (v * scale_values(b)[:, :, None]).reshape(codes.shape)


def roundtrip_rows(x: np.ndarray) -> np.ndarray:
    return dequantize_rows(*quantize_rows(x))


def pack(codes: np.ndarray) -> np.ndarray:
    """Codes [..., K] -> bytes [..., K/2], the even element in the low half."""
    c = np.asarray(codes, np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    q = np.asarray(q, np.uint8)
    return np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], -1)


def forward(x, w1, w2, topk_idx, topk_prob):
    """The expert MLP with MXFP4 operands, unrounded: x [T, H], w1 [E, 2I, H]
    (gate rows first), w2 [E, H, I].  A slot whose expert id is no expert's
    leaves nothing.  Returns the layer's output and, per expert, what the
    tests' allowances need."""
    x = np.asarray(x, np.float64)
    T, k = topk_idx.shape
    E, H, I = w2.shape
    xq = roundtrip_rows(x)
    out = np.zeros((T, H))
    parts = []
    for e in range(E):
        t, j = np.nonzero(topk_idx == e)
        if t.size == 0:
            continue
        w1q, w2q = roundtrip_rows(w1[e]), roundtrip_rows(w2[e])
        a = xq[t] @ w1q.T
        g, u = a[:, :I], a[:, I:]
        p = np.asarray(topk_prob, np.float64)[t, j][:, None]
        with np.errstate(over="ignore"):
            h = p * moe.silu(g) * u
        y = roundtrip_rows(h) @ w2q.T
        np.add.at(out, t, y)
        parts.append(dict(e=e, t=t, a=xq[t], w1q=w1q, w2q=w2q, g=g, u=u, p=p, h=h, y=y))
    return dict(out=out, parts=parts)
