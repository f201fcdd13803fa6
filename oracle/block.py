"""The block-scaled FP8 operators from their definitions, in fp64 NumPy.

Scales are fp32 values (they are stored as such) and a code is the e4m3 value
nearest to the fp32 quotient v / s, ties to even; everything else is fp64.
"""

import numpy as np

from . import formats as F

BLOCK = 128


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def quantize_rows(v):
    """v [M, K] fp64 -> (codes u8 [M, K], scales fp32 [M, K / 128 rounded up])."""
    v = np.asarray(v, dtype=np.float64)
    M, K = v.shape
    q = np.zeros((M, K), np.uint8)
    s = np.zeros((M, blocks(K)), np.float32)
    for b in range(blocks(K)):
        c = v[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b] = (np.abs(c).max(axis=1) / 448.0).astype(np.float32)
        d = s[:, b].astype(np.float64)[:, None]
        t = np.where(d > 0, c / np.where(d > 0, d, 1.0), 0.0).astype(np.float32)
        q[:, b * BLOCK:(b + 1) * BLOCK] = F.e4m3_encode(F.e4m3_round(t.astype(np.float64)))
    return q, s


def quantize_weight(w):
    """w [N, K] -> (codes u8 [N, K], scales fp32 [N / 128, K / 128], rounded up)."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    q = np.zeros((N, K), np.uint8)
    s = np.zeros((blocks(N), blocks(K)), np.float32)
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            c = w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            a = np.float32(np.abs(c).max() / 448.0)
            s[i, j] = a
            if a > 0:
                t = (c / np.float64(a)).astype(np.float32)
                q[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = F.e4m3_encode(F.e4m3_round(t.astype(np.float64)))
    return q, s


def dequantize_rows(q, s):
    K = q.shape[1]
    return F.e4m3_decode(q) * np.repeat(s.astype(np.float64), BLOCK, axis=1)[:, :K]


def dequantize_weight(q, s):
    N, K = q.shape
    wide = np.repeat(np.repeat(s.astype(np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return F.e4m3_decode(q) * wide[:N, :K]


def rmsnorm(x, weight=None, eps=1e-6, residual=None):
    """(v, r): the norm of r = x + residual, and r."""
    r = np.asarray(x, np.float64)
    if residual is not None:
        r = r + residual
    v = r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    return (v if weight is None else v * weight), r


def silu_mul(x):
    K = x.shape[1] // 2
    g, u = np.asarray(x[:, :K], np.float64), np.asarray(x[:, K:], np.float64)
    return g / (1.0 + np.exp(-g)) * u


def linear(q, s, wq, ws, bias=None):
    y = dequantize_rows(q, s) @ dequantize_weight(wq, ws).T
    return y if bias is None else y + bias


def experts(q, s, wq, ws, offsets, bias=None):
    """Rows offsets[e] .. offsets[e + 1] of q by the weight of expert e; NaN
    where no expert has a row."""
    y = np.full((q.shape[0], wq.shape[1]), np.nan)
    for e in range(wq.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            y[a:b] = linear(q[a:b], s[a:b], wq[e], ws[e], None if bias is None else bias[e])
    return y
