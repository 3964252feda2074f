"""Plain 64-bit references of the operators around the layer: residual add and
RMS norm, sorted token rows, their gradients, and 4-bit expert weights.  numpy
only; shares nothing with the GPU code."""
from __future__ import annotations

import numpy as np


def bf16(a) -> np.ndarray:
    """The nearest bf16 values (ties to even) of fp32 values, as fp32."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return np.where(np.isnan(a), np.float32(np.nan), r.view(np.float32))


def stored(a, act: str) -> np.ndarray:
    """fp32 values as a row of the activation type holds them."""
    a = np.asarray(a, np.float32)
    return bf16(a) if act == "bf16" else a


def rmsnorm(r, weight, eps) -> np.ndarray:
    r = np.asarray(r, np.float64)
    return r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rmsnorm_backward(r, weight, eps, dy, dsum=None):
    """(dx, dweight) of rmsnorm(r) for the output gradient dy; dsum is added to dx."""
    r, w, dy = (np.asarray(a, np.float64) for a in (r, weight, dy))
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    n, g = r * rstd, dy * w
    dx = rstd * (g - n * np.mean(g * n, axis=1, keepdims=True))
    return dx + (0.0 if dsum is None else np.asarray(dsum, np.float64)), np.sum(dy * n, axis=0)


def combine(y, pos, w, n_rows) -> np.ndarray:
    """out[t] = sum_k w[t, k] y[pos[t, k]]; positions outside [0, n_rows) have no row."""
    T, K = w.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for k in range(K):
            p = pos[t * K + k]
            if 0 <= p < n_rows:
                out[t] += float(w[t, k]) * np.asarray(y[p], np.float64)
    return out


def combine_backward_w(dout, y, pos, K) -> np.ndarray:
    """dw[t, k] = <dout[t], y[pos[t, k]]>, 0 for a slot without a row."""
    T = dout.shape[0]
    dw = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            p = pos[t * K + k]
            if 0 <= p < T * K:
                dw[t, k] = np.dot(np.asarray(dout[t], np.float64), np.asarray(y[p], np.float64))
    return dw


def quantize_int4(w, group):
    """(codes [rows, cols] 0..15, scales [rows, cols / group] as fp32) of bf16 values w."""
    w = np.asarray(w, np.float32)
    g = w.reshape(w.shape[0], -1, group)
    s = bf16(np.abs(g).max(axis=2) / np.float32(7.0))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, np.rint(g / s[..., None]), 0.0)
    return (np.clip(q, -8, 7) + 8).astype(np.uint8).reshape(w.shape), s


def pack_nibbles(codes) -> np.ndarray:
    """Two codes a byte, the even column in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def dequantize_int4(codes, scales, group) -> np.ndarray:
    return (codes.astype(np.float64) - 8.0) * np.repeat(np.asarray(scales, np.float64), group, axis=-1)


def swiglu(x, w13, w2) -> np.ndarray:
    x = np.asarray(x, np.float64)
    gu = x @ w13.T
    g, u = np.split(gu, 2, axis=1)
    return (g / (1.0 + np.exp(-g)) * u) @ w2.T
