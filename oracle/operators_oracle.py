"""The operators that stand beside the SSD in a layer in float64 NumPy, from their
definitions: the gated delta rule. Independent of the HIP code.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    v = np.asarray(v, np.float64)
    t = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, t) / (1.0 + t)


def unit(v, eps):
    """v / sqrt(sum v^2 + eps) over the last axis; zeros stay zeros."""
    n = np.sqrt((v * v).sum(-1, keepdims=True) + eps)
    return np.divide(v, n, out=np.zeros_like(v), where=n > 0)


def delta(x, dt, A, k, q, beta, scale, state):
    """The gated delta rule, one position after the other: x [B, L, H, P], dt, beta
    [B, L, H], A [H], k, q [B, L, G, N], state [B, H, P, N]. Returns y, the state after,
    and both with every term taken by its magnitude (for rounding bounds)."""
    B, L, H, P = x.shape
    r = H // k.shape[2]
    k, q = np.repeat(k, r, 2), np.repeat(q, r, 2)
    s, mag = state.copy(), np.abs(state)
    y, ymag = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(L):
        a = np.exp(dt[:, t] * A)[..., None, None]
        s *= a
        mag *= a
        sk = np.matmul(s, k[:, t, :, :, None])[..., 0]
        mk = np.matmul(mag, np.abs(k[:, t, :, :, None]))[..., 0]
        b = beta[:, t, :, None]
        s += (b * (x[:, t] - sk))[..., None] * k[:, t, :, None, :]
        mag += np.minimum(np.abs(b) * (np.abs(x[:, t]) + mk), 1e300)[..., None] * np.abs(k[:, t, :, None, :])
        # a write replaces what the key held: the magnitude of what a stable rule keeps
        mag = np.minimum(mag, np.abs(s) + np.sqrt((s * s).sum(-1, keepdims=True)) + np.abs(x[:, t])[..., None])
        y[:, t] = scale * np.matmul(s, q[:, t, :, :, None])[..., 0]
        ymag[:, t] = abs(scale) * np.matmul(mag, np.abs(q[:, t, :, :, None]))[..., 0]
    return y, s, ymag, mag


def activation(v, act):
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "relu2":
        return np.maximum(v, 0.0) ** 2
    if act == "silu":
        return v * sigmoid(v)
    if act == "sigmoid":
        return sigmoid(v)
    if act == "gelu":
        from scipy.special import ndtr
        return v * ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)))
    return np.asarray(v, np.float64)


def rms(v, eps):
    """1 / sqrt(mean(v^2) + eps) of rows, 0 where that is infinite."""
    m = (v * v).mean(-1, keepdims=True) + eps
    return np.where(m > 0, 1.0 / np.sqrt(np.where(m > 0, m, 1.0)), 0.0)


def block_norm(x, post, gate, res, res_scale, weight, eps):
    """r and y of a block's norms: x [rows, cols], gate and res [rows, cols] (1, 0 for none)."""
    r = x * rms(x, eps) * post * gate + res_scale * res
    return r, r * rms(r, eps) * weight
