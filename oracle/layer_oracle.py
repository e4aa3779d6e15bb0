"""The steps around the SSD in a Mamba-2 layer in float64 NumPy, from their
definitions: causal convolution with SiLU and softplus, residual and gated
RMSNorm with 8-bit rows, the 8-bit product. Independent of the HIP code.
"""
from __future__ import annotations

import numpy as np


def rhaz(v):
    """Round half away from zero."""
    v = np.asarray(v, np.float64)
    return np.trunc(v + np.copysign(0.5, v))


def silu(u):
    u = np.asarray(u, np.float64)
    with np.errstate(over="ignore"):
        return u / (1.0 + np.exp(-u))


def softplus(v):
    return np.logaddexp(0.0, np.asarray(v, np.float64))


def conv_history(ring, pos, width):
    """The width - 1 inputs before position pos[b] of each sequence, oldest first
    ([B, width - 1, Cd]; zeros before a sequence's start)."""
    B, cd = len(pos), ring.shape[-1]
    out = np.zeros((B, width - 1, cd))
    for b in range(B):
        for j in range(width - 1):
            p = int(pos[b]) - (width - 1) + j
            if p >= 0:
                out[b, j] = ring[b, p % width]
    return out


def conv(xbc, weight, bias, history):
    """u [B, L, Cd] and sum |w x| + |b| (for rounding bounds): xbc [B, L, Cd],
    weight [Cd, W], bias [Cd], history [B, W - 1, Cd]."""
    W, L = weight.shape[1], xbc.shape[1]
    full = np.concatenate([history, xbc], 1)
    u = np.zeros(xbc.shape) + bias
    mag = np.zeros(xbc.shape) + np.abs(bias)
    for j in range(W):
        u += full[:, j:j + L] * weight[:, j]
        mag += np.abs(full[:, j:j + L] * weight[:, j])
    return u, mag


def ring_after(ring, xbc, pos, ends, width):
    """The ring [B, width, Cd] after the inputs of positions pos[b] .. pos[b] + ends[b] - 1."""
    out = ring.copy()
    for b in range(xbc.shape[0]):
        for t in range(max(0, int(ends[b]) - width), int(ends[b])):
            out[b, (int(pos[b]) + t) % width] = xbc[b, t]
    return out


def rms_rows(r, groups, weight, eps):
    """r / sqrt(mean(r^2) + eps) * weight, the mean over each of `groups` runs of a row."""
    g = r.reshape(r.shape[0], groups, -1)
    n = g / np.sqrt(np.mean(g * g, axis=-1, keepdims=True) + eps)
    return n.reshape(r.shape) * weight


def row_codes(y):
    """(codes, steps) of rows: step = max|y| / 127 (1 for a row of zeros)."""
    step = np.abs(y).max(axis=-1) / 127.0
    step = np.where(step > 0, step, 1.0)
    return np.clip(rhaz(y / step[:, None]), -127, 127), step


def matmul_i8(a, a_step, w, w_step, bias):
    """a_step w_step (a @ w.T) + bias; the sums are whole numbers, exact in float64."""
    y = a.astype(np.float64) @ w.astype(np.float64).T
    return y * a_step[:, None] * w_step + bias
