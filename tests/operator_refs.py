"""The encoder layer's attention operators in float64, written from their definitions (CPU, NumPy)."""
import math

import numpy as np


def frequencies(dims, theta, scaling="none", factor=1.0, original_length=8192, beta_fast=32.0, beta_slow=1.0):
    """Angle per position of each rotated pair, and the factor of cos and sin."""
    j = np.arange(dims // 2)
    if scaling == "ntk" and dims > 2:
        theta = theta * factor ** (dims / (dims - 2))
    w = theta ** (-2.0 * j / dims)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "yarn":
        def pair(turns):
            return dims * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(theta))
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), dims - 1)
        g = np.clip((j - low) / max(high - low, 1e-3), 0, 1)
        return w * (1 - g) + w / factor * g, 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    return w, 1.0


def norm(x, kind, eps, gain=None):
    """x [..., d] normalised over its last axis."""
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if gain is None else y * gain


def rotate(x, pos, w, amplitude, layout):
    """x [T, H, d] at positions pos [T]; the first 2 len(w) elements of every head turn."""
    a = (pos.astype(np.float64)[:, None] * w)[:, None, :]
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    h, y = len(w), x.copy()
    i, j = (slice(0, h), slice(h, 2 * h)) if layout == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def row_positions(cu, T):
    """Index of each token in its row; -1 past the last row."""
    pos = np.full(T, -1, np.int64)
    for a, b in zip(cu[:-1], cu[1:]):
        pos[a:b] = np.arange(b - a)
    return pos


def diff_lambda(lq1, lk1, lq2, lk2, lambda_init):
    return math.exp(float(lq1 @ lk1)) - math.exp(float(lq2 @ lk2)) + lambda_init


def diff_attention(q, k, v, cu, lam, lambda_init, gain, eps, window, scale=0.125):
    """q [T, 2H, 64], k [T, 2G, 64], v [T, G, 128] -> (out [T, H, 128], (D, rms, sums)): the output, the difference
    before the norm, its root mean square and, per element, sum p0 |v| + |lambda| sum p1 |v| (what errors of the
    probabilities are multiplied by).  Zero past the last row."""
    T, H, G = q.shape[0], q.shape[1] // 2, v.shape[1]
    D, A = np.zeros((T, H, 128)), np.zeros((T, H, 128))
    for a, b in zip(cu[:-1], cu[1:]):
        if b <= a:
            continue
        i = np.arange(b - a)
        hidden = np.abs(i[:, None] - i[None, :]) > window if window >= 0 else None
        for h in range(H):
            g = h // (H // G)
            for x, f in ((0, 1.0), (1, -lam)):
                s = (q[a:b, 2 * h + x] @ k[a:b, 2 * g + x].T) * scale
                if hidden is not None:
                    s = np.where(hidden, -np.inf, s)
                e = np.exp(s - s.max(-1, keepdims=True))
                p = e / e.sum(-1, keepdims=True)
                D[a:b, h] += f * (p @ v[a:b, g])
                A[a:b, h] += abs(f) * (p @ np.abs(v[a:b, g]))
    if gain is None:
        return D, (D, None, A)
    rms = np.sqrt((D * D).mean(-1, keepdims=True) + eps)
    return (1 - lambda_init) * gain * D / rms, (D, rms, A)
