"""FP64 oracle of the operators around a block's products: norms with gate and
residual sum, tokens sorted by expert and brought back, and the gradients of
these.  TEST INFRASTRUCTURE ONLY, in NumPy and plain loops, from the definitions
in ``include/w4_block.h``; it shares no code with the library.

Arrays are float64 values (of what the library holds in BF16 or FP32) and
Python integers.
"""
from __future__ import annotations

import numpy as np


def _f32(x) -> float:
    return float(np.float32(x))


def rms(x, eps):
    return np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + _f32(eps))


def block_norm(h, y=None, y_weight=None, z_weight=None, gate=None, a=1.0, b=1.0, eps=1e-6, add=0.0):
    """(h', z) for h, y [T, D]."""
    x = h
    if y is not None:
        u = y if y_weight is None else y / rms(y, eps) * (y_weight + _f32(add))
        x = _f32(a) * h + _f32(b) * (u if gate is None else gate * u)
    return x, (x if z_weight is None else x / rms(x, eps) * (z_weight + _f32(add)))


def block_norm_grad(h, y=None, dh_out=None, dz=None, y_weight=None, z_weight=None, gate=None, a=1.0, b=1.0, eps=1e-6,
                    add=0.0):
    """dict of dh, dy, d_y_weight, d_z_weight and d_gate (a token's own; sum it for a shared gate)."""
    x, _ = block_norm(h, y, y_weight, z_weight, gate, a, b, eps, add)
    zero = np.zeros_like(x)
    dz = zero if dz is None else dz
    d = zero if dh_out is None else dh_out
    out = {}
    if z_weight is None:
        d = d + dz
    else:
        r = rms(x, eps)
        n = x / r
        g = dz * (z_weight + _f32(add))
        d = d + (g - n * np.mean(g * n, axis=-1, keepdims=True)) / r
        out["d_z_weight"] = (dz * n).sum(axis=0)
    if y is None:
        out["dh"] = d
        return out
    out["dh"] = _f32(a) * d
    d = _f32(b) * d
    n = y if y_weight is None else y / rms(y, eps)
    w = 1.0 if y_weight is None else y_weight + _f32(add)
    if gate is not None:
        out["d_gate"] = d * (n * w)
        d = d * gate
    if y_weight is None:
        out["dy"] = d
        return out
    out["d_y_weight"] = (d * n).sum(axis=0)
    g = d * w
    out["dy"] = (g - n * np.mean(g * n, axis=-1, keepdims=True)) / rms(y, eps)
    return out


def moe_sort(experts, num_experts, capacity=0):
    """(row_start, row_of, source) of experts [T][top]."""
    flat = [int(e) for row in experts for e in row]
    row_start, source = [0], []
    row_of = [-1] * len(flat)
    for e in range(num_experts):
        taken = [i for i, x in enumerate(flat) if x == e]
        if capacity > 0:
            taken = taken[:capacity]
        for i in taken:
            row_of[i] = len(source)
            source.append(i)
        row_start.append(len(source))
    return row_start, np.array(row_of, dtype=np.int64).reshape(np.shape(experts)), source + [-1] * (len(flat) - len(source))


def combine(y, row_of, weights=None, add=None, tokens=None):
    """(out, size) [T, N]: the sum and the sum of its terms' magnitudes."""
    T, top = np.shape(row_of)
    out = np.zeros((T, y.shape[1])) if add is None else add.copy()
    size = np.abs(out)
    for t in range(T):
        for j in range(top):
            if 0 <= row_of[t][j] < len(y):
                term = y[row_of[t][j]] * (1.0 if weights is None else float(weights[t][j]))
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_grad(dout, y, row_of, weights=None):
    """(dy, dweights, size of dweights' terms); rows of dy without a choice are NaN."""
    T, top = np.shape(row_of)
    dy = np.full(y.shape, np.nan)
    dw, size = np.zeros((T, top)), np.zeros((T, top))
    for t in range(T):
        for j in range(top):
            r = row_of[t][j]
            if 0 <= r < len(y):
                dy[r] = dout[t] * (1.0 if weights is None else float(weights[t][j]))
                dw[t, j] = dout[t] @ y[r]
                size[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, size
