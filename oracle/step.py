"""FP64 oracle of the decode step's operators: the 4-bit key/value cache, norm
and rotation, attention, tables and sampling.  TEST INFRASTRUCTURE ONLY, in
NumPy and plain loops, from the definitions in ``include/w4_step.h``; it
shares no code with the library.

Arrays are bit patterns where the library takes BF16 or FP16 (uint16), and
float64 otherwise.
"""
from __future__ import annotations

import math

import numpy as np

from . import bf16_bits, bf16_to_f64

GROUP = 128


def round_to_bf16(x) -> np.ndarray:
    """float64 -> bfloat16 bits the way a kernel does: to float32, then to bfloat16."""
    with np.errstate(over="ignore"):
        return bf16_bits(np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64))


# ------------------------------------------------------------------- cache
def quantise(bits):
    """bfloat16 bits [..., D] -> codes uint8 [..., D], (s, m) float16 [..., groups, 2]."""
    x = bf16_to_f64(bits)
    size = min(x.shape[-1], GROUP)
    x = x.reshape(*x.shape[:-1], -1, size)
    sound = np.isfinite(x).all(axis=-1)
    x = np.clip(np.where(np.isfinite(x), x, 0.0), -65504, 65504).astype(np.float32)
    low, high = x.min(axis=-1), x.max(axis=-1)
    s = ((high - low) * np.float32(1.0 / 15.0)).astype(np.float16)
    m = low.astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(s > 0, np.float32(1) / s.astype(np.float32), np.float32(0)).astype(np.float32)
    q = np.clip(np.rint((x - m.astype(np.float32)[..., None]) * inv[..., None]), 0, 15).astype(np.uint8)
    q[~sound] = 0
    meta = np.stack((np.where(sound, s, np.float16(np.nan)), np.where(sound, m, np.float16(0))), axis=-1)
    return q.reshape(*q.shape[:-2], -1), meta.astype(np.float16)


def dequantise(q, meta):
    """codes [..., D] and (s, m) [..., groups, 2] -> float64 [..., D]."""
    s = np.asarray(meta, dtype=np.float64)
    size = q.shape[-1] // s.shape[-2]
    return q.astype(np.float64) * np.repeat(s[..., 0], size, axis=-1) + np.repeat(s[..., 1], size, axis=-1)


def pack(q) -> np.ndarray:
    """codes [..., D] -> int32 words [..., D / 8], nibble j of word p for d = 8p + j."""
    w = q.reshape(*q.shape[:-1], -1, 8).astype(np.uint64)
    out = np.zeros(w.shape[:-1], dtype=np.uint64)
    for j in range(8):
        out |= w[..., j] << np.uint64(4 * j)
    return out.astype(np.uint32).view(np.int32)


def unpack(words) -> np.ndarray:
    w = np.asarray(words).view(np.uint32)
    return np.stack([(w >> np.uint32(4 * j)) & np.uint32(15) for j in range(8)], axis=-1).reshape(
        *w.shape[:-1], -1).astype(np.uint8)


class Cache:
    """The cache's four arrays on the host, in the library's layout."""

    def __init__(self, num_blocks, block, heads, dim):
        self.blocks, self.block, self.heads, self.dim = num_blocks, block, heads, dim
        g = max(1, dim // GROUP)
        self.k_codes = np.zeros((num_blocks, heads, block, dim // 8), np.int32)
        self.v_codes = np.zeros((num_blocks, heads, block // 4, dim // 8, 4), np.int32)
        self.k_meta = np.zeros((num_blocks, heads, g, block, 2), np.float16)
        self.v_meta = np.zeros_like(self.k_meta)

    def put(self, slot, k_bits, v_bits):
        """One token's keys and values, bfloat16 bits [heads, dim]; a slot outside is ignored."""
        if not 0 <= slot < self.blocks * self.block:
            return
        p, o = divmod(int(slot), self.block)
        q, meta = quantise(k_bits)
        self.k_codes[p, :, o], self.k_meta[p, :, :, o] = pack(q), meta
        q, meta = quantise(v_bits)
        self.v_codes[p, :, o // 4, :, o % 4], self.v_meta[p, :, :, o] = pack(q), meta

    def values(self, slots):
        """(keys, values) float64 [n, heads, dim]."""
        p, o = np.asarray(slots) // self.block, np.asarray(slots) % self.block
        return (dequantise(unpack(self.k_codes[p, :, o]), self.k_meta[p, :, :, o]),
                dequantise(unpack(self.v_codes[p, :, o // 4, :, o % 4]), self.v_meta[p, :, :, o]))


# -------------------------------------------------------- norm and rotation
def norm_rope(bits, weight_bits, cos_sin, positions, rot, interleaved, eps, weight_add):
    """bfloat16 bits [T, heads, D] -> float64 [T, heads, D].  Rows of negative position are NaN here."""
    x = bf16_to_f64(bits)
    if weight_bits is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + float(np.float32(eps))) * (
            bf16_to_f64(weight_bits) + weight_add)
    out = x.copy()
    half = rot // 2
    for t in range(x.shape[0]):
        if not rot:
            continue
        if not 0 <= positions[t] < len(cos_sin):
            out[t] = np.nan
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(cos_sin[positions[t], i]), float(cos_sin[positions[t], half + i])
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


# --------------------------------------------------------------- attention
def visible(pos, kv, window, sinks):
    j = np.arange(max(kv, 0))
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    return see


def attention(q_bits, cache: Cache, table, kv_lens, q_start, scale, window=0, sinks=0, weights=2.0 ** -8):
    """(out, noise) float64 [T, q_heads, D]; rows in no request are NaN.

    ``noise`` bounds the error of a computation that forms scores in FP32 from
    exact products, rounds each weight times its value's scale by ``weights``
    of itself (once to BF16: 2^-8; to two BF16 parts: 2^-16) and sums in FP32: see ``tests/test_gpu_step.py``."""
    T, hq, d = q_bits.shape
    g = hq // cache.heads
    out = np.full((T, hq, d), np.nan)
    noise = np.zeros((T, hq, d))
    q = bf16_to_f64(q_bits)
    size = min(d, GROUP)
    for b in range(len(kv_lens)):
        first, last = int(q_start[b]), int(q_start[b + 1])
        kv = max(int(kv_lens[b]), 0)
        if last <= first:
            continue
        place = np.arange(kv)
        slots = np.asarray(table[b], dtype=np.int64)[place // cache.block] * cache.block + place % cache.block
        p, o = slots // cache.block, slots % cache.block
        with np.errstate(invalid="ignore"):
            keys, values = cache.values(slots) if kv else (np.zeros((0, cache.heads, d)),) * 2
        ks = np.asarray(cache.k_meta[p, :, :, o], dtype=np.float64)  # [kv, heads, groups, 2]
        vs = np.repeat(np.asarray(cache.v_meta[p, :, :, o], dtype=np.float64)[..., 0], size, axis=-1)
        codes = unpack(cache.v_codes[p, :, o // 4, :, o % 4]).astype(np.float64) if kv else np.zeros_like(keys)
        for i in range(first, last):
            see = visible(kv - (last - first) + i - first, kv, window, sinks)
            for h in range(hq):
                if not see.any():
                    out[i, h] = 0.0
                    continue
                k, v = keys[see, h // g], values[see, h // g]
                z = scale * (k @ q[i, h])
                top = z.max()
                with np.errstate(invalid="ignore"):
                    w = np.exp(z - top)
                    w /= w.sum()
                    out[i, h] = w @ v
                # scores: sums of up to 40 terms as large as (136 s + |m|) times the sum of |x|, exp2's argument
                x = np.abs(q[i, h]).reshape(-1, size).sum(axis=-1)
                size_of = (136.0 * ks[see, h // g, :, 0] + np.abs(ks[see, h // g, :, 1])) @ x
                delta = 2.0 ** -24 * (40 * scale * size_of + 4 * np.abs(z) + 4 * abs(top) + 8)
                noise[i, h] = (2 * (w * delta) @ np.abs(v - out[i, h]) + 2 * (w @ delta) * np.abs(w @ (v - out[i, h])) +
                               weights * (w @ np.abs(vs[see, h // g] * (codes[see, h // g] - 8))) +
                               2.0 ** -18 * (w @ np.abs(v)) + 2.0 ** -8 * np.abs(out[i, h]))
    return out, noise


# ------------------------------------------------------------------ tables
def plan(cached, new, table, free, free_count, block, rows):
    """Everything w4_kv4_plan writes, as (q_start, kv_lens, positions, slots, table, counts)."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    left = min(max(int(free_count), 0), len(free))
    given = needed = 0
    q_start, kv, positions, slots = [0], [], [], []
    for b in range(len(cached)):
        c, n = max(int(cached[b]), 0), max(int(new[b]), 0)
        for col in range(min(-(-c // block), width), min(-(-(c + n) // block), width)):
            needed += 1
            if given < left:
                table[b, col] = free[left - 1 - given]
                given += 1
            else:
                table[b, col] = -1
        for pos in range(c, c + n):
            page = table[b, pos // block] if pos // block < width else -1
            positions.append(pos)
            slots.append(page * block + pos % block if page >= 0 else -1)
        q_start.append(q_start[-1] + n)
        kv.append(c + n)
    pad = lambda v: (v + [-1] * rows)[:rows]  # noqa: E731
    return q_start, kv, pad(positions), pad(slots), table, [left - given, needed - given]


# ---------------------------------------------------------------- sampling
def sample(bits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) -> int:
    """One row: bfloat16 bits [vocab] -> token."""
    x = bf16_to_f64(bits)
    x = np.where(np.isnan(x), -np.inf, x) + 0.0  # -0 -> +0
    order = np.argsort(-x, kind="stable")
    top = x[order[0]]
    if top == -np.inf:
        return -1
    if not temperature > 0:
        return int(order[0])
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / float(np.float32(temperature))))
    keep = len(x) if top_k <= 0 else min(top_k, len(x))
    if top_p < 1:
        goal, before, n = float(np.float32(top_p)) * math.fsum(w[:keep]), 0.0, 0
        sums = np.concatenate(([0.0], np.cumsum(w)))
        n = int(np.sum(sums[:keep] < goal))
        keep = max(1, n)
    if min_p > 0:
        keep = min(keep, max(1, int(np.sum(w >= float(np.float32(min_p))))))
    goal = min(u, 1 - 2.0 ** -40) * float(np.cumsum(w)[keep - 1])  # never past the last token with a weight
    at = int(np.sum(np.cumsum(w) <= goal))
    return int(order[min(at, keep - 1)])
