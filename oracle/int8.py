"""Rotary positions and the int8 cache in plain numpy: what their calls return,
from the definitions in include/tq.h ("Rotary positions, and the int8 cache's
writer, reader and single-token attention").  Codes and scales are the format's
own fp32 / binary16 arithmetic; rotations, norms and attention are float64."""
from __future__ import annotations

import math

import numpy as np

TOP = np.float32(127 * 65504)


def frequencies(rot_dim, base, kind="plain", factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """-> (radians per position of each pair, magnitude)"""
    if kind == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    j = np.arange(rot_dim // 2)
    f = base ** (-2.0 * j / rot_dim)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "rotations":
        w = np.clip((original_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0, 1)
        return w * f + (1 - w) * f / factor, 1.0
    if kind == "pairs":
        pair = lambda b: rot_dim * math.log(original_len / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = max(min(math.ceil(pair(beta_slow)), rot_dim - 1), lo)
        hi = hi + 0.001 if hi == lo else hi
        w = 1 - np.clip((j - lo) / (hi - lo), 0, 1)
        return w * f + (1 - w) * f / factor, 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    return f, 1.0


def turned(x, positions, freqs, layout="half", magnitude=1.0, norm=None, eps=0.0, inverse=False):
    """Rows x [n][heads][d] normed and rotated, float64 (rows of negative positions: as position 0)."""
    y = np.asarray(x, np.float64)
    if norm is not None:
        with np.errstate(all="ignore"):
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    t = np.maximum(np.asarray(positions, np.float64), 0)[:, None] * np.asarray(freqs)[None] * (-1 if inverse else 1)
    rot = 2 * len(freqs)
    first = np.arange(rot // 2) if layout == "half" else np.arange(0, rot, 2)
    second = first + rot // 2 if layout == "half" else first + 1
    z = (y[..., first] + 1j * y[..., second]) * (magnitude * np.exp(1j * t))[:, None]
    out = y.copy()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def quantise(x):
    """Rows [..., D] (rounded to fp32 first) -> codes int8 [..., D], scales float16 [...]."""
    x = np.asarray(x, np.float32)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), -TOP, TOP)
    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float16)
    sf = s.astype(np.float32)[..., None]
    c = np.clip(np.rint(x / np.where(sf > 0, sf, np.float32(1))), -127, 127)
    return np.where(sf > 0, c, 0).astype(np.int8), s


def values(codes, scales):
    return codes.astype(np.float64) * scales.astype(np.float64)[..., None]


class Cache:
    """Planes of one cache, as in tq_int8."""

    def __init__(self, n_kv_heads, head_dim, n_cells):
        self.n_kv_heads, self.head_dim, self.n_cells = n_kv_heads, head_dim, n_cells
        self.rows = np.zeros((n_cells, n_kv_heads, head_dim), np.int8)
        self.scales = np.zeros((n_cells, n_kv_heads), np.float16)

    def set_rows(self, x, slots):
        c, s = quantise(x)
        for r, slot in enumerate(slots):
            if 0 <= slot < self.n_cells:
                self.rows[slot], self.scales[slot] = c[r], s[r]

    def gather(self, table, length, page_size, head):
        """Values [length][D] of one sequence's cells; a page that is not in the cache as a whole: zeros."""
        t = np.arange(length)
        page = np.asarray(table)[t // page_size].astype(np.int64)
        bad = (page < 0) | (page >= self.n_cells // page_size)
        cell = np.where(bad, 0, page) * page_size + t % page_size
        v = values(self.rows[cell, head], self.scales[cell, head])
        v[bad] = 0.0
        return v


def attention(kc: Cache, vc: Cache, tables, lens, page_size, q, scale, weight_bits):
    """Single-token attention: (out, bound) [n_seq][n_heads][Dv].

    ``bound``: what the library's arithmetic may move a result by before it is rounded.  The products' sums are fp32
    ones of Dk terms, error 2^-22 of the largest sum there could be (four roundings' worth: the order is the tensor
    cores'), which a weight takes as a relative error; the exponent's argument is rounded once more.  Weights carry
    ``weight_bits`` bits, rounded to nearest: 2^-bits relative, and in any case in steps of binary16's smallest number:
    the largest weight p s^V is at least 2^12, so each of them is off by 2^-37 at most against it.  Sums of weights and
    values are fp32, and the tensor cores cut theirs: 2^-13 in all (below 2^11 roundings in a row here)."""
    n, heads, _ = q.shape
    group = heads // vc.n_kv_heads
    out = np.zeros((n, heads, vc.head_dim))
    bound = np.zeros_like(out)
    for s in range(n):
        length = int(lens[s])
        if length == 0:
            continue
        for h in range(heads):
            k = kc.gather(tables[s], length, page_size, h // group)
            v = vc.gather(tables[s], length, page_size, h // group)
            x = scale * (k @ q[s, h])
            p = np.exp(x - x.max())
            p /= p.sum()
            out[s, h] = p @ v
            mag = np.max(np.abs(q[s, h])) * np.max(np.abs(k), initial=0.0)
            err = abs(scale) * 2.0 ** -22 * mag * kc.head_dim + 2.0 ** -23 * (np.max(np.abs(x)) + 1) + 2.0 ** -13
            a = p @ np.abs(v)
            low = length * 2.0 ** -37 * np.max(np.abs(v))
            bound[s, h] = 2.0 ** -weight_bits * a + err * (a + np.abs(out[s, h])) + low
    return out, bound
