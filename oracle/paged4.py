"""The paged 4-bit cache in plain numpy: what its calls return, from their
definitions (include/tq.h, "Paged 4-bit cache").  Codes and scales are the
format's own fp32 / binary16 arithmetic; attention is float64."""
from __future__ import annotations

import numpy as np


def width(head_dim: int) -> int:
    return 64 if head_dim <= 64 else 128 if head_dim <= 128 else 256


def quantise(x: np.ndarray):
    """Rows [..., D] -> codes uint8 [..., D], scale and offset float16 [...]."""
    x = np.asarray(x, np.float32)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), np.float32(-65504), np.float32(65504))
    lo, hi = x.min(-1), x.max(-1)
    m = lo.astype(np.float16)
    s = ((hi - lo) / np.float32(15)).astype(np.float16)
    sf, mf = s.astype(np.float32)[..., None], m.astype(np.float32)[..., None]
    c = np.rint((x - mf) / np.where(sf > 0, sf, np.float32(1)))
    return np.where(sf > 0, np.clip(c, 0, 15), 0).astype(np.uint8), s, m


def pack(codes: np.ndarray) -> np.ndarray:
    """Codes [..., D] -> bytes [..., width(D) / 2], zero codes beyond D."""
    d = codes.shape[-1]
    full = np.zeros((*codes.shape[:-1], width(d)), np.uint8)
    full[..., :d] = codes
    return full[..., 0::2] | full[..., 1::2] << 4


def unpack(packed: np.ndarray, head_dim: int) -> np.ndarray:
    c = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), np.uint8)
    c[..., 0::2] = packed & 15
    c[..., 1::2] = packed >> 4
    return c[..., :head_dim]


def values(codes, scale, offset) -> np.ndarray:
    """scale * code + offset in float64."""
    return (codes.astype(np.float64) * scale.astype(np.float64)[..., None]
            + offset.astype(np.float64)[..., None])


class Cache:
    """Planes of one cache, as in tq_paged4."""

    def __init__(self, n_kv_heads, head_dim, page_size, n_pages):
        self.n_kv_heads, self.head_dim, self.page_size, self.n_pages = n_kv_heads, head_dim, page_size, n_pages
        self.codes = np.zeros((n_pages, n_kv_heads, page_size, width(head_dim) // 2), np.uint8)
        self.scales = np.zeros((n_pages, n_kv_heads, page_size, 2), np.float16)

    def set_rows(self, x, slots):
        c, s, m = quantise(x)
        p = pack(c)
        for r, slot in enumerate(slots):
            if 0 <= slot < self.n_pages * self.page_size:
                page, at = divmod(int(slot), self.page_size)
                self.codes[page, :, at] = p[r]
                self.scales[page, :, at, 0] = s[r]
                self.scales[page, :, at, 1] = m[r]

    def rows(self, table, length, head):
        """(scale * code + offset, scale * code) [length][D] of one sequence's cells; a page id outside the
        cache reads as zero rows."""
        cells = np.arange(length)
        page = np.asarray(table)[cells // self.page_size].astype(np.int64)
        bad = (page < 0) | (page >= self.n_pages)
        page = np.where(bad, 0, page)
        at = cells % self.page_size
        c = unpack(self.codes[page, head, at], self.head_dim).astype(np.float64)
        sm = self.scales[page, head, at].astype(np.float64)
        sc = c * sm[:, :1]
        v = sc + sm[:, 1:]
        v[bad] = 0.0
        sc[bad] = 0.0
        return v, sc


def softmax_map(q, k, v, sc, ends, scale, score_error=0.0):
    """One map: rows q [n][Dk] over keys < ends[i] -> (out, bound).  ``bound`` is what a rounding of every weight
    p_t s_t by 2^-11 and of every p_t by 2^-13 can move the output by, with weights below 2^-14 of the largest
    rounded in steps of 2^-24 (the library's binary16 weights), plus relative weight errors of ``score_error``."""
    out = np.zeros((q.shape[0], v.shape[1]))
    bound = np.zeros_like(out)
    step = (np.max(np.abs(sc), initial=0.0)) * 2.0 ** -24
    for i in range(q.shape[0]):
        n = max(0, min(int(ends[i]), k.shape[0]))
        if n == 0:
            continue
        x = scale * (k[:n] @ q[i])
        p = np.exp(x - x.max())
        p /= p.sum()
        out[i] = p @ v[:n]
        a = p @ np.abs(v[:n])
        bound[i] = 2.0 ** -11 * (p @ sc[:n]) + (2.0 ** -13 + score_error) * (a + np.abs(out[i]) + p @ sc[:n]) + n * step
    return out, bound


def rms_limit(kc: Cache, vc: Cache, table, length, q, n_heads, scale, dtype, causal=True, lam=None):
    """-> (exact output [rows][n_heads][Dv] of one sequence's last rows, rms that its error stays below).

    The prompt kernel rounds every weight and every value to binary16 and the output to ``dtype``.  A rounding of half a
    step h moves a number x by at most h |x|, evenly spread, so by h |x| / sqrt(3) rms; the terms' errors are
    independent, and a term p v carries two: 2 (h p v)^2 / 3 each, added to the square of what rounding the exact output
    itself leaves."""
    maps, group = (1, n_heads // vc.n_kv_heads) if lam is None else (2, n_heads // vc.n_kv_heads)
    n, h = q.shape[0], 2.0 ** -11
    out = np.zeros((n, n_heads, vc.head_dim))
    var = np.zeros_like(out)
    ends = length - n + 1 + np.arange(n) if causal else np.full(n, length)
    for head in range(n_heads):
        hv = head // group
        v = vc.rows(table, length, hv)[0]
        for m in range(maps):
            x = scale * q[:, maps * head + m] @ kc.rows(table, length, maps * hv + m)[0].T
            x[np.arange(length)[None] >= ends[:, None]] = -np.inf
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            f = 1.0 if m == 0 else -lam[head]
            out[:, head] += f * (p @ v)
            var[:, head] += 2 * h * h / 3 * f * f * ((p * p) @ (v * v))
    own = round_to(out, dtype) - out
    return out, float(np.sqrt(np.mean(own * own) + np.mean(var)))


def round_to(x, dtype):
    """float64 values rounded to binary16 or bfloat16 (ties to even), normal numbers."""
    if dtype == "float16":
        return x.astype(np.float16).astype(np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def attention(kc: Cache, vc: Cache, tables, lens, q, q_start, n_heads, scale, causal=True, lam=None,
              norm_weight=None, eps=0.0, out_scale=1.0):
    """Every attention call: (out, bound) [rows][n_heads][Dv]; rows outside q_start stay NaN.  lam: differential."""
    maps = 1 if lam is None else 2
    group = n_heads // vc.n_kv_heads
    q = np.asarray(q, np.float64)
    out = np.full((q.shape[0], n_heads, vc.head_dim), np.nan)
    bound = np.zeros_like(out)
    for s, length in enumerate(lens):
        r0, r1 = int(q_start[s]), int(q_start[s + 1])
        if r0 == r1:
            continue
        ends = length - (r1 - r0) + np.arange(r1 - r0) + 1 if causal else np.full(r1 - r0, length)
        for hv in range(vc.n_kv_heads):
            v, sc = vc.rows(tables[s], length, hv)
            ks = [kc.rows(tables[s], length, maps * hv + m)[0] for m in range(maps)]
            for h in range(hv * group, (hv + 1) * group):
                got = []
                for m in range(maps):
                    qm = q[r0:r1, maps * h + m]
                    # fp32 accumulation of Dk products: relative 2^-24 each, against the largest possible sum
                    mag = np.max(np.abs(qm), initial=0.0) * np.max(np.abs(ks[m]), initial=0.0)
                    err = 2.0 ** -22 * abs(scale) * mag * kc.head_dim
                    got.append(softmax_map(qm, ks[m], v, sc, ends, scale, err))
                o, b = got[0]
                if lam is not None:
                    o, b = o - lam[h] * got[1][0], b + abs(lam[h]) * got[1][1] + 2.0 ** -22 * np.abs(o)
                    if norm_weight is not None:
                        r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
                        b = r * (b + np.abs(o) * r * r * (np.abs(o) * b).mean(-1, keepdims=True)) + 2.0 ** -20 * np.abs(o) * r
                        o, b = o * r * norm_weight, b * np.abs(norm_weight)
                    o, b = o * out_scale, b * abs(out_scale)
                out[r0:r1, h], bound[r0:r1, h] = o, b
    return out, bound


def page_plan(seq_len, n_new, page_size, block_table, free_pages, free_count, n_rows):
    """-> (ok, block_table, free_pages, free_count, seq_len, q_start, page_start, slots, positions), one by one."""
    table, free = np.array(block_table), np.array(free_pages)
    n, cap = len(seq_len), table.shape[1] * page_size
    pages = lambda c: -(-int(c) // page_size)  # noqa: E731
    old, new = [int(x) for x in seq_len], [int(x) for x in n_new]
    after = [a + b for a, b in zip(old, new)]
    ok = all(0 <= a <= cap and 0 <= b <= cap for a, b in zip(old, after))
    back = sum(max(0, pages(a) - pages(b)) for a, b in zip(old, after)) if ok else 0
    more = sum(max(0, pages(b) - pages(a)) for a, b in zip(old, after)) if ok else 0
    count = int(free_count)
    ok = ok and count >= 0 and count + back <= len(free) and count + back - more >= 0
    ok = ok and sum(max(0, b) for b in new) <= n_rows
    slots, positions = np.full(n_rows, -1, np.int64), np.full(n_rows, -1, np.int32)
    q_start, page_start = np.zeros(n + 1, np.int32), np.zeros(n + 1, np.int32)
    if not ok:
        return False, table, free, count, np.array(old, np.int32), q_start, page_start, slots, positions
    for s in range(n):
        for j in range(pages(after[s]), pages(old[s])):
            free[count] = table[s, j]
            count += 1
    r = 0
    for s in range(n):
        page_start[s + 1] = page_start[s]
        for j in range(pages(old[s]), pages(after[s])):
            count -= 1
            table[s, j] = free[count]
            page_start[s + 1] += 1
        for pos in range(old[s], after[s]):
            slots[r] = int(table[s, pos // page_size]) * page_size + pos % page_size
            positions[r] = pos
            r += 1
        q_start[s + 1] = r
    return True, table, free, count, np.array(after, np.int32), q_start, page_start, slots, positions
