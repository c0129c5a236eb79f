"""The 4-bit paged key/value cache in plain numpy, 64 bits, for the tests.

Written from include/spear_ec_kv.h alone: quantization of one vector, the
cache's byte layout, and attention by its definition, one row and head at a
time.  bf16 arrays are uint16 bits; fp16 scales uint16 bits.

Tolerances of an attention output are counted from the header's arithmetic,
with u = 2^-24 half a step of fp32 and p_j = exp(S_j - m) / l:
  * a score is a sum of D products of q with codes up to 15 in magnitude, less
    z times the sum of q, accumulated in fp32 in any order, then a few
    products: |dS| <= (D + 16) u * scale * s_j * 30 * sum|q|.  A relative error
    of p_j is at most twice the largest dS, plus exp's and its argument's
    rounding, under 2^-18;
  * p_j s_j, or p_j and v_j apart, are rounded to fp16, half a step: 2^-11 of
    themselves each.  Below fp16's normal range half a step is 2^-25 of what 1
    stands for: of a value, 2^-25 of the largest scale of its 16 tokens; of a
    p_j s_j, 2^-25 of the row's largest p times its largest s;
  * O's sum runs over products with codes up to 15 and zero-points up to 15,
    in fp32: relative to sum p_j s_j 30, (n/16 + 64) u;
  * the output is rounded once to bf16: half a step, at most 2^-8 relative.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def bf16_to_f64(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(a):
    """Finite values, nearest even in one step."""
    a = np.asarray(a, np.float64)
    _, e = np.frexp(np.abs(a))
    quantum = np.ldexp(1.0, np.maximum(e - 1, -126) - 7)
    r = np.copysign(np.rint(np.abs(a) / quantum) * quantum, a).astype(np.float32)
    return (r.view(np.uint32) >> 16).astype(np.uint16)


def half_step_bf16(a):
    _, e = np.frexp(np.abs(np.asarray(a, np.float64)))
    return np.ldexp(1.0, np.maximum(e - 1, -126) - 8)


def quantize(x, asym):
    """One vector -> (codes, scale bits, zero-point)."""
    lo, hi = min(0.0, float(np.min(x))), max(0.0, float(np.max(x)))
    with np.errstate(over="ignore"):
        s = np.float16((hi - lo) / 15.0 if asym else max(hi, -lo) / 7.0)
    if np.isinf(s):
        s = np.float16(65504.0)
    if s == 0:
        s = np.float16(1.0)
    d = float(s)
    if asym:
        z = int(min(15.0, max(0.0, np.rint(-lo / d))))
        c = np.clip(np.rint(x / d) + z, 0, 15)
    else:
        z = 8
        c = np.clip(np.rint(x / d), -8, 7) + 8
    return c.astype(np.uint8), s.view(np.uint16), z


def rotate(x, pos, cos_sin, dim, interleaved):
    """x [..., D] at position pos."""
    if cos_sin is None:
        return x
    y = np.array(x, np.float64)
    c, s = cos_sin[pos, :dim // 2].astype(np.float64), cos_sin[pos, dim // 2:dim].astype(np.float64)
    i = np.arange(dim // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class Cache:
    """Host copy of a cache: codes, scales (bits) and zeros arrays of the header's layout."""

    def __init__(self, kv_heads, D, page, pages, asym, fill=0):
        nb = page // 16
        self.G, self.D, self.page, self.pages, self.asym = kv_heads, D, page, pages, asym
        self.codes = np.full((pages, kv_heads, nb, 16 * D), fill, np.uint8)
        # slots never written may hold anything: NaN scales show a read of them
        self.scales = np.full((pages, kv_heads, nb, 2, 16), 0x7E00 if fill else 0, np.uint16)
        self.zeros = np.full((pages, kv_heads, nb, 16), fill, np.uint8) if asym else None

    def _at(self, table_row, pos):
        return int(table_row[pos // self.page]), pos % self.page // 16, pos % 16

    def put(self, table_row, pos, head, which, codes, scale, z):
        pg, blk, j = self._at(table_row, pos)
        D = self.D
        packed = codes[0::2] | (codes[1::2] << 4)
        if which == 0:
            self.codes[pg, head, blk, j * (D // 2):(j + 1) * (D // 2)] = packed
        else:
            self.codes[pg, head, blk, 8 * D + j::16] = packed
        self.scales[pg, head, blk, which, j] = scale
        if self.asym:
            old = int(self.zeros[pg, head, blk, j])
            self.zeros[pg, head, blk, j] = (old & 0xF0) | z if which == 0 else (old & 15) | (z << 4)

    def parts(self, table_row, n, head, which, first=0):
        """(codes - z, s) of tokens first .. n."""
        t = np.arange(first, n)
        pg = np.asarray(table_row)[t // self.page]
        blk, j = t % self.page // 16, t % 16
        rows = self.codes[pg, head, blk]
        D = self.D
        if which == 0:
            b = np.take_along_axis(rows, j[:, None] * (D // 2) + np.arange(D // 2), 1)
        else:
            b = np.take_along_axis(rows, 8 * D + 16 * np.arange(D // 2) + j[:, None], 1)
        c = np.stack([b & 15, b >> 4], -1).reshape(len(t), D).astype(np.float64)
        z = 8.0
        if self.asym:
            z = (self.zeros[pg, head, blk, j] >> (4 * which)) & 15
            z = z.astype(np.float64)[:, None]
        s = self.scales[pg, head, blk, which, j].view(np.float16).astype(np.float64)
        return c - z, s


def append(cache, q, k, v, offsets, lens, table, cos_sin=None, dim=0, interleaved=False):
    """Stores k, v in `cache`; returns q rotated (float64)."""
    q = bf16_to_f64(q)
    out = np.array(q)
    k, v = bf16_to_f64(k), bf16_to_f64(v)
    for b in range(len(lens)):
        n = offsets[b + 1] - offsets[b]
        for i in range(n):
            t, pos = offsets[b] + i, lens[b] - n + i
            if pos < 0:
                out[t] = 0
                continue
            out[t] = rotate(q[t], pos, cos_sin, dim, interleaved)
            kr = rotate(k[t], pos, cos_sin, dim, interleaved)
            for h in range(cache.G):
                cache.put(table[b], pos, h, 0, *quantize(kr[h], cache.asym))
                cache.put(table[b], pos, h, 1, *quantize(v[t, h], cache.asym))
    return out


def attention(cache, q, offsets, lens, table, scale, window=0):
    """(out, lse, tolerance of out, tolerance of lse) in float64."""
    q = bf16_to_f64(q)
    T, H, D = q.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol, ltol = np.zeros((T, H, D)), np.zeros((T, H))
    R = H // cache.G
    for b in range(len(lens)):
        n = offsets[b + 1] - offsets[b]
        if n == 0 or lens[b] <= 0:
            continue
        for g in range(cache.G):
            kc, ks = cache.parts(table[b], lens[b], g, 0)
            vc, vs = cache.parts(table[b], lens[b], g, 1)
            for i in range(n):
                t, pos = offsets[b] + i, lens[b] - n + i
                if pos < 0:
                    continue
                lo = max(0, pos - window + 1) if window else 0
                sl = slice(lo, pos + 1)
                m_keys = pos + 1 - lo
                for h in range(g * R, (g + 1) * R):
                    S = (kc[sl] @ q[t, h]) * ks[sl] * scale
                    m = S.max()
                    e = np.exp(S - m)
                    l = e.sum()
                    p = e / l
                    out[t, h] = (p * vs[sl]) @ vc[sl]
                    lse[t, h] = m + np.log(l)
                    dS = scale * ks[sl].max() * (D + 16) * U * 30 * np.abs(q[t, h]).sum()
                    pv = p * vs[sl]
                    tol[t, h] = ((2 * dS + 2.0 ** -10 + 2.0 ** -18) * (pv @ np.abs(vc[sl]))
                                 + 2.0 ** -25 * (p.max() * vs[sl].max() * 15 * m_keys + vs[sl].max())
                                 + (m_keys / 16 + 64) * U * 30 * pv.sum())
                    tol[t, h] += half_step_bf16(np.abs(out[t, h]) + tol[t, h])
                    ltol[t, h] = dS + 2.0 ** -20 * (1 + abs(lse[t, h]))
    return out, lse, tol, ltol
