"""fp64 oracle of the 8-bit key/value cache: numpy, one row and one block at a
time, written from the definitions (codes, power-of-two scales, outward
bounds, softmax, whole-number block scores).

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64
E4M3, INT8 = 0, 1
LARGEST = {E4M3: 448.0, INT8: 127.0}


def e4m3_value(byte: int) -> float:
    sign, e, f = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and f == 7:
        return math.nan
    v = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
    return -v if sign else v


_E4M3 = np.array([e4m3_value(b) for b in range(256)])
_POSITIVE = _E4M3[:127]


def values(codes, fmt):
    """Code bytes (uint8) as float64."""
    return _E4M3[codes] if fmt == E4M3 else codes.view(np.int8).astype(np.float64)


def v_order():
    """Byte of token t inside a channel's 64 bytes of V."""
    out = np.empty(BLOCK, np.int64)
    for t in range(BLOCK):
        j, h, c, e = t // 16, t // 8 % 2, t // 2 % 4, t % 2
        out[t] = 16 * c + 4 * j + 2 * h + e
    return out


def round_code(x, fmt):
    """Nearest code value, ties to even."""
    x = np.asarray(x, np.float64)
    if fmt == INT8:
        return np.rint(x)
    a = np.abs(x)
    i = np.searchsorted(_POSITIVE, a, side="right") - 1  # the code at or below
    lo, hi = _POSITIVE[i], _POSITIVE[np.minimum(i + 1, 126)]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    return np.copysign(np.where(up, hi, lo), x)


def scale_of(amax: float, fmt) -> float:
    """The smallest power of two, 2^-126 at least, with amax <= M times it."""
    s = 2.0 ** -126
    while amax > LARGEST[fmt] * s:
        s *= 2
    return s


class Cache:
    """k, v [pages][hkv][64][d] code values, scales [pages][hkv][2], bounds [pages][hkv][2][d]."""

    def __init__(self, pages, hkv, d, fmt):
        self.fmt, self.hkv, self.d = fmt, hkv, d
        self.k, self.v = np.zeros((pages, hkv, BLOCK, d)), np.zeros((pages, hkv, BLOCK, d))
        self.scales, self.bounds = np.zeros((pages, hkv, 2)), np.zeros((pages, hkv, 2, d))

    @classmethod
    def of(cls, k, v, scales, bounds, fmt):
        """From the library's arrays (uint8 codes, V in its order)."""
        c = cls(k.shape[0], k.shape[1], k.shape[3], fmt)
        c.k, c.v = values(k, fmt), values(v, fmt)[..., v_order()].swapaxes(2, 3)
        c.scales, c.bounds = scales.astype(np.float64), bounds.astype(np.float64)
        return c

    def append(self, table, lens, k, v, cu):
        """k, v float64 [rows][hkv][d]."""
        for i, length in enumerate(lens):
            n = cu[i + 1] - cu[i]
            for b in range(0, (length + BLOCK - 1) // BLOCK):
                rows = [(p, cu[i] + p - (length - n)) for p in range(b * BLOCK, min(length, b * BLOCK + BLOCK))
                        if p >= length - n]
                if not rows:
                    continue
                page = table[i][b]
                fresh = rows[0][0] == b * BLOCK
                inside = [p - b * BLOCK for p, _ in rows]
                for h in range(self.hkv):
                    for w, (codes, x) in enumerate(((self.k, k), (self.v, v))):
                        new = x[[r for _, r in rows], h]
                        if fresh:
                            codes[page, h] = 0
                        old = 0.0 if fresh else self.scales[page, h, w]
                        if not np.isfinite(new).all() or math.isnan(old):
                            self.scales[page, h, w] = math.nan
                            continue
                        s = max(scale_of(np.abs(new).max(), self.fmt), old)
                        if s != old and not fresh:
                            codes[page, h] = round_code(codes[page, h] * (old / s), self.fmt)
                        codes[page, h, inside] = round_code(new / s, self.fmt)
                        if w == 0:
                            unit = s if self.fmt == INT8 else 4 * s
                            lo, hi = np.floor(new.min(0) / unit), np.ceil(new.max(0) / unit)
                            if not fresh:
                                lo = np.minimum(lo, np.floor(self.bounds[page, h, 0] * (old / s)))
                                hi = np.maximum(hi, np.ceil(self.bounds[page, h, 1] * (old / s)))
                            self.bounds[page, h] = lo, hi
                        self.scales[page, h, w] = s

    def sequence(self, row, length):
        """Dequantised (k, v) [length][hkv][d] of a sequence."""
        pages = list(row[:(length + BLOCK - 1) // BLOCK])
        out = []
        for w, codes in enumerate((self.k, self.v)):
            x = codes[pages] * self.scales[pages][:, :, w, None, None]
            out.append(x.transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.d)[:length])
        return out

    def attention(self, table, lens, q, cu, scale, blocks=None):
        """q float64 [rows][hq][d] -> o, lse [hq][rows], and what their error bounds need: a = sum p |v| of each
        output, x = the largest sum |q k| scale of a row's keys, and z = max(p s) sum |code| over the keys with
        p s < 2^-13 max(p s), s the V scale of the key's block."""
        rows, hq, d = q.shape
        g = hq // self.hkv
        o, a, z = (np.zeros((rows, hq, d)) for _ in range(3))
        lse, x = np.full((hq, rows), -np.inf), np.zeros((hq, rows))
        for i, length in enumerate(lens):
            if length <= 0:
                continue
            k, v = self.sequence(table[i], length)
            for t in range(cu[i], cu[i + 1]):
                pos = length - (cu[i + 1] - t)
                if pos < 0:
                    continue
                for h in range(self.hkv):
                    keys = np.arange(pos + 1)
                    if blocks is not None:
                        keys, last = [], -1
                        chosen = [int(b) for b in blocks[t, h]]
                        for j, b in enumerate(chosen):
                            if b > (chosen[j - 1] if j else -1) and 0 <= b * BLOCK <= pos:
                                keys += range(b * BLOCK, min(pos + 1, b * BLOCK + BLOCK))
                        keys = np.array(keys, np.int64)
                    if not len(keys):
                        continue
                    s = q[t, h * g:(h + 1) * g] @ k[keys, h].T * scale
                    top = s.max(1, keepdims=True)
                    p = np.exp(s - top)
                    total = p.sum(1, keepdims=True)
                    lse[h * g:(h + 1) * g, t] = (top + np.log(total))[:, 0]
                    o[t, h * g:(h + 1) * g] = p / total @ v[keys, h]
                    a[t, h * g:(h + 1) * g] = p / total @ np.abs(v[keys, h])
                    sv = self.scales[np.asarray(table[i])[keys // BLOCK], h, 1]
                    ps = p / total * sv
                    with np.errstate(invalid="ignore"):
                        low = ps < 2.0 ** -13 * ps.max(1, keepdims=True)
                        z[t, h * g:(h + 1) * g] = ps.max(1, keepdims=True) * (low @ (np.abs(v[keys, h]) / sv[:, None]))
                    x[h * g:(h + 1) * g, t] = (np.abs(q[t, h * g:(h + 1) * g]) @ np.abs(k[keys, h]).T * scale).max(1)
        return o, lse, a, x, z

    def select(self, table, lens, q, cu, count, keep_first, keep_last, max_pages=None):
        rows, hq, d = q.shape
        g = hq // self.hkv
        out = np.full((rows, self.hkv, count), -1, np.int64)
        for i, length in enumerate(lens):
            for t in range(cu[i], cu[i + 1]):
                pos = length - (cu[i + 1] - t)
                have = pos // BLOCK + 1 if pos >= 0 else 0
                for h in range(self.hkv):
                    x = np.where(np.isfinite(q[t, h * g:(h + 1) * g]), q[t, h * g:(h + 1) * g], 0.0)
                    c = np.rint(x / scale_of(np.abs(x).max(), INT8)).astype(np.int64)
                    up, down = np.maximum(c, 0).sum(0), np.minimum(c, 0).sum(0)
                    pages = list(table[i][:have])
                    u = (self.bounds[pages, h, 1].astype(np.int64) @ up + self.bounds[pages, h, 0].astype(np.int64) @ down)
                    score = u.astype(np.float32) * self.scales[pages, h, 0].astype(np.float32)
                    rank = [(not (b < keep_first or b >= have - keep_last), not np.isnan(score[b]),
                             -score[b] if not np.isnan(score[b]) else 0, b) for b in range(have)]
                    chosen = sorted(r[3] for r in sorted(rank)[:count])
                    out[t, h, :len(chosen)] = chosen
        return out
