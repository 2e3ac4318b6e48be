"""fp64 oracle of the 4-bit key/value cache: numpy, one row at a time, written from the definitions (e2m1 codes,
power-of-two scales, places of codes and scales, softmax).

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
SIZES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([SIZES, -SIZES])


def round_code(x):
    """Code of the nearest value, ties to the even code, with the sign of x (of zeros too); x within [-6, 6]."""
    x = np.asarray(x, np.float64)
    far = np.abs(np.abs(x)[..., None] - SIZES)
    best = far.min(-1, keepdims=True)
    tied = far == best
    even = tied & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tied.argmax(-1))
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def scale_byte(amax: float) -> int:
    """Exponent plus 127 of the smallest power of two, 2^-126 at least, with amax <= 6 times it; 255 if it is no number."""
    if not np.isfinite(amax):
        return 255
    e = -126
    while amax > 6 * 2.0 ** e:
        e += 1
    return e + 127


def scale_value(byte):
    return np.where(np.asarray(byte) == 255, np.nan, 2.0 ** (np.asarray(byte, np.float64) - 127))


def k_place(ch: int, d: int):
    """(byte of a token's row, half) of a channel."""
    g, c, b, e = ch // 32, ch % 32 // 8, ch % 8 // 2, ch % 2
    return d // 8 * c + 4 * g + b, e


def v_place(token: int, ch: int):
    """(row, byte, half) of a token's channel."""
    i, h, r = ch // 16, ch % 16 // 8, ch % 8
    s, p, c, e = token // 16, token % 16 // 8, token % 8 // 2, token % 2
    return i, 64 * r + 16 * c + 8 * h + 2 * s + p, e


def scale_place(token: int) -> int:
    return 8 * (token % 8) + token // 8


class Cache:
    """The library's three arrays, read and written code by code."""

    def __init__(self, k, v, scales):
        self.k, self.v, self.scales = k.copy(), v.copy(), scales.copy()
        self.hkv, self.d = k.shape[1], 2 * k.shape[3]

    def _row(self, page, head, token, which):
        """A row's codes and scale bytes."""
        d = self.d
        out = np.empty(d, np.uint8)
        for ch in range(d):
            if which == "k":
                byte, e = k_place(ch, d)
                x = self.k[page, head, token, byte]
            else:
                i, byte, e = v_place(token, ch)
                x = self.v[page, head, i, byte]
            out[ch] = x >> 4 if e else x & 15
        s = self.scales[page, head, :, scale_place(token)]
        return out, (np.repeat(s[:-1], 32) if which == "k" else np.repeat(s[-1:], d))

    def _write(self, page, head, token, which, x):
        d = self.d
        step = 32 if which == "k" else d
        for a in range(0, d, step):
            byte = scale_byte(np.abs(x[a:a + step]).max())
            most = 3.0 if byte == 253 else 6.0  # 4 * 2^126 is past the end of bf16 and fp32
            code = np.zeros(step, np.uint8) if byte == 255 else round_code(np.clip(x[a:a + step] / scale_value(byte), -most, most))
            self.scales[page, head, a // 32 if which == "k" else d // 32, scale_place(token)] = byte
            for ch in range(a, a + step):
                if which == "k":
                    at, e = k_place(ch, d)
                    where = self.k[page, head, token]
                else:
                    i, at, e = v_place(token, ch)
                    where = self.v[page, head, i]
                where[at] = where[at] & (0x0f if e else 0xf0) | int(code[ch - a]) << 4 * e

    def append(self, table, lens, k, v, cu):
        for i, l in enumerate(lens):
            for r in range(cu[i], cu[i + 1]):
                p = l - (cu[i + 1] - r)
                if p < 0:
                    continue
                for h in range(self.hkv):
                    self._write(table[i][p // BLOCK], h, p % BLOCK, "k", k[r, h])
                    self._write(table[i][p // BLOCK], h, p % BLOCK, "v", v[r, h])

    def values(self, pages, head):
        """K and V [tokens][d] of these pages and one head, whole arrays at a time."""
        d = self.d
        s = scale_value(self.scales[pages, head][:, :, [scale_place(t) for t in range(BLOCK)]])
        at, half = (np.array(x) for x in zip(*(k_place(c, d) for c in range(d))))
        k = VALUES[self.k[pages, head][:, :, at] >> (4 * half).astype(np.uint8) & 15]
        k = k * np.repeat(s[:, :-1], 32, axis=1).swapaxes(1, 2)
        places = np.array([[v_place(t, c) for c in range(d)] for t in range(BLOCK)])
        v = VALUES[self.v[pages, head][:, places[..., 0], places[..., 1]] >> (4 * places[..., 2]).astype(np.uint8) & 15]
        return k.reshape(-1, d), (v * s[:, -1][:, :, None]).reshape(-1, d)

    def sequence(self, row, length):
        """K and V [length][hkv][d] of a sequence."""
        pages = np.asarray(row[:(length + BLOCK - 1) // BLOCK], np.int64)
        both = [self.values(pages, h) for h in range(self.hkv)]
        return tuple(np.stack([x[w][:length] for x in both], 1) for w in (0, 1))

    def attention(self, table, lens, q, cu, scale):
        """(o, lse [hq][rows], sum of p |v|, largest sum of |q k| scale [rows][hq], sum of |v|) of the rows."""
        rows, hq, d = q.shape
        g = hq // self.hkv
        o, lse = np.zeros((rows, hq, d)), np.full((hq, rows), -np.inf)
        weight, size, plain = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq, d))
        for i, l in enumerate(lens):
            if l == 0 or cu[i] == cu[i + 1]:
                continue
            pages = np.asarray(table[i][:(l + BLOCK - 1) // BLOCK], np.int64)
            for h in range(self.hkv):
                k, v = self.values(pages, h)
                for r in range(cu[i], cu[i + 1]):
                    n = l - (cu[i + 1] - r) + 1
                    if n <= 0:
                        continue
                    x = q[r, h * g:(h + 1) * g] @ k[:n].T * scale
                    top = x.max(1, keepdims=True)
                    p = np.exp(x - top)
                    total = p.sum(1, keepdims=True)
                    o[r, h * g:(h + 1) * g] = p / total @ v[:n]
                    lse[h * g:(h + 1) * g, r] = (top + np.log(total))[:, 0]
                    weight[r, h * g:(h + 1) * g] = p / total @ np.abs(v[:n])
                    plain[r, h * g:(h + 1) * g] = np.abs(v[:n]).sum(0)
                    size[r, h * g:(h + 1) * g] = (np.abs(q[r, h * g:(h + 1) * g]) @ np.abs(k[:n]).T * scale).max(1)
        return o, lse, weight, size, plain
