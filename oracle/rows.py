"""Oracle of the block tables, the slot maps and the rotary positions: a stack of pages in Python lists, one row at a
time, angles in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np

BLOCK = 64


def assign(free, table, held, lens):
    """One call on a stack of free pages (a list, its top last), tables and held (lists, changed in place).  Returns
    whether every sequence got its pages."""
    columns = len(table[0])
    want = [-(-min(max(l, 0), columns * BLOCK) // BLOCK) for l in lens]
    for i in reversed(range(len(lens))):
        while held[i] > want[i]:
            held[i] -= 1
            free.append(int(table[i][held[i]]))
    for i in range(len(lens)):
        if want[i] - held[i] > len(free):
            return False
        while held[i] < want[i]:
            table[i][held[i]] = free.pop()
            held[i] += 1
    return True


def rows(lens, cu, count, table=None, num_pages=0):
    """(sequence, position, slot) of `count` rows."""
    seq, pos, slot = (np.full(count, -1, np.int64) for _ in range(3))
    for i, l in enumerate(lens):
        for r in range(cu[i], min(cu[i + 1], count)):
            p = max(l, 0) - (cu[i + 1] - r)
            seq[r], pos[r] = i, p
            if table is not None and p >= 0 and 0 <= table[i][p // BLOCK] < num_pages:
                slot[r] = int(table[i][p // BLOCK]) * BLOCK + p % BLOCK
    return seq, pos, slot


def turn(x, pos, freqs, neighbours=False, backward=False, factor=1.0):
    """x [rows][heads][d] float64 with its pairs turned; rows at negative positions as they are."""
    out = np.array(x, np.float64)
    half = len(freqs)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        angle = np.asarray(pos, np.float64) * freqs[i] * (-1 if backward else 1)
        c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return np.where((np.asarray(pos) >= 0)[:, None, None], out, x)
