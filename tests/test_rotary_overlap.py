"""Rotary positions: calls whose outputs overlap their inputs, the other tensor's rows or themselves are refused, all
others go on.  No GPU is needed: the calls have no positions, which is looked at behind the overlaps."""
import ctypes
import itertools

import numpy as np
import pytest

import packed_varlen_attention_aware_gb300 as pkg
from packed_varlen_attention_aware_gb300 import binding
from packed_varlen_attention_aware_gb300 import build as native_build

BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return pkg.load()


def _refusal(lib, q, k, rows, d, kind=2):
    """The reason why a call is refused; q, k: (in, out) of (at, row stride, head stride, heads) in elements."""
    size = 4 if kind == 2 else 2
    sides = [None if x is None else binding.RotaryRows(BASE + size * x[0][0], BASE + size * x[1][0], *x[0][1:3], *x[1][1:3], x[0][3]) for x in (q, k)]
    assert lib.hdp_rotary(*sides, rows, d, kind, None, ctypes.c_void_p(256), 2, 0, 1.0, None) == pkg.HDP_ERR_INVALID_ARGUMENT
    return pkg.hdp_last_error_message().removeprefix("hdp_rotary: ")


FREE = "position or freqs is NULL"
OTHERS, OWN, ITSELF = "rows of the other", "its input or not overlap", "rows and heads of an output"


def test_views_of_one_projection(lib):
    """q, k and v side by side: in place where the heads are apart, not where they share one."""
    R = 12 * 64
    view = lambda a, b, at=0: (at + a * 64, R, 64, b - a)
    both = lambda x: (x, x)
    for rows in (1, 2, 9):
        assert FREE in _refusal(lib, both(view(0, 8)), both(view(8, 10)), rows, 64)
        assert FREE in _refusal(lib, both(view(8, 10)), both(view(0, 8)), rows, 64, 0)
        assert OTHERS in _refusal(lib, both(view(0, 5)), both(view(4, 12)), rows, 64)
        assert OTHERS in _refusal(lib, both(view(4, 12)), both(view(0, 5)), rows, 64, 1)
        assert OTHERS in _refusal(lib, both(view(0, 8)), both((7 * 64 + 63, R, 64, 1)), rows, 64)
        assert FREE in _refusal(lib, both(view(0, 8)), both((8 * 64, R, 32, 4)), rows, 32)  # heads of another pitch
        assert OTHERS in _refusal(lib, both(view(0, 8)), both((7 * 64, R, 32, 4)), rows, 32)
        assert FREE in _refusal(lib, both((0, R, 128, 6)), both((64, R, 128, 6)), rows, 64)  # heads of q and k in turn
    # out of place: q's output in k's input, and the two outputs in each other
    far = 1 << 16
    assert OTHERS in _refusal(lib, (view(0, 4), view(8, 12)), (view(6, 9), view(0, 3, far)), 5, 64)
    assert OTHERS in _refusal(lib, (view(6, 9), view(0, 3, far)), (view(0, 4), view(8, 12)), 5, 64)
    assert OTHERS in _refusal(lib, (view(0, 4), view(0, 4, far)), (view(4, 8), view(3, 7, far)), 5, 64)
    assert FREE in _refusal(lib, (view(0, 4), view(0, 4, far)), (view(0, 8), view(4, 12, far)), 5, 64)
    assert OWN in _refusal(lib, (view(0, 4), view(1, 5)), None, 5, 64)
    assert OWN in _refusal(lib, (view(0, 4), (R, R, 64, 4)), None, 5, 64)  # a row further on
    assert FREE in _refusal(lib, (view(0, 4), (R, R, 64, 4)), None, 1, 64)
    assert FREE in _refusal(lib, (view(0, 4), view(4, 8)), None, 5, 64)


def test_heads_outside_rows_and_single_ones(lib):
    S = 9 * 64
    x = lambda at, heads: ((at, 64, S, heads),) * 2
    assert FREE in _refusal(lib, x(0, 3), x(3 * S, 2), 9, 64) and OTHERS in _refusal(lib, x(0, 3), x(2 * S, 2), 9, 64)
    assert FREE in _refusal(lib, ((0, 128, S, 1),) * 2, ((64, 128, 5, 1),) * 2, 4, 64)  # one head each: their strides say nothing
    assert FREE in _refusal(lib, ((0, 7, 128, 4),) * 2, ((64, 9, 128, 4),) * 2, 1, 64)  # one row
    assert OTHERS in _refusal(lib, ((0, 128, S, 1),) * 2, ((63, 128, 5, 1),) * 2, 4, 64)


def test_outputs_over_themselves(lib):
    far = 1 << 16
    for out in ((far, 0, 64, 2), (far, 63, 64, 1), (far, 64, 64, 2), (far, 200, 63, 3), (far, 128, 64, 3), (far, -128, 64, 3)):
        assert ITSELF in _refusal(lib, ((0, 512, 64, out[3]), out), None, 4, 64), out
    for out in ((far, 192, 64, 3), (far, 64, 256, 2), (far, -192, 64, 3), (far, 128, 64 * 3, 2)):
        assert FREE in _refusal(lib, ((0, 512, 64, out[3]), out), None, 4, 64), out
    assert FREE in _refusal(lib, ((0, 0, 0, 3), (far, 192, 64, 3)), None, 4, 64)  # a broadcast input


def test_strides_that_leave_memory(lib):
    assert ITSELF in _refusal(lib, ((0, 64, 64, 1), (64, 1 << 60, 64, 1)), None, 2 ** 31 - 1, 64)
    assert OWN in _refusal(lib, ((0, 1 << 60, 64, 1), (1 << 16, 64, 64, 1)), None, 2 ** 20, 64)
    least, most = -2 ** 63, 2 ** 63 - 1  # strides that are never taken
    assert FREE in _refusal(lib, ((0, most, 64, 2),) * 2, ((128, least, most, 1),) * 2, 1, 64)
    assert OTHERS in _refusal(lib, ((0, least, least, 1),) * 2, ((63, most, most, 1),) * 2, 1, 64)


def _elements(x, rows, d):
    return [x[0] + i * x[1] + h * x[2] + c for i, h, c in itertools.product(range(rows), range(x[3]), range(d))]


def test_drawn_layouts_against_every_element(lib):
    """Layouts of a few rows and heads close together: what is refused has an element in common, or rows of different
    strides; what is not has none."""
    rng = np.random.default_rng(0)
    seen = {FREE: 0, OTHERS: 0, OWN: 0, ITSELF: 0}
    for _ in range(6000):
        rows, d = int(rng.integers(1, 5)), int(rng.integers(2, 5))
        draw = lambda heads: (int(rng.integers(0, 90)), int(rng.choice([12, 16, 20, 24, 3, -16, 0])), int(rng.choice([d, 4, 5, 8, 40, -4, 0])), heads)
        sides = []
        for heads in rng.integers(1, 5, 2):
            a, b = draw(int(heads)), draw(int(heads))
            if rng.random() < 0.7:  # the strides of a common buffer
                b = (b[0],) + a[1:]
            sides.append((a, a) if rng.random() < 0.4 else (a, b))
        if rng.random() < 0.7:
            sides[1] = tuple((x[0], sides[0][0][1], sides[0][0][2] if rng.random() < 0.7 else x[2], x[3]) for x in sides[1])
        if any(a[0] == b[0] and a[1:] != b[1:] for a, b in sides):
            continue
        q, k = sides if rng.random() < 0.8 else (sides[0], None)
        why = _refusal(lib, q, k, rows, d)
        given = [x for x in (q, k) if x is not None]
        sets = [[set(_elements(y, rows, d)) for y in x] for x in given]
        itself = [len(_elements(x[1], rows, d)) != len(s[1]) for x, s in zip(given, sets)]
        own = [x[0] != x[1] and bool(s[0] & s[1]) for x, s in zip(given, sets)]
        cross = k is not None and bool(sets[0][1] & (sets[1][0] | sets[1][1]) or sets[1][1] & sets[0][0])
        shared = any(itself) or any(own) or cross
        kind = next(x for x in seen if x in why)
        seen[kind] += 1
        alike = rows == 1 or len({y[1] for x in given for y in x}) == 1
        assert kind == FREE if not shared and alike else kind != FREE if shared else True, (q, k, rows, d, why)
        if kind == ITSELF:
            assert any(itself)
    assert min(seen.values()) > 200, seen
