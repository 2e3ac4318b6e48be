"""Pins of the oracles of the 4-bit cache, the block tables and the rotary positions: closed forms, permutations,
invariants, the packed attention oracle."""
import math

import numpy as np
import pytest

from oracle import attention_f64
from oracle import kv_cache4 as k4
from oracle import rows as ro


def test_codes_are_the_nearest_values_and_ties_go_to_the_even_code():
    grid = np.arange(-6, 6.001, 2.0 ** -8)
    codes = k4.round_code(grid)
    far = np.abs(grid[:, None] - k4.VALUES)
    assert (np.abs(grid - k4.VALUES[codes]) == far.min(1)).all()
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert k4.VALUES[k4.round_code(ties)].tolist() == [0, 1, 1, 2, 2, 4, 4]
    assert k4.VALUES[k4.round_code(-ties)].tolist() == [0, -1, -1, -2, -2, -4, -4]
    assert np.array_equal(k4.round_code(k4.VALUES[1:8]), np.arange(1, 8))


def test_scale_is_the_smallest_power_of_two():
    for a in (0.0, 2.0 ** -140, 6 * 2.0 ** -126, 1e-30, 0.7, 6.0, 6.01, 12.0, 3e38):
        s = float(k4.scale_value(k4.scale_byte(a)))
        assert math.frexp(s)[0] == 0.5 and a <= 6 * s
        assert s == 2.0 ** -126 or a > 3 * s
    assert k4.scale_byte(math.inf) == k4.scale_byte(math.nan) == 255 and math.isnan(k4.scale_value(255))


@pytest.mark.parametrize("d", [64, 128])
def test_places_are_permutations(d):
    assert sorted(k4.k_place(c, d) for c in range(d)) == [(b, e) for b in range(d // 2) for e in range(2)]
    v = {k4.v_place(t, c) for t in range(64) for c in range(d)}
    assert v == {(i, b, e) for i in range(d // 16) for b in range(512) for e in range(2)}
    assert sorted(k4.scale_place(t) for t in range(64)) == list(range(64))


@pytest.mark.parametrize("d", [64, 128])
def test_rows_come_back_within_half_a_step_whatever_the_order(d):
    rng = np.random.default_rng(d)
    n, hkv = 70, 2
    x, y = rng.normal(size=(2, n, hkv, d)) * np.exp2(rng.integers(-9, 9, size=(2, n, hkv, 1)))
    make = lambda: k4.Cache(rng.integers(0, 256, (2, hkv, 64, d // 2), np.uint8), rng.integers(0, 256, (2, hkv, d // 16, 512), np.uint8),
                            rng.integers(0, 256, (2, hkv, d // 32 + 1, 64), np.uint8))
    whole, pieces = make(), make()
    whole.append([[1, 0]], [n], x, y, [0, n])
    for a, z in ((0, 33), (33, 34), (34, 70)):
        pieces.append([[1, 0]], [z], x[a:z], y[a:z], [0, z - a])
    got, again = whole.sequence([1, 0], n), pieces.sequence([1, 0], n)
    for g, a, ref, step in zip(got, again, (x, y), (32, d)):
        assert np.array_equal(g, a)
        top = np.abs(ref.reshape(n, hkv, -1, step)).max(-1)
        s = np.vectorize(lambda t: float(k4.scale_value(k4.scale_byte(t))))(top).repeat(step, -1)
        near = np.where(np.abs(ref) <= 2 * s, 0.25, np.where(np.abs(ref) <= 4 * s, 0.5, 1.0)) * s
        assert (np.abs(g - ref) <= near).all()
    k, v = whole._row(0, 1, 5, "k"), whole._row(0, 1, 5, "v")
    assert np.array_equal(k4.VALUES[k[0]] * k4.scale_value(k[1]), got[0][69, 1]) and np.array_equal(k4.VALUES[v[0]] * k4.scale_value(v[1]), got[1][69, 1])


def test_attention_over_the_cache_is_the_packed_attention_of_its_values():
    rng = np.random.default_rng(3)
    lens, hq, hkv, d = [70, 5], 4, 2, 64
    cu = [0, 70, 75]
    cache = k4.Cache(np.zeros((3, hkv, 64, d // 2), np.uint8), np.zeros((3, hkv, d // 16, 512), np.uint8), np.zeros((3, hkv, 3, 64), np.uint8))
    table = [[2, 0], [1, 0]]
    cache.append(table, lens, *rng.normal(size=(2, 75, hkv, d)), cu)
    q = rng.normal(size=(75, hq, d))
    o, lse, weight, size, plain = cache.attention(table, lens, q, cu, 0.1)
    k, v = (np.concatenate(x) for x in zip(*(cache.sequence(t, l) for t, l in zip(table, lens))))
    ro_, rl = attention_f64(q, k, v, np.array(cu, np.int32), hq, hkv, d, 0.1)
    assert np.abs(o - np.asarray(ro_).reshape(o.shape)).max() < 1e-12 and np.abs(lse - np.asarray(rl).reshape(lse.shape)).max() < 1e-12
    assert (weight >= np.abs(o) - 1e-12).all() and (size > 0).all() and (plain >= weight - 1e-12).all()


def test_a_stack_of_pages_by_hand():
    free, table, held = [9, 8, 7, 6, 5], [[-1] * 3 for _ in range(3)], [0, 0, 0]
    assert ro.assign(free, table, held, [65, 0, 64])
    assert (table, held, free) == ([[5, 6, -1], [-1] * 3, [7, -1, -1]], [2, 0, 1], [9, 8])
    assert not ro.assign(free, table, held, [1, 130, 129])  # one comes back: three for the second, none for the third
    assert (table, held, free) == ([[5, 6, -1], [6, 8, 9], [7, -1, -1]], [1, 3, 1], [])
    assert ro.assign(free, table, held, [0, 0, 0])
    assert free == [7, 9, 8, 6, 5]


def test_taking_and_giving_back_leaves_the_stack():
    rng = np.random.default_rng(5)
    free, table, held = list(rng.permutation(40)), [[-1] * 6 for _ in range(7)], [0] * 7
    a, b = rng.integers(0, 200, 7), rng.integers(200, 384, 7)
    assert ro.assign(free, table, held, a)
    before = list(free), list(held)
    assert ro.assign(free, table, held, b) and ro.assign(free, table, held, a)
    assert (free, held) == before


def test_rows_of_documents_and_of_requests():
    seq, pos, slot = ro.rows([3, 0, 2], [0, 3, 3, 5], 7)
    assert seq.tolist() == [0, 0, 0, 2, 2, -1, -1] and pos.tolist() == [0, 1, 2, 0, 1, -1, -1] and (slot == -1).all()
    seq, pos, slot = ro.rows([66, 1], [0, 2, 4], 4, [[4, 2], [9, 0]], 5)
    assert pos.tolist() == [64, 65, -1, 0] and slot.tolist() == [128, 129, -1, -1]  # page 9 is none


@pytest.mark.parametrize("neighbours", [False, True])
def test_turns_keep_lengths_and_depend_on_distances(neighbours):
    rng = np.random.default_rng(7)
    x, y = rng.normal(size=(2, 4, 1, 10))
    f = np.array([1.0, 0.3, 0.01])
    pos = np.array([0, 5, 1000, 12345])
    a = ro.turn(x, pos, f, neighbours)
    assert np.allclose((a ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(a[..., 6:], x[..., 6:]) and np.array_equal(a[0], x[0])
    assert np.allclose((a * ro.turn(y, pos, f, neighbours)).sum(-1), (x * y).sum(-1))
    later = (ro.turn(x, pos + 77, f, neighbours) * ro.turn(y, pos + 70, f, neighbours)).sum(-1)
    assert np.allclose(later, (ro.turn(x, pos + 7, f, neighbours) * ro.turn(y, pos, f, neighbours)).sum(-1))
    back = ro.turn(a, pos, f, neighbours, backward=True, factor=2.0)
    assert np.allclose(back[1:, :, :6], 2 * x[1:, :, :6]) and np.array_equal(back[..., 6:], x[..., 6:])
    one = np.zeros((1, 1, 4))
    one[0, 0, 0] = 1.0
    quarter = ro.turn(one, [1], np.array([math.pi / 2, 0.0]), neighbours)[0, 0]
    assert np.allclose(quarter, [0, 1, 0, 0] if neighbours else [0, 0, 1, 0])


@pytest.mark.parametrize("neighbours", [False, True])
def test_the_gradient_of_a_turn_against_differences(neighbours):
    rng = np.random.default_rng(8)
    x, g = rng.normal(size=(2, 3, 2, 6))
    f, pos = np.array([0.9, 0.05]), [3, 0, 250]
    dx = ro.turn(g, pos, f, neighbours, backward=True, factor=1.3)
    loss = lambda z: (ro.turn(z, pos, f, neighbours, factor=1.3) * g).sum()
    wide = dx.copy()
    wide[..., 4:] = g[..., 4:]
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 0.5
        assert abs(loss(x + e) - loss(x - e) - wide[i]) < 1e-12
