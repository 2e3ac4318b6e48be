"""Pins of the cache oracle: its codes against PyTorch's e4m3 type and exhaustive search, its scales and bounds against
their definitions, its attention against the packed attention oracle, its block choice against brute force."""
import math

import numpy as np
import pytest
import torch

from oracle import attention_f64
from oracle import kv_cache as kc


def test_e4m3_values_and_rounding_match_the_torch_type():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    got = kc.values(codes.numpy(), kc.E4M3)
    assert np.array_equal(np.isnan(ref), np.isnan(got)) and np.array_equal(ref[~np.isnan(ref)], got[~np.isnan(got)])
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)) * torch.logspace(-4, 2, 20000)
    x = torch.cat([x, torch.tensor([0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])]).clamp(-448, 448)
    assert np.array_equal(kc.round_code(x.double().numpy(), kc.E4M3), x.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("fmt", [kc.E4M3, kc.INT8])
def test_scale_is_the_smallest_power_of_two(fmt):
    for a in (0.0, 2.0 ** -140, 1e-30, 0.7, 1.0, 127.0, 127.5, 448.0, 449.0, 3e38):
        s = kc.scale_of(a, fmt)
        assert math.frexp(s)[0] == 0.5 and a <= kc.LARGEST[fmt] * s
        assert s == 2.0 ** -126 or a > kc.LARGEST[fmt] * s / 2


def test_v_order_is_a_permutation():
    assert sorted(kc.v_order()) == list(range(64))


@pytest.mark.parametrize("fmt", [kc.E4M3, kc.INT8])
def test_append_in_pieces_stays_within_its_error_bound_and_bounds_nest(fmt):
    rng = np.random.default_rng(1)
    n, hkv, d = 150, 2, 64
    x, y = rng.normal(size=(2, n, hkv, d)) * np.exp2(np.arange(n) / 25)[:, None, None]
    whole, pieces = kc.Cache(3, hkv, d, fmt), kc.Cache(3, hkv, d, fmt)
    table = [[2, 0, 1]]
    whole.append(table, [n], x, y, [0, n])
    for t in range(n):
        pieces.append(table, [t + 1], x[t:t + 1], y[t:t + 1], [0, 1])
    assert np.array_equal(whole.scales, pieces.scales) and np.array_equal(whole.bounds, pieces.bounds)
    for c, steps in ((whole, 0.5), (pieces, 1.0)):
        k, v = c.sequence(table[0], n)
        for got, ref, w in ((k, x, 0), (v, y, 1)):
            s = np.repeat(c.scales[table[0]][:, :, w], 64, axis=0)[:n, :, None]
            step = s if fmt == kc.INT8 else np.maximum(s * 2.0 ** -9, 2.0 ** (np.floor(np.log2(np.abs(ref))) - 3))
            slack = 2.0 ** -9 * s if fmt == kc.E4M3 and steps == 1.0 else 0  # one subnormal step
            assert (np.abs(got - ref) <= (0.5 if fmt == kc.E4M3 else steps) * step * (1 + 1e-12) + slack).all()
    unit = whole.scales[:, :, 0] * (1 if fmt == kc.INT8 else 4)
    for b in range(3):
        rows = x[b * 64:(b + 1) * 64]
        assert (whole.bounds[table[0][b], :, 0] * unit[table[0][b]][:, None] <= rows.min(0)).all()
        assert (whole.bounds[table[0][b], :, 1] * unit[table[0][b]][:, None] >= rows.max(0)).all()


def test_attention_over_the_cache_is_the_packed_attention_of_its_values():
    rng = np.random.default_rng(2)
    lens, hq, hkv, d = [70, 5], 4, 2, 64
    cu = np.array([0, 70, 75], np.int32)
    c = kc.Cache(3, hkv, d, kc.INT8)
    table = [[1, 2], [0, 0]]
    c.append(table, lens, rng.normal(size=(75, hkv, d)), rng.normal(size=(75, hkv, d)), cu)
    q = rng.normal(size=(75, hq, d))
    o, lse, _, _, _ = c.attention(table, lens, q, cu, 0.125)
    k, v = (np.concatenate(x) for x in zip(c.sequence(table[0], 70), c.sequence(table[1], 5)))
    o_ref, lse_ref = attention_f64(q, k, v, cu, hq, hkv, d, 0.125)
    assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, lse_ref, atol=1e-12)
    every = np.broadcast_to(np.arange(2), (75, hkv, 2))
    o2, lse2, _, _, _ = c.attention(table, lens, q, cu, 0.125, every)
    assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2, atol=1e-12)


def test_block_score_bounds_every_key_and_forced_blocks_are_kept():
    rng = np.random.default_rng(3)
    n, hq, hkv, d = 640, 4, 1, 64
    c = kc.Cache(10, hkv, d, kc.INT8)
    table, cu = [list(range(10))], [0, 1]
    c.append(table, [n], rng.normal(size=(n, hkv, d)), rng.normal(size=(n, hkv, d)), [0, n])
    q = np.rint(rng.normal(size=(1, hq, d)) * 30)
    q[0, 0, 0] = 127  # whole numbers that the rounding of q leaves alone
    k, _ = c.sequence(table[0], n)
    best = (q[0] @ k[:, 0].T).reshape(hq, 10, 64).max(2).sum(0)  # per block: sum over heads of the largest product
    up, down = np.maximum(q[0], 0).sum(0), np.minimum(q[0], 0).sum(0)
    score = (c.bounds[:, 0, 1] @ up + c.bounds[:, 0, 0] @ down) * c.scales[:, 0, 0]
    assert (score >= best - 0.5 * c.scales[:, 0, 0] * np.abs(q).sum()).all()
    got = c.select(table, [n], q, cu, 4, 1, 1)[0, 0]
    middle = sorted(range(1, 9), key=lambda b: (-score[b], b))[:2]
    assert list(got) == sorted([0, 9] + middle)
    assert list(c.select(table, [n], q, cu, 12, 1, 1)[0, 0]) == list(range(10)) + [-1, -1]
