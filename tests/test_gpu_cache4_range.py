"""Attention over the 4-bit cache where a score's sum of products passes fp32's end before the row's factor brings it
back, and NaN scales over codes that are not zero: both may come out as -infinity, as a masked score does."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from oracle import kv_cache4 as k4
from test_gpu_cache4 import _bf16, _check, _cu, _f64, _garbage, _i32, _pair, _random_cache, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.fixture(autouse=True)
def _no_report_left():
    yield
    pkg.hdp_device_status()


def _far_below(tokens, d, rng, near=()):
    """K rows whose 64 first channels are -2^108: with q of 2^-107 their products sum to -128, on the way to it to
    -2^128 of fp32 where q and K are scaled apart; the tokens in `near` have channels of 0 and stay inside."""
    k = np.zeros((tokens, 1, d))
    k[:, :, :64] = -2.0 ** 108
    for t in near:
        k[t, :, rng.integers(0, 64, 3)] = 0
    return _bf16(k)


def _small_query(rows, hq, d):
    q = np.zeros((rows, hq, d))
    q[:, :, :64] = 2.0 ** -107
    return _bf16(q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("sign", [-1, 1])
def test_sums_beyond_the_end_in_a_short_sequence(d, runs, sign):
    """Ten tokens of which one has a sum inside fp32, one row, one head: a CTA for the unit, and by runs.  Scores of -15.75
    and nine times -16, or the same with the other sign."""
    rng = np.random.default_rng(d)
    cache, ref = _pair(_garbage(1, 1, d, rng))
    k, v = _far_below(10, d, rng), _bf16(rng.normal(size=(10, 1, d)))
    k[0, 0, 0] = 0
    pkg.cache_append(cache, _i32([[0]]), _i32([10]), k.cuda(), v.cuda(), cu=_i32([0, 10]))
    ref.append([[0]], [10], _f64(k), _f64(v), [0, 10])
    q = sign * _small_query(1, 1, d)
    o, lse = pkg.cache_attention(cache, _i32([[0]]), _i32([10]), q.cuda(), cu=_i32([0, 1]) if runs else None, scale=0.125)
    want = ref.attention([[0]], [10], _f64(q), [0, 1], 0.125)
    assert np.isclose(want[1][0, 0], np.log(np.exp(-sign * 15.75) + 9 * np.exp(-sign * 16.0)))
    _check(o, lse, want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 3])
def test_sums_beyond_the_end_in_runs_of_many_blocks(d, rows):
    """40 blocks of such keys, one in eight of them inside fp32, shared by 500 sequences: runs of a dozen blocks and more,
    in which small P have a budget after the first."""
    rng = np.random.default_rng(d + rows)
    n, tokens = 500, 40 * 64 - 7
    table, pages = _table([tokens], rng)
    cache, ref = _pair(_garbage(pages, 1, d, rng))
    k = _far_below(tokens, d, rng, near=np.flatnonzero(rng.random(tokens) < 0.125))
    v = _bf16(rng.normal(size=(tokens, 1, d)) + 0.5)
    pkg.cache_append(cache, _i32(table), _i32([tokens]), k.cuda(), v.cuda(), cu=_i32([0, tokens]))
    ref.append(table, [tokens], _f64(k), _f64(v), [0, tokens])
    q = _small_query(n * rows, 1, d)
    cu = np.arange(n + 1) * rows
    o, lse = pkg.cache_attention(cache, _i32(np.repeat(table, n, 0)), _i32([tokens] * n), q.cuda(), cu=_i32(cu), scale=0.125)
    one = ref.attention(table, [tokens], _f64(q[:rows]), [0, rows], 0.125)
    _check(o, lse, tuple(np.tile(x, (1, n) if i == 1 else (n,) + (1,) * (x.ndim - 1)) for i, x in enumerate(one)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [0.01, 0.125, 1.0])
def test_drawn_keys_near_the_end_of_the_range(d, size):
    """K of one sign near bf16's end and q that brings it back, groups that pass the end or do not, sequences of a few
    tokens to many blocks, scores from flat to peaked."""
    rng = np.random.default_rng(int(1000 * size) + d)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), 40))] + [1, 64, 65, 128]
    new = [min(l, int(rng.integers(0, 4))) for l in lens]
    table, pages = _table(lens, rng)
    cache, ref = _pair(_garbage(pages, 2, d, rng))
    k = -np.exp2(rng.uniform(105, 110, (sum(lens), 2, d))) * (rng.random((sum(lens), 2, d)) < 0.9)
    v = rng.normal(size=k.shape)
    k, v = _bf16(k), _bf16(v)
    cu = _cu(lens)
    pkg.cache_append(cache, _i32(table), _i32(lens), k.cuda(), v.cuda(), cu=_i32(cu))
    back = pkg.cache_read(cache, _i32(table), _i32(lens), sum(lens), cu=_i32(cu))
    ref = k4.Cache(*(x.cpu().numpy() for x in (cache.k, cache.v, cache.scales)))
    assert np.array_equal(_f64(back[0])[:lens[0]], ref.sequence(table[0], lens[0])[0])
    q = _bf16(np.exp2(rng.uniform(-108, -106, (sum(new), 4, d))) * (rng.random((sum(new), 4, 1)) < 0.8) * size)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(_cu(new)), scale=0.125)
    _check(o, lse, ref.attention(table, lens, _f64(q), _cu(new), 0.125))


@pytest.mark.parametrize("d,size", [(64, 1.0), (64, 4.0), (128, 1.0), (128, 3.0)])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("token", [3, 64 * 30 + 9, 64 * 39 + 5])
def test_nan_scales_over_codes_that_are_not_zero(d, size, sign, token):
    """One token's K scale of 32 channels is NaN and its products are all of one sign, in whole tiles of eight rows (rows that
    pad a tile are zeros, and zero times NaN is noticed): every row that sees it is NaN, in the first block, inside a long
    run, and in a block that is not seen whole; with flat scores and with peaked ones, which may lose small P."""
    rng = np.random.default_rng(d + token)
    n, tokens = 400, 64 * 39 + 20
    table, (cache, ref) = _random_cache([tokens], 1, d, rng, low=124)
    page, at = table[0, token // 64], token % 64
    ref.k[page, 0, at] = 0x22  # all codes 1
    ref.scales[page, 0, 1, k4.scale_place(at)] = 255
    cache.k.copy_(torch.tensor(ref.k)), cache.scales.copy_(torch.tensor(ref.scales))
    q = rng.normal(size=(n, 8, d)) * size
    q[:, :, 32:64] = sign * np.abs(q[:, :, 32:64])
    q = _bf16(q)
    o, lse = pkg.cache_attention(cache, _i32(np.repeat(table, n, 0)), _i32([tokens] * n), q.cuda())
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    o, lse = pkg.cache_attention(cache, _i32(table), _i32([token]), q[:1].cuda())  # the tokens in front of it: nothing is NaN
    _check(o, lse, ref.attention(table, [token], _f64(q[:1]), [0, 1], d ** -0.5))


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("rows", [1, 2])
def test_nan_scales_in_a_few_tokens(sign, rows):
    """The same in a CTA that has the whole unit, and in tiles of 16 rows."""
    rng = np.random.default_rng(7)
    d, lens = 64, [10, 10]
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    ref.k[table[1, 0], 0, 4] = 0x22
    ref.scales[table[1, 0], 0, 0, k4.scale_place(4)] = 255
    cache.k.copy_(torch.tensor(ref.k)), cache.scales.copy_(torch.tensor(ref.scales))
    q = _bf16(sign * np.abs(rng.normal(size=(2 * rows, 8, d))))
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=None if rows == 1 else _i32([0, 2, 4]))
    assert torch.isnan(o[rows:]).all() and torch.isnan(lse[:, rows:]).all()
    assert torch.isfinite(o[:rows]).all() and torch.isfinite(lse[:, :rows]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("runs", [False, True])
def test_scores_of_the_largest_magnitude(d, runs):
    """Scores of 1.75 * 2^126, 0 and their negatives: the largest has all of the weight, whichever sign it has."""
    rng = np.random.default_rng(d)
    n, tokens = 3, 100
    table, pages = _table([tokens] * n, rng)
    cache, ref = _pair(_garbage(pages, 1, d, rng))
    k, v = np.zeros((n * tokens, 1, d)), _bf16(rng.normal(size=(n * tokens, 1, d)))
    k[:, 0, 0] = -2.0 ** 100  # sequence 2: all the same
    k[70, 0, 0], k[tokens + 9, 0, 0] = 2.0 ** 100, 0  # sequence 0: one far above; 1: one between
    k = _bf16(k)
    lens, cu = _i32([tokens] * n), _i32(_cu([tokens] * n))
    pkg.cache_append(cache, _i32(table), lens, k.cuda(), v.cuda(), cu=cu)
    held = _f64(pkg.cache_read(cache, _i32(table), lens, n * tokens, cu=cu)[1])
    q = np.zeros((n, 2, d))
    q[:, :, 0] = 1.75 * 2.0 ** 26
    o, lse = pkg.cache_attention(cache, _i32(table), lens, _bf16(q).cuda(), cu=_i32(range(n + 1)) if runs else None, scale=1.0)
    for i, row in ((0, held[70, 0]), (1, held[tokens + 9, 0])):
        assert np.abs(_f64(o)[i] - row).max() <= 2.0 ** -8 * np.abs(row).max()
    mean, size = held[2 * tokens:, 0].mean(0), np.abs(held[2 * tokens:, 0]).mean(0)
    assert (np.abs(_f64(o)[2] - mean) <= 2.0 ** -8 * np.abs(mean) + (2.0 ** -11 + 2.0 ** -18) * size).all()
    top = 1.75 * 2.0 ** 126
    assert np.abs(_f64(lse) / top - [1, 0, -1]).max() <= 2.0 ** -20
