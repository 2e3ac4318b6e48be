"""The 4-bit cache on the GPU against its fp64 oracle: codes and scales bit for bit, rows read back exactly, attention
within what its roundings allow."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from oracle import kv_cache4 as k4

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


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _bf16(x):
    return torch.as_tensor(np.asarray(x)).to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _garbage(pages, hkv, d, rng):
    return (rng.integers(0, 256, (pages, hkv, 64, d // 2), np.uint8), rng.integers(0, 256, (pages, hkv, d // 16, 512), np.uint8),
            rng.integers(0, 256, (pages, hkv, d // 32 + 1, 64), np.uint8))


def _pair(arrays):
    """The same cache on the GPU and in the oracle."""
    return pkg.KVCache4(*(torch.tensor(a, device="cuda") for a in arrays)), k4.Cache(*arrays)


def _same(cache, ref):
    for name, a, b in zip(("k", "v", "scales"), (cache.k, cache.v, cache.scales), (ref.k, ref.v, ref.scales)):
        a = a.cpu().numpy()
        assert np.array_equal(a, b), (name, np.argwhere(a != b)[:5].tolist())


def _table(lens, rng, spare=0):
    need = [-(-l // 64) for l in lens]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -7, np.int32)  # entries behind the last block may hold anything
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    return table, len(order)


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


# ---------------------------------------------------------------- writing and reading

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_rows_in_pieces_are_the_oracles_bit_for_bit(d, hkv):
    """Prompts, drafts and single tokens of sequences of 0 to 200 tokens in a pool of garbage; rows behind the last are not read."""
    rng = np.random.default_rng(d + hkv)
    final = [1, 64, 200, 65, 0, 130]
    table, pages = _table(final, rng, spare=2)
    cache, ref = _pair(_garbage(pages, hkv, d, rng))
    lens = np.zeros(6, np.int64)
    for step in ([1, 63, 70, 65, 0, 128], [0, 1, 0, 0, 0, 1], None, [0, 0, 129, 0, 0, 0]):
        if step is None:  # one token for each: sequences at their end write their last row again
            new = np.ones(6, np.int64)
            lens = np.minimum(lens + 1, final)
            cu = None
        else:
            new = np.asarray(step)
            lens = lens + new
            cu = _cu(new)
        rows = int(new.sum())
        k, v = (_bf16(rng.normal(size=(rows + 3, hkv, d)) * np.exp2(rng.integers(-12, 12, (rows + 3, hkv, 1)))) for _ in "kv")
        if cu is None:
            k, v = k[:rows], v[:rows]
        else:
            k[rows:] = v[rows:] = float("nan")
        pkg.cache_append(cache, _i32(table), _i32(lens), k.cuda(), v.cuda(), cu=None if cu is None else _i32(cu))
        ref.append(table, lens, _f64(k), _f64(v), _cu(new))
        _same(cache, ref)
    assert lens.tolist() == final
    back = pkg.cache_read(cache, _i32(table), _i32(final), sum(final) + 2, cu=_i32(_cu(final)))
    want = [np.concatenate(x) for x in zip(*(ref.sequence(table[i], l) for i, l in enumerate(final)))]
    for got, w in zip(back, want):
        assert np.array_equal(_f64(got)[:sum(final)], w)


@pytest.mark.parametrize("d", [64, 128])
def test_every_kind_of_value(d):
    """Borders of the scales, ties, zeros, subnormal numbers, the largest ones, infinities and NaN, each among ordinary rows."""
    rng = np.random.default_rng(d)
    rows = rng.normal(size=(24, 1, d))
    rows[0] = 0
    rows[1] = -0.0
    rows[2, 0, :] = np.tile([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], d // 8)
    rows[3] = -rows[2] * 2.0 ** 40
    rows[4, 0, 5] = 6.03125  # a step above six times one
    rows[5] = 2.0 ** -133
    rows[6, 0, :] = np.linspace(-1, 1, d) * 2.0 ** -126
    rows[7, 0, 7] = 3.3895313892515355e38
    rows[8, 0, 3], rows[9, 0, d - 1], rows[10, 0, 32] = np.inf, -np.inf, np.nan
    rows[11, 0, ::7] = 2.0 ** -120
    rows[12:] *= np.exp2(rng.integers(-120, 120, (12, 1, 1)))
    x = _bf16(rows)
    cache, ref = _pair(_garbage(1, 1, d, rng))
    pkg.cache_append(cache, _i32([[0]]), _i32([24]), x.cuda(), x.flip(0).cuda(), cu=_i32([0, 24]))
    with np.errstate(invalid="ignore"):
        ref.append([[0]], [24], _f64(x), _f64(x.flip(0)), [0, 24])
    _same(cache, ref)
    k, v = pkg.cache_read(cache, _i32([[0]]), _i32([24]), 24, cu=_i32([0, 24]))
    wk, wv = ref.sequence([0], 24)
    assert np.array_equal(_f64(k), wk, equal_nan=True) and np.array_equal(_f64(v), wv, equal_nan=True)
    assert np.isnan(wk).sum() == 3 * 32 and np.isnan(wv).sum() == 3 * d
    one, again = _pair(_garbage(1, 1, d, rng))  # the kernel for single tokens
    for r in range(24):
        pkg.cache_append(one, _i32([[0]]), _i32([r + 1]), x[r:r + 1].cuda(), x[23 - r:24 - r].cuda())
    assert all(torch.equal(a[..., :24] if i == 1 else a, b[..., :24] if i == 1 else b) for i, (a, b) in
               enumerate(zip(pkg.cache_read(one, _i32([[0]]), _i32([24]), 24, cu=_i32([0, 24]))[0].nan_to_num(7).unbind(0), k.nan_to_num(7).unbind(0))))


def test_rows_outside_the_tables():
    """Rows at negative positions are not written and read as zeros, pages outside the pool and lengths outside the table
    are reported, nothing else changes."""
    rng = np.random.default_rng(4)
    d, hkv = 64, 2
    cache, ref = _pair(_garbage(4, hkv, d, rng))
    x = _bf16(rng.normal(size=(5, hkv, d)))
    pkg.cache_append(cache, _i32([[2]]), _i32([3]), x.cuda(), x.cuda(), cu=_i32([0, 5]))  # three tokens, five rows
    ref.append([[2]], [3], _f64(x), _f64(x), [0, 5])
    _same(cache, ref)
    k, v = pkg.cache_read(cache, _i32([[2]]), _i32([3]), 5, cu=_i32([0, 5]))
    assert not k[:2].any() and not v[:2].any() and np.array_equal(_f64(k)[2:], ref.sequence([2], 3)[0])
    for table, lens, cu in (([[4]], [5], [0, 5]), ([[-1]], [5], [0, 5]), ([[1]], [70], [0, 0]), ([[1]], [-3], [0, 5])):
        pkg.hdp_device_status()
        pkg.cache_append(cache, _i32(table), _i32(lens), x.cuda(), x.cuda(), cu=_i32(cu))
        k, v = pkg.cache_read(cache, _i32(table), _i32(lens), 5, cu=_i32(cu))
        o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), torch.ones((5, 4, d), dtype=torch.bfloat16, device="cuda"), cu=_i32(cu))
        with pytest.raises(pkg.HdpError, match="outside"):  # of sequences without rows too
            pkg.hdp_device_status()
        if cu[1]:
            assert not k.any() and not v.any() and not o.any() and (lse == -np.inf).all()
        _same(cache, ref)


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of codes."""
    pages, hkv, d = 140000, 8, 128
    cache = pkg.KVCache4.empty(pages, hkv, d)
    rng = np.random.default_rng(9)
    table = np.array([[pages - 1, 3], [pages - 2, pages - 3]], np.int32)
    lens, new = [70, 128], [70, 128]
    k, v = (_bf16(rng.normal(size=(198, hkv, d))) for _ in "kv")
    pkg.cache_append(cache, _i32(table), _i32(lens), k.cuda(), v.cuda(), cu=_i32(_cu(new)))
    small = table.copy()
    small[table > 3] = pages - 1 - table[table > 3]
    arrays = [a[[pages - 1, pages - 2, pages - 3, 3]].cpu().numpy() for a in (cache.k, cache.v, cache.scales)]
    ref = k4.Cache(*(np.zeros_like(a) for a in arrays))
    ref.append(small, lens, _f64(k), _f64(v), _cu(new))
    kr, vr = pkg.cache_read(cache, _i32(table), _i32(lens), 198, cu=_i32(_cu(new)))
    for i, (a, z) in enumerate(((0, 70), (70, 198))):
        for got, want in zip((kr, vr), ref.sequence(small[i], lens[i])):
            assert np.array_equal(_f64(got)[a:z], want)
    q = _bf16(rng.normal(size=(2, 8, d)))
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    _check(o, lse, ref.attention(small, lens, _f64(q), [0, 1, 2], d ** -0.5))


# ---------------------------------------------------------------- attention

def _check(o, lse, want, rows=None):
    """o is rounded to bf16 (2^-8 of it) from a sum whose P is rounded to fp16 (2^-11 of each weight) and whose scores are
    fp32 sums of up to 128 products, each of the matrix instruction's additions cut at 2^-23 of its largest at worst: 2^-16
    of the sum of magnitudes, s.  A score that is off by s multiplies a weight by e^s at most and, through the row sum, by
    e^s again: off by e^2s - 1 of it (which is 2 s where s is small).  Weights below 2^-126 of a row's largest need not
    count: of each key that loses 2^-126 |v| at most."""
    ro, rl, weight, size, plain = want
    rows = np.arange(ro.shape[0]) if rows is None else rows
    s = 2.0 ** -16 * size[rows]
    do = np.abs(_f64(o)[rows] - ro[rows])
    limit = (2.0 ** -8 * np.abs(ro[rows]) + (2.0 ** -11 + np.expm1(2 * np.minimum(s, 300)) + 2.0 ** -18)[..., None] * weight[rows]
             + 2.0 ** -126 * plain[rows] + 2.0 ** -133)
    assert (do <= limit).all(), (float((do / limit).max()), np.argwhere(do > limit)[:4].tolist())
    got, ref = _f64(lse)[:, rows], rl[:, rows]
    none = np.isinf(ref)
    assert np.array_equal(none, np.isinf(got)) and (got[none] < 0).all()
    dl = np.abs(got[~none] - ref[~none])
    bound = s.T[~none] + 2.0 ** -18 + 2.0 ** -22 * np.abs(ref[~none])
    assert (dl <= bound).all(), float((dl / bound).max())


def _random_cache(lens, hkv, d, rng, spread=3, low=120):
    table, pages = _table(lens, rng, spare=1)
    k, v, s = _garbage(pages, hkv, d, rng)
    s[:] = rng.integers(low, low + spread, s.shape)
    return table, _pair((k, v, s))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 2), (2, 3), (1, 8), (1, 16), (3, 5)])
@pytest.mark.parametrize("most", [1, 3, 20])
def test_attention_is_the_oracles(d, hkv, g, most):
    """Lengths around the blocks' borders, none to 20 rows a sequence, rows behind the last, garbage in unwritten places."""
    rng = np.random.default_rng(d + 7 * hkv + g + most)
    lens = [1, 0, 63, 64, 65, 200, 129, 5]
    new = [1] * 8 if most == 1 else [min(l, int(rng.integers(0, most + 1))) for l in lens]
    table, (cache, ref) = _random_cache(lens, hkv, d, rng)
    rows = sum(new) + (0 if most == 1 else 2)
    q = _bf16(rng.normal(size=(rows, hkv * g, d)))
    if most > 1:
        q[sum(new):] = float("nan")
    cu = None if most == 1 else _i32(_cu(new))
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=cu)
    _check(o, lse, ref.attention(table, lens, np.nan_to_num(_f64(q)), _cu(new), d ** -0.5), np.arange(sum(new)))
    again, lse2 = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=cu)
    assert torch.equal(again[:sum(new)], o[:sum(new)]) and torch.equal(lse[:, :sum(new)], lse2[:, :sum(new)])


@pytest.mark.parametrize("lens,hkv,g,d", [([40000, 3, 70000], 8, 4, 128), ([150000], 8, 1, 64), ([6000] * 40, 2, 4, 64), ([1] * 900, 1, 2, 64)])
def test_long_and_many_sequences(lens, hkv, g, d):
    """Runs of many blocks, handed out in pieces, and sequences that pieces share; 900 sequences."""
    rng = np.random.default_rng(len(lens) + d)
    table, (cache, ref) = _random_cache(lens, hkv, d, rng)
    q = _bf16(rng.normal(size=(len(lens), hkv * g, d)))
    ws = torch.full((pkg.hdp_fourbit_attention_workspace_bytes(cache, hkv * g),), 0xff, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty((hkv * g, len(lens)), device="cuda")
    pkg.hdp_fourbit_attention(cache, _i32(table), _i32(lens), q.cuda(), d ** -0.5, ws, o, lse)
    _check(o, lse, ref.attention(table, lens, _f64(q), np.arange(len(lens) + 1), d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
def test_very_different_scales(d):
    """V scales over 2^-60 .. 2^60 between tokens, K groups over 2^-40 .. 2^5, rows of q of any size."""
    rng = np.random.default_rng(d)
    lens = [190, 70, 64]
    table, (cache, ref) = _random_cache(lens, 2, d, rng)
    s = ref.scales
    s[:, :, :-1] = rng.integers(87, 132, s[:, :, :-1].shape)
    s[:, :, -1] = rng.integers(67, 188, s[:, :, -1].shape)
    cache.scales.copy_(torch.tensor(s))
    q = _bf16(rng.normal(size=(3, 8, d)) * np.exp2([[-3], [-100], [2], [-6], [0], [-126], [-4], [-5]])[None])
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    _check(o, lse, ref.attention(table, lens, _f64(q), [0, 1, 2, 3], d ** -0.5))


@pytest.mark.parametrize("shift", [-126, -90, 40, 64, 65, 100, 120])
def test_keys_of_any_size_with_queries_that_bring_them_back(shift):
    """K scales near 2^shift, q near 2^-shift: scores of ordinary size."""
    rng = np.random.default_rng(shift + 200)
    lens, d = [100, 64, 7], 64
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    ref.scales[:, :, :-1] = np.clip(rng.integers(0, 6, ref.scales[:, :, :-1].shape) + shift + 125, 1, 254)
    cache.scales.copy_(torch.tensor(ref.scales))
    q = _bf16(rng.normal(size=(3, 4, d)) * 2.0 ** -shift)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    _check(o, lse, ref.attention(table, lens, _f64(q), [0, 1, 2, 3], d ** -0.5))


def _one_channel(ref, page, token, ch, code):
    """K's code of a channel, where it was 0."""
    at, e = k4.k_place(ch, ref.d)
    ref.k[page, 0, token, at] |= code << 4 * e


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 4])
@pytest.mark.parametrize("seen", [64, 40])
def test_large_scales_of_values_that_weigh_nothing_cost_no_range(d, rows, seen):
    """Key 0 has the row's weight and a V scale of 2^-53; keys 2, 5, 8 .. have V scales of 2^60 and weights of 2^-235 or
    less; key 1 has a weight of 2^-74 and alone a value in channel 0.  In one block, and behind a block of ordinary keys."""
    rng = np.random.default_rng(d + rows)
    lens = [seen, 64 + seen]
    table = np.array([[2, -7], [0, 1]], np.int32)
    k, v, s = _garbage(3, 1, d, rng)
    ref = k4.Cache(k, v, s)
    ref.k[:] = 0
    ref.scales[:] = 127
    for page in (2, 1, 0):
        ref.v[page, 0] |= 0x22  # no zeros among the other codes: |code| >= 1
        for t in range(64):
            _one_channel(ref, page, t, 0, 0xF if page == 0 or t % 3 == 2 else 4 if t == 0 else 2 if t > 1 else 0)  # -6, 2, 1; 0
            vs = 74 if t == 0 else 95 if t == 1 else 187 if t % 3 == 2 else 74
            ref.scales[page, 0, -1, k4.scale_place(t)] = 60 if page == 0 else vs
            i, byte, e = k4.v_place(t, 0)
            ref.v[page, 0, i, byte] = ref.v[page, 0, i, byte] & (0x0F if e else 0xF0) | (3 if t == 1 and page else 0) << 4 * e
    cache = pkg.KVCache4(*(torch.tensor(a, device="cuda") for a in (ref.k, ref.v, ref.scales)))
    q = np.zeros((2 * rows, 2, d))
    q[:, :, 0] = 26.0  # scores of 52, 26, 0 and -156: weights 1, 2^-37.5, 2^-75, 2^-300
    q = _bf16(q)
    cu = np.arange(3) * rows
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(cu), scale=1.0)
    want = ref.attention(table, lens, _f64(q), cu, 1.0)
    assert (want[0][:, :, 0] > 0).all()
    _check(o, lse, want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("before", [0, 64])
def test_nan_scales_among_the_largest(d, before):
    """V scales of 2^116 and more, one token's NaN: the output is NaN wherever that token is seen."""
    rng = np.random.default_rng(d + before)
    lens = [before + 64, before + 64]
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    ref.scales[:, :, -1] = rng.integers(243, 248, ref.scales[:, :, -1].shape)
    page = table[1, before // 64]
    ref.scales[page, 0, -1, k4.scale_place(20)] = 255
    for ch in range(d):
        i, byte, e = k4.v_place(20, ch)
        ref.v[page, 0, i, byte] &= 0x0F if e else 0xF0
    cache.v.copy_(torch.tensor(ref.v)), cache.scales.copy_(torch.tensor(ref.scales))
    q = _bf16(rng.normal(size=(2, 4, d)) * 0.05)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("rows", [1, 3])
def test_tiny_scales_beside_huge_ones(rows):
    """Channels with K scales of 2^-98 decide the scores; others have 2^70 and meet zeros of q."""
    rng = np.random.default_rng(29 + rows)
    lens, d = [64, 200, 66], 64
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    ref.scales[:, :, 0] = 29
    ref.scales[:, :, 1] = rng.choice([1, 197], ref.scales[:, :, 1].shape)
    cache.scales.copy_(torch.tensor(ref.scales))
    q = rng.normal(size=(3 * rows, 4, d)) * 2.0 ** 97
    q[:, :, 32:] = 0
    q = _bf16(q)
    cu = np.arange(4) * rows
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(cu))
    _check(o, lse, ref.attention(table, lens, _f64(q), cu, d ** -0.5))


def test_small_weights_count_where_the_heavy_ones_values_are_zero():
    """Within a block one key has all of a row's weight but 10^-9 .. 10^-30, and zero codes of V in half of the channels."""
    rng = np.random.default_rng(11)
    d, lens = 64, [64, 100]
    table, (cache, ref) = _random_cache(lens, 1, d, rng, spread=1, low=125)
    ref.scales[:, :, :-1] = 127
    for page in range(ref.k.shape[0]):
        ref.k[page] = 0
        at, e = k4.k_place(0, d)
        for t in range(64):
            ref.k[page, 0, t, at] = (2 if t == 9 else 1 + t % 2 * 8) << 4 * e  # 1 and +-0.5
        for ch in range(0, d, 2):
            i, byte, e = k4.v_place(9, ch)
            ref.v[page, 0, i, byte] &= 0x0f if e else 0xf0
    cache.k.copy_(torch.tensor(ref.k)), cache.v.copy_(torch.tensor(ref.v)), cache.scales.copy_(torch.tensor(ref.scales))
    q = np.zeros((2, 4, d))
    q[:, :, 0] = [40, 80, 100, 140]
    q = _bf16(q)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), scale=1.0)
    _check(o, lse, ref.attention(table, lens, _f64(q), [0, 1, 2], 1.0))


def test_nan_scales():
    """A NaN scale of a seen key makes the row NaN, of V only its output; behind the row's position it does nothing."""
    rng = np.random.default_rng(12)
    d, lens = 128, [130, 130, 130, 130]
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    ref.scales[table[0, 1], 0, 2, k4.scale_place(3)] = 255
    ref.scales[table[1, 2], 0, -1, k4.scale_place(1)] = 255
    ref.scales[table[2, 2], 0, :, [k4.scale_place(t) for t in range(2, 64)]] = 255
    cache.scales.copy_(torch.tensor(ref.scales))
    q = _bf16(rng.normal(size=(4, 4, d)))
    o, lse = (_f64(x) for x in pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda()))
    assert np.isnan(o[:2]).all() and np.isnan(lse[:, 0]).all() and np.isfinite(lse[:, 1:]).all()
    ok, rl = ref.attention(table[2:], lens[2:], _f64(q)[2:], [0, 1, 2], d ** -0.5)[:2]
    assert np.abs(o[2:] - ok).max() <= 2.0 ** -7 * np.abs(ok).max() and np.abs(lse[:, 2:] - rl).max() < 1e-4


def test_infinite_queries_and_scores_beyond_the_end():
    d = 64
    rng = np.random.default_rng(13)
    table, (cache, ref) = _random_cache([100, 100], 1, d, rng)
    q = _bf16(rng.normal(size=(2, 2, d)))
    q[0, 0, 5] = float("inf")
    q[0, 1, 6] = float("nan")
    o, lse = pkg.cache_attention(cache, _i32(table), _i32([100, 100]), q.cuda())
    assert torch.isnan(o[0]).all() and torch.isfinite(o[1]).all()


def test_drawn_shapes():
    rng = np.random.default_rng(21)
    for _ in range(24):
        d, hkv, g = int(rng.choice([64, 128])), int(rng.integers(1, 5)), int(rng.integers(1, 9))
        n = int(rng.integers(1, 20))
        lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), n))]
        new = [int(rng.integers(0, min(l, 9) + 1)) for l in lens]
        if not sum(new):
            continue
        table, (cache, ref) = _random_cache(lens, hkv, d, rng, spread=int(rng.integers(1, 20)), low=int(rng.integers(105, 125)))
        q = _bf16(rng.normal(size=(sum(new), hkv * g, d)))
        o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(_cu(new)), scale=0.05)
        _check(o, lse, ref.attention(table, lens, _f64(q), _cu(new), 0.05))


# ---------------------------------------------------------------- calls around the ordinary ones

def test_a_captured_step_is_replayed_with_new_lengths_and_two_streams_overlap():
    rng = np.random.default_rng(31)
    d, hkv, hq, n = 128, 2, 8, 5
    lens = np.array([70, 1, 640, 127, 300])
    table, (cache, ref) = _random_cache([l + 3 for l in lens], hkv, d, rng)
    gl, gt = _i32(lens), _i32(table)
    k, v, q = (torch.zeros((n, h, d), dtype=torch.bfloat16, device="cuda") for h in (hkv, hkv, hq))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkg.cache_attention(cache, gt, gl, q)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.cache_append(cache, gt, gl, k, v)
        o, lse = pkg.cache_attention(cache, gt, gl, q)
    for step in range(3):
        new = [_bf16(rng.normal(size=(n, h, d))) for h in (hkv, hkv, hq)]
        for to, x in zip((k, v, q), new):
            to.copy_(x)
        gl.copy_(_i32(lens + step + 1))
        graph.replay()
        ref.append(table, lens + step + 1, _f64(new[0]), _f64(new[1]), np.arange(n + 1))
        _check(o, lse, ref.attention(table, lens + step + 1, _f64(new[2]), np.arange(n + 1), d ** -0.5))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams * 3:
        s.wait_stream(torch.cuda.current_stream())
        outs.append(pkg.cache_attention(cache, gt, gl, q, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in outs)


def test_a_step_without_rows():
    cache = pkg.KVCache4.empty(2, 2, 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    table, lens, cu = _i32([[0], [1]]), _i32([5, 6]), _i32([0, 0, 0])
    pkg.cache_append(cache, table, lens, none, none, cu=cu)
    assert pkg.cache_read(cache, table, lens, 0, cu=cu)[0].shape == (0, 2, 64)
    o, lse = pkg.cache_attention(cache, table, lens, torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), cu=cu)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)


def test_what_a_4_bit_cache_is_not_for():
    cache = pkg.KVCache4.empty(2, 2, 64)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    table, lens = _i32([[0], [1]]), _i32([5, 6])
    with pytest.raises(TypeError, match="no lists"):
        pkg.cache_attention(cache, table, lens, q, blocks=torch.zeros((2, 2, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="hdp_cache_select"):
        pkg.cache_select(cache, table, lens, q, 1)
    with pytest.raises(TypeError, match="q must be"):
        pkg.cache_attention(cache, table, lens, q.float())
    with pytest.raises(ValueError, match="v must have shape"):
        pkg.KVCache4(cache.k, cache.v[:, :, :2].contiguous(), cache.scales)
