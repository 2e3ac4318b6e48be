"""The 8-bit cache's attention where numbers get large, small or far apart: one key with nearly all of the weight, scores
of any size, K and V scales at both ends of their range.  Against 64 bits on the values that the cache holds."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg

pytestmark = pytest.mark.gpu
FMTS = [pkg.HDP_CACHE_E4M3, pkg.HDP_CACHE_INT8]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _randn(shape, seed, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def _cache_of(k, v, fmt, seqs=1):
    """A cache of the rows k, v [keys][hkv][d], pages in no order; a table in which `seqs` sequences share the pages; and
    the rows as the cache holds them, in 64 bits."""
    keys, hkv, d = k.shape
    pages = (keys + 63) // 64
    cache = pkg.KVCache.empty(pages, hkv, d, fmt)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(keys)).int().cuda()[None]
    lens, cu = _i32([keys]), _i32([0, keys])
    pkg.cache_append(cache, table, lens, k.bfloat16().cuda(), v.bfloat16().cuda(), cu=cu)
    held = pkg.cache_read(cache, table, lens, keys, cu=cu)
    return cache, table.expand(seqs, pages).contiguous(), *(x.double() for x in held)


def _exact(q, k, v, scale, pos=None, blocks=None):
    """(o, lse, a, x) in 64 bits of rows q that see the keys up to their pos (all): a = sum p |v| of each output, x = each
    row's largest sum |q k| scale."""
    rows, hq, d = q.shape
    keys, hkv, _ = k.shape
    q = q.double().view(rows, hkv, hq // hkv, d)
    s = torch.einsum("rhgd,nhd->rhgn", q, k) * scale
    x = torch.einsum("rhgd,nhd->rhgn", q.abs(), k.abs()) * scale
    at = torch.arange(keys, device="cuda")
    if pos is not None:
        s = s.masked_fill(at > torch.as_tensor(pos, device="cuda")[:, None, None, None], -torch.inf)
    if blocks is not None:
        chosen = (blocks[..., None] == at // 64).any(2)  # [rows][hkv][keys]
        s = s.masked_fill(~chosen[:, :, None], -torch.inf)
    p = s.softmax(-1)
    o, a = (torch.einsum("rhgn,nhd->rhgd", p, y).reshape(rows, hq, d) for y in (v, v.abs()))
    x = x.masked_fill(torch.isneginf(s), 0).amax(-1).reshape(rows, hq)
    return o, s.logsumexp(-1).reshape(rows, hq).t(), a, x


def _check(o, lse, exact, same_scores=False):
    """Bounds, from the roundings alone; nothing is added for small probabilities.
    Scores: products of fp16 operands are exact; 128 fp32 additions and four multiplications are off by at most 2^-16 of
    x, and so is log2(e) in them: d_s.  Keys that are equal bit by bit have equal scores, so where all are (same_scores)
    d_s moves the LSE alone.
    P: d_s and exp2's 2^-22, and its rounding to fp16, half a step, 2^-11 of it (it is scaled into fp16's normal numbers).
    So o is off by (2^-11 + 2 d_s + 2^-18) a, and by half a bf16 step, 2^-8, of |o|; twice 2^-11 are allowed.  fp32 ends at
    2^-126 of the largest p s: not in reach of any case here.
    LSE: d_s, and 2^-20 for the logarithm and the sum, relative to max(1, |lse|)."""
    want, lse_want, a, x = exact
    ds = 2.0 ** -16 * x
    off = (lse.double() - lse_want).abs() - ds.t() - 2.0 ** -20 * lse_want.abs().clamp(min=1)
    assert (off <= 0).all(), f"lse over by {off.max()}"
    ds = 0 if same_scores else ds[..., None]
    err = (o.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -18 + 2 * ds) * a
    assert (err <= tol).all(), f"o over by {(err - tol).max()}: {o.double()[err > tol][:4].tolist()} for {want[err > tol][:4].tolist()}"


def _sink(n, hkv, d, weight, seed):
    """Keys of which the first takes `weight` of a row whose channel 0 is 8, with V = 0; the others' scores are close
    together and their V has a mean."""
    k, v = _randn((n, hkv, d), seed), _randn((n, hkv, d), seed + 1) + 0.5
    k[:, :, 0] = 0
    k[0] = 0
    v[0] = 0
    k[0, :, 0] = float(np.log(n * weight / (1 - weight)) / (8 * d ** -0.5))
    return k, v


def _sink_rows(rows, hq, d, seed):
    q = _randn((rows, hq, d), seed, 0.5)
    q[:, :, 0] = 8
    return q.bfloat16().cuda()


# ---------------------------------------------------------------- probabilities of any size

@pytest.mark.parametrize("weight", [0.9, 0.99, 0.999, 0.9999, 1 - 1e-7])
@pytest.mark.parametrize("fmt,hq,d", [(0, 8, 64), (1, 8, 64), (1, 32, 128)])
def test_one_key_with_nearly_all_of_the_weight(fmt, hq, d, weight):
    """160 sequences of 8 heads share 8,192 keys: a warp has most of a (sequence, head), the heavy key among it, and
    what the other keys leave in the output is 1 - weight of it."""
    n, seqs, hkv, scale = 8192, 160, 8, d ** -0.5
    k, v = _sink(n, hkv, d, weight, 3)
    cache, table, k, v = _cache_of(k, v, fmt, seqs)
    q = _sink_rows(seqs, hq, d, 5)
    o, lse = pkg.cache_attention(cache, table, _i32([n] * seqs), q)
    _check(o, lse, _exact(q, k, v, scale))


@pytest.mark.parametrize("fmt", FMTS)
def test_one_key_with_nearly_all_of_the_weight_drafts(fmt):
    """The same for three tokens of each sequence, 12 rows of a head's group."""
    n, seqs, new, hq, hkv, d = 4096, 100, 3, 16, 4, 128
    k, v = _sink(n, hkv, d, 0.9999, 7)
    cache, table, k, v = _cache_of(k, v, fmt, seqs)
    q = _sink_rows(seqs * new, hq, d, 8)
    o, lse = pkg.cache_attention(cache, table, _i32([n] * seqs), q, cu=_i32(np.arange(seqs + 1) * new))
    _check(o, lse, _exact(q, k, v, d ** -0.5, pos=np.tile(np.arange(n - new, n), seqs)))


@pytest.mark.parametrize("fmt,d", [(0, 128), (1, 64)])
def test_one_key_with_nearly_all_of_the_weight_chosen_blocks(fmt, d):
    n, seqs, hq, hkv = 4096, 60, 8, 2
    k, v = _sink(n, hkv, d, 0.9999, 9)
    cache, table, k, v = _cache_of(k, v, fmt, seqs)
    q = _sink_rows(seqs, hq, d, 10)
    blocks = torch.rand((seqs, hkv, 64), generator=torch.Generator().manual_seed(1)).topk(24, 2).indices
    blocks[:, :, 0] = 0  # the heavy key's
    blocks = blocks.sort(2).values.int().cuda()
    o, lse = pkg.cache_attention(cache, table, _i32([n] * seqs), q, blocks=blocks)
    _check(o, lse, _exact(q, k, v, d ** -0.5, blocks=blocks))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,d", [(1, 64), (4, 128), (12, 64)])
@pytest.mark.parametrize("heavy", [0, 70, 150])
def test_probabilities_over_the_range_of_fp32(fmt, hq, d, heavy):
    """Scores 0 to -85 in steps of one and V of one channel each, so an output is one probability: from 1 to 1e-37, in
    the heavy key's own block and in others."""
    n = 192
    k, v = torch.zeros((n, 1, d)), torch.zeros((n, 1, d))
    at = torch.arange(n)
    k[:, 0, 0] = -(20.0 + at % 64)  # whole numbers below 2^7; e4m3 rounds the upper ones
    k[heavy, 0, 0] = 0
    v[at, 0, at % 64] = 1
    v[heavy] = 0
    cache, table, k, v = _cache_of(k, v, fmt)
    q = torch.zeros((1, hq, d))
    q[:, :, 0] = torch.linspace(1, 0.7, hq) * d ** 0.5
    q = q.bfloat16().cuda()
    o, lse = pkg.cache_attention(cache, table, _i32([n]), q)
    exact = _exact(q, k, v, d ** -0.5)
    assert (exact[0][0, 0, 1:60] > 0).all() and exact[0][0, 0, :60].min() < 1e-30
    _check(o, lse, exact)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bits", [18, 24, 30, 60])
def test_one_channel_of_v_much_larger_in_one_block(fmt, bits):
    """2^bits in channel 0 of 64 keys: the other channels' outputs come from the other blocks."""
    n, seqs, hkv, d = 8192, 160, 8, 64
    k, v = _randn((n, hkv, d), 11), _randn((n, hkv, d), 12) + 0.5
    v[640:704, :, 0] = 2.0 ** bits
    cache, table, k, v = _cache_of(k, v, fmt, seqs)
    q = _randn((seqs, hkv, d), 13).bfloat16().cuda()
    o, lse = pkg.cache_attention(cache, table, _i32([n] * seqs), q)
    _check(o, lse, _exact(q, k, v, 0.125))


# ---------------------------------------------------------------- scores of any size

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("std", [1e7, 1e9, 1e15, 1e33])
@pytest.mark.parametrize("order,sign", [(1, 1), (1, -1), (-1, 1), (-1, -1)])
def test_large_scores_and_scales_far_apart(fmt, std, order, sign):
    """One key takes all: its V, whatever its block's scale and the others'."""
    d, n, hq = 64, 256, 2
    k, v = _randn((n, 1, d), 31), _randn((n, 1, d), 32)
    v *= torch.exp2((torch.arange(n) // 64 * 20.0 - 30) * order)[:, None, None]
    cache, table, k, v = _cache_of(k, v, fmt)
    q = (_randn((1, hq, d), 33, std) * sign).bfloat16().cuda()
    exact = _exact(q, k, v, 0.125)
    s = torch.einsum("hd,nd->hn", q[0].double(), k[:, 0]) * 0.125
    first, second = s.topk(2, 1).values.unbind(1)
    assert (first - second > 800 + 2 * 2.0 ** -16 * exact[3][0]).all()  # e^-800 is 0 in 64 bits; the scores' errors
    o, lse = pkg.cache_attention(cache, table, _i32([n]), q)
    _check(o, lse, exact, same_scores=True)  # the weight is 1 for one key, with no error


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [1.0, 1e4, 1e6, 3e7, 1e12, -1e7, -1e12, -3e30, -1e36])
@pytest.mark.parametrize("seqs,new", [(1, 1), (40, 1), (30, 3)])
def test_equal_keys_with_scores_of_any_size(fmt, size, seqs, new):
    """All keys are the same: the output is the mean of V, however the keys are split over warps and joined, and the
    V scales differ from block to block."""
    n, hq, hkv, d = 20011, 8, 2, 64
    k = _randn((1, hkv, d), 41).sign().expand(n, hkv, d)
    v = (_randn((n, hkv, d), 42) + 1) * torch.exp2(torch.arange(n) // 64 % 7 - 3.0)[:, None, None]
    cache, table, k, v = _cache_of(k, v, fmt, seqs)
    q = k[:1].float().repeat_interleave(hq // hkv, 1).expand(seqs * new, hq, d) * (size * torch.linspace(0.5, 1, hq, device="cuda")[:, None] / 8)
    q = q.bfloat16()
    cu = None if new == 1 else _i32(np.arange(seqs + 1) * new)
    o, lse = pkg.cache_attention(cache, table, _i32([n] * seqs), q, cu=cu)
    pos = np.tile(np.arange(n - new, n), seqs)
    _check(o, lse, _exact(q, k, v, 0.125, pos=pos), same_scores=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ks", [3e36, 3e-36])
@pytest.mark.parametrize("hq", [2, 12])
def test_keys_and_queries_at_opposite_ends_of_the_range(fmt, ks, hq):
    """|K| of 3e36 and q of 3e-37, or the other way round: scores of order one."""
    n, d = 200, 64
    k, v = _randn((n, 1, d), 51, ks), _randn((n, 1, d), 52)
    cache, table, k, v = _cache_of(k, v, fmt)
    q = _randn((1, hq, d), 53, 1 / ks).bfloat16().cuda()
    o, lse = pkg.cache_attention(cache, table, _i32([n]), q)
    _check(o, lse, _exact(q, k, v, 0.125))


def test_the_smallest_v_in_long_sequences():
    """V of 2^-121 (a scale of 2^-126) over 1.1M keys of equal weight: the mean, to the last bit but the roundings."""
    n, seqs, hkv, d = 1100000, 152, 8, 64
    k = torch.zeros((n, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.full((n, hkv, d), 1.5 * 2.0 ** -121, dtype=torch.bfloat16, device="cuda")
    pages = (n + 63) // 64
    cache = pkg.KVCache.empty(pages, hkv, d, 1)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    pkg.cache_append(cache, table, _i32([n]), k, v, cu=_i32([0, n]))
    assert (cache.scales[:, :, 1] == 2.0 ** -126).all()
    o, lse = pkg.cache_attention(cache, table.expand(seqs, pages).contiguous(), _i32([n] * seqs),
                                 torch.ones((seqs, hkv, d), dtype=torch.bfloat16, device="cuda"))
    # probabilities are powers of two here and codes equal: sums of 1.1M of them in fp32 are off by 2^-24 an addition at
    # most, one for the 64 keys of a step, 2^-24 * 17188 < 2^-9; then half a bf16 step
    assert ((o.double() / (1.5 * 2.0 ** -121) - 1).abs() <= 2.0 ** -8 + 2.0 ** -9).all()
    assert ((lse.double() - np.log(n)).abs() <= 2.0 ** -9).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_read_at_the_smallest_scales(fmt, d):
    """Every code at scales of 2^-126 to 2^-122 and 2^119: the nearest bf16 to code * scale, exact from 2^-124 on."""
    exponents = [-126, -125, -124, -123, -122, 119]
    pages = len(exponents)
    cache = pkg.KVCache.empty(pages, 1, d, fmt)
    codes = torch.arange(64 * d, device="cuda").view(64, d) % 254
    codes = (codes - 127).to(torch.int8).view(torch.uint8) if fmt else torch.where(codes < 127, codes, codes + 1).to(torch.uint8)
    cache.k.copy_(codes.expand(pages, 1, 64, d))
    at = torch.tensor([16 * (t // 2 % 4) + 4 * (t // 16) + 2 * (t // 8 % 2) + t % 2 for t in range(64)], device="cuda")
    cache.v[..., at] = codes.t().expand(pages, 1, d, 64)
    cache.scales.copy_(torch.tensor([2.0 ** e for e in exponents], device="cuda")[:, None, None].expand(pages, 1, 2))
    n = 64 * pages
    k, v = pkg.cache_read(cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None], _i32([n]), n, cu=_i32([0, n]))
    value = codes.view(torch.int8).double() if fmt else codes.view(torch.float8_e4m3fn).double()
    want = (value[None] * cache.scales[:, 0, :1, None].double()).view(n, 1, d)
    step = torch.where(want.abs() < 2.0 ** -126, 2.0 ** -133, 0.0)  # of bf16's subnormal numbers
    exact = torch.tensor([bool(fmt) or e >= -124 for e in exponents], device="cuda").repeat_interleave(64)[:, None, None]
    for got in (k.double(), v.double()):
        assert torch.equal(got[exact.expand_as(got)], want[exact.expand_as(got)])
        assert ((got - want).abs() <= step / 2).all()
