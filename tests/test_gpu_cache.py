"""The 8-bit key/value cache on the GPU against the fp64 oracle: codes, scales, bounds and chosen blocks exactly,
attention within bounds that are derived from its roundings (see _check_attention)."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from oracle import kv_cache as kc

pytestmark = pytest.mark.gpu
FMTS = [pkg.HDP_CACHE_E4M3, pkg.HDP_CACHE_INT8]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def _table(lens, rng, spare=0, columns=0):
    """Pages in no order, and a table whose unused entries are out of range."""
    need = [max(0, (l + 63) // 64) for l in lens]
    pages = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), columns, 1)), -7, np.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = pages[at:at + m]
        at += m
    return max(1, len(pages)), table


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _filled(pages, hkv, d, fmt, byte=0x5a):
    c = pkg.KVCache.empty(pages, hkv, d, fmt)
    for t in (c.k, c.v, c.bounds):
        t.fill_(byte)
    c.scales.fill_(3.0)
    return c


def _oracle(cache):
    return kc.Cache.of(cache.k.cpu().numpy(), cache.v.cpu().numpy(), cache.scales.cpu().numpy(),
                       cache.bounds.cpu().numpy(), cache.format)


def _random_cache(lens, hkv, d, fmt, seed, spare=1):
    """A cache written through the library, and the oracle's view of its bytes."""
    rng = np.random.default_rng(seed)
    pages, table = _table(lens, rng, spare)
    cache = _filled(pages, hkv, d, fmt)
    rows = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = _bf16((rows, hkv, d), seed), _bf16((rows, hkv, d), seed + 1)
    k[:, :, : d // 8] *= 6
    v *= torch.exp2(torch.arange(rows) % 7 - 3.0).to(torch.bfloat16)[:, None, None]
    if rows:
        pkg.cache_append(cache, _i32(table), _i32(lens), k.cuda(), v.cuda(), cu=_i32(cu))
        pkg.hdp_device_status()
    return cache, table, _oracle(cache)


def _check_attention(o, lse, ref, what=""):
    """Bounds, from the roundings alone.
    Scores: products of fp16 operands are exact, 128 fp32 additions and four multiplications are off by at most 2^-16 of
    x = the row's largest sum |q k| scale (128 * 2^-23, truncating); the query row's shift loses at most 2^-39 of its
    largest element.  Call that d_s.
    P: d_s and exp2's error, and its rounding to fp16: half a step, 2^-11, for P >= 2^-14, 2^-25 absolute below, each
    once more for the product with its block's power of two.  P is held relative to 2^M, M a whole number with
    2^M <= 2 max(p s), so the absolute part sums to at most 2 * 2^-25 * 2 max(p s) |code| over the keys with
    p s < 2^-13 max(p s): 2^-23 z.  A P of 2^-14 or more is a normal number in fp16, and its product with the power of
    two is exact or falls under the absolute part.
    So o is off by (2^-11 + 2 d_s + 2^-18) a + 2^-23 z with a = sum p |v|, and by half a bf16 step, 2^-8, of |o|; twice
    2^-11 are allowed.  LSE: d_s, and 2^-20 for the logarithm and the sum, relative to max(1, |lse|)."""
    o_ref, lse_ref, a, x, z = ref
    o, lse = _f64(o), _f64(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(lse_ref)), what
    seen = ~np.isneginf(lse_ref)
    ds = 2.0 ** -16 * x
    err = np.abs(np.where(seen, lse, 0) - np.where(seen, lse_ref, 0))
    over = err - ds - 2.0 ** -20 * np.maximum(1, np.abs(np.where(seen, lse_ref, 0)))
    assert over.max(initial=0.0) <= 0, f"{what}: lse {err.max()}"
    tol = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -10 + 2.0 ** -18 + 2 * ds.T[:, :, None]) * a + 2.0 ** -23 * z
    bad = np.abs(o - o_ref) - tol
    assert np.isfinite(o).all(), what
    assert bad.max(initial=0.0) <= 0, f"{what}: o over by {bad.max()}, |o| {np.abs(o_ref).max()}"
    assert (o[~seen.T] == 0).all()


# ---------------------------------------------------------------- writing and reading

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv", [(128, 8), (64, 3)])
def test_append_matches_the_oracle_code_for_code(fmt, d, hkv):
    """Prompts, chunks that end and begin inside blocks, single tokens and steps that enlarge scales; pages that no
    call names keep their bytes, and so do the rows behind the last sequence's."""
    rng = np.random.default_rng(d + fmt)
    final = [200, 1, 64, 129, 65, 40]
    pages, table = _table(final, rng, spare=3, columns=6)
    cache = _filled(pages, hkv, d, fmt)
    start = _oracle(cache)
    ref = kc.Cache.of(cache.k.cpu().numpy(), cache.v.cpu().numpy(), cache.scales.cpu().numpy(),
                      cache.bounds.cpu().numpy(), fmt)
    steps = [([100, 0, 63, 128, 1, 0], 1.0), ([30, 0, 1, 0, 33, 7], 3.0), ([1, 1, 0, 1, 1, 1], 0.1),
             ([69, 0, 0, 0, 30, 32], 40.0)]
    lens, seed = np.zeros(6, np.int64), 5
    for new, std in steps:
        lens = lens + new
        cu = np.concatenate([[0], np.cumsum(new)])
        rows = int(cu[-1]) + 3  # three rows of no sequence behind
        k, v = _bf16((rows, hkv, d), seed, std), _bf16((rows, hkv, d), seed + 1, std)
        k[0, 0, 0] = 0
        seed += 2
        pkg.cache_append(cache, _i32(table), _i32(lens), k.cuda(), v.cuda(), cu=_i32(cu))
        pkg.hdp_device_status()
        ref.append(table, lens, _f64(k), _f64(v), cu)
        got = _oracle(cache)
        for name in ("scales", "bounds", "k", "v"):
            x, y = getattr(got, name), getattr(ref, name)
            assert np.array_equal(x, y), f"{name} after {new}: {np.count_nonzero(x != y)} of {x.size} differ"
    unused = sorted(set(range(pages)) - set(table[table >= 0].tolist()))
    assert unused and np.array_equal(got.k[unused], start.k[unused]) and np.array_equal(got.scales[unused], start.scales[unused])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_one_for_each_sequence(fmt, d):
    """cu None: 130 steps of three sequences of different lengths, bit for bit as the oracle, and written again after
    two tokens are taken back."""
    rng = np.random.default_rng(7)
    pages, table = _table([140, 150, 160], rng)
    cache = _filled(pages, 2, d, fmt)
    ref = _oracle(cache)
    lens = np.array([3, 60, 31])
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = _bf16((94, 2, d), 1), _bf16((94, 2, d), 2)
    pkg.cache_append(cache, _i32(table), _i32(lens), k.cuda(), v.cuda(), cu=_i32(cu))
    ref.append(table, lens, _f64(k), _f64(v), cu)
    ks, vs = _bf16((130, 3, 2, d), 3), _bf16((130, 3, 2, d), 4)
    ks[40] *= 100
    for s in range(130):
        lens = lens + (1 if s != 70 else -1)  # step 70 overwrites the last two tokens' places
        pkg.cache_append(cache, _i32(table), _i32(lens), ks[s].cuda(), vs[s].cuda())
        ref.append(table, lens, _f64(ks[s]), _f64(vs[s]), [0, 1, 2, 3])
    got = _oracle(cache)
    for name in ("scales", "bounds", "k", "v"):
        assert np.array_equal(getattr(got, name), getattr(ref, name)), name


@pytest.mark.parametrize("fmt", FMTS)
def test_extreme_values(fmt):
    """Zeros, the smallest and largest bf16 numbers and values at the codes' borders; an infinity or NaN makes its
    block and head NaN and nothing else, until the block is begun again."""
    d, hkv = 64, 2
    cache = _filled(3, hkv, d, fmt)
    table, lens = [[2, 0, 1]], [140]
    x = _bf16((140, hkv, d), 9)
    x[:64, 0] = 0
    x[:64, 1] = torch.tensor([2.0 ** -133, -2.0 ** -126, 2.0 ** -120, 0]).to(torch.bfloat16).repeat(16)
    x[64:128, 0] = torch.tensor([3.38e38, -3.38e38, 1e38, 1e30]).to(torch.bfloat16).repeat(16)
    x[64:128, 1] = torch.tensor([127.0, 127.5, 448.0, -449.0]).to(torch.bfloat16).repeat(16)
    ref = _oracle(cache)
    pkg.cache_append(cache, _i32(table), _i32(lens), x.cuda(), x.flip(0).contiguous().cuda(), cu=_i32([0, 140]))
    ref.append(table, lens, _f64(x), _f64(x.flip(0)), [0, 140])
    got = _oracle(cache)
    for name in ("scales", "bounds", "k", "v"):
        assert np.array_equal(getattr(got, name), getattr(ref, name)), name
    bad = _bf16((1, hkv, d), 10)
    bad[0, 1, 5] = float("nan") if fmt else float("inf")
    ok = _bf16((1, hkv, d), 11)
    pkg.cache_append(cache, _i32(table), _i32([141]), bad.cuda(), ok.cuda())
    k, v = pkg.cache_read(cache, _i32(table), _i32([141]), 141, cu=_i32([0, 141]))
    nan = torch.isnan(k).cpu()
    assert nan[128:, 1].all() and not nan[:128].any() and not nan[:, 0].any() and not torch.isnan(v).any()
    pkg.cache_append(cache, _i32(table), _i32([142]), ok.cuda(), ok.cuda())  # a later row does not hide it
    assert torch.isnan(cache.scales[1, 1, 0]) and not torch.isnan(cache.scales[1, 0]).any()
    pkg.cache_append(cache, _i32(table), _i32([129]), ok.cuda(), ok.cuda())  # the block begins again
    assert torch.isfinite(cache.scales).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv", [(128, 2), (64, 5)])
def test_read_gives_code_times_scale(fmt, d, hkv):
    lens = [130, 0, 64, 1, 63, 200]
    cache, table, ref = _random_cache(lens, hkv, d, fmt, 3)
    for new in ([130, 0, 64, 1, 63, 200], [70, 0, 1, 1, 0, 136]):
        cu = np.concatenate([[0], np.cumsum(new)])
        rows = int(cu[-1])
        k = torch.full((rows + 2, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
        v = torch.full_like(k, 7.0)
        pkg.hdp_cache_read(cache, _i32(table), _i32(lens), k, v, cu=_i32(cu))
        pkg.hdp_device_status()
        want = [ref.sequence(table[i], l) for i, l in enumerate(lens)]
        for w, got in ((0, k), (1, v)):
            x = np.concatenate([want[i][w][l - m:] for i, (l, m) in enumerate(zip(lens, new))])
            assert np.array_equal(_f64(got)[:rows], x)
            assert (got[rows:] == 7).all()
    # single tokens, one of them of an empty sequence (zeros)
    k, v = pkg.cache_read(cache, _i32(table), _i32(lens), 6)
    for i, l in enumerate(lens):
        kr, vr = ref.sequence(table[i], l)
        assert np.array_equal(_f64(k[i]), kr[-1] if l else np.zeros((hkv, d)))
        assert np.array_equal(_f64(v[i]), vr[-1] if l else np.zeros((hkv, d)))
    # more rows than tokens: the first ones read as zeros
    k, v = pkg.cache_read(cache, _i32(table[:1]), _i32([130]), 133, cu=_i32([0, 133]))
    assert (k[:3] == 0).all() and (v[:3] == 0).all() and np.array_equal(_f64(k[3:]), ref.sequence(table[0], 130)[0])


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_before_the_sequence_and_of_empty_sequences_are_not_written(fmt):
    cache = _filled(3, 2, 64, fmt)
    ref = _oracle(cache)
    table = np.array([[1, -7], [2, 0]], np.int32)
    k, v = _bf16((8, 2, 64), 1), _bf16((8, 2, 64), 2)
    pkg.cache_append(cache, _i32(table), _i32([0, 3]), k.cuda(), v.cuda(), cu=_i32([0, 2, 8]))
    pkg.cache_append(cache, _i32(table), _i32([0, 4]), k[:2].cuda(), v[:2].cuda())  # one of an empty sequence
    pkg.hdp_device_status()
    ref.append(table[1:], [3], _f64(k[5:]), _f64(v[5:]), [0, 3])  # the last three of six rows
    ref.append(table[1:], [4], _f64(k[1:2]), _f64(v[1:2]), [0, 1])
    got = _oracle(cache)
    for name in ("scales", "bounds", "k", "v"):
        assert np.array_equal(getattr(got, name), getattr(ref, name)), name


def test_page_shared_by_two_sequences_and_rows_written_twice():
    """A common prefix page read by both sequences; the second half of a draft overwritten with other tokens reads as
    those, within the larger scale that the first left."""
    cache = pkg.KVCache.empty(4, 1, 64, 1)
    table = _i32([[0, 1], [0, 2]])
    prefix = _bf16((64, 1, 64), 1).cuda()
    pkg.cache_append(cache, table[:1], _i32([64]), prefix, prefix, cu=_i32([0, 64]))
    tail = _bf16((2, 1, 64), 2).cuda()
    pkg.cache_append(cache, table, _i32([65, 65]), tail, tail)
    k, _ = pkg.cache_read(cache, table, _i32([65, 65]), 130, cu=_i32([0, 65, 130]))
    assert torch.equal(k[:64], k[65:129]) and not torch.equal(k[64], k[129])
    pkg.cache_append(cache, table, _i32([66, 66]), tail * 64, tail * 64)
    pkg.cache_append(cache, table, _i32([66, 66]), tail, tail)
    k, _ = pkg.cache_read(cache, table, _i32([66, 66]), 2)
    step = cache.scales[[1, 2], :, 0][..., None]
    assert ((k.float() - tail.float()).abs() <= step / 2).all() and (step > 0.25).all()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 4, 64), (6, 2, 128), (32, 1, 64), (9, 1, 128), (2, 2, 128),
                                      (24, 8, 64)])
def test_one_token_of_each_sequence(fmt, hq, hkv, d):
    lens = [1, 64, 65, 0, 128, 1000, 63, 2, 319]
    cache, table, ref = _random_cache(lens, hkv, d, fmt, 11)
    q = _bf16((len(lens), hq, d), 21)
    cu = np.arange(len(lens) + 1)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    pkg.hdp_device_status()
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, d ** -0.5), f"{hq}/{hkv} d={d}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (5, 1, 128), (32, 2, 64)])
def test_several_tokens_of_each_sequence(fmt, hq, hkv, d):
    """1 to 70 rows a sequence, some with more rows than tokens, one with none; the rows behind the last sequence's
    keep what their outputs held."""
    lens, new = [70, 300, 5, 64, 0, 129, 3], [70, 5, 1, 2, 3, 0, 6]
    cache, table, ref = _random_cache(lens, hkv, d, fmt, 13)
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1])
    q = _bf16((rows + 4, hq, d), 22, 2.0)
    o = torch.full((rows + 4, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, rows + 4), 7.0, device="cuda")
    ws = torch.empty(pkg.hdp_cache_attention_workspace_bytes(cache, hq), dtype=torch.uint8, device="cuda").fill_(0xff)
    pkg.hdp_cache_attention(cache, _i32(table), _i32(lens), q.cuda(), d ** -0.5, ws, o, lse, cu=_i32(cu))
    pkg.hdp_device_status()
    _check_attention(o[:rows], lse[:, :rows], ref.attention(table, lens, _f64(q[:rows]), cu, d ** -0.5))
    assert (o[rows:] == 7).all() and (lse[:, rows:] == 7).all()


@pytest.mark.parametrize("fmt,hq,hkv,d,lens", [
    (0, 4, 1, 128, [20000]), (1, 1, 1, 64, [33333]), (0, 16, 2, 64, [9000, 17, 4097]), (1, 32, 8, 128, [3000] * 5)])
def test_long_sequences_are_split_and_joined(fmt, hq, hkv, d, lens):
    cache, table, ref = _random_cache(lens, hkv, d, fmt, 17)
    q = _bf16((len(lens), hq, d), 23)
    args = (cache, _i32(table), _i32(lens), q.cuda())
    o, lse = pkg.cache_attention(*args)
    pkg.hdp_device_status()
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), np.arange(len(lens) + 1), d ** -0.5))
    for _ in range(3):
        o2, lse2 = pkg.cache_attention(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt,hq,hkv,d,lens,new", [
    (1, 16, 8, 64, [600000, 130, 250001, 64, 7000], 1), (0, 8, 8, 128, [200000, 100100], 1), (0, 8, 4, 64, [400000, 90000], 5)])
def test_runs_whose_ends_are_handed_out(fmt, hq, hkv, d, lens, new):
    """More than 20 blocks for each warp of the device: pieces of runs go to whoever comes free, with the same result
    every time; against PyTorch in 64 bits on the values that the cache holds."""
    g = torch.Generator(device="cuda").manual_seed(3)
    need = [(l + 63) // 64 for l in lens]
    pages = sum(need)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    for i, m in enumerate(need):
        table[i, :m] = order[sum(need[:i]):sum(need[:i]) + m]
    cache = pkg.KVCache.empty(pages, hkv, d, fmt)
    for t in (cache.k, cache.v):
        x = torch.randint(-90, 91, t.shape, generator=g, device="cuda", dtype=torch.int8)
        t.copy_(x.view(torch.uint8) if fmt else (x.float() * 3).to(torch.float8_e4m3fn).view(torch.uint8))
    cache.scales.copy_(torch.exp2(torch.randint(-8, -5, cache.scales.shape, generator=g, device="cuda").float()))
    rows = len(lens) * new
    q = torch.randn((rows, hq, d), generator=g, device="cuda").bfloat16()
    cu = None if new == 1 else _i32(np.arange(len(lens) + 1) * new)
    dl = _i32(lens)
    o, lse = pkg.cache_attention(cache, table, dl, q, cu=cu)
    pkg.hdp_device_status()
    for _ in range(4):
        o2, lse2 = pkg.cache_attention(cache, table, dl, q, cu=cu)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # captured and replayed, beside an eager call on another stream, and with other queries in place
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    q_in = q.clone()
    with torch.cuda.graph(graph):
        og, lg = pkg.cache_attention(cache, table, dl, q_in, cu=cu)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        o2, lse2 = pkg.cache_attention(cache, table, dl, q, cu=cu, stream=side)
        side.synchronize()
        torch.cuda.current_stream().synchronize()
        assert torch.equal(o, og) and torch.equal(lse, lg) and torch.equal(o, o2) and torch.equal(lse, lse2)
    q_in.copy_(-q)
    graph.replay()
    o2, lse2 = pkg.cache_attention(cache, table, dl, -q, cu=cu)
    assert torch.equal(o2, og) and torch.equal(lse2, lg) and not torch.equal(o, og)
    whole = _i32(np.concatenate([[0], np.cumsum(lens)]))
    k, v = pkg.cache_read(cache, table, dl, sum(lens), cu=whole)
    grp = hq // hkv
    for i, l in enumerate(lens):
        for h in range(hkv):
            kh, vh = (x[sum(lens[:i]):sum(lens[:i]) + l, h].double() for x in (k, v))
            for r in range(new):
                seen = l - new + 1 + r
                qq = q[i * new + r, h * grp:(h + 1) * grp].double()
                sc = qq @ kh[:seen].T * d ** -0.5
                p = sc.softmax(1)
                ref, a = p @ vh[:seen], p @ vh[:seen].abs()
                ds = 2.0 ** -16 * (qq.abs() @ kh[:seen].abs().T * d ** -0.5).amax(1)
                err = (o[i * new + r, h * grp:(h + 1) * grp].double() - ref).abs()
                # as in _check_attention, with scales s of 2^-8 to 2^-6 and codes up to 270: where p s < 2^-13 max(p s),
                # p < 2^-11 max p
                top = p.amax(1, keepdim=True)
                z = top * 2.0 ** -6 * (p < 2.0 ** -11 * top).double().sum(1, keepdim=True) * 270
                tol = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -18 + 2 * ds[:, None]) * a + 2.0 ** -23 * z
                assert (err <= tol).all(), (i, h, r, float((err - tol).max()))
                want = torch.logsumexp(sc, 1)
                got = lse[h * grp:(h + 1) * grp, i * new + r].double()
                assert ((got - want).abs() <= ds + 2.0 ** -20 * want.abs().clamp(min=1)).all()


def _poisoned(cache, table, lens, q, scale, cu=None, blocks=None):
    """The call with a workspace and outputs of garbage (0x7f7f7f7f is a large float)."""
    rows, hq, d = q.shape
    ws = torch.full((pkg.hdp_cache_attention_workspace_bytes(cache, hq),), 0x7f, dtype=torch.uint8, device="cuda")
    o, lse = torch.full_like(q, 1e30), torch.full((hq, rows), 1e30, device="cuda")
    pkg.hdp_cache_attention(cache, table, lens, q, scale, ws, o, lse, cu=cu, blocks=blocks)
    pkg.hdp_device_status()
    return o, lse


@pytest.mark.parametrize("blocks", [3048, 3053, 3061, 3090])
def test_a_last_run_of_few_blocks(blocks):
    """On 152 SMs the last warp with work has 1 to 3 blocks, fewer than its copies run ahead: it goes on to pieces of
    other runs before its own is done."""
    length, hkv, d = blocks * 64 - 3, 8, 64
    g = torch.Generator(device="cuda").manual_seed(blocks)
    cache = pkg.KVCache.empty(blocks, hkv, d, 1)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(-90, 91, t.shape, generator=g, device="cuda", dtype=torch.int8).view(torch.uint8))
    cache.scales.fill_(2.0 ** -7)
    table = torch.randperm(blocks, generator=g, device="cuda").int()[None]
    q = torch.randn((1, hkv, d), generator=g, device="cuda").bfloat16()
    o, lse = _poisoned(cache, table, _i32([length]), q, 0.125)
    k, v = pkg.cache_read(cache, table, _i32([length]), length, cu=_i32([0, length]))
    for h in range(hkv):
        sc = k[:, h].double() @ q[0, h].double() * 0.125
        p = sc.softmax(0)
        want = torch.logsumexp(sc, 0)
        ds = 2.0 ** -16 * (k[:, h].double().abs() @ q[0, h].double().abs() * 0.125).max()
        assert (lse[h, 0].double() - want).abs() <= ds + 2.0 ** -20 * want.abs()
        # as in _check_attention; all keys below 2^-13 of the largest probability or not, one scale
        a, z = p @ v[:, h].double().abs(), p.max() * (p < 2.0 ** -13 * p.max()).sum() * 90 * 2.0 ** -7
        ref = p @ v[:, h].double()
        assert ((o[0, h].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -18 + 2 * ds) * a + 2.0 ** -23 * z).all()


@pytest.mark.parametrize("count", [200, 203, 207, 252])
def test_a_last_run_of_few_list_entries(count):
    lens = [int(x) for x in np.random.default_rng(count).integers(0, 140, 165)]
    lens[-1] = 65
    cache, table, ref = _random_cache(lens, 4, 64, 0, 7)
    q = _bf16((165, 48, 64), 8)
    blocks = np.full((165, 4, count), -1, np.int32)
    blocks[:, :, 0], blocks[:, :, 1], blocks[:, :, count - 1] = 0, 1, 2
    blocks[:, 1, 0] = -1
    o, lse = _poisoned(cache, _i32(table), _i32(lens), q.cuda(), 0.125, blocks=_i32(blocks))
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), np.arange(166), 0.125, blocks))


def test_many_rows_of_one_sequence():
    """A prompt's rows all at once: 88 tiles of query rows over one cache."""
    lens, new = [700, 40], [700, 3]
    cache, table, ref = _random_cache(lens, 2, 64, 1, 15)
    cu = np.array([0, 700, 703])
    q = _bf16((703, 4, 64), 16)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(cu))
    pkg.hdp_device_status()
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, 0.125))


def test_many_sequences_against_one_at_a_time():
    """700 sequences: what a sequence gets does not depend on its neighbours beyond the order of its sums."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 200, 700)]
    cache, table, ref = _random_cache(lens, 2, 64, 1, 19)
    q = _bf16((700, 4, 64), 24)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    pkg.hdp_device_status()
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), np.arange(701), 0.125))


@pytest.mark.parametrize("fmt", FMTS)
def test_scales_far_apart_and_large_scores(fmt):
    """V blocks 2^60 apart, in either order, and scores of several hundred: the largest products decide."""
    d, lens = 64, [256]
    for order in (1, -1):
        cache = _filled(4, 1, d, fmt)
        k, v = _bf16((256, 1, d), 31), _bf16((256, 1, d), 32)
        v = (v.float() * torch.exp2((torch.arange(256) // 64 * 20.0 - 30) * order)[:, None, None]).to(torch.bfloat16)
        pkg.cache_append(cache, _i32([[3, 1, 0, 2]]), _i32(lens), k.cuda(), v.cuda(), cu=_i32([0, 256]))
        ref = _oracle(cache)
        for std in (1.0, 60.0, 1e-20, 1e15):
            q = _bf16((1, 2, d), 33, std)
            o, lse = pkg.cache_attention(cache, _i32([[3, 1, 0, 2]]), _i32(lens), q.cuda())
            want = ref.attention([[3, 1, 0, 2]], lens, _f64(q), [0, 1], 0.125)
            if std < 1e10:
                _check_attention(o, lse, want, f"std {std}")
            else:  # one key takes all
                assert torch.isfinite(o).all() and np.allclose(_f64(lse), want[1], rtol=2 ** -16)


def test_nan_reaches_the_rows_that_see_it_and_no_others():
    d, fmt = 64, pkg.HDP_CACHE_E4M3
    lens = [130, 100]
    cache, table, _ = _random_cache(lens, 2, d, fmt, 41)
    cache.k[table[0][2], :, 2:] = 0x7f  # NaN codes behind the newest token
    cache.v[table[0][2]] = torch.where(torch.tensor(kc.v_order().argsort() >= 2, device="cuda"), 0x7f, cache.v[table[0][2]].int()).to(torch.uint8)
    q = _bf16((2, 4, d), 42)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    cache.scales[table[1][0], 1, 0] = float("nan")
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    assert torch.isnan(o[1, 2:]).all() and torch.isnan(lse[2:, 1]).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[1, :2]).all()
    cache.scales[table[1][0], 1] = torch.tensor([1.0, float("nan")])
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    assert torch.isnan(o[1, 2:]).all() and torch.isfinite(lse).all()
    q[0, 1, 3] = float("nan")
    cache.scales[table[1][0], 1] = 1.0
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[1, 0]) and torch.isnan(o).sum() == d


def test_a_pool_larger_than_4_gib():
    """Pages whose byte offsets pass 2^32, in K and V."""
    hkv, d, pages = 8, 128, 70000
    cache = pkg.KVCache.empty(pages, hkv, d, 1)
    table = np.array([[69999, 3, 65537, 69998]], np.int32)
    k, v = _bf16((200, hkv, d), 51), _bf16((200, hkv, d), 52)
    pkg.cache_append(cache, _i32(table), _i32([200]), k.cuda(), v.cuda(), cu=_i32([0, 200]))
    used = torch.tensor(table[0].astype(np.int64), device="cuda")
    ref = kc.Cache.of(*(x[used].cpu().numpy() for x in (cache.k, cache.v, cache.scales, cache.bounds)), 1)
    own = kc.Cache(4, hkv, d, 1)
    own.append([[0, 1, 2, 3]], [200], _f64(k), _f64(v), [0, 200])
    assert np.array_equal(ref.k, own.k * (own.scales[..., :1, None] > 0)) and np.array_equal(ref.scales, own.scales)
    q = _bf16((1, 8, d), 53)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32([200]), q.cuda())
    _check_attention(o, lse, own.attention([[0, 1, 2, 3]], [200], _f64(q), [0, 1], d ** -0.5))
    b = pkg.cache_select(cache, _i32(table), _i32([200]), q.cuda(), 3)
    assert np.array_equal(b.cpu().numpy(), own.select([[0, 1, 2, 3]], [200], _f64(q), [0, 1], 3, 1, 1))
    kr, vr = pkg.cache_read(cache, _i32(table), _i32([200]), 200, cu=_i32([0, 200]))
    assert np.array_equal(_f64(vr), own.sequence([0, 1, 2, 3], 200)[1])
    pkg.hdp_device_status()


# ---------------------------------------------------------------- choosing blocks, attention over them

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,hkv,d,count,first,last", [(32, 8, 128, 3, 1, 1), (4, 4, 64, 1, 0, 0), (32, 1, 128, 5, 2, 3),
                                                       (6, 2, 64, 8, 0, 2), (256, 2, 64, 4, 1, 1)])
def test_select_matches_the_oracle(fmt, hq, hkv, d, count, first, last):
    lens, new = [1000, 64, 0, 65, 700, 2000], [1, 2, 1, 0, 5, 3]
    cache, table, ref = _random_cache(lens, hkv, d, fmt, 61)
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1])
    q = _bf16((rows + 1, hq, d), 62)
    q[1] = 0
    q[2, 0, 0] = float("inf")
    blocks = torch.full((rows + 1, hkv, count), -9, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkg.hdp_cache_select_workspace_bytes(cache, _i32(table), rows + 1), dtype=torch.uint8, device="cuda")
    pkg.hdp_cache_select(cache, _i32(table), _i32(lens), q.cuda(), first, last, ws, blocks, cu=_i32(cu))
    pkg.hdp_device_status()
    want = ref.select(table, lens, _f64(q[:rows]), cu, count, first, last)
    assert np.array_equal(blocks[:rows].cpu().numpy(), want)
    assert (blocks[rows:] == -9).all()


def test_select_ties_take_the_lower_block_and_nan_the_first_place():
    d, n = 64, 100 * 64
    cache = pkg.KVCache.empty(100, 1, d, 1)
    table = np.arange(100, dtype=np.int32)[None]
    x = _bf16((64, 1, d), 71).repeat(100, 1, 1)  # every block the same
    pkg.cache_append(cache, _i32(table), _i32([n]), x.cuda(), x.cuda(), cu=_i32([0, n]))
    q = _bf16((1, 2, d), 72).cuda()
    b = pkg.cache_select(cache, _i32(table), _i32([n]), q, 7, keep_first=0, keep_last=2)
    assert b[0, 0].tolist() == [0, 1, 2, 3, 4, 98, 99]
    cache.scales[50, 0, 0] = float("nan")
    b = pkg.cache_select(cache, _i32(table), _i32([n]), q, 3, keep_first=0, keep_last=1)
    assert b[0, 0].tolist() == [0, 50, 99]


@pytest.mark.parametrize("blocks,count", [(4096, 100), (4097, 1000), (32768, 256), (33000, 300), (70000, 5000)])
def test_select_among_many_blocks(blocks, count):
    """Every size class of the search; scores with many ties."""
    d = 64
    g = torch.Generator().manual_seed(blocks)
    bounds = torch.randint(-3, 4, (blocks, 1, 2, d), generator=g).sort(2).values.to(torch.int8)
    scales = torch.exp2(torch.randint(-2, 1, (blocks, 1, 2), generator=g).float())
    cache = pkg.KVCache(torch.empty((blocks, 1, 64, d), dtype=torch.uint8, device="cuda"),
                        torch.empty((blocks, 1, d, 64), dtype=torch.uint8, device="cuda"), scales.cuda(), bounds.cuda(), 1)
    table = torch.randperm(blocks, generator=g).to(torch.int32)[None]
    q = torch.randint(-1, 2, (1, 2, d), generator=g).to(torch.bfloat16)
    got = pkg.cache_select(cache, table.cuda(), _i32([blocks * 64 - 5]), q.cuda(), count, keep_first=3, keep_last=4)
    pkg.hdp_device_status()
    x = torch.round(q[0].double() * 64).long()  # largest magnitude 1: 2^-6 is the smallest power with 1 <= 127 * it
    bd = bounds[table[0].long(), 0].long()
    score = (bd[:, 1] @ x.clamp(min=0).sum(0) + bd[:, 0] @ x.clamp(max=0).sum(0)).float() * scales[table[0].long(), 0, 0]
    score[:3] = score[-4:] = float("inf")
    want = score.sort(descending=True, stable=True).indices[:count].sort().values
    assert torch.equal(got[0, 0].cpu().long(), want)


@pytest.mark.parametrize("blocks,rows,count", [(3000, 30, 100), (20000, 30, 512), (1500, 140, 64), (6000, 30, 600)])
def test_select_for_many_rows(blocks, rows, count):
    """Rows enough to fill the device: scores and choice in one kernel, 1 to 8 CTAs a row; a count beyond what they
    take goes through memory."""
    d = 64
    g = torch.Generator().manual_seed(blocks)
    bounds = torch.randint(-90, 91, (blocks, 1, 2, d), generator=g).sort(2).values.to(torch.int8)
    scales = torch.exp2(torch.randint(-1, 1, (blocks, 1, 2), generator=g).float())
    cache = pkg.KVCache(torch.empty((blocks, 1, 64, d), dtype=torch.uint8, device="cuda"),
                        torch.empty((blocks, 1, d, 64), dtype=torch.uint8, device="cuda"), scales.cuda(), bounds.cuda(), 0)
    table = torch.randperm(blocks, generator=g).to(torch.int32)[None]
    q = torch.randint(-127, 128, (rows, 3, d), generator=g).to(torch.bfloat16)
    q[:, 0, 0] = 127  # whole numbers that the rounding of q leaves alone
    length = blocks * 64 - 20
    got = pkg.cache_select(cache, table.cuda(), _i32([length]), q.cuda(), count, cu=_i32([0, rows]), keep_first=2, keep_last=3)
    pkg.hdp_device_status()
    bd, sc = bounds[table[0].long(), 0].long(), scales[table[0].long(), 0, 0]
    for r in range(rows):
        have = (length - rows + r) // 64 + 1
        x = q[r].long()
        score = (bd[:have, 1] @ x.clamp(min=0).sum(0) + bd[:have, 0] @ x.clamp(max=0).sum(0)).float() * sc[:have]
        score[:2] = score[have - 3:] = float("inf")
        want = score.sort(descending=True, stable=True).indices[:count].sort().values
        assert torch.equal(got[r, 0].cpu().long(), want), r


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 4, 64), (20, 1, 64)])
def test_attention_over_chosen_blocks(fmt, hq, hkv, d):
    lens, new = [1000, 64, 0, 65, 700, 3], [1, 2, 1, 1, 5, 4]
    cache, table, ref = _random_cache(lens, hkv, d, fmt, 81)
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1])
    q = _bf16((rows, hq, d), 82)
    blocks = pkg.cache_select(cache, _i32(table), _i32(lens), q.cuda(), 4, cu=_i32(cu))
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(cu), blocks=blocks)
    pkg.hdp_device_status()
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, d ** -0.5, blocks.cpu().numpy()))
    # entries that have to be skipped: before, twice, descending, beyond the row, beyond the table, negative
    odd = torch.tensor([[0, 0, 3, 1, 2, 9, 15, 400, -1, 2 ** 31 - 1]], dtype=torch.int32).expand(rows, hkv, 10).contiguous()
    odd[:, 0] = -1  # a head that attends to nothing
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(cu), blocks=odd.cuda())
    pkg.hdp_device_status()
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, d ** -0.5, odd.numpy()))
    # all blocks: the dense result, up to the order of its sums
    every = torch.arange(16, dtype=torch.int32, device="cuda").expand(rows, hkv, 16).contiguous()
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda(), cu=_i32(cu), blocks=every)
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, d ** -0.5))


def test_rows_of_no_sequence_keep_their_outputs_with_blocks():
    cache, table, _ = _random_cache([100], 1, 64, 0, 91)
    q = _bf16((5, 2, 64), 92).cuda()
    o, lse = torch.full((5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 5), 7.0, device="cuda")
    ws = torch.empty(pkg.hdp_cache_attention_workspace_bytes(cache, 2), dtype=torch.uint8, device="cuda")
    blocks = torch.zeros((5, 1, 2), dtype=torch.int32, device="cuda")
    pkg.hdp_cache_attention(cache, _i32(table), _i32([100]), q, 0.125, ws, o, lse, cu=_i32([0, 2]), blocks=blocks)
    assert (o[2:] == 7).all() and (lse[:, 2:] == 7).all() and (o[:2] != 7).any()


# ---------------------------------------------------------------- bad tables, streams, graphs

def test_pages_and_lengths_outside_are_reported_and_never_touched():
    lens = [200]
    cache, table, ref = _random_cache(lens, 2, 64, 1, 95, spare=0)
    q = _bf16((1, 4, 64), 96)
    bad = table.copy()
    bad[0, 1] = 10 ** 6
    o, lse = pkg.cache_attention(cache, _i32(bad), _i32(lens), q.cuda())
    with pytest.raises(pkg.HdpError) as e:
        pkg.hdp_device_status()
    assert e.value.status == pkg.HDP_ERR_INVALID_ARGUMENT and "page" in str(e.value)
    pkg.hdp_device_status()  # cleared
    without = np.array([0, 2, 3])[None, None].repeat(2, 1)
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), [0, 1], 0.125, without))
    k, v = pkg.cache_read(cache, _i32(bad), _i32(lens), 200, cu=_i32([0, 200]))
    assert (k[64:128] == 0).all() and np.array_equal(_f64(k[128:]), ref.sequence(table[0], 200)[0][128:])
    before = [t.clone() for t in (cache.k, cache.v, cache.scales, cache.bounds)]
    bad[0, :] = -1
    x = _bf16((200, 2, 64), 97).cuda()
    pkg.cache_append(cache, _i32(bad), _i32(lens), x, x, cu=_i32([0, 200]))
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.scales, cache.bounds)))
    with pytest.raises(pkg.HdpError):
        pkg.hdp_device_status()
    # a length beyond the table counts as the table's end; a negative one as none
    o, lse = pkg.cache_attention(cache, _i32(table), _i32([10 ** 9]), q.cuda())
    o2, lse2 = pkg.cache_attention(cache, _i32(table), _i32([256]), q.cuda())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32([-5]), q.cuda())
    assert (o == 0).all() and torch.isneginf(lse).all()
    with pytest.raises(pkg.HdpError):
        pkg.hdp_device_status()
    b = pkg.cache_select(cache, _i32([[int(table[0, 0]), 99, int(table[0, 2]), int(table[0, 3])]]), _i32(lens), q.cuda(), 3, keep_first=0)
    assert (b == _i32([0, 2, 3])).all()
    with pytest.raises(pkg.HdpError):
        pkg.hdp_device_status()


def test_two_threads_on_one_stream():
    """Calls from two threads interleave on the default stream; each has its own workspace."""
    import threading

    lens = [120000, 90000]
    pages = sum((l + 63) // 64 for l in lens)
    cache = pkg.KVCache.empty(pages, 8, 64, 1)
    cache.k.random_(0, 256)
    cache.v.random_(0, 256)
    cache.scales.fill_(2.0 ** -6)
    cache.bounds.random_(-100, 100)
    table = torch.zeros((2, 1875), dtype=torch.int32, device="cuda")
    table[0] = torch.arange(1875)
    table[1, :1407] = torch.arange(1875, pages)
    qs = [_bf16((2, 16, 64), i).cuda() for i in range(2)]
    dl = _i32(lens)
    want = [(*pkg.cache_attention(cache, table, dl, q), pkg.cache_select(cache, table, dl, q, 50)) for q in qs]
    torch.cuda.synchronize()
    wrong = []

    def many(i):
        for _ in range(60):
            got = (*pkg.cache_attention(cache, table, dl, qs[i]), pkg.cache_select(cache, table, dl, qs[i], 50))
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)

    threads = [threading.Thread(target=many, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    pkg.hdp_device_status()


def test_another_stream_and_no_rows():
    lens = [300, 20]
    cache, table, ref = _random_cache(lens, 2, 64, 0, 101)
    q = _bf16((2, 4, 64), 102).cuda()
    args = (cache, _i32(table), _i32(lens), q)
    o, lse = pkg.cache_attention(*args)
    b = pkg.cache_select(*args, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = pkg.cache_attention(*args, stream=s)
    b2 = pkg.cache_select(*args, 2, stream=s.cuda_stream)
    k2, v2 = pkg.cache_read(cache, args[1], args[2], 2, stream=s)
    s.synchronize()
    k, v = pkg.cache_read(cache, args[1], args[2], 2)
    assert all(torch.equal(x, y) for x, y in ((o, o2), (lse, lse2), (b, b2), (k, k2), (v, v2)))
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu = _i32([0, 0, 0])
    o, lse = pkg.cache_attention(cache, args[1], args[2], none, cu=cu)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert pkg.cache_select(cache, args[1], args[2], none, 2, cu=cu).shape == (0, 2, 2)
    kv = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    pkg.cache_append(cache, args[1], args[2], kv, kv, cu=cu)


def test_prompt_then_decoding_steps_in_a_graph():
    """The operators as they are used together: a packed prompt goes through the attention and into the cache, then a
    captured step (append, choose, attend to all and to the chosen blocks, advance the lengths) is replayed; a second
    graph with a workspace of its own runs on another stream meanwhile."""
    hq, hkv, d, fmt = 8, 2, 128, pkg.HDP_CACHE_INT8
    prompt, steps = [100, 447, 64], 30
    T = sum(prompt)
    final = [p + steps for p in prompt]
    rng = np.random.default_rng(1)
    pages, table = _table(final, rng)
    cache = pkg.KVCache.empty(pages, hkv, d, fmt)
    q, k, v = _bf16((T, hq, d), 1).cuda(), _bf16((T, hkv, d), 2).cuda(), _bf16((T, hkv, d), 3).cuda()
    lens = _i32(prompt)
    o, lse, plan = pkg.attention(q, k, v, lens, 8192)
    cu = _i32(np.concatenate([[0], np.cumsum(prompt)]))
    tb = _i32(table)
    pkg.cache_append(cache, tb, lens, k, v, cu=cu)
    # the prompt's attention over the cache is the packed attention of what the cache holds
    kr, vr = pkg.cache_read(cache, tb, lens, T, cu=cu)
    o1, lse1 = pkg.cache_attention(cache, tb, lens, q, cu=cu)
    o2, lse2, _ = pkg.attention(q, kr, vr, lens, 8192, plan=plan)
    # o2 is within 1.5e-2 of the exact result (the attention's tolerance), o1 within half a bf16 step, 2^-8 |o|, and
    # twice 2^-11 sum p |v| <= 2^-10 max |v|; lse2 within 2e-3, lse1 within 2^-16 * 64 (sum |q k| scale stays below 64)
    off = (o1.float() - o2.float()).abs() - 1.5e-2 - 2.0 ** -8 * o2.float().abs() - 2.0 ** -10 * vr.float().abs().max()
    assert off.max() <= 0 and (lse1 - lse2).abs().max() <= 3e-3
    plan.destroy()

    def buffers():
        return dict(q=torch.empty((3, hq, d), dtype=torch.bfloat16, device="cuda"),
                    k=torch.empty((3, hkv, d), dtype=torch.bfloat16, device="cuda"),
                    v=torch.empty((3, hkv, d), dtype=torch.bfloat16, device="cuda"))

    x = buffers()

    def step():
        lens.add_(1)
        pkg.cache_append(cache, tb, lens, x["k"], x["v"])
        blocks = pkg.cache_select(cache, tb, lens, x["q"], 3)
        return (*pkg.cache_attention(cache, tb, lens, x["q"]), blocks,
                *pkg.cache_attention(cache, tb, lens, x["q"], blocks=blocks))

    for t in x.values():
        t.normal_()
    lens0, state = lens.clone(), [t.clone() for t in (cache.k, cache.v, cache.scales, cache.bounds)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    fixed = (q[:3].contiguous(), _i32(prompt))
    with torch.cuda.graph(other):
        still = pkg.cache_attention(cache, tb, fixed[1], fixed[0])
    lens.copy_(lens0)
    for t, s in zip((cache.k, cache.v, cache.scales, cache.bounds), state):
        t.copy_(s)
    want_still = pkg.cache_attention(cache, tb, fixed[1], fixed[0])
    ref = _oracle(cache)
    now = np.array(prompt)
    gen = torch.Generator().manual_seed(9)
    for s in range(steps):
        for name, t in x.items():
            t.copy_(torch.randn(t.shape, generator=gen).to(torch.bfloat16))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        now = now + 1
        ref.append(table, now, _f64(x["k"]), _f64(x["v"]), [0, 1, 2, 3])
        if s % 10 == 9:
            cu1 = np.arange(4)
            assert lens.tolist() == now.tolist()
            blocks = outs[2].cpu().numpy()
            assert np.array_equal(blocks, ref.select(table, now, _f64(x["q"]), cu1, 3, 1, 1))
            _check_attention(outs[0], outs[1], ref.attention(table, now, _f64(x["q"]), cu1, d ** -0.5))
            _check_attention(outs[3], outs[4], ref.attention(table, now, _f64(x["q"]), cu1, d ** -0.5, blocks))
    # two graphs at once: the prompt's blocks are read by one while the other attends
    side.wait_stream(torch.cuda.current_stream())
    lens.sub_(1)
    torch.cuda.current_stream().synchronize()
    full = [t.clone() for t in outs]
    for _ in range(5):
        lens.sub_(0)
        with torch.cuda.stream(side):
            other.replay()
        pkg.cache_attention(cache, tb, lens, x["q"])
    torch.cuda.synchronize()
    still2 = pkg.cache_attention(cache, tb, fixed[1], fixed[0])
    assert torch.equal(still[0], still2[0]) and torch.equal(still[1], still2[1])
    assert all(torch.equal(a, b) for a, b in zip(full, outs)) and want_still[0].shape == still[0].shape
    pkg.hdp_device_status()


# ---------------------------------------------------------------- drawn calls

@pytest.mark.parametrize("seed", [3304] + list(range(40)))
def test_drawn_calls(seed):
    """Everything at once on drawn shapes: several appends (prompts, chunks, single tokens, scales that grow), then
    attention, the choice of blocks, attention over them and reading back, for drawn numbers of rows."""
    import random

    r, rng = random.Random(seed), np.random.default_rng(seed)
    fmt, d, hkv = r.choice(FMTS), r.choice([64, 128]), r.choice([1, 1, 2, 3, 4, 8])
    hq, n = hkv * r.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 17, 33]), r.choice([1, 1, 2, 3, 5, 9, 40])
    top = r.choice([3, 70, 300, 1500]) if n > 3 else r.choice([1, 65, 300, 3000, 9000])
    lens = [r.choice([0, 1, 63, 64, 65, r.randint(0, top), r.randint(0, top)]) for _ in range(n)]
    pages, table = _table([max(l, 1) for l in lens], rng, spare=r.randint(0, 3), columns=r.randint(0, 60))
    cache = _filled(pages, hkv, d, fmt, byte=r.randint(0, 126))
    ref, tb = _oracle(cache), _i32(table)
    now, step = [0] * n, 0
    while now != lens:
        new = [min(l - c, r.choice([0, 1, 1, 5, 64, 100, 10000])) for l, c in zip(lens, now)]
        if not sum(new):
            continue
        step += 1
        now = [c + m for c, m in zip(now, new)]
        cu = np.concatenate([[0], np.cumsum(new)])
        k, v = (_bf16((int(cu[-1]), hkv, d), seed + 50 * step + w, 2.0 ** r.randint(-4, 4)) for w in range(2))
        pkg.cache_append(cache, tb, _i32(now), k.cuda(), v.cuda(), cu=_i32(cu))
        ref.append(table, now, _f64(k), _f64(v), cu)
    got = _oracle(cache)
    used = sorted({int(table[i, b]) for i, l in enumerate(lens) for b in range((l + 63) // 64)})
    for name in ("scales", "bounds", "k", "v"):
        assert np.array_equal(getattr(got, name)[used], getattr(ref, name)[used]), name

    single = r.random() < 0.3
    new = [1] * n if single else [r.choice([0, 1, 1, 2, 3, 9, r.randint(0, l + 2) if l < 100 else 4]) for l in lens]
    new[0] = max(new[0], 1)
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1])
    q, cud, scale = _bf16((rows, hq, d), seed + 3, r.choice([0.3, 1, 3])), None if single else _i32(cu), d ** -0.5
    o, lse = _poisoned(cache, tb, _i32(lens), q.cuda(), scale, cu=cud)
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, scale), "all")
    count = r.choice([1, 2, 3, 8, 40, 200])
    first = r.randint(0, min(2, count))
    last = r.randint(0, min(2, count - first))
    b = pkg.cache_select(cache, tb, _i32(lens), q.cuda(), count, cu=cud, keep_first=first, keep_last=last)
    want = ref.select(table, lens, _f64(q), cu, count, first, last)
    assert np.array_equal(b.cpu().numpy(), want)
    o, lse = _poisoned(cache, tb, _i32(lens), q.cuda(), scale, cu=cud, blocks=b)
    _check_attention(o, lse, ref.attention(table, lens, _f64(q), cu, scale, want), "chosen")
    k, v = pkg.cache_read(cache, tb, _i32(lens), rows, cu=cud)
    for i, l in enumerate(lens):
        none = max(0, new[i] - l)
        for x, y in zip((k, v), ref.sequence(table[i], l)):
            assert np.array_equal(_f64(x[cu[i] + none:cu[i + 1]]), y[l - new[i] + none:]) and (x[cu[i]:cu[i] + none] == 0).all()
    pkg.hdp_device_status()
