"""Attention over the 4-bit cache where its paths meet: scores spread from nothing to far, blocks on no page, rows at the
beginning, one sequence over the whole GPU, streams, devices' workspaces of garbage."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from oracle import kv_cache4 as k4
from test_gpu_cache4 import _bf16, _check, _cu, _f64, _i32, _random_cache

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


def _attend(cache, table, lens, q, new, scale):
    """With a workspace of garbage."""
    hq = q.shape[1]
    cu = None if new is None else _i32(_cu(new))
    ws = torch.full((pkg.hdp_fourbit_attention_workspace_bytes(cache, hq),), 0xa5, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty((hq, q.shape[0]), device="cuda")
    pkg.hdp_fourbit_attention(cache, _i32(table), _i32(lens), q.cuda(), scale, ws, o, lse, cu=cu)
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 4])
@pytest.mark.parametrize("size", [0.0, 0.02, 0.5, 1.0, 1.5, 2.0, 4.0, 20.0])
def test_scores_spread_from_nothing_to_far(d, rows, size):
    """From blocks that all stay under the first references to ones that none does, and those that change in between."""
    rng = np.random.default_rng(int(size * 100) + d + rows)
    lens = [700, 64, 129, 1, 190]
    new = [min(l, rows) for l in lens]
    table, (cache, ref) = _random_cache(lens, 2, d, rng, spread=4, low=124)
    q = _bf16(rng.normal(size=(sum(new), 8, d)) * size)
    q[:, 3] *= 8  # one head far larger than its neighbours
    o, lse = _attend(cache, table, lens, q, new, d ** -0.5)
    _check(o, lse, ref.attention(table, lens, _f64(q), _cu(new), d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0, 4.0, 8.0])
@pytest.mark.parametrize("zeros", [0.0, 0.7, 0.97])
def test_peaked_rows_over_many_blocks_with_zeros_in_v(d, size, zeros):
    """Runs of several blocks whose scores deviate by nats, so that small weights meet channels in which the heavy keys are
    zero: what they add counts all the same."""
    rng = np.random.default_rng(int(size) + d + int(100 * zeros))
    lens = [4000] * 20
    table, (cache, ref) = _random_cache(lens, 4, d, rng, spread=3, low=124)
    for half in (0x0F, 0xF0):
        ref.v[rng.random(ref.v.shape) < zeros] &= half
    cache.v.copy_(torch.tensor(ref.v))
    q = _bf16(rng.normal(size=(20, 8, d)) * 0.5 * size)
    o, lse = pkg.cache_attention(cache, _i32(table), _i32(lens), q.cuda())
    _check(o, lse, ref.attention(table, lens, _f64(q), np.arange(21), d ** -0.5))


@pytest.mark.parametrize("rising", [False, True])
def test_scores_that_rise_and_fall_from_block_to_block(rising):
    """Each block's scores lie some bits beyond the last one's: references are made anew again and again, or are far above."""
    rng = np.random.default_rng(5)
    d, lens = 64, [1500, 900]
    table, (cache, ref) = _random_cache(lens, 1, d, rng, spread=1, low=125)
    for i, l in enumerate(lens):
        for b in range(-(-l // 64)):
            ref.scales[table[i, b], 0, :-1] = 116 + (b if rising else 22 - b) // 2
            ref.scales[table[i, b], 0, -1] = 120 + b % 9
    cache.scales.copy_(torch.tensor(ref.scales))
    q = _bf16(rng.normal(size=(2, 4, d)))
    o, lse = _attend(cache, table, lens, q, None, 1.0)
    _check(o, lse, ref.attention(table, lens, _f64(q), [0, 1, 2], 1.0))


@pytest.mark.parametrize("d", [64, 128])
def test_blocks_on_no_page_are_left_out(d):
    """Bad pages at the beginning, inside, several at once and at the end of sequences that share warps and CTAs."""
    rng = np.random.default_rng(d + 1)
    lens = [64 * 40, 64 * 40 + 17, 130, 64, 64 * 70]
    table, (cache, ref) = _random_cache(lens, 2, d, rng)
    gone = {0: [0, 7, 8, 9], 1: [40], 2: [1], 3: [0], 4: list(range(20, 60)) + [69]}
    bad = table.copy()
    for i, blocks in gone.items():
        bad[i, blocks] = rng.choice([-1, 10 ** 6], len(blocks))
    q = _bf16(rng.normal(size=(5, 4, d)))
    o, lse = _attend(cache, bad, lens, q, None, d ** -0.5)
    with pytest.raises(pkg.HdpError, match="outside"):
        pkg.hdp_device_status()
    want = []
    for i, l in enumerate(lens):  # the oracle sees the other tokens only, in their order, a whole block of garbage never
        keep = [b for b in range(-(-l // 64)) if b not in gone[i]]
        n = sum(min(64, l - 64 * b) for b in keep)
        want.append(ref.attention(table[i:i + 1, keep] if keep else [[0]], [n], _f64(q)[i:i + 1], [0, 1], d ** -0.5))
    _check(o, lse, tuple(np.concatenate([w[k] for w in want], axis=1 if k == 1 else 0) for k in range(5)))


@pytest.mark.parametrize("d,g", [(64, 1), (128, 4), (64, 8)])
def test_many_rows_of_a_sequence(d, g):
    """Rows of a whole prompt: every row sees another number of keys, tiles of rows read the cache again; some rows come
    before the sequence's first token."""
    rng = np.random.default_rng(d + g)
    lens, new = [150, 200, 40], [150, 30, 45]
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    q = _bf16(rng.normal(size=(sum(new), g, d)))
    o, lse = _attend(cache, table, lens, q, new, d ** -0.5)
    _check(o, lse, ref.attention(table, lens, _f64(q), _cu(new), d ** -0.5))
    assert not o[180:185].any() and (lse[:, 180:185] == -np.inf).all()


def test_one_head_of_one_sequence_over_the_whole_gpu():
    rng = np.random.default_rng(8)
    lens, d = [700001], 64
    table, (cache, ref) = _random_cache(lens, 1, d, rng)
    q = _bf16(rng.normal(size=(1, 2, d)))
    o, lse = _attend(cache, table, lens, q, None, 0.125)
    _check(o, lse, ref.attention(table, lens, _f64(q), [0, 1], 0.125))


@pytest.mark.parametrize("n,longest", [(1, 64), (3, 300), (40, 64), (300, 130), (1217, 70)])
def test_fewer_and_more_units_than_warps(n, longest):
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, longest + 1, n)]
    table, (cache, ref) = _random_cache(lens, 1, 64, rng)
    q = _bf16(rng.normal(size=(n, 3, 64)))
    o, lse = _attend(cache, table, lens, q, None, 0.125)
    _check(o, lse, ref.attention(table, lens, _f64(q), np.arange(n + 1), 0.125))


def test_results_do_not_depend_on_what_else_a_page_or_the_workspace_holds():
    """Bit for bit, with other codes and scales (NaN among them) in tokens behind the sequences."""
    rng = np.random.default_rng(10)
    d, lens = 128, [100, 1, 65, 640]
    table, (cache, ref) = _random_cache(lens, 2, d, rng)
    q = _bf16(rng.normal(size=(4, 8, d)))
    o, lse = _attend(cache, table, lens, q, None, d ** -0.5)
    for i, l in enumerate(lens):
        for t in range(l % 64, 64 if l % 64 else 0):
            page = table[i, l // 64]
            ref.scales[page, :, :, k4.scale_place(t)] = rng.choice([0, 1, 60, 127, 190, 191, 255], (2, d // 32 + 1))
            ref.k[page, :, t] = rng.integers(0, 256, (2, d // 2))
    cache.k.copy_(torch.tensor(ref.k)), cache.scales.copy_(torch.tensor(ref.scales))
    again, lse2 = _attend(cache, table, lens, q, None, d ** -0.5)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


def test_inputs_that_die_while_another_stream_reads_them():
    rng = np.random.default_rng(12)
    d, lens = 64, [3000] * 8
    table, (cache, ref) = _random_cache(lens, 2, d, rng)
    q = _bf16(rng.normal(size=(8, 4, d))).cuda()
    want = _attend(cache, table, lens, q, None, 0.125)
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        a, b, c = _i32(table), _i32(lens), q.clone()
        side.wait_stream(torch.cuda.current_stream())
        got.append(pkg.cache_attention(cache, a, b, c, scale=0.125, stream=side))
        seq, pos, slot = pkg.cache_rows(b, 8, page_table=a, num_pages=cache.num_pages, stream=side)
        turned = pkg.rotary(c, None, pos, torch.ones(8, dtype=torch.float64, device="cuda"), stream=side)[0]
        del a, b, c
        torch.full((8, 4, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.zeros((8, table.shape[1]), dtype=torch.int32, device="cuda")
    side.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(lse, want[1]) for o, lse in got)
    assert seq.tolist() == list(range(8)) and pos.tolist() == [2999] * 8 and slot.tolist() == [int(t[46]) * 64 + 55 for t in table]
    assert torch.equal(turned, pkg.rotary(q, None, _i32([2999] * 8), torch.ones(8, dtype=torch.float64, device="cuda"))[0])
