"""Block tables, slot maps and rotary positions on the GPU against their oracles, and a prompt and decoding steps that use
all of them together."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from oracle import kv_cache4 as k4
from oracle import rows as ro

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


def _f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- block tables

class _Both:
    """A pool and its sequences on the GPU and in the oracle."""

    def __init__(self, pages, n, columns, rng):
        self.free, self.table, self.held = [int(x) for x in rng.permutation(pages)], [[-1] * columns for _ in range(n)], [0] * n
        self.pool = pkg.PagePool(_i32(self.free), _i32([pages]))
        self.gt, self.gh = _i32(self.table), _i32(self.held)

    def assign(self, lens):
        pkg.cache_assign(self.pool, self.gt, self.gh, _i32(lens))
        fits = ro.assign(self.free, self.table, self.held, lens)
        self.check()
        return fits

    def check(self):
        assert self.gh.cpu().tolist() == self.held
        assert self.pool.count.item() == len(self.free) and self.pool.free[:len(self.free)].cpu().tolist() == self.free
        assert np.array_equal(self.gt.cpu().numpy(), np.asarray(self.table))


@pytest.mark.parametrize("n,columns", [(1, 1), (1, 40), (7, 9), (300, 5), (1023, 3), (2048, 2), (2049, 3), (5000, 2)])
def test_tables_follow_lengths_that_grow_and_shrink(n, columns):
    """One CTA and a cluster, one and several rounds of sequences, giving and taking in one call."""
    rng = np.random.default_rng(n)
    both = _Both(n * columns, n, columns, rng)
    for step in range(6):
        lens = rng.integers(0, columns * 64 + 1, n) * (rng.random(n) < 0.8) if step != 3 else np.zeros(n, int)
        assert both.assign(lens.tolist())


def test_taking_pages_and_giving_them_back_leaves_everything_as_it_was():
    rng = np.random.default_rng(1)
    both = _Both(900, 90, 10, rng)
    a = rng.integers(0, 300, 90)
    both.assign(a.tolist())
    before = list(both.free), list(both.held)
    both.assign((a + rng.integers(0, 300, 90)).tolist())
    both.assign(a.tolist())
    assert (both.free, both.held) == before


@pytest.mark.parametrize("n,columns", [(5, 4), (400, 30), (3000, 2)])
def test_a_pool_that_runs_out(n, columns):
    """Sequences in front get theirs, the first that lacks too many and the later ones keep what they have; it is reported."""
    rng = np.random.default_rng(n + 1)
    both = _Both(n * columns // 2, n, columns, rng)
    ran_out = 0
    for _ in range(5):
        if not both.assign((rng.integers(0, columns + 1, n) * 64).tolist()):
            ran_out += 1
            with pytest.raises(pkg.HdpError, match="ran out") as e:
                pkg.hdp_device_status()
            assert e.value.status == pkg.HDP_ERR_OUT_OF_MEMORY
        pkg.hdp_device_status()
    assert ran_out


def test_one_sequence_takes_and_gives_many_pages():
    rng = np.random.default_rng(2)
    both = _Both(40000, 2, 33000, rng)
    assert both.assign([2097152, 65]) and both.assign([100, 2000000]) and both.assign([0, 0])


def test_lengths_and_counts_outside_their_ranges_are_bounded_and_reported():
    rng = np.random.default_rng(3)
    both = _Both(20, 3, 4, rng)
    pkg.cache_assign(both.pool, both.gt, both.gh, _i32([-5, 1000, 64]))
    ro.assign(both.free, both.table, both.held, [0, 256, 64])
    both.check()
    with pytest.raises(pkg.HdpError, match="outside"):
        pkg.hdp_device_status()
    both.gh.copy_(_i32([-1, 9, 1]))  # counts that are none
    pkg.cache_assign(both.pool, both.gt, both.gh, _i32([0, 256, 64]))
    with pytest.raises(pkg.HdpError, match="outside"):
        pkg.hdp_device_status()
    assert both.pool.free[:15].cpu().tolist() == both.free and both.pool.count.item() == 15
    pool = pkg.PagePool(_i32([1, 2, 3]), _i32([7]))
    pkg.cache_assign(pool, _i32([[0]]), _i32([0]), _i32([0]))
    with pytest.raises(pkg.HdpError, match="outside"):
        pkg.hdp_device_status()
    assert pool.count.item() == 3
    pool = pkg.PagePool(_i32([1, 2, 3]), _i32([3]))  # a page that is given back twice does not fall off the stack's end
    held = _i32([2])
    pkg.cache_assign(pool, _i32([[8, 9]]), held, _i32([0]))
    with pytest.raises(pkg.HdpError, match="outside"):
        pkg.hdp_device_status()
    assert pool.count.item() == 3 and pool.free.cpu().tolist() == [1, 2, 3] and held.item() == 0


# ---------------------------------------------------------------- slot maps

def _maps(lens, cu, count, table=None, pages=0):
    got = pkg.cache_rows(_i32(lens), count, cu=None if cu is None else _i32(cu), page_table=None if table is None else _i32(table),
                         num_pages=pages if table is not None else None)
    want = ro.rows(lens, list(range(len(lens) + 1)) if cu is None else cu, count, table, pages)
    for name, g, w in zip(("sequence", "position", "slot"), got, want):
        if g is not None:
            assert np.array_equal(g.cpu().numpy(), w), name
    return got


@pytest.mark.parametrize("seed", range(6))
def test_rows_of_requests_with_empty_ones_and_rows_behind_the_last(seed):
    rng = np.random.default_rng(seed)
    n = [1, 3, 40, 700, 2000, 33][seed]
    lens = rng.integers(0, 640, n)
    new = np.minimum(lens, rng.integers(0, [700, 700, 700, 3, 2, 200][seed], n)) * (rng.random(n) < 0.7)
    table = rng.integers(0, 77, (n, 10))
    cu = np.concatenate([[0], np.cumsum(new)])
    _maps(lens.tolist(), cu.tolist(), int(cu[-1]) + seed * 50, table, 77)
    _maps(lens.tolist(), None, n, table, 77) if (lens > 0).all() else None


def test_documents_single_tokens_and_rows_before_the_beginning():
    seq, pos, slot = _maps([5, 0, 1, 130, 0], [0, 5, 5, 6, 136, 136], 140)
    assert slot is None and pos[6:9].tolist() == [0, 1, 2]
    _maps([3, 1], None, 2, [[2], [0]], 3)
    _maps([2, 5], [0, 6, 9], 9, [[1], [2]], 4)  # four rows more than tokens
    _maps([1] * 5000, list(range(5001)), 5001)
    pkg.hdp_device_status()
    _maps([3, 3], [0, 3, 6], 6, [[3], [-1]], 3)  # pages outside the pool
    with pytest.raises(pkg.HdpError, match="outside"):
        pkg.hdp_device_status()


# ---------------------------------------------------------------- rotary positions

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _turn_check(got, x, pos, f, neighbours, backward, factor):
    """One rounding to the type; in fp32 the angle (2^-24 of up to pi), the cosine and sine (an ulp each), the factor, two
    products and a sum: below 2^-20 of |a| + |b|."""
    ref = ro.turn(_f64(x), pos, f, neighbours, backward, factor)
    half = len(f)
    a = np.abs(_f64(x))
    size = np.zeros_like(a)
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if neighbours else (slice(0, half), slice(half, 2 * half))
    size[..., first] = size[..., second] = a[..., first] + a[..., second]
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * eps
    limit = eps * np.abs(ref) + (1 + eps) * 2.0 ** -20 * factor * size + tiny
    off = np.abs(_f64(got) - ref)
    assert (off <= limit).all(), (float((off / limit).max()), np.argwhere(off > limit)[:4].tolist())
    assert np.array_equal(_f64(got)[..., 2 * half:], _f64(x)[..., 2 * half:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (128, 64), (64, 32), (96, 48), (64, 38), (64, 2), (256, 256), (10, 6), (2, 2)])
def test_turns_of_every_layout(dtype, neighbours, d, rot):
    rng = np.random.default_rng(d + rot)
    for rows, hq, hkv, apart in ((1, 1, 1, False), (37, 5, 2, True), (700, 3, 1, False)):
        x = torch.tensor(rng.normal(size=(rows, hq + 2 * hkv, d))).to(dtype).cuda()
        q, k = x[:, :hq], x[:, hq:hq + hkv]
        if apart:  # heads outside, rows inside
            q, k = (y.transpose(0, 1).contiguous().transpose(0, 1) for y in (q, k))
        pos = rng.integers(0, 2 ** 31, rows) if rows == 37 else rng.integers(0, 5000, rows)
        f = np.exp(-rng.uniform(0, 12, rot // 2))
        gf = torch.tensor(f, device="cuda")
        before = x.clone()
        for backward in (False, True):
            turn = pkg.rotary_backward if backward else pkg.rotary
            a, b = turn(q, k, _i32(pos), gf, neighbours=neighbours, factor=1.25)
            _turn_check(a, q, pos, f, neighbours, backward, 1.25)
            _turn_check(b, k, pos, f, neighbours, backward, 1.25)
        assert torch.equal(x, before)
        c, e = q.clone(), k.clone()
        assert pkg.rotary(c, e, _i32(pos), gf, neighbours=neighbours, inplace=True)[0] is c
        a, b = pkg.rotary(q, k, _i32(pos), gf, neighbours=neighbours)
        assert torch.equal(a, c) and torch.equal(b, e)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_at_any_alignment_turn_alike(dtype):
    """Views one element behind an aligned address, and strides that are no multiples of 16 bytes."""
    rng = np.random.default_rng(5)
    whole = torch.tensor(rng.normal(size=33 * 7 * 65 + 1)).to(dtype).cuda()
    odd = whole[1:].view(33, 7, 65)[:, :, :64]
    pos, f = _i32(rng.integers(0, 9999, 33)), torch.tensor(np.exp(-rng.uniform(0, 9, 24)), device="cuda")
    for neighbours in (False, True):
        a, none = pkg.rotary(odd, None, pos, f, neighbours=neighbours)
        b = pkg.rotary(None, odd.contiguous(), pos, f, neighbours=neighbours)[1]
        assert none is None and torch.equal(a, b)


def test_rows_that_are_both_q_and_k():
    """Turned out of place they may be both; where one is written over the other's rows the call is refused."""
    x = torch.randn(9, 2, 64, device="cuda")
    f, pos = torch.ones(32, device="cuda", dtype=torch.float64), _i32(np.arange(9))
    a, b = pkg.rotary(x, x, pos, f)
    assert torch.equal(a, b)
    before, y = x.clone(), torch.empty_like(x)
    for out in ((x, x), (x, y), (y, x), (y, y)):
        with pytest.raises(pkg.HdpError, match="rows of the other"):
            pkg.hdp_rotary(x, x, pos, f, *out)
    with pytest.raises(pkg.HdpError, match="rows of the other"):
        pkg.rotary(x, x, pos, f, inplace=True)
    assert torch.equal(x, before)
    pkg.rotary(x, x[:, :0], pos, f, inplace=True)  # no heads: nothing is shared
    assert torch.equal(x, a)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("d,rot,pitch,offset", [(64, 48, 66, 0), (64, 46, 66, 2), (64, 36, 64, 0), (128, 6, 136, 0), (128, 126, 128, 0), (7, 6, 8, 0), (250, 250, 250, 0)])
def test_every_way_through_a_head_turns_alike(dtype, neighbours, d, rot, pitch, offset):
    """By 16 bytes, pieces, two elements and one, in place and not; infinities behind rot stay, and what lies between
    rows is left alone."""
    rng = np.random.default_rng(rot)
    whole = torch.tensor(rng.normal(size=21 * 5 * pitch + offset)).to(dtype).cuda()
    x = whole[offset:].view(21, 5, pitch)[:, :, :d]
    if rot < d:
        x[:, :, rot::3] = float("inf")
    before = whole.clone()
    f = torch.tensor(np.exp(-rng.uniform(0, 9, rot // 2)), device="cuda")
    pos = rng.integers(0, 9999, 21)
    a, b = pkg.rotary(x[:, :4], x[:, 4:], _i32(pos), f, neighbours=neighbours, factor=0.75)
    assert torch.equal(whole, before)
    for got, src in ((a, x[:, :4]), (b, x[:, 4:])):
        _turn_check(got[..., :rot], src[..., :rot], pos, f.cpu().numpy(), neighbours, False, 0.75)
        assert torch.equal(got[..., rot:], src[..., rot:])
    pkg.rotary(x[:, :4], x[:, 4:], _i32(pos), f, neighbours=neighbours, factor=0.75, inplace=True)
    assert torch.equal(x, torch.cat((a, b), 1))
    between = torch.ones_like(whole, dtype=torch.bool)
    between[offset:].view(21, 5, pitch)[:, :, :d] = False
    assert torch.equal(whole[between], before[between])


def test_rows_at_negative_positions_and_other_rows_between_are_left_alone():
    rng = np.random.default_rng(6)
    x = torch.tensor(rng.normal(size=(9, 6, 64))).to(torch.bfloat16).cuda()
    x[4] = float("nan")
    before = x.clone()
    pos, f = _i32([3, -1, 5, -7, -1, 0, 9, -2 ** 31, 1]), torch.tensor([1.0, 0.5], dtype=torch.float64, device="cuda")
    pkg.rotary(x[:, :2], x[:, 2:3], pos, f, inplace=True)
    still = pos.cpu() < 0
    assert torch.equal(x[still].view(torch.int16), before[still].view(torch.int16)) and torch.equal(x[:, 3:].view(torch.int16), before[:, 3:].view(torch.int16))
    assert torch.equal(x[..., 4:].view(torch.int16), before[..., 4:].view(torch.int16)) and not torch.equal(x[0, :3], before[0, :3])


def test_far_positions_keep_their_angle():
    """cos and sin at two thousand million positions, from the pair (1, 0)."""
    pos = np.array([0, 1, 2097151, 2 ** 24 + 1, 2 ** 31 - 1])
    f = np.array([1.0, 0.7310585786300049, 1e-3, 1e-7, 3.0])
    x = torch.zeros((5, 1, 10), device="cuda")
    x[:, :, :5] = 1
    y = _f64(pkg.rotary(x, None, _i32(pos), torch.tensor(f, device="cuda"))[0])[:, 0]
    angle = np.array([[float(int(p) * np.longdouble(t) % (2 * np.longdouble("3.14159265358979323846264338327950288"))) for t in f] for p in pos])
    assert np.abs(y[:, :5] - np.cos(angle)).max() < 6e-7 and np.abs(y[:, 5:] - np.sin(angle)).max() < 6e-7


def test_rotary_refusals_on_the_gpu():
    x, pos, f = torch.zeros((3, 2, 8), device="cuda"), _i32([0, 1, 2]), torch.ones(4, dtype=torch.float64, device="cuda")
    for bad in (dict(q=x.double()), dict(q=x.to(torch.int32)), dict(k=x.half()), dict(q=x[0]), dict(position=pos.long()), dict(position=pos[:2]),
                dict(freqs=f.float()), dict(k=x[:2]), dict(k=torch.zeros((3, 2, 6), device="cuda")), dict(q=x.transpose(1, 2)),
                dict(q=x[:1].expand(3, 2, 8), k=None, inplace=True)):
        with pytest.raises((TypeError, ValueError)):
            pkg.rotary(**{**dict(q=x, k=x, position=pos, freqs=f), **bad})
    with pytest.raises(pkg.HdpError, match="rot"):
        pkg.rotary(x, x, pos, torch.ones(5, dtype=torch.float64, device="cuda"))
    with pytest.raises(pkg.HdpError, match="factor"):
        pkg.rotary(x, x, pos, f, factor=0.0)
    a = pkg.rotary(x[:1].expand(3, 2, 8), None, pos, f)[0]  # read, a row may stand for several
    assert a.shape == (3, 2, 8)
    assert pkg.rotary(x[:0], x[:0], pos[:0], f)[0].shape == (0, 2, 8)


# ---------------------------------------------------------------- together

def _attention_ref(q, k, v, lens, scale):
    """Causal attention of whole documents in fp64, from q, k, v lists of [tokens][heads][d]."""
    out = []
    for x, y, z in zip(q, k, v):
        g = x.shape[1] // y.shape[1]
        y, z = (np.repeat(t, g, axis=1).transpose(1, 0, 2) for t in (y, z))
        s = x.transpose(1, 0, 2) @ y.transpose(0, 2, 1) * scale
        s = np.where(np.tril(np.ones(s.shape[1:], bool)), s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        out.append((p / p.sum(-1, keepdims=True) @ z).transpose(1, 0, 2))
    return out


@pytest.mark.parametrize("neighbours", [False, True])
def test_packed_attention_of_turned_rows_and_its_gradient(neighbours):
    """positions -> turn -> attention -> its backward -> turn back: the gradients of the projection's q and k are those of
    the whole by differences in fp64."""
    rng = np.random.default_rng(40)
    lens, hq, hkv, d = [70, 1, 33], 2, 1, 64
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    fused = torch.tensor(rng.normal(size=(T, hq + 2 * hkv, d)) * 0.5).to(torch.bfloat16).cuda()
    v = fused[:, hq + hkv:].contiguous()
    freqs, factor = pkg.rotary_frequencies(48, base=100.0, scaling="parts", by=4, trained=64)
    _, pos, _ = pkg.cache_rows(_i32(lens), T, cu=_i32(cu))
    q, k = pkg.rotary(fused[:, :hq], fused[:, hq:hq + hkv], pos, freqs, neighbours=neighbours, factor=factor)
    o, lse, plan = pkg.attention(q, k, v, _i32(lens), 256)
    dout = torch.tensor(rng.normal(size=(T, hq, d))).to(torch.bfloat16).cuda()
    dq, dk, dv = pkg.attention_backward(plan, q, k, v, o, lse, dout)
    gq, gk = pkg.rotary_backward(dq, dk, pos, freqs, neighbours=neighbours, factor=factor)
    pkg.hdp_device_status()
    plan.destroy()
    x, f, p, w = _f64(fused), freqs.cpu().numpy(), pos.cpu().numpy(), _f64(dout)
    split = lambda y: [y[a:b] for a, b in zip(cu, cu[1:])]

    def out(a, b):
        turned = [ro.turn(y, p, f, neighbours, factor=factor) for y in (a, b)]
        return np.concatenate(_attention_ref(split(turned[0]), split(turned[1]), split(x[:, hq + hkv:]), lens, d ** -0.5))

    base = x[:, :hq], x[:, hq:hq + hkv]
    assert np.abs(_f64(o) - out(*base)).max() <= 1.5e-2
    for got, which in ((gq, 0), (gk, 1)):
        got, want, seen = _f64(got), [], []
        for i in [(r, h, c) for r in (0, 3, 69, 71, 90, 103) for h in range(base[which].shape[1]) for c in (0, 1, 23, 24, 47, 48, 63)]:
            e = np.zeros_like(base[which])
            e[i] = 1e-4
            a, b = ([y + s * e if j == which else y for j, y in enumerate(base)] for s in (1, -1))
            want.append(((out(*a) - out(*b)) * w).sum() / 2e-4)
            seen.append(got[i])
        want, seen = np.array(want), np.array(seen)
        # the backward's own bar (2e-2 of the largest) and the bf16 roundings of q, k and of the turned gradients
        assert np.abs(want - seen).max() <= 3e-2 * np.abs(want).max(), (which, np.abs(want - seen).max(), np.abs(want).max())


@pytest.mark.parametrize("d", [64, 128])
def test_a_served_batch_from_prompts_to_decoding(d):
    """Pages from a pool, positions from the lengths, turned q and k, the cache written and attended to, step after step in
    a captured graph; a sequence is finished and its pages go to another."""
    rng = np.random.default_rng(41 + d)
    n, hq, hkv, columns = 4, 4, 2, 5
    pool, ref_pool = pkg.PagePool.full(14), list(range(13, -1, -1))
    table, rt = _i32(np.full((n, columns), -1)), [[-1] * columns for _ in range(n)]
    held, rh = _i32([0] * n), [0] * n
    cache = pkg.KVCache4.empty(14, hkv, d)
    for t in (cache.k, cache.v, cache.scales):
        t.zero_()
    ref = k4.Cache(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.scales)))
    freqs, factor = pkg.rotary_frequencies(d // 2, scaling="linear", by=2.0)
    f = freqs.cpu().numpy()
    scale = d ** -0.5
    lens = np.array([100, 63, 0, 250])
    glens = _i32(lens)

    def step(q, k, v, cu, rows):
        pkg.cache_assign(pool, table, held, glens)
        _, pos, slot = pkg.cache_rows(glens, rows, cu=cu, page_table=table, num_pages=14)
        tq, tk = pkg.rotary(q, k, pos, freqs, neighbours=True, factor=factor)
        pkg.cache_append(cache, table, glens, tk, v, cu=cu)
        o, lse = pkg.cache_attention(cache, table, glens, tq, cu=cu, scale=scale)
        return tq, tk, pos, slot, o, lse

    def check(out, v, new):
        tq, tk, pos, slot, o, lse = out
        assert ro.assign(ref_pool, rt, rh, lens.tolist())
        assert held.cpu().tolist() == rh and pool.free[:len(ref_pool)].cpu().tolist() == ref_pool
        cu = np.concatenate([[0], np.cumsum(new)])
        want = ro.rows(lens.tolist(), cu, int(cu[-1]), rt, 14)
        assert np.array_equal(pos.cpu().numpy(), want[1]) and np.array_equal(slot.cpu().numpy(), want[2])
        ref.append(rt, lens, _f64(tk), _f64(v), cu)
        for i in range(n):
            m = -(-int(lens[i]) // 64)
            if m:
                assert all(np.array_equal(a, b) for a, b in zip(ref.sequence(rt[i], int(lens[i])), k4.Cache(
                    *(t.cpu().numpy() for t in (cache.k, cache.v, cache.scales))).sequence(rt[i], int(lens[i]))))
        wo, wl, weight, size, _ = ref.attention(rt, lens.tolist(), _f64(tq), cu, scale)
        live = np.isfinite(wl)
        limit = 2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2.0 ** -15 * size + 2.0 ** -18)[..., None] * weight + 1e-30
        assert (np.abs(_f64(o) - wo) <= limit).all() and np.abs(_f64(lse)[live] - wl[live]).max() < 1e-3

    make = lambda rows, h: torch.tensor(rng.normal(size=(rows, h, d))).to(torch.bfloat16).cuda()
    rows = int(lens.sum())
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
    q, k, v = make(rows, hq), make(rows, hkv), make(rows, hkv)
    out = step(q, k, v, cu, rows)
    check(out, v, lens)
    _ = _f64(out[0]), ro.turn(_f64(q), out[2].cpu().numpy(), f, True, factor=factor)
    assert np.abs(_[0] - _[1]).max() <= 2.0 ** -8 * np.abs(_[1]).max() + 1e-5

    lens = np.array([101, 64, 1, 251])
    glens.copy_(_i32(lens))
    q, k, v = make(n, hq), make(n, hkv), make(n, hkv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check(step(q, k, v, None, n), v, [1] * n)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(q, k, v, None, n)
    for i in range(4):
        lens = lens + 1
        if i == 2:  # the long one is finished; its place is taken by a new sequence that begins with a token
            lens[3] = 1
        glens.copy_(_i32(lens))
        for t, h in ((q, hq), (k, hkv), (v, hkv)):
            t.copy_(make(n, h))
        graph.replay()
        check(out, v, [1] * n)
    pkg.hdp_device_status()
