"""Calls of the 8-bit cache around the ordinary ones: steps without rows, empty block lists, inputs that die while another
stream still reads them, two graphs that overlap, bounds of values far below their block's scale."""
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


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16).cuda()


def _filled(lens, hkv, d, fmt, seed):
    """A cache of sequences of these lengths: (cache, table, lens)."""
    need = [(l + 63) // 64 for l in lens]
    table = torch.zeros((len(lens), max(need) + 1), dtype=torch.int32)
    order = torch.randperm(sum(need) + len(lens), generator=torch.Generator().manual_seed(seed)).int()
    at = 0
    for i, m in enumerate(need):
        table[i, :m + 1] = order[at:at + m + 1]
        at += m + 1
    cache = pkg.KVCache.empty(len(order), hkv, d, fmt)
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
    pkg.cache_append(cache, table.cuda(), _i32(lens), _bf16((sum(lens), hkv, d), seed), _bf16((sum(lens), hkv, d), seed + 1), cu=cu)
    return cache, table.cuda(), _i32(lens)


# ---------------------------------------------------------------- bounds

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("single", [False, True])
def test_bounds_are_rounded_outwards_below_the_smallest_float(fmt, single):
    """Values whose share of the block's scale is below 2^-149 still widen the bounds, whether they come with the
    large one, before it or after it: bounds are a function of the rows alone."""
    d, hkv, big = 64, 2, 1e30
    row = torch.zeros((3, hkv, d))
    row[:, 0, 1], row[:, 0, 2], row[:, 1, 3] = -1e-38, 3e-37, -2.0 ** -133
    row[1, :, 0] = big  # the scale grows by some 2^200
    row[1, 0, 5], row[2, 0, 6] = 2.0 ** -126, -2.0 ** -126
    row = row.to(torch.bfloat16)
    table = _i32([[0]])
    cache, ref = pkg.KVCache.empty(1, hkv, d, fmt), kc.Cache(1, hkv, d, fmt)
    f64 = row.double().numpy()
    if single:
        for r in range(3):
            pkg.cache_append(cache, table, _i32([r + 1]), row[r:r + 1].cuda(), row[r:r + 1].cuda())
            ref.append([[0]], [r + 1], f64[r:r + 1], f64[r:r + 1], [0, 1])
    else:
        for a, z in ((0, 1), (1, 3)):
            pkg.cache_append(cache, table, _i32([z]), row[a:z].cuda(), row[a:z].cuda(), cu=_i32([0, z - a]))
            ref.append([[0]], [z], f64[a:z], f64[a:z], [0, z - a])
    got = cache.bounds.cpu().numpy()
    assert np.array_equal(got, ref.bounds), [(i.tolist(), got[tuple(i)], ref.bounds[tuple(i)]) for i in np.argwhere(got != ref.bounds)]
    whole = pkg.KVCache.empty(1, hkv, d, fmt)
    pkg.cache_append(whole, table, _i32([3]), row.cuda(), row.cuda(), cu=_i32([0, 3]))
    assert torch.equal(whole.bounds, cache.bounds)
    assert (got[0, 0, 0, 1], got[0, 0, 1, 2], got[0, 1, 0, 3]) == (-1, 1, -1)


# ---------------------------------------------------------------- steps without rows, empty lists

def test_an_empty_list_of_blocks_is_not_all_blocks():
    cache, table, lens = _filled([100, 70], 2, 64, 0, 1)
    q = _bf16((2, 4, 64), 3)
    with pytest.raises(ValueError, match="blocks"):
        pkg.cache_attention(cache, table, lens, q, blocks=torch.empty((2, 2, 0), dtype=torch.int32, device="cuda"))
    pkg.hdp_device_status()


def test_a_step_without_rows_goes_through_all_calls():
    cache, table, lens = _filled([100, 70], 2, 64, 1, 2)
    cu = _i32([0, 0, 0])
    before = [t.clone() for t in (cache.k, cache.v, cache.scales, cache.bounds)]
    kv, q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    pkg.cache_append(cache, table, lens, kv, kv, cu=cu)
    blocks = pkg.cache_select(cache, table, lens, q, 3, cu=cu)
    assert blocks.shape == (0, 2, 3)
    for b in (None, blocks):
        o, lse = pkg.cache_attention(cache, table, lens, q, cu=cu, blocks=b)
        assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    k, v = pkg.cache_read(cache, table, lens, 0, cu=cu)
    assert k.shape == v.shape == (0, 2, 64)
    pkg.hdp_device_status()
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.scales, cache.bounds)))


# ---------------------------------------------------------------- choice of blocks

@pytest.mark.parametrize("blocks,rows,count,hkv", [(700, 1, 3, 2), (4096, 3, 512, 1), (4097, 40, 64, 2), (9000, 99, 20, 1),
                                                   (700, 50, 16, 2), (5000, 101, 64, 1), (9000, 52, 33, 2), (20000, 100, 512, 1)])
def test_select_with_and_without_a_kernel_for_the_scores(blocks, rows, count, hkv):
    """On both sides of the rule (100 rows times heads), 1 to 8 CTAs a row and head, rows of unequal lengths."""
    d = 64
    g = torch.Generator().manual_seed(blocks + rows)
    bounds = torch.randint(-90, 91, (blocks, hkv, 2, d), generator=g).sort(2).values.to(torch.int8)
    scales = torch.exp2(torch.randint(-1, 1, (blocks, hkv, 2), generator=g).float())
    cache = pkg.KVCache(torch.empty((blocks, hkv, 64, d), dtype=torch.uint8, device="cuda"),
                        torch.empty((blocks, hkv, d, 64), dtype=torch.uint8, device="cuda"), scales.cuda(), bounds.cuda(), 0)
    table = torch.stack([torch.randperm(blocks, generator=g) for _ in range(rows)]).int()
    q = torch.randint(-127, 128, (rows, hkv, d), generator=g).to(torch.bfloat16)
    q[:, :, 0] = 127  # whole numbers that the rounding of q leaves alone
    lens = torch.randint(1, blocks * 64 + 1, (rows,), generator=g).int()
    lens[0] = blocks * 64
    got = pkg.cache_select(cache, table.cuda(), lens.cuda(), q.cuda(), count, keep_first=1, keep_last=min(2, count - 1)).cpu()
    pkg.hdp_device_status()
    for r in range(rows):
        have = (int(lens[r]) - 1) // 64 + 1
        page = table[r, :have].long()
        for h in range(hkv):
            x, b = q[r, h].long(), bounds[page, h].long()
            score = (b[:, 1] @ x.clamp(min=0) + b[:, 0] @ x.clamp(max=0)).float() * scales[page, h, 0]
            score[:1] = score[max(0, have - min(2, count - 1)):] = float("inf")
            want = score.sort(descending=True, stable=True).indices[:count].sort().values
            assert torch.equal(got[r, h, :len(want)].long(), want) and (got[r, h, len(want):] == -1).all(), (r, h)


# ---------------------------------------------------------------- streams and graphs

def test_inputs_that_die_while_another_stream_reads_them():
    """Temporaries as arguments of a call on another stream: what the caller's stream allocates next must not be given
    their memory before the call has read them."""
    cache, table, lens = _filled([1000, 700], 2, 64, 1, 4)
    q, k, v = _bf16((2, 8, 64), 5), _bf16((2, 2, 64), 6), _bf16((2, 2, 64), 7)
    cu = _i32([0, 1, 2])
    state = [t.clone() for t in (cache.k, cache.v, cache.scales, cache.bounds)]

    def calls(stream, t):
        """All calls, with arguments that only the call holds (t makes them)."""
        now = lens + 1
        pkg.cache_append(cache, t(table), t(now), t(k), t(v), cu=t(cu), stream=stream)
        b = pkg.cache_select(cache, t(table), t(now), t(q), 4, cu=t(cu), stream=stream)
        return (b, *pkg.cache_attention(cache, t(table), t(now), t(q), cu=t(cu), stream=stream),
                *pkg.cache_attention(cache, t(table), t(now), t(q), cu=t(cu), blocks=b, stream=stream),
                *pkg.cache_read(cache, t(table), t(now), 2, cu=t(cu), stream=stream))

    want = calls(None, lambda x: x)
    side = torch.cuda.Stream()
    for again in range(2):  # the first time for the memory pools' sake
        for x, y in zip((cache.k, cache.v, cache.scales, cache.bounds), state):
            x.copy_(y)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)  # half a second in front of the calls
        got = calls(side, torch.clone)
        junk = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in [512] * 200 + [2048] * 50 + [4096] * 50]
        torch.cuda.current_stream().synchronize()
        waiting = not side.query()
        side.synchronize()
        del junk
    if not waiting:
        pytest.skip("the host took longer than the delay: the calls ran before the temporaries' memory was given out again")
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pkg.hdp_device_status()


def test_streams_that_torch_does_not_own():
    """A raw handle, an external stream and any object with a handle: the same results, and nothing noted on them."""
    cache, table, lens = _filled([300, 70], 2, 64, 1, 12)
    q, k = _bf16((2, 4, 64), 13), _bf16((2, 2, 64), 14)
    lens.add_(1)
    pkg.cache_append(cache, table, lens, k, k)
    want = pkg.cache_attention(cache, table, lens, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    class Other:
        cuda_stream = side.cuda_stream

    for stream in (side.cuda_stream, torch.cuda.ExternalStream(side.cuda_stream), Other()):
        pkg.cache_append(cache, table, lens, k, k, stream=stream)
        side.synchronize()
        if not isinstance(stream, Other):  # outputs need a stream that torch can allocate on
            got = pkg.cache_attention(cache, table, lens, q, stream=stream)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(pkg.cache_attention(cache, table, lens, q), want))


def test_a_captured_call_on_a_forked_stream():
    """Inside a capture, attention on another stream than the capture's, with a temporary as its input."""
    cache, table, lens = _filled([1000, 700], 2, 64, 0, 8)
    q = _bf16((2, 8, 64), 9)
    want = pkg.cache_attention(cache, table, lens, -q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        negative = -q
        side.wait_stream(torch.cuda.current_stream())
        outs = pkg.cache_attention(cache, table, lens, negative, stream=side)
        del negative
        torch.cuda.current_stream().wait_stream(side)
        blank = [torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    for _ in range(3):
        for t in outs:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and not any(t.any() for t in blank)
    del graph, outs, blank
    torch.cuda.synchronize()
    assert torch.equal(pkg.cache_attention(cache, table, lens, -q)[0], want[0])


def test_two_graphs_overlap():
    """Captured steps of two models on two streams, replayed without waiting for each other, each with the results that
    it has alone."""
    models = []
    for m, (lens, hq, hkv, d, fmt) in enumerate([([40000, 100, 9000], 8, 2, 128, 1), ([30000] * 4, 4, 4, 64, 0)]):
        cache, table, dl = _filled([l - 1 for l in lens], hkv, d, fmt, 11 + m)
        dl.add_(1)
        n = len(lens)
        q, k, v = _bf16((n, hq, d), 21 + m), _bf16((n, hkv, d), 31 + m), _bf16((n, hkv, d), 41 + m)

        def step(cache=cache, table=table, dl=dl, q=q, k=k, v=v):
            pkg.cache_append(cache, table, dl, k, v)  # the same rows at the same places: nothing changes after the first
            b = pkg.cache_select(cache, table, dl, q, 20)
            return (b, *pkg.cache_attention(cache, table, dl, q), *pkg.cache_attention(cache, table, dl, q, blocks=b),
                    *pkg.cache_read(cache, table, dl, dl.shape[0]))

        step()
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        models.append((graph, torch.cuda.Stream(), outs, want, step))  # step keeps the graph's inputs
    for _ in range(5):
        for _, _, outs, _, _ in models:
            for t in outs:
                t.fill_(7)
        torch.cuda.synchronize()
        for _ in range(6):
            for graph, stream, _, _, _ in models:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, outs, want, _ in models:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    pkg.hdp_device_status()
