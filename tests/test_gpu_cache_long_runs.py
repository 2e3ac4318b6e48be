"""Attention over the caches where one warp has a very long run: its sums may not drift.  All sequences share a few pages,
which hold every block's keys again, so that the outputs are those of these pages alone."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["4bit", "int8", "e4m3"])
@pytest.mark.parametrize("tokens,d,new", [(131072, 128, 1), (131072, 64, 3), (2097152, 64, 1)])
def test_long_runs_keep_their_sums(kind, tokens, d, new):
    """A warp for each sequence.  Off by: bf16's rounding, 2^-8 of an output; P's, 2^-11 of each weight; scores that are fp32
    sums of d products, 2^-16 of their magnitudes, twice; 2^-18 for exponentials and logarithms.  And by fp32's own sums: at
    2M tokens a lane adds 2^18 weights, the last of them to a sum in which half a step is 2^-24 * 2^18 = 2^-6 of such a
    weight, 2^-7 on the way there; there are 512 different ones, so that 2^-7 / sqrt(3 * 512) = 2^-12.3 of the sum is left.
    Of the output's sums likewise: 2^15 blocks' of 8 kinds, 2^-10 / sqrt(3 * 8) = 2^-12.3.  2^-10 is allowed for each.
    On average over outputs that are not equal bf16 numbers all of these go both ways: the rounding of 150,000 outputs
    leaves 2^-9 / sqrt(3 * 150,000) = 2^-18 of their mean, what a row's outputs share less than 2^-12 / sqrt(4,800) = 2^-18;
    2^-14 is allowed."""
    n = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(tokens + d)
    pages, one = 8, lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache = pkg.KVCache4.empty(pages, 1, d) if kind == "4bit" else pkg.KVCache.empty(pages, 1, d, {"int8": pkg.HDP_CACHE_INT8, "e4m3": pkg.HDP_CACHE_E4M3}[kind])
    k, v = (torch.randn(64 * pages, 1, d, generator=g, device="cuda") for _ in "kv")
    v = v.abs()
    v[:, :, :d // 2] = 1.5
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    pkg.cache_append(cache, table, one(64 * pages), k.bfloat16(), v.bfloat16(), cu=one(0, 64 * pages))
    k, v = (x[:, 0].double() for x in pkg.cache_read(cache, table, one(64 * pages), 64 * pages, cu=one(0, 64 * pages)))
    q = (torch.randn(n * new, 4, d, generator=g, device="cuda") * 0.5).bfloat16()
    cu = None if new == 1 else torch.arange(n + 1, dtype=torch.int32, device="cuda") * new
    lens = torch.full((n,), tokens + new - 1, dtype=torch.int32, device="cuda")
    wide = torch.cat((table.repeat(n, tokens // 64 // pages), torch.zeros((n, 1), dtype=torch.int32, device="cuda")), 1)
    o, lse = pkg.cache_attention(cache, wide, lens, q, cu=cu)
    o, lse = (x.double() for x in (o.view(n, new, 4, d)[:, 0], lse.t().reshape(n, new, 4)[:, 0]))  # the first row sees whole pages
    q = q.view(n, new, 4, d)[:, 0].double()
    x, size = q @ k.t() * d ** -0.5, (q.abs() @ k.abs().t() * d ** -0.5).amax(-1, keepdim=True)
    want, rows = x.softmax(-1) @ v, x.logsumexp(-1) + np.log(tokens / (64 * pages))
    sums = 2.0 ** -10 * tokens / 2 ** 21
    off = (o - want).abs()
    limit = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15 * size + 2.0 ** -18 + 2 * sums) * want  # V is positive: want is the sum of weight |v|
    assert (off <= limit).all(), float((off / limit).max())
    assert (o / want - 1)[..., d // 2:].mean().abs() <= 2.0 ** -14
    assert ((lse - rows).abs() <= 2.0 ** -16 * size[..., 0] + 2.0 ** -18 + sums).all()
