"""Query rows with an infinity or NaN over the caches of 8 and of 4 bits: they are NaN whatever the keys are, as long as
they see one, and nothing else is."""
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


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _empty(kind, pages, hkv, d):
    return pkg.KVCache4.empty(pages, hkv, d) if kind == "4bit" else pkg.KVCache.empty(pages, hkv, d, {"int8": pkg.HDP_CACHE_INT8, "e4m3": pkg.HDP_CACHE_E4M3}[kind])


@pytest.mark.parametrize("kind", ["4bit", "int8", "e4m3"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("tokens,rows,listed", [(10, 1, False), (64, 1, False), (500, 1, False), (300, 3, False), (500, 1, True)])
def test_rows_with_an_infinity_or_nan_are_nan(kind, bad, tokens, rows, listed):
    """Channel 0 of all keys is positive, so that the products of a row with an infinity there are all of one sign."""
    if listed and kind == "4bit":
        pytest.skip("no lists of blocks")
    rng = np.random.default_rng(tokens + rows)
    hkv, d = 2, 64
    pages = -(-tokens // 64)
    cache, table = _empty(kind, pages, hkv, d), _i32(rng.permutation(pages))[None]
    k, v = (torch.tensor(rng.normal(size=(tokens, hkv, d))).bfloat16().cuda() for _ in "kv")
    k[:, :, 0] = k[:, :, 0].abs() + 1
    pkg.cache_append(cache, table, _i32([tokens]), k, v, cu=_i32([0, tokens]))
    q = torch.tensor(rng.normal(size=(rows, 8, d))).bfloat16().cuda()
    cu = _i32([0, rows])
    blocks = torch.arange(pages, dtype=torch.int32, device="cuda").expand(rows, hkv, pages).contiguous() if listed else None
    want = pkg.cache_attention(cache, table, _i32([tokens]), q, cu=cu, blocks=blocks)
    q[-1, 2, 0] = q[0, 7, 0] = bad
    for with_cu in (cu, None) if rows == 1 else (cu,):
        o, lse = pkg.cache_attention(cache, table, _i32([tokens]), q, cu=with_cu, blocks=blocks)
        gone = torch.zeros((rows, 8), dtype=torch.bool, device="cuda")
        gone[-1, 2] = gone[0, 7] = True
        assert torch.isnan(o[gone]).all() and torch.isnan(lse.t()[gone]).all()
        assert torch.isfinite(o[~gone]).all() and torch.isfinite(lse.t()[~gone]).all()
        assert ((lse - want[1]).t()[~gone].abs() < 1e-5).all() and ((o - want[0])[~gone].abs() <= 2.0 ** -7 * want[0][~gone].abs() + 2.0 ** -9).all()


@pytest.mark.parametrize("kind", ["4bit", "int8", "e4m3"])
def test_rows_before_the_first_token_see_no_key_whatever_they_hold(kind):
    rng = np.random.default_rng(3)
    cache, table = _empty(kind, 1, 1, 64), _i32([[0]])
    x = torch.tensor(rng.normal(size=(5, 1, 64))).bfloat16().cuda().abs() + 1
    pkg.cache_append(cache, table, _i32([5]), x, x, cu=_i32([0, 5]))
    q = torch.zeros((7, 4, 64), dtype=torch.bfloat16, device="cuda")
    q[:3, :, 0] = -float("inf")
    o, lse = pkg.cache_attention(cache, table, _i32([5]), q, cu=_i32([0, 7]))  # rows 0 and 1 stand before the first token
    assert not o[:2].any() and torch.isneginf(lse[:, :2]).all()
    assert torch.isnan(o[2]).all() and torch.isnan(lse[:, 2]).all() and torch.isfinite(o[3:]).all() and torch.isfinite(lse[:, 3:]).all()
