"""Refusals of the cache calls: the C entry points check sizes, pointers and alignment before any CUDA call, the
binding checks types, shapes and devices.  No GPU is needed."""
import ctypes

import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from packed_varlen_attention_aware_gb300 import binding
from packed_varlen_attention_aware_gb300 import build as native_build

INVALID, UNSUPPORTED = pkg.HDP_ERR_INVALID_ARGUMENT, pkg.HDP_ERR_UNSUPPORTED
V = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return pkg.load()


def _cache(**changes):
    f = dict(k=256, v=256, scales=256, bounds=256, num_pages=4, hkv=2, d=64, format=0, page_table=256, lens=256,
             num_seqs=3, max_pages=2)
    f.update(changes)
    return binding.CacheStruct(**f)


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(scales=None), INVALID), (dict(bounds=None), INVALID),
    (dict(page_table=None), INVALID), (dict(lens=None), INVALID), (dict(num_pages=0), INVALID), (dict(hkv=0), INVALID),
    (dict(num_seqs=0), INVALID), (dict(max_pages=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(format=2), INVALID), (dict(k=264), INVALID), (dict(v=257), INVALID), (dict(bounds=260), INVALID),
    (dict(scales=260), INVALID), (dict(num_seqs=(1 << 24) + 1), UNSUPPORTED), (dict(hkv=65536), UNSUPPORTED)]


def _append(lib, c, cu=V(256), rows=3, k=V(256), v=V(256)):
    return lib.hdp_cache_append(c, cu, rows, k, v, None)


def _read(lib, c, cu=V(256), rows=3, k=V(256), v=V(256)):
    return lib.hdp_cache_read(c, cu, rows, k, v, None)


def _attend(lib, c, cu=V(256), rows=3, q=V(256), hq=4, scale=0.1, blocks=None, count=0, ws=V(256), nbytes=1 << 40, o=V(256),
            lse=V(256)):
    return lib.hdp_cache_attention(c, cu, rows, q, hq, scale, blocks, count, ws, nbytes, o, lse, None)


def _select(lib, c, cu=V(256), rows=3, q=V(256), hq=4, count=2, first=0, last=1, ws=V(256), nbytes=1 << 40, blocks=V(256)):
    return lib.hdp_cache_select(c, cu, rows, q, hq, count, first, last, ws, nbytes, blocks, None)


@pytest.mark.parametrize("call", [_append, _read, _attend, _select])
def test_a_cache_that_is_not_one(lib, call):
    assert call(lib, None) == INVALID
    for changes, status in BAD_CACHES:
        rows = changes.get("num_seqs", 3)
        assert call(lib, _cache(**changes), rows=max(rows, 1)) == status, changes
        assert pkg.hdp_last_error_message().startswith("hdp_cache_")
    assert call(lib, _cache(), rows=-1) == INVALID
    assert call(lib, _cache(), rows=1 << 31) == INVALID
    assert call(lib, _cache(), cu=None, rows=4) == INVALID  # one row for each of three sequences
    assert call(lib, _cache(), rows=0) == pkg.HDP_OK


@pytest.mark.parametrize("call", [_append, _read])
def test_rows_that_cannot_be_moved(lib, call):
    for bad in (dict(k=None), dict(v=None), dict(k=V(264)), dict(v=V(258))):
        assert call(lib, _cache(), **bad) == INVALID, bad


def test_attention_refusals(lib):
    c = _cache()
    for bad in (dict(hq=0), dict(hq=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(count=4),
                dict(blocks=V(256), count=0), dict(blocks=V(256), count=-1), dict(q=None), dict(o=None), dict(lse=None),
                dict(q=V(264)), dict(o=V(264))):
        assert _attend(lib, c, **bad) == INVALID, bad
    assert _attend(lib, _cache(hkv=1), rows=1 << 30, hq=4) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.hdp_cache_attention_workspace_bytes(None, 4, ctypes.byref(n)) == INVALID
    assert lib.hdp_cache_attention_workspace_bytes(c, 3, ctypes.byref(n)) == INVALID
    assert lib.hdp_cache_attention_workspace_bytes(_cache(d=80), 4, ctypes.byref(n)) == UNSUPPORTED
    assert lib.hdp_cache_attention_workspace_bytes(c, 4, None) == INVALID


def test_select_refusals(lib):
    c = _cache()
    for bad in (dict(hq=0), dict(hq=5), dict(count=0), dict(first=-1), dict(last=-1), dict(first=2, last=1),
                dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(q=None), dict(blocks=None), dict(q=V(260)), dict(ws=None),
                dict(nbytes=3 * 2 * 2 * 4 - 1), dict(ws=V(128))):
        assert _select(lib, c, **bad) == INVALID, bad
    assert _select(lib, c, hq=2 * 129) == UNSUPPORTED
    assert _select(lib, _cache(max_pages=1 << 30), rows=1 << 20) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.hdp_cache_select_workspace_bytes(c, 3, ctypes.byref(n)) == pkg.HDP_OK and n.value == 256
    assert lib.hdp_cache_select_workspace_bytes(c, -1, ctypes.byref(n)) == INVALID
    assert lib.hdp_cache_select_workspace_bytes(None, 3, ctypes.byref(n)) == INVALID


def test_the_binding_wants_cuda_tensors_of_the_right_types():
    k = torch.zeros((2, 1, 64, 64), dtype=torch.uint8)
    with pytest.raises(TypeError, match="CUDA"):
        pkg.KVCache(k, k, torch.zeros((2, 1, 2)), torch.zeros((2, 1, 2, 64), dtype=torch.int8), 0)
    with pytest.raises(ValueError, match="k must be"):
        pkg.KVCache(k[0], k, None, None, 0)


def test_an_empty_list_of_blocks_is_refused():
    """Width 0 must not be taken for "every block": its tensor has no address."""
    cache = object.__new__(pkg.KVCache)
    cache.hkv, cache._dev = 2, 0
    for shape in ((3, 2, 0), (0, 2, 0), (3, 2), (0,), ()):
        with pytest.raises(ValueError, match="blocks must be"):
            cache._blocks_of(torch.empty(shape, dtype=torch.int32), 3)
    assert cache._blocks_of(None, 3) == (0, None)


def test_no_rows_and_a_list_without_an_address(lib):
    assert _attend(lib, _cache(), rows=0, blocks=None, count=4, q=None, o=None, lse=None, ws=None) == pkg.HDP_OK
    assert _attend(lib, _cache(), rows=0, blocks=V(256), count=4) == pkg.HDP_OK
    assert _attend(lib, _cache(), rows=1, blocks=None, count=4) == INVALID
    assert _attend(lib, _cache(), rows=0, blocks=None, count=-1) == INVALID
    assert _attend(lib, _cache(), rows=0, blocks=V(256), count=0) == INVALID
