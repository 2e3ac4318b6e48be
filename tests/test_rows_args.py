"""Refusals of the 4-bit cache, the block tables and the rotary positions: the C entry points check before any CUDA call,
the binding checks types, shapes and devices.  No GPU is needed."""
import ctypes
import math

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
    f = dict(k=256, v=256, scales=256, num_pages=4, hkv=2, d=64, page_table=256, lens=256, num_seqs=3, max_pages=2)
    f.update(changes)
    return binding.Cache4Struct(**f)


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(scales=None), INVALID), (dict(page_table=None), INVALID),
    (dict(lens=None), INVALID), (dict(num_pages=0), INVALID), (dict(hkv=0), INVALID), (dict(num_seqs=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(k=264), INVALID),
    (dict(v=257), INVALID), (dict(scales=260), INVALID), (dict(num_seqs=(1 << 24) + 1), UNSUPPORTED), (dict(hkv=65536), UNSUPPORTED)]


def _append(lib, c, cu=V(256), rows=3, k=V(256), v=V(256)):
    return lib.hdp_fourbit_append(c, cu, rows, k, v, None)


def _read(lib, c, cu=V(256), rows=3, k=V(256), v=V(256)):
    return lib.hdp_fourbit_read(c, cu, rows, k, v, None)


def _attend(lib, c, cu=V(256), rows=3, q=V(256), hq=4, scale=0.1, ws=V(256), nbytes=1 << 40, o=V(256), lse=V(256)):
    return lib.hdp_fourbit_attention(c, cu, rows, q, hq, scale, ws, nbytes, o, lse, None)


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_a_cache_that_is_not_one(lib, call):
    assert call(lib, None) == INVALID
    for changes, status in BAD_CACHES:
        assert call(lib, _cache(**changes), rows=max(changes.get("num_seqs", 3), 1)) == status, changes
        assert pkg.hdp_last_error_message().startswith("hdp_fourbit_")
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
    for bad in (dict(hq=0), dict(hq=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(q=None), dict(o=None),
                dict(lse=None), dict(q=V(264)), dict(o=V(264))):
        assert _attend(lib, c, **bad) == INVALID, bad
    assert _attend(lib, _cache(hkv=1), rows=1 << 30, hq=4) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.hdp_fourbit_attention_workspace_bytes(None, 4, ctypes.byref(n)) == INVALID
    assert lib.hdp_fourbit_attention_workspace_bytes(c, 3, ctypes.byref(n)) == INVALID
    assert lib.hdp_fourbit_attention_workspace_bytes(_cache(d=80), 4, ctypes.byref(n)) == UNSUPPORTED
    assert lib.hdp_fourbit_attention_workspace_bytes(c, 4, None) == INVALID


def test_assign_refusals(lib):
    ok = dict(free=V(256), count=V(256), pages=4, table=V(256), held=V(256), lens=V(256), n=3, cols=2)
    call = lambda **x: lib.hdp_cache_assign(*{**ok, **x}.values(), None)
    for name in ("free", "count", "table", "held", "lens"):
        assert call(**{name: None}) == INVALID, name
    for name in ("pages", "n", "cols"):
        assert call(**{name: 0}) == INVALID and call(**{name: -1}) == INVALID, name
    assert call(n=(1 << 24) + 1) == UNSUPPORTED


def test_row_map_refusals(lib):
    ok = dict(table=V(256), lens=V(256), cu=V(256), n=3, cols=2, pages=4, rows=5, seq=V(256), pos=V(256), slot=V(256))
    call = lambda **x: lib.hdp_cache_rows(*{**ok, **x}.values(), None)
    for bad in (dict(lens=None), dict(n=0), dict(rows=-1), dict(rows=1 << 31), dict(cu=None), dict(table=None), dict(cols=0), dict(pages=0)):
        assert call(**bad) == INVALID, bad
    assert call(n=(1 << 24) + 1) == UNSUPPORTED
    assert call(rows=0) == pkg.HDP_OK and call(rows=0, table=None, slot=None, cols=0, pages=0) == pkg.HDP_OK


def _rows(**changes):
    f = dict(in_=256, out=512, in_row_stride=256, in_head_stride=64, out_row_stride=256, out_head_stride=64, heads=4)
    f.update(changes)
    return binding.RotaryRows(**f)


def test_rotary_refusals(lib):
    ok = dict(q=_rows(), k=None, rows=3, d=64, type=0, pos=V(256), freqs=V(256), rot=64, flags=0, factor=1.0)
    call = lambda **x: lib.hdp_rotary(*{**ok, **x}.values(), None)
    for bad in (dict(q=None), dict(rows=-1), dict(rows=1 << 31), dict(d=1), dict(rot=0), dict(rot=63), dict(rot=66), dict(type=3), dict(type=-1),
                dict(flags=4), dict(factor=0.0), dict(factor=-1.0), dict(factor=math.inf), dict(factor=math.nan), dict(pos=None), dict(freqs=None),
                dict(freqs=V(260)), dict(k=_rows()), dict(k=_rows(in_=1024)), dict(k=_rows(out=256)), dict(k=_rows(in_=512, out=1024)),
                dict(q=_rows(heads=-1)), dict(q=_rows(heads=(1 << 20) + 1)), dict(q=_rows(in_=None)), dict(q=_rows(out=None)),
                dict(q=_rows(in_=257)), dict(q=_rows(out=513)), dict(type=2, q=_rows(in_=258)), dict(q=_rows(out=256, out_row_stride=512)),
                dict(k=_rows(out=256, out_head_stride=128))):
        assert call(**bad) == INVALID, bad
        assert pkg.hdp_last_error_message().startswith("hdp_rotary: ")
    assert call(d=258, rot=64) == UNSUPPORTED
    assert call(rows=0) == call(rows=0, q=_rows(in_=None, out=None, out_row_stride=1)) == call(q=_rows(heads=0)) == pkg.HDP_OK


def test_the_binding_wants_cuda_tensors_of_the_right_types():
    byte = lambda *s: torch.zeros(s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        pkg.KVCache4(byte(2, 1, 64, 32), byte(2, 1, 4, 512), byte(2, 1, 3, 64))
    with pytest.raises(ValueError, match="k must be"):
        pkg.KVCache4(byte(1, 64, 32), None, None)
    with pytest.raises(TypeError, match="CUDA"):
        pkg.PagePool(i32(4), i32(1))
    with pytest.raises(TypeError, match="CUDA"):
        pkg.cache_rows(i32(4), 4)
    x = torch.zeros((3, 2, 8))
    with pytest.raises(TypeError, match="CUDA"):
        pkg.rotary(x, x, i32(3), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError, match="one of them"):
        pkg.hdp_rotary(None, None, i32(3), torch.zeros(4, dtype=torch.float64), None, None)


def test_a_4_bit_cache_has_no_lists_of_blocks():
    cache = object.__new__(pkg.KVCache4)
    cache.hkv, cache._dev = 2, 0
    with pytest.raises(TypeError, match="no lists"):
        cache._blocks_of(torch.empty((3, 2, 4), dtype=torch.int32), 3)
    assert cache._blocks_of(None, 3) == (0, None)
    with pytest.raises(TypeError, match="hdp_cache_select is not for"):
        cache._call("hdp_cache_select", None)


def test_outputs_whose_rows_overlap_are_found():
    x = torch.zeros(4 * 3 * 8)
    assert binding._apart(x.view(4, 3, 8)) and binding._apart(x.view(3, 4, 8).transpose(0, 1)) and binding._apart(x[:8].view(1, 1, 8))
    assert not binding._apart(x.as_strided((4, 3, 8), (0, 8, 1))) and not binding._apart(x.as_strided((2, 3, 8), (16, 8, 1)))
    assert not binding._apart(x.as_strided((2, 2, 8), (4, 16, 1)))


def test_frequencies():
    f, factor = pkg.rotary_frequencies(8, base=10000.0, device="cpu")
    assert f.dtype == torch.float64 and factor == 1.0 and torch.allclose(f, torch.tensor([1, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.allclose(pkg.rotary_frequencies(8, scaling="linear", by=4, device="cpu")[0], f / 4)
    g = pkg.rotary_frequencies(8, scaling="base", by=4, device="cpu")[0]
    assert g[0] == 1 and math.isclose(g[-1], f[-1] / 4)  # the slowest pair goes four times slower
    g, factor = pkg.rotary_frequencies(64, scaling="parts", by=4, trained=4096, device="cpu")
    f = pkg.rotary_frequencies(64, device="cpu")[0]
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.allclose(g[turns < 1], f[turns < 1] / 4)
    assert (g <= f).all() and (g >= f / 4 * (1 - 1e-12)).all() and math.isclose(factor, 0.1 * math.log(4) + 1)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=0), dict(rot=8, scaling="other"), dict(rot=8, by=0), dict(rot=8, scaling="parts"),
                dict(rot=8, scaling="parts", trained=10, fast=1, slow=1)):
        with pytest.raises(ValueError):
            pkg.rotary_frequencies(**{"device": "cpu", **bad})
