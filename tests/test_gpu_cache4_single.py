"""Single tokens written into the 4-bit cache, values of every kind, against the oracle's bytes."""
import numpy as np
import pytest

import packed_varlen_attention_aware_gb300 as pkg
from test_gpu_cache4 import _bf16, _f64, _garbage, _i32, _pair, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_single_tokens_of_every_kind_are_the_oracles_bit_for_bit(d, hkv):
    """Codes and scales of K and of V, and what is left of the bytes that two tokens share: borders of the scales, ties,
    zeros, subnormal numbers, the largest ones, infinities and NaN."""
    rng = np.random.default_rng(d + hkv)
    rows = rng.normal(size=(70, hkv, d)) * np.exp2(rng.integers(-120, 120, (70, hkv, 1)))
    rows[0] = 0
    rows[1] = -0.0
    rows[2] = np.tile([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], d // 8)
    rows[3] = -rows[2] * 2.0 ** 40
    rows[4, :, 5] = 6.03125 * 2.0 ** 118
    rows[5] = 2.0 ** -133
    rows[6] = np.linspace(-1, 1, d) * 2.0 ** -126
    rows[7, :, 7] = 3.3895313892515355e38
    rows[8, :, 3], rows[9, :, d - 1], rows[10, :, 32] = np.inf, -np.inf, np.nan
    rows[11, :, ::7] = 2.0 ** -120
    k = _bf16(rows)
    v = k.flip(0)
    cache, ref = _pair(_garbage(2, hkv, d, rng))
    for r in range(70):
        pkg.cache_append(cache, _i32([[1, 0]]), _i32([r + 1]), k[r:r + 1].cuda(), v[r:r + 1].cuda())
        with np.errstate(invalid="ignore"):
            ref.append([[1, 0]], [r + 1], _f64(k[r:r + 1]), _f64(v[r:r + 1]), [0, 1])
    _same(cache, ref)
    back = pkg.cache_read(cache, _i32([[1, 0]]), _i32([70]), 70, cu=_i32([0, 70]))
    for got, want in zip(back, ref.sequence([1, 0], 70)):
        assert np.array_equal(_f64(got), want, equal_nan=True)
