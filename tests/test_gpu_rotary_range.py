"""Rotary positions: angles of any frequency at the farthest positions."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from test_gpu_rows import _f64, _i32

pytestmark = pytest.mark.gpu

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def _angle(pos, f):
    """pos * f within half a turn, as a fraction worked out exactly and rounded once."""
    x = Fraction(int(pos)) * Fraction(float(f))
    return float(x - 2 * PI * round(x / (2 * PI)))


@pytest.mark.parametrize("neighbours", [False, True])
def test_angles_of_any_frequency_at_far_positions(neighbours):
    """From the pair (1, 0) in fp32.  The fraction of a turn is exact to 2^-31 (2^-28.3 radians) and, as a fraction of half
    a turn, rounded to fp32 once (2^-25, times pi: 2^-23.3 radians); cosine and sine are off by two units of 2^-24 at most."""
    f = np.array([1.0, 0.7310585786300049, 3.0, 100.0, 1234.5678, 2.0 ** 30 + 0.5, 4.5e15, -5.25, -0.3, 1e-7, 3e-13, 1e-18, 1e-300, 5e-324, 0.0, 2 * np.pi])
    pos = np.array([0, 1, 2, 2097151, 2 ** 24 + 1, 123456789, 2 ** 31 - 2, 2 ** 31 - 1])
    n = len(f)
    x = torch.zeros((len(pos), 1, 2 * n), device="cuda")
    x[:, :, 0::2 if neighbours else 1] = 1
    if not neighbours:
        x[:, :, n:] = 0
    y = _f64(pkg.rotary(x, None, _i32(pos), torch.tensor(f, device="cuda"), neighbours=neighbours)[0])[:, 0]
    c, s = (y[:, 0::2], y[:, 1::2]) if neighbours else (y[:, :n], y[:, n:])
    angle = np.array([[_angle(p, t) for t in f] for p in pos])
    limit = 2.0 ** -28.3 + 2.0 ** -23.3 + 2.0 ** -23
    off = np.maximum(np.abs(c - np.cos(angle)), np.abs(s - np.sin(angle)))
    assert off.max() <= limit, [(int(pos[i]), float(f[j]), float(off[i, j])) for i, j in np.argwhere(off > limit)[:6]]
