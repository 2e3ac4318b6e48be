"""Rotary positions in place on views of one projection: apart they are turned, overlapping they are refused and left."""
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def _inputs():
    x = torch.randn(33, 12, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    return x, torch.arange(33, dtype=torch.int32, device="cuda"), torch.rand(32, dtype=torch.float64, device="cuda")


def test_views_that_share_a_head_are_refused():
    x, pos, f = _inputs()
    before = x.clone()
    for a, b in ((x[:, :5], x[:, 4:]), (x[:, 4:], x[:, :5]), (x[:, :8], x[:, 7:8]), (x[:, 2:3], x), (x[1:], x[:-1])):
        with pytest.raises(pkg.HdpError, match="rows of the other"):
            pkg.rotary(a, b, pos[:a.shape[0]], f, inplace=True)
        with pytest.raises(pkg.HdpError, match="rows of the other"):
            pkg.hdp_rotary(a, b, pos[:a.shape[0]], f, torch.empty_like(a), b)
    with pytest.raises(pkg.HdpError, match="its input or not overlap"):
        pkg.hdp_rotary(x[1:], None, pos[:32], f, x[:-1], None)
    assert torch.equal(x, before)


@pytest.mark.parametrize("q,k", [(slice(0, 8), slice(8, 10)), (slice(6, 12), slice(0, 2)), (slice(0, 12, 2), slice(1, 12, 2)), (slice(0, 9, 3), slice(10, 11))])
def test_views_that_share_none_are_turned(q, k):
    x, pos, f = _inputs()
    before = x.clone()
    want = pkg.rotary(before[:, q], before[:, k], pos, f)
    pkg.rotary(x[:, q], x[:, k], pos, f, inplace=True)
    assert torch.equal(x[:, q], want[0]) and torch.equal(x[:, k], want[1])
    rest = sorted(set(range(12)) - set(range(12)[q]) - set(range(12)[k]))
    assert torch.equal(x[:, rest], before[:, rest])
