"""Rotary positions: rows at negative positions are left alone on every way through a head."""
import numpy as np
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg
from test_gpu_rows import TYPES, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("d,rot,pitch,offset", [(128, 128, 128, 0), (128, 64, 128, 0), (64, 48, 66, 0), (64, 46, 66, 2), (64, 46, 66, 1),
                                               (64, 36, 64, 0), (64, 30, 64, 0), (128, 126, 128, 0), (10, 6, 10, 0)])
def test_rows_at_negative_positions_on_every_way_through_a_head(dtype, neighbours, d, rot, pitch, offset):
    """In place and into outputs that hold something: nothing of those rows is written, whatever they hold; the others are
    what they are without them."""
    rng = np.random.default_rng(rot + offset)
    whole = torch.tensor(rng.normal(size=23 * 5 * pitch + offset)).to(dtype).cuda()
    x = whole[offset:].view(23, 5, pitch)[:, :, :d]
    pos = rng.integers(0, 9999, 23)
    gone = np.isin(np.arange(23), [0, 5, 6, 7, 13, 22])
    pos[gone] = [-1, -2 ** 31, -7, -1, -64, -3]
    f = torch.tensor(np.exp(-rng.uniform(0, 9, rot // 2)), device="cuda")
    keep, away = torch.tensor(~gone, device="cuda"), torch.tensor(gone, device="cuda")
    want = pkg.rotary(x[keep][:, :3], x[keep][:, 3:], _i32(pos[~gone]), f, neighbours=neighbours)
    x[away] = float("nan")
    outs = [torch.full((23, h, d), 7.0, dtype=dtype, device="cuda") for h in (3, 2)]
    pkg.hdp_rotary(x[:, :3], x[:, 3:], _i32(pos), f, *outs, neighbours=neighbours)
    for o, w in zip(outs, want):
        assert torch.equal(o[keep], w) and (o[away] == 7).all()
    before = whole.clone()
    pkg.rotary(x[:, :3], x[:, 3:], _i32(pos), f, neighbours=neighbours, inplace=True)
    assert torch.equal(x[keep], torch.cat(want, 1)) and torch.isnan(x[away]).all()
    x[keep] = before[offset:].view(23, 5, pitch)[:, :, :d][keep]
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    assert torch.equal(whole.view(bits), before.view(bits))
