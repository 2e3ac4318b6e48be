"""Rotary positions beside autograd: no history, in-place turns that a backward pass notices, and the explicit backward
call in a torch.autograd.Function."""
import pytest
import torch

import packed_varlen_attention_aware_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def _inputs(requires_grad):
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k = (torch.randn(21, h, 32, device="cuda", generator=g).requires_grad_(requires_grad) for h in (4, 2))
    return q, k, torch.arange(21, dtype=torch.int32, device="cuda") * 37, torch.rand(12, dtype=torch.float64, device="cuda")


def test_what_is_returned_has_no_history():
    q, k, pos, f = _inputs(True)
    a, b = pkg.rotary(q, k, pos, f)
    assert a.grad_fn is None and not a.requires_grad and b.grad_fn is None and q._version == k._version == 0


@pytest.mark.parametrize("turn", [pkg.rotary, pkg.rotary_backward])
def test_a_backward_pass_notices_what_was_turned_in_place(turn):
    q, k, pos, f = _inputs(True)
    x = q * 1.0
    y = x * x  # keeps x
    x = x.detach()
    turn(x, None, pos, f, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    fused = torch.zeros(21, 6, 32, device="cuda")
    turn(fused[:, :4], fused[:, 4:], pos, f, inplace=True)
    assert fused._version > 0
    with torch.inference_mode():
        z = torch.ones(21, 6, 32, device="cuda")
        turn(z[:, :4], None, pos, f, inplace=True)
    turn(z[:, 4:], None, pos, f, inplace=True)  # a tensor without versions


def test_the_backward_call_in_an_autograd_function():
    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, pos, f):
            ctx.save_for_backward(pos, f)
            return pkg.rotary(q, k, pos, f, factor=1.5)

        @staticmethod
        def backward(ctx, dq, dk):
            return (*pkg.rotary_backward(dq, dk, *ctx.saved_tensors, factor=1.5), None, None)

    q, k, pos, f = _inputs(True)
    a, b = Turn.apply(q, k, pos, f)
    wa, wb = torch.randn_like(a), torch.randn_like(b)
    ((a * wa).sum() + (b * wb).sum()).backward()
    # the turn is linear: its gradient along any direction u is the turned u, <w, R u> = <R^T w, u>
    u, v = torch.randn_like(a), torch.randn_like(b)
    ru, rv = pkg.rotary(u, v, pos, f, factor=1.5)
    for w, r, grad, x in ((wa, ru, q.grad, u), (wb, rv, k.grad, v)):
        left, right = (w.double() * r.double()).sum(), (grad.double() * x.double()).sum()
        size = (w.double().abs() * r.double().abs()).sum() + (grad.double().abs() * x.double().abs()).sum()
        assert (left - right).abs() <= 2.0 ** -20 * size  # each product off by 2^-20 of its size at most
