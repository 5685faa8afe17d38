"""The loss's gradients come from kernels and have no graph of their own: asking for
their gradients is an error. On the CPU, with an engine that stands in for the kernels."""
import pytest
import torch


class Engine:
    """loss = sum(H^2) sum(W^2): gradients 2 H sum(W^2) and 2 W sum(H^2)."""
    e4m3 = False

    def __init__(self, compute_dW):
        self.compute_dW, self.dW = compute_dW, None

    def forward(self, H, H_ref, W, ids, mask, adv):
        return (H * H).sum().reshape(1) * (W * W).sum(), H.new_zeros(1), None, None

    def backward(self, H, W, ids, mask, adv, grad_loss, dH=None):
        dH.copy_(2 * grad_loss * H * (W * W).sum())
        self.dW = 2 * grad_loss * W * (H * H).sum() if self.compute_dW else None
        return dH


@pytest.mark.parametrize("compute_dW", [False, True])
@pytest.mark.parametrize("outer", [lambda v: v, lambda v: 3 * v, lambda v: v.square()], ids=["loss", "scaled", "square"])
def test_second_derivatives_of_the_loss_are_refused(outer, compute_dW):
    import grpo_loss_gb300 as G
    H = torch.randn(4, 3, requires_grad=True)
    W = torch.randn(5, 3, requires_grad=compute_dW)
    ids = mask = adv = torch.zeros(4)
    f = lambda: outer(G.grpo_loss(H, None, W, ids, mask, adv, Engine(compute_dW))[0])  # noqa: E731
    (want,) = torch.autograd.grad(outer((H * H).sum() * (W * W).sum()), H)
    (got,) = torch.autograd.grad(f(), H)
    assert torch.allclose(got, want)
    (gH,) = torch.autograd.grad(f(), H, create_graph=True)
    assert torch.allclose(gH, want)
    with pytest.raises(RuntimeError, match="once differentiable"):
        torch.autograd.grad(gH.pow(2).sum() + H.pow(2).sum(), H)
