"""The policy loss's sums, and what a ratio that is not a number reaches."""
import math

import numpy as np
import pytest
import torch

from tests.operator_reference import f64

U = 2.0 ** -24                                      # half a float32 step, relative


@pytest.mark.gpu
@pytest.mark.parametrize("token_adv", [False, True])
@pytest.mark.parametrize("ratio", ["token", "sequence_token"])
@pytest.mark.parametrize("T", [20, 300, 9000])
def test_without_an_advantage_no_ratio_counts(T, ratio, token_adv):
    """Whatever it is: tokens without an advantage have the gradient of their KL term."""
    import grpo_loss_gb300 as G
    B = 30
    g = torch.Generator(device="cuda").manual_seed(T)
    q = -torch.rand(B, T, generator=g, device="cuda")
    old = q + 0.1 * torch.randn(B, T, generator=g, device="cuda")
    ref = q + 0.1 * torch.randn(B, T, generator=g, device="cuda")
    mask = torch.rand(B, T, generator=g, device="cuda") < 0.9
    mask[:, :2] = True
    old[::3, 0], old[1::3, 0], old[2::3, 0] = math.nan, -math.inf, math.inf
    adv = torch.zeros((B, T) if token_adv else (B,), device="cuda")
    for r, beta in ((None, 0.0), (ref, 0.1)):
        loss, d, stats = G.policy_loss(q, adv, mask, old, r, ratio=ratio, beta=beta)
        x = np.zeros((B, T)) if r is None else f64(r) - f64(q)
        m = mask.cpu().numpy()
        c = m / (B * m.sum(1, keepdims=True))
        k, e = np.expm1(x) - x, np.expm1(x)
        # e^x - 1: its argument's rounding, half a step of |x| <= 1, and a few of its own
        assert np.all(np.abs(f64(d) + c * beta * e) <= c * beta * (8 * U * np.abs(e) + 4 * U * np.abs(x)))
        assert abs(loss.item() - (c * beta * k).sum()) <= 1e-4 * (c * beta * k).sum()
        assert stats[1] == stats[2] == 0
