"""The policy loss's sums over many tokens, and what a ratio that is not a number reaches."""
import math

import numpy as np
import pytest
import torch

from tests.operator_reference import f64

U = 2.0 ** -24                                      # half a float32 step, relative


@pytest.mark.gpu
@pytest.mark.parametrize("token_adv", [False, True])
def test_one_long_sequence_of_equal_tokens(token_adv):
    """Tokens that are alike: every partial sum rounds the same way, and nothing averages
    out. Per token the values are off by 20 half steps at most (the exponential's argument,
    series and products); a thread adds 36 pairs before its sum is kept in two floats, a half
    step each of what has been added up; the rest is wider than float32."""
    import grpo_loss_gb300 as G
    T = 3 * 2 ** 25 + 5
    w, x = 0.3, -0.4
    q = torch.full((1, T), -1.0, device="cuda")
    old, ref = q - w, q + x
    wf, xf = (q[0, 0].double() - old[0, 0].double()).item(), (ref[0, 0].double() - q[0, 0].double()).item()
    mask = torch.ones(1, T, dtype=torch.bool, device="cuda")
    adv = torch.full((1, T) if token_adv else (1,), -0.7, device="cuda")
    A = -adv.flatten()[0].double().item()
    rel = (20 + 36 + 4) * U
    for reduce, divisor in (("token", None), ("constant", 1000.0)):
        loss, d, stats = G.policy_loss(q, adv, mask, old, ref, clip=(0.2, 0.2), beta=0.05, reduce=reduce, divisor=divisor, dlogp=None)
        n = T / (T if divisor is None else divisor)
        k, r = math.expm1(xf) - xf, math.exp(wf)
        # the advantage's part is summed as c A n and c A (r - 1), each with its own error
        want = n * (A * r + 0.05 * k)
        assert abs(loss.item() - want) <= rel * n * (A + A * (r - 1) + 0.05 * k)
        got = f64(stats)
        assert abs(got[0] - k) <= rel * k and abs(got[3] - r) <= rel * (r - 1) + 2 * U * r and got[1] == got[2] == 0
        each = n / T * (A * r - 0.05 * math.expm1(xf))
        assert abs(d.min().item() - each) <= 30 * U * abs(each) and d.max() == d.min()


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


@pytest.mark.gpu
@pytest.mark.parametrize("token_adv", [False, True])
@pytest.mark.parametrize("T", [60, 3000])
def test_far_tokens_among_others(T, token_adv):
    """Tokens too far from the drawing policy for the series, and on a bound, beside others
    of the same lane."""
    from tests.test_policy_loss import check, inputs
    q, adv, mask, old, ref = inputs(7, T, seed=11, fill=0.8, token_adv=token_adv)
    live = torch.where(mask, torch.ones_like(q), torch.full_like(q, math.nan))
    old[:, 5::97] = ((q - 0.01)[:, 5::97] + 90.0) * live[:, 5::97]      # a ratio near 0
    old[:, 9::83] = q[:, 9::83] * live[:, 9::83]                        # a ratio of 1
    ref[:, 7::71] = (q[:, 7::71] - 85.0) * live[:, 7::71]
    for kw in (dict(clip=(0.0, 0.0)), dict(clip=(0.2, 0.28), dual_clip=3.0)):
        check(q, adv, mask, old, ref, beta=0.01, **kw)
        check(q, adv, mask, old, ref, beta=0.01, reduce="token", **kw)
