"""The policy loss of a sequence's ratio, by what its gradient is the gradient of: with an
advantage for each sequence of the loss itself, with one for each token of the surrogate in
which every token has the sequence's ratio times its own probability over itself held
constant."""
import numpy as np
import pytest
import torch

from tests.operator_reference import f64
from tests.test_policy_loss import inputs


def surrogate(z, at, old, ref, mask, A, clip=(0.2, 0.2), dual=np.inf, beta=0.0, reduce="sequence", divisor=1.0, own=True):
    """The loss at log-probabilities z in float64, with token ratios r(at) e^(z - at), or with
    own = False the ratio r(z) of the sequence itself."""
    loss, total, B = 0.0, mask.sum(), len(mask)
    for b in range(B):
        t = np.flatnonzero(mask[b])
        if not len(t):
            continue
        mean = ((at if own else z)[b, t] - old[b, t]).mean()
        r = np.exp(mean + (z[b, t] - at[b, t] if own else 0.0 * z[b, t]))
        a = A[b, t] if A.ndim == 2 else np.full(len(t), A[b])
        l = np.where(a > 0, -a * np.minimum(r, 1 + clip[1]), -a * np.maximum(np.minimum(r, dual), 1 - clip[0]))
        x = ref[b, t] - z[b, t]
        c = {"sequence": 1.0 / (B * len(t)), "token": 1.0 / total, "constant": 1.0 / divisor}[reduce]
        loss += c * (l + beta * (np.expm1(x) - x)).sum()
    return loss


@pytest.mark.gpu
@pytest.mark.parametrize("ratio,token_adv,own", [("sequence_token", True, True), ("sequence_token", False, True), ("sequence_token", False, False),
                                                 ("sequence", False, False), ("sequence", True, True)])
@pytest.mark.parametrize("B,T", [(6, 40), (5, 300)])
def test_gradient_against_differences(B, T, ratio, token_adv, own):
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(B, T, seed=7, fill=0.6, token_adv=token_adv)
    m = mask.cpu().numpy()
    fix = lambda t: np.where(m, f64(t), 0.0)  # noqa: E731
    A = fix(adv) if token_adv else f64(adv)
    rng = np.random.default_rng(3)
    for kw in (dict(beta=0.1), dict(beta=0.0, reduce="token", dual_clip=1.5), dict(beta=0.05, reduce="constant", divisor=9.0, clip=(0.01, 0.02))):
        loss, d, _ = G.policy_loss(q, adv, mask, old, ref, ratio=ratio, **kw)
        kw = {{"dual_clip": "dual"}.get(k, k): v for k, v in kw.items()}
        f = lambda z: surrogate(z, fix(q), fix(old), fix(ref), m, A, own=own, **kw)  # noqa: E731
        assert abs(loss.item() - f(fix(q))) <= 1e-5 * abs(loss.item()) + 1e-7
        for _ in range(4):
            # float32's error on the gradient is some 20 half steps of 2^-24 of each of its terms, the
            # differences' own 1e-16 of the loss over the step and the step's second order: below 1e-9
            v, h = rng.standard_normal(q.shape) * m, 1e-6
            num = (f(fix(q) + h * v) - f(fix(q) - h * v)) / (2 * h)
            assert abs(num - (f64(d) * v).sum()) <= 1e-5 * np.abs(f64(d) * v).sum() + 1e-9


@pytest.mark.gpu
def test_names():
    """Of an advantage for each sequence both names are one; of one for each token
    ``policy_loss`` takes the shorter name for the longer."""
    import grpo_loss_gb300 as G
    for token_adv in (False, True):
        q, adv, mask, old, ref = inputs(5, 3000, token_adv=token_adv)
        a, b = (G.policy_loss(q, adv, mask, old, ref, ratio=r, beta=0.05) for r in ("sequence", "sequence_token"))
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("ratio,token_adv", [("sequence", False), ("sequence_token", False), ("sequence_token", True)])
def test_autograd(ratio, token_adv):
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(5, 400, token_adv=token_adv)
    leaf = torch.where(mask, q, torch.zeros_like(q)).requires_grad_(True)
    loss, _ = G.clipped_policy_loss(leaf, adv, mask, old, ref, beta=0.05, ratio=ratio)
    loss.backward()
    want = G.policy_loss(q, adv, mask, old, ref, beta=0.05, ratio=ratio)
    assert torch.equal(loss.detach(), want[0][0]) and torch.equal(leaf.grad, want[1])


def test_autograd_asks_for_the_name_of_a_surrogate():
    """A gradient that is not that of the number returned is not handed to autograd
    under the name of one that is."""
    import grpo_loss_gb300 as G
    q = torch.zeros(3, 8, requires_grad=True)
    mask = torch.ones(3, 8, dtype=torch.bool)
    with pytest.raises(ValueError, match="sequence_token"):
        G.clipped_policy_loss(q, torch.ones(3, 8), mask, torch.zeros(3, 8), ratio="sequence")
    for adv in (torch.ones(3, 8), torch.ones(3)):   # (refused for where it lies)
        with pytest.raises(ValueError, match="CUDA"):
            G.clipped_policy_loss(q, adv, mask, torch.zeros(3, 8), ratio="sequence_token")
    with pytest.raises(ValueError, match="CUDA"):
        G.clipped_policy_loss(q, torch.ones(3), mask, torch.zeros(3, 8), ratio="sequence")
