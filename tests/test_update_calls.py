"""Calls of the operators of a rollout's further updates that their documentation allows, at
the edges of what it allows, and calls that it does not."""
import math

import pytest
import torch

from grpo_loss_gb300 import _lib as L

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_rows_leave_no_gradient_of_a_gate_on_the_host(monkeypatch, dtype):
    """(The library's call, which has nothing to do, is left out.)"""
    import grpo_loss_gb300 as G
    monkeypatch.setattr(L, "_device_of", lambda t, name: t.device)
    monkeypatch.setattr(L, "_call", lambda *a: None)
    x, w = torch.zeros(0, 8), torch.ones(8)
    for n in (1, 3):
        buf = torch.full((n, 8), math.nan)
        dg = G.residual_norm_bwd(x, x, x, w, torch.zeros(0), torch.zeros(0), x=x, gate=torch.ones(n, 8, dtype=dtype), dgate=buf,
                                 need_params=False)[6]
        assert dg is buf and not buf.any()


@pytest.mark.gpu
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_rows_leave_no_gradient_of_a_gate(dtype, post):
    import grpo_loss_gb300 as G
    d = 64
    x, w, none = torch.zeros(0, d, device="cuda", dtype=dtype), torch.ones(d, device="cuda"), torch.zeros(0, device="cuda")
    kw = dict(post_weight=w, post_mean=none, post_rstd=none) if post else {}
    for n in (1, 5):
        gate, side = torch.ones(n, d, device="cuda", dtype=dtype), torch.cuda.Stream()
        for stream in (None, side):
            buf = torch.full((n, d), math.nan, device="cuda")
            torch.cuda.synchronize()
            given = G.residual_norm_bwd(x, x, x, w, none, none, x=x, gate=gate, dgate=buf, stream=stream, **kw)
            junk = torch.full((n, d), math.nan, device="cuda")      # what an allocation may find
            del junk
            made = G.residual_norm_bwd(x, x, x, w, none, none, x=x, gate=gate, stream=stream, **kw)
            torch.cuda.synchronize()
            assert given[6] is buf and not buf.any() and made[6].shape == (n, d) and not made[6].any()
            assert not any(t.any() for t in made[2:6] if t is not None)
    # a learned gate keeps the gradient that it has
    leaf = torch.ones(d, device="cuda", dtype=dtype, requires_grad=True)
    leaf.grad = torch.full_like(leaf, 2.0)
    xs = torch.zeros(0, 4, d, device="cuda", dtype=dtype, requires_grad=True)
    h, y = G.residual_norm(xs, xs.detach(), w, post_weight=w if post else None, gate=leaf)
    (h.float().sum() + y.float().sum()).backward()
    assert (leaf.grad == 2).all() and xs.grad.shape == xs.shape
