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


def _stand_in(monkeypatch):
    """residual_norm's forward by its formula on the host, without the norms."""
    import grpo_loss_gb300 as G

    def fwd(x, r, w, b, pw, pb, gate, scale, eps, rms):
        g = 1.0 if gate is None else gate.repeat_interleave(len(x) // len(gate), 0)
        return r + scale * g * x, r * w, None, None, None, None
    monkeypatch.setattr(G, "residual_norm_fwd", fwd)
    return G.residual_norm


@pytest.mark.parametrize("lead,gate", [
    ((2, 6), ()), ((2, 6), (2,)), ((2, 6), (2, 1)), ((2, 6), (1, 1)), ((2, 6), (1,)), ((2, 6), (2, 6)), ((2, 6), (12,)),
    ((4, 3, 5), (4, 3)), ((4, 3, 5), (4,)), ((4, 3, 5), (4, 3, 1)), ((4, 3, 5), (4, 1, 1)), ((4, 3, 5), (4, 3, 5)), ((4, 3, 5), (60,)),
    ((12,), (4,)), ((12,), (12,)), ((12,), (1,)), ((12,), (4, 3)), ((12,), (4, 1)), ((), ()), ((), (1,)), ((1, 6), (1, 6)),
    ((1, 6), (6,)), ((3, 3), (3,))])
def test_gates_that_have_leading_dimensions(monkeypatch, lead, gate):
    """A gate's dimensions are x's leading ones, and count for all that follow; x that is
    flat takes gates whose rows divide its own."""
    f = _stand_in(monkeypatch)
    g = torch.Generator().manual_seed(1)
    x, r, s = (torch.randn(*v, 8, generator=g, dtype=torch.float64) for v in (lead, lead, gate))
    w = torch.ones(8, dtype=torch.float64)
    rows, n = math.prod(lead), math.prod(gate)
    each = s.reshape(n, 1, 8).expand(n, rows // n, 8).reshape(x.shape)
    h, _ = f(x, r, w, gate=s, scale=0.5)
    assert h.shape == x.shape and torch.equal(h, r + 0.5 * each * x)


@pytest.mark.parametrize("lead,gate", [
    ((2, 6), (6,)), ((2, 6), (1, 6)), ((2, 6), (3,)), ((2, 6), (4,)), ((2, 6), (6, 1)), ((2, 6), (6, 2)), ((2, 6), (2, 3)),
    ((4, 3, 5), (3,)), ((4, 3, 5), (12,)), ((4, 3, 5), (1, 3)), ((4, 3, 5), (1, 3, 5)), ((4, 3, 5), (4, 1, 5)), ((4, 3, 5), (3, 4)),
    ((4, 3, 5), (5,)), ((12,), (5,)), ((12,), (24,)), ((12,), (0,))])
def test_gates_that_lie_otherwise_are_refused(monkeypatch, lead, gate):
    """A gate for each position of x [sequences, positions, d], above all: its rows divide
    x's, but are not shared by runs of them."""
    f = _stand_in(monkeypatch)
    with pytest.raises(ValueError, match="gate"):
        f(torch.zeros(*lead, 8), torch.zeros(*lead, 8), torch.ones(8), gate=torch.ones(*gate, 8))


def test_a_residual_of_another_shape_is_refused(monkeypatch):
    f = _stand_in(monkeypatch)
    x = torch.zeros(2, 6, 8)
    for shape in ((6, 2, 8), (12, 8), (1, 12, 8), (2, 6, 4), (2, 3, 8)):
        with pytest.raises(ValueError, match="residual"):
            f(x, torch.zeros(shape), torch.ones(8))
    with pytest.raises(ValueError, match="gate"):
        f(x, x, torch.ones(8), gate=torch.ones(2, 6, 4))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [100, 300000, 3000000])
def test_a_nan_reaches_the_factor_of_an_infinite_bound(n):
    """In one launch, and in several."""
    import grpo_loss_gb300 as G
    for dtype in (F32, BF16):
        for norm_type in (2.0, math.inf):
            for at in (None, 0, 37, n - 1):
                g = torch.ones(n, device="cuda", dtype=dtype)
                if at is not None:
                    g[at] = math.nan
                grads, some = [g[:n // 2], g[n // 2:]], at is not None
                norm, factor = G.grad_norm(grads, norm_type, max_norm=math.inf)
                assert math.isnan(norm.item()) == math.isnan(factor.item()) == some and (some or factor.item() == 1)
                out, f = [torch.zeros_like(t) for t in grads], torch.zeros(1, device="cuda")
                norm = G.clip_grad_norm(grads, math.inf, norm_type, out=out, factor=f)
                assert math.isnan(norm.item()) == math.isnan(f.item()) == some
                assert all(torch.isnan(t).all() if some else torch.equal(t, u) for t, u in zip(out, grads))
                g[0] = math.inf                      # (an infinite norm under an infinite bound: not clipped)
                _, factor = G.grad_norm(grads, norm_type, max_norm=math.inf)
                assert math.isnan(factor.item()) if some and at != 0 else factor.item() == 1


def test_lists_of_nothing_are_looked_at(monkeypatch):
    """Outputs beside no gradients, and results that are not on a GPU."""
    import grpo_loss_gb300 as G
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="expected 0 tensors in out, got 1"):
        G.clip_grad_norm([], 1.0, out=[torch.zeros(3)])
    for kw in (dict(norm=torch.zeros(1)), dict(factor=torch.zeros(1)), dict(norm=torch.zeros(1), workspace=torch.zeros(1 << 20))):
        with pytest.raises(ValueError, match="CUDA"):
            G.clip_grad_norm([], 1.0, **kw)
        with pytest.raises(ValueError, match="CUDA"):
            G.grad_norm([], max_norm=1.0, **kw)
