"""Layer norm and RMS norm against float64, forward and backward, within bounds
on float32 evaluation in any order plus the rounding of the outputs' type."""
import ctypes

import numpy as np
import pytest
import torch

from grpo_loss_gb300 import _lib as L
from tests.operator_reference import U, f64, norm_bwd, norm_fwd

F32, BF16 = torch.float32, torch.bfloat16


def inputs(rows, d, dtype, pdtype, bias=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + rows * 31 + d)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (n(rows, d) * (1 + n(d).abs()) + 0.5 * n(d)).to(dtype)
    w, b = (1 + 0.2 * n(d)).to(pdtype), (0.3 * n(d)).to(pdtype) if bias else None
    return x, w, b, (n(rows, d) * 0.01).to(dtype)


def near(got, want, bound, dtype=F32):
    got = f64(got)
    tol = bound + U[dtype] * (np.abs(want) + bound)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / np.maximum(tol, 1e-300))


def check(x, w, b, dy, rms=False, eps=1e-5, **out):
    import grpo_loss_gb300 as G
    fwd = {k: v for k, v in out.items() if k in ("y",)}
    y, mean, rstd = G.layernorm_fwd(x, w, b, eps=eps, rms=rms, **fwd)
    torch.cuda.synchronize()
    x64, w64 = f64(x), f64(w)
    want = norm_fwd(x64, w64, None if b is None else f64(b), eps, rms)
    near(y, want[0], want[3], x.dtype)
    near(rstd, want[2], want[5])
    if rms:
        assert mean is None
    else:
        near(mean, want[1], want[4])
    dx, dw, db = G.layernorm_bwd(x, w, dy, mean, rstd, rms=rms, bias=b is not None)
    torch.cuda.synchronize()
    ref = norm_bwd(x64, w64, f64(dy), None if rms else f64(mean), f64(rstd), rms)
    near(dx, ref[0], ref[3], x.dtype)
    near(dw, ref[1], ref[4])
    if b is None:
        assert db is None
    else:
        near(db, ref[2], ref[5])
    return y, mean, rstd, dx, dw, db


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 4096), (3, 2), (5, 33), (64, 257), (7, 1536), (130, 2880), (2, 65536),
                                    (1001, 64), (19, 4100), (700, 520), (3, 16387), (33, 8192), (305, 1000)])
def test_sizes_and_types(rows, d, rms):
    for dtype, pdtype in ((F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)):
        x, w, b, dy = inputs(rows, d, dtype, pdtype, bias=not rms)
        check(x, w, b, dy, rms)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 303, 304, 305, 609, 2500])
def test_column_sums_over_row_counts(rows):
    x, w, b, dy = inputs(rows, 192, BF16, BF16)
    check(x, w, b, dy)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_large_mean_and_constant_rows(dtype):
    """The variance is taken about the mean: no cancellation of large squares."""
    x, w, b, dy = inputs(9, 1000, F32, F32)
    x = (x * 0.01 + 100).to(dtype)
    x[3] = 2.5                                     # variance 0: rstd = 1 / sqrt(eps)
    x[4] = 0.0
    check(x, w, b, dy.to(dtype))


@pytest.mark.gpu
def test_rows_with_no_gradient_and_frozen_parameters():
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(40, 768, BF16, F32)
    dy[::2] = 0
    y, mean, rstd, dx, dw, db = check(x, w, b, dy)
    assert not dx[::2].any()
    only, none, none2 = G.layernorm_bwd(x, w, dy, mean, rstd, bias=False, need_dweight=False)
    assert none is None and none2 is None and torch.equal(only, dx)
    a, dw1, none = G.layernorm_bwd(x, w, dy, mean, rstd, bias=False)
    c, none2, db1 = G.layernorm_bwd(x, w, dy, mean, rstd, need_dweight=False)
    assert torch.equal(a, dx) and torch.equal(c, dx) and torch.equal(dw1, dw) and torch.equal(db1, db)
    assert none is None and none2 is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,d", [(0, 512), (1, 512), (3, 509), (8, 1000)])
def test_strided_and_unaligned_rows(dtype, offset, d):
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(21, 1100, dtype, dtype)
    cut = lambda t: t[:, offset:offset + d]  # noqa: E731
    yb = torch.zeros_like(x)
    args = cut(x), w[offset:offset + d], b[offset:offset + d], cut(dy)
    y, mean, rstd, dx, dw, db = check(*args, y=cut(yb))
    assert not yb[:, :offset].any() and not yb[:, offset + d:].any()      # nothing beside the rows
    whole = [t.contiguous() for t in args]
    again = check(*whole)
    for s, t in zip((y, mean, rstd, dx, dw, db), again):
        assert torch.allclose(s.float(), t.float(), rtol=1e-2 if dtype == BF16 else 1e-4, atol=1e-6)
    buf = torch.zeros_like(dy)
    got = G.layernorm_bwd(args[0], args[1], args[3], mean, rstd, dx=cut(buf))[0]
    assert torch.equal(got, dx) and not buf[:, :offset].any() and not buf[:, offset + d:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(4000, 3), (5000, 67), (3000, 129), (2000, 513), (1700, 1001), (1300, 2881), (700, 5003),
                                    (400, 9999), (330, 16383), (90, 1001), (77, 67)])
def test_odd_widths_over_many_rows(rows, d):
    """Rows that begin anywhere in a 16-byte granule, several of them a CTA."""
    for dtype, pdtype, rms in ((BF16, BF16, False), (F32, F32, False), (BF16, F32, True)):
        x, w, b, dy = inputs(rows, d, dtype, pdtype, bias=not rms)
        x[0] *= 3.0
        check(x, w, b, dy, rms)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_and_operands_that_lie_differently(dtype):
    """Bases off a 16-byte boundary, odd strides, operands that differ in both;
    NaN beside the rows stays out of them."""
    import grpo_loss_gb300 as G
    rows, d = 900, 257
    x, w, b, dy = inputs(rows, d, dtype, dtype)

    def laid(t, base, ld):
        flat = torch.full((base + rows * ld,), float("nan"), dtype=dtype, device="cuda")
        view = flat[base:].view(rows, ld)[:, :d]
        view.copy_(t)
        return view

    for bases, lds in (((1, 1), (261, 261)), ((5, 5), (257, 257)), ((0, 3), (264, 264)), ((2, 2), (259, 275)), ((8, 0), (264, 257))):
        xs, gs = laid(x, bases[0], lds[0]), laid(dy, bases[1], lds[1])
        y, mean, rstd, dx, dw, db = check(xs, w, b, gs)
        out = laid(torch.zeros_like(x), bases[0], lds[0])
        assert torch.equal(G.layernorm_bwd(xs, w, gs, mean, rstd, dx=out)[0], dx)
        assert torch.equal(G.layernorm_fwd(xs, w, b, y=out)[0], y)


@pytest.mark.gpu
def test_another_stream_owns_what_it_makes():
    """A workspace made by a call on a side stream is not handed to the current
    stream's next tensors while the call runs."""
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(20000, 1024, BF16, BF16)
    y, mean, rstd = G.layernorm_fwd(x, w, b)
    want = G.layernorm_bwd(x, w, dy, mean, rstd)
    size = G._lib.layernorm_workspace_size(G._lib.LayernormProblem(20000, 1024, 1024, 0, 1024, 1024, 0.0, 0, 1, 1))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        ys, ms, rs = G.layernorm_fwd(x, w, b, stream=side)
        got = G.layernorm_bwd(x, w, dy, ms, rs, stream=side)
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(ys, y) and all(torch.equal(s, t) for s, t in zip(got, want))
        del junk


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 512, 1000, 4096, 8192])
def test_outputs_off_a_boundary_have_the_same_bits(d, dtype):
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(400, d, dtype, dtype)
    y, mean, rstd, dx, dw, db = check(x, w, b, dy)
    off = lambda: torch.empty(400 * d + 1, dtype=dtype, device="cuda")[1:].view(400, d)  # noqa: E731
    other = G.layernorm_fwd(x, w, b, y=off())
    assert all(torch.equal(s, t) for s, t in zip(other, (y, mean, rstd)))
    dx2, dw2, db2 = G.layernorm_bwd(x, w, dy, mean, rstd, dx=off())
    assert torch.equal(dx2, dx)
    ref = norm_bwd(f64(x), f64(w), f64(dy), f64(mean), f64(rstd), False)
    near(dw2, ref[1], ref[4])                      # (other rows share a group's partial sums)
    near(db2, ref[2], ref[5])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(50, 1024), (50, 1021), (3, 65536)])
def test_in_place(rows, d):
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(rows, d, BF16, BF16)
    y, mean, rstd, dx, dw, db = check(x, w, b, dy)
    x2, g1, x3 = x.clone(), dy.clone(), x.clone()
    assert torch.equal(G.layernorm_fwd(x2, w, b, y=x2)[0], y)
    for r in (G.layernorm_bwd(x, w, g1, mean, rstd, dx=g1), G.layernorm_bwd(x3, w, dy, mean, rstd, dx=x3)):
        assert torch.equal(r[0], dx) and torch.equal(r[1], dw) and torch.equal(r[2], db)


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of sum(dy * y) in float64 along random directions."""
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(6, 96, F32, F32)
    for rms in (False, True):
        bb = None if rms else b
        _, mean, rstd = G.layernorm_fwd(x, w, bb, rms=rms)
        dx, dw, db = G.layernorm_bwd(x, w, dy, mean, rstd, rms=rms, bias=not rms)
        x64, w64, dy64 = f64(x), f64(w), f64(dy)
        f = lambda a, c: float((norm_fwd(a, c, None, 1e-5, rms)[0] * dy64).sum())  # noqa: E731
        rng = np.random.default_rng(1)
        for _ in range(4):
            v, h = rng.standard_normal(x64.shape), 1e-5
            num = (f(x64 + h * v, w64) - f(x64 - h * v, w64)) / (2 * h)
            # float32 evaluation: some units in the last place of the terms' magnitudes
            assert abs(num - (f64(dx) * v).sum()) <= 1e-5 * np.abs(f64(dx) * v).sum()
            v = rng.standard_normal(w64.shape)
            num = (f(x64, w64 + h * v) - f(x64, w64 - h * v)) / (2 * h)
            assert abs(num - (f64(dw) * v).sum()) <= 1e-5 * np.abs(f64(dw) * v).sum()


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_autograd(rms):
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(24, 320, F32, F32)
    b = None if rms else b
    leaves = [t.clone().requires_grad_(True) for t in (x, w) + (() if rms else (b,))]
    y = G.layer_norm(leaves[0].view(4, 6, 320), leaves[1], None if rms else leaves[2], rms=rms)
    assert y.shape == (4, 6, 320)
    (y * dy.view(4, 6, 320)).sum().backward()
    _, mean, rstd = G.layernorm_fwd(x, w, b, rms=rms)
    want = G.layernorm_bwd(x, w, dy, mean, rstd, rms=rms, bias=not rms)
    for leaf, t in zip(leaves, want):
        assert torch.equal(leaf.grad, t)
    z = x.clone().requires_grad_(True)             # a broadcast gradient; frozen parameters
    G.layer_norm(z, w, b, rms=rms).sum().backward()
    ones = G.layernorm_bwd(x, w, torch.ones_like(x), mean, rstd, rms=rms, bias=False, need_dweight=False)
    assert torch.equal(z.grad, ones[0])


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_second_derivatives_are_refused(monkeypatch, rms):
    """Gradients that come from kernels have no graph of their own: a penalty on them
    would silently add nothing. (The kernels are stood in for by their formulas.)"""
    import grpo_loss_gb300 as G

    def fwd(x, w, b, eps=1e-5, rms=False):
        mean = None if rms else x.mean(1)
        c = x if rms else x - mean[:, None]
        rstd = ((c * c).mean(1) + eps).rsqrt()
        return c * rstd[:, None] * w, mean, rstd

    def bwd(x, w, dy, mean, rstd, rms=False, bias=True, need_dweight=True):
        h = (x if rms else x - mean[:, None]) * rstd[:, None]
        g = dy * w
        dx = rstd[:, None] * (g - (0 if rms else g.mean(1, keepdim=True)) - h * (g * h).mean(1, keepdim=True))
        return dx, (dy * h).sum(0), None
    monkeypatch.setattr(G, "layernorm_fwd", fwd)
    monkeypatch.setattr(G, "layernorm_bwd", bwd)
    x = torch.randn(4, 8, dtype=torch.float64, requires_grad=True)
    w = torch.ones(8, dtype=torch.float64, requires_grad=True)
    (want,) = torch.autograd.grad(torch.nn.functional.rms_norm(x, (8,), w, 1e-5).pow(2).sum() if rms else
                                  torch.nn.functional.layer_norm(x, (8,), w, None).pow(2).sum(), x)
    (got,) = torch.autograd.grad(G.layer_norm(x, w, rms=rms).pow(2).sum(), x)
    assert torch.allclose(got, want)
    for loss in (lambda y: y.pow(2).sum(), lambda y: y.sum()):      # dy with a graph, and without
        gx, gw = torch.autograd.grad(loss(G.layer_norm(x, w, rms=rms)), (x, w), create_graph=True)
        for g in (gx, gw):
            with pytest.raises(RuntimeError, match="once differentiable"):
                torch.autograd.grad(g.pow(2).sum() + x.pow(2).sum(), x, retain_graph=True)


@pytest.mark.gpu
def test_no_rows():
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(1, 64, F32, F32)
    y, mean, rstd = G.layernorm_fwd(x[:0], w, b)
    assert y.shape == (0, 64) and mean.numel() == rstd.numel() == 0
    dx, dw, db = G.layernorm_bwd(x[:0], w, dy[:0], mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.gpu
def test_rows_past_two_to_the_31_elements():
    import grpo_loss_gb300 as G
    d, rows = 4096, 524289 + 1024                  # 2.15e9 elements
    x = torch.zeros(rows, d, device="cuda", dtype=BF16)
    tail, w, b, dy = inputs(64, d, BF16, BF16)
    x[-64:] = tail
    y, mean, rstd = G.layernorm_fwd(x, w, b)
    alone = G.layernorm_fwd(tail, w, b)
    for s, t in zip((y, mean, rstd), alone):
        assert torch.equal(s[-64:], t)
    g = torch.zeros_like(x)
    g[-64:] = dy
    dx, dw, db = G.layernorm_bwd(x, w, g, mean, rstd)
    want = G.layernorm_bwd(tail, w, dy, alone[1], alone[2])
    assert torch.equal(dx[-64:], want[0]) and not dx[:-64].any()
    bound = 80 * 2.0 ** -24
    assert (dw - want[1]).abs().max() <= bound * f64(dy.abs()).sum(0).max() * 10
    assert (db - want[2]).abs().max() <= bound * f64(dy.abs()).sum(0).max()


@pytest.mark.gpu
def test_repeats_streams_and_graphs():
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(900, 1536, BF16, BF16)
    y, mean, rstd = G.layernorm_fwd(x, w, b)
    want = (y, mean, rstd) + G.layernorm_bwd(x, w, dy, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = G.layernorm_fwd(x, w, b)
        a = a + G.layernorm_bwd(x, w, dy, a[1], a[2])
    side.synchronize()
    outs = [torch.empty_like(t) for t in want]
    pr = L.LayernormProblem(900, 1536, 0, 0, 0, 0, 1e-5, 0, L.GRPO_BF16, L.GRPO_BF16)
    ws = torch.empty(L.layernorm_workspace_size(pr), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.layernorm_fwd(x, w, b, y=outs[0], mean=outs[1], rstd=outs[2])
        G.layernorm_bwd(x, w, dy, outs[1], outs[2], dx=outs[3], dweight=outs[4], dbias=outs[5], workspace=ws)
    for t in outs:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for s, t, o in zip(want, a, outs):
        assert torch.equal(s, t) and torch.equal(s, o)


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (python -m grpo_loss_gb300.build)")
    return L.lib()


@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, 1), ("d", 0, 1), ("ld_x", 99, 1), ("ld_y", 1, 1), ("ld_dy", -5, 1), ("ld_dx", 99, 1),
    ("eps", -1.0, 1), ("eps", float("nan"), 1), ("rms", 2, 1), ("dtype", 2, 1), ("param_dtype", 7, 1),
    ("d", 65537, 2), ("rows", 1 << 31, 2)])
def test_refuses_bad_problems_on_the_host(lib, field, value, status):
    pr = L.LayernormProblem(4, 100, 0, 0, 0, 0, 1e-5, 0, L.GRPO_F32, L.GRPO_F32)
    setattr(pr, field, value)
    at, size = ctypes.c_void_p(256), ctypes.c_size_t(0)
    r = ctypes.byref(pr)
    assert lib.grpo_layernorm_workspace_size(r, ctypes.byref(size)) == status
    assert lib.grpo_layernorm_fwd(r, at, at, at, at, at, at, None) == status
    assert lib.grpo_layernorm_bwd(r, at, at, at, at, at, at, at, at, at, 1 << 40, None) == status


def test_refuses_bad_pointers_on_the_host(lib):
    pr = L.LayernormProblem(4, 100, 0, 0, 0, 0, 1e-5, 0, L.GRPO_F32, L.GRPO_BF16)
    r, at, odd = ctypes.byref(pr), ctypes.c_void_p(256), ctypes.c_void_p(257)
    put = lambda n, i, v: [v if j == i else at for j in range(n)]  # noqa: E731
    assert lib.grpo_layernorm_fwd(None, *[at] * 6, None) == 1
    for i in (0, 1, 3):
        assert lib.grpo_layernorm_fwd(r, *put(6, i, None), None) == 1
    for i in range(6):
        assert lib.grpo_layernorm_fwd(r, *put(6, i, odd), None) == 2
    for i in (0, 1, 2, 3, 4, 5):
        assert lib.grpo_layernorm_bwd(r, *put(8, i, None), at, 1 << 40, None) == 1
    for i in range(8):
        assert lib.grpo_layernorm_bwd(r, *put(8, i, odd), at, 1 << 40, None) == 2
    pr.rms = 1                                     # an RMS norm has no bias
    assert lib.grpo_layernorm_fwd(r, *[at] * 6, None) == 1
    assert lib.grpo_layernorm_bwd(r, *[at] * 8, at, 1 << 40, None) == 1


@pytest.mark.gpu
def test_refuses_a_short_workspace_and_wrong_tensors():
    import grpo_loss_gb300 as G
    x, w, b, dy = inputs(10, 64, F32, F32)
    y, mean, rstd = G.layernorm_fwd(x, w, b)
    with pytest.raises(L.GrpoError) as e:
        G.layernorm_bwd(x, w, dy, mean, rstd, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    for bad, word in ((dict(weight=w[:5]), "elements"), (dict(bias=b.bfloat16()), "float32"), (dict(x=x.half()), "float32 or"),
                      (dict(x=x.t()), "contiguous"), (dict(y=x[:5]), "shape"), (dict(weight=w.cpu()), "on cuda"),
                      (dict(y=torch.empty(1, 64, device="cuda").expand(10, 64)), "row stride")):
        with pytest.raises(ValueError, match=word):
            G.layernorm_fwd(**{"x": x, "weight": w, "bias": b, **bad})
    with pytest.raises(ValueError, match="mean"):
        G.layernorm_bwd(x, w, dy, None, rstd)
    with pytest.raises(ValueError, match="must be"):
        G.layernorm_bwd(x, w, dy.bfloat16(), mean, rstd)
