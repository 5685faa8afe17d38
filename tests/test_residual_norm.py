"""The norms behind and before a block with its gate and residual scale against float64,
forward and backward, within bounds on float32 evaluation in any order plus the
rounding of the outputs' type."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from grpo_loss_gb300 import _lib as L
from tests.operator_reference import U, f64
from tests.update_reference import residual_norm_bwd, residual_norm_fwd

F32, BF16 = torch.float32, torch.bfloat16
FWD = ("h", "y", "mean", "rstd", "post_mean", "post_rstd")
BWD = ("dx", "dresidual", "dweight", "dbias", "dpost_weight", "dpost_bias", "dgate")


def inputs(rows, d, dtype, pdtype=F32, rms=False, bias=True, post=True, gate=None, gdtype=None, seed=0, laid=None):
    """A dict of the forward's tensors and of dy and dh. ``gate``: rows of it, or None.
    ``laid(t)`` places each [rows, d] matrix."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + rows * 31 + d)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    laid = laid or (lambda t: t)
    bias = bias and not rms
    s = dict(x=laid((n(rows, d) * (1 + n(d).abs()) + 0.3 * n(d)).to(dtype)), residual=laid((n(rows, d) * 2 + n(d)).to(dtype)),
             weight=(1 + 0.2 * n(d)).to(pdtype), bias=(0.3 * n(d)).to(pdtype) if bias else None,
             post_weight=(0.5 + 0.2 * n(d)).to(pdtype) if post else None,
             post_bias=(0.2 * n(d)).to(pdtype) if post and bias else None,
             gate=None if gate is None else (0.5 + n(gate, d)).to(gdtype or dtype))
    if gate == rows and rows > 1:
        s["gate"] = laid(s["gate"].to(dtype))
    s["dy"], s["dh"] = laid((n(rows, d) * 0.01).to(dtype)), laid((n(rows, d) * 0.01).to(dtype))
    return s


def near(name, got, want, bound):
    u, got = U[got.dtype], f64(got)
    tol = bound + u * (np.abs(want) + bound) + 1e-38
    assert got.shape == want.shape, name
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol), \
        (name, np.max(np.abs(got - want) / tol), np.unravel_index(np.argmax(np.abs(got - want) / tol), got.shape))


def z(t):
    return None if t is None else f64(t)


def check(s, scale=1.0, rms=False, eps=1e-5, dh=True, fwd=None, bwd=None):
    import grpo_loss_gb300 as G
    args = [s[k] for k in ("x", "residual", "weight", "bias", "post_weight", "post_bias", "gate")]
    got = dict(zip(FWD, G.residual_norm_fwd(*args, scale=scale, eps=eps, rms=rms, **(fwd or {}))))
    torch.cuda.synchronize()
    val, err = residual_norm_fwd(*[z(t) for t in args], scale, eps, rms)
    for k in FWD:
        assert (got[k] is None) == (k not in val or (rms and "mean" in k)), k
        if got[k] is not None:
            near(k, got[k], val[k], err[k])
    back = G.residual_norm_bwd(s["dy"], s["dh"] if dh else None, got["h"], s["weight"], got["mean"], got["rstd"], x=s["x"],
                               post_weight=s["post_weight"], post_bias=s["post_bias"], post_mean=got["post_mean"],
                               post_rstd=got["post_rstd"], gate=s["gate"], scale=scale, rms=rms,
                               bias=s["bias"] is not None, **(bwd or {}))
    torch.cuda.synchronize()
    back = dict(zip(BWD, back))
    val, err = residual_norm_bwd(f64(s["dy"]), z(s["dh"]) if dh else None, f64(got["h"]), f64(s["weight"]), z(got["mean"]),
                                 f64(got["rstd"]), f64(s["x"]), z(s["post_weight"]), z(s["post_bias"]), z(got["post_mean"]),
                                 z(got["post_rstd"]), z(s["gate"]), scale, rms)
    have = {"dx": True, "dresidual": True, "dweight": True, "dbias": s["bias"] is not None,
            "dpost_weight": s["post_weight"] is not None, "dpost_bias": s["post_bias"] is not None,
            "dgate": s["gate"] is not None}
    for k in BWD:
        assert (back[k] is not None) == have[k], k
        if have[k]:
            near(k, back[k], val[k], err[k])
    return got, back


KINDS = [dict(post=False), dict(post=True), dict(post=True, rms=True), dict(post=False, gate=1), dict(post=True, gate=1, rms=True),
         dict(post=False, gate="all"), dict(post=True, gate="all"), dict(post=True, gate="seq"), dict(post=False, gate="seq", rms=True)]
IDS = ["%s-%s-%s" % ("post" if k["post"] else "plain", k.get("gate"), "rms" if k.get("rms") else "layer") for k in KINDS]


def of_kind(kind, rows):
    """The gate's rows: a third of the rows to each where that divides, else the most that do."""
    gate = kind.get("gate")
    if gate == "seq":
        gate = next(n for n in (3, 5, 7, 2, 1) if rows % n == 0)
    return dict(kind, gate=rows if gate == "all" else gate)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 4096), (3, 2), (6, 33), (63, 257), (21, 1536), (135, 2880), (2, 32768),
                                    (1001, 64), (21, 4100), (700, 520), (33, 8192), (305, 1000), (12, 16384), (9, 9999)])
def test_sizes_and_types(rows, d, kind):
    kw = of_kind(kind, rows)
    for dtype, pdtype, gdtype in ((F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, F32)):
        s = inputs(rows, d, dtype, pdtype, gdtype=gdtype, **kw)
        check(s, scale=0.7 if dtype == BF16 else 1.0, rms=kind.get("rms", False))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("dtype,rows,d", [(F32, 480, 4099), (F32, 300, 8200), (BF16, 480, 8195), (BF16, 300, 16392), (BF16, 75, 30001),
                                          (F32, 75, 20004)])
def test_long_rows(dtype, rows, d, kind):
    """Several rows to each of those that work at a time, whole pieces and not."""
    s = inputs(rows, d, dtype, **of_kind(kind, rows))
    _, first = check(s, scale=0.7, rms=kind.get("rms", False))
    _, again = check(s, scale=0.7, rms=kind.get("rms", False))
    assert all(torch.equal(first[k], again[k]) for k in BWD if first[k] is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(50, 512), (33, 257), (9, 5000), (2, 32768)])
def test_a_gate_of_another_type_than_the_rows(rows, d):
    for dtype, gdtype, gate in ((BF16, F32, rows), (F32, BF16, rows), (BF16, F32, 1), (F32, BF16, 1)):
        s = inputs(rows, d, dtype, F32)
        s["gate"] = torch.randn(gate, d, device="cuda", generator=torch.Generator("cuda").manual_seed(d)).to(gdtype)
        _, back = check(s, scale=0.7)
        assert back["dgate"].dtype == (gdtype if gate == rows else F32)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,per", [(2, 1), (303, 101), (304, 2), (608, 76), (609, 3), (2500, 100), (2400, 7 * 0 + 800), (5000, 1250)])
def test_gates_over_row_counts(rows, per):
    """Gates whose rows are shared by a few rows and by many, and end anywhere."""
    for d, dtype in ((192, BF16), (65, F32)):
        check(inputs(rows, d, dtype, gate=rows // per), scale=0.5)
        check(inputs(rows, d, dtype, gate=rows // per, post=False, rms=True), scale=0.5, rms=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_large_mean_and_constant_rows(dtype):
    """Variances are taken about the mean: no cancellation of large squares."""
    s = inputs(9, 1000, F32)
    for k in ("x", "residual"):
        s[k] = s[k] * 0.01 + 100
        s[k][3] = 2.5
        s[k][4] = 0.0
    s = {k: v.to(dtype) if k in ("x", "residual", "dy", "dh") else v for k, v in s.items()}
    s["gate"] = torch.ones(1, 1000, device="cuda")
    check(s)
    s["post_weight"] = s["post_bias"] = None
    check(s)


@pytest.mark.gpu
def test_the_norm_is_of_the_stream_before_its_rounding():
    import grpo_loss_gb300 as G
    s = inputs(64, 512, BF16, BF16, post=False, bias=False)
    h, y, mean, rstd, _, _ = G.residual_norm_fwd(s["x"], s["residual"], s["weight"], eps=0.0)
    exact = s["residual"].double() + s["x"].double()
    assert not torch.equal(h.double(), exact) and torch.equal(h, exact.to(BF16))
    assert (mean.double() - exact.mean(1)).abs().max() <= 1e-5 * exact.abs().mean()
    only, _, _ = G.layernorm_fwd(exact.float(), s["weight"], eps=0.0)
    assert torch.equal(only.to(BF16), y) or (only - y.float()).abs().max() <= 2.0 ** -8 * only.abs().max() * 1.01


@pytest.mark.gpu
def test_what_may_be_left_out():
    import grpo_loss_gb300 as G
    s = inputs(40, 768, BF16, F32, gate=8)
    got, back = check(s, scale=0.3)
    check(s, scale=0.3, dh=False)
    call = lambda **kw: G.residual_norm_bwd(  # noqa: E731
        s["dy"], s["dh"], got["h"], s["weight"], got["mean"], got["rstd"], x=s["x"], post_weight=s["post_weight"],
        post_bias=s["post_bias"], post_mean=got["post_mean"], post_rstd=got["post_rstd"], gate=s["gate"], scale=0.3, **kw)
    r = dict(zip(BWD, call(need_params=False, need_dgate=False)))
    assert [k for k in BWD if r[k] is not None] == ["dx", "dresidual"]
    assert torch.equal(r["dx"], back["dx"]) and torch.equal(r["dresidual"], back["dresidual"])
    r = dict(zip(BWD, call(need_params=False)))
    assert torch.equal(r["dgate"], back["dgate"]) and torch.equal(r["dx"], back["dx"]) and r["dweight"] is None
    r = dict(zip(BWD, call(need_dgate=False, bias=False)))
    assert torch.equal(r["dpost_weight"], back["dpost_weight"]) and r["dbias"] is None and r["dgate"] is None
    p = inputs(40, 768, BF16, F32, post=False)
    got, back = check(p)
    assert back["dx"] is back["dresidual"]          # one gradient for both
    buf = torch.empty_like(p["x"])
    got2, back2 = check(p, bwd=dict(dx=buf))
    assert back2["dx"] is buf and torch.equal(buf, back["dx"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [dict(post=True), dict(post=True, gate="all"), dict(post=False, gate="seq", rms=True)], ids=str)
@pytest.mark.parametrize("offset,d,ld", [(0, 512, 1100), (1, 512, 1100), (3, 509, 1099), (8, 1000, 1100), (4, 258, 264), (2, 257, 261)])
def test_strided_and_unaligned_rows(offset, d, ld, kind, dtype):
    rows = 21

    def laid(t):
        flat = torch.full((rows, ld), float("nan"), dtype=t.dtype, device="cuda")
        flat[:, offset:offset + d] = t
        return flat[:, offset:offset + d]

    kw = of_kind(kind, rows)
    rms = kind.get("rms", False)
    whole = inputs(rows, d, dtype, dtype, **kw)
    cut = inputs(rows, d, dtype, dtype, laid=laid, **kw)
    new = lambda: laid(torch.zeros(rows, d, dtype=dtype, device="cuda"))  # noqa: E731
    outs = dict(h=new(), y=new()), dict(dx=new(), dresidual=new())
    if kind.get("gate") == "all":
        outs[1]["dgate"] = new()
    a, b = check(whole, rms=rms), check(cut, rms=rms, fwd=outs[0], bwd=outs[1])
    for s, t in zip(a, b):
        for k in s:
            assert (s[k] is None) == (t[k] is None)
            if s[k] is not None:
                assert torch.allclose(s[k].float(), t[k].float(), rtol=2e-2 if dtype == BF16 else 1e-4, atol=1e-5)
    for o in (outs[0]["h"], outs[0]["y"], outs[1]["dx"], outs[1]["dresidual"]):
        beside = o.as_strided((rows, ld), (ld, 1), o.storage_offset() - offset).clone()
        beside[:, offset:offset + d] = float("nan")
        assert torch.isnan(beside).all()            # nothing beside the rows


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_operands_that_lie_differently(dtype):
    """Bases and strides of every operand of its own."""
    rows, d, at = 90, 257, [0]

    def laid(t):
        at[0] += 1
        base, ld = at[0] % 5, d + at[0] % 7
        flat = torch.full((base + rows * ld,), float("nan"), dtype=t.dtype, device="cuda")
        view = flat[base:].view(rows, ld)[:, :d]
        view.copy_(t)
        return view

    for kw in (dict(post=True, gate=rows), dict(post=False, gate=1), dict(post=True, gate=9)):
        check(inputs(rows, d, dtype, dtype, laid=laid, **kw))
        check(inputs(rows, d - 1, dtype, dtype, laid=lambda t: laid(torch.nn.functional.pad(t, (0, 1)))[:, :d - 1], **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(4000, 3), (5000, 67), (3000, 129), (2000, 513), (1700, 1001), (1300, 2881), (600, 5003)])
def test_odd_widths_over_many_rows(rows, d):
    for dtype, kw in ((BF16, dict(post=True)), (F32, dict(post=True, rms=True, gate=1)), (BF16, dict(post=False, gate=rows)),
                      (F32, dict(post=False, gate=10)), (BF16, dict(post=False))):
        check(inputs(rows, d, dtype, dtype, **kw), rms=kw.get("rms", False), scale=0.9)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [k for k in KINDS if k.get("gate") != "seq"] + [dict(post=True, gate=1)], ids=str)
@pytest.mark.parametrize("dtype,rows,d,ld", [(BF16, 2051, 1001, 1001), (BF16, 1030, 254, 258), (F32, 1027, 1003, 1003), (F32, 600, 66, 70),
                                             (BF16, 300, 508, 512), (BF16, 2049, 2047, 2049), (BF16, 2050, 8177, 8177), (F32, 1031, 4089, 4091), (F32, 1025, 8150, 8150), (BF16, 2049, 9001, 9001)])
def test_rows_that_are_cut_alike(dtype, rows, d, ld, kind):
    """Rows in granules that hold the end of the row before, or what is beside the rows."""
    def laid(t):
        flat = torch.full((rows, ld), float("nan"), dtype=t.dtype, device="cuda")
        flat[:, :d] = t
        return flat[:, :d]

    s = inputs(rows, d, dtype, BF16, laid=laid, **of_kind(kind, rows))
    kw = dict(scale=0.6, rms=kind.get("rms", False))
    new = lambda: laid(torch.zeros(rows, d, dtype=dtype, device="cuda"))  # noqa: E731
    fwd, bwd = dict(h=new(), y=new()), dict(dx=new(), dresidual=new())
    got, back = check(s, fwd=fwd, bwd=bwd, **kw)
    for o in (fwd["h"], fwd["y"], bwd["dx"], bwd["dresidual"]):
        assert torch.isnan(o.as_strided((rows, ld), (ld, 1))[:, d:]).all()
    # a row that is not finite is its own affair
    bad, at = dict(s), rows // 2
    for k in ("x", "residual", "dy", "dh"):
        bad[k] = laid(s[k])
        bad[k][at] = float("inf")
    import grpo_loss_gb300 as G
    args = [bad[k] for k in ("x", "residual", "weight", "bias", "post_weight", "post_bias", "gate")]
    # (laid out as those it is compared with: sums of rows that are cut otherwise run in another order)
    h, y, mean, rstd, pm, pr = G.residual_norm_fwd(*args, h=new(), y=new(), **kw)
    dx, dr = G.residual_norm_bwd(bad["dy"], bad["dh"], h, s["weight"], mean, rstd, x=bad["x"], post_weight=s["post_weight"],
                                 post_bias=s["post_bias"], post_mean=pm, post_rstd=pr, gate=s["gate"], dx=new(), dresidual=new(), **kw)[:2]
    others = torch.arange(rows, device="cuda") != at
    for t, want in ((h, got["h"]), (y, got["y"]), (dx, back["dx"]), (dr, back["dresidual"])):
        assert torch.equal(t[others], want[others])


@pytest.mark.gpu
def test_in_place_where_rows_share_granules():
    import grpo_loss_gb300 as G
    s = inputs(2500, 1021, BF16, BF16, gate=1)
    got, back = check(s, scale=0.5)
    args = lambda x, r: (x, r, s["weight"], s["bias"], s["post_weight"], s["post_bias"], s["gate"], 0.5)  # noqa: E731
    for _ in range(5):
        x, r = s["x"].clone(), s["residual"].clone()
        h, y = G.residual_norm_fwd(*args(x, r), h=r, y=x)[:2]
        assert torch.equal(h, got["h"]) and torch.equal(y, got["y"])
        dy, dh = s["dy"].clone(), s["dh"].clone()
        dx, dr = G.residual_norm_bwd(dy, dh, h, s["weight"], got["mean"], got["rstd"], x=s["x"], post_weight=s["post_weight"],
                                     post_bias=s["post_bias"], post_mean=got["post_mean"], post_rstd=got["post_rstd"],
                                     gate=s["gate"], scale=0.5, dx=dy, dresidual=dh)[:2]
        assert torch.equal(dx, back["dx"]) and torch.equal(dr, back["dresidual"])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(50, 1024), (50, 1021), (3, 32768)])
def test_in_place(rows, d):
    import grpo_loss_gb300 as G
    s = inputs(rows, d, BF16, BF16, gate=1)
    got, back = check(s, scale=0.5)
    args = lambda x, r: (x, r, s["weight"], s["bias"], s["post_weight"], s["post_bias"], s["gate"], 0.5)  # noqa: E731
    for h_is, y_is in (("residual", None), ("x", None), ("residual", "x"), ("x", "residual"), (None, "x"), (None, "residual")):
        x, r = s["x"].clone(), s["residual"].clone()
        own = {"x": x, "residual": r, None: None}
        h, y = G.residual_norm_fwd(*args(x, r), h=own[h_is], y=own[y_is])[:2]
        assert torch.equal(h, got["h"]) and torch.equal(y, got["y"])
    for dx_is in ("dy", "dh", "h", "x", None):
        for dr_is in ("dy", "dh", "h", None):
            if dx_is == dr_is:
                continue
            own = {k: t.clone() for k, t in (("dy", s["dy"]), ("dh", s["dh"]), ("h", got["h"]), ("x", s["x"]))}
            own[None] = None
            r = G.residual_norm_bwd(own["dy"], own["dh"], own["h"], s["weight"], got["mean"], got["rstd"], x=own["x"],
                                    post_weight=s["post_weight"], post_bias=s["post_bias"], post_mean=got["post_mean"],
                                    post_rstd=got["post_rstd"], gate=s["gate"], scale=0.5, dx=own[dx_is],
                                    dresidual=own[dr_is])
            for k, t in zip(BWD, r):
                assert torch.equal(t, back[k]), (k, dx_is, dr_is)


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of sum(dy y) + sum(dh h) in float64 along random directions."""
    import grpo_loss_gb300 as G
    rng = np.random.default_rng(1)
    for rms, post, gate in ((False, True, 3), (True, True, None), (False, False, 6), (True, False, 1)):
        s = inputs(6, 96, F32, rms=rms, post=post, gate=gate)
        args = [s[k] for k in ("x", "residual", "weight", "bias", "post_weight", "post_bias", "gate")]
        h, y, mean, rstd, pm, pr = G.residual_norm_fwd(*args, scale=0.6, rms=rms)
        r = G.residual_norm_bwd(s["dy"], s["dh"], h, s["weight"], mean, rstd, x=s["x"], post_weight=s["post_weight"],
                                post_bias=s["post_bias"], post_mean=pm, post_rstd=pr, gate=s["gate"], scale=0.6, rms=rms,
                                bias=s["bias"] is not None)
        a64 = [z(t) for t in args]
        dy, dh = f64(s["dy"]), f64(s["dh"])

        def f(a):
            v, _ = residual_norm_fwd(*a, 0.6, 1e-5, rms)
            return float((v["y"] * dy).sum() + (v["h"] * dh).sum())
        for i, g in zip(range(7), r):
            if a64[i] is None:
                continue
            g = f64(g)
            for _ in range(3):
                v, step = rng.standard_normal(a64[i].shape), 1e-5
                plus = [t if j != i else t + step * v for j, t in enumerate(a64)]
                minus = [t if j != i else t - step * v for j, t in enumerate(a64)]
                num = (f(plus) - f(minus)) / (2 * step)
                assert abs(num - (g * v).sum()) <= 2e-5 * np.abs(g * v).sum() + 1e-8, (i, rms, post, gate)


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_autograd(rms):
    import grpo_loss_gb300 as G
    s = inputs(24, 320, F32, rms=rms, gate=4)
    names = [k for k in ("x", "residual", "weight", "bias", "post_weight", "post_bias", "gate") if s[k] is not None]
    leaf = {k: s[k].clone().requires_grad_(True) for k in names}
    kw = {k: leaf[k] for k in names if k not in ("x", "residual", "weight", "gate")}
    h, y = G.residual_norm(leaf["x"].view(4, 6, 320), leaf["residual"].view(4, 6, 320), leaf["weight"], **kw,
                           gate=leaf["gate"], scale=0.4, rms=rms)
    assert h.shape == y.shape == (4, 6, 320)
    ((y * s["dy"].view(4, 6, 320)).sum() + (h * s["dh"].view(4, 6, 320)).sum()).backward()
    _, back = check(s, scale=0.4, rms=rms)
    order = dict(zip(("x", "residual", "weight", "bias", "post_weight", "post_bias", "gate"), BWD))
    for k in names:
        assert torch.equal(leaf[k].grad, back[order[k]]), k
    # one output alone, broadcast gradients, frozen parameters, a gate for each channel
    for which in (0, 1):
        x, r = s["x"].clone().requires_grad_(True), s["residual"].clone().requires_grad_(True)
        G.residual_norm(x, r, s["weight"], gate=s["gate"][0], rms=rms)[which].sum().backward()
        one = torch.ones_like(s["x"])
        h, _, m, rs, _, _ = G.residual_norm_fwd(s["x"], s["residual"], s["weight"], gate=s["gate"][:1], rms=rms)
        want = G.residual_norm_bwd(one * which, one * (1 - which), h, s["weight"], m, rs, x=s["x"], gate=s["gate"][:1], rms=rms)
        assert torch.allclose(x.grad, want[0], rtol=1e-5, atol=1e-7) and torch.allclose(r.grad, want[1], rtol=1e-5, atol=1e-7)


def test_second_derivatives_are_refused(monkeypatch):
    """(The kernels are stood in for by the formulas of a plain sum.)"""
    import grpo_loss_gb300 as G
    monkeypatch.setattr(G, "residual_norm_fwd", lambda x, r, w, *a: (r + x, (r + x) * w, None, None, None, None))
    monkeypatch.setattr(G, "residual_norm_bwd", lambda dy, dh, h, w, *a, **k: (
        (g := dy * w + (0 if dh is None else dh)), g, (dy * h).sum(0), None, None, None, None))
    x = torch.randn(4, 8, dtype=torch.float64, requires_grad=True)
    r = torch.randn(4, 8, dtype=torch.float64)
    w = torch.full((8,), 2.0, dtype=torch.float64, requires_grad=True)
    for f in (lambda h, y: y.sum(), lambda h, y: h.pow(2).sum(), lambda h, y: (h * y).sum()):
        gx, gw = torch.autograd.grad(f(*G.residual_norm(x, r, w)), (x, w), create_graph=True, allow_unused=True)
        for g in (gx, gw):
            with pytest.raises(RuntimeError, match="once differentiable"):
                torch.autograd.grad(g.pow(2).sum() + x.pow(2).sum(), x, retain_graph=True)


@pytest.mark.gpu
def test_no_rows():
    import grpo_loss_gb300 as G
    s = inputs(3, 64, F32, gate=3)
    none = {k: v[:0] if k in ("x", "residual", "dy", "dh", "gate") else v for k, v in s.items()}
    h, y, m, r, pm, pr = G.residual_norm_fwd(none["x"], none["residual"], s["weight"], s["bias"], s["post_weight"], s["post_bias"],
                                             none["gate"])
    assert h.shape == y.shape == (0, 64) and m.numel() == r.numel() == pm.numel() == pr.numel() == 0
    back = G.residual_norm_bwd(none["dy"], none["dh"], h, s["weight"], m, r, x=none["x"], post_weight=s["post_weight"],
                               post_bias=s["post_bias"], post_mean=pm, post_rstd=pr, gate=none["gate"])
    assert back[0].shape == (0, 64) and back[6].shape == (0, 64)
    assert not any(t.any() for t in back[2:6])


@pytest.mark.gpu
def test_rows_past_two_to_the_31_elements():
    import grpo_loss_gb300 as G
    d, rows, n = 4096, 524289 + 1023, 64            # 2.15e9 elements
    tail = inputs(n, d, BF16, BF16, post=False, rms=True, gate=1)
    x, res = (torch.zeros(rows, d, device="cuda", dtype=BF16) for _ in range(2))
    x[-n:], res[-n:] = tail["x"], tail["residual"]
    h, y, _, r, _, _ = G.residual_norm_fwd(x, res, tail["weight"], gate=tail["gate"], rms=True, h=res)
    want = G.residual_norm_fwd(tail["x"], tail["residual"], tail["weight"], gate=tail["gate"], rms=True)
    assert torch.equal(h[-n:], want[0]) and torch.equal(y[-n:], want[1]) and torch.equal(r[-n:], want[3]) and not h[:-n].any()
    dy = y.zero_()
    dy[-n:] = tail["dy"]
    back = G.residual_norm_bwd(dy, None, h, tail["weight"], None, r, x=x, gate=tail["gate"], rms=True, dx=x, dresidual=dy)
    alone = G.residual_norm_bwd(tail["dy"], None, want[0], tail["weight"], None, want[3], x=tail["x"], gate=tail["gate"], rms=True)
    assert torch.equal(back[0][-n:], alone[0]) and torch.equal(back[1][-n:], alone[1])
    assert not back[0][:-n].any() and not back[1][:-n].any()
    for i in (2, 6):                                # other walkers take the rows: another order of the sums
        assert (back[i] - alone[i]).abs().max() <= 1e-4 * alone[i].abs().max()


@pytest.mark.gpu
def test_repeats_streams_and_graphs():
    import grpo_loss_gb300 as G
    s = inputs(900, 1536, BF16, BF16, gate=9)
    args = [s[k] for k in ("x", "residual", "weight", "bias", "post_weight", "post_bias", "gate")]

    def both(stream=None, fwd=None, bwd=None):
        f = G.residual_norm_fwd(*args, stream=stream, **(fwd or {}))
        b = G.residual_norm_bwd(s["dy"], s["dh"], f[0], s["weight"], f[2], f[3], x=s["x"], post_weight=s["post_weight"],
                                post_bias=s["post_bias"], post_mean=f[4], post_rstd=f[5], gate=s["gate"], stream=stream,
                                **(bwd or {}))
        return f + b
    want = both()
    size = L.residual_norm_workspace_size(L.ResidualNormProblem(900, 1536, *[0] * 10, 100, 1e-5, 1.0, 0, 1, 1, 1))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = both(side)
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(None, dict(zip(FWD, outs)), dict(zip(BWD, outs[6:]), workspace=ws))
    for _ in range(2):
        for t in outs + [ws]:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (python -m grpo_loss_gb300.build)")
    return L.lib()


def problem(**kw):
    p = L.ResidualNormProblem(4, 100, *[0] * 10, 2, 1e-5, 1.0, 0, L.GRPO_F32, L.GRPO_BF16, L.GRPO_F32)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def fwd(lib, p, args=None):
    at = ctypes.c_void_p(256)
    other = ctypes.c_void_p(512)
    args = args or [at] * 8 + [other] + [at] * 4
    return lib.grpo_residual_norm_fwd(None if p is None else ctypes.byref(p), *args, None)


def bwd(lib, p, args=None):
    at, other = ctypes.c_void_p(256), ctypes.c_void_p(512)
    args = args or [at] * 12 + [other] + [at] * 6
    return lib.grpo_residual_norm_bwd(None if p is None else ctypes.byref(p), *args, at, 1 << 40, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(d=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(rms=2), 1), (dict(dtype=2), 1), (dict(param_dtype=7), 1), (dict(gate_dtype=-1), 1), (dict(gate_rows=-1), 1),
    (dict(d=32769), 2), (dict(rows=1 << 31), 2)] + [(dict(**{k: v}), 1) for k, v in (
        ("ld_x", 99), ("ld_residual", 1), ("ld_h", -5), ("ld_y", 99), ("ld_gate", 99), ("ld_dy", 99), ("ld_dh", 99),
        ("ld_dx", 99), ("ld_dresidual", 99), ("ld_dgate", 99))])
def test_refuses_bad_problems_on_the_host(lib, kw, status):
    p, size = problem(**kw), ctypes.c_size_t(0)
    assert lib.grpo_residual_norm_workspace_size(ctypes.byref(p), ctypes.byref(size)) == status
    assert fwd(lib, p) == status and bwd(lib, p) == status


def test_refuses_bad_pointers_on_the_host(lib):
    at, other, odd = ctypes.c_void_p(256), ctypes.c_void_p(512), ctypes.c_void_p(257)
    f = [at] * 8 + [other] + [at] * 4               # x res w b pw pb gate h y mean rstd pmean prstd
    b = [at] * 12 + [other] + [at] * 6              # dy dh h w mean rstd x pw pb pm pr gate dx dres dw db dpw dpb dgate
    put = lambda v, i, w: [w if j == i else t for j, t in enumerate(v)]  # noqa: E731
    p = problem()
    assert fwd(lib, None) == 1 and bwd(lib, None) == 1
    for i in (0, 1, 2, 4, 7, 8):                    # (post_weight: beside a post_bias)
        assert fwd(lib, p, put(f, i, None)) == 1
    for i in range(13):
        assert fwd(lib, p, put(f, i, odd)) == 2
    assert fwd(lib, p, put(f, 8, at)) == 1          # h is y
    for i in (0, 2, 3, 4, 5, 6, 7, 9, 10, 11, 13):
        assert bwd(lib, p, put(b, i, None)) == 1, i
    for i in range(19):
        assert bwd(lib, p, put(b, i, odd)) == 2, i
    assert bwd(lib, p, put(b, 12, at)) == 1         # dx is dresidual
    for rows in (0, 3):                             # gate rows that do not divide
        p.gate_rows = rows
        assert fwd(lib, p) == 1 and bwd(lib, p) == 1
    p = problem(rms=1)                              # an RMS norm has no bias
    assert fwd(lib, p) == 1 and bwd(lib, p) == 1
    assert fwd(lib, p, put(f, 3, None)) == 1 and bwd(lib, p, put(b, 15, None)) == 1


def test_refuses_wrong_tensors(monkeypatch):
    import grpo_loss_gb300 as G
    monkeypatch.setattr(L, "_device_of", lambda t, name: t.device)
    x, w, r = torch.zeros(6, 8), torch.ones(8), torch.zeros(6)
    for bad, word in ((dict(x=x[0]), "2-D"), (dict(x=x.half()), "float32 or"), (dict(residual=x.bfloat16()), "float32"),
                      (dict(residual=x[:3]), "shape"), (dict(weight=w[:5]), "elements"), (dict(bias=w.bfloat16()), "float32"),
                      (dict(gate=w), "2-D"), (dict(gate=torch.zeros(4, 8)), "divides"), (dict(gate=torch.zeros(0, 8)), "divides"),
                      (dict(gate=torch.zeros(3, 7)), "shape"), (dict(gate=torch.zeros(3, 8).half()), "float32 or"),
                      (dict(y=torch.zeros(1, 8).expand(6, 8)), "row stride"), (dict(x=torch.zeros(8, 6).t()), "contiguous")):
        with pytest.raises(ValueError, match=word):
            G.residual_norm_fwd(**{"x": x, "residual": x, "weight": w, **bad})
    ok = dict(dy=x, dh=x, h=x, weight=w, mean=r, rstd=r)
    for bad, word in ((dict(mean=None), "mean"), (dict(gate=torch.zeros(3, 8)), "x is needed"), (dict(post_weight=w, x=x), "statistics"),
                      (dict(dgate=x), "gate"), (dict(dy=x.bfloat16()), "float32"), (dict(dh=x[:2]), "shape"),
                      (dict(gate=torch.zeros(3, 8), x=x, dgate=torch.zeros(3, 8).bfloat16()), "float32")):
        with pytest.raises(ValueError, match=word):
            G.residual_norm_bwd(**{**ok, **bad})


@pytest.mark.gpu
def test_refuses_a_short_workspace():
    import grpo_loss_gb300 as G
    s = inputs(10, 64, F32, post=False)
    h, y, m, r, _, _ = G.residual_norm_fwd(s["x"], s["residual"], s["weight"])
    with pytest.raises(L.GrpoError) as e:
        G.residual_norm_bwd(s["dy"], s["dh"], h, s["weight"], m, r, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3


def test_kernels_have_no_read_only_loads():
    """Their outputs may be their inputs, and a read-only load is defined only for memory
    that the kernel does not write."""
    csrc = os.path.join(os.path.dirname(L.__file__), "csrc")
    for name in ("residual_norm.cu", "residual_norm_bwd.cuh", "pieces.cuh", "policy.cu", "grad_norm.cu"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//[^\n]*|/\*.*?\*/", " ", f.read(), flags=re.S)
        assert not re.findall(r"__ldg\b|__restrict__|ld\.global\.nc", code), name
