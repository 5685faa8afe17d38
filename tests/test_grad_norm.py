"""The norm of many gradients, clipping by it, and the optimizer step that takes the
factor, against float64."""
import ctypes
import math

import numpy as np
import pytest
import torch

from grpo_loss_gb300 import _lib as L
from tests.operator_reference import U, f64

F32, BF16 = torch.float32, torch.bfloat16
SIZES = [1, 2, 3, 7, 8, 31, 257, 1000, 4096, 4097, 8191, 70001, 0, 5, 300000]


def gradients(sizes, dtypes=(F32, BF16), seed=0, packed=False, std=1e-2, offset=0):
    """One tensor a size, of the types in turn; ``packed``: views of one buffer a type,
    ``offset`` elements behind a boundary."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kinds = [dtypes[i % len(dtypes)] for i in range(len(sizes))]
    made = [(torch.randn(n, generator=g, device="cuda") * std).to(k) for n, k in zip(sizes, kinds)]
    if not packed:
        return made
    flat = {k: torch.zeros(offset + sum(n for n, t in zip(sizes, kinds) if t == k), dtype=k, device="cuda") for k in dtypes}
    at, views = dict.fromkeys(dtypes, offset), []
    for t in made:
        view = flat[t.dtype][at[t.dtype]:at[t.dtype] + t.numel()]
        view.copy_(t)
        at[t.dtype] += t.numel()
        views.append(view)
    return views


def norm_of(grads, kind=2.0):
    flat = np.concatenate([f64(g).ravel() for g in grads] + [np.zeros(1)])
    return np.sqrt((flat ** 2).sum()) if kind == 2.0 else np.abs(flat).max()


# float32 sums of 64 squares at most before float64 takes over, in either order: each at
# most 64 roundings off; the root halves it, and the result is rounded once
REL = 64 * 2.0 ** -24 / 2 + 2.0 ** -24


def check_clip(grads, max_norm, kind=2.0, eps=1e-6, out=None):
    import grpo_loss_gb300 as G
    want = norm_of(grads, kind)
    factor = min(1.0, max_norm / (want + eps))
    before = [f64(g) for g in grads]
    norm = G.clip_grad_norm(grads, max_norm, norm_type=kind, eps=eps, out=out)
    torch.cuda.synchronize()
    assert norm.shape == (1,) and abs(norm.item() - want) <= REL * want
    for b, g, o in zip(before, grads, out or grads):
        tol = np.abs(b * factor) * (REL + 2 * 2.0 ** -24 + U[g.dtype] * 1.001) + 1e-40
        assert np.all(np.abs(f64(o) - b * factor) <= tol)
        if out is not None:
            assert np.array_equal(f64(g), b)
    return norm


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F32, BF16)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("packed,offset", [(False, 0), (True, 0), (True, 1), (True, 5)])
def test_norm_and_clip(packed, offset, dtypes, kind):
    import grpo_loss_gb300 as G
    make = lambda s: gradients(SIZES, dtypes, s, packed, offset=offset)  # noqa: E731
    grads = make(1)
    want = norm_of(grads, kind)
    assert abs(G.grad_norm(grads, norm_type=kind).item() - want) <= REL * want
    for max_norm in (want * 0.37, want * 2):
        check_clip(make(1), max_norm, kind)
        check_clip(make(1), max_norm, kind, out=make(2))
        mixed = make(3)                             # outputs that lie otherwise than their gradients
        check_clip(gradients(SIZES, dtypes, 1), max_norm, kind, out=mixed)
    for i, n in enumerate(SIZES):                   # each size alone
        g = make(4)[i]
        got, want = G.grad_norm([g], norm_type=kind).item(), norm_of([g], kind)
        assert abs(got - want) <= REL * want


@pytest.mark.gpu
def test_what_is_beside_a_tensor_stays():
    flat = torch.ones(5000, device="cuda")
    view = flat[3:4000]
    check_clip([view], 1.0)
    assert (flat[:3] == 1).all() and (flat[4000:] == 1).all() and (view < 0.1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 100, 1000, 1001, 2500])
def test_many_tensors(n):
    import grpo_loss_gb300 as G
    g = torch.Generator(device="cuda").manual_seed(n)
    grads = gradients([1 + (7 * i) % 300 for i in range(n)], seed=n)
    check_clip(grads, norm_of(grads) / 3)
    check_clip(gradients([1 + (7 * i) % 300 for i in range(n)], seed=n), 1e-3, math.inf)
    del g
    assert G.grad_norm([]).item() == 0.0 and G.clip_grad_norm([], 1.0).item() == 0.0
    assert G.grad_norm(grads[:0], max_norm=2.0)[1].item() == 1.0


@pytest.mark.gpu
def test_more_tensors_than_all_launches_hold():
    grads = list(torch.full((17003, 2), 0.5, device="cuda").unbind(0))
    check_clip(grads, 1.0)
    check_clip(list(torch.full((17003, 2), 0.5, device="cuda").unbind(0)), 0.1, math.inf)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_sizes(dtype):
    """Squares that float32 does not hold, side by side with others and alone; zeros."""
    import grpo_loss_gb300 as G
    for std in (1e-38, 1e-30, 1e-20, 1e-12, 1e10, 1e19, 1e30):
        for n in (5, 5000, 200000):
            grads = gradients([n], (dtype,), 5, std=std)
            want = norm_of(grads)
            assert abs(G.grad_norm(grads).item() - want) <= REL * want + 1e-45
            assert abs(G.grad_norm(grads, norm_type=math.inf).item() - norm_of(grads, math.inf)) == 0
    grads = [g for s in (1e-30, 1e-15, 1.0, 1e22, 1e25) for g in gradients([3000, 40], (dtype,), 6, std=s)]
    want = norm_of(grads)
    assert abs(G.grad_norm(grads).item() - want) <= REL * want
    mix = gradients([100000], (dtype,), 7, std=1e-25)[0]
    mix[::1000] = 1e-3
    mix[5] = 3e24
    assert abs(G.grad_norm([mix]).item() - norm_of([mix])) <= REL * norm_of([mix])
    assert G.grad_norm([torch.zeros(100000, dtype=dtype, device="cuda")]).item() == 0.0
    big = torch.full((1 << 20,), 3e38, device="cuda")            # the norm itself beyond float32
    norm, factor = G.grad_norm([big], max_norm=1.0)
    assert norm.item() == math.inf and abs(factor.item() - 1 / (3e38 * 1024)) <= 1e-45


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_not_finite(dtype):
    import grpo_loss_gb300 as G
    for kind in (2.0, math.inf):
        for at in (0, 3, 4099, 9999):
            g = gradients([10000], (dtype,), 8)[0]
            g[at] = -math.inf
            norm, factor = G.grad_norm([g], kind, max_norm=1.0)
            assert norm.item() == math.inf and factor.item() == 0
            g[(at + 77) % 10000] = math.nan
            norm, factor = G.grad_norm([g], kind, max_norm=1.0)
            assert math.isnan(norm.item()) and math.isnan(factor.item())
    g = gradients([100], (dtype,), 8)[0]
    g[5] = math.inf
    G.clip_grad_norm([g], 1.0)
    assert math.isnan(g[5].item()) and not g[:5].any()
    g = gradients([100], (dtype,), 9)[0]
    same = g.clone()
    G.clip_grad_norm([g], math.inf)                 # no limit
    assert torch.equal(g, same)
    G.clip_grad_norm([g], 0.0)
    assert not g.any()


@pytest.mark.gpu
def test_a_factor_of_one_changes_nothing():
    import grpo_loss_gb300 as G
    grads = gradients(SIZES, seed=11)
    same, out = [g.clone() for g in grads], [torch.empty_like(g) for g in grads]
    G.clip_grad_norm(grads, 1e9)
    G.clip_grad_norm(grads, 1e9, out=out)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(grads, same, out))


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[100], [3000, 50], [5000000, 17], [200000] * 30])
def test_repeats_streams_and_graphs(sizes):
    import grpo_loss_gb300 as G
    grads = gradients(sizes, seed=12)
    out = [torch.empty_like(g) for g in grads]
    want = G.clip_grad_norm(grads, 0.5, out=out).clone()
    kept = [t.clone() for t in out]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        for t in out:
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        norm = G.clip_grad_norm(grads, 0.5, out=out, stream=side)
        junk = [torch.full((1 << 17,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, kept))
        del junk
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.clip_grad_norm(grads, 0.5, out=out, norm=norm)
    for _ in range(3):
        for t in out + [norm]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, kept))


@pytest.mark.gpu
def test_elements_past_two_to_the_31():
    import grpo_loss_gb300 as G
    g = torch.zeros((1 << 31) + 4099, dtype=BF16, device="cuda")
    g[-3:] = 4.0
    g[0] = 1.0
    assert abs(G.grad_norm([g]).item() - 7.0) <= REL * 7
    G.clip_grad_norm([g], 3.5, eps=0.0)
    assert (g[-3:] == 2.0).all() and g[0] == 0.5 and not g[1:-3].any()


KINDS = [(F32, F32, False), (BF16, BF16, False), (BF16, F32, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,gdtype,master", KINDS, ids=["f32", "bf16", "master"])
def test_a_step_takes_the_factor(dtype, gdtype, master, bits):
    """The step with the factor on the device is that with the same number as its
    grad_scale, bit by bit; a factor of one that of no factor."""
    import grpo_loss_gb300 as G
    sizes = [1, 33, 4096, 70001]
    grads = gradients(sizes, (gdtype,), 20, std=1.0)

    def run(**kw):
        params = [p.clone() for p in gradients(sizes, (dtype,), 21)]
        opt = G.AdamW(params, lr=1e-3, state_bits=bits, master=master)
        for _ in range(3):
            opt.step(grads, **kw)
        return opt.params + opt.exp_avg + opt.exp_avg_sq + [t for t in opt.masters if t is not None]
    norm, factor = G.grad_norm(grads, max_norm=1.0)
    assert 0 < factor.item() < 0.5
    for a, b in zip(run(factor=factor), run(grad_scale=factor.item())):
        assert torch.equal(a, b)
    two = torch.full((1,), 2.0, device="cuda")
    for a, b in zip(run(factor=two, grad_scale=0.25), run(grad_scale=0.5)):
        assert torch.equal(a, b)
    for a, b in zip(run(factor=torch.ones(1, device="cuda")), run()):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (python -m grpo_loss_gb300.build)")
    return L.lib()


def test_refuses_bad_calls_on_the_host(lib):
    at, odd = ctypes.c_void_p(256), ctypes.c_void_p(257)
    table = (L.GradTensor * 2)()
    for t in table:
        t.n, t.grad, t.out, t.dtype = 10, 256, 512, L.GRPO_F32
    p = ctypes.addressof(table)

    def both(tensors=p, n=2, kind=2, max_norm=1.0, eps=0.0, norm=at, factor=at):
        a = lib.grpo_grad_norm(tensors, n, kind, max_norm, eps, norm, factor, at, 1 << 40, None)
        assert lib.grpo_clip_grad_norm(tensors, n, kind, max_norm, eps, norm, factor, at, 1 << 40, None) == a
        return a
    for kw in (dict(tensors=None), dict(n=-1), dict(kind=1), dict(kind=3), dict(max_norm=-1.0), dict(max_norm=math.nan),
               dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(norm=None)):
        assert both(**kw) == 1, kw
    assert both(norm=odd) == 2 and both(factor=odd) == 2
    assert lib.grpo_clip_grad_norm(p, 2, 2, 1.0, 0.0, at, None, at, 1 << 40, None) == 1    # the factor is needed
    for field, value, status in (("n", -1, 1), ("dtype", 2, 1), ("grad", None, 1), ("grad", 258, 2), ("n", 1 << 41, 2)):
        keep = getattr(table[1], field)
        setattr(table[1], field, value)
        assert both() == status, field
        setattr(table[1], field, keep)
    for value, status in ((None, 1), (513, 2)):
        table[0].out = value
        assert lib.grpo_clip_grad_norm(p, 2, 2, 1.0, 0.0, at, at, at, 1 << 40, None) == status
        table[0].out = 512


def test_refuses_more_elements_than_their_chunks_can_be_counted(lib):
    table = (L.GradTensor * 64)()
    for t in table:
        t.n, t.grad, t.out, t.dtype = (1 << 34) + 1, 256, 256, L.GRPO_BF16
    at = ctypes.c_void_p(256)
    for fn in (lib.grpo_grad_norm, lib.grpo_clip_grad_norm):
        assert fn(ctypes.addressof(table), 64, 2, 1.0, 0.0, at, at, at, 1 << 40, None) == 2


@pytest.mark.parametrize("call", ["grad_norm", "clip_grad_norm"])
def test_refuses_wrong_tensors_on_the_host(monkeypatch, call):
    import grpo_loss_gb300 as G
    f = getattr(G, call)
    g = torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        f([g], max_norm=1.0)
    with pytest.raises(ValueError, match="must be a tensor"):
        f([None], max_norm=1.0)
    with pytest.raises(ValueError, match="norm_type"):
        f([g], max_norm=1.0, norm_type=1.0)
    with pytest.raises(ValueError, match="max_norm"):
        f([g], max_norm=-1.0)
    with pytest.raises(ValueError, match="max_norm"):
        f([g], max_norm=math.nan)


@pytest.mark.gpu
def test_refuses_wrong_tensors():
    import grpo_loss_gb300 as G
    g = torch.zeros(8, 8, device="cuda")
    for grads, word in (([g, g.half()], "float32 or"), ([g, g.t()], "contiguous"), ([g, g.cpu()], "CUDA"), ([g, 3.0], "tensor")):
        with pytest.raises(ValueError, match=word):
            G.grad_norm(grads)
    for out in ([g.bfloat16()], [g[:4]], [g.t()], [torch.zeros(8, 8)], [None]):
        with pytest.raises(ValueError, match="out\\[0\\]"):
            G.clip_grad_norm([g], 1.0, out=out)
    with pytest.raises(ValueError, match="expected 1"):
        G.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(L.GrpoError) as e:           # (a short list needs none)
        G.grad_norm([g] * 40, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(ValueError, match="elements"):
        G.grad_norm([g], norm=torch.zeros(2, device="cuda"))


@pytest.mark.gpu
def test_overlapping_tensors_are_refused_where_they_are_written():
    import grpo_loss_gb300 as G
    flat = torch.ones(100, device="cuda")
    other = torch.empty(50, device="cuda")
    a, b = flat[:50], flat[49:99]
    G.grad_norm([a, b, a])                          # only read: counted as often as given
    G.clip_grad_norm([a, a], 1.0, out=[other, torch.empty_like(other)])
    for grads, out in (([a, b], None), ([a, a], None), ([a, flat[50:]], [other, other]), ([a], [b]), ([a, flat[50:]], [flat[50:], a]),
                       ([a, b], [a, other])):
        before = flat.clone()
        with pytest.raises(ValueError, match="overlap"):
            G.clip_grad_norm(grads, 1.0, out=out)
        assert torch.equal(flat, before)
    G.clip_grad_norm([a, flat[50:]], 1.0)           # side by side
    G.clip_grad_norm([a, flat[50:]], 1.0, out=[a, other])
    G.clip_grad_norm([flat[:0], a, flat[10:10]], 1.0)
    # one that lies inside another, with a third between their ends
    x, y = flat[:100], flat[60:70]
    with pytest.raises(ValueError, match="overlap"):
        G.clip_grad_norm([x, flat[10:20], y], 1.0, out=[torch.empty_like(x), torch.empty(10, device="cuda"), y])


@pytest.mark.gpu
def test_written_tensors_are_known_to_be_written():
    import grpo_loss_gb300 as G
    g, out, norm, factor = (torch.ones(8, device="cuda") for _ in range(4))
    norm, factor = norm[:1], factor[:1]
    seen = [t._version for t in (g, out, norm, factor)]
    G.grad_norm([g], max_norm=1.0, norm=norm, factor=factor)
    assert [t._version > v for t, v in zip((g, out, norm, factor), seen)] == [False, False, True, True]
    G.clip_grad_norm([g], 1.0, out=[out])
    assert out._version > seen[1] and g._version == seen[0]
    G.clip_grad_norm([g], 1.0)
    assert g._version > seen[0]
