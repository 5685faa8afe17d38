"""AdamW over many tensors against float64: states in 32 bits within bounds on
float32 evaluation; 8-bit codes equal to the dithered ones of the float64 values
except where those lie within the evaluation's error of a border."""
import ctypes
import math

import numpy as np
import pytest
import torch

from grpo_loss_gb300 import _lib as L
from tests.operator_reference import adamw, block_scale, block_values, dither, dithered_steps, f64

F32, BF16 = torch.float32, torch.bfloat16
HYPER = dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
SIZES = [1, 31, 32, 33, 64, 1000, 4095, 4096, 4097, 70001]
SALT_M, SALT_V, SALT_P = 0, 0x55555555, 0xAAAAAAAA


def tensors(sizes, dtype, gdtype, seed=0, flat=0):
    """Parameters and gradients; with ``flat`` views into one buffer at offsets
    off any alignment but the element's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    def make(dt, std):
        if not flat:
            return [(torch.randn(n, generator=g, device="cuda") * std).to(dt) for n in sizes]
        big = (torch.randn(sum(sizes) + flat, generator=g, device="cuda") * std).to(dt)
        at = np.cumsum([flat] + list(sizes))
        return [big[a:a + n] for a, n in zip(at, sizes)]
    return make(dtype, 0.02), make(gdtype, 1e-3)


def check_step(before, opt, grads, step, grad_scale=1.0, lr=None):
    """``opt`` holds what a step made of the copies ``before``."""
    h = HYPER
    lr = h["lr"] if lr is None else lr
    for i, g in enumerate(grads):
        n = g.numel()
        p0, w0, m0, v0, ms0, vs0 = (None if b[i] is None else b[i] for b in before)
        eight = ms0 is not None
        m64, v64 = (block_values(m0, ms0), block_values(v0, vs0)) if eight else (f64(m0).ravel(), f64(v0).ravel())
        x64 = f64(p0 if w0 is None else w0).ravel()
        x, m, v, ex, em, ev = adamw(x64, f64(g).ravel(), m64, v64, step, lr, *h["betas"], h["eps"],
                                    opt.weight_decay[i], grad_scale)
        x = np.where(m == 0, x64 * (1 - lr * opt.weight_decay[i]), x)     # a zero gradient's 0 / 0 is 0
        if not eight:
            assert np.all(np.abs(f64(opt.exp_avg[i]).ravel() - m) <= em + 1e-44)
            assert np.all(np.abs(f64(opt.exp_avg_sq[i]).ravel() - v) <= ev + 1e-44)
        else:
            for val, q, s, salt, err, floor in ((m, opt.exp_avg[i], opt.exp_avg_scale[i], SALT_M, em, 0),
                                                (v, opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], SALT_V, ev, 1)):
                scale, want = s.cpu().numpy().astype(int), block_scale(val)
                top = np.pad(np.abs(val), (0, -n % 32)).reshape(-1, 32).max(1)
                edge = np.abs(top / np.exp2(want - 127.0) / 448 - 1) < 1e-5
                edge |= np.abs(top / np.exp2(want - 127.0) / 224 - 1) < 1e-5
                assert np.all((scale == want) | edge)
                unit, steps = dithered_steps(val, scale, dither(n, step, salt))
                got = block_values(q, s) / unit
                slack = err / unit + 2.0 ** -20
                lo, hi = np.floor(steps - slack), np.floor(steps + slack)
                if floor:          # at least the smallest step of a block that is not zero
                    least = np.exp2(np.repeat(scale, 32)[:n] - 136.0) / unit * (np.repeat(top, 32)[:n] > 0)
                    lo, hi = np.maximum(lo, least), np.maximum(hi, least)
                sign = np.where(val < 0, -1, 1)
                assert np.all((got * sign >= lo) & (got * sign <= hi)), i
        if w0 is not None:
            assert np.all(np.abs(f64(opt.masters[i]).ravel() - x) <= ex + 2.0 ** -24 * np.abs(x))
            assert torch.equal(opt.params[i], opt.masters[i].to(BF16))
        elif opt.params[i].dtype == F32:
            assert np.all(np.abs(f64(opt.params[i]).ravel() - x) <= ex + 2.0 ** -24 * np.abs(x))
        else:
            q = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 7)
            steps = np.abs(x) / q + dither(n, step, SALT_P)
            slack = (ex + 2.0 ** -24 * np.abs(x)) / q + 2.0 ** -16
            got = np.abs(f64(opt.params[i]).ravel()) / q
            assert np.all((got >= np.floor(steps - slack)) & (got <= np.floor(steps + slack))), i


def copies(opt):
    return [[None if t is None else t.clone() for t in ts] for ts in
            (opt.params, opt.masters, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)]


KINDS = [(F32, F32, False), (F32, BF16, False), (BF16, BF16, False), (BF16, F32, False), (BF16, F32, True),
         (BF16, BF16, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,gdtype,master", KINDS,
                         ids=["f32-f32", "f32-bf16", "bf16-bf16", "bf16-f32", "master-f32", "master-bf16"])
@pytest.mark.parametrize("flat", [0, 1, 3])
def test_three_steps(dtype, gdtype, master, bits, flat):
    import grpo_loss_gb300 as G
    params, _ = tensors(SIZES, dtype, gdtype, 1, flat)
    opt = G.AdamW(params, state_bits=bits, master=master, **HYPER)
    for step in (1, 2, 3):
        _, grads = tensors(SIZES, dtype, gdtype, 10 + step, flat)
        if step == 2:
            grads[5][:40] = 0
        before = copies(opt)
        opt.step(grads, grad_scale=0.5 if step == 3 else 1.0, lr=1e-3 if step == 2 else None)
        torch.cuda.synchronize()
        assert opt.step_count == step
        check_step(before, opt, grads, step, 0.5 if step == 3 else 1.0, 1e-3 if step == 2 else None)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_wide_ranges_and_zeros(bits):
    """Tiny, huge and zero gradients side by side in blocks; a tensor whose
    gradients are all zero keeps zero states."""
    import grpo_loss_gb300 as G
    p, _ = tensors([4096, 100, 4096], F32, F32, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (4096, 100, 4096)]
    grads[0] *= torch.exp2(torch.randint(-60, 30, (4096,), generator=g, device="cuda").float())
    grads[1].zero_()
    grads[2][::7] = 0
    opt = G.AdamW(p, state_bits=bits, **HYPER)
    for step in (1, 2):
        before = copies(opt)
        opt.step(grads)
        torch.cuda.synchronize()
        check_step(before, opt, grads, step)
    assert not opt.exp_avg[1].any() and not opt.exp_avg_sq[1].any()


@pytest.mark.gpu
def test_not_finite_gradients_stay_in_their_block():
    import grpo_loss_gb300 as G
    for bits in (8, 32):
        p, grads = tensors([4096], BF16, F32, 6)
        grads[0][100], grads[0][2000] = math.nan, math.inf
        opt = G.AdamW(p, state_bits=bits, **HYPER)
        opt.step(grads)
        opt.step([torch.zeros_like(grads[0])])
        bad = ~torch.isfinite(p[0].float())
        if bits == 8:
            want = torch.zeros_like(bad)
            want[96:128], want[1984:2016] = True, True
        else:
            want = torch.zeros_like(bad)
            want[100], want[2000] = True, True
        assert torch.equal(bad, want)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_of_mixed_kinds(bits):
    """More tensors than one launch's table holds, empty ones and every mix of
    types in one call: as each tensor alone."""
    import grpo_loss_gb300 as G
    g = torch.Generator(device="cuda").manual_seed(9)
    kinds = [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)]
    sizes = [(i * 37) % 301 for i in range(1200)]
    params = [torch.randn(n, generator=g, device="cuda").to(kinds[i % 4][0]) for i, n in enumerate(sizes)]
    grads = [torch.randn(n, generator=g, device="cuda").to(kinds[i % 4][1]) for i, n in enumerate(sizes)]
    wd = [0.1 * (i % 3) for i in range(1200)]
    hyper = {**HYPER, "weight_decay": wd}
    alone = [p.clone() for p in params]
    opt = G.AdamW(params, state_bits=bits, **hyper)
    opt.step(grads)
    for i in range(0, 1200, 7):
        one = G.AdamW([alone[i]], state_bits=bits, **{**HYPER, "weight_decay": wd[i]})
        one.step([grads[i]])
        assert torch.equal(alone[i], params[i]) and torch.equal(one.exp_avg[0], opt.exp_avg[i])
        assert torch.equal(one.exp_avg_sq[0], opt.exp_avg_sq[i])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
def test_step_into_other_buffers(bits, master):
    import grpo_loss_gb300 as G
    params, grads = tensors(SIZES, BF16, F32, 2)
    opt = G.AdamW(params, state_bits=bits, master=master, **HYPER)
    opt.step(grads)
    other = G.AdamW([torch.full_like(p, 7.0) for p in params], state_bits=bits, master=master, **HYPER)
    before, versions = copies(opt), [p._version for p in params]
    opt.step(grads, out=other)
    for ts, ks in zip(copies(opt), before):         # the source stays
        for t, k in zip(ts, ks):
            assert (t is None and k is None) or torch.equal(t, k)
    assert other.step_count == 2 and opt.step_count == 1
    assert versions == [p._version for p in params]
    opt.step(grads)
    assert all(p._version > v for p, v in zip(params, versions))         # autograd sees the change
    for ts, ks in zip(copies(opt), copies(other)):
        for t, k in zip(ts, ks):
            assert (t is None and k is None) or torch.equal(t, k)


@pytest.mark.gpu
def test_dither_keeps_small_changes():
    """Where a step moves a value by far less than half a code, the mean over
    steps still moves by it: v reaches the mean square of the gradients and a
    bf16 parameter with no master follows its float32 counterpart."""
    import grpo_loss_gb300 as G
    n, steps = 4096, 1500
    g = torch.Generator(device="cuda").manual_seed(5)
    opt = G.AdamW([torch.zeros(n, device="cuda")], state_bits=8, lr=0.0, weight_decay=0.0, betas=(0.9, 0.99))
    for _ in range(steps):
        opt.step([torch.randn(n, generator=g, device="cuda")])
    v = torch.from_numpy(block_values(opt.exp_avg_sq[0], opt.exp_avg_sq_scale[0]))
    # E[g^2] = 1; its running mean has a deviation of sqrt(2 * 0.01 / 1.99) = 0.1, 4096 values
    # average that out, and a code's step of an eighth at most is what rounding could keep
    assert abs(v.mean().item() - 1.0) < 0.125 / 2
    p = torch.full((n,), 1.0, device="cuda", dtype=BF16)
    low = G.AdamW([p], lr=1e-4, weight_decay=0.0)                 # a bf16 step at 1 is 2^-8 or 2^-7
    for _ in range(100):
        low.step([torch.ones(n, device="cuda", dtype=BF16)])
    assert abs(p.double().mean().item() - 0.99) < 2.0 ** -9


@pytest.mark.gpu
def test_more_than_two_to_the_31_elements():
    import grpo_loss_gb300 as G
    n = (1 << 31) + 4096 + 5
    p = torch.ones(n, device="cuda", dtype=BF16)
    g = torch.zeros(n, device="cuda", dtype=BF16)
    tail = torch.randn(4096 + 5, device="cuda").to(BF16)
    g[-tail.numel():] = tail
    opt = G.AdamW([p], state_bits=8, lr=1e-2, weight_decay=0.0)
    opt.step([g])
    assert bool((p[: 1 << 31] == 1).all())
    small = torch.ones(tail.numel(), device="cuda", dtype=BF16)
    one = G.AdamW([small], state_bits=8, lr=1e-2, weight_decay=0.0)
    one.step([tail])                                # 2^31 is whole blocks: the same scales
    assert torch.equal(one.exp_avg_scale[0], opt.exp_avg_scale[0][-one.exp_avg_scale[0].numel():])
    assert (p[-tail.numel():].float() - small.float()).abs().max() <= 2.0 ** -7


@pytest.mark.gpu
def test_repeats_streams_and_graphs():
    import grpo_loss_gb300 as G
    for bits in (8, 32):
        params, grads = tensors([5000, 77], BF16, BF16, 2)
        opt = G.AdamW(params, state_bits=bits, master=True, **HYPER)
        opt.step(grads)
        outs = [G.AdamW([p.clone() for p in params], state_bits=bits, master=True, **HYPER) for _ in range(3)]
        opt.step(grads, out=outs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        opt.step(grads, out=outs[1], stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step(grads, out=outs[2], step=2)
        graph.replay()
        torch.cuda.synchronize()
        for o in outs[1:]:
            for ts, ks in zip(copies(o), copies(outs[0])):
                for t, k in zip(ts, ks):
                    assert (t is None and k is None) or torch.equal(t, k)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_same_bits_on_and_off_a_boundary(dtype, bits):
    """Elements that are taken in pieces and one by one, and moments that are those
    of float32 operations one after the other."""
    import grpo_loss_gb300 as G
    n = 20000
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    p, grads = rand().to(dtype), [rand() * 1e-3 for _ in range(4)]
    shifted = torch.empty(n + 1, dtype=dtype, device="cuda")[1:].copy_(p)
    a, b = (G.AdamW([t], state_bits=bits, lr=1e-2) for t in (p, shifted))
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for x in grads:
        off = torch.empty(n + 1, device="cuda")[1:].copy_(x)
        a.step([x])
        b.step([off])
        m, v = 0.9 * m + (1 - 0.9) * x, 0.999 * v + (1 - 0.999) * x * x
        for s, t in zip((a.params, a.exp_avg, a.exp_avg_sq), (b.params, b.exp_avg, b.exp_avg_sq)):
            assert torch.equal(s[0], t[0])
        if bits == 32:
            assert torch.equal(a.exp_avg[0], m) and torch.equal(a.exp_avg_sq[0], v)
        else:
            assert torch.equal(a.exp_avg_scale[0], b.exp_avg_scale[0])
            assert torch.equal(a.exp_avg_sq_scale[0], b.exp_avg_sq_scale[0])

@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-40, 1e-50, 1.17e-38])
def test_a_tiny_eps_is_not_none(eps, bits):
    """Below float32's normal range, too, an element with no moments stays: 0 / eps."""
    import grpo_loss_gb300 as G
    for n in (7, 4096):                                      # one by one, and in pieces
        g = torch.Generator(device="cuda").manual_seed(n)
        p = torch.randn(n, generator=g, device="cuda")
        grad = torch.randn(n, generator=g, device="cuda")
        grad[::2] = 0.0
        grad[n // 2: n // 2 + 64] = 0.0                      # whole blocks, too
        still = grad == 0
        before = p.clone()
        G.AdamW([p], lr=1e-3, eps=eps, weight_decay=0.0, state_bits=bits).step([grad])
        torch.cuda.synchronize()
        assert torch.isfinite(p).all()
        assert torch.equal(p[still], before[still])
        moved = grad != 0                                    # the first step moves by lr: m / sqrt(v) is a sign
        off = (p.double() - (before.double() - 1e-3 * grad.sign().double()))[moved].abs()
        # the update to 2^-20 (roundings of m, v and the constants 2^-24 each, root and quotient 2^-22), p to 2^-24
        assert bool((off <= 1e-3 * 2.0 ** -20 + 2.0 ** -24 * (before[moved].abs().double() + 1e-3)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_run_goes_on_from_its_lists(bits):
    """Saved and restored, by copies into the tensors or by other tensors in the lists."""
    import grpo_loss_gb300 as G
    sizes = [5000, 77]
    params, _ = tensors(sizes, BF16, F32, 2)
    steps = [tensors(sizes, BF16, F32, 20 + i)[1] for i in range(3)]
    opt = G.AdamW(params, state_bits=bits, master=True, **HYPER)
    for g in steps[:2]:
        opt.step(g)
    saved, count = copies(opt), opt.step_count
    opt.step(steps[2])
    for replace in (False, True):
        again = G.AdamW([torch.zeros_like(p) for p in params], state_bits=bits, master=True, **HYPER)
        again.step([torch.zeros_like(g) for g in steps[0]])          # its table is made
        for mine, theirs in zip((again.params, again.masters, again.exp_avg, again.exp_avg_sq, again.exp_avg_scale,
                                 again.exp_avg_sq_scale), saved):
            for i, t in enumerate(theirs):
                if t is not None and replace:
                    mine[i] = t.clone()
                elif t is not None:
                    mine[i].copy_(t)
        again.step_count = count
        again.step(steps[2])
        torch.cuda.synchronize()
        for ts, ks in zip(copies(again), copies(opt)):
            for t, k in zip(ts, ks):
                assert (t is None and k is None) or torch.equal(t, k)



# ---------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (python -m grpo_loss_gb300.build)")
    return L.lib()


def _call(lib, config=None, tensor=None, n=1, out=None):
    c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, state_bits=8, step=1)
    c.update(config or {})
    at = 4096
    t = dict(n=64, grad=at, param=at, master=None, m=at, v=at, m_scale=at, v_scale=at, weight_decay=0.1,
             param_dtype=L.GRPO_BF16, grad_dtype=L.GRPO_F32)
    t.update(tensor or {})
    arr = (L.AdamwTensor * 1)(L.AdamwTensor(**t))
    to = None if out is None else (L.AdamwTensor * 1)(L.AdamwTensor(**{**t, **out}))
    return lib.grpo_adamw_step(ctypes.byref(L.AdamwConfig(**c)), arr, to, n, None)


@pytest.mark.parametrize("config", [dict(lr=-1.0), dict(lr=math.nan), dict(beta1=1.0), dict(beta2=-0.1),
                                    dict(beta1=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(grad_scale=math.nan),
                                    dict(state_bits=16), dict(step=0)], ids=str)
def test_refuses_bad_settings_on_the_host(lib, config):
    assert _call(lib, config) == 1


@pytest.mark.parametrize("tensor,status", [
    (dict(n=-1), 1), (dict(grad=None), 1), (dict(param=None), 1), (dict(m=None), 1), (dict(v=None), 1),
    (dict(m_scale=None), 1), (dict(v_scale=None), 1), (dict(weight_decay=-0.1), 1), (dict(weight_decay=math.inf), 1),
    (dict(param_dtype=2), 1), (dict(grad_dtype=5), 1), (dict(master=4096, param_dtype=0), 1),
    (dict(grad=4098), 2), (dict(param=4097), 2),
    (dict(master=4098), 2), (dict(n=(1 << 40) + 1), 2)], ids=str)
def test_refuses_bad_tensors_on_the_host(lib, tensor, status):
    assert _call(lib, tensor=tensor) == status


def test_refuses_states_of_the_other_width(lib):
    assert _call(lib, dict(state_bits=32)) == 1                          # scales beside float32 states
    assert _call(lib, dict(state_bits=32), dict(m_scale=None, v_scale=None, m=4098)) == 2
    assert _call(lib, n=-1) == 1
    assert lib.grpo_adamw_step(None, None, None, 0, None) == 1


@pytest.mark.parametrize("out,status", [
    (dict(n=63), 1), (dict(param_dtype=0), 1), (dict(master=4096), 1), (dict(param=None), 1), (dict(m=None), 1),
    (dict(m_scale=None), 1), (dict(param=4097), 2)], ids=str)
def test_refuses_outputs_of_another_kind(lib, out, status):
    assert _call(lib, out=out) == status


def test_binding_refuses_wrong_tensors():
    import grpo_loss_gb300 as G
    with pytest.raises(ValueError, match="state_bits"):
        G.AdamW([], state_bits=4)
    with pytest.raises(ValueError, match="CUDA"):
        G.AdamW([torch.zeros(3)])
    with pytest.raises(ValueError, match="weight_decay"):
        G.AdamW([], weight_decay=[0.1])
    G.AdamW([]).step([])
    with pytest.raises(ValueError, match="gradients"):
        G.AdamW([]).step([torch.zeros(3)])


@pytest.fixture
def calls(monkeypatch):
    """Steps on the host alone: what each would have launched, tensor by tensor."""
    got = []
    monkeypatch.setattr(L, "_ptr", lambda t, name: t.data_ptr())
    monkeypatch.setattr(L, "adamw_step", lambda config, tensors, out, n, device, stream=None: got.append(
        [{f: getattr(t[i], f) for f, _ in L.AdamwTensor._fields_} for t in (tensors, out) if t is not None for i in range(n)]))
    return got


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_that_shrank_where_it_is(calls, bits):
    """The same address with fewer elements: refused while the states are longer,
    and taken with its own size once they are not."""
    import grpo_loss_gb300 as G
    p, q = torch.zeros(1000, 64), torch.zeros(5)
    opt = G.AdamW([p, q], state_bits=bits)
    p.data = p.data[:10]
    with pytest.raises(ValueError, match="elements"):
        opt.step([torch.zeros(10, 64), torch.zeros(5)])
    with pytest.raises(ValueError, match="elements"):        # and again: nothing was half bound
        opt.step([torch.zeros(10, 64), torch.zeros(5)])
    assert not calls and opt.step_count == 0
    for ts in (opt.exp_avg, opt.exp_avg_sq):
        ts[0] = ts[0][:10]
    for ts in (opt.exp_avg_scale, opt.exp_avg_sq_scale):
        ts[0] = None if bits == 32 else ts[0][:20]
    opt.step([torch.zeros(10, 64), torch.zeros(5)])
    assert [t["n"] for t in calls[0]] == [640, 5]


def test_a_parameter_that_changed_where_it_is(calls):
    import grpo_loss_gb300 as G
    p = torch.zeros(8, 8)
    opt, out = G.AdamW([p]), G.AdamW([torch.zeros(8, 8)])
    opt.step([torch.zeros(8, 8)], out=out)
    p.data = p.data.t()                                       # a square: shape and size stay
    with pytest.raises(ValueError, match="contiguous"):
        opt.step([torch.zeros(8, 8)])
    p.data = p.data.t().view(4, 16)
    opt.step([torch.zeros(4, 16)])
    with pytest.raises(ValueError, match="out must be"):      # which has the old shape
        opt.step([torch.zeros(4, 16)], out=out)
    whole = torch.zeros(64)
    opt, out = G.AdamW([whole]), G.AdamW([torch.zeros(64)])
    opt.step([whole], out=out)
    out.params[0].data = out.params[0].data[:32]
    with pytest.raises(ValueError, match="elements"):
        opt.step([whole], out=out)
    opt.params[0] = whole.view(BF16)[:64]                     # the same address and length, another type
    opt.step([torch.zeros(64)])
    assert calls[-1][0]["param_dtype"] == L.GRPO_BF16


def test_a_state_that_shrank_where_it_is(calls):
    import grpo_loss_gb300 as G
    opt = G.AdamW([torch.zeros(64, dtype=BF16)], master=True)
    for ts in (opt.exp_avg, opt.exp_avg_sq, opt.masters):
        keep = ts[0]
        ts[0] = keep[:32]
        with pytest.raises(ValueError, match="elements"):
            opt.step([torch.zeros(64)])
        ts[0] = keep
    opt.step([torch.zeros(64)])
    assert len(calls) == 1


def test_weight_decay_acts_when_it_is_changed(calls):
    """As lr, betas and eps do; with another AdamW's buffers, too."""
    import grpo_loss_gb300 as G
    ps, gs = [torch.zeros(8), torch.zeros(8)], [torch.zeros(8), torch.zeros(8)]
    opt = G.AdamW(ps, weight_decay=0.5)
    opt.step(gs)
    opt.weight_decay[0] = 0.25
    opt.step(gs)
    opt.weight_decay = [0.0, 0.125]
    opt.step(gs, out=G.AdamW([p.clone() for p in ps]))
    opt.weight_decay = 0.75
    opt.step(gs)
    assert [[t["weight_decay"] for t in c[:2]] for c in calls] == [[0.5, 0.5], [0.25, 0.5], [0.0, 0.125], [0.75, 0.75]]
    for bad in ([0.1], [0.1] * 3, ["a", 0.1]):
        opt.weight_decay = bad
        with pytest.raises(ValueError):
            opt.step(gs)
    assert len(calls) == 4


@pytest.mark.parametrize("bad", [None, 1.0, np.zeros(8, np.float32)], ids=["none", "number", "array"])
def test_refuses_gradients_that_are_not_tensors(calls, bad):
    import grpo_loss_gb300 as G
    opt = G.AdamW([torch.zeros(8), torch.zeros(8)])
    with pytest.raises(ValueError, match=r"grads\[1\] must be a tensor"):
        opt.step([torch.zeros(8), bad])
    assert not calls and opt.step_count == 0


def test_refuses_buffers_that_overlap(calls):
    """A tensor given twice (tied weights) would be updated by two parts of one launch
    at a time; neighbours in one buffer are no overlap, and empty ones never are."""
    import grpo_loss_gb300 as G
    flat = torch.zeros(100)
    for params in ([flat, torch.zeros(3), flat], [flat[:60], flat[50:]], [flat, flat[10:20]], [flat.view(10, 10), flat]):
        with pytest.raises(ValueError, match=r"overlaps"):
            G.AdamW(params)
    opt = G.AdamW([flat[:50], flat[50:], torch.zeros(0), flat[:0], torch.zeros(0)])
    opt.step([torch.zeros(50), torch.zeros(50)] + [torch.zeros(0)] * 3)
    opt.exp_avg[1] = opt.exp_avg[0]
    with pytest.raises(ValueError, match="overlaps"):
        opt.step([torch.zeros(50), torch.zeros(50)] + [torch.zeros(0)] * 3)
    assert len(calls) == 1


@pytest.mark.gpu
def test_binding_refuses_wrong_gpu_tensors():
    import grpo_loss_gb300 as G
    p = torch.zeros(4, 6, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        G.AdamW([p.t()])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        G.AdamW([p.half()])
    opt = G.AdamW([p])
    for g, word in ((torch.zeros(6, 4, device="cuda"), "shape"), (torch.zeros(4, 6), "on cuda"),
                    (torch.zeros(6, 4, device="cuda").t(), "contiguous"), (p.half(), "float32 or")):
        with pytest.raises(ValueError, match=word):
            opt.step([g])
    with pytest.raises(ValueError, match="out must be"):
        opt.step([p], out=opt)
    with pytest.raises(ValueError, match="out must be"):
        opt.step([p], out=G.AdamW([p.clone()], state_bits=8))
    with pytest.raises(L.GrpoError):
        opt.step([p], step=0)
    assert opt.step_count == 0
