"""The clipped policy loss against float64, with its gradient and statistics, within
bounds on float32 evaluation; its refusals; the head's backward from it."""
import ctypes
import math

import numpy as np
import pytest
import torch

from grpo_loss_gb300 import _lib as L
from tests.operator_reference import f64
from tests.update_reference import policy

F32 = torch.float32


def inputs(B, T, seed=0, fill=0.4, pad=0, token_adv=False, spread=0.25, device="cuda"):
    """Strided [B, T] views when ``pad``; masks with holes, whole rows empty; what is
    masked is not finite."""
    g = torch.Generator().manual_seed(seed * 1009 + B * 31 + T)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    old = -(n(B, T + pad) * 1.4 - 1).exp()
    q = old + spread * n(B, T + pad) + 0.1 * n(B, 1)
    ref = q + 0.2 * n(B, T + pad) * (1 + 10 * (torch.rand(B, T + pad, generator=g) < 0.02))
    length = (fill + (1 - fill) * torch.rand(B, generator=g)) * T
    mask = (torch.arange(T + pad)[None, :] < length[:, None]) & (torch.rand(B, T + pad, generator=g) < 0.95)
    if B > 2:
        mask[1] = False
    adv = n(B, T + pad) if token_adv else n(B)
    adv[0] = 0.0
    for t, bad in ((old, -math.inf), (ref, math.nan), (q, math.inf)):
        t[~mask] = bad
    if token_adv:
        adv[~mask] = math.nan
    cut = lambda t: t.to(device)[:, :T] if t.dim() == 2 else t.to(device)  # noqa: E731
    return cut(q), cut(adv), cut(mask), cut(old), cut(ref)


def check(q, adv, mask, old, ref, **kw):
    import grpo_loss_gb300 as G
    out = {k: kw.pop(k) for k in ("loss", "dlogp", "stats", "workspace") if k in kw}
    loss, dlogp, stats = G.policy_loss(q, adv, mask, old, ref, **kw, **out)
    torch.cuda.synchronize()
    z = lambda t: None if t is None else f64(t)  # noqa: E731
    names = {"dual_clip": "dual"}
    want = policy(f64(q), f64(adv), mask.cpu().numpy(), z(old), z(ref), **{names.get(k, k): v for k, v in kw.items()})
    assert abs(loss.item() - want[0]) <= want[3] + 1e-37, (loss.item(), want[0], want[3])
    d = f64(dlogp)
    assert np.all(np.abs(d - want[1]) <= want[4] + 1e-44), np.nanmax(np.abs(d - want[1]) / (want[4] + 1e-44))
    assert not d[mask.cpu().numpy() == 0].any()
    assert np.all(np.abs(f64(stats) - want[2]) <= want[5] + 1e-37), (stats, want[2])
    return loss, dlogp, stats


@pytest.mark.gpu
@pytest.mark.parametrize("ratio", ["token", "sequence"])
@pytest.mark.parametrize("reduce", ["sequence", "token", "constant"])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (5, 7), (70, 31), (4, 33), (9, 1000), (3, 2048), (2, 2049), (5, 8191), (2, 70001)])
def test_sizes(B, T, reduce, ratio):
    for token_adv, pad, dual, beta in ((False, 0, None, 0.04), (True, 3, 3.0, 0.2)):
        x = inputs(B, T, pad=pad, token_adv=token_adv)
        check(*x, ratio=ratio, reduce=reduce, divisor=1000.0 if reduce == "constant" else None, beta=beta,
              dual_clip=dual, clip=(0.2, 0.28))


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(2000, 3), (5000, 17), (700, 129), (33, 4100), (300, 900)])
def test_many_sequences(B, T):
    x = inputs(B, T, seed=1)
    for ratio in ("token", "sequence"):
        check(*x, ratio=ratio, beta=0.01)
        check(*x, ratio=ratio, beta=0.01, reduce="token")


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 32768), (1, 32769), (1024, 32), (1025, 31), (33, 1000), (130, 255), (3, 10001), (8, 24576), (8, 24577), (500, 393)])
def test_on_either_side_of_one_launch(B, T):
    """The most tokens and sequences that one launch takes, and more, with rows on and off
    16-byte boundaries."""
    for pad, token_adv, ratio in ((0, False, "token"), (4, True, "sequence"), (1, False, "sequence")):
        x = inputs(B, T, seed=2, pad=pad, token_adv=token_adv)
        check(*x, ratio=ratio, reduce="token", beta=0.02, dual_clip=2.0)


@pytest.mark.gpu
def test_what_may_be_left_out():
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(6, 300)
    check(q, adv, mask, None, None)                 # no old policy: ratio 1; no reference: no KL term
    check(q, adv, mask, None, None, ratio="sequence", reduce="token")
    check(q, adv, mask, old, None, beta=0.3)
    check(q, adv, mask, old, ref, beta=0.0)         # the KL as a statistic
    check(q, adv, mask, None, ref, beta=0.1)
    check(q, adv, mask, old, ref, clip=(math.inf, math.inf), beta=0.1)     # no bounds
    check(q, adv, mask, old, ref, clip=(1.0, 0.0), beta=0.1, dual_clip=1.0)
    loss, dlogp, stats = check(q, adv, mask, old, ref, beta=0.1)
    only, none, same = G.policy_loss(q, adv, mask, old, ref, beta=0.1, need_dlogp=False)
    assert none is None and torch.equal(only, loss) and torch.equal(same, stats)
    u8 = G.policy_loss(q, adv, mask.to(torch.uint8) * 7, old, ref, beta=0.1)
    assert all(torch.equal(s, t) for s, t in zip(u8, (loss, dlogp, stats)))


@pytest.mark.gpu
def test_empty_masks_and_no_tokens():
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(6, 300)
    for reduce in ("sequence", "token"):
        for ratio in ("token", "sequence"):
            loss, dlogp, stats = check(q, adv, torch.zeros_like(mask), old, ref, reduce=reduce, ratio=ratio, beta=0.1)
            assert loss.item() == 0 and not dlogp.any() and not stats.any()
    for B, T in ((0, 5), (5, 0), (0, 0)):
        z = torch.empty(B, T, device="cuda")
        loss, dlogp, stats = G.policy_loss(z, torch.ones(B, device="cuda"), z.bool(), z, z, beta=0.1)
        assert loss.item() == 0 and dlogp.shape == (B, T) and not stats.any()


@pytest.mark.gpu
def test_on_the_bounds():
    """A ratio of exactly 1 with clip 0 is not clipped; one float step beyond is."""
    import grpo_loss_gb300 as G
    q = torch.full((1, 4), -1.0, device="cuda")
    old = q.clone()
    up, down = torch.nextafter(q[0, 1], q[0, 1] * 0), torch.nextafter(q[0, 2], q[0, 2] * 2)
    q[0, 1], q[0, 2] = up, down
    m = torch.ones(1, 4, dtype=torch.bool, device="cuda")
    _, d, s = G.policy_loss(q, torch.ones(1, device="cuda"), m, old, clip=(0.0, 0.0))
    assert d[0, 0] == -0.25 and d[0, 1] == 0 and d[0, 2] != 0 and s[2] == 0.25 and s[1] == 0
    _, d, s = G.policy_loss(q, -torch.ones(1, device="cuda"), m, old, clip=(0.0, 0.0))
    assert d[0, 0] == 0.25 and d[0, 1] != 0 and d[0, 2] == 0 and s[1] == 0.25 and s[2] == 0
    # around log(1.2): the border lies between two floats
    b = math.log(1.2)
    lo = torch.tensor(b, dtype=F32)
    lo = lo if lo.double() <= b else torch.nextafter(lo, lo * 0)
    q = torch.stack([lo, torch.nextafter(lo, lo * 2)]).cuda()[None]
    _, d, s = G.policy_loss(q, torch.ones(1, device="cuda"), m[:, :2], torch.zeros_like(q), clip=(0.2, 0.2))
    assert d[0, 0] != 0 and d[0, 1] == 0
    # the difference of two floats beside it, which rounds onto it
    big = torch.tensor(4.0) + lo
    for step in (-2, -1, 0, 1, 2):
        v = torch.tensor(big.item() + step * 2.0 ** -21, dtype=F32)
        o = torch.tensor(4.0 + 2.0 ** -22, dtype=F32)
        exact = v.double().item() - o.double().item()
        _, d, s = G.policy_loss(v.cuda().view(1, 1), torch.ones(1, device="cuda"), m[:, :1], o.cuda().view(1, 1))
        assert (d.item() == 0) == (exact > b)


@pytest.mark.gpu
def test_far_ratios_and_nans():
    import grpo_loss_gb300 as G
    q = torch.tensor([[0.0, 0.0, -200.0, 0.0]], device="cuda")
    old = torch.tensor([[-200.0, -1.0, 0.0, -math.inf]], device="cuda")
    m = torch.ones(1, 4, dtype=torch.bool, device="cuda")
    f = lambda A, **kw: G.policy_loss(q, torch.tensor([A], device="cuda"), m, old, **kw)  # noqa: E731
    loss, d, s = f(0.0)                             # no advantage: no loss, whatever the ratio
    assert loss.item() == 0 and not d.any()
    loss, d, s = f(1.0)                             # held at 1.2, or near 0
    assert abs(loss.item() + 3 * 1.2 / 4) < 1e-6 and not d.any()
    loss, d, s = f(-1.0, dual_clip=3.0)
    assert abs(loss.item() - (3.0 + math.e + 0.8 + 3.0) / 4) < 1e-5 and d[0, 1] != 0 and not d[0, [0, 2, 3]].any()
    assert f(-1.0)[0].item() == math.inf
    q[0, 1] = math.nan                              # a valid token's NaN is seen
    loss, d, s = f(1.0)
    assert math.isnan(loss.item()) and math.isnan(d[0, 1].item()) and not d[0, 0].any()


@pytest.mark.gpu
def test_gradient_against_differences():
    """Central differences of the float64 loss."""
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(5, 40, seed=3, fill=1.0)
    m = mask.cpu().numpy()
    rng = np.random.default_rng(0)
    for kw in (dict(beta=0.1), dict(beta=0.1, ratio="sequence", reduce="token"), dict(beta=0.0, reduce="constant", divisor=9.0)):
        _, d, _ = G.policy_loss(q, adv, mask, old, ref, **kw)
        fix = lambda t: np.where(m, f64(t), 0.0)  # noqa: E731
        f = lambda z: policy(z, f64(adv), m, fix(old), fix(ref), **kw)[0]  # noqa: E731
        for _ in range(5):
            v, h = rng.standard_normal(q.shape) * m, 1e-6
            num = (f(fix(q) + h * v) - f(fix(q) - h * v)) / (2 * h)
            # float32's error on the gradient, and the step's second order
            assert abs(num - (f64(d) * v).sum()) <= 1e-5 * np.abs(f64(d) * v).sum() + 1e-9


@pytest.mark.gpu
def test_autograd():
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(5, 400)
    leaf = torch.where(mask, q, torch.zeros_like(q)).requires_grad_(True)
    loss, stats = G.clipped_policy_loss(leaf, adv, mask, old, ref, beta=0.05)
    assert loss.shape == () and not stats.requires_grad
    (3.0 * loss).backward()
    want = G.policy_loss(q, adv, mask, old, ref, beta=0.05)
    assert torch.equal(loss.detach(), want[0][0]) and torch.equal(stats, want[2])
    assert torch.equal(leaf.grad, want[1] * 3.0)
    with torch.no_grad():
        assert torch.equal(G.clipped_policy_loss(leaf, adv, mask, old, ref, beta=0.05)[0], loss)


@pytest.mark.gpu
def test_in_place_and_given_outputs():
    import grpo_loss_gb300 as G
    for ratio in ("token", "sequence"):
        q, adv, mask, old, ref = inputs(4, 5000, token_adv=True, pad=5)
        loss, dlogp, stats = check(q, adv, mask, old, ref, ratio=ratio, beta=0.1)
        for which in range(4):
            x = [t.clone() if t.is_contiguous() else t for t in (q, adv, old, ref)]
            x[which] = x[which].clone()
            to = x[which]
            got = G.policy_loss(x[0], x[1], mask, x[2], x[3], ratio=ratio, beta=0.1, dlogp=to)
            assert got[1] is to and torch.equal(to, dlogp) and torch.equal(got[0], loss) and torch.equal(got[2], stats)
        buf = torch.full((4, 5003), 7.0, device="cuda")
        G.policy_loss(q, adv, mask, old, ref, ratio=ratio, beta=0.1, dlogp=buf[:, 2:5002])
        assert torch.equal(buf[:, 2:5002], dlogp) and (buf[:, :2] == 7).all() and (buf[:, 5002:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(8, 64), (8, 20480), (300, 50)])
def test_repeats_streams_and_graphs(B, T):
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(B, T)
    kw = dict(beta=0.1, reduce="token")
    want = G.policy_loss(q, adv, mask, old, ref, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = G.policy_loss(q, adv, mask, old, ref, stream=side, **kw)
        junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(want, got))
        del junk
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.policy_loss(q, adv, mask, old, ref, loss=outs[0], dlogp=outs[1], stats=outs[2], **kw)
    for _ in range(3):
        for t in outs:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(want, outs))
    # a workspace that held other things
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    got = G.policy_loss(q, adv, mask, old, ref, workspace=ws, **kw)
    assert all(torch.equal(s, t) for s, t in zip(want, got))


@pytest.mark.gpu
def test_tokens_past_two_to_the_31():
    import grpo_loss_gb300 as G
    B, T, n = 2, (1 << 30) + 4096, 4096             # 2.1e9 tokens; the last few are valid
    q = torch.zeros(B, T, device="cuda")
    mask = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    tail = inputs(1, n, fill=1.0)
    q[1, -n:] = tail[0][0]
    mask[1, -n:] = tail[2][0]
    old = torch.zeros_like(q)
    old[1, -n:] = tail[3][0]
    A = torch.ones(B, device="cuda")
    loss, d, stats = G.policy_loss(q, A, mask, old, reduce="token", dlogp=q)
    alone = G.policy_loss(tail[0], A[:1], tail[2], tail[3], reduce="token")
    assert torch.equal(d[1, -n:], alone[1][0]) and not d[0].any() and not d[1, :-n].any()
    assert abs(loss.item() - alone[0].item()) <= 2 ** -22 * abs(loss.item()) and torch.allclose(stats, alone[2], rtol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dW", [(F32, True), (torch.bfloat16, False), (torch.bfloat16, True), (torch.float8_e4m3fn, True)])
def test_the_heads_backward_from_dlogp(dtype, dW):
    """On the policy that drew the tokens, the loss's own dlogp gives the loss's own dH
    and dW; and in general dlogp is the gradient by logp that it is taken for."""
    import grpo_loss_gb300 as G
    B, T, d, V, grp = 8, 160, 128, 700, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    data = F32 if dtype == torch.float8_e4m3fn else dtype
    Hp, W = n(B * T, d).to(data), (0.2 * n(V, d)).to(data)
    Hr = (Hp.float() + 0.2 * n(B * T, d)).to(data)
    ids = torch.randint(0, V, (B * T,), generator=g, device="cuda", dtype=torch.int32)
    mask = (torch.rand(B, T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    mask[3] = 0
    adv = n(B)
    eng = G.GRPOLoss(B, T, d, V, grp, dtype=dtype, compute_dW=dW)
    loss, kl, logp, logp_ref = eng.forward(Hp, Hr, W, ids, mask.view(-1), adv)
    want = eng.backward(Hp, W, ids, mask.view(-1), adv, 0.5).clone()
    want_dW = eng.dW.clone() if dW else None
    mine, dlogp, stats = G.policy_loss(logp.view(B, T), adv, mask, None, logp_ref.view(B, T), beta=eng.problem.beta)
    assert abs(mine.item() - loss.item()) <= 1e-5 * abs(loss.item()) + 1e-7
    assert abs(stats[0].item() - kl.item()) <= 1e-5 * kl.item()
    dlogp[mask == 0] = math.nan                     # not looked at
    got = eng.backward(Hp, W, ids, mask.view(-1), None, 0.5, dlogp=dlogp.view(-1))
    eng.check()
    # the coefficients agree to float32, the bf16 dZ that is made of them to a rounding of a few
    rel = lambda a, b: ((a.float() - b.float()).norm() / b.float().norm()).item()  # noqa: E731
    assert rel(got, want) <= 2.0 ** -8 and not got.view(B, T, d)[3].any()
    if dW:
        assert rel(eng.dW, want_dW) <= 2.0 ** -8
    twice = eng.backward(Hp, W, ids, mask.view(-1), None, 1.0, dlogp=dlogp.view(-1) * 0.5)
    assert torch.equal(twice, got)                  # a power of two


def test_second_derivatives_are_refused(monkeypatch):
    """Gradients that come from kernels have no graph of their own. (The kernel is stood
    in for by a formula.)"""
    import grpo_loss_gb300 as G

    def loss(logp, adv, mask, need_dlogp=True, **kw):
        return logp.pow(2).sum().reshape(1), 2 * logp, torch.zeros(4)
    monkeypatch.setattr(G, "policy_loss", loss)
    q = torch.randn(3, 4, dtype=torch.float64, requires_grad=True)
    (g,) = torch.autograd.grad(G.clipped_policy_loss(q, None, None)[0], q)
    assert torch.allclose(g, 2 * q)
    (g,) = torch.autograd.grad(3 * G.clipped_policy_loss(q, None, None)[0], q, create_graph=True)
    assert torch.allclose(g, 6 * q)
    with pytest.raises(RuntimeError, match="once differentiable"):
        torch.autograd.grad(g.pow(2).sum() + q.sum(), q)


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (python -m grpo_loss_gb300.build)")
    return L.lib()


def problem(**kw):
    p = L.PolicyProblem(4, 100, 0, 0, 0, 0, 0, 0, 0.2, 0.2, 0.0, 0.1, 0.0, 0, 0, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 1), (dict(seq_len=-1), 1), (dict(ld_logp=99), 1), (dict(ld_old=1), 1), (dict(ld_ref=-1), 1),
    (dict(ld_adv=99), 1), (dict(ld_mask=99), 1), (dict(ld_dlogp=99), 1), (dict(clip_low=-0.1), 1),
    (dict(clip_high=-0.1), 1), (dict(clip_low=math.nan), 1), (dict(clip_high=math.nan), 1), (dict(dual_clip=0.5), 1),
    (dict(dual_clip=-1.0), 1), (dict(dual_clip=math.nan), 1), (dict(beta=math.inf), 1), (dict(beta=math.nan), 1),
    (dict(ratio=2), 1), (dict(ratio=-1), 1), (dict(reduce=3), 1), (dict(reduce=-1), 1), (dict(token_adv=2), 1),
    (dict(reduce=2), 1), (dict(reduce=2, divisor=-1.0), 1), (dict(reduce=2, divisor=math.inf), 1),
    (dict(num_seqs=1 << 31), 2), (dict(seq_len=1 << 31), 2), (dict(num_seqs=1 << 30, seq_len=1 << 30), 2)])
def test_refuses_bad_problems_on_the_host(lib, kw, status):
    at, size = ctypes.c_void_p(256), ctypes.c_size_t(0)
    r = ctypes.byref(problem(**kw))
    assert lib.grpo_policy_loss_workspace_size(r, ctypes.byref(size)) == status
    assert lib.grpo_policy_loss(r, *[at] * 9, 1 << 40, None) == status


def test_refuses_bad_pointers_on_the_host(lib):
    r, at, odd = ctypes.byref(problem()), ctypes.c_void_p(256), ctypes.c_void_p(257)
    put = lambda i, v: [v if j == i else at for j in range(8)]  # noqa: E731
    assert lib.grpo_policy_loss(None, *[at] * 9, 1 << 40, None) == 1
    for i in (0, 3, 4, 5):                          # logp, adv, mask, loss
        assert lib.grpo_policy_loss(r, *put(i, None), at, 1 << 40, None) == 1
    for i in (0, 1, 2, 3, 5, 6, 7):                 # all but the mask
        assert lib.grpo_policy_loss(r, *put(i, odd), at, 1 << 40, None) == 2


def test_refuses_bad_dlogp_calls_on_the_host(lib):
    p = L.make_problem(8, 64, 256, 1024, 4)
    at = ctypes.c_void_p(256)
    r = ctypes.byref(p)
    put = lambda n, i: [None if j == i else at for j in range(n)]  # noqa: E731
    for i in range(6):
        assert lib.grpo_loss_bwd_dlogp(r, *put(6, i), 1.0, at, None, at, 1 << 50, None) == 1
    assert lib.grpo_loss_bwd_dlogp(r, *[at] * 6, math.nan, at, None, at, 1 << 50, None) == 1
    assert lib.grpo_loss_bwd_dlogp(r, *[at] * 6, 1.0, at, at, at, 1 << 50, None) == 1     # dW without compute_dW
    assert lib.grpo_loss_bwd_dlogp_e4m3(r, *[at] * 8, 1.0, at, None, at, 1 << 50, None) == 1
    p.dtype = L.GRPO_E4M3
    assert lib.grpo_loss_bwd_dlogp(r, *[at] * 6, 1.0, at, None, at, 1 << 50, None) == 1
    for i in range(8):
        assert lib.grpo_loss_bwd_dlogp_e4m3(r, *put(8, i), 1.0, at, None, at, 1 << 50, None) == 1


def test_refuses_wrong_arguments(monkeypatch):
    import grpo_loss_gb300 as G
    monkeypatch.setattr(L, "_device_of", lambda t, name: t.device)
    q, adv, mask, old, ref = inputs(3, 8, device="cpu")
    for bad, word in ((dict(logp=q[0]), "2-D"), (dict(logp=q.double()), "float32"), (dict(mask=mask.int()), "bool or uint8"),
                      (dict(mask=mask[:, :5]), "shape"), (dict(advantages=adv[:2]), "elements"),
                      (dict(advantages=torch.zeros(3, 7)), "shape"), (dict(logp_old=old.t().contiguous().t()), "contiguous"),
                      (dict(clip=0.2), "clip"), (dict(clip=(0.1, 0.2, 0.3)), "clip"), (dict(ratio="both"), "ratio"), (dict(reduce="sum"), "reduce"), (dict(reduce="constant"), "divisor"),
                      (dict(divisor=3.0), "divisor"), (dict(dlogp=torch.zeros(1, 8).expand(3, 8)), "row stride"),
                      (dict(loss=torch.zeros(2)), "elements"), (dict(stats=torch.zeros(3)), "elements")):
        with pytest.raises(ValueError, match=word):
            G.policy_loss(**{"logp": q, "advantages": adv, "mask": mask, **bad})


@pytest.mark.gpu
def test_refuses_a_short_workspace_and_the_host():
    import grpo_loss_gb300 as G
    q, adv, mask, old, ref = inputs(300, 800)       # (few tokens need none)
    with pytest.raises(L.GrpoError) as e:
        G.policy_loss(q, adv, mask, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(ValueError, match="CUDA"):
        G.policy_loss(q.cpu(), adv, mask)
