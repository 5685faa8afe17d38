"""The operators of a rollout's further updates as one update uses them: a block with norms
on both sides, the head's log-probabilities, the clipped loss, its gradient back through
the head and the norms, the gradients' norm, and the step that takes the factor. Against
the same update in float64, and captured into a graph."""
import math

import numpy as np
import pytest
import torch

from tests.operator_reference import f64
from tests.update_reference import policy, residual_norm_bwd, residual_norm_fwd

B, T, D, V, GROUP = 8, 48, 64, 320, 4
KW = dict(clip=(0.2, 0.28), beta=0.05)


def tensors(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    N = B * T
    p = dict(weight=1 + 0.2 * n(D), post=0.5 + 0.2 * n(D), gate=0.5 + 0.3 * n(1, D), head=0.3 * n(V, D))
    x, res = n(N, D), n(N, D)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    mask = torch.rand(B, T, generator=g, device="cuda") < 0.9
    mask[2] = False
    return p, x, res, ids, mask, n(B), n(B, T)


class Update:
    """One update, every buffer its own; run() leaves the new parameters in p."""

    def __init__(self, seed=0):
        import grpo_loss_gb300 as G
        self.G = G
        self.p, self.x, self.res, self.ids, self.mask, self.adv, self.noise = tensors(seed)
        self.u8 = self.mask.to(torch.uint8).view(-1)
        self.eng = G.GRPOLoss(B, T, D, V, GROUP, dtype=torch.float32, compute_dW=True, ref_logp_given=True)
        self.eng.logp_ref.zero_()
        self.names = ["weight", "post", "gate", "head"]
        self.opt = G.AdamW([self.p[k] for k in self.names], lr=1e-2, weight_decay=0.0)
        y = self.forward()
        logp = self.logp(y).clone().view(B, T)
        self.old = torch.where(self.mask, logp + 0.1 * self.noise, logp)    # another policy drew the tokens
        self.ref = torch.where(self.mask, logp - 0.1 * self.noise.flip(0), logp)

    def forward(self):
        self.h, y, _, self.rstd, _, self.prstd = self.G.residual_norm_fwd(
            self.x, self.res, self.p["weight"], post_weight=self.p["post"], gate=self.p["gate"], scale=0.5, rms=True)
        return y

    def logp(self, y):
        return self.eng.forward(y, None, self.p["head"], self.ids, self.u8, self.adv, logp_ref=self.eng.logp_ref)[2]

    def run(self):
        G, p = self.G, self.p
        y = self.forward()
        self.now = self.logp(y).view(B, T)
        self.loss, self.dlogp, self.stats = G.policy_loss(self.now, self.adv, self.mask, self.old, self.ref, **KW)
        self.dy = self.eng.backward(y, p["head"], self.ids, self.u8, None, dlogp=self.dlogp.view(-1))
        _, _, dw, _, dpw, _, dgate = G.residual_norm_bwd(
            self.dy, None, self.h, p["weight"], None, self.rstd, x=self.x, post_weight=p["post"], post_rstd=self.prstd,
            gate=p["gate"], scale=0.5, rms=True)
        self.grads = [dw, dpw, dgate, self.eng.dW]
        self.norm, self.factor = G.grad_norm(self.grads, max_norm=0.5)
        self.opt.step(self.grads, factor=self.factor, step=1)


@pytest.mark.gpu
def test_an_update_against_float64():
    u = Update()
    p0 = {k: f64(t) for k, t in u.p.items()}
    u.run()
    u.eng.check()
    torch.cuda.synchronize()
    m = u.mask.cpu().numpy()
    val, _ = residual_norm_fwd(f64(u.x), f64(u.res), p0["weight"], None, p0["post"], None, p0["gate"], 0.5, 1e-5, True)
    z = val["y"] @ p0["head"].T
    z -= z.max(1, keepdims=True)
    lse = np.log(np.exp(z).sum(1, keepdims=True))
    ids = u.ids.cpu().numpy()
    logp = (z - lse)[np.arange(B * T), ids].reshape(B, T)
    # the head multiplies in bf16: its products are off by 2^-8 of their terms' sizes at most, some 0.01 here
    assert np.abs(f64(u.now) - logp)[m].max() < 0.05
    # from the head's own log-probabilities on, float32
    loss, dlogp, stats, e_loss, e_dlogp, e_stats = policy(f64(u.now), f64(u.adv), m, f64(u.old), f64(u.ref), **KW)
    assert abs(u.loss.item() - loss) <= e_loss and np.all(np.abs(f64(u.dlogp) - dlogp) <= e_dlogp + 1e-44)
    assert stats[1] + stats[2] > 0.01               # some tokens are clipped, or this tests little
    soft = np.exp(z - lse)
    dz = -dlogp.reshape(-1, 1) * soft
    dz[np.arange(B * T), ids] += dlogp.ravel()
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    # dZ, y and W are bf16 in the head's products: each rounding 2^-9 rms of its operand, and the logits' own error
    assert rel(f64(u.dy), dz @ p0["head"]) < 0.03 and rel(f64(u.eng.dW), dz.T @ val["y"]) < 0.03
    back, err = residual_norm_bwd(f64(u.dy), None, f64(u.h), p0["weight"], None, f64(u.rstd), f64(u.x), p0["post"], None, None,
                                  f64(u.prstd), p0["gate"], 0.5, True)
    for got, k in zip(u.grads, ("dweight", "dpost_weight", "dgate")):
        assert np.all(np.abs(f64(got) - back[k].reshape(got.shape)) <= err[k].reshape(got.shape) * 1.01 + 2.0 ** -24 * np.abs(f64(got)))
    norm = math.sqrt(sum((f64(g) ** 2).sum() for g in u.grads))
    assert abs(u.norm.item() - norm) <= 1e-5 * norm and abs(u.factor.item() - min(1, 0.5 / (norm + 1e-6))) <= 1e-5
    # a first step of AdamW moves every parameter by lr g / (|g| + eps / sqrt(1 - b2)) or so
    for k, g in zip(u.names, u.grads):
        g64 = f64(g) * f64(u.factor)[0]
        want = p0[k] - 1e-2 * g64 / (np.abs(g64) + 1e-8)
        assert np.abs(f64(u.p[k]) - want.reshape(p0[k].shape)).max() <= 1e-5


@pytest.mark.gpu
def test_an_update_is_the_same_on_a_side_stream_and_in_a_graph():
    want = Update(1)
    want.run()
    torch.cuda.synchronize()
    keep = [t.clone() for t in [want.loss, want.dlogp, want.stats, want.norm, want.factor] + [want.p[k] for k in want.names]]
    side = Update(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side.run()
    s.synchronize()
    graphed = Update(1)
    graphed.run()                                   # (warm; then from the same state again)
    state = Update(1)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        state.run()
    g.replay()
    torch.cuda.synchronize()
    for u in (side, graphed, state):
        got = [u.loss, u.dlogp, u.stats, u.norm, u.factor] + [u.p[k] for k in u.names]
        for a, b in zip(got, keep):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_graphs_with_workspaces_of_their_own_overlap():
    """Two captured calls on two streams at once, each with its own workspace."""
    import grpo_loss_gb300 as G
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    made = []
    for k in range(2):
        q, o = n(64, 5000) - 3, n(64, 5000) * 0.1
        o = q + o
        m, A = torch.rand(64, 5000, generator=g, device="cuda") < 0.8, n(64)
        x, dy, w = n(4000, 512), n(4000, 512), 1 + 0.1 * n(512)
        h, y, _, r, _, pr = G.residual_norm_fwd(x, dy, w, post_weight=w, rms=True)
        grads = [n(3_000_001), n(70_000)]
        out = [torch.empty_like(t) for t in grads]
        f = lambda q=q, o=o, m=m, A=A, x=x, dy=dy, w=w, h=h, r=r, pr=pr, grads=grads, out=out: (  # noqa: E731
            *G.policy_loss(q, A, m, o, reduce="token"),
            *[t for t in G.residual_norm_bwd(dy, x, h, w, None, r, x=x, post_weight=w, post_rstd=pr, rms=True) if t is not None],
            G.clip_grad_norm(grads, 1.0, out=out), *out)
        want = [t.clone() for t in f()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = f()
        made.append((graph, outs, want, torch.cuda.Stream(), f))   # (f holds the tensors that the graph reads)
    for _ in range(5):
        for graph, _, _, s, _ in made:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _, _ in made:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.gpu
def test_the_example_runs_with_several_updates_a_rollout():
    from tests.test_examples import load
    rewards, greedy = load().run(2, seed=0, quiet=True, updates=3)
    assert len(rewards) == 2 and all(0.0 <= r <= 1.0 for r in rewards) and 0.0 <= greedy <= 1.0
