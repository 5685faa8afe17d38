"""GRPO iterations of a small recurrent policy, start to end on the library: each
token is drawn with ``sample`` from logits behind ``layernorm_fwd``, the loss and
its gradients with respect to the hidden states and the head are ``GRPOLoss``'s,
the norm's gradients ``layer_norm``'s, and one ``AdamW`` call with 8-bit states
and float32 masters updates every tensor.

With more than one update for each rollout, the policy has moved away from the one that
drew the tokens: the later ones take ``policy_loss`` of the ratio to the drawn
log-probabilities, whose gradient goes back through the head, and clip the gradients by
their norm.

The reward of a completion is the share of its tokens that lie in the first
eighth of the vocabulary; its mean starts near 1/8 and is over 0.9 after 25 iterations.

    python examples/grpo_iterations.py [iterations [updates for each]]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import grpo_loss_gb300 as G  # noqa: E402

VOCAB, HIDDEN, LENGTH, GROUPS, GROUP = 1024, 256, 16, 4, 64
END = VOCAB - 1  # a completion ends behind this token
BF16 = torch.bfloat16


class Policy:
    """h_t = embed[token_t] + tanh(h_(t-1) mix), x_t = layer_norm(h_t), logits = x_t head^T."""

    def __init__(self, seed: int, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).to(BF16).requires_grad_(True)

        self.embed = normal(VOCAB, HIDDEN, std=1.0)
        self.mix = normal(HIDDEN, HIDDEN, std=HIDDEN ** -0.5)
        self.weight = torch.ones(HIDDEN, dtype=BF16, device=device, requires_grad=True)
        self.bias = torch.zeros(HIDDEN, dtype=BF16, device=device, requires_grad=True)
        self.head = normal(VOCAB, HIDDEN, std=HIDDEN ** -0.5)
        self.params = [self.embed, self.mix, self.weight, self.bias, self.head]

    def advance(self, h, tokens):
        return self.embed[tokens.long()] + torch.tanh(h @ self.mix)

    @torch.no_grad()
    def generate(self, prompts, temperature=None, generator=None, **cuts):
        """(tokens int32 [B, LENGTH], their mask, log-probabilities) behind one prompt token each."""
        B, dev = prompts.shape[0], prompts.device
        ids = torch.empty(B, LENGTH, dtype=torch.int32, device=dev)
        mask, logp = torch.empty(B, LENGTH, dtype=torch.uint8, device=dev), torch.empty(B, LENGTH, device=dev)
        T = None if temperature is None else torch.full((B,), temperature, device=dev)
        h, last, live = torch.zeros(B, HIDDEN, dtype=BF16, device=dev), prompts, torch.ones(B, dtype=torch.uint8, device=dev)
        for t in range(LENGTH):
            h = self.advance(h, last)
            x, _, _ = G.layernorm_fwd(h, self.weight.detach(), self.bias.detach())
            u = torch.rand(B, generator=generator, device=dev)
            last, lp = G.sample(x @ self.head.T, u, temperature=T, **cuts)
            ids[:, t], mask[:, t], logp[:, t] = last, live, lp
            live = live * (last != END)  # the end token itself counts
        return ids, mask, logp

    def hidden(self, prompts, ids):
        """x_t for every position of given completions, [B * LENGTH, HIDDEN]."""
        h = torch.zeros(prompts.shape[0], HIDDEN, dtype=BF16, device=prompts.device)
        hs = []
        for t in range(LENGTH):
            h = self.advance(h, prompts if t == 0 else ids[:, t - 1])
            hs.append(h)
        return G.layer_norm(torch.stack(hs, 1).view(-1, HIDDEN), self.weight, self.bias)


def run(iterations: int = 40, seed: int = 0, state_bits: int = 8, quiet: bool = False, updates: int = 1):
    """Mean reward of every iteration, and of a greedy completion at the end."""
    B = GROUPS * GROUP
    policy, first = Policy(seed), Policy(seed)  # `first` stays: the reference model
    loss_of = G.GRPOLoss(B, LENGTH, HIDDEN, VOCAB, GROUP, compute_dW=True, ref_logp_given=True)
    ref_of = G.GRPOLoss(B, LENGTH, HIDDEN, VOCAB, GROUP)
    opt = G.AdamW(policy.params, lr=3e-2, weight_decay=[0.0] * 4 + [0.01], state_bits=state_bits, master=True)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rewards = []
    for it in range(iterations):
        prompts = torch.randint(VOCAB, (GROUPS,), generator=g, device="cuda").int().repeat_interleave(GROUP)
        ids, mask, logp = policy.generate(prompts, generator=g)
        reward = ((ids < VOCAB // 8) * mask).sum(1) / mask.sum(1)
        adv = loss_of.advantages(reward)
        flat, live = ids.view(-1), mask.view(-1)
        with torch.no_grad():
            x_ref = first.hidden(prompts, ids)
            logp_ref = ref_of.forward(x_ref, x_ref, first.head.detach(), flat, live, adv)[2]
        clipped = norm = None
        for update in range(updates):
            x = policy.hidden(prompts, ids)
            loss, kl, now, _ = loss_of.forward(x.detach(), None, policy.head.detach(), flat, live, adv, logp_ref=logp_ref)
            if update == 0:
                logp_now, dlogp = now.clone(), None
            else:
                loss, dlogp, clipped = G.policy_loss(now.view(B, LENGTH), adv, mask, logp, logp_ref.view(B, LENGTH),
                                                     clip=(0.2, 0.28), beta=loss_of.problem.beta)
                dlogp = dlogp.view(-1)
            x.backward(loss_of.backward(x.detach(), policy.head.detach(), flat, live, adv, dlogp=dlogp))
            grads, factor = [p.grad for p in policy.params[:-1]] + [loss_of.dW], None
            if updates > 1:
                norm, factor = G.grad_norm(grads, max_norm=1.0)
            opt.step(grads, factor=factor)
            for p in policy.params:
                p.grad = None
        rewards.append(reward.mean().item())
        if not quiet:
            off = ((logp - logp_now.view_as(logp)).abs() * mask).max().item()
            print("iteration %2d  reward %.3f  loss %+.4f  kl %.4f  |logp drawn - logp of the loss| <= %.4f" % (
                it, rewards[-1], loss.item(), kl.item(), off))
            if clipped is not None:
                print("              clipped %.3f low, %.3f high  gradient norm %.3f" % (
                    clipped[1].item(), clipped[2].item(), norm.item()))
    loss_of.check()
    ids, mask, _ = policy.generate(prompts, temperature=0.0)
    last = (((ids < VOCAB // 8) * mask).sum(1) / mask.sum(1)).mean().item()
    if not quiet:
        print("greedy reward %.3f" % last)
    return rewards, last


if __name__ == "__main__":
    run(int(sys.argv[1]) if len(sys.argv) > 1 else 40, updates=int(sys.argv[2]) if len(sys.argv) > 2 else 1)
