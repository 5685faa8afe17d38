"""Cases of the operators of a GRPO update beyond the first of a rollout, with
their plain forms.

Such an update takes, next to the fused loss head: the clipped policy loss with
its KL term and the gradient by every token's log-probability; the norms behind
and before a block with the block's gate and residual scale, forward and
backward; and the global norm of all gradients with the clipping by it. The
cases below are those operators at this repository's head shapes and at generic
odd ones.

``run`` computes the plain form (elementary torch operations) while ``own`` is
False and calls the package's kernels while it is True.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5                                          # of the norms
CLIP_EPS = 1e-6                                     # beside the gradients' norm


def listed():
    return [
        # the tokens of eight short completions: the latency of a loss
        dict(name="policy_short", op="policy", B=8, T=64, fill=0.5, pad=0, ratio="token", reduce="sequence",
             beta=0.04, dual=0.0, token_adv=False, old=True),
        # 8 generations of 20480 tokens, the second update of a rollout
        dict(name="policy_20k", op="policy", B=8, T=20480, fill=1.0, pad=0, ratio="token", reduce="sequence",
             beta=0.04, dual=0.0, token_adv=False, old=True),
        # a large ragged batch, one weight for every token of it, an advantage for each token
        dict(name="policy_tokens", op="policy", B=509, T=8191, fill=0.5, pad=0, ratio="token", reduce="token",
             beta=0.001, dual=3.0, token_adv=True, old=True),
        # long completions whose ratio is one for the whole sequence, no reference model, rows cut from wider ones
        dict(name="policy_sequences", op="policy", B=256, T=32768, fill=0.25, pad=4, ratio="sequence",
             reduce="sequence", beta=0.0, dual=0.0, token_adv=False, old=True),
        # one token being generated, norms on both sides of its block
        dict(name="block_fwd_1", op="block_fwd", rows=1, d=4096, dtype="bf16", params="bf16", rms=True, bias=False,
             post=True, gate="none", seqs=1, scale=1.0),
        # a training batch of 8 x 20480 tokens through the same norms
        dict(name="block_fwd_batch", op="block_fwd", rows=163840, d=4096, dtype="bf16", params="bf16", rms=True,
             bias=False, post=True, gate="none", seqs=1, scale=1.0),
        # float32 rows of 7 sequences, each gated by what conditions it
        dict(name="block_fwd_gated_f32", op="block_fwd", rows=7 * 1877, d=1536, dtype="f32", params="f32", rms=False,
             bias=True, post=False, gate="seq", seqs=7, scale=1.0),
        # gradients of a ragged batch with a learned gate for every channel
        dict(name="block_bwd_channel", op="block_bwd", rows=13081, d=2880, dtype="bf16", params="f32", rms=False,
             bias=True, post=False, gate="channel", seqs=1, scale=0.7),
        # gradients over the whole training batch
        dict(name="block_bwd_batch", op="block_bwd", rows=163840, d=4096, dtype="bf16", params="bf16", rms=True,
             bias=False, post=True, gate="none", seqs=1, scale=1.0),
        # the gradients of a handful of norm weights and biases: launch latency
        dict(name="norm_small", op="norm", shapes="4096,4096,1536,1536,2880,257", dtype="f32", packed=False,
             norm=2.0),
        # the low-rank factors of a fine-tune in one packed buffer, clipped into another
        dict(name="clip_factors", op="clip", shapes=",".join(["16x4096", "14336x16", "8x1536", "1027x8", "257"] * 12),
             dtype="bf16", packed=True, norm=2.0, max_norm=1.0),
        # a full fine-tune's float32 dW and the gradients of its last norm
        dict(name="clip_head", op="clip", shapes="151936x1536,1536", dtype="f32", packed=False, norm=2.0,
             max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "policy", "block_fwd", "block_bwd", "norm", "clip"])
    if op == "policy":
        T = _log_int(rng, 1, 110000)
        B = _log_int(rng, 1, max(1, min(4096, 256 * 32768 // T)))
        return dict(op=op, B=B, T=T, fill=rng.choice([1.0, 0.5, 0.0]), pad=rng.choice([0, 0, 1, 4]),
                    ratio=rng.choice(["token", "token", "sequence"]),
                    reduce=rng.choice(["sequence", "token", "constant"]),
                    beta=rng.choice([0.0, 0.04, round(rng.uniform(0.001, 0.2), 4)]),
                    dual=rng.choice([0.0, 3.0]), token_adv=rng.random() < 0.4, old=rng.random() < 0.85)
    if op in ("block_fwd", "block_bwd"):
        d = rng.choice([4096, 1536, 2880, 512, _log_int(rng, 64, 16384)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 163840 * 4096 // d // (2 if dtype == "f32" else 1)
        gate = rng.choice(["none", "none", "channel", "seq", "element"])
        if gate == "element":
            most = most * 2 // 3
        rows, seqs = _log_int(rng, 1, min(163840, most)), 1
        if gate == "seq":
            seqs = _log_int(rng, 1, min(rows, 512))
            rows = rows // seqs * seqs
        rms = rng.random() < 0.5
        return dict(op=op, rows=rows, d=d, dtype=dtype, params=rng.choice(["f32", dtype]), rms=rms,
                    bias=(not rms) and rng.random() < 0.7, post=rng.random() < 0.5, gate=gate, seqs=seqs,
                    scale=rng.choice([1.0, round(rng.uniform(0.1, 1.0), 3)]))
    n = rng.choice([rng.randint(1, 24), _log_int(rng, 1, 400)])
    shapes, room = [], 200_000_000
    for _ in range(n):
        size = min(_log_int(rng, 1, 30_000_000), room // 8 + 1)
        room -= size
        shapes.append(str(size))
    case = dict(op=op, shapes=",".join(shapes), dtype=rng.choice(["bf16", "f32", "mixed"]),
                packed=rng.random() < 0.5, norm=rng.choice([2.0, 2.0, math.inf]))
    if op == "clip":
        case["max_norm"] = rng.choice([1.0, round(rng.uniform(0.01, 5.0), 3)])
    return case


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _kinds(case):
    """The type of each gradient: every third is float32 in a mixed list."""
    n = len(_shapes(case))
    return [("f32" if i % 3 == 2 else "bf16") if case["dtype"] == "mixed" else case["dtype"] for i in range(n)]


def work(case):
    if case["op"] == "policy":
        n = case["B"] * case["T"]
        valid = n * (1 + case["fill"]) / 2         # of a masked token the mask alone is read
        reads = 4 + 4 * case["old"] + 4 * (case["beta"] > 0) + 4 * case["token_adv"]
        return {"bytes": 5 * n + reads * valid, "flops": 40 * valid}
    if case["op"] in ("block_fwd", "block_bwd"):
        R, d, es, ps = case["rows"], case["d"], SIZE[case["dtype"]], SIZE[case["params"]]
        vecs = (1 + case["bias"]) * (1 + case["post"])
        gate = {"none": 0, "channel": d * ps, "seq": case["seqs"] * d * es, "element": R * d * es}[case["gate"]]
        stats = 4 * R * (1 if case["rms"] else 2) * (1 + case["post"])
        if case["op"] == "block_fwd":
            return {"bytes": 4 * R * d * es + vecs * d * ps + gate + stats, "flops": (10 + 8 * case["post"]) * R * d}
        inner = case["post"] or case["gate"] != "none"      # the block's output is read again
        alone = not inner and case["scale"] == 1.0          # the block's gradient is the stream's
        dgate = {"none": 0, "channel": 4 * d, "seq": 4 * case["seqs"] * d, "element": R * d * es}[case["gate"]]
        return {"bytes": (5 + inner - alone) * R * d * es + (1 + case["post"]) * d * ps + gate + dgate +
                4 * vecs * d + stats, "flops": (16 + 16 * case["post"]) * R * d}
    size = sum(math.prod(s) * SIZE[k] for s, k in zip(_shapes(case), _kinds(case)))
    n = sum(math.prod(s) for s in _shapes(case))
    return {"bytes": size * (2 if case["op"] == "clip" else 1) + 4, "flops": (3 if case["op"] == "clip" else 2) * n}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dtype).mul_(std)

    def uniform(n, lo=0.0, hi=1.0):
        return torch.rand(n, generator=gen, device=DEV).mul_(hi - lo).add_(lo)

    if case["op"] == "policy":
        return _prepare_policy(case, normal, uniform)
    if case["op"] in ("block_fwd", "block_bwd"):
        return _prepare_block(case, normal, uniform)
    # gradients: a size of its own for every tensor, rare rows smaller than others
    s = {"case": case, "grads": [], "out": [], "flat": {}}
    shapes, kinds = _shapes(case), _kinds(case)
    flat = {}
    if case["packed"]:                              # views of one buffer a type, one behind the other
        for kind in sorted(set(kinds)):
            n = sum(math.prod(sh) for sh, k in zip(shapes, kinds) if k == kind)
            flat[kind] = [torch.empty(n, device=DEV, dtype=DTYPES[kind]) for _ in range(2)] + [0]
            s["flat"][kind] = flat[kind][1]
    for shape, kind in zip(shapes, kinds):
        g = normal(shape)
        g.mul_(normal((shape[0],) + (1,) * (len(shape) - 1)).mul_(1.5).exp_().mul_(1e-4))
        if case["packed"]:
            at, n = flat[kind][2], math.prod(shape)
            view, to = (t[at:at + n].view(shape) for t in flat[kind][:2])
            view.copy_(g)
            flat[kind][2] += n
            s["grads"].append(view)
            s["out"].append(to)
        else:
            s["grads"].append(g.to(DTYPES[kind]))
            s["out"].append(torch.empty_like(s["grads"][-1]))
    return s


def _prepare_policy(case, normal, uniform):
    B, T = case["B"], case["T"]
    wide = T + case["pad"]                          # rows may be cut from wider ones
    lengths = (uniform(B, case["fill"], 1.0) * T).round()
    at = torch.arange(wide, device=DEV)
    mask = at[None, :] < lengths[:, None]
    # log-probabilities of drawn tokens: mostly near 0, some far below
    logp_old = normal((B, wide), 1.5).sub_(1.0).exp_().neg_()
    # an update or two later: a shift for each sequence and one for each token
    shift = normal((B, wide), 0.15).add_(normal((B, 1), 0.03)).mul_(logp_old.abs().sqrt())
    logp = (logp_old + shift).clamp_(max=0.0)
    logp_ref = normal((B, wide), 0.2).mul_(logp_old.abs().sqrt()).add_(logp).clamp_(max=0.0)
    # the padding holds what a generator leaves there
    logp_old.masked_fill_(~mask, -math.inf)
    adv = normal((B, wide)) if case["token_adv"] else normal((B,))
    if not case["token_adv"]:
        adv.mul_((uniform(B) < 0.9).float())        # prompts whose answers were all alike teach nothing
    return {"case": case, "logp": logp[:, :T], "mask": mask[:, :T], "adv": adv[:, :T] if case["token_adv"] else adv,
            "old": logp_old[:, :T] if case["old"] else None, "ref": logp_ref[:, :T] if case["beta"] > 0 else None,
            "divisor": float(B * T)}


def _prepare_block(case, normal, uniform):
    R, d, dt, dp = case["rows"], case["d"], DTYPES[case["dtype"]], DTYPES[case["params"]]
    loud = torch.where(uniform(d) < 0.01, 12.0, 1.0)
    s = {"case": case, "residual": normal((R, d), 1.0, dt).mul_(loud.to(dt)).add_(normal((d,), 0.3).to(dt)),
         "x": normal((R, d), 0.6, dt).add_(normal((d,), 0.1).to(dt)),
         "weight": normal((d,), 0.1).add_(1.0).to(dp), "bias": normal((d,), 0.1).to(dp) if case["bias"] else None,
         "post_weight": normal((d,), 0.1).add_(0.5).to(dp) if case["post"] else None,
         "post_bias": normal((d,), 0.1).to(dp) if case["post"] and case["bias"] else None, "gate": None}
    if case["gate"] == "channel":
        s["gate"] = normal((1, d), 0.1).add_(0.3).to(dp)
    elif case["gate"] == "seq":
        s["gate"] = normal((case["seqs"], d), 0.5, dt)
    elif case["gate"] == "element":
        s["gate"] = normal((R, d), 1.0, dt).sigmoid_()
    if case["op"] == "block_fwd":
        return s
    # what the forward pass kept
    h, stats = torch.empty_like(s["residual"]), [[], [], [], []]
    for at in range(0, R, 8192):
        x = s["x"][at:at + 8192].double()
        p = x
        if case["post"]:
            m, r = _stats64(x, case["rms"])
            stats[2].append(m[:, 0].float())
            stats[3].append(r[:, 0].float())
            p = (x - m) * r * s["post_weight"].double()
            p = p + s["post_bias"].double() if s["post_bias"] is not None else p
        if s["gate"] is not None:
            per = R // len(s["gate"])
            p = p * s["gate"][torch.arange(at, at + len(p), device=DEV) // per].double()
        z = s["residual"][at:at + 8192].double() + case["scale"] * p
        m, r = _stats64(z, case["rms"])
        stats[0].append(m[:, 0].float())
        stats[1].append(r[:, 0].float())
        h[at:at + 8192] = z.to(dt)
    del s["residual"]
    s["h"] = h
    keys = ("mean", "rstd", "post_mean", "post_rstd")
    s.update({k: torch.cat(v) if v and not (case["rms"] and "mean" in k) else None for k, v in zip(keys, stats)})
    s["dy"] = normal((R, d), 1e-3, dt)
    s["dh"] = normal((R, d), 1e-3, dt)
    live = (uniform(R) < 0.9).to(dt)[:, None]      # masked tokens have no gradient
    s["dy"].mul_(live)
    s["dh"].mul_(live)
    return s


def _stats64(x, rms):
    m = x.mean(1, keepdim=True) * (0.0 if rms else 1.0)
    return m, (((x - m) ** 2).mean(1, keepdim=True) + EPS).rsqrt()


# --------------------------------------------------------------- one pass
CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "policy":
        return _plain_policy(s, case)
    if case["op"] == "block_fwd":
        return _plain_block_fwd(s, case)
    if case["op"] == "block_bwd":
        return _plain_block_bwd(s, case)
    return _plain_clip(s, case)


def _run_own(s, case):
    import grpo_loss_gb300 as G
    if case["op"] == "policy":
        loss, dlogp, stats = G.policy_loss(s["logp"], s["adv"], s["mask"], logp_old=s["old"], logp_ref=s["ref"],
                                           clip=(CLIP_LOW, CLIP_HIGH), dual_clip=case["dual"] or None,
                                           beta=case["beta"], ratio=case["ratio"], reduce=case["reduce"],
                                           divisor=s["divisor"] if case["reduce"] == "constant" else None)
        return {"loss": loss, "dlogp": dlogp, "stats": stats}
    if case["op"] == "block_fwd":
        h, y, mean, rstd, post_mean, post_rstd = G.residual_norm_fwd(
            s["x"], s["residual"], s["weight"], s["bias"], post_weight=s["post_weight"], post_bias=s["post_bias"],
            gate=s["gate"], scale=case["scale"], eps=EPS, rms=case["rms"])
        return {"h": h, "y": y, "mean": mean, "rstd": rstd, "post_mean": post_mean, "post_rstd": post_rstd}
    if case["op"] == "block_bwd":
        keys = ("dx", "dresidual", "dweight", "dbias", "dpost_weight", "dpost_bias", "dgate")
        return dict(zip(keys, G.residual_norm_bwd(
            s["dy"], s["dh"], s["h"], s["weight"], s["mean"], s["rstd"], x=s["x"], post_weight=s["post_weight"],
            post_bias=s["post_bias"], post_mean=s["post_mean"], post_rstd=s["post_rstd"], gate=s["gate"],
            scale=case["scale"], rms=case["rms"], bias=case["bias"])))
    if case["op"] == "norm":
        return {"norm": G.grad_norm(s["grads"], norm_type=case["norm"])}
    norm = G.clip_grad_norm(s["grads"], case["max_norm"], norm_type=case["norm"], eps=CLIP_EPS, out=s["out"])
    return {"norm": norm, "out": _joined(s)}


def _joined(s):
    """Packed gradients as their buffers, others one by one, the many of a long
    list from its beginning, middle and end (64 outputs at most)."""
    if s["flat"]:
        return s["flat"]
    out, n = s["out"], len(s["out"])
    return out if n <= 48 else out[:16] + out[n // 2 - 8:n // 2 + 8] + out[-16:]


def _plain_policy(s, case):
    """In float64: a token near the border of the clip is on one side of it, and
    e^x - 1 - x has few digits left near 0."""
    mask = s["mask"]
    valid = mask.double()
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    logp = torch.where(mask, s["logp"].double(), zero)
    count, total = valid.sum(1, keepdim=True), valid.sum()
    if s["old"] is None:
        w = torch.zeros_like(logp)
    else:
        w = torch.where(mask, logp - s["old"].double(), zero)
        if case["ratio"] == "sequence":
            w = (w.sum(1, keepdim=True) / count.clamp(min=1)).expand_as(w)
    r = w.exp()
    A = s["adv"].double()
    A = torch.where(mask, A, zero) if case["token_adv"] else A[:, None].expand_as(w)
    up, down = r > 1 + CLIP_HIGH, r < 1 - CLIP_LOW
    far = r > case["dual"] if case["dual"] else torch.zeros_like(up)
    high = ((A > 0) & up) | ((A < 0) & far)
    low = (A < 0) & down
    held = torch.where(A > 0, r.clamp(max=1 + CLIP_HIGH),
                       r.clamp(min=1 - CLIP_LOW, max=case["dual"] or math.inf))
    loss = torch.where(A == 0, zero, -A * held)
    grad = torch.where(high | low | (A == 0), zero, -A * r)
    k = zero
    if s["ref"] is not None:
        x = torch.where(mask, s["ref"].double() - logp, zero)
        k = x.exp() - 1 - x
        loss = loss + case["beta"] * k
        grad = grad - case["beta"] * (x.exp() - 1)
    if case["reduce"] == "sequence":
        c = 1.0 / (len(valid) * count.clamp(min=1))
    else:
        c = 1.0 / (total.clamp(min=1) if case["reduce"] == "token" else torch.full_like(total, s["divisor"]))
    c = c * valid
    n = total.clamp(min=1)
    stats = torch.stack([(k * valid).sum() / n, (low * valid).sum() / n, (high * valid).sum() / n,
                         (r * valid).sum() / n])
    return {"loss": (c * loss).sum().float().view(1), "dlogp": torch.where(mask, c * grad, zero).float(),
            "stats": stats.float()}


def _gate_rows(gate, rows):
    return gate.float().repeat_interleave(rows // len(gate), 0) if 1 < len(gate) < rows else gate.float()


def _plain_norm(x, weight, bias, rms):
    mean = None if rms else x.mean(1)
    c = x if rms else x - mean[:, None]
    rstd = 1.0 / ((c * c).mean(1) + EPS).sqrt()
    y = c * rstd[:, None] * weight.float()
    return y if bias is None else y + bias.float(), mean, rstd


def _plain_block_fwd(s, case):
    p, post_mean, post_rstd = s["x"].float(), None, None
    if case["post"]:
        p, post_mean, post_rstd = _plain_norm(p, s["post_weight"], s["post_bias"], case["rms"])
    if s["gate"] is not None:
        p = p * _gate_rows(s["gate"], len(p))
    h = s["residual"].float() + case["scale"] * p
    y, mean, rstd = _plain_norm(h, s["weight"], s["bias"], case["rms"])
    dt = s["x"].dtype
    return {"h": h.to(dt), "y": y.to(dt), "mean": mean, "rstd": rstd, "post_mean": post_mean, "post_rstd": post_rstd}


def _plain_norm_bwd(g, x, weight, mean, rstd, bias):
    """(dx, dweight, dbias) of a norm, all in float32."""
    hat = (x if mean is None else x - mean[:, None]) * rstd[:, None]
    dweight, dbias = (g * hat).sum(0), g.sum(0) if bias else None
    g = g * weight.float()
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(1, keepdim=True)
    return dx * rstd[:, None], dweight, dbias


def _plain_block_bwd(s, case):
    dt, gate, x = s["h"].dtype, s["gate"], s["x"].float()
    g, dweight, dbias = _plain_norm_bwd(s["dy"].float(), s["h"].float(), s["weight"], s["mean"], s["rstd"],
                                        case["bias"])
    g = g + s["dh"].float()
    dresidual = g.to(dt)
    g = g * case["scale"]
    dgate = dpost_weight = dpost_bias = None
    if gate is not None:
        p = x
        if case["post"]:
            c = x if case["rms"] else x - s["post_mean"][:, None]
            p = c * s["post_rstd"][:, None] * s["post_weight"].float()
            p = p if s["post_bias"] is None else p + s["post_bias"].float()
        dgate = g * p
        if len(gate) < len(g):
            dgate = dgate.view(len(gate), -1, dgate.shape[1]).sum(1)
        else:
            dgate = dgate.to(gate.dtype)            # a gate for every row is an activation
        g = g * _gate_rows(gate, len(g))
    if case["post"]:
        g, dpost_weight, dpost_bias = _plain_norm_bwd(g, x, s["post_weight"], s["post_mean"], s["post_rstd"],
                                                      case["bias"])
    return {"dx": g.to(dt), "dresidual": dresidual, "dweight": dweight, "dbias": dbias,
            "dpost_weight": dpost_weight, "dpost_bias": dpost_bias, "dgate": dgate}


def _plain_clip(s, case):
    if case["norm"] == 2.0:
        norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    else:
        norm = torch.stack([g.abs().max().double() for g in s["grads"]]).max()
    if case["op"] == "norm":
        return {"norm": norm.float().view(1)}
    factor = (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    for g, to in zip(s["grads"], s["out"]):
        to.copy_(g.float() * factor)
    return {"norm": norm.float().view(1), "out": _joined(s)}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """From the definitions, in float64: sequence by sequence in slices for the
    loss, row by row in slices for the norms, tensor by tensor for the clip."""
    s = prepare(case, seed)
    if case["op"] == "policy":
        return _exact_policy(s, case)
    if case["op"] == "block_fwd":
        return _exact_block_fwd(s, case)
    if case["op"] == "block_bwd":
        return _exact_block_bwd(s, case)
    return _exact_clip(s, case)


def _exact_policy(s, case):
    """The objective min(r A, clip(r) A) and its KL term as they stand, the
    gradient from their derivatives by cases."""
    total = max(1, int(s["mask"].sum()))
    B, T = s["logp"].shape
    dlogp = torch.zeros(B, T, dtype=torch.float64, device=DEV)
    sums = torch.zeros(5, dtype=torch.float64, device=DEV)
    rows = max(1, 4_000_000 // T)
    for at in range(0, B, rows):
        cut = slice(at, min(B, at + rows))
        mask = s["mask"][cut]
        n = mask.sum(1).clamp(min=1)
        b, t = mask.nonzero(as_tuple=True)          # the valid tokens alone
        q = s["logp"][cut][b, t].double()
        w = q - s["old"][cut][b, t].double() if s["old"] is not None else torch.zeros_like(q)
        if case["ratio"] == "sequence" and s["old"] is not None:
            w = (torch.zeros(len(n), dtype=torch.float64, device=DEV).index_add_(0, b, w) / n)[b]
        A = s["adv"][cut][b, t].double() if case["token_adv"] else s["adv"][cut][b].double()
        r = torch.exp2(w / math.log(2.0))
        bounded = torch.minimum(torch.maximum(r, torch.full_like(r, 1 - CLIP_LOW)), torch.full_like(r, 1 + CLIP_HIGH))
        free = r if not case["dual"] else torch.where((A < 0) & (r > case["dual"]), case["dual"], r)
        gain = torch.minimum(free * A, bounded * A)
        flows = (A != 0) & (free * A <= bounded * A) & (free == r)
        x = s["ref"][cut][b, t].double() - q if s["ref"] is not None else torch.zeros_like(q)
        kl = torch.expm1(x) - x
        c = torch.full_like(q, {"token": 1.0 / total, "constant": 1.0 / s["divisor"], "sequence": 0.0}[case["reduce"]])
        if case["reduce"] == "sequence":
            c = 1.0 / (B * n[b].double())
        dlogp[cut][b, t] = c * (-(A * r) * flows - case["beta"] * torch.expm1(x))
        cut_off = (A != 0) & ~flows
        sums += torch.stack([(c * (case["beta"] * kl - gain)).sum(), kl.sum(), (cut_off & (r < 1)).sum().double(),
                             (cut_off & (r > 1)).sum().double(), r.sum()])
    return {"loss": sums[:1], "dlogp": dlogp, "stats": sums[1:] / total}


def _exact_stats(x, rms):
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    if rms:
        var, mean = var + mean ** 2, mean * 0
    return mean, (var + EPS) ** -0.5


def _exact_gate(s, at, n):
    g = s["gate"]
    per = s["case"]["rows"] // len(g)
    return g.double()[torch.div(torch.arange(at, at + n, device=DEV), per, rounding_mode="floor")] if len(g) > 1 else g.double()


def _exact_post(s, x, mean, rstd):
    out = (x - mean) * rstd * s["post_weight"].double()
    return out if s["post_bias"] is None else out + s["post_bias"].double()


def _exact_block_fwd(s, case):
    wide = s["x"].dtype == torch.float32
    out = {k: [] for k in ("h", "y", "mean", "rstd", "post_mean", "post_rstd")}
    zero = torch.zeros_like(s["weight"]).double()
    for at in range(0, case["rows"], 8192):
        p = s["x"][at:at + 8192].double()
        if case["post"]:
            m, r = _exact_stats(p, case["rms"])
            out["post_mean"].append(m[:, 0])
            out["post_rstd"].append(r[:, 0])
            p = _exact_post(s, p, m, r)
        if s["gate"] is not None:
            p = p * _exact_gate(s, at, len(p))
        h = torch.add(s["residual"][at:at + 8192].double(), p, alpha=case["scale"])
        m, r = _exact_stats(h, case["rms"])
        y = torch.addcmul(zero if s["bias"] is None else s["bias"].double(), (h - m) * s["weight"].double(), r)
        for k, v in (("h", h), ("y", y)):
            out[k].append(v if wide else v.float())
        out["mean"].append(m[:, 0])
        out["rstd"].append(r[:, 0])
    return {k: torch.cat(v) if v and not (case["rms"] and "mean" in k) else None for k, v in out.items()}


def _exact_norm_bwd(g, hat, rstd, weight, rms):
    gw = g * weight.double()
    d = gw.shape[1]
    dx = gw - hat * (torch.einsum("rd,rd->r", gw, hat)[:, None] / d)
    if not rms:
        dx = dx - (gw @ torch.ones(d, 1, dtype=torch.float64, device=DEV)) / d
    return dx * rstd


def _exact_block_bwd(s, case):
    wide, gate = s["h"].dtype == torch.float32, s["gate"]
    d = s["h"].shape[1]

    def sums():
        return torch.zeros(d, dtype=torch.float64, device=DEV)

    dw, db, dpw, dpb = sums(), sums(), sums(), sums()
    dgate, dxs, drs = [], [], []
    shared = gate is not None and case["gate"] != "element"
    if shared:
        dgate = torch.zeros(gate.shape, dtype=torch.float64, device=DEV)
    for at in range(0, case["rows"], 8192):
        cut = slice(at, at + 8192)

        def hat_of(t, mean, rstd):
            r = s[rstd][cut].double()[:, None]
            return (t - (0.0 if case["rms"] else s[mean][cut].double()[:, None])) * r, r

        dy = s["dy"][cut].double()
        hat, r = hat_of(s["h"][cut].double(), "mean", "rstd")
        dw += torch.einsum("rd,rd->d", dy, hat)
        db += dy.sum(0)
        g = s["dh"][cut].double() + _exact_norm_bwd(dy, hat, r, s["weight"], case["rms"])
        drs.append(g if wide else g.float())
        dx = g * case["scale"]
        if case["post"]:
            phat, pr = hat_of(s["x"][cut].double(), "post_mean", "post_rstd")
        if gate is not None:
            p = s["x"][cut].double()
            if case["post"]:
                p = phat * s["post_weight"].double()
                p = p if s["post_bias"] is None else p + s["post_bias"].double()
            dp = dx * p
            if shared:
                per = case["rows"] // len(gate)
                dgate.index_add_(0, torch.arange(at, at + len(dp), device=DEV) // per, dp)
            else:
                dgate.append(dp if wide else dp.float())
            dx = dx * _exact_gate(s, at, len(dp))
        if case["post"]:
            dpw += torch.einsum("rd,rd->d", dx, phat)
            dpb += dx.sum(0)
            dx = _exact_norm_bwd(dx, phat, pr, s["post_weight"], case["rms"])
        dxs.append(dx if wide else dx.float())
    return {"dx": torch.cat(dxs), "dresidual": torch.cat(drs), "dweight": dw, "dbias": db if case["bias"] else None,
            "dpost_weight": dpw if case["post"] else None,
            "dpost_bias": dpb if case["post"] and case["bias"] else None,
            "dgate": None if gate is None else dgate if shared else torch.cat(dgate)}


def _exact_clip(s, case):
    parts = [torch.linalg.vector_norm(g, case["norm"], dtype=torch.float64) for g in s["grads"]]
    norm = torch.linalg.vector_norm(torch.stack(parts), case["norm"])
    if case["op"] == "norm":
        return {"norm": norm.view(1)}
    factor = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
    s["out"] = [torch.mul(g.double(), factor) for g in s["grads"]]
    for kind in s["flat"]:
        s["flat"][kind] = torch.cat([t.flatten() for t, k in zip(s["out"], _kinds(case)) if k == kind])
    return {"norm": norm.view(1), "out": _joined(s)}
