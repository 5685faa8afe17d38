"""Cases of the operators around the GRPO loss head, with their plain forms.

A GRPO iteration runs, next to the loss itself: the norm that produces the
hidden states the head reads (and, after the loss's dH, the norm's gradients),
the draw of completion tokens from the head's logits, and the optimizer step
that applies dW and the other gradients. The cases below are those three
operators at this repository's head shapes and at generic odd ones.

``run`` computes the plain form (elementary torch operations) while ``own`` is
False and calls the package's kernels while it is True.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}

# Additive recurrence of the rounding dither (see _dither): the fractional
# parts 1/r and 1/r^2 of the plastic number r = 1.3247..., times 2^32.
DITHER_STEP, DITHER_INDEX = 0xC13FA9A9, 0x91E10DA5
DITHER_M, DITHER_V, DITHER_P = 0x00000000, 0x55555555, 0xAAAAAAAA


def listed():
    return [
        # one sequence being generated: the latency of a single draw
        dict(name="sample_1", op="sample", rows=1, V=128256, dtype="bf16", temperature=1.0,
             top_k=0, top_p=0.95, min_p=0.0, mixed=False, banned=0.0),
        # a group of 8 generations of one prompt, plain softmax sampling from float32 logits
        dict(name="sample_group_f32", op="sample", rows=8, V=128256, dtype="f32",
             temperature=0.9, top_k=0, top_p=1.0, min_p=0.0, mixed=False, banned=0.0),
        # generations under a grammar that bans half of the vocabulary, all cut-offs on
        dict(name="sample_61_banned", op="sample", rows=61, V=151936, dtype="bf16",
             temperature=0.6, top_k=20, top_p=0.95, min_p=0.02, mixed=False, banned=0.5),
        # a full rollout batch, every request with its own temperature and cut-offs
        dict(name="sample_512_mixed", op="sample", rows=512, V=201088, dtype="bf16",
             temperature=1.0, top_k=50, top_p=0.9, min_p=0.05, mixed=True, banned=0.0),
        # the norm of one token on its way to the head while generating
        dict(name="norm_fwd_1", op="norm_fwd", rows=1, d=4096, dtype="bf16", params="bf16",
             rms=False, bias=True),
        # the norm before the head over a whole training batch
        dict(name="norm_fwd_batch_rms", op="norm_fwd", rows=262144, d=2880, dtype="bf16",
             params="bf16", rms=True, bias=False),
        # gradients of a ragged float32 batch
        dict(name="norm_bwd_ragged_f32", op="norm_bwd", rows=13081, d=1536, dtype="f32",
             params="f32", rms=False, bias=True),
        # gradients over a whole training batch of 8 x 20480 tokens
        dict(name="norm_bwd_batch", op="norm_bwd", rows=163840, d=4096, dtype="bf16",
             params="bf16", rms=False, bias=True),
        # a step over a handful of norm weights and biases: launch latency
        dict(name="adamw_norms", op="adamw", shapes="4096,4096,1536,1536,2880,257", dtype="f32",
             grad="f32", master=False, bits=32, step=7),
        # a step over the low-rank factors of a fine-tune, 8-bit states
        dict(name="adamw_factors_8bit", op="adamw",
             shapes=",".join(["16x4096", "14336x16", "8x1536", "1027x8"] * 12), dtype="bf16",
             grad="bf16", master=False, bits=8, step=100),
        # a full fine-tune's lm_head with float32 master weights and its float32 dW
        dict(name="adamw_head", op="adamw", shapes="151936x1536,1536", dtype="bf16", grad="f32",
             master=True, bits=32, step=3),
        # the same head with no master weights and 8-bit states
        dict(name="adamw_head_8bit", op="adamw", shapes="151936x1536,1536", dtype="bf16",
             grad="f32", master=False, bits=8, step=1000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "norm_fwd", "norm_bwd", "adamw", "adamw"])
    if op == "sample":
        rows = _log_int(rng, 1, 512)
        V = rng.choice([_log_int(rng, 1000, 201088), 128256, 151936, 201088])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, V=V, dtype=dtype,
                    temperature=round(rng.uniform(0.3, 1.5), 3),
                    top_k=rng.choice([0, 0, 1, rng.randint(2, 1000)]),
                    top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                    min_p=rng.choice([0.0, round(rng.uniform(0.001, 0.2), 4)]),
                    mixed=rng.random() < 0.3, banned=rng.choice([0.0, 0.0, 0.5, 0.99]))
    if op in ("norm_fwd", "norm_bwd"):
        d = rng.choice([4096, 1536, 2880, 512, _log_int(rng, 64, 16384)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 163840 * 4096 // d // (2 if dtype == "f32" else 1)
        rms = rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, min(262144, most)), d=d, dtype=dtype,
                    params=rng.choice(["f32", dtype]), rms=rms, bias=(not rms) and rng.random() < 0.7)
    n = rng.randint(1, 24)
    shapes, room = [], 200_000_000
    for _ in range(n):
        size = _log_int(rng, 16, 30_000_000)
        if size > room:
            size = 1 + room // 100
        room -= size
        shapes.append(str(size))
    dtype = rng.choice(["bf16", "f32"])
    return dict(op=op, shapes=",".join(shapes), dtype=dtype, grad=rng.choice(["bf16", "f32"]),
                master=dtype == "bf16" and rng.random() < 0.5, bits=rng.choice([8, 32]),
                step=_log_int(rng, 1, 5000))


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _elements(case):
    return sum(math.prod(s) for s in _shapes(case))


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "sample":
        n = case["rows"] * case["V"]
        return {"bytes": n * es + case["rows"] * 28, "flops": 4 * n}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        R, d, ps = case["rows"], case["d"], SIZE[case["params"]]
        stats = 4 * R * (1 if case["rms"] else 2)
        vecs = 1 + case["bias"]
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * R * d * es + vecs * d * ps + stats, "flops": 8 * R * d}
        return {"bytes": 3 * R * d * es + d * ps + 4 * vecs * d + stats, "flops": 14 * R * d}
    n = _elements(case)
    per = 2 * es + SIZE[case["grad"]] - (es if case["master"] else 0)
    per += 8 if case["master"] else 0               # with masters the parameter is only written
    per += 16 if case["bits"] == 32 else 4 + 4 / 32
    return {"bytes": per * n, "flops": 15 * n}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dtype).mul_(std)

    def uniform(n, lo=0.0, hi=1.0):
        return torch.rand(n, generator=gen, device=DEV).mul_(hi - lo).add_(lo)

    if case["op"] == "sample":
        R, V = case["rows"], case["V"]
        # next-token logits: a power law over a random order of the vocabulary,
        # whose exponent differs from row to row, plus noise
        rank = torch.randperm(V, generator=gen, device=DEV).add_(1).float().log_()
        logits = normal((R, V), 1.0)
        logits.sub_(rank[torch.arange(V, device=DEV)] * uniform(R, 0.7, 2.2)[:, None])
        if case["banned"] > 0:
            logits.masked_fill_((uniform(V) < case["banned"])[None, :], -math.inf)
            logits[:, V // 2] = 0.0                 # the grammar leaves something to say
        s = {"case": case, "logits": logits.to(dt), "u": uniform(R),
             "temperature": torch.full((R,), case["temperature"], device=DEV),
             "top_k": torch.full((R,), case["top_k"], device=DEV, dtype=torch.int32),
             "top_p": torch.full((R,), case["top_p"], device=DEV),
             "min_p": torch.full((R,), case["min_p"], device=DEV)}
        if case["mixed"]:                           # each request asks for some of the cut-offs
            s["temperature"] *= uniform(R, 0.5, 1.5)
            s["temperature"][uniform(R) < 0.1] = 0.0            # greedy requests
            s["top_k"] *= (uniform(R) < 0.5).int()
            s["top_p"] = torch.where(uniform(R) < 0.5, s["top_p"], 1.0)
            s["min_p"] *= (uniform(R) < 0.3).float()
        return s
    if case["op"] in ("norm_fwd", "norm_bwd"):
        R, d, dp = case["rows"], case["d"], DTYPES[case["params"]]
        x = normal((R, d), 1.0, dt)
        x.mul_(torch.where(uniform(d) < 0.01, 12.0, 1.0).to(dt))   # a few loud channels
        x.add_(normal((d,), 0.3).to(dt))
        s = {"case": case, "x": x, "weight": normal((d,), 0.1).add_(1.0).to(dp),
             "bias": normal((d,), 0.1).to(dp) if case["bias"] else None}
        if case["op"] == "norm_bwd":
            s["dy"] = normal((R, d), 1e-3, dt)
            s["dy"].mul_((uniform(R) < 0.9).to(dt)[:, None])       # masked tokens have no gradient
            s["mean"], s["rstd"] = [], []
            for part in x.split(16384):                            # what the forward pass kept
                part = part.double()
                m = part.mean(1) * (0.0 if case["rms"] else 1.0)
                s["mean"].append(m.float())
                s["rstd"].append((((part - m[:, None]) ** 2).mean(1) + EPS).rsqrt().float())
            s["mean"], s["rstd"] = torch.cat(s["mean"]), torch.cat(s["rstd"])
            if case["rms"]:
                s["mean"] = None
        return s
    # adamw: parameters, gradients and the states of a run that is under way
    s = {"case": case, "params": [], "grads": [], "masters": [], "m": [], "v": [], "m_scale": [],
         "v_scale": []}
    for shape in _shapes(case):
        rows = (shape[0],) + (1,) * (len(shape) - 1)
        size = normal(rows).mul_(1.5).exp_().mul_(1e-4)            # rare rows have small gradients
        p = normal(shape, 0.02)
        s["params"].append(p.to(dt))
        s["masters"].append(p if case["master"] else None)
        s["grads"].append(normal(shape).mul_(size).to(DTYPES[case["grad"]]))
        m = normal(shape, 0.2).mul_(size)
        v = normal(shape, 0.3).add_(1.0).mul_(size).square_()
        if case["bits"] == 32:
            s["m"].append(m)
            s["v"].append(v)
        else:
            for key, t in (("m", m), ("v", v)):
                q, e = _encode(t, torch.full((1,), 0.5, device=DEV), key == "v")
                s[key].append(q)
                s[key + "_scale"].append(e)
    if own:                                         # the optimizer object that a program keeps
        import grpo_loss_gb300 as G
        s["opt"] = G.AdamW(s["params"], state_bits=case["bits"], **_hyper(case))
        s["out"] = G.AdamW([torch.empty_like(p) for p in s["params"]], state_bits=case["bits"],
                           **_hyper(case))
        for i in range(len(s["params"])):
            for mine, key in ((s["opt"].exp_avg, "m"), (s["opt"].exp_avg_sq, "v"),
                              (s["opt"].exp_avg_scale, "m_scale"),
                              (s["opt"].exp_avg_sq_scale, "v_scale"), (s["opt"].masters, "masters")):
                if s[key] and s[key][i] is not None:
                    mine[i].copy_(s[key][i].view(mine[i].dtype))
    return s


EPS = 1e-5                                          # of the norms


def _hyper(case):
    return dict(lr=2e-5, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, master=case["master"])


# --------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "sample":
        return _plain_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    if case["op"] == "norm_fwd":
        return _plain_norm_fwd(s["x"], s["weight"], s["bias"], case["rms"])
    if case["op"] == "norm_bwd":
        return _plain_norm_bwd(s["x"], s["weight"], s["dy"], s["mean"], s["rstd"], case["rms"], case["bias"])
    h, eight = _hyper(case), case["bits"] == 8
    n = len(s["params"])
    rows = [_plain_adamw(s["params"][i], s["masters"][i], s["grads"][i], s["m"][i], s["v"][i],
                         s["m_scale"][i] if eight else None, s["v_scale"][i] if eight else None,
                         case["step"], h) for i in range(n)]
    return _adamw_outputs(*[list(c) for c in zip(*rows)])


def _run_own(s, case):
    import grpo_loss_gb300 as G
    if case["op"] == "sample":
        tokens, logp = G.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                top_p=s["top_p"], min_p=s["min_p"])
        return {"tokens": tokens, "logp": logp}
    if case["op"] == "norm_fwd":
        y, mean, rstd = G.layernorm_fwd(s["x"], s["weight"], s["bias"], eps=EPS, rms=case["rms"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_bwd":
        dx, dw, db = G.layernorm_bwd(s["x"], s["weight"], s["dy"], s["mean"], s["rstd"],
                                     rms=case["rms"], bias=case["bias"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    o = s["out"]
    s["opt"].step(s["grads"], step=case["step"], out=o)
    return _adamw_outputs(o.params, o.masters, o.exp_avg, o.exp_avg_sq, o.exp_avg_scale, o.exp_avg_sq_scale)


def _adamw_outputs(params, masters, m, v, m_scale, v_scale):
    """8-bit states as the numbers they stand for: e4m3 values and the powers
    of two of their blocks. Of many tensors the first and last few are given
    one by one and the others joined by kind (64 outputs at most)."""
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    kinds = {"params": params, "masters": masters,
             "m": [t.view(f8) if t.dtype == torch.uint8 else t for t in m],
             "v": [t.view(f8) if t.dtype == torch.uint8 else t for t in v],
             "m_scale": [t.view(e8) for t in (m_scale or []) if t is not None],
             "v_scale": [t.view(e8) for t in (v_scale or []) if t is not None]}
    out = {}
    for kind, ts in kinds.items():
        ts = [t for t in ts if t is not None]
        if ts:
            out[kind] = ts if len(ts) <= 9 else ts[:4] + ts[-4:]
    return out


def _plain_sample(logits, u, temperature, top_k, top_p, min_p):
    """In float64: a token is decided by which side of a border u falls on."""
    z = logits.double()
    z = torch.where(torch.isnan(z), -math.inf, z)
    V = z.shape[1]
    zmax = z.max(1, keepdim=True).values
    warm = temperature > 0
    T = torch.where(warm, temperature, 1.0).double()[:, None]
    d = torch.where(z == zmax, 0.0, (z - zmax) / T)
    cut = -40.0 * math.log(2.0)                     # less likely than 2^-40 of the top: never drawn
    w = torch.where(d < cut, 0.0, d.exp())
    logz = w.sum(1).log()
    ws, order = torch.sort(z, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    rank = torch.arange(V, device=z.device)[None, :]
    k = torch.where(top_k > 0, top_k, V)[:, None]
    ws = torch.where((rank < k) & (ws >= min_p.double().clamp(max=1.0)[:, None]), ws, 0.0)
    upto = ws.cumsum(1)
    p = torch.where(top_p < 1, top_p, 2.0).double()[:, None]
    ws = torch.where((upto - ws < p * upto[:, -1:]) | (rank == 0), ws, 0.0)
    upto = torch.zeros_like(w).scatter_(1, order, ws).cumsum(1)
    tokens = (upto <= u.double()[:, None] * upto[:, -1:]).sum(1)
    tokens = torch.where(warm, tokens, order[:, 0])
    logp = d.gather(1, tokens[:, None])[:, 0] - logz
    some = zmax[:, 0] > -math.inf                   # a row with nothing left: no token
    return {"tokens": torch.where(some, tokens, -1).int(),
            "logp": torch.where(some, logp, -math.inf).float()}


def _plain_norm_fwd(x, weight, bias, rms):
    xf = x.float()
    mean = None if rms else xf.mean(1)
    c = xf if rms else xf - mean[:, None]
    rstd = 1.0 / ((c * c).mean(1) + EPS).sqrt()
    y = c * rstd[:, None] * weight.float()
    if bias is not None:
        y = y + bias.float()
    return {"y": y.to(x.dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(x, weight, dy, mean, rstd, rms, bias):
    g = dy.float()
    xhat = (x.float() if rms else x.float() - mean[:, None]) * rstd[:, None]
    dweight = (g * xhat).sum(0)
    dbias = g.sum(0) if bias else None
    g = g * weight.float()
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if not rms:
        dx = dx - g.mean(1, keepdim=True)
    return {"dx": (dx * rstd[:, None]).to(x.dtype), "dweight": dweight, "dbias": dbias}


def _dither(n, step, salt):
    """Sixteen bits for each element of a tensor at each step: an additive
    recurrence in the element's index and the step, so that over the steps
    a value between two codes is rounded up its share of the times."""
    i = torch.arange(n, device=DEV, dtype=torch.int64)
    return ((i * DITHER_INDEX + (step * DITHER_STEP + salt)) & 0xFFFFFFFF) >> 16


def _blocks(t):
    """[blocks of 32, 32], the last one filled up with zeros."""
    t = t.reshape(-1)
    return torch.nn.functional.pad(t, (0, -t.numel() % 32)).view(-1, 32)


def _encode(t, dither, positive):
    """e4m3 codes with one power of two for each 32 values: the smallest that
    brings them to 448 or less. ``dither``: a fraction of a code step for each
    value, added before rounding towards zero. ``positive``: values of a
    non-zero block are one step of the smallest code at least."""
    b = _blocks(t)
    amax = b.abs().amax(1)
    e = ((amax.view(torch.int32) + 0x1FFFFF) >> 23).sub(8).clamp(min=0)
    fine = amax < math.inf
    e = torch.where(fine, e, 255)
    up = torch.where(fine, 254 - e, 127).to(torch.int32) << 23
    y = b.abs() * up.view(torch.float32)[:, None]
    # a code step is 2^-9 below 2^-6 and an eighth of the power of two below y above
    step = (y.clamp(min=2.0 ** -6).view(torch.int32) & 0x7F800000).view(torch.float32) * 0.125
    part = _blocks(dither.expand(t.shape) if dither.numel() == 1 else dither)
    y = torch.floor(y.double() / step.double() + part.double()).float() * step
    if positive:
        y = torch.where((amax > 0)[:, None], y.clamp(min=2.0 ** -9), y)
    codes = torch.copysign(y, b).view(-1)[: t.numel()].view(t.shape).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), e.to(torch.uint8)


def _decode(codes, e):
    scale = torch.where(e == 0, 1 << 22, e.to(torch.int32) << 23).to(torch.int32).view(torch.float32)
    scale = torch.where(e == 255, math.nan, scale)
    return (_blocks(codes.view(torch.float8_e4m3fn).float()) * scale[:, None]).view(-1)[: codes.numel()].view(codes.shape)


def _plain_adamw(p, master, g, m, v, m_scale, v_scale, step, h):
    b1, b2 = h["betas"]
    eight = m_scale is not None
    x, g = (p if master is None else master).float(), g.float()
    m, v = (_decode(m, m_scale), _decode(v, v_scale)) if eight else (m, v)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    root = v.sqrt() / math.sqrt(1 - b2 ** step)
    x = x * (1 - h["lr"] * h["weight_decay"]) - h["lr"] / (1 - b1 ** step) * m / (root + h["eps"])
    if master is not None or p.dtype == torch.float32:
        out = x.to(p.dtype)
    else:                                           # bf16 with no master: dithered, not to nearest
        up = x.view(torch.int32) + _dither(x.numel(), step, DITHER_P).view(x.shape).int()
        out = (up & -65536).view(torch.float32).bfloat16()
    if eight:
        m, m_scale = _encode(m, _dither(m.numel(), step, DITHER_M).view(m.shape) / 65536.0, False)
        v, v_scale = _encode(v, _dither(v.numel(), step, DITHER_V).view(v.shape) / 65536.0, True)
    return out, None if master is None else x, m, v, m_scale, v_scale


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """From the definitions, in float64: row by row on the host for the
    sampler, in slices on the device for the others."""
    if case["op"] == "sample" and case["rows"] * case["V"] > 30_000_000:
        return None
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "norm_fwd":
        return _exact_norm_fwd(s, case["rms"])
    if case["op"] == "norm_bwd":
        return _exact_norm_bwd(s, case["rms"])
    return _exact_adamw(s, case)


def _exact_sample(s):
    Z = s["logits"].float().cpu().numpy().astype(np.float64)
    par = [s[k].cpu().numpy().astype(np.float64) for k in ("u", "temperature", "top_k", "top_p", "min_p")]
    tokens, logp = [], []
    for z, u, T, k, p, mp in zip(Z, *par):
        z = np.where(np.isnan(z), -np.inf, z)
        top = z.max()
        if top == -np.inf:
            tokens.append(-1)
            logp.append(-np.inf)
            continue
        with np.errstate(invalid="ignore"):
            x = np.where(z == top, 0.0, (z - top) / (T if T > 0 else 1.0))
        w = np.exp2(x / math.log(2.0))
        w[x < -40 * math.log(2.0)] = 0.0
        if T > 0:
            kept = np.flatnonzero(w >= max(mp, 1e-300))
            kept = kept[np.lexsort((kept, -z[kept]))]
            kept = kept[: int(k)] if k > 0 else kept
            if p < 1:
                share = np.concatenate([[0.0], np.cumsum(w[kept])])
                kept = kept[: max(1, int(np.searchsorted(share[:-1], p * share[-1], side="left")))]
            kept = np.sort(kept)
            c = np.cumsum(w[kept])
            at = int(kept[min(int(np.searchsorted(c, u * c[-1], side="right")), len(kept) - 1)])
        else:
            at = int(z.argmax())
        tokens.append(at)
        logp.append(x[at] - math.log(w.sum()))
    return {"tokens": np.array(tokens, np.int32), "logp": np.array(logp)}


def _exact_norm_fwd(s, rms):
    ys, means, rstds = [], [], []
    for x in s["x"].split(8192):
        x = x.double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        if rms:
            var, mean = var + mean ** 2, mean * 0
        r = (var + EPS) ** -0.5
        y = torch.addcmul((s["bias"] if s["bias"] is not None else torch.zeros_like(s["weight"])).double(),
                          (x - mean) * s["weight"].double(), r)
        ys.append(y.float() if s["x"].dtype != torch.float32 else y)
        means.append(mean[:, 0])
        rstds.append(r[:, 0])
    return {"y": torch.cat(ys), "mean": None if rms else torch.cat(means), "rstd": torch.cat(rstds)}


def _exact_norm_bwd(s, rms):
    d = s["x"].shape[1]
    w, wide = s["weight"].double(), s["x"].dtype == torch.float32
    dw, db, dxs = torch.zeros_like(w), torch.zeros_like(w), []
    at = 0
    for x, dy in zip(s["x"].split(8192), s["dy"].split(8192)):
        r = s["rstd"][at:at + len(x)].double()[:, None]
        mu = 0.0 if rms else s["mean"][at:at + len(x)].double()[:, None]
        at += len(x)
        h, dy = (x.double() - mu) * r, dy.double()
        dw += torch.einsum("rd,rd->d", dy, h)
        db += dy.sum(0)
        dyw = dy * w
        inner = torch.einsum("rd,rd->r", dyw, h)[:, None] / d
        dx = r * (dyw - h * inner - (0.0 if rms else (dyw @ torch.ones_like(w))[:, None] / d))
        dxs.append(dx if wide else dx.float())
    return {"dx": torch.cat(dxs), "dweight": dw, "dbias": db if s["case"]["bias"] else None}


def _exact_adamw(s, case):
    h, t, eight = _hyper(case), case["step"], case["bits"] == 8
    (b1, b2), rows = h["betas"], []

    def values(q, e):
        q = q.view(torch.float8_e4m3fn).double().flatten()
        return q * torch.exp2(e.double() - 127).repeat_interleave(32)[: q.numel()]

    def dithered(y, lowest, digits, salt):
        """y >= 0 on the grid of so many binary digits, steps no finer than that of 2^lowest."""
        i = torch.arange(y.numel(), device=y.device)
        u = torch.remainder(i * DITHER_INDEX + t * DITHER_STEP + salt, 2 ** 32).div(65536, rounding_mode="floor") / 65536.0
        q = torch.exp2(torch.frexp(y).exponent.sub(1).clamp(min=lowest).double() - digits)
        return (y / q + u).floor() * q

    def blocks8(x, salt, positive):
        pad = torch.cat([x, x.new_zeros(-x.numel() % 32)]).view(-1, 32)
        most = pad.abs().max(1).values.clamp(min=448 * 2.0 ** -127)
        e = torch.ceil(torch.log2(most / 448.0))
        y = dithered((pad.abs() / torch.exp2(e)[:, None]).view(-1)[: x.numel()], -6, 3, salt)
        if positive:
            y = y.clamp(min=2.0 ** -9)
        return torch.copysign(y, x), torch.exp2(e)

    for i, g in enumerate(s["grads"]):
        g = g.double().flatten()
        m = values(s["m"][i], s["m_scale"][i]) if eight else s["m"][i].double().flatten()
        v = values(s["v"][i], s["v_scale"][i]) if eight else s["v"][i].double().flatten()
        x = (s["params"][i] if s["masters"][i] is None else s["masters"][i]).double().flatten()
        m = torch.lerp(g, m, b1)
        v = torch.lerp(g * g, v, b2)
        x = x - h["lr"] * (h["weight_decay"] * x + m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + h["eps"]))
        shape = s["params"][i].shape
        p = x if s["masters"][i] is not None or case["dtype"] == "f32" else \
            torch.copysign(dithered(x.abs(), -126, 7, DITHER_P), x)
        me = ve = None
        if eight:
            (m, me), (v, ve) = blocks8(m, DITHER_M, False), blocks8(v, DITHER_V, True)
        rows.append((p.view(shape), None if s["masters"][i] is None else x.view(shape), m.view(shape), v.view(shape), me, ve))
        del g, x
    kinds, out = [list(c) for c in zip(*rows)], {}
    for kind, ts in zip(("params", "masters", "m", "v", "m_scale", "v_scale"), kinds):
        ts = [t for t in ts if t is not None]
        if ts:
            out[kind] = ts if len(ts) <= 9 else ts[:4] + ts[-4:]
    return out
