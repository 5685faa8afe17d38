"""Float64 definitions of the operators around the loss head, on the host,
written from their formulas for the tests."""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def f64(t):
    return t.detach().double().cpu().numpy()


def sample_row(z, u, T=1.0, k=0, p=1.0, q=0.0):
    """(token, logp) of one row of logits (float64 array)."""
    z = np.where(np.isnan(z), -np.inf, z)
    top = z.max()
    if top == -np.inf:
        return -1, -np.inf
    warm = T > 0
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.where(z == top, 0.0, (z - top) / (T if warm else 1.0))
    w = np.where(x < -40 * math.log(2.0), 0.0, np.exp(np.maximum(x, -1e4)))
    if warm:
        order = np.lexsort((np.arange(z.size), -z))
        if k > 0:
            order = order[:k]
        if q > 0:
            order = order[w[order] >= min(q, 1.0)]
        if p < 1:
            before = np.concatenate([[0.0], np.cumsum(w[order])])
            stays = before[:-1] < p * before[-1]
            stays[0] = True
            order = order[stays]
        kept = np.sort(order)
        c = np.cumsum(w[kept])
        u = min(max(u, 0.0) if u == u else 0.0, 1 - 2.0 ** -24)
        at = int(kept[int(np.argmax(c > u * c[-1]))])
    else:
        at = int(np.argmax(z))
    return at, x[at] - math.log(w.sum())


def sum_bound(n):
    """Relative error of a float32 sum of n terms, of the terms' magnitudes, in
    any order whose longest chain is n / 32 + 40 additions."""
    return (n / 32 + 40) * 2.0 ** -24


def norm_fwd(x, w, b, eps, rms):
    """y, mean, rstd and bounds on the errors of a float32 evaluation."""
    u, d = 2.0 ** -24, x.shape[1]
    mean = np.zeros((len(x), 1)) if rms else x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    core = (x - mean) * rstd * w
    y = core + (0 if b is None else b)
    e_mean = 0 if rms else sum_bound(d) * np.abs(x).mean(1, keepdims=True) + u * np.abs(mean)
    # the sum of squares, the shift of the mean in it (second order) and 1 / sqrt
    e_rstd = rstd * (sum_bound(d) + 8 * u) + rstd ** 3 * e_mean ** 2
    e_y = np.abs(core) * (e_rstd / rstd + 4 * u) + rstd * np.abs(w) * (e_mean + u * np.abs(x)) + 2 * u * np.abs(y)
    return y, mean[:, 0], rstd[:, 0], e_y, e_mean if rms else e_mean[:, 0], e_rstd[:, 0]


def norm_bwd(x, w, dy, mean, rstd, rms):
    """dx, dw, db and bounds on the errors of a float32 evaluation from the same
    float32 statistics."""
    u, d, R = 2.0 ** -24, x.shape[1], len(x)
    r = rstd[:, None]
    h = (x - (0 if rms else mean[:, None])) * r
    g = dy * w
    c1 = 0 if rms else g.mean(1, keepdims=True)
    c2 = (g * h).mean(1, keepdims=True)
    dx = r * (g - c1 - h * c2)
    e1 = 0 if rms else sum_bound(d) * np.abs(g).mean(1, keepdims=True)
    e2 = (sum_bound(d) + 4 * u) * np.abs(g * h).mean(1, keepdims=True)
    e_dx = np.abs(r) * (8 * u * (np.abs(g) + np.abs(c1) + np.abs(h * c2)) + e1 + np.abs(h) * e2)
    bound = (R + 16) * u
    return (dx, (dy * h).sum(0), dy.sum(0), e_dx, bound * np.abs(dy * h).sum(0) + 1e-30,
            bound * np.abs(dy).sum(0) + 1e-30)


def dither(n, step, salt):
    i = np.arange(n, dtype=np.uint64)
    return (((i * np.uint64(0x91E10DA5) + np.uint64(step * 0xC13FA9A9 + salt)) & np.uint64(0xFFFFFFFF))
            >> np.uint64(16)).astype(np.float64) / 65536.0


def block_values(codes, scale):
    """Float64 values of e4m3 codes with one power of two for each 32."""
    v = codes.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(-1)
    e = np.repeat(scale.cpu().numpy().astype(np.float64), 32)[: v.size]
    return np.where(e == 255, np.nan, v * np.exp2(e - 127))


def block_scale(x):
    """Scale bytes of the blocks of 32 of a float64 array."""
    b = np.pad(np.abs(x), (0, -x.size % 32)).reshape(-1, 32).max(1)
    e = np.ceil(np.log2(np.maximum(b, 1e-300) / 448.0)) + 127
    return np.where(np.isfinite(b), np.clip(e, 0, None), 255).astype(int)


def dithered_steps(x, scale, u):
    """(step size, number of steps down to which |x| + dither is cut) on the
    e4m3 grid under the scale bytes."""
    s = np.exp2(np.repeat(scale, 32)[: x.size] - 127.0)
    y = np.abs(x) / s
    q = np.exp2(np.clip(np.floor(np.log2(np.maximum(y, 1e-300))), -6, None) - 3)
    return q * s, y / q + u


def adamw(x, g, m, v, step, lr, b1, b2, eps, wd, grad_scale=1.0):
    """x, m, v in float64 and bounds on the errors of a float32 evaluation."""
    u = 2.0 ** -24
    g = g * grad_scale
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    e_m = 5 * u * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    upd = lr / (1 - b1 ** step) * m2 / (np.sqrt(v2) / math.sqrt(1 - b2 ** step) + eps)
    x2 = x * (1 - lr * wd) - upd
    rel = e_m / np.maximum(np.abs(m2), 1e-300)
    return x2, m2, v2, 4 * u * np.abs(x) + np.abs(upd) * (rel + 16 * u), e_m, 8 * u * v2
