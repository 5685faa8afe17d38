"""Float64 definitions of the operators of a rollout's further updates, on the host,
written from their formulas for the tests."""
import numpy as np

from tests.operator_reference import norm_bwd, norm_fwd, sum_bound

U = 2.0 ** -24                                      # half a float32 step, relative


def policy(logp, adv, mask, old=None, ref=None, clip=(0.2, 0.2), dual=None, beta=0.0, ratio="token",
           reduce="sequence", divisor=None):
    """loss, dlogp, stats and bounds on the errors of a float32 evaluation; float64
    arrays, adv [B] or [B, T]."""
    B, T = logp.shape
    live = mask != 0
    count, total = live.sum(1), max(int(live.sum()), 1)
    loss, e_loss, dlogp, e_dlogp = 0.0, 0.0, np.zeros((B, T)), np.zeros((B, T))
    kl = low = high = rs = e_kl = e_rs = 0.0
    for b in range(B):
        t = np.flatnonzero(live[b])
        q = logp[b, t]
        w = q - old[b, t] if old is not None else np.zeros(len(t))
        if ratio == "sequence" and len(t):
            w = np.full(len(t), w.mean())
        with np.errstate(over="ignore", invalid="ignore"):
            r = np.exp(w)
        A = adv[b, t] if adv.ndim == 2 else np.full(len(t), adv[b])
        top = np.where(A > 0, 1 + clip[1], np.inf if dual is None else dual)
        bottom = np.where(A > 0, 0.0, max(1 - clip[0], 0.0))
        held = np.clip(r, bottom, top)
        flows = held == r
        with np.errstate(over="ignore", invalid="ignore"):
            l = np.where(A == 0, 0.0, -A * held)
            g = np.where((A == 0) | ~flows, 0.0, -A * r)
            x = ref[b, t] - q if ref is not None else np.zeros(len(t))
            k = np.expm1(x) - x
            ex = np.expm1(x)
        c = 1.0 / (B * max(count[b], 1)) if reduce == "sequence" else 1.0 / total if reduce == "token" else 1.0 / divisor
        # e^w is off by the rounding of w (half a step of it) and of the function (two steps),
        # e^x - 1 by that of x and its own; the products by half a step each
        e_r = r * U * (np.abs(w) + 6)
        e_x = np.abs(np.exp(np.minimum(x, 700))) * np.abs(x) * U + 6 * U * np.abs(ex)
        e_k = 8 * U * np.abs(k) + np.abs(ex) * np.abs(x) * U + 4 * U * np.minimum(np.abs(k), np.abs(x))
        e_k += np.where(np.abs(x) >= 0.5, 2 * U * (np.abs(ex) + np.abs(x)), 0.0)
        e_l = np.where(A == 0, 0.0, np.abs(A) * (e_r + 4 * U * held)) + abs(beta) * (e_k + 3 * U * np.abs(k)) + U * np.abs(l)
        e_g = np.where(g == 0, 0.0, np.abs(A) * (e_r + 4 * U * r)) + abs(beta) * (e_x + 3 * U * np.abs(ex))
        loss += (c * (l + beta * k)).sum()
        e_loss += (c * e_l).sum()
        dlogp[b, t] = c * (g - beta * ex)
        e_dlogp[b, t] = c * (e_g + 4 * U * (np.abs(g) + abs(beta) * np.abs(ex)))
        kl, rs = kl + k.sum(), rs + r.sum()
        e_kl, e_rs = e_kl + e_k.sum(), e_rs + e_r.sum()
        cut = ~flows & (A != 0)
        low, high = low + (cut & (r < 1)).sum(), high + (cut & (r > 1)).sum()
    stats = np.array([kl, low, high, rs]) / total
    e_stats = np.array([e_kl, 0.0, 0.0, e_rs]) / total + 2 * U * np.abs(stats)
    return loss, dlogp, stats, e_loss + 2 * U * abs(loss), e_dlogp, e_stats


def gate_rows(gate, rows):
    return np.repeat(gate, rows // len(gate), 0)


def residual_norm_fwd(x, res, w, b=None, pw=None, pb=None, gate=None, scale=1.0, eps=1e-5, rms=False):
    """h, y, mean, rstd, post_mean, post_rstd and bounds on a float32 evaluation's errors,
    in a dict each."""
    val, err = {}, {}
    p, e_p = x, 0.0
    if pw is not None:
        p, val["post_mean"], val["post_rstd"], e_p, err["post_mean"], err["post_rstd"] = norm_fwd(x, pw, pb, eps, rms)
    g = scale * (1.0 if gate is None else gate_rows(gate, len(x)))
    h = res + g * p
    e_h = np.abs(g) * e_p + 3 * U * np.abs(g * p) + U * np.abs(h)
    val["h"], err["h"] = h, e_h
    y, val["mean"], val["rstd"], e_y, err["mean"], err["rstd"] = norm_fwd(h, w, b, eps, rms)
    # what h is off goes through the norm: its own term, the mean's, and the size's along h
    r, c = val["rstd"][:, None], h - (0.0 if rms else val["mean"][:, None])
    k = c * r
    e_m = 0.0 if rms else e_h.mean(1, keepdims=True)
    e_r = (np.abs(k) * (e_h + e_m) * r).mean(1, keepdims=True)      # relative
    val["y"], err["y"] = y, e_y + np.abs(w) * (r * (e_h + e_m) + np.abs(k) * e_r) * 1.01
    if not rms:
        err["mean"] = err["mean"] + e_m[:, 0]
    err["rstd"] = err["rstd"] + 1.01 * (e_r * r)[:, 0]
    return val, err


def residual_norm_bwd(dy, dh, h, w, mean, rstd, x=None, pw=None, pb=None, pmean=None, prstd=None, gate=None, scale=1.0,
                      rms=False):
    """dx, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate and bounds on a
    float32 evaluation's errors, in a dict each."""
    val, err = {}, {}
    R, d = h.shape
    dz, val["dweight"], val["dbias"], e_dz, err["dweight"], err["dbias"] = norm_bwd(h, w, dy, mean, rstd, rms)
    g = dz + (0.0 if dh is None else dh)
    e_g = e_dz + U * np.abs(g)
    val["dresidual"], err["dresidual"] = g, e_g
    gt = 1.0 if gate is None else gate_rows(gate, R)
    q = scale * gt * g
    e_q = np.abs(scale * gt) * e_g + 3 * U * np.abs(q)
    many = (R + 16) * U
    if pw is not None:
        k = (x - (0.0 if rms else pmean[:, None])) * prstd[:, None]
        e_hat = 3 * U * np.abs(k)
    if gate is not None:
        p = x if pw is None else k * pw + (0.0 if pb is None else pb)
        e_p = 0.0 if pw is None else 3 * U * (np.abs(k * pw) + np.abs(p))
        v = scale * g * p
        e_v = np.abs(scale) * (e_g * np.abs(p) + np.abs(g) * e_p) + 3 * U * np.abs(v)
        n = len(gate)
        fold = lambda a: a.reshape(n, -1, d).sum(1)  # noqa: E731
        val["dgate"], err["dgate"] = fold(v), fold(e_v) + (0.0 if n == R else (R // n + 16) * U) * fold(np.abs(v))
    if pw is None:
        val["dx"], err["dx"] = q, e_q
    else:
        dx, val["dpost_weight"], val["dpost_bias"], e_dx, e_pw, e_pb = norm_bwd(x, pw, q, pmean, prstd, rms)
        # what q is off, through the norm: itself, and the means of it and of its product with k
        qw = e_q * np.abs(pw)
        through = qw + (0.0 if rms else qw.mean(1, keepdims=True)) + np.abs(k) * (qw * np.abs(k)).mean(1, keepdims=True)
        # the sums may be taken of dh's part and dy's apart, each larger than their difference
        parts = np.abs(scale * gt * pw) * (np.abs(g) + np.abs(dz) + np.abs(dy * w) * rstd[:, None])
        extra = sum_bound(d) * (parts.mean(1, keepdims=True) * (0.0 if rms else 1.0) +
                                np.abs(k) * (parts * np.abs(k)).mean(1, keepdims=True))
        val["dx"], err["dx"] = dx, e_dx + np.abs(prstd[:, None]) * (through + 4 * extra)
        err["dpost_weight"] = e_pw + (e_q * np.abs(k) + np.abs(q) * e_hat).sum(0)
        err["dpost_bias"] = e_pb + e_q.sum(0)
    err["dweight"] = err["dweight"] + 3 * U * np.abs(dy * (h - (0.0 if rms else mean[:, None])) * rstd[:, None]).sum(0)
    assert many > 0
    return val, err
