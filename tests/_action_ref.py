"""Policies over many actions, gated layers and gradient norms in 64 bits, from
their definitions (numpy), with bounds for what fp32 arithmetic may lose.

u = 2^-24.  The bounds count: a rounding of a result as half a step of its type;
a sum of n terms as 8 u (sqrt(n) + 8) of its magnitudes (random rounding errors);
__expf(d) as 2 u (2 + 1.2 |d|) of itself (its documented error in units in the
last place, which are 2 u at most)."""
import numpy as np

import _trunk_ref as R

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def softmax_rows(logits, action, mask=None):
    """dict of logp, H, lp, p, d, logs, and bounds of the errors of logp, H, p (relative)."""
    l = np.asarray(logits, np.float64)
    M, V = l.shape
    if mask is not None:
        l = np.where(np.asarray(mask) != 0, l, -np.inf)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = l.max(1)
        d = l - np.where(np.isneginf(m), 0.0, m)[:, None]
        e = np.exp(d)
        s = e.sum(1)
        logs = np.log(s)
        lp = d - logs[:, None]
        p = np.where(s[:, None] == 0, 0.0, e / s[:, None])
        finite = np.where(p > 0, lp, 0.0)
        H = -(p * finite).sum(1)
        a = np.asarray(action)
        has = (a >= 0) & (a < V)
        at = lp[np.arange(M), np.where(has, a, 0)]
        la = l[np.arange(M), np.where(has, a, 0)]
        logp = np.where(has, np.where(np.isneginf(la), -np.inf, at), 0.0)
        dd = np.where(p > 0, d, 0.0)
        T, E2 = (p * -dd).sum(1), (p * dd * dd).sum(1)
        n = 8 * U * (np.sqrt(V) + 8)
        ls = np.where(s == 0, 0.0, logs)
        rs = 2 * U * (2 + 1.2 * T) + n
        b_lp = np.where(np.isfinite(logp), U * (np.abs(np.where(has, dd[np.arange(M), np.where(has, a, 0)], 0)) +
                                                np.abs(ls) * 3 + np.abs(np.where(np.isfinite(logp), logp, 0)) + 2)
                        + rs, 0.0)
        b_H = rs + 2 * U * (2 * T + 1.2 * E2) + T * (rs + n) + U * (4 * T + 4 * np.abs(ls) + H + 2)
        rp = 2 * U * (2 + 1.2 * np.abs(dd)) + U * np.abs(dd) + rs[:, None] + 4 * U
    kept = has & ~np.isneginf(logp)
    return dict(logp=logp, H=H, lp=finite, p=p, d=dd, logs=ls, kept=kept, b_logp=b_lp, b_H=b_H, rp=rp)


def policy_loss(logits, action, old, adv, scale, ref=None, weight=None, mask=None, lo=0.2, hi=0.2, kl=0.0,
                ent=0.0):
    """(softmax_rows' dict, dlogits, its bound before rounding, stats [8], their bounds)."""
    z = softmax_rows(logits, action, mask)
    M, V = np.asarray(logits).shape
    f64 = lambda v: np.asarray(v, np.float64)
    w = np.ones(M) if weight is None else f64(weight)
    use = z["kept"] & (w != 0)
    pick = lambda v: np.where(use, f64(v), 0.0)
    logp, A = pick(z["logp"]), pick(adv)
    x = logp - pick(old)
    r = np.exp(x)
    s1, s2 = r * A, np.clip(r, 1 - lo, 1 + hi) * A
    pg = -np.minimum(s1, s2)
    c = np.where(s1 <= s2, -s1, 0.0)
    dx = np.where(use, z["b_logp"] + U * np.abs(x), 0.0)
    rr = dx + 6 * U                                     # of r, relative
    b_c, b_pg = np.abs(c) * rr, np.abs(s1) * rr + np.abs(pg) * 4 * U
    k = np.zeros(M)
    b_k = np.zeros(M)
    if ref is not None:
        y = pick(ref) - logp
        k = np.exp(y) - y - 1
        dy = z["b_logp"] + U * np.abs(y)
        c = c + kl * (1 - np.exp(y))
        b_c = b_c + kl * (np.exp(y) * dy + 6 * U * np.abs(np.expm1(y)))
        b_k = np.abs(np.expm1(y)) * dy + 6 * U * (np.abs(np.expm1(y)) + np.abs(y))
    W = np.where(use, scale * w, 0.0)
    hot = np.zeros((M, V))
    rows = np.flatnonzero(use)
    hot[rows, np.asarray(action)[rows]] = 1.0
    p, inner = z["p"], z["lp"] + z["H"][:, None]
    g = W[:, None] * (c[:, None] * (hot - p) + ent * p * inner)
    g = np.where(use[:, None], g, 0.0)
    size = np.abs(c)[:, None] * (hot + p) + ent * p * (np.abs(z["d"]) + np.abs(z["H"] - z["logs"])[:, None] + 1e-9)
    b_g = np.abs(W)[:, None] * (b_c[:, None] * (hot + p) + size * (8 * U + z["rp"])
                                + ent * p * (z["b_H"] + z["b_logp"] + 4 * U * np.abs(z["logs"]))[:, None])
    b_g = np.where(use[:, None], b_g, 0.0)
    H = np.where(use, z["H"], 0.0)
    out = ((r < 1 - lo) | (r > 1 + hi)).astype(float)
    terms = [pg + kl * k - ent * H, pg, k, H, out, np.expm1(x) - x, np.ones(M)]
    b_x = np.abs(np.expm1(x)) * dx + 6 * U * (np.abs(np.expm1(x)) + np.abs(x))
    bounds = [b_pg + kl * b_k + ent * z["b_H"], b_pg, b_k, z["b_H"], 0 * b_x, b_x, 0 * b_x]
    stats = np.array([(W * t).sum() for t in terms] + [float((~z["kept"]).sum())])
    b_s = np.array([(np.abs(W) * (b + 2 * U * np.abs(t))).sum() + 2 * U * abs(v)
                    for b, t, v in zip(bounds, terms, stats)] + [0.0]) + 1e-30
    return z, g, b_g, stats, b_s


_C, _A = 2 * np.sqrt(2 / np.pi), 0.044715


def act(name, x):
    """R.act, but gelu as x sigmoid: 1 + tanh(v) has no digits left in 64 bits either
    from v = -18 on (an activation of -7), where e^(2 v) is far from 0 still."""
    x = np.asarray(x, np.float64)
    return x * R.sigmoid(_C * (x + _A * x ** 3)) if name == "gelu" else R.act(name, x)


def act_grad(name, x):
    x = np.asarray(x, np.float64)
    if name != "gelu":
        return R.act_grad(name, x)
    q = R.sigmoid(_C * (x + _A * x ** 3))
    return q + x * q * (1 - q) * _C * (1 + 3 * _A * x * x)


def gated(name, g, u):
    """(y, dy/dg, dy/du)."""
    return act(name, g) * u, act_grad(name, g) * u, act(name, g)
