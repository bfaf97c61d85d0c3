"""The recurrent trunk's operators in 64 bits, from their definitions (numpy)."""
import numpy as np

U32 = 2.0 ** -24     # unit roundoff of fp32
U16 = 2.0 ** -9      # of bf16


def layernorm(x, gamma, beta, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    dev = x - mean[:, None]
    rstd = 1 / np.sqrt((dev * dev).mean(1) + eps)
    return dev * rstd[:, None] * gamma + beta, mean, rstd


def layernorm_grad(dy, x, gamma, mean, rstd, dres=None):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - mean[:, None]) * rstd[:, None]
    q = dy * gamma
    dx = rstd[:, None] * (q - q.mean(1, keepdims=True) - xh * (q * xh).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    return dx, (dy * xh).sum(0), dy.sum(0)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-np.asarray(x, np.float64)))


def cleared(T, N, done, done0):
    """[T][N]: the state entering step t is cleared."""
    c = np.zeros((T, N), bool)
    if done is not None:
        c[1:] = np.asarray(done)[:-1] != 0
    if done0 is not None:
        c[0] = np.asarray(done0) != 0
    return c


def scan(p, h0=None, done=None, done0=None):
    """(h [T][N][H], entering states [T][N][H]) step by step."""
    p = np.asarray(p, np.float64)
    T, N, H2 = p.shape
    H = H2 // 2
    c = cleared(T, N, done, done0)
    h = np.zeros((N, H)) if h0 is None else np.asarray(h0, np.float64)
    hs, ent = np.empty((T, N, H)), np.empty((T, N, H))
    with np.errstate(invalid="ignore"):
        for t in range(T):
            h = np.where(c[t][:, None], 0.0, h)
            ent[t] = h
            z = sigmoid(p[t, :, :H])
            h = (1 - z) * h + z * p[t, :, H:]
            hs[t] = h
    return hs, ent


def scan_grad(dh, p, h0=None, done=None, done0=None, dhT=None):
    """(dp, dh0, gradient that reaches each state)."""
    p, dh = np.asarray(p, np.float64), np.asarray(dh, np.float64)
    T, N, H2 = p.shape
    H = H2 // 2
    c = cleared(T, N, done, done0)
    _, ent = scan(p, h0, done, done0)
    u = np.zeros((N, H)) if dhT is None else np.asarray(dhT, np.float64)
    dp, gs = np.empty_like(p), np.empty((T, N, H))
    for t in range(T - 1, -1, -1):
        z, cand = sigmoid(p[t, :, :H]), p[t, :, H:]
        g = gs[t] = dh[t] + u
        dp[t, :, H:] = g * z
        dp[t, :, :H] = g * (cand - ent[t]) * z * (1 - z)
        u = np.where(c[t][:, None], 0.0, (1 - z) * g)
    return dp, u, gs


_C, _A = np.sqrt(2 / np.pi), 0.044715


def act(name, x):
    x = np.asarray(x, np.float64)
    if name == "tanh":
        return np.tanh(x)
    if name == "relu":
        return np.maximum(x, 0)
    if name == "silu":
        return x * sigmoid(x)
    if name == "gelu":
        return 0.5 * x * (1 + np.tanh(_C * (x + _A * x ** 3)))
    return x


def act_grad(name, x):
    x = np.asarray(x, np.float64)
    if name == "tanh":
        return 1 - np.tanh(x) ** 2
    if name == "relu":
        return (x > 0).astype(np.float64)
    if name == "silu":
        s = sigmoid(x)
        return s * (1 + x * (1 - s))
    if name == "gelu":
        t = np.tanh(_C * (x + _A * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * _C * (1 + 3 * _A * x * x)
    return np.ones_like(x)
