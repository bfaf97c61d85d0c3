"""Gated linear layers on the GPU against the 64-bit reference.

Bounds: a sum of n products on the tensor cores is off by (n / 16 + 8) 2^-23 of
its magnitudes (one truncation a 16-term step), an fp32 one by 8 u (sqrt(n) + 8).
An activation passes its argument's error on (slopes are below 1.13) and adds its
own: 2^-11 of itself for the hardware's tanh (bf16 results alone), 2e-6 for the
others.  Results are rounded once."""
import numpy as np
import pytest

import _action_ref as A
from _gpu import host
from test_gpu_trunk_ops import dev, f64, out, within

pytestmark = pytest.mark.gpu
CODES = {"none": -1, "tanh": 0, "relu": 1, "silu": 2, "gelu": 3}


@pytest.fixture(scope="module")
def P():
    import policy_rl_gb300
    return policy_rl_gb300


def zeroed(n):
    import torch
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def sum_bound(a, b, dtype):
    """Error of a b^T, both in 64 bits."""
    n = a.shape[1]
    size = np.abs(a) @ np.abs(b).T
    return ((n / 16 + 8) * 2.0 ** -23 if dtype == "bf16" else 8 * A.U * (np.sqrt(n) + 8)) * size


def own_error(act, dtype):
    return 2.0 ** -11 if act == "tanh" and dtype == "bf16" else 2e-6


def check_forward(P, M, N, K, dtype, act="silu", bias=True, pre=True, pitches=(None,) * 4, seed=0):
    rng = np.random.default_rng(seed)
    px, pw, py, pp = pitches
    x = dev(rng.normal(size=(M, K)), dtype, px)
    w = dev(rng.normal(size=(2 * N, K)) / np.sqrt(K), dtype, pw)
    b = dev(0.3 * rng.normal(size=2 * N)) if bias else None
    y, q = out((M, N), dtype, py), out((M, 2 * N), dtype, pp) if pre else None
    work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, K, x.dtype, ldx=x.stride(0), ldw=w.stride(0)))
    P.ppo_gated_linear_forward(x, w, y, b, CODES[act], q, work)
    P.ppo_work_status(work)
    X, W = f64(x), f64(w)
    r = X @ W.T + (f64(b) if bias else 0.0)
    e = sum_bound(X, W, dtype) + 2 * A.U * np.abs(r)
    g, u, eg, eu = r[:, :N], r[:, N:], e[:, :N], e[:, N:]
    ry, dg, du = A.gated(act, g, u)
    bound = 1.13 * (np.abs(u) + eu) * eg + np.abs(du) * eu + own_error(act, dtype) * np.abs(ry) + 4 * A.U * np.abs(ry)
    if act == "relu":
        bound = (np.abs(u) + eu) * eg + np.maximum(g, 0) * eu + 4 * A.U * np.abs(ry)
    within(y, ry, bound + A.HALF[dtype] * (np.abs(ry) + bound) + 1e-30, "y")
    if pre:
        within(q, r, e + A.HALF[dtype] * (np.abs(r) + e), "pre")
    gaps(y, N, py)
    if pre:
        gaps(q, 2 * N, pp)
    return x, w, y


def gaps(t, n, pitch):
    """Nothing between the rows is written."""
    import torch
    if pitch and pitch > n and t.shape[0] > 1:
        assert torch.isnan(torch.as_strided(t, (t.shape[0] - 1, pitch - n), (pitch, 1), n)).all()


def check_backward(P, M, N, J, dtype, act="silu", with_y=True, pitches=(None,) * 5, seed=0, in_place=False):
    rng = np.random.default_rng(seed)
    pz, pw, pi, po, py = pitches
    dz = dev(rng.normal(size=(M, J)), dtype, pz)
    w2 = dev(rng.normal(size=(J, N)) / np.sqrt(J), dtype, pw)
    pre = dev(1.5 * rng.normal(size=(M, 2 * N)), dtype, pi)
    g, u = f64(pre)[:, :N], f64(pre)[:, N:]
    dp = pre if in_place else out((M, 2 * N), dtype, po)
    y = out((M, N), dtype, py) if with_y else None
    work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, 1, dz.dtype, J=J, lddz=dz.stride(0), ldw2=w2.stride(0)))
    P.ppo_gated_linear_backward_data(dz, w2, pre, dp, CODES[act], y, work)
    P.ppo_work_status(work)
    Z, W = f64(dz), f64(w2)
    d, e = Z @ W, sum_bound(Z, W.T, dtype)
    ry, sg, su = A.gated(act, g, u)
    own = own_error(act, dtype)
    slope = A.act_grad(act, g)
    # the slope's own error: exponentials and a product of a few terms below 1.2
    # of |g| with gelu' (its polynomial's terms cancel the exponential's argument)
    es = 0.0 if act in ("relu", "none") else 8e-6 * (1 + np.abs(g))
    r0, r1 = d * u * slope, d * su
    b0 = np.abs(u * slope) * e + (np.abs(d) + e) * np.abs(u) * es + 6 * A.U * np.abs(r0)
    b1 = np.abs(su) * e + (np.abs(d) + e) * np.abs(su) * own + 6 * A.U * np.abs(r1)
    h = A.HALF[dtype]
    within(dp[:, :N], r0, b0 + h * (np.abs(r0) + b0) + 1e-30, "dp gate")
    within(dp[:, N:], r1, b1 + h * (np.abs(r1) + b1) + 1e-30, "dp up")
    if with_y:
        by = own * np.abs(ry) + 4 * A.U * np.abs(ry)
        within(y, ry, by + h * (np.abs(ry) + by) + 1e-30, "y")
        gaps(y, N, py)
    if not in_place:
        gaps(dp, 2 * N, po)


# one row; few; odd; more than a tile; several tiles a CTA; sums that are split
SIZES = [(1, 1, 1), (1, 512, 128), (1, 2048, 512), (2, 33, 70), (3, 7, 5), (4, 100, 1397), (8, 256, 256), (17, 40, 64), (33, 512, 512),
         (64, 65, 130), (100, 128, 64), (129, 127, 96), (128, 128, 64), (200, 300, 256), (300, 136, 1000), (513, 1001, 200),
         (20, 3, 1), (64, 1, 9), (48, 129, 64), (49, 200, 4000),
         (1000, 64, 72), (2049, 520, 128), (70, 2048, 2048), (5000, 24, 40)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(P, M, N, K, dtype):
    check_forward(P, M, N, K, dtype, seed=M + N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,J", SIZES)
def test_backward(P, M, N, J, dtype):
    check_backward(P, M, N, J, dtype, seed=M + N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", list(CODES))
def test_activations(P, act, dtype):
    for M in (1, 5, 300):
        check_forward(P, M, 136, 96, dtype, act, seed=3)
        check_forward(P, M, 136, 96, dtype, act, bias=False, pre=False, seed=4)
        check_backward(P, M, 136, 96, dtype, act, seed=5)
        check_backward(P, M, 136, 96, dtype, act, with_y=False, seed=6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 6, 150, 400])
@pytest.mark.parametrize("N,K,pitches", [(64, 72, (80, 88, 72, 136)), (64, 72, (77, 75, 65, 131)), (61, 70, (72, 72, 64, 128)),
                                         (130, 130, (131, 130, 130, 261)), (192, 64, (64, 64, 200, 392))])
def test_pitches(P, M, N, K, pitches, dtype):
    px, pw, py, pp = pitches
    check_forward(P, M, N, K, dtype, pitches=pitches, seed=M)
    check_backward(P, M, N, K, dtype, pitches=(px, max(N, pw), pp, pp, py), seed=M)


def test_large_tiles(P):
    """Tiles enough for several a pair of CTAs, in both directions."""
    check_forward(P, 20000, 512, 64, "bf16", seed=1)
    check_forward(P, 9001, 1000, 72, "bf16", "gelu", seed=2)
    check_backward(P, 20000, 512, 64, "bf16", seed=3)
    check_backward(P, 9001, 1000, 72, "bf16", "gelu", seed=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_in_place(P, dtype):
    for M, N, J in ((1, 8, 8), (40, 61, 24), (700, 520, 128)):
        check_backward(P, M, N, J, dtype, in_place=True, seed=M)


def test_long_sums(P):
    check_forward(P, 40, 24, 70000, "bf16", seed=1)
    check_backward(P, 40, 24, 70000, "bf16", seed=2)


@pytest.mark.parametrize("M", [1, 40, 1000])
def test_special_values(P, M):
    """Infinities and NaN stay in their rows and columns."""
    import torch
    N, K = 64, 48
    rng = np.random.default_rng(1)
    for dtype in ("f32", "bf16"):
        x, w = dev(rng.normal(size=(M, K)), dtype), dev(rng.normal(size=(2 * N, K)), dtype)
        work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, K, x.dtype, J=K))
        y, y2 = out((M, N), dtype), out((M, N), dtype)
        P.ppo_gated_linear_forward(x, w, y, None, CODES["silu"], None, work)
        w[5, 0], w[N + 9, 3] = float("nan"), float("inf")
        P.ppo_gated_linear_forward(x, w, y2, None, CODES["silu"], None, work)
        cols = [c for c in range(N) if c not in (5, 9)]
        assert torch.equal(y[:, cols], y2[:, cols])
        assert torch.isnan(y2[:, 5]).all() and (~torch.isfinite(y2[:, 9])).all()


def test_special_values_in_fp32_on_the_tensor_cores(P):
    """The planes of an infinity do not add up: what it reaches is summed again."""
    import torch
    M, N, K = 1000, 512, 160
    rng = np.random.default_rng(1)
    x, w = dev(rng.normal(size=(M, K))), dev(rng.normal(size=(2 * N, K)) / 12)
    dz, w2 = dev(rng.normal(size=(M, K))), dev(rng.normal(size=(K, N)) / 12)
    pre = dev(rng.normal(size=(M, 2 * N)))
    work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, K, x.dtype, J=K))
    w[N + 9, 3] = float("inf")
    w[40, 5] = 3.4e38           # bf16 rounds it to infinity
    x[17, 5] = 0.0
    w2[2, 33] = float("inf")
    y, q, dp = out((M, N)), out((M, 2 * N)), out((M, 2 * N))
    P.ppo_gated_linear_forward(x, w, y, None, CODES["relu"], q, work)
    P.ppo_gated_linear_backward_data(dz, w2, pre, dp, CODES["relu"], None, work)
    with np.errstate(invalid="ignore", over="ignore"):
        r = f64(x) @ f64(w).T
        d = f64(dz) @ f64(w2)
    assert np.array_equal(np.sign(f64(q)[:, N + 9]), np.sign(r[:, N + 9])) and torch.isinf(q[:, N + 9]).all()
    ok = np.abs(r[:, 40]) < 3e38
    assert ok[17] and np.allclose(f64(q)[ok, 40], r[ok, 40], rtol=1e-5)
    assert (np.isinf(f64(q)[:, 40]) == (np.abs(r[:, 40]) > 3.4028235e38)).all()
    assert torch.isfinite(q[:, [c for c in range(2 * N) if c not in (40, N + 9)]]).all()
    u = f64(pre)[:, N + 33]
    g = f64(pre)[:, 33]
    assert (np.isinf(f64(dp)[:, 33]) == ((g > 0) & (u != 0))).all() and not np.isfinite(f64(dp)[:, N + 33]).any()
    assert np.array_equal(np.sign(f64(dp)[g > 0, N + 33]), np.sign(d[g > 0, 33]))


def test_few_rows(P):
    """One to eight rows: groups of warps along the sum, columns that do not fill a block."""
    for M in range(1, 10):
        for N, K in ((1, 3), (2, 2000), (37, 129), (300, 4096), (3000, 64)):
            for dtype in ("f32", "bf16"):
                check_forward(P, M, N, K, dtype, seed=M, pitches=(K + 1, None, N + 3, None) if N == 37 else (None,) * 4)


@pytest.mark.parametrize("M,N,K", [(300, 200, 96), (1, 200, 96), (33, 200, 1024), (64, 4000, 96), (4, 1024, 4096)])
def test_streams_graphs_and_determinism(P, M, N, K):
    import torch
    rng = np.random.default_rng(2)
    x, w = dev(rng.normal(size=(M, K)), "bf16"), dev(rng.normal(size=(2 * N, K)), "bf16")
    dz, w2 = dev(rng.normal(size=(M, K)), "bf16"), dev(rng.normal(size=(K, N)), "bf16")
    y, pre, dp, y2 = (out(s, "bf16") for s in ((M, N), (M, 2 * N), (M, 2 * N), (M, N)))
    work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, K, x.dtype, J=K))

    def go(stream=None):
        P.ppo_gated_linear_forward(x, w, y, None, CODES["gelu"], pre, work, stream)
        P.ppo_gated_linear_backward_data(dz, w2, pre, dp, CODES["gelu"], y2, work, stream)

    go()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, pre, dp, y2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    go(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, pre, dp, y2)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(2):
        for t in (y, pre, dp, y2):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, pre, dp, y2)))


def test_refusals(P):
    M, N, K = 8, 16, 24
    x, w, y = dev(np.zeros((M, K)), "bf16"), dev(np.zeros((2 * N, K)), "bf16"), out((M, N), "bf16")
    work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, K, x.dtype, J=K))
    with pytest.raises(ValueError):
        P.ppo_gated_linear_forward(x, w[:N], y, work=work)
    with pytest.raises(ValueError):
        P.ppo_gated_linear_forward(x, w.float(), y, work=work)
    for bad in (dict(work=None), dict(work=work[:16]), dict(work=work, act=9), dict(work=work[8:])):
        with pytest.raises(P.PpoError):
            P.ppo_gated_linear_forward(x, w, y, **bad)
    base = out((M * N + 8,), "bf16")
    with pytest.raises(P.PpoError):
        P.ppo_gated_linear_forward(x, w, base[4:4 + M * N].view(M, N), work=work)
    wide = out((M, 4 * N), "bf16")
    pre, dz, w2 = wide[:, :2 * N], dev(np.zeros((M, K)), "bf16"), dev(np.zeros((K, N)), "bf16")
    with pytest.raises(P.PpoError):      # in place, another pitch
        P.ppo_gated_linear_backward_data(dz, w2, pre, wide.view(-1)[:M * 2 * N].view(M, 2 * N), work=work)
    for size in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 1 << 28, 4)):
        with pytest.raises(P.PpoError):
            P.ppo_gated_linear_workspace_bytes(*size, x.dtype)
