"""The trunk operators at the limits of their plans: widths that fill a shared-
memory size exactly, very many rows of few columns, rows padded in the
workspace, values near the ends of the types' ranges, very long sums, and
shapes that reach the variants for large problems.  Bounds as in
test_gpu_trunk_ops.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

import _trunk_ref as R
from test_gpu_trunk_ops import (P, check_linear, check_ln, check_scan, dev, f64, ln_inputs, out,  # noqa: F401
                                prod_bound, rounding, scan_inputs, tdt, within)

pytestmark = pytest.mark.gpu
U32, U16 = R.U32, R.U16
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("dtype,M,N,K", [("bf16", 4096, 512, 100), ("bf16", 65536, 64, 20),
                                         ("f32", 700, 640, 636), ("f32", 3000, 130, 100)])
@pytest.mark.parametrize("bias", [True, False])
def test_weight_gradient_of_widths_four_past_eight(P, dtype, M, N, K, bias):
    """K % 8 = 4: rows of partial products are padded, rows of dW are not.  The
    workspace holds what earlier calls may have left, and dW and db lie in larger
    buffers whose other elements stay."""
    import torch
    rng = np.random.default_rng(M + K)
    dz, x = dev(rng.normal(size=(M, N)), dtype), dev(rng.normal(size=(M, K)), dtype)
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, tdt(dtype)), dtype=torch.uint8, device="cuda")
    work[256:] = 0x7f
    room, roomb = torch.full((N * K + 64,), 5.0, device="cuda"), torch.full((N + 64,), 5.0, device="cuda")
    dw, db = room[:N * K].view(N, K), roomb[:N]
    P.ppo_linear_backward_weight(dz, x, dw, db=db if bias else None, work=work)
    P.ppo_work_status(work)
    Z, X = f64(dz), f64(x)
    within(dw, Z.T @ X, prod_bound(dtype, Z.T, X, M), "dw")
    if bias:
        within(db, Z.sum(0), 8 * U32 * (np.sqrt(M) + 8) * np.abs(Z).sum(0), "db")
    assert bool((room[N * K:] == 5.0).all()) and bool((roomb[N if bias else 0:] == 5.0).all())


def test_a_refused_call_leaves_no_error_behind():
    """The status word cannot be waited for inside a graph capture: that call says
    so, and the calls after it are not blamed for it."""
    code = (f"import sys; sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]\n"
            "import torch\n"
            "import policy_rl_gb300 as P\n"
            "from test_gpu_trunk_ops import check_linear, check_ln, check_scan\n"
            "work, side = torch.zeros(256, dtype=torch.uint8, device='cuda'), torch.cuda.Stream()\n"
            "def refused():\n"
            "    try:\n"
            "        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):\n"
            "            try:\n"
            "                P.ppo_work_status(work, stream=side)\n"
            "            except P.PpoError as e:\n"
            "                assert 'PPO_ERR_CUDA' in str(e)\n"
            "                return True\n"
            "    except RuntimeError:\n"
            "        return True\n"
            "for check in (lambda: check_ln(P, 9, 40, 'f32'), lambda: check_scan(P, 3, 2, 8, 'f32', 1),\n"
            "              lambda: check_linear(P, 20, 24, 16, 'f32')):\n"
            "    assert refused()\n"
            "    torch.cuda.synchronize()\n"
            "    check()\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype,widths", [("f32", (1532, 1534, 1536, 1537, 1801, 2048)),
                                          ("bf16", (3576, 3584, 3585, 3847, 4096))])
def test_layernorm_backward_of_rows_that_fill_48_kb(dtype, widths):
    """Widths whose rows on their way take 48 KB beside what the kernel holds
    statically: in a process of their own and in ascending order, so that no wider
    call has gone before."""
    code = (f"import sys; sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]\n"
            "import policy_rl_gb300 as P\nfrom test_gpu_trunk_ops import check_ln\n"
            f"for D in {widths}:\n"
            "    for res in (False, True):\n"
            f"        check_ln(P, 40, D, {dtype!r}, res=res, seed=D)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(600000, 1, 16), (600000, 1, 7), (1000000, 1, 33), (530001, 3, 5), (524281, 2, 8)])
def test_linear_forward_of_very_many_rows_and_few_columns(P, M, N, K, dtype):
    """A value head over a large rollout."""
    import torch
    rng = np.random.default_rng(K)
    x, w, b = dev(rng.normal(size=(M, K)), dtype), dev(rng.normal(size=(N, K)), dtype), dev(rng.normal(size=N))
    y = out((M, N), dtype)
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, tdt(dtype)), dtype=torch.uint8, device="cuda")
    P.ppo_linear_forward(x, w, y, bias=b, work=work)
    P.ppo_work_status(work)
    X, W = f64(x), f64(w)
    ry = X @ W.T + f64(b)
    within(y, ry, rounding(dtype, ry) + prod_bound(dtype, X, W.T, K) + 2 * U32 * (np.abs(ry) + np.abs(f64(b))), "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["tanh", "relu", "silu", "gelu"])
@pytest.mark.parametrize("M,N,K", [(5, 40, 24), (300, 256, 264), (700, 640, 640)])
def test_slopes_of_large_pre_activations(P, M, N, K, act, dtype):
    """Finite values whose squares leave fp32's range: the slope is 0 or 1 there,
    and a NaN stays in its element."""
    import torch
    rng = np.random.default_rng(M)
    code = {"tanh": 0, "relu": 1, "silu": 2, "gelu": 3}[act]
    dz, w = dev(rng.normal(size=(M, N)), dtype), dev(rng.normal(size=(N, K)) / np.sqrt(K), dtype)
    pre = 1.5 * rng.normal(size=(M, K))
    large = [16, 17, 40, 100, 1e4, 1e10, 1.5e19, 2e19, 1e20, 3e38]
    for i, v in enumerate(large):
        pre[i % M, 2 * i], pre[i % M, 2 * i + 1] = v, -v
    pre[M - 1, K - 1] = np.nan
    pre, dx = dev(pre, dtype), out((M, K), dtype)
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, tdt(dtype)), dtype=torch.uint8, device="cuda")
    P.ppo_linear_backward_data(dz, w, dx, pre=pre, act=code, work=work)
    P.ppo_work_status(work)
    Z, W, X = f64(dz), f64(w), f64(pre)
    rd = Z @ W
    ref = rd * R.act_grad(act, np.where(np.isnan(X), 0.0, X))
    bound = rounding(dtype, ref) + 1.2 * prod_bound(dtype, Z, W, N) + 64 * U32 * np.abs(rd) + 4 * U32 * np.abs(ref)
    bound[M - 1, K - 1] = np.inf
    got = f64(dx)
    if act != "relu":
        assert np.isnan(got[M - 1, K - 1])
    got[M - 1, K - 1] = 0.0
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (X[bad], got[bad], ref[bad])


@pytest.mark.parametrize("K", [1 << 18, 1 << 20])
def test_bf16_products_of_very_long_sums(P, K):
    """The tensor cores truncate what they add, which over positive terms is a
    drift; rounding to nearest has none.  The mean relative error of many results
    is below six standard errors of a bf16 rounding, (U16 / sqrt 3) / sqrt(count),
    and what 32 truncated steps of a window and fp32 sums leave, 1e-5."""
    import torch
    M = N = 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    x = torch.rand(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(N, K, generator=g, device="cuda", dtype=torch.bfloat16)
    y, work = out((M, N), "bf16"), torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, x.dtype), dtype=torch.uint8,
                                               device="cuda")
    rows = torch.arange(0, M, 32, device="cuda")
    ref = sum(x[rows, k:k + 65536].double() @ w[rows, k:k + 65536].double().t() for k in range(0, K, 65536))
    limit = 6 * U16 / np.sqrt(3 * ref.numel()) + 1e-5
    P.ppo_linear_forward(x, w, y, work=work)
    err = y[rows][:, rows].double() / ref - 1
    assert abs(float(err.mean())) < limit, float(err.mean())
    assert float(err.abs().max()) < 1.01 * U16
    # the data gradient of [M][K] by [K][N] sums over K as well
    wt = w.t().contiguous()
    P.ppo_linear_backward_data(x, wt, y, work=work)
    P.ppo_work_status(work)
    err = y[rows][:, rows].double() / ref - 1
    assert abs(float(err.mean())) < limit and float(err.abs().max()) < 1.01 * U16


def test_views_of_one_environment(P):
    """[T, 1, W] slices of a rollout have one pitch and are taken as they lie."""
    import torch
    T, N, H = 150, 5, 40
    rng = np.random.default_rng(3)
    full, dfull = dev(rng.normal(size=(T, N, 2 * H)), "bf16"), dev(rng.normal(size=(T, N, H)), "bf16")
    h, dp = torch.zeros(T, N, H, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(full)
    carry, want_h, want_dp = out((2, 1, H)), out((T, 1, H), "bf16"), out((T, 1, 2 * H), "bf16")
    for n in (0, 2):
        P.ppo_gated_scan_forward(full[:, n:n + 1].contiguous(), want_h, carry=carry)
        P.ppo_gated_scan_forward(full[:, n:n + 1], h[:, n:n + 1], carry=carry)
        P.ppo_gated_scan_backward(dfull[:, n:n + 1].contiguous(), full[:, n:n + 1].contiguous(), carry, want_dp)
        P.ppo_gated_scan_backward(dfull[:, n:n + 1], full[:, n:n + 1], carry, dp[:, n:n + 1])
        assert torch.equal(h[:, n:n + 1], want_h) and torch.equal(dp[:, n:n + 1], want_dp)
    assert not h[:, [1, 3, 4]].any() and not dp[:, [1, 3, 4]].any()


def test_trunk_takes_gradients_of_odd_pitch(P):
    """dy as columns of a wider buffer (logits beside a value), against 64-bit
    autograd with the bound of test_trunk_in_bf16.  (Not bit for bit what rows of
    even pitch give: layer norm sums rows of unequal pitches in another order.)"""
    import torch
    from test_gpu_trunk import build, reference, run
    t, made = build(20, 6, 64, 32, 96, torch.bfloat16)
    ref = reference(t, made)
    wide = torch.zeros(20, 6, 65, dtype=torch.bfloat16, device="cuda")
    wide[..., :64] = made["dy"]
    made["dy"] = wide[..., :64]
    got = run(t, made)
    for k, r in ref.items():
        err = float((got[k].double() - r).norm() / r.norm())
        assert err <= 3e-2, (k, err)


# ---- variants that only large problems reach ---------------------------------------
@pytest.mark.parametrize("act,pact,res,dres,pre,K,pitch", [
    ("relu", "relu", False, False, False, 1000, None),
    ("none", "none", False, True, False, 1000, None),
    ("relu", "none", True, False, False, 1032, None),
    ("none", "relu", True, True, False, 1032, None),
    ("gelu", "silu", True, True, True, 1000, None),
    ("relu", "relu", False, False, False, 997, (999, 1001, 1003)),
    ("none", "none", True, True, False, 1031, (1033, 1035, 1001)),
    ("gelu", "relu", True, True, True, 997, (1001, 997, 1007))])
def test_linear_with_many_tiles_a_pair(P, act, pact, res, dres, pre, K, pitch):
    """308 tiles of 256 x 256 forward (and 308 or 385 backward): four and more for each
    pair of CTAs, each epilogue with its boxes moved by TMA or, of odd pitch, by hand."""
    check_linear(P, 19500, 1000, K, "bf16", act=act, pact=pact, res=res, dres=dres, pre=pre, pitch=pitch, seed=K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", [(140, 1217, 128), (135, 1207, 129), (300, 2440, 64)])
def test_scan_walked_by_warps_over_many_tiles(P, T, N, H, dtype):
    """More than 155,648 channels: forward, each warp walks its channels alone and
    leaves the carry of every 128th step, which the backward pass starts from."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    p = (1.5 * rn(T, N, 2 * H) - 0.5).to(tdt(dtype))
    done, done0 = (rn(T, N) > 1.6).float(), (rn(N) > 0.5).float()
    h0, dh, dhT = rn(N, H), rn(T, N, H).to(tdt(dtype)), rn(N, H)
    h, hT, carry = out((T, N, H), dtype), out((N, H)), out((P.ppo_scan_blocks(T), N, H))
    dp, dh0 = out((T, N, 2 * H), dtype), out((N, H))
    P.ppo_gated_scan_forward(p, h, h0=h0, done=done, done0=done0, hT=hT, carry=carry)
    P.ppo_gated_scan_backward(dh, p, carry, dp, done=done, done0=done0, dhT=dhT, dh0=dh0)
    # step by step in 64 bits, on the device
    state, ent, S = h0.double(), [], 0.0
    for t in range(T):
        state = torch.where((done0 if t == 0 else done[t - 1])[:, None] != 0, 0.0, state)
        ent.append(state)
        S = max(S, float(state.abs().max()), float(p[t, :, H:].abs().max()))
        if t % 128 == 0:
            assert float((carry[t // 128].double() - state).abs().max()) <= 1e-5 * S
        z = torch.sigmoid(p[t, :, :H].double())
        state = (1 - z) * state + z * p[t, :, H:].double()
        lost = 2 * U16 * state.abs() if dtype == "bf16" else 0.0
        assert bool(((h[t].double() - state).abs() <= lost + 1e-5 * max(S, float(state.abs().max()))).all()), t
    assert float((hT.double() - state).abs().max()) <= 1e-5 * S
    u, G = dhT.double(), 0.0
    for t in range(T - 1, -1, -1):
        z, c = torch.sigmoid(p[t, :, :H].double()), p[t, :, H:].double()
        q = dh[t].double() + u
        G = max(G, float(q.abs().max()))
        want = torch.cat([q * (c - ent[t]) * z * (1 - z), q * z], 1)
        lost = 2 * U16 * want.abs() if dtype == "bf16" else 0.0
        assert bool(((dp[t].double() - want).abs() <= lost + 1e-5 * G * (1 + 2 * S)).all()), t
        u = torch.where((done0 if t == 0 else done[t - 1])[:, None] != 0, 0.0, (1 - z) * q)
    assert float((dh0.double() - u).abs().max()) <= 1e-5 * G


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(1000, 513), (3001, 33), (700, 1397), (500, 4101), (330, 8201)])
def test_layernorm_in_place_of_odd_widths(P, M, D, dtype):
    """Aligned pieces reach into the rows beside: in place, rows that other blocks write."""
    import torch
    _, x, ga, be = ln_inputs(M, D, dtype, 5)
    y, st = torch.empty_like(x), out((M, 2))
    P.ppo_layernorm_forward(x, ga, be, y, stats=st)
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    dy, dres = (torch.randn(M, D, generator=g, device="cuda").to(x.dtype) for _ in range(2))
    dx, dxr = torch.empty_like(x), torch.empty_like(x)
    P.ppo_layernorm_backward(dy, x, ga, st, dx)
    P.ppo_layernorm_backward(dy, x, ga, st, dxr, dres=dres)
    for _ in range(5):
        a, b, c, d = x.clone(), dy.clone(), dy.clone(), dres.clone()
        P.ppo_layernorm_forward(a, ga, be, a)
        P.ppo_layernorm_backward(b, x, ga, st, b)
        P.ppo_layernorm_backward(c, x, ga, st, c, dres=dres)
        P.ppo_layernorm_backward(dy, x, ga, st, d, dres=d)
        assert torch.equal(a, y) and torch.equal(b, dx) and torch.equal(c, dxr) and torch.equal(d, dxr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D,pitch", [(700, 8200, None), (310, 16393, None), (1000, 4099, 4101)])
def test_layernorm_of_long_rows_several_a_block(P, M, D, pitch, dtype):
    """Rows that are read once per reduction; a block adds up several rows' parameter
    gradients in its partial row."""
    check_ln(P, M, D, dtype, pitch=pitch, seed=M)
    check_ln(P, M, D, dtype, pitch=pitch, res=False, seed=M)


def test_layernorm_past_32_bit_offsets_against_the_reference(P):
    import torch
    M, D = 540000, 4096                     # 2.2e9 elements
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    x, dy = (torch.zeros(M, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x[rows] = torch.randn(5, D, generator=g, device="cuda").to(torch.bfloat16)
    dy[rows] = torch.randn(5, D, generator=g, device="cuda").to(torch.bfloat16)
    ga, be = 1 + 0.2 * torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    X, Z, st, dg, db = f64(x[rows]), f64(dy[rows]), out((M, 2)), out((D,)), out((D,))
    work = out((P.ppo_layernorm_backward_workspace_bytes(M, D) // 4,))
    y = torch.empty_like(x)
    P.ppo_layernorm_forward(x, ga, be, y, stats=st)
    P.ppo_layernorm_backward(dy, x, ga, st, dy, dgamma=dg, dbeta=db, work=work)      # in place
    ry, mean, rstd = R.layernorm(X, f64(ga), f64(be), 1e-5)
    rdx, rdg, rdb = R.layernorm_grad(Z, X, f64(ga), mean, rstd)
    # as in check_ln: a row's values relative to its deviation are off by `lost`
    lost = 16 * U32 * (np.sqrt(D) + 8) * (np.abs(X).mean(1) * rstd + 1)[:, None]
    within(y[rows], ry, 2 * U16 * np.abs(ry) + lost * (np.abs(ry) + np.abs(f64(ga)) + np.abs(f64(be))), "y")
    xh, q = np.abs((X - mean[:, None]) * rstd[:, None]), np.abs(Z * f64(ga))
    size = rstd[:, None] * (q + q.mean(1, keepdims=True) + (xh + 1) * (q * (xh + 1)).mean(1, keepdims=True))
    within(dy[rows], rdx, 2 * U16 * np.abs(rdx) + 2 * lost * (size + np.abs(rdx)), "dx")
    n = 8 * U32 * (np.sqrt(5) + 8)
    within(dg, rdg, n * (np.abs(Z) * xh).sum(0) + (np.abs(Z) * lost * (xh + 1)).sum(0), "dgamma")
    within(db, rdb, n * np.abs(Z).sum(0), "dbeta")
    want = be.to(torch.bfloat16)
    assert bool((y[2:M // 2] == want).all()) and not bool(dy[2:M // 2].any())
    assert bool((y[M // 2 + 1:M - 2] == want).all()) and not bool(dy[M // 2 + 1:M - 2].any())


# ---- fp32 products by planes with elements that bf16 cannot hold ------------------------
def test_f32_weight_gradient_infinities_in_many_slices_of_the_sum(P):
    """Slices of a long sum are finished apart: infinities of one sign, of both signs
    in one slice and in distant ones, infinity times zero, NaN, and large finite
    values, each in its row of dW and its element of db alone."""
    import torch
    rng = np.random.default_rng(21)
    M, N, K = 40000, 72, 68
    dz, x = rng.normal(size=(M, N)), rng.normal(size=(M, K))
    inf = np.inf
    dz[11, 0] = dz[39990, 0] = inf                  # rows of dW: 0 .. 6
    dz[11, 1], dz[39990, 1] = inf, -inf
    dz[20000, 2], dz[20001, 2] = -inf, inf
    dz[30000, 3], x[30000, 5] = inf, 0.0
    dz[7, 4] = np.nan
    dz[[9, 25000], 5], x[[9, 25000]] = 3.4e38, np.clip(x[[9, 25000]], -0.4, 0.4)
    dz[39999, 6] = -inf
    dz, x = dev(dz), dev(x)
    dw, db = out((N, K)), out((N,))
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, x.dtype), dtype=torch.uint8, device="cuda")
    P.ppo_linear_backward_weight(dz, x, dw, db=db, work=work)
    P.ppo_work_status(work)
    Z, X, W, B = f64(dz), f64(x), f64(dw), f64(db)
    with np.errstate(invalid="ignore", over="ignore"):
        rw, rb = Z.T @ X, Z.sum(0)
        # (the product of an infinity and the rest, without what a library may do with it)
        for n in (0, 1, 2, 3, 4, 6):
            rw[n] = (Z[:, n, None] * X).sum(0)
    special = np.arange(7)
    for n in (0, 1, 2, 3, 4, 6):
        assert np.array_equal(np.isnan(W[n]), np.isnan(rw[n])), n
        ok = ~np.isnan(rw[n])
        assert np.array_equal(W[n][ok], rw[n][ok]), n
        assert B[n] == rb[n] or np.isnan(B[n]) and np.isnan(rb[n]), n
    rest = np.setdiff1d(np.arange(N), special[[0, 1, 2, 3, 4, 6]])
    assert (np.abs(W[rest] - rw[rest]) <= prod_bound("f32", Z[:, rest].T, X, M)).all()
    # (6.8e38 leaves fp32's range in the sum of the column, not in its products)
    assert B[5] == inf
    rest = np.arange(7, N)
    assert (np.abs(B[rest] - rb[rest]) <= 8 * U32 * (np.sqrt(M) + 8) * np.abs(Z[:, rest]).sum(0)).all()


def test_f32_products_with_an_infinity_take_no_thousand_times_longer(P):
    """One infinity in a gradient of 300,000 rows: its row of dW and its column sum are
    computed again, which may take 100 times the product (0.4 ms), not 1,000."""
    import torch
    M, N, K = 300000, 64, 64
    dz, x = torch.randn(M, N, device="cuda"), torch.randn(M, K, device="cuda")
    dw, db = out((N, K)), out((N,))
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, x.dtype), dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def ms():
        took = []
        for _ in range(4):
            a.record()
            P.ppo_linear_backward_weight(dz, x, dw, db=db, work=work)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        return min(took)
    plain = ms()
    dz[5, 7] = float("inf")
    assert ms() < 100 * plain
    assert bool(torch.isinf(dw[7]).all()) and bool(torch.isinf(db[7])) and int(torch.isfinite(dw).sum()) == (N - 1) * K


# ---- nothing but the outputs is written ------------------------------------------------
@pytest.fixture
def framed(monkeypatch):
    """Outputs of the checks lie in larger buffers of NaN: before (`front` elements),
    after and between their rows nothing may change."""
    import torch
    import test_gpu_trunk_ops as ops
    frames = []

    def framed_out(shape, dtype="f32", pitch=None):
        front, pitch, rows = check.front, pitch or shape[-1], int(np.prod(shape[:-1]))
        flat = torch.full((front + rows * pitch + 64,), float("nan"), dtype=tdt(dtype), device="cuda")
        frames.append((flat, front, rows, pitch, shape[-1]))
        return flat[front:-64].view(*shape[:-1], pitch)[..., :shape[-1]]

    def check():
        assert frames
        for flat, front, rows, pitch, width in frames:
            assert bool(flat[:front].isnan().all()) and bool(flat[-64:].isnan().all())
            gap = flat[front:-64].view(rows, pitch)[:, width:]
            assert bool(gap.isnan().all()), (rows, pitch, width, gap.isnan().logical_not().nonzero()[:3].tolist())
    check.front = 64
    monkeypatch.setattr(ops, "out", framed_out)
    return check


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pre,res,dres", [(False, False, False), (True, False, True), (False, True, False),
                                          (True, True, True)])
@pytest.mark.parametrize("M,N,K,pitch", [(50, 31, 21, (24, 24, 32)), (552, 6, 1, (8, 8, 8)), (300, 245, 335, (336, 336, 248)),
                                         (700, 1003, 999, (1000, 1000, 1008)), (4220, 18, 270, (272, 272, 24)),
                                         (260, 130, 71, (75, 73, 131))])
def test_linear_writes_its_outputs_alone(P, framed, M, N, K, pitch, pre, res, dres, dtype):
    """Rows that end inside 16 bytes, from 16-byte boundaries: what follows them in the
    buffer (other columns of a wider matrix) stays."""
    check_linear(P, M, N, K, dtype, act="gelu", pact="relu" if dres else "none", pre=pre, res=res, dres=dres,
                 pitch=pitch, seed=M)
    framed()


@pytest.mark.parametrize("act,pact,res,dres,pre", [("relu", "relu", False, False, False), ("none", "none", False, True, False),
                                                   ("gelu", "silu", True, True, True)])
def test_linear_with_many_tiles_a_pair_writes_its_outputs_alone(P, framed, act, pact, res, dres, pre):
    check_linear(P, 19500, 1001, 998, "bf16", act=act, pact=pact, res=res, dres=dres, pre=pre,
                 pitch=(1000, 1000, 1008), seed=3)
    framed()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layernorm_and_scan_write_their_outputs_alone(P, framed, dtype):
    framed.front = 0      # (check_ln looks between rows from the buffer's start on)
    for M, D, pitch in [(19, 61, 64), (333, 1397, 1400), (70, 4099, 4104), (5000, 33, 35), (700, 8203, 8208), (9, 7, None)]:
        check_ln(P, M, D, dtype, pitch=pitch, seed=D)
    framed.front = 64
    for T, N, H, pitch in [(1, 9, 61, 184), (7, 5, 33, 104), (140, 3, 61, 184), (1100, 2, 31, 96), (33, 4, 130, None)]:
        check_scan(P, T, N, H, dtype, seed=T, pitch=pitch)
    framed()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pitch", [(1, 753, 21, (24, 24, 760)), (38, 1, 1889, (1896, 1896, 8)), (1, 1, 14, (16, 16, 8)),
                                         (1, 468, 1152, (1152, 1152, 472)), (300, 1, 45, (48, 48, 8)),
                                         (1, 244, 201, (208, 203, 246)), (1, 1397, 1001, None)])
def test_linear_of_single_rows(P, framed, M, N, K, pitch, dtype):
    """One row has no pitch of its own: the workspace of whichever is named is enough."""
    check_linear(P, M, N, K, dtype, act="gelu", pact="silu", dres=True, pitch=pitch, seed=N)
    framed()
