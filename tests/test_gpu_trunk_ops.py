"""The recurrent trunk's operators on the GPU against the 64-bit reference.

Bounds are derived, not fitted.  u = 2^-24, U = 2^-9 (bf16).  A result rounded
to bf16 is off by at most U |y| for the rounding (2 U |y| is allowed) plus what
fp32 lost before it; a sum of n fp32 terms by c sqrt(n) u sum|terms| (random
rounding errors; c = 8), and on the tensor cores by (n / 16 + 8) 2^-23 sum|terms|
(one truncation a 16-term step)."""
import numpy as np
import pytest

import _trunk_ref as R
from _gpu import host

pytestmark = pytest.mark.gpu
U32, U16 = R.U32, R.U16


@pytest.fixture(scope="module")
def P():
    import policy_rl_gb300
    return policy_rl_gb300


def tdt(dtype):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]


def dev(x, dtype="f32", pitch=None):
    """x on the device, with rows of `pitch` elements where given."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(tdt(dtype))
    if pitch is None:
        return t
    big = torch.full((*t.shape[:-1], pitch), 7.0, dtype=t.dtype, device="cuda")
    big[..., :t.shape[-1]] = t
    return big[..., :t.shape[-1]]


def out(shape, dtype="f32", pitch=None):
    import torch
    big = torch.full((*shape[:-1], pitch or shape[-1]), float("nan"), dtype=tdt(dtype), device="cuda")
    return big[..., :shape[-1]]


def f64(t):
    return host(t.float()).astype(np.float64)


def within(x, ref, bound, what):
    err = np.abs(f64(x) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err):.3g} at "
                           f"{np.argwhere(bad)[0]}, bound there {np.broadcast_to(bound, err.shape)[tuple(np.argwhere(bad)[0])]:.3g}")


def rounding(dtype, ref):
    return (2 * U16 if dtype == "bf16" else 0) * np.abs(ref)


# ---- layer norm ------------------------------------------------------------------
LN_SHAPES = [(1, 1), (1, 512), (3, 7), (5, 16), (64, 512), (33, 64), (257, 100), (129, 256), (77, 513),
             (40, 1000), (31, 1397), (9, 4104), (5, 5001), (3, 8192), (4, 10008), (2, 20001), (2500, 24)]


def ln_inputs(M, D, dtype, seed, pitch=None):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, D)) * rng.uniform(0.5, 4, (M, 1)) + rng.normal(size=(M, 1))
    x = dev(x, dtype, pitch)
    ga, be = dev(1 + 0.2 * rng.normal(size=D)), dev(rng.normal(size=D))
    return rng, x, ga, be


def check_ln(P, M, D, dtype, pitch=None, res=True, params=True, seed=0):
    rng, x, ga, be = ln_inputs(M, D, dtype, seed, pitch)
    dy = dev(rng.normal(size=(M, D)), dtype, pitch)
    dres = dev(rng.normal(size=(M, D)), dtype, pitch) if res else None
    y, dx = out((M, D), dtype, pitch), out((M, D), dtype, pitch)
    st, dg, db = out((M, 2)), out((D,)), out((D,))
    work = out((P.ppo_layernorm_backward_workspace_bytes(M, D) // 4,))
    P.ppo_layernorm_forward(x, ga, be, y, stats=st)
    P.ppo_layernorm_backward(dy, x, ga, st, dx, dgamma=dg if params else None,
                             dbeta=db if params else None, dres=dres, work=work if params else None)
    xr, yr = f64(x), f64(dy)
    ry, mean, rstd = R.layernorm(xr, f64(ga), f64(be), 1e-5)
    # mean off by c sqrt(D) u mean|x|; a row's values, relative to its deviation, by that over sigma
    lost = 16 * U32 * (np.sqrt(D) + 8) * (np.abs(xr).mean(1) * rstd + 1)[:, None]
    within(st[:, 0], mean, 8 * U32 * (np.sqrt(D) + 8) * np.abs(xr).mean(1) + 1e-30, "mean")
    within(st[:, 1], rstd, 2 * lost[:, 0] * rstd, "rstd")
    within(y, ry, rounding(dtype, ry) + lost * (np.abs(ry) + np.abs(f64(ga)) + np.abs(f64(be))), "y")
    rdx, rdg, rdb = R.layernorm_grad(yr, xr, f64(ga), mean, rstd, None if dres is None else f64(dres))
    q = np.abs(yr * f64(ga))
    xh = np.abs((xr - mean[:, None]) * rstd[:, None])
    size = rstd[:, None] * (q + q.mean(1, keepdims=True) + (xh + 1) * (q * (xh + 1)).mean(1, keepdims=True))
    within(dx, rdx, rounding(dtype, rdx) + 2 * lost * (size + np.abs(rdx)), "dx")
    if params:
        n = 8 * U32 * (np.sqrt(M) + 8)
        within(dg, rdg, n * (np.abs(yr) * xh).sum(0) + (np.abs(yr) * lost * (xh + 1)).sum(0), "dgamma")
        within(db, rdb, n * np.abs(yr).sum(0), "dbeta")
    if pitch:   # nothing between the rows is written
        import torch
        for t in (y, dx):
            gap = torch.as_strided(t, (M, pitch - D), (pitch, 1), D)
            assert torch.isnan(gap[:-1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", LN_SHAPES)
def test_layernorm(P, M, D, dtype):
    check_ln(P, M, D, dtype, seed=M * 31 + D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,pitch", [(64, 72), (64, 67), (500, 512), (1000, 1001)])
def test_layernorm_strided_rows(P, D, pitch, dtype):
    check_ln(P, 19, D, dtype, pitch=pitch, seed=D)


def test_layernorm_optional_arguments(P):
    check_ln(P, 70, 96, "bf16", res=False)
    check_ln(P, 70, 96, "f32", params=False)
    rng, x, ga, be = ln_inputs(12, 40, "f32", 3)
    y = out((12, 40))
    P.ppo_layernorm_forward(x, None, None, y)
    within(y, R.layernorm(f64(x), 1.0, 0.0, 1e-5)[0], 1e-5, "no gamma, beta")


def test_layernorm_in_place(P):
    import torch
    _, x, ga, be = ln_inputs(1000, 512, "bf16", 5)
    y = torch.empty_like(x)
    st = out((1000, 2))
    P.ppo_layernorm_forward(x, ga, be, y, stats=st)
    dy, dres = torch.randn_like(x), torch.randn_like(x)
    dx = torch.empty_like(x)
    P.ppo_layernorm_backward(dy, x, ga, st, dx, dres=dres)
    d2 = dres.clone()
    P.ppo_layernorm_backward(dy, x, ga, st, d2, dres=d2)
    P.ppo_layernorm_backward(dy, x, ga, st, dy, dres=dres)
    P.ppo_layernorm_forward(x, ga, be, x)
    assert torch.equal(x, y) and torch.equal(d2, dx) and torch.equal(dy, dx)


def test_layernorm_constant_rows_and_large_mean(P):
    # a constant row: deviations 0, y = beta, rstd = 1/sqrt(eps)
    x = dev(np.full((3, 48), 1234.5))
    ga, be, y, st = dev(np.ones(48)), dev(np.arange(48.0)), out((3, 48)), out((3, 2))
    P.ppo_layernorm_forward(x, ga, be, y, stats=st)
    assert (host(y) == np.arange(48.0)).all() and np.allclose(host(st)[:, 1], 1e5 ** 0.5, rtol=1e-6)
    # a mean 1,000 times the deviation loses digits of x, not of the variance
    rng = np.random.default_rng(2)
    x = dev(1000 + rng.normal(size=(5, 600)))
    ga, be, y = dev(np.ones(600)), dev(np.zeros(600)), out((5, 600))
    P.ppo_layernorm_forward(x, ga, be, y)
    within(y, R.layernorm(f64(x), 1.0, 0.0, 1e-5)[0], 5e-4, "large mean")


def test_layernorm_nan_stays_in_its_row(P):
    _, x, ga, be = ln_inputs(70, 64, "bf16", 9)
    x[13, 5] = float("nan")
    x[41, 0] = float("inf")
    y = out((70, 64), "bf16")
    P.ppo_layernorm_forward(x, ga, be, y)
    bad = ~np.isfinite(f64(y)).all(1)
    assert list(np.flatnonzero(bad)) == [13, 41]


def test_layernorm_deterministic_and_on_another_stream(P):
    import torch
    _, x, ga, be = ln_inputs(5000, 512, "bf16", 11)
    dy = torch.randn_like(x)
    work = out((P.ppo_layernorm_backward_workspace_bytes(5000, 512) // 4,))
    got = []
    for s in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        y, st, dx, dg, db = (torch.empty_like(x), out((5000, 2)), torch.empty_like(x), out((512,)),
                             out((512,)))
        torch.cuda.synchronize()
        P.ppo_layernorm_forward(x, ga, be, y, stats=st, stream=s)
        P.ppo_layernorm_backward(dy, x, ga, st, dx, dgamma=dg, dbeta=db, work=work, stream=s)
        s.synchronize()
        got.append((y, st, dx, dg, db))
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], g))


def test_layernorm_past_32_bit_offsets(P):
    import torch
    M, D = 540000, 4096                     # 2.2e9 elements
    x = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    x[rows] = torch.randn(5, D, device="cuda").to(torch.bfloat16)
    ga, be = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    st = torch.empty(M, 2, device="cuda")
    P.ppo_layernorm_forward(x, ga, be, x, stats=st)      # in place
    y, mean, rstd = R.layernorm(0.0 * f64(x[rows]), 1.0, 0.0, 1e-5)
    got = f64(x[rows])
    assert np.abs(got.mean(1)).max() < 1e-3 and np.abs((got ** 2).mean(1) - 1).max() < 1e-2
    assert float(x[5:M // 2].abs().max()) == 0.0


# ---- gated scan -------------------------------------------------------------------
def scan_inputs(T, N, H, dtype, seed, pitch=None, done_p=0.05, shift=-1.0):
    rng = np.random.default_rng(seed)
    p = np.concatenate([1.5 * rng.normal(size=(T, N, H)) + shift, rng.normal(size=(T, N, H))], 2)
    p = dev(p, dtype, pitch)
    done = dev((rng.random((T, N)) < done_p).astype(np.float32))
    done0 = dev((rng.random(N) < 0.3).astype(np.float32))
    return rng, p, done, done0, dev(rng.normal(size=(N, H)))


def check_scan(P, T, N, H, dtype, seed, pitch=None, done_p=0.05, use=("done", "done0", "h0", "dhT"),
               shift=-1.0):
    rng, p, done, done0, h0 = scan_inputs(T, N, H, dtype, seed, pitch, done_p, shift)
    done, done0 = done if "done" in use else None, done0 if "done0" in use else None
    h0 = h0 if "h0" in use else None
    dh = dev(rng.normal(size=(T, N, H)), dtype, pitch and pitch - H)
    dhT = dev(rng.normal(size=(N, H))) if "dhT" in use else None
    h, hT = out((T, N, H), dtype, pitch and pitch - H), out((N, H))
    carry = out((P.ppo_scan_blocks(T), N, H))
    dp, dh0 = out((T, N, 2 * H), dtype, pitch), out((N, H))
    P.ppo_gated_scan_forward(p, h, h0=h0, done=done, done0=done0, hT=hT, carry=carry)
    P.ppo_gated_scan_backward(dh, p, carry, dp, done=done, done0=done0, dhT=dhT, dh0=dh0)
    n = lambda t: None if t is None else f64(t)
    rh, ent = R.scan(n(p), n(h0), n(done), n(done0))
    rdp, rdh0, g = R.scan_grad(n(dh), n(p), n(h0), n(done), n(done0), n(dhT))
    # a step's gate and product are off by some 20 u of what it adds, and each
    # rounding of the state by u of it, remembered for 1 / z steps (z > 0.01)
    S = max(np.abs(rh).max(), np.abs(ent).max(), np.abs(n(p)[..., H:]).max())
    G = np.abs(g).max()
    within(h, rh, rounding(dtype, rh) + 1e-5 * S, "h")
    within(hT, rh[-1], 1e-5 * S, "hT")
    within(carry, ent[::128], 1e-5 * S, "carry")
    within(dp, rdp, rounding(dtype, rdp) + 1e-5 * G * (1 + 2 * S), "dp")
    within(dh0, rdh0, 1e-5 * G, "dh0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", [
    (1, 1, 1), (1, 7, 33), (1, 300, 64), (2, 3, 8), (15, 2, 20), (16, 4, 64), (17, 1, 65),
    (32, 5, 30), (33, 40, 64), (63, 2, 96), (64, 3, 32), (127, 3, 64), (128, 2, 62), (129, 5, 32),
    (256, 1, 130), (300, 3, 37), (1000, 2, 64), (1025, 1, 16), (4097, 1, 32), (2000, 9, 7)])
def test_scan(P, T, N, H, dtype):
    check_scan(P, T, N, H, dtype, seed=T * 7 + N * 3 + H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", [(140, 37, 129), (130, 200, 256), (20, 700, 128), (5, 900, 130)])
def test_scan_many_channels(P, T, N, H, dtype):
    check_scan(P, T, N, H, dtype, seed=T)


@pytest.mark.parametrize("use", [(), ("done",), ("done0", "h0"), ("h0",), ("dhT",)])
def test_scan_optional_arguments(P, use):
    check_scan(P, 150, 3, 40, "bf16", seed=1, use=use)


@pytest.mark.parametrize("T", [1, 20, 200])
def test_scan_every_state_cleared(P, T):
    check_scan(P, T, 4, 48, "f32", seed=2, done_p=1.1)


@pytest.mark.parametrize("pitch", [3 * 64, 150, 141])
def test_scan_strided_rows(P, pitch):
    check_scan(P, 140, 3, 64, "bf16", seed=3, pitch=pitch)
    check_scan(P, 140, 3, 64, "f32", seed=3, pitch=pitch)


def test_scan_slow_gates_over_a_long_sequence(P):
    # z around 0.02: the state of one tile reaches many tiles on
    check_scan(P, 3000, 2, 64, "f32", seed=4, done_p=0.0, shift=-2.5)


def test_scan_cleared_state_does_not_leak(P):
    """NaN and infinities before a clear stay before it; gates at +-inf keep or
    replace the state."""
    T, N, H = 300, 2, 64
    _, p, _, _, h0 = scan_inputs(T, N, H, "f32", 6, done_p=0.0)
    done = np.zeros((T, N), np.float32)
    done[[40, 150, 260], 0] = 1
    p[10, 0, H + 3] = float("nan")            # candidate of step 10: poisons channel 3 up to step 40
    p[100, 0, H + 5] = float("inf")
    h0[1, 7] = float("nan")                   # environment 1 is cleared on entry
    p[200, 1, :H] = float("-inf")             # z = 0: the state stays (to the rounding of a join)
    p[201, 1, :H] = float("inf")              # z = 1: the state is the candidate
    done0 = dev(np.array([0.0, 1.0]))
    d = dev(done)
    h, hT, carry = out((T, N, H)), out((N, H)), out((3, N, H))
    P.ppo_gated_scan_forward(p, h, h0=h0, done=d, done0=done0, hT=hT, carry=carry)
    hh, (ref, _) = f64(h), R.scan(f64(p), f64(h0), done, [0, 1])
    assert np.array_equal(np.isfinite(hh), np.isfinite(ref))
    assert np.isnan(hh[10:41, 0, 3]).all() and np.isfinite(hh[41:, 0, 3]).all()
    assert np.isfinite(hh[:, 1]).all() and np.abs(hh[200, 1] - hh[199, 1]).max() <= 1e-5 * np.abs(hh[:, 1]).max()
    assert (hh[201, 1] == f64(p)[201, 1, H:]).all()
    fin = np.isfinite(ref)
    assert np.abs(hh[fin] - ref[fin]).max() < 1e-4
    # backward: a NaN that reaches a state after the clear does not pass it
    dh = np.ones((T, N, H), np.float32)
    dh[200, 0, 9] = np.nan
    p2 = dev(np.nan_to_num(f64(p), nan=0.1, posinf=1, neginf=-1))
    P.ppo_gated_scan_forward(p2, h, done=d, hT=hT, carry=carry)
    dp, dh0 = out((T, N, 2 * H)), out((N, H))
    P.ppo_gated_scan_backward(dev(dh), p2, carry, dp, done=d, dh0=dh0)
    bad = np.isnan(f64(dp)[:, 0, 9])
    assert bad[151:201].all() and not bad[:151].any() and not bad[201:].any()
    assert np.isfinite(f64(dh0)).all()


def test_scan_steps_one_by_one_equal_the_sequence(P):
    import torch
    T, N, H = 70, 33, 130
    _, p, done, done0, h0 = scan_inputs(T, N, H, "bf16", 8)
    h, hT = out((T, N, H), "bf16"), out((N, H))
    P.ppo_gated_scan_forward(p, h, h0=h0, done=done, done0=done0, hT=hT)
    state = h0.clone()
    step = out((1, N, H), "bf16")
    for t in range(T):
        P.ppo_gated_scan_forward(p[t:t + 1], step, h0=state, hT=state,
                                 done0=done0 if t == 0 else done[t - 1])
        # (a different order of the same fp32 sums, each rounded to bf16 once)
        assert (step[0].float() - h[t].float()).abs().max() < 2 * U16 * float(h[t].abs().max())
    assert float((state - hT).abs().max()) < 1e-5 * float(h.abs().max() + 1)
    assert torch.isfinite(state).all()


def test_scan_deterministic(P):
    import torch
    _, p, done, done0, h0 = scan_inputs(700, 3, 256, "bf16", 10)
    dh = torch.randn(700, 3, 256, device="cuda").to(torch.bfloat16)
    got = []
    for _ in range(3):
        h, hT, carry = out((700, 3, 256), "bf16"), out((3, 256)), out((6, 3, 256))
        dp, dh0 = out((700, 3, 512), "bf16"), out((3, 256))
        P.ppo_gated_scan_forward(p, h, h0=h0, done=done, done0=done0, hT=hT, carry=carry)
        P.ppo_gated_scan_backward(dh, p, carry, dp, done=done, done0=done0, dh0=dh0)
        got.append((h, hT, carry, dp, dh0))
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], g))


def test_scan_in_place_states_and_many_tiles(P):
    import torch
    T, N, H = 1500, 2, 96
    _, p, done, done0, h0 = scan_inputs(T, N, H, "f32", 12)
    h, hT, carry = out((T, N, H)), out((N, H)), out((P.ppo_scan_blocks(T), N, H))
    P.ppo_gated_scan_forward(p, h, h0=h0, done=done, done0=done0, hT=hT, carry=carry)
    s = h0.clone()
    P.ppo_gated_scan_forward(p, h, h0=s, done=done, done0=done0, hT=s)
    assert torch.equal(s, hT)
    dh, dhT, dp = torch.randn_like(h), torch.randn_like(hT), torch.empty_like(p)
    a, b = dhT.clone(), torch.empty_like(dhT)
    P.ppo_gated_scan_backward(dh, p, carry, dp, done=done, done0=done0, dhT=dhT, dh0=b)
    P.ppo_gated_scan_backward(dh, p, carry, dp, done=done, done0=done0, dhT=a, dh0=a)
    assert torch.equal(a, b)


def test_scan_past_32_bit_offsets(P):
    import torch
    T, N, H = 3, 12000, 32000                # 2.3e9 elements of p
    p = torch.zeros(T, N, 2 * H, dtype=torch.bfloat16, device="cuda")
    p[:, -3:] = torch.randn(T, 3, 2 * H, device="cuda").to(torch.bfloat16)
    h = torch.empty(T, N, H, dtype=torch.bfloat16, device="cuda")
    P.ppo_gated_scan_forward(p, h)
    ref, _ = R.scan(f64(p[:, -3:]))
    within(h[:, -3:], ref, 2 * U16 * np.abs(ref) + 1e-5 * 6, "h")
    assert float(h[:, :-3].abs().max()) == 0.0


# ---- linear ---------------------------------------------------------------------------
def prod_bound(dtype, a, b, n):
    """What a sum of n products loses, from the sum of their magnitudes."""
    mag = np.abs(a) @ np.abs(b)
    return ((n / 16 + 8) * 2.0 ** -23 if dtype == "bf16" else 8 * U32 * (np.sqrt(n) + 8)) * mag


def check_linear(P, M, N, K, dtype, act="none", pact="none", res=True, dres=False, pre=True, bias=True,
                 pitch=None, seed=0):
    """pitch: (x, w, dz / outputs) row pitches."""
    rng = np.random.default_rng(seed)
    codes = {"none": -1, "tanh": 0, "relu": 1, "silu": 2, "gelu": 3}
    px, pw, pz = pitch or (None, None, None)
    x, w = dev(rng.normal(size=(M, K)), dtype, px), dev(rng.normal(size=(N, K)) / np.sqrt(K), dtype, pw)
    b = dev(rng.normal(size=N)) if bias else None
    r = dev(rng.normal(size=(M, N)), dtype, pz) if res else None
    y, pr = out((M, N), dtype, pz), out((M, N), dtype, pz) if pre else None
    dz = dev(rng.normal(size=(M, N)), dtype, pz)
    pp = dev(1.5 * rng.normal(size=(M, K)), dtype, px) if pact != "none" else None
    dr = dev(rng.normal(size=(M, K)), dtype, px) if dres else None
    dx, dw, db = out((M, K), dtype, px), out((N, K)), out((N,))
    import torch
    nb = P.ppo_linear_workspace_bytes(M, N, K, tdt(dtype), px or 0, pw or 0, pz or 0)
    work = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    P.ppo_linear_forward(x, w, y, bias=b, act=codes[act], res=r, pre=pr, work=work)
    P.ppo_linear_backward_data(dz, w, dx, pre=pp, act=codes[pact], res=dr, work=work)
    P.ppo_linear_backward_weight(dz, x, dw, db=db, work=work)
    P.ppo_work_status(work)
    X, W, Z = f64(x), f64(w), f64(dz)
    rp = X @ W.T + (0 if b is None else f64(b))
    lost = prod_bound(dtype, X, W.T, K) + 2 * U32 * np.abs(rp)
    # the activations themselves: fp32 to a few u; tanh before a bf16 rounding
    # by the hardware approximation, 2^-10.9
    ea = 2.0 ** -10.5 if dtype == "bf16" else 16 * U32
    ra = R.act(act, rp)
    ry = ra + (0 if r is None else f64(r))
    within(y, ry, rounding(dtype, ry) + 1.2 * lost + (ea * np.abs(ra) + 16 * U32 * (np.abs(rp) + 1)
           if act != "none" else 0) + 4 * U32 * np.abs(ra), "y")
    if pre:
        within(pr, rp, rounding(dtype, rp) + lost, "pre")
    rd = Z @ W
    ld = prod_bound(dtype, Z, W, N)
    s = R.act_grad(pact, f64(pp)) if pp is not None else 1.0
    rdx = rd * s + (0 if dr is None else f64(dr))
    within(dx, rdx, rounding(dtype, rdx) + 1.2 * ld + 64 * U32 * np.abs(rd) + 4 * U32 * np.abs(rdx), "dx")
    within(dw, Z.T @ X, prod_bound(dtype, Z.T, X, M), "dw")
    within(db, Z.sum(0), 8 * U32 * (np.sqrt(M) + 8) * np.abs(Z).sum(0), "db")


LIN_SHAPES = [(1, 1, 1), (1, 16, 16), (1, 512, 256), (2, 7, 9), (3, 2048, 512), (17, 100, 72), (33, 512, 1024),
              (64, 64, 64), (65, 130, 200), (128, 256, 512), (129, 257, 65), (200, 1000, 1397), (255, 264, 136),
              (300, 72, 2056), (1000, 24, 40), (1111, 512, 256), (4100, 40, 520)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", LIN_SHAPES)
def test_linear(P, M, N, K, dtype):
    check_linear(P, M, N, K, dtype, act="gelu", pact="silu", dres=True, seed=M + N + K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "tanh", "relu", "silu", "gelu"])
@pytest.mark.parametrize("M", [5, 140])
def test_linear_activations(P, act, M, dtype):
    check_linear(P, M, 136, 88, dtype, act=act, pact=act, seed=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pitch", [(96, 80, 128), (77, 76, 105), (80, 75, 100)])
def test_linear_strided_rows(P, pitch, dtype):
    check_linear(P, 150, 100, 75, dtype, act="tanh", pact="gelu", dres=True, pitch=pitch, seed=5)
    check_linear(P, 9, 100, 75, dtype, act="tanh", pact="gelu", dres=True, pitch=pitch, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_optional_arguments(P, dtype):
    check_linear(P, 70, 48, 56, dtype, res=False, pre=False, bias=False)
    check_linear(P, 3, 48, 56, dtype, res=False, pre=False, bias=False)


@pytest.mark.parametrize("dtype,M,N,K", [("bf16", 6000, 512, 1024), ("bf16", 20011, 136, 264), ("f32", 3001, 300, 200)])
def test_linear_large(P, dtype, M, N, K):
    check_linear(P, M, N, K, dtype, act="gelu", pact="gelu", seed=6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [7, 3000])
def test_linear_weight_gradient_accumulates(P, M, dtype):
    import torch
    rng = np.random.default_rng(7)
    N, K = 136, 264
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, tdt(dtype)), dtype=torch.uint8, device="cuda")
    dz, x = dev(rng.normal(size=(M, N)), dtype), dev(rng.normal(size=(M, K)), dtype)
    one, oneb, two, twob = out((N, K)), out((N,)), out((N, K)), out((N,))
    P.ppo_linear_backward_weight(dz, x, one, db=oneb, work=work)
    two.fill_(3.0)
    twob.fill_(-2.0)
    P.ppo_linear_backward_weight(dz, x, two, db=twob, accumulate=True, work=work)
    assert torch.equal(two, one + 3.0) and torch.equal(twob, oneb - 2.0)


def test_linear_in_place_residual_and_determinism(P):
    import torch
    rng = np.random.default_rng(8)
    for M in (9, 700):
        x, w = dev(rng.normal(size=(M, 512)), "bf16"), dev(rng.normal(size=(256, 512)) / 23, "bf16")
        r = dev(rng.normal(size=(M, 256)), "bf16")
        work = torch.zeros(P.ppo_linear_workspace_bytes(M, 256, 512, x.dtype), dtype=torch.uint8,
                           device="cuda")
        y = torch.empty_like(r)
        P.ppo_linear_forward(x, w, y, res=r, work=work)
        again = torch.empty_like(r)
        P.ppo_linear_forward(x, w, again, res=r, work=work)
        P.ppo_linear_forward(x, w, r, res=r, work=work)
        assert torch.equal(y, again) and torch.equal(y, r)
        dz, dr = dev(rng.normal(size=(M, 256)), "bf16"), dev(rng.normal(size=(M, 512)), "bf16")
        a = torch.empty_like(dr)
        P.ppo_linear_backward_data(dz, w, a, res=dr, work=work)
        P.ppo_linear_backward_data(dz, w, dr, res=dr, work=work)
        assert torch.equal(a, dr)
        P.ppo_work_status(work)


def test_linear_nan_stays_in_its_row(P):
    import torch
    rng = np.random.default_rng(9)
    for M in (20, 300):
        x, w = dev(rng.normal(size=(M, 72)), "bf16"), dev(rng.normal(size=(40, 72)), "bf16")
        x[7, 3] = float("nan")
        y = out((M, 40), "bf16")
        work = torch.zeros(P.ppo_linear_workspace_bytes(M, 40, 72, x.dtype), dtype=torch.uint8, device="cuda")
        P.ppo_linear_forward(x, w, y, act=3, work=work)
        assert list(np.flatnonzero(~np.isfinite(f64(y)).all(1))) == [7]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 5, 4104), (2, 33, 2056), (3, 16, 7), (4, 1030, 520), (5, 9, 1032), (8, 1001, 300),
                                   (16, 64, 1024), (23, 40, 2051), (40, 24, 136)])
def test_linear_few_rows(P, M, N, K, dtype):
    check_linear(P, M, N, K, dtype, act="gelu", seed=11 + M)
    check_linear(P, M, N, K, dtype, act="silu", bias=False, res=False, pitch=(K + 3, K + 5, max(N, K) + 1), seed=12 + M)


@pytest.mark.parametrize("M", [1, 6, 200])
def test_linear_one_output_per_row(P, M):
    check_linear(P, M, 1, 260, "bf16", seed=13)
    check_linear(P, M, 1, 260, "f32", seed=13)


@pytest.mark.parametrize("pitch", [None, (645, 643, 650), (648, 641, 644)])
def test_linear_f32_in_planes(P, pitch):
    """Sizes that take the tensor cores."""
    check_linear(P, 700, 641, 639, "f32", act="tanh", pact="gelu", dres=True, pitch=pitch, seed=14)


def test_linear_f32_infinities_nan_and_what_rounds_to_infinity(P):
    """An element that bf16 rounds to an infinity, an infinity, a NaN, sums past
    fp32's range: as the fp32 product has them, in their rows alone."""
    import torch
    rng = np.random.default_rng(15)
    M, N, K = 700, 640, 640
    x, w = dev(rng.normal(size=(M, K))), dev(rng.normal(size=(N, K)) / 25)
    x[3, 5] = float("inf")
    x[9, 1] = float("nan")
    x[20] = 0.0
    x[20, 7] = 3.4e38           # bf16's largest is 3.39e38
    x[31] = 3.0e38
    w[:, 7] = w[:, 7].abs().clamp(max=0.5) + 0.01
    w[0] = 1.0                  # x[31] w[0] leaves fp32's range
    w[1, 5] = 0.0               # infinity times zero
    y = out((M, N))
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, x.dtype), dtype=torch.uint8, device="cuda")
    P.ppo_linear_forward(x, w, y, work=work)
    P.ppo_work_status(work)
    Y, X, W = f64(y), f64(x), f64(w)
    rest = np.setdiff1d(np.arange(M), [3, 9, 31])
    ref = X[rest] @ W.T
    within(y[torch.from_numpy(rest).cuda()], ref, prod_bound("f32", X[rest], W.T, K), "rows without special values")
    sign = np.sign(W[:, 5])
    assert np.isnan(Y[3, 1]) and (np.delete(Y[3], 1) == np.delete(sign, 1) * np.inf).all()
    assert np.isnan(Y[9]).all()
    assert Y[31, 0] == np.inf


def test_linear_f32_weight_gradient_with_infinities_and_nan(P):
    import torch
    rng = np.random.default_rng(16)
    M, N, K = 700, 640, 640
    dz, x = dev(rng.normal(size=(M, N))), dev(rng.normal(size=(M, K)))
    dz[3, 5] = float("inf")
    dz[4, 6] = float("nan")
    dz[5, 7], x[5] = 3.4e38, x[5].clamp(-0.5, 0.5)
    dw, db = out((N, K)), out((N,))
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, x.dtype), dtype=torch.uint8, device="cuda")
    P.ppo_linear_backward_weight(dz, x, dw, db=db, work=work)
    P.ppo_work_status(work)
    Z, X, W, B = f64(dz), f64(x), f64(dw), f64(db)
    rest = np.setdiff1d(np.arange(N), [5, 6])
    bound = prod_bound("f32", Z[:, rest].T, X, M)
    assert (np.abs(W[rest] - Z[:, rest].T @ X) <= bound).all()
    assert (np.abs(B[rest] - Z[:, rest].sum(0)) <= 8 * U32 * (np.sqrt(M) + 8) * np.abs(Z[:, rest]).sum(0)).all()
    assert (W[5] == np.sign(X[3]) * np.inf).all() and B[5] == np.inf
    assert np.isnan(W[6]).all() and np.isnan(B[6])


def test_linear_past_32_bit_offsets(P):
    import torch
    M, N, K = 1100000, 2048, 64             # 2.3e9 outputs
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, K, device="cuda").to(torch.bfloat16)
    w = (torch.randn(N, K, device="cuda") / 8).to(torch.bfloat16)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, x.dtype), dtype=torch.uint8, device="cuda")
    P.ppo_linear_forward(x, w, y, work=work)
    ref = f64(x[-5:]) @ f64(w).T
    within(y[-5:], ref, 2 * U16 * np.abs(ref) + 1e-5, "y")
    assert float(y[:-5].abs().max()) == 0.0
    dx = torch.empty_like(x)
    P.ppo_linear_backward_data(y, w, dx, work=work)
    dw = torch.empty(N, K, device="cuda")
    P.ppo_linear_backward_weight(y, x, dw, work=work)
    Y = f64(y[-5:])
    rdx = Y @ f64(w)
    within(dx[-5:], rdx, 2 * U16 * np.abs(rdx) + prod_bound("bf16", Y, f64(w), N), "dx")
    within(dw, Y.T @ f64(x[-5:]), prod_bound("bf16", Y.T, f64(x[-5:]), 64), "dw")
    P.ppo_work_status(work)


# ---- differences through the kernels themselves ------------------------------------------
def test_gradients_against_differences_of_the_forward_kernels(P):
    """(L(a + e v) - L(a - e v)) / 2e against <dL/da, v> in fp32: the
    differences are off by e^2 of the third derivative and by u |L| / e."""
    import torch
    e = 2e-2
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")

    def check(f, a, grad, what):
        v = rn(*a.shape)
        v /= v.norm()
        num = (f(a + e * v) - f(a - e * v)) / (2 * e)
        ana = float((grad.double() * v.double()).sum())
        assert abs(num - ana) < 2e-3 * float(grad.double().norm()), (what, num, ana)

    x, ga, be, w = rn(6, 40), 1 + 0.2 * rn(40), rn(40), rn(6, 40)
    y, st, dx, dg, db = (torch.empty_like(x), out((6, 2)), torch.empty_like(x), out((40,)), out((40,)))
    work = out((P.ppo_layernorm_backward_workspace_bytes(6, 40) // 4,))

    def ln(a, b, c):
        P.ppo_layernorm_forward(a, b, c, y, stats=st)
        return float((y.double() * w.double()).sum())
    ln(x, ga, be)
    P.ppo_layernorm_backward(w, x, ga, st.clone(), dx, dgamma=dg, dbeta=db, work=work)
    check(lambda a: ln(a, ga, be), x, dx, "layer norm x")
    check(lambda a: ln(x, a, be), ga, dg, "gamma")
    check(lambda a: ln(x, ga, a), be, db, "beta")

    T, N, H = 37, 2, 24
    p, h0, w, wT = rn(T, N, 2 * H), rn(N, H), rn(T, N, H), rn(N, H)
    done = (torch.rand(T, N, generator=g, device="cuda") < 0.1).float()
    h, hT, carry, dp, dh0 = (torch.empty_like(w), torch.empty_like(h0), out((1, N, H)),
                             torch.empty_like(p), torch.empty_like(h0))

    def sc(a, b):
        P.ppo_gated_scan_forward(a, h, h0=b, done=done, hT=hT, carry=carry)
        return float((h.double() * w.double()).sum() + (hT.double() * wT.double()).sum())
    sc(p, h0)
    P.ppo_gated_scan_backward(w, p, carry, dp, done=done, dhT=wT, dh0=dh0)
    check(lambda a: sc(a, h0), p, dp.clone(), "scan p")
    check(lambda a: sc(p, a), h0, dh0.clone(), "scan h0")

    # linear after an activation: x = silu(q), y = x W^T + b
    M, N, K = 11, 20, 28
    q, W, b, w = rn(M, K), rn(N, K), rn(N), rn(M, N)
    y, dq, dw, db = torch.empty_like(w), torch.empty_like(q), torch.empty_like(W), torch.empty_like(b)
    work = torch.zeros(P.ppo_linear_workspace_bytes(M, N, K, q.dtype), dtype=torch.uint8, device="cuda")
    silu = lambda t: t * torch.sigmoid(t)

    def li(a, B, c):
        P.ppo_linear_forward(silu(a), B, y, bias=c, work=work)
        return float((y.double() * w.double()).sum())
    P.ppo_linear_backward_data(w, W, dq, pre=q, act=2, work=work)
    P.ppo_linear_backward_weight(w, silu(q), dw, db=db, work=work)
    check(lambda a: li(a, W, b), q, dq, "linear q")
    check(lambda a: li(q, a, b), W, dw, "linear W")
    check(lambda a: li(q, W, a), b, db, "linear b")


# ---- the binding's refusals ----------------------------------------------------------------
def test_binding_refuses_wrong_tensors(P):
    import torch
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        P.ppo_layernorm_forward(x.half(), None, None, torch.empty_like(x).half())
    with pytest.raises(ValueError):
        P.ppo_layernorm_forward(x, torch.ones(7, device="cuda"), None, torch.empty_like(x))
    with pytest.raises(ValueError):
        P.ppo_layernorm_forward(x.t(), None, None, torch.empty(8, 4, device="cuda"))
    with pytest.raises(ValueError):
        P.ppo_gated_scan_forward(torch.zeros(2, 3, 8, device="cuda"), torch.zeros(2, 3, 5, device="cuda"))
    with pytest.raises(ValueError):
        P.ppo_linear_forward(x, torch.zeros(5, 9, device="cuda"), torch.zeros(4, 5, device="cuda"))
    with pytest.raises(P.PpoError):
        P.ppo_linear_forward(x, torch.zeros(5, 8, device="cuda"), torch.zeros(4, 5, device="cuda"))
    base = torch.zeros(100, device="cuda")
    with pytest.raises(P.PpoError):     # a base that is not 16-byte aligned
        P.ppo_layernorm_forward(base[1:33].view(4, 8), None, None, x)
