"""The trunk operators' 64-bit reference: its gradients against central
differences and its scan against closed forms (CPU); argument refusals that
need no device."""
import ctypes

import numpy as np
import pytest

import _trunk_ref as R

EPS = 1e-5


def central(f, x, v, e=1e-6):
    return (f(x + e * v) - f(x - e * v)) / (2 * e)


def test_layernorm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    x, w = rng.normal(size=(5, 7)) + 2, rng.normal(size=(5, 7))
    ga, be = rng.normal(size=7), rng.normal(size=7)
    _, mean, rstd = R.layernorm(x, ga, be, EPS)
    dx, dg, db = R.layernorm_grad(w, x, ga, mean, rstd)
    for arg, grad, f in ((x, dx, lambda a: (R.layernorm(a, ga, be, EPS)[0] * w).sum()),
                         (ga, dg, lambda a: (R.layernorm(x, a, be, EPS)[0] * w).sum()),
                         (be, db, lambda a: (R.layernorm(x, ga, a, EPS)[0] * w).sum())):
        v = rng.normal(size=arg.shape)
        assert abs(central(f, arg, v) - (grad * v).sum()) < 1e-7


def test_scan_gradient_matches_differences():
    rng = np.random.default_rng(1)
    T, N, H = 9, 3, 4
    p, h0 = rng.normal(size=(T, N, 2 * H)), rng.normal(size=(N, H))
    w, wT = rng.normal(size=(T, N, H)), rng.normal(size=(N, H))
    done, done0 = (rng.random((T, N)) < 0.25).astype(float), np.array([1.0, 0, 0])

    def loss(pp, hh):
        hs, _ = R.scan(pp, hh, done, done0)
        return (hs * w).sum() + (hs[-1] * wT).sum()

    dp, dh0, _ = R.scan_grad(w, p, h0, done, done0, wT)
    vp, vh = rng.normal(size=p.shape), rng.normal(size=h0.shape)
    assert abs(central(lambda a: loss(a, h0), p, vp) - (dp * vp).sum()) < 1e-7
    assert abs(central(lambda a: loss(p, a), h0, vh) - (dh0 * vh).sum()) < 1e-7
    assert (dh0[0] == 0).all()          # cleared on entry


def test_scan_closed_form():
    # constant gate z and candidate c from h0: h_t = c + (1 - z)^(t + 1) (h0 - c)
    T, pz, c = 40, 0.3, 1.7
    p = np.empty((T, 1, 2))
    p[..., 0], p[..., 1] = pz, c
    h, _ = R.scan(p, np.array([[-2.0]]))
    a = 1 - R.sigmoid(pz)
    assert np.allclose(h[:, 0, 0], c + a ** np.arange(1, T + 1) * (-2.0 - c), atol=1e-12)


@pytest.mark.parametrize("name", ["none", "tanh", "relu", "silu", "gelu"])
def test_activation_slopes_match_differences(name):
    x = np.linspace(-6, 6, 121) + 0.013
    assert np.abs(central(lambda a: R.act(name, a), x, 1.0) - R.act_grad(name, x)).max() < 1e-8


def test_refusals_before_any_launch():
    from policy_rl_gb300 import _abi, build
    build.build()
    L = _abi.load()
    p, q = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
    INV, ALIGN = 1, 2
    ln = lambda dt=1, x=p, ldx=64, M=4, D=64, eps=1e-5, y=p, ldy=64: L.ppo_layernorm_forward(
        dt, x, ldx, M, D, p, p, eps, y, ldy, p, None)
    assert ln(dt=2) == ln(dt=-1) == ln(x=None) == ln(y=None) == INV
    assert ln(M=0) == ln(M=-1) == ln(D=0) == ln(ldx=63) == ln(ldy=63) == INV
    assert ln(eps=-1.0) == ln(eps=float("nan")) == ln(ldy=128) == INV     # in place, two pitches
    assert ln(x=q) == ln(y=q) == ALIGN
    sz = ctypes.c_size_t()
    assert L.ppo_layernorm_backward_workspace_bytes(0, 8, ctypes.byref(sz)) == INV
    assert L.ppo_layernorm_backward_workspace_bytes(7, 8, ctypes.byref(sz)) == 0
    need = sz.value
    assert need >= 2 * 8 * 4
    lb = lambda stats=p, dg=p, work=p, wb=need, dy=p: L.ppo_layernorm_backward(
        1, dy, 8, p, 8, 7, 8, p, stats, None, 0, ctypes.c_void_p(0x2000), 8, dg, p, work, wb, None)
    assert lb(stats=None) == lb(work=None) == lb(wb=need - 1) == lb(dy=None) == INV
    assert lb(work=q) == lb(dg=q) == ALIGN
    sf = lambda dt=0, P=p, ldp=16, T=3, N=2, H=8, h=p, ldh=8, h0=None: L.ppo_gated_scan_forward(
        dt, P, ldp, None, None, h0, T, N, H, h, ldh, None, None, None)
    assert sf(dt=7) == sf(P=None) == sf(h=None) == sf(T=0) == sf(N=0) == sf(H=0) == INV
    assert sf(ldp=15) == sf(ldh=7) == INV
    odd = ctypes.c_void_p(0x1002)
    assert sf(h0=odd) == sf(P=odd) == ALIGN
    sb = lambda carry=p, dp=p, lddp=16: L.ppo_gated_scan_backward(
        0, p, 8, p, 16, None, None, carry, None, 3, 2, 8, dp, lddp, None, None)
    assert sb(carry=None) == sb(dp=None) == sb(lddp=15) == INV
    assert sb(carry=odd) == sb(dp=odd) == ALIGN
    ws = lambda dt=1, M=5, N=6, K=7: L.ppo_linear_workspace_bytes(dt, M, N, K, 0, 0, 0,
                                                                  ctypes.byref(sz))
    assert ws(dt=3) == ws(M=0) == ws(N=0) == ws(K=0) == INV
    assert ws() == 0
    big = 1 << 40
    lf = lambda act=0, x=p, ldx=8, y=p, res=None, ldres=8, work=p, wb=big: L.ppo_linear_forward(
        1, x, ldx, p, 8, p, act, res, ldres, 5, 6, 7, y, 8, None, 0, work, wb, None)
    assert lf(act=4) == lf(act=-2) == lf(x=None) == lf(y=None) == lf(ldx=6) == INV
    assert lf(work=None) == lf(wb=16) == lf(res=p, ldres=16) == INV
    assert lf(x=q) == lf(work=q) == ALIGN
    ld = lambda act=0, pre=p: L.ppo_linear_backward_data(1, p, 8, p, 8, pre, 8, act, None, 0, 5, 6, 7,
                                                         p, 8, p, 16, None)
    assert ld(pre=None) == ld() == INV
    assert L.ppo_linear_backward_weight(1, p, 8, p, 8, 5, 6, 7, None, None, 0, p, big, None) == INV
    assert L.ppo_linear_backward_weight(1, p, 8, q, 8, 5, 6, 7, p, None, 0, p, big, None) == ALIGN
    assert L.ppo_work_status(None, None) == INV and L.ppo_work_status(q, None) == ALIGN
