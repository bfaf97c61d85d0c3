"""The 64-bit reference of the policy loss and the gated layer against differences (CPU)."""
import numpy as np
import pytest

import _action_ref as A


@pytest.mark.parametrize("masked", [False, True])
def test_loss_gradient_is_the_loss_s_difference(masked):
    rng = np.random.default_rng(3)
    M, V = 12, 7
    l = rng.normal(size=(M, V)) * 2
    a = rng.integers(0, V, M)
    mask = rng.random((M, V)) < 0.7 if masked else None
    if masked:
        mask[np.arange(M), a] = True
        mask[4, a[4]] = False
        mask[7] = False
    a[2] = -1
    base = A.softmax_rows(l, a, mask)["logp"]
    old = np.where(np.isfinite(base), base, 0) - np.array([-0.5, -0.1, 0.05, 0.5])[np.arange(M) % 4]
    kw = dict(old=old, adv=rng.normal(size=M), scale=0.3, ref=old + 0.2, weight=rng.random(M), mask=mask, kl=0.4,
              ent=0.2, hi=0.3)
    g = A.policy_loss(l, a, **kw)[1]
    h = 1e-6
    for i in range(M):
        for j in range(V):
            d = np.zeros_like(l)
            d[i, j] = h
            diff = (A.policy_loss(l + d, a, **kw)[3][0] - A.policy_loss(l - d, a, **kw)[3][0]) / (2 * h)
            assert abs(diff - g[i, j]) <= 1e-8, (i, j)
    assert (g[2] == 0).all() and (not masked or ((g[4] == 0).all() and (g[7] == 0).all()))


def test_rows_without_anything():
    z = A.softmax_rows(np.zeros((3, 4)), [1, -1, 9], np.array([[0, 0, 0, 0], [1, 1, 0, 0], [1, 1, 1, 1]]))
    assert np.isneginf(z["logp"][0]) and z["H"][0] == 0 and list(z["kept"]) == [False, False, False]
    assert z["logp"][1] == 0 and np.isclose(z["H"][1], np.log(2)) and z["logp"][2] == 0


@pytest.mark.parametrize("act", ["none", "tanh", "relu", "silu", "gelu"])
def test_gated_slopes(act):
    rng = np.random.default_rng(5)
    g, u, h = rng.normal(size=50) * 2, rng.normal(size=50), 1e-6
    y, dg, du = A.gated(act, g, u)
    assert np.allclose((A.gated(act, g + h, u)[0] - A.gated(act, g - h, u)[0]) / (2 * h), dg, atol=1e-7)
    assert np.allclose((A.gated(act, g, u + h)[0] - A.gated(act, g, u - h)[0]) / (2 * h), du, atol=1e-7)
