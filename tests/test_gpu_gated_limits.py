"""Gated linear layers at the ends of the types' ranges."""
import numpy as np
import pytest

import _action_ref as A
from test_gpu_gated import CODES, P, zeroed  # noqa: F401
from test_gpu_trunk_ops import dev, f64, out

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act,gate", [("relu", -3.0), ("silu", -300.0), ("gelu", -30.0), ("tanh", 30.0), ("none", 1.0)])
@pytest.mark.parametrize("M,N,J", [(1, 64, 32), (40, 61, 24), (700, 520, 128), (2000, 520, 136)])
def test_large_finite_pre_activations(P, M, N, J, act, gate, dtype):
    """A closed gate's slope is 0, or small, however large the other projection: their product with
    the gradient is representable where the gradient's with that projection is not."""
    import torch
    rng = np.random.default_rng(M)
    side = rng.integers(0, 2, (M, N)) * 2.0 - 1
    dz = dev(np.full((M, J), 1.0), dtype)
    w2 = dev(np.full((J, N), 1.0), dtype)                # d = J
    pre = torch.empty(M, 2 * N, device="cuda", dtype=dz.dtype)
    pre[:, :N] = gate
    top = 126 if act != "none" else 110                  # (the gate's own gradient is not an infinity)
    pre[:, N:] = dev(side * 2.0 ** top, dtype)
    dp, y = out((M, 2 * N), dtype), out((M, N), dtype)
    work = zeroed(P.ppo_gated_linear_workspace_bytes(M, N, 1, dz.dtype, J=J))
    P.ppo_gated_linear_backward_data(dz, w2, pre, dp, CODES[act], y, work)
    P.ppo_work_status(work)
    ry, sg, su = A.gated(act, np.float64(gate), side * 2.0 ** top)
    if act == "tanh":                                    # (1 - tanh^2 has no digits left there)
        sg = 4 * np.exp(-2 * gate) / (1 + np.exp(-2 * gate)) ** 2 * side * 2.0 ** top
    # (an exponential is off by 2 + 1.2 x its argument units in the last place, four at most of
    # them and of roundings beside it: 1e-4; bf16's rounding; the hardware's tanh)
    tol = 1e-4 + (A.HALF["bf16"] + 2.0 ** -11 if dtype == "bf16" else 0)
    for got, want in ((dp[:, :N], J * sg), (dp[:, N:], np.broadcast_to(J * su, (M, N))), (y, ry)):
        got = f64(got)
        want = np.where(np.abs(want) < 2.0 ** -120, 0.0, want)
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= tol * np.abs(want) + 2.0 ** -100).all()
