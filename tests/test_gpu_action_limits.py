"""Log-probability, entropy and policy loss at the limits of their plans: the longest rows.
Bounds as in test_gpu_action.py."""
import numpy as np
import pytest

import _action_ref as A
from test_gpu_action import P, flags, ints, make, within_inf  # noqa: F401
from test_gpu_trunk_ops import dev, f64, out, tdt, within

pytestmark = pytest.mark.gpu
KL, ENT = 0.3, 0.05


def loss(P, l, g, c, scale, mask=None, ref=True):
    """(logp, entropy, stats); dlogits go to g."""
    M = l.shape[0]
    lp, H, st = out((M,)), out((M,)), out((8,))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    P.ppo_action_loss_grad(l, ints(c["a"]), dev(c["old"]), dev(c["adv"]), g, scale,
                           logp_ref=dev(c["ref"]) if ref else None, weight=dev(c["weight"]), mask=mask, clip_low=0.2,
                           clip_high=0.28, kl_coef=KL, ent_coef=ENT, logp=lp, entropy=H, stats=st, work=work)
    return lp, H, st


def close(got, c, l64, dtype, scale, times=1):
    """Against the formula, every row `times` times over."""
    g, lp, H, st = got
    z, rg, b_g, rs, b_s = A.policy_loss(l64, c["a"], c["old"], c["adv"], np.float32(scale), c["ref"], c["weight"],
                                        c["mask"], 0.2, 0.28, KL, ENT)
    for k in range(times):
        part = slice(k * len(l64), (k + 1) * len(l64))
        within_inf(lp[part], z["logp"], z["b_logp"], "logp")
        within(H[part], z["H"], z["b_H"], "entropy")
        within(g[part], rg, b_g + A.HALF[dtype] * np.abs(rg) + 4 * A.U * np.abs(rg) + 1e-38, "dlogits")
    within(st, times * rs, times * (b_s + 4 * A.U * np.abs(rs) + 4 * A.U * (np.abs(rs[1:4]).sum())), "stats")


# 65,537 pieces of 16 bytes hold such a row where it is fp32 and starts between two of them
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("times", [1, 80])       # few rows, and one for each SM
@pytest.mark.parametrize("V,pitch,out_pitch", [(262137, 262137, 262137), (262140, 262141, 262141),
                                               (262141, 262141, 262141), (262143, 262143, 262144),
                                               (262142, 262144, 262143), (262144, 262145, 262147)])
def test_the_longest_rows(P, V, pitch, out_pitch, times, masked):
    import torch
    c = make(2, V, "f32", V, masked)
    M = 2 * times
    many = dict(c, **{k: np.tile(c[k], times) for k in ("a", "old", "adv", "ref", "weight")})
    l = torch.zeros(M, pitch, device="cuda")[:, :V]
    l.copy_(c["l"].repeat(times, 1))
    room = torch.full((M * out_pitch + 64,), 7.0, device="cuda")
    g = room[1:1 + M * out_pitch].view(M, out_pitch)[:, :V]
    g.fill_(float("nan"))
    lp, H, st = loss(P, l, g, many, 0.5, flags(np.tile(c["mask"], (times, 1))) if masked else None)
    close((g, lp, H, st), c, f64(c["l"]), "f32", 0.5, times)
    assert (room[0] == 7) and (room[1 + M * out_pitch:] == 7).all()
    if out_pitch > V:
        assert (torch.as_strided(room, (M, out_pitch - V), (out_pitch, 1), 1 + V) == 7).all()
