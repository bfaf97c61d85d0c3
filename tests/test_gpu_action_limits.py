"""Log-probability, entropy and policy loss at the limits of their plans: the longest rows,
logits far from 0 on both sides of where they are taken relative to the maximum,
finite logits of the type's lowest value.  Bounds as in test_gpu_action.py."""
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


def far_rows(M, V, base, dtype, seed):
    """Rows whose logits lie around `base`."""
    rng = np.random.default_rng(seed)
    return dev(base + 2 * rng.normal(size=(M, V)), dtype)


def check_rows(P, l, dtype, seed, scale=0.25):
    """The loss on l, with ratios as in make()."""
    M, V = l.shape
    c = make(M, V, dtype, seed, False)
    c["a"] = np.random.default_rng(seed).integers(0, V, M)
    c["a"][0] = int(f64(l)[0].argmax())
    base = A.softmax_rows(f64(l), c["a"])["logp"]
    c["old"] = (base - np.array([-0.5, -0.1, 0.02, 0.1, 0.5])[np.arange(M) % 5]).astype(np.float32)
    c["ref"] = (base + 0.3 * np.random.default_rng(seed).normal(size=M)).astype(np.float32)
    c["weight"] = np.ones(M, np.float32)
    g = out((M, V), dtype)
    close((g, *loss(P, l, g, c, scale)), c, f64(l), dtype, scale)


# lanes of a warp, a warp, blocks of 128 to 1,024 threads, clusters
LENGTHS = [(5, 9), (5, 300), (5, 1000), (5, 3000), (5, 9000), (3, 20001), (3, 70000), (2, 131072)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("base", [100, -1000, 5000, -30000, 60000, -60000])
@pytest.mark.parametrize("M,V", LENGTHS)
def test_logits_around_a_large_number(P, M, V, base, dtype):
    """What all logits share cancels, whichever warp a logit is in."""
    check_rows(P, far_rows(M, V, base, dtype, V), dtype, V)


@pytest.mark.parametrize("base", [65536, -65536, 65540.5, -65531.5, 65900, 120000, -120000, 140000])
@pytest.mark.parametrize("M,V", LENGTHS)
def test_logits_around_the_border(P, M, V, base):
    """Past |maximum| = 65,536 a warp takes fp32 logits relative to its own: rows of which
    some warps do so and others do not."""
    check_rows(P, far_rows(M, V, base, "f32", V), "f32", V)


@pytest.mark.parametrize("top,rest", [(65537.25, 65533.0), (65536.0, 65535.5), (-65533.0, -65537.25), (65580.0, 65530.0)])
@pytest.mark.parametrize("M,V", LENGTHS[3:] + [(160, 9000), (160, 40001)])
def test_one_warp_across_the_border(P, M, V, top, rest):
    """One logit of a row lies on the border's other side."""
    import torch
    rng = np.random.default_rng(V)
    l = dev(rest + 0.25 * rng.integers(-1, 1, (min(M, 4), V)))
    for i in range(l.shape[0]):
        l[i, (i * 7919 + V // 3) % V] = top
    check_rows(P, l.repeat(M // l.shape[0], 1) if M > 4 else l, "f32", V)


@pytest.mark.parametrize("base", [32512, 32768, -32768, 33024])
@pytest.mark.parametrize("M,V", [(5, 300), (5, 9000), (3, 20001), (2, 131072)])
def test_bf16_logits_around_the_border(P, M, V, base):
    rng = np.random.default_rng(V)
    check_rows(P, dev(base + 128.0 * rng.integers(-2, 3, (M, V)), "bf16"), "bf16", V)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 300, 1000, 5000, 20001, 131072])
def test_an_action_of_the_lowest_logit(P, V, dtype):
    """A finite logit counts, however low (masks are often made so): such an action's row is kept,
    with a ratio of 0; logp is the logit less the row's log-sum, or the lowest number."""
    import torch
    low = torch.finfo(tdt(dtype)).min
    rng = np.random.default_rng(V)
    l = dev(rng.normal(size=(7, V)), dtype)
    a = np.full(7, V - 2)
    for i, x in enumerate((low, low, -2.5e38, -1e31, low, -5e29, low)):
        l[i, V - 2] = x
    l[1, 0] = 1e6                   # rows taken relative to their maximum
    l[4, 0] = 2e38
    l[5, 0] = 6e29
    l[6, :] = low
    l[6, V - 2] = low / 2
    l64 = f64(l)
    z = A.softmax_rows(l64, a)
    want = np.maximum(z["logp"], -np.finfo(np.float32).max)
    lp, H = out((7,)), out((7,))
    P.ppo_action_logp(l, ints(a), logp=lp, entropy=H)
    within(lp, want, 4 * A.U * np.abs(want) + z["b_logp"] * (np.abs(want) < 1), "logp")
    within(H, z["H"], z["b_H"], "entropy")
    # the loss: an advantage of 0 leaves the entropy's gradient, the same as for another action
    zero, one = dev(np.zeros(7)), dev(np.ones(7))
    other = ints([1] * 7)
    got, st = [], out((8,))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    for act in (ints(a), other):
        g = out((7, V), dtype)
        P.ppo_action_loss_grad(l, act, zero, zero, g, 0.5, ent_coef=ENT, stats=st, work=work)
        got.append(g)
        assert float(st[7]) == 0 and float(st[6]) == 3.5
        assert abs(float(st[3]) - 0.5 * z["H"].sum()) <= 0.5 * z["b_H"].sum() + 16 * A.U * z["H"].sum()
    assert torch.isfinite(got[0]).all() and torch.equal(got[0], got[1])
    # and an advantage that counts is multiplied by a ratio of 0 (row 6: of 1)
    g = out((7, V), dtype)
    P.ppo_action_loss_grad(l, ints(a), zero, one, g, 0.5, ent_coef=ENT, stats=st, work=work)
    assert torch.equal(g[:6], got[0][:6])
    # -inf alone means that there is no such action
    l[0, V - 2] = float("-inf")
    P.ppo_action_loss_grad(l, ints(a), zero, one, g, 0.5, ent_coef=ENT, stats=st, work=work)
    assert float(st[7]) == 1 and (g[0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [11, 29, 301, 5003])
def test_masks_inside_a_buffer(P, V, dtype):
    """Masks that start anywhere, between bytes that say something else."""
    import torch
    M = 5
    c = make(M, V, dtype, V, True)
    for at in range(1, 10):
        room = torch.full((M * V + 32,), at % 2, dtype=torch.uint8, device="cuda")
        mask = room[at:at + M * V].view(M, V)
        mask.copy_(flags(c["mask"]))
        g = out((M, V), dtype, V + at % 3)
        close((g, *loss(P, c["l"], g, c, 0.25, mask)), c, f64(c["l"]), dtype, 0.25)


@pytest.mark.parametrize("V", [5, 300, 5000, 131072])
def test_a_reference_without_its_term(P, V):
    """kl_coef = 0 with log-probabilities so far apart that e^y is no fp32 number: the KL estimate
    says so, the loss and its gradient are those without a reference."""
    import torch
    M = 4
    l = dev(np.random.default_rng(V).normal(size=(M, V)))
    l[:, 1] = -120.0
    a, adv, zero = ints([1] * M), dev([1.0, -1.0, 0.5, -2.0]), dev(np.zeros(M))
    old, ref = torch.empty(M, device="cuda"), dev([0.0, -1.0, -100.0, -130.0])
    P.ppo_action_logp(l, a, logp=old)
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    got = []
    for r in (None, ref):
        g, st = out((M, V)), out((8,))
        P.ppo_action_loss_grad(l, a, old, adv, g, 0.25, logp_ref=r, ent_coef=ENT, stats=st, work=work)
        got.append((g, st))
    assert torch.isfinite(got[1][0]).all() and torch.equal(got[0][0], got[1][0])
    assert torch.equal(got[0][1][[0, 1, 3, 4, 5, 6, 7]], got[1][1][[0, 1, 3, 4, 5, 6, 7]])
    assert torch.isinf(got[1][1][2])


@pytest.mark.parametrize("clip_high", [0.2, float("inf")])
@pytest.mark.parametrize("V", [5, 300, 5000, 131072])
def test_an_advantage_of_zero(P, V, clip_high):
    """It makes 0 of any ratio e^x, of those that are no fp32 number too: such rows have the entropy's
    gradient alone.  An infinite x stays what the formula makes of it."""
    import torch
    M = 5
    l = dev(np.random.default_rng(V).normal(size=(M, V)))
    a, zero = ints([1] * M), dev(np.zeros(M))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    same, far = torch.empty(M, device="cuda"), dev([-100.0, -700.0, -1e9, -3e38, 1e9])
    P.ppo_action_logp(l, a, logp=same)
    got = []
    for old in (same, far):
        g, st = out((M, V)), out((8,))
        P.ppo_action_loss_grad(l, a, old, zero, g, 0.25, clip_high=clip_high, ent_coef=ENT, stats=st, work=work)
        got.append((g, st))
    assert torch.isfinite(got[1][0]).all() and torch.equal(got[0][0], got[1][0])
    assert torch.equal(got[0][1][[0, 1, 2, 3, 6, 7]], got[1][1][[0, 1, 2, 3, 6, 7]]) and float(got[1][1][1]) == 0
    # (four ratios above every finite bound, one below)
    assert float(got[1][1][4]) == (0.25 * 5 if clip_high < 1 else 0.25)
    g = out((M, V))
    P.ppo_action_loss_grad(l, a, dev([-np.inf, 0, 0, 0, 0]), zero, g, 0.25, ent_coef=ENT)
    assert torch.isnan(g[0]).all() and torch.isfinite(g[1:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", [(16452, 5), (65536, 5), (100003, 5), (300007, 2), (1000003, 3), (40000, 30), (70001, 60),
                                 (9001, 300), (2003, 2000), (700, 9000)])
def test_sums_over_many_equal_rows(P, M, V, dtype):
    """Sums of equal terms, whose roundings do not cancel.  u = 2^-24: sums over a thread's rows and over
    blocks are compensated, and joined with their roundings kept (2 u each, 1 where a block's and the
    whole one are rounded): 6 u of a sum without signs; 8 u more for the terms' own products."""
    l = dev(np.broadcast_to(np.linspace(-1, 1, V), (M, V)), dtype)
    scale = np.float32(1.0 / M)
    z = A.softmax_rows(f64(l[:1]), [0])
    lp, H, st = out((M,)), out((M,)), out((8,))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    one = dev(np.ones(M))
    old = dev(np.full(M, z["logp"][0] - 0.1))
    P.ppo_action_loss_grad(l, ints(np.zeros(M)), old, one, out((M, V), dtype), scale, logp=lp, entropy=H, stats=st, work=work)
    total = float(scale) * M
    got = f64(st)
    assert got[7] == 0 and got[4] == 0 and abs(got[6] - total) <= 6 * A.U * total, got[6] / total - 1
    for k, term, own in ((3, z["H"][0], z["b_H"][0]), (1, -np.exp(float(z["logp"][0]) - f64(old)[0]), 2 * z["b_logp"][0])):
        assert abs(got[k] - total * term) <= total * (own + 14 * A.U * abs(term)), (k, got[k], total * term)
