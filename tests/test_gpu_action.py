"""Log-probability, entropy and policy loss over any number of actions on the GPU
against the 64-bit reference; the bounds are derived in _action_ref."""
import numpy as np
import pytest

import _action_ref as A
from _gpu import host
from test_gpu_trunk_ops import dev, f64, out, tdt, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import policy_rl_gb300
    return policy_rl_gb300


def ints(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def flags(x, pitch=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    if pitch is None:
        return t
    big = torch.ones(t.shape[0], pitch, dtype=t.dtype, device="cuda")
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def make(M, V, dtype, seed, masked, pitch=None):
    """Inputs whose ratios lie on both sides of the clip and inside it, 0.05 from its
    borders (in the logarithm) at least."""
    rng = np.random.default_rng(seed)
    l = dev(rng.normal(size=(M, V)) * 2, dtype, pitch)
    a = rng.integers(0, V, M)
    mask = None
    if masked:
        mask = rng.random((M, V)) < 0.6
        mask[np.arange(M), a] = np.arange(M) % 11 != 10
        mask[np.arange(M) % 13 == 12] = False
    a[np.arange(M) % 7 == 6] = -1
    a[np.arange(M) % 17 == 16] = V
    base = A.softmax_rows(f64(l), a, mask)["logp"]
    base = np.where(np.isfinite(base), base, 0)
    old = (base - np.array([-0.5, -0.1, 0.02, 0.1, 0.5])[np.arange(M) % 5]).astype(np.float32)
    return dict(rng=rng, l=l, a=a, mask=mask, old=old, adv=rng.normal(size=M).astype(np.float32),
                ref=(base + 0.3 * rng.normal(size=M)).astype(np.float32),
                weight=(rng.random(M) * (rng.random(M) < 0.8)).astype(np.float32))


def run_loss(P, c, dtype, pitch=None, ref=True, weight=True, in_place=False, mask_pitch=None, out_pitch=None, **kw):
    M, V = c["l"].shape
    g = c["l"] if in_place else out((M, V), dtype, out_pitch or pitch)
    lp, H, st = out((M,)), out((M,)), out((8,))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    mask = None if c["mask"] is None else flags(c["mask"], mask_pitch)
    P.ppo_action_loss_grad(c["l"], ints(c["a"]), dev(c["old"]), dev(c["adv"]), g, 1.0 / M,
                           logp_ref=dev(c["ref"]) if ref else None, weight=dev(c["weight"]) if weight else None,
                           mask=mask, logp=lp, entropy=H, stats=st, work=work, **kw)
    return g, lp, H, st


def check_loss(P, M, V, dtype, seed=0, masked=False, pitch=None, ref=True, weight=True, kl=0.3, ent=0.05, **kw):
    c = make(M, V, dtype, seed, masked, pitch)
    logits = f64(c["l"])
    g, lp, H, st = run_loss(P, c, dtype, pitch, ref, weight, clip_low=0.2, clip_high=0.28, kl_coef=kl,
                            ent_coef=ent, **kw)
    z, rg, b_g, rs, b_s = A.policy_loss(logits, c["a"], c["old"], c["adv"], np.float32(1.0 / M),
                                        c["ref"] if ref else None, c["weight"] if weight else None, c["mask"], 0.2,
                                        0.28, kl, ent)
    # (the coefficients reach the kernel as fp32: 2^-24 of each term)
    within_inf(lp, z["logp"], z["b_logp"], "logp")
    within(H, z["H"], z["b_H"], "entropy")
    within(g, rg, b_g + A.HALF[dtype] * np.abs(rg) + 4 * A.U * np.abs(rg) + 1e-38, "dlogits")
    within(st, rs, b_s + 4 * A.U * np.abs(rs) + 4 * A.U * (np.abs(rs[1:4]).sum()), "stats")
    if c["mask"] is not None:
        assert (host(g.float())[~c["mask"]] == 0).all()
    return c, g


def within_inf(x, ref, bound, what):
    got = f64(x)
    assert (np.isneginf(got) == np.isneginf(ref)).all(), what
    ok = np.isfinite(ref)
    err = np.abs(got[ok] - ref[ok])
    assert (err <= bound[ok]).all(), (what, (err / bound[ok]).max())


SHAPES = [(1, 1), (1, 2), (5, 3), (33, 7), (64, 9), (257, 18), (40, 31), (9, 32), (70, 63), (21, 64), (19, 100), (12, 257),
          (30, 512), (7, 1001), (5, 1397), (6, 2048), (3, 2051), (4, 4100), (3, 8191), (2, 12345), (3, 16384), (2, 20001),
          (2, 32768), (2, 33001), (3, 50257), (1, 65536), (2, 70001), (1, 131072), (1, 200003), (2, 262144)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", SHAPES)
def test_loss(P, M, V, dtype):
    check_loss(P, M, V, dtype, seed=M * 31 + V)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", SHAPES[1:])
def test_loss_masked(P, M, V, dtype):
    check_loss(P, M, V, dtype, seed=M * 37 + V, masked=True)


# rows enough that the kernels are chosen for throughput: blocks of 128, 256 and 512 threads, two
# blocks a row, clusters of 2, 4 and 8 blocks of 1,024, two lanes a row
@pytest.mark.parametrize("M,V,dtype,masked",
                         [(160, 8000, "bf16", True), (700, 8001, "bf16", False), (161, 4000, "f32", True),
                          (170, 12345, "bf16", True), (900, 16000, "bf16", False), (170, 8004, "f32", False),
                          (333, 32768, "bf16", True), (320, 20011, "bf16", False), (160, 16383, "f32", True),
                          (170, 50257, "bf16", True), (153, 65536, "bf16", False), (155, 20001, "f32", True),
                          (160, 70001, "bf16", True), (160, 40000, "f32", False), (155, 140000, "bf16", True),
                          (153, 70004, "f32", False), (153, 132001, "f32", True),
                          (16385, 18, "f32", True), (20000, 31, "bf16", True), (16384, 8, "bf16", False),
                          (40000, 3, "f32", True), (70001, 2, "bf16", False), (5000, 60, "bf16", True),
                          (30001, 60, "bf16", True), (13001, 150, "bf16", True), (7000, 301, "bf16", False),
                          (3300, 900, "bf16", True), (30000, 33, "f32", False), (14000, 100, "f32", True),
                          (6500, 252, "f32", False), (3300, 500, "f32", True),
                          (3001, 250, "f32", True), (2000, 1000, "bf16", True), (2500, 2040, "bf16", False)])
def test_many_rows_of_every_length(P, M, V, dtype, masked):
    check_loss(P, M, V, dtype, seed=M + V, masked=masked)


@pytest.mark.parametrize("M", [1, 63, 1000, 5003])
def test_many_rows(P, M):
    check_loss(P, M, 18, "f32", seed=M, masked=True)
    check_loss(P, M, 129, "bf16", seed=M)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pitch,out_pitch,mask_pitch",
                         [(64, 72, None, 80), (61, 67, None, 61), (500, 512, 501, 503), (1000, 1001, 1000, 1003),
                          (5000, 5003, 5001, 5007), (40001, 40003, 40008, 40001)])
def test_pitches(P, V, pitch, out_pitch, mask_pitch, dtype):
    """Rows of any pitch, each matrix its own; nothing between rows is written."""
    import torch
    M = 21 if V < 40000 else 5
    _, g = check_loss(P, M, V, dtype, seed=V, masked=True, pitch=pitch, out_pitch=out_pitch, mask_pitch=mask_pitch)
    p = out_pitch or pitch
    if p > V:
        gap = torch.as_strided(g, (M, p - V), (p, 1), V)
        assert torch.isnan(gap[:-1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 61, 1000, 4099, 50257])
def test_offsets_inside_a_buffer(P, V, dtype):
    """Bases on their elements' alignment only; guards before and behind are kept."""
    import torch
    M = 6
    c = make(M, V, dtype, V, False)
    big = torch.full((M * V + 16,), 5.0, dtype=tdt(dtype), device="cuda")
    dst = torch.full((M * V + 16,), 7.0, dtype=tdt(dtype), device="cuda")
    # (the order of a row's sums follows its place in memory: against the formula, not bit by bit)
    _, rg, b_g, _, _ = A.policy_loss(f64(c["l"]), c["a"], c["old"], c["adv"], np.float32(1.0 / M), c["ref"], c["weight"])
    for at in (1, 3, 8):
        c2 = dict(c)
        c2["l"] = big[at:at + M * V].view(M, V)
        c2["l"].copy_(c["l"])
        g = dst[at:at + M * V].view(M, V)
        a = (ints(c["a"]), dev(c["old"]), dev(c["adv"]))
        P.ppo_action_loss_grad(c2["l"], *a, g, 1.0 / M, logp_ref=dev(c["ref"]), weight=dev(c["weight"]))
        within(g, rg, b_g + (A.HALF[dtype] + 4 * A.U) * np.abs(rg) + 1e-38, "dlogits")
        assert (dst[:at] == 7).all() and (dst[at + M * V:] == 7).all()
        dst.fill_(7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 100, 3000, 20001, 131072])
def test_in_place(P, V, dtype):
    import torch
    c = make(9, V, dtype, V, True)
    want = run_loss(P, c, dtype)
    got = run_loss(P, c, dtype, in_place=True)
    for x, y in zip(want, got):
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))


@pytest.mark.parametrize("M,V", [(20000, 7), (3000, 121), (1000, 1001), (700, 8001), (400, 20001), (200, 50257),
                                 (160, 70001)])
def test_in_place_many_odd_rows(P, M, V):
    """Neighbouring rows share 16 bytes at their ends, and are written while others are read."""
    import torch
    c = make(M, V, "bf16", V, False)
    want = run_loss(P, c, "bf16")
    got = run_loss(P, c, "bf16", in_place=True)
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("V", [18, 1000, 50257])
def test_logp_equals_the_loss_s(P, V):
    """The forward form gives the same numbers, whatever it is asked for."""
    import torch
    c = make(40, V, "bf16", V, True)
    _, lp, H, _ = run_loss(P, c, "bf16")
    lp2, H2, lp3, H3 = (out((40,)) for _ in range(4))
    mask = flags(c["mask"])
    P.ppo_action_logp(c["l"], ints(c["a"]), logp=lp2, entropy=H2, mask=mask)
    P.ppo_action_logp(c["l"], ints(c["a"]), logp=lp3, mask=mask)
    P.ppo_action_logp(c["l"], None, entropy=H3, mask=mask)
    assert torch.equal(lp, lp2) and torch.equal(lp, lp3) and torch.equal(H, H2) and torch.equal(H, H3)


def test_optional_arguments(P):
    check_loss(P, 50, 40, "f32", ref=False, weight=False, kl=0.0, ent=0.0)
    check_loss(P, 50, 40, "bf16", ref=False, weight=True, kl=0.7, ent=0.0)
    check_loss(P, 50, 40, "bf16", ref=True, weight=False, kl=0.0, ent=0.1)


@pytest.mark.parametrize("V", [9, 300, 5000, 131072])
def test_special_values(P, V):
    """Covered infinities and NaN do not matter; left-out rows and rows of weight 0 may
    hold anything beside their logits; uncovered NaN stay in their row."""
    import torch
    M = 8
    for dtype in ("f32", "bf16"):
        c = make(M, V, dtype, V, True)
        c["a"][:] = np.arange(M)
        c["mask"][:] = True
        c["mask"][:, V - 1] = False
        c["mask"][1, 1] = False                 # row 1: its action is not allowed
        c["mask"][2] = False                    # row 2: nothing is
        c["a"][3] = -5
        if V > 20:
            c["l"][5, 7] = float("-inf")        # allowed, of probability 0
        want = [t.clone() for t in run_loss(P, c, dtype)]
        hidden = c["l"].clone()
        for i, bad in enumerate((float("nan"), float("inf"), float("-inf"), torch.finfo(tdt(dtype)).min)):
            hidden[i::4, V - 1] = bad
            hidden[2, i::4] = bad
        odd = dict(c, l=hidden, old=c["old"].copy(), adv=c["adv"].copy(), ref=c["ref"].copy(),
                   weight=c["weight"].copy())
        for r in (1, 2, 3):
            odd["old"][r] = odd["adv"][r] = odd["ref"][r] = odd["weight"][r] = np.nan
        got = run_loss(P, odd, dtype)
        for x, y in zip(want, got):
            assert torch.equal(x, y)
        assert (got[0][1:4] == 0).all() and torch.isfinite(got[0]).all() and host(got[3])[7] == 3
        # weight 0: nothing else of the row's matters
        odd["weight"][4] = 0.0
        clean = [t.clone() for t in run_loss(P, odd, dtype)]
        odd["old"][4] = odd["adv"][4] = odd["ref"][4] = np.inf
        got = run_loss(P, odd, dtype)
        assert torch.equal(clean[0], got[0]) and torch.equal(clean[3], got[3]) and (got[0][4] == 0).all()
        # a NaN that is not covered
        nan = dict(odd, l=hidden.clone())
        nan["l"][6, 0] = float("nan")
        got = run_loss(P, nan, dtype)
        assert torch.isnan(got[1][6]) and torch.isnan(got[2][6])
        assert torch.isnan(got[0][6][torch.from_numpy(c["mask"][6]).cuda()]).all() and (got[0][6, V - 1] == 0).all()
        rest = [r for r in range(M) if r != 6]
        assert torch.equal(got[0][rest], clean[0][rest])


def test_large_logits(P):
    """Logits far apart, of the type's size, and rows that one action owns."""
    for dtype in ("f32", "bf16"):
        l = np.array([[1e30, 0, -1e30, 5], [-3e38, -3e38, -3e38, -3e38], [3e38, -3e38, 0, 0], [80, 0, 0, 0]])
        x = dev(l, dtype)
        lp, H = out((4,)), out((4,))
        P.ppo_action_logp(x, ints([0, 2, 0, 1]), logp=lp, entropy=H)
        assert np.allclose(host(lp), [0, -np.log(4), 0, -80], atol=1e-5)
        assert np.allclose(host(H), [0, np.log(4), 0, 0], atol=1e-5)


def test_differences(P):
    """The gradient against differences of the loss that the kernel itself returns."""
    c = make(6, 10, "f32", 4, True)
    g = host(run_loss(P, c, "f32", kl_coef=0.3, ent_coef=0.05)[0]).astype(np.float64)
    h = 2.0 ** -6
    for i, j in [(0, 1), (1, 4), (2, 9), (3, 0), (4, int(c["a"][4])), (5, 3)]:
        both = []
        for s in (h, -h):
            moved = dict(c, l=c["l"].clone())
            moved["l"][i, j] += s
            both.append(float(host(run_loss(P, moved, "f32", kl_coef=0.3, ent_coef=0.05)[3])[0]))
        # third-order remainder h^2 / 6 times a derivative of order 1 / M, and fp32 losses of order 1
        assert abs((both[0] - both[1]) / (2 * h) - g[i, j]) <= 4 * h * h + 8 * A.U / h


def test_offsets_past_32_bits(P):
    """Rows that start more than 2^32 elements into their buffer."""
    import torch
    M, V, pitch = 3, 1000, 1_600_000_001
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * (2 * pitch + V) * 2 + 2**30:
        pytest.skip("needs 20 GB")
    big = torch.zeros(2 * pitch + V, dtype=torch.bfloat16, device="cuda")
    l = big.as_strided((M, V), (pitch, 1))
    c = make(M, V, "bf16", 5, False)
    l.copy_(c["l"])
    _, rg, b_g, _, _ = A.policy_loss(f64(c["l"]), c["a"], c["old"], c["adv"], np.float32(1.0 / M), c["ref"], c["weight"])
    got = run_loss(P, dict(c, l=l), "bf16", in_place=True)
    within(got[0], rg, b_g + (A.HALF["bf16"] + 4 * A.U) * np.abs(rg) + 1e-38, "dlogits")


def test_an_infinite_ratio(P):
    """r = inf: a good action's slope is 0, as its surrogate is flat; a bad one's infinite."""
    import torch
    l, g, st = dev(np.zeros((3, 4))), out((3, 4)), out((8,))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    for adv, good in ((1.0, True), (-1.0, False)):
        P.ppo_action_loss_grad(l, ints([1, 2, 3]), dev([-200.0, 0.0, 0.0]), dev([adv, 0.0, 0.0]), g, 1.0, stats=st,
                               work=work)
        assert (g[1:] == 0).all()
        if good:
            assert (g[0] == 0).all() and abs(float(st[1]) + 1.2) < 1e-6
        else:
            assert not torch.isfinite(g[0]).all() and torch.isinf(st[1])


@pytest.mark.parametrize("M,V", [(300, 3001), (40, 131072), (200, 70001), (900, 40)])
def test_streams_graphs_and_determinism(P, M, V):
    import torch
    c = make(M, V, "bf16", 8, True)
    want = [t.clone() for t in run_loss(P, c, "bf16")]
    side = torch.cuda.Stream()
    a, old, adv, mask = ints(c["a"]), dev(c["old"]), dev(c["adv"]), flags(c["mask"])
    ref, w = dev(c["ref"]), dev(c["weight"])
    g, st = out((M, V), "bf16"), out((8,))
    work = out((P.ppo_action_loss_workspace_bytes() // 4,))
    torch.cuda.synchronize()
    kw = dict(logp_ref=ref, weight=w, mask=mask, stats=st, work=work)
    P.ppo_action_loss_grad(c["l"], a, old, adv, g, 1 / M, stream=side, **kw)
    side.synchronize()
    assert torch.equal(g, want[0]) and torch.equal(st, want[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.ppo_action_loss_grad(c["l"], a, old, adv, g, 1 / M, **kw)
    for _ in range(2):
        g.zero_(), st.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g, want[0]) and torch.equal(st, want[3])


def test_two_streams_at_once(P):
    """Calls that overlap, a workspace each."""
    import torch
    cs = [make(2000, 5001, "bf16", k, False) for k in range(2)]
    want = [[t.clone() for t in run_loss(P, c, "bf16")] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    made = [(ints(c["a"]), dev(c["old"]), dev(c["adv"]), dev(c["ref"]), dev(c["weight"]), out((2000, 5001), "bf16"),
             out((8,)), out((P.ppo_action_loss_workspace_bytes() // 4,))) for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, (a, old, adv, ref, w, g, st, work) in zip(cs, streams, made):
            P.ppo_action_loss_grad(c["l"], a, old, adv, g, 1 / 2000, logp_ref=ref, weight=w, stats=st, work=work,
                                   stream=s)
    torch.cuda.synchronize()
    for (first, _, _, stats), m in zip(want, made):
        assert torch.equal(first, m[5]) and torch.equal(stats, m[6])


def test_refusals(P):
    import torch
    c = make(4, 8, "f32", 1, False)
    a, v = ints(c["a"]), dev(c["old"])
    g = out((4, 8))
    ok = dict(logits=c["l"], action=a, logp_old=v, adv=v, dlogits=g, scale=1.0)
    for bad in (dict(clip_low=-0.1), dict(clip_high=float("nan")), dict(stats=out((8,))),
                dict(stats=out((8,)), work=out((16,)))):
        with pytest.raises(P.PpoError):
            P.ppo_action_loss_grad(**{**ok, **bad})
    for bad in (dict(action=a.long()), dict(action=a[:3]), dict(adv=v.double()), dict(dlogits=out((4, 9))),
                dict(mask=torch.ones(4, 8, device="cuda")), dict(mask=torch.ones(4, 7, dtype=torch.bool, device="cuda")),
                dict(logits=c["l"].half())):
        with pytest.raises(ValueError):
            P.ppo_action_loss_grad(**{**ok, **bad})
    with pytest.raises(P.PpoError):
        P.ppo_action_logp(c["l"], None, logp=v)
    wide = torch.empty(1, 262145, device="cuda")
    with pytest.raises(P.PpoError):
        P.ppo_action_logp(wide, None, entropy=out((1,)))
