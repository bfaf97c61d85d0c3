"""A gated trunk, a head over many actions, the policy loss and the clip, run together
as they train, against 64-bit autograd of their formulas.

fp32 bounds: an output passes about twenty sums of up to 300 terms, forward and
backward, each off by 8 u (sqrt(n) + 8) of its magnitudes at most (u = 2^-24):
4e-4 of the largest element is ten times their sum.  bf16: every tensor
between two operators is rounded once, by 2^-8 at most and in root mean square by
2^-9 / sqrt(3) of an element's size: of the 8 of a block forward, as many
backward, and the head's 3, over one block sqrt(19) 2^-9 / sqrt(3) = 5e-3 of the
norm; the loss's slope is steep in the log-probability (a ratio multiplies its error
by up to e^0.5, the KL term adds as much), so 5e-2 is allowed."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
LOSS = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.2, ent_coef=0.05)


def build(T, N, D, H, F, V, dtype, act="silu", blocks=1):
    import torch
    from policy_rl_gb300.trunk import ActionHead, GradClip, RecurrentTrunk
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    M = T * N
    trunk = RecurrentTrunk(T, N, D, H, F, blocks=blocks, dtype=dtype, act=act, generator=g, gated=True)
    head = ActionHead(M, D, V, dtype=dtype, generator=g)
    for part in (trunk, head):
        for v in part.params.values():
            if v.dim() == 1:
                v += 0.2 * torch.randn(v.shape, generator=g, device="cuda")
        part.load_params()
    head.params["W"] *= 10
    head.load_params()
    made = dict(x=torch.randn(T, N, D, generator=g, device="cuda").to(dtype),
                done=(torch.rand(T, N, generator=g, device="cuda") < 0.05).float(),
                action=torch.randint(0, V, (M,), generator=g, device="cuda").to(torch.int32),
                adv=torch.randn(M, generator=g, device="cuda"),
                mask=torch.rand(M, V, generator=g, device="cuda") < 0.7,
                weight=torch.rand(M, generator=g, device="cuda"))
    rows = torch.arange(M, device="cuda")
    made["mask"][rows, made["action"].long()] = True
    made["action"][rows % 9 == 8] = -1
    return trunk, head, GradClip(trunk, head), made


def reference(trunk, head, made, old=None, ref=None):
    """Log-probabilities and, with old and ref, the loss and all gradients by autograd in 64 bits."""
    import torch
    par = {k: (trunk._w[k] if k in trunk._w else v).double().clone().requires_grad_(True)
           for k, v in trunk.params.items()}
    hw, hb = head._w.double().clone().requires_grad_(True), head.params["b"].double().clone().requires_grad_(True)
    x = made["x"].double().clone().requires_grad_(True)
    fn = {2: torch.nn.functional.silu, 3: lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[trunk.act]
    y = x
    for b in range(trunk.blocks):
        n = torch.nn.functional.layer_norm(y, (trunk.D,), par[b, "g1"], par[b, "c1"], trunk.eps)
        p = n @ par[b, "Wp"].T + par[b, "bp"]
        z, c = torch.sigmoid(p[..., :trunk.H]), p[..., trunk.H:]
        h, hs = torch.zeros_like(c[0]), []
        for s in range(trunk.T):
            if s:
                h = torch.where(made["done"][s - 1][:, None] != 0, 0.0, h)
            h = (1 - z[s]) * h + z[s] * c[s]
            hs.append(h)
        y = y + torch.stack(hs) @ par[b, "Wo"].T + par[b, "bo"]
        n = torch.nn.functional.layer_norm(y, (trunk.D,), par[b, "g2"], par[b, "c2"], trunk.eps)
        q = n @ par[b, "W1"].T + par[b, "b1"]
        y = y + (fn(q[..., :trunk.F]) * q[..., trunk.F:]) @ par[b, "W2"].T + par[b, "b2"]
    l = (y.reshape(head.M, head.D) @ hw.T + hb).masked_fill(~made["mask"], -torch.inf)
    lp = torch.log_softmax(l, 1)
    a = made["action"].long()
    kept = a >= 0
    at = lp.gather(1, a.clamp(min=0)[:, None])[:, 0]
    at = torch.where(kept, at, 0.0)
    if old is None:
        return at.detach()
    ent = -(lp.exp() * lp.masked_fill(~made["mask"], 0.0)).sum(1)
    adv, w = made["adv"].double(), made["weight"].double() * kept / head.M
    r = torch.exp(at - old)
    pg = -torch.minimum(r * adv, r.clamp(1 - LOSS["clip_low"], 1 + LOSS["clip_high"]) * adv)
    kl = torch.exp(ref - at) - (ref - at) - 1
    loss = (w * (pg + LOSS["kl_coef"] * kl - LOSS["ent_coef"] * ent)).sum()
    loss.backward()
    return {"loss": loss.detach(), "dx": x.grad, "W": hw.grad, "b": hb.grad, **{k: v.grad for k, v in par.items()}}


def step(trunk, head, clip, made, old, ref, stats, max_norm):
    y = trunk.forward(made["x"], made["done"])
    dy = head.loss_grad(y, made["action"], old, made["adv"], 1.0 / head.M, logp_ref=ref, weight=made["weight"],
                        mask=made["mask"], stats=stats, **LOSS)
    dx = trunk.backward(dy)
    return dx, clip.clip(max_norm)


def ready(trunk, head, made):
    import torch
    lp = reference(trunk, head, made)
    rows = torch.arange(head.M, device="cuda")
    off = torch.tensor([-0.5, -0.1, 0.02, 0.1, 0.5], device="cuda", dtype=torch.float64)[rows % 5]
    return (lp - off).float(), (lp + 0.3 * torch.sin(rows.double())).float()


SHAPES = [(1, 5, 24, 16, 40, 9), (37, 9, 72, 33, 100, 18), (20, 30, 64, 48, 136, 1001), (64, 20, 256, 128, 512, 5000)]


@pytest.mark.parametrize("T,N,D,H,F,V", SHAPES)
@pytest.mark.parametrize("kind,act", [("f32", "silu"), ("f32", "gelu"), ("bf16", "silu")])
def test_a_training_step(T, N, D, H, F, V, kind, act):
    import torch
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    trunk, head, clip, made = build(T, N, D, H, F, V, dtype, act)
    old, ref = ready(trunk, head, made)
    want = reference(trunk, head, made, old.double(), ref.double())
    stats = torch.empty(8, device="cuda")
    dx, norm = step(trunk, head, clip, made, old, ref, stats, 0.0)      # no clip
    trunk.check(), head.check()
    got = {"dx": dx, **head.grads, **trunk.grads}
    assert abs(float(stats[0] - want["loss"])) <= (2e-4 if kind == "f32" else 3e-2) * (abs(float(want["loss"])) + 1)
    for k, r in want.items():
        if k == "loss":
            continue
        d = got[k].double() - r
        err = float(d.abs().max() / r.abs().max()) if kind == "f32" else float(d.norm() / r.norm())
        assert err <= (4e-4 if kind == "f32" else 5e-2), (k, err)
    # the same step once more, clipped to half its norm
    total = sum(float((g.double() ** 2).sum()) for part in (trunk, head) for g in part.grads.values()) ** 0.5
    assert abs(float(norm) - total) <= 1e-5 * total
    before = {k: v.clone() for part in (trunk, head) for k, v in part.grads.items()}
    step(trunk, head, clip, made, old, ref, stats, total / 2)
    for part in (trunk, head):
        for k, v in part.grads.items():
            assert torch.allclose(v, before[k] * 0.5, rtol=1e-5, atol=0), k


def test_two_blocks_in_fp32():
    import torch
    trunk, head, clip, made = build(30, 6, 48, 32, 96, 50, torch.float32, blocks=2)
    old, ref = ready(trunk, head, made)
    want = reference(trunk, head, made, old.double(), ref.double())
    dx, _ = step(trunk, head, clip, made, old, ref, torch.empty(8, device="cuda"), 0.0)
    got = {"dx": dx, **head.grads, **trunk.grads}
    for k, r in want.items():
        if k != "loss":
            assert float((got[k].double() - r).abs().max() / r.abs().max()) <= 8e-4, k


def test_gated_acting_steps_equal_the_rollout():
    import torch
    trunk, _, _, made = build(20, 6, 48, 32, 96, 50, torch.float32)
    y = trunk.forward(made["x"], made["done"]).clone()
    state = trunk.state()
    for s in range(trunk.T):
        o = trunk.step(made["x"][s], state, made["done"][s - 1] if s else None)
        assert float((o - y[s]).abs().max()) <= 2e-4 * float(y.abs().max())


def test_a_training_step_in_a_graph():
    """Captured and replayed, beside an eager step of the same parts."""
    import torch
    trunk, head, clip, made = build(20, 30, 64, 48, 136, 1001, torch.bfloat16)
    old, ref = ready(trunk, head, made)
    stats = torch.empty(8, device="cuda")
    dx, norm = step(trunk, head, clip, made, old, ref, stats, 0.1)
    want = [t.clone() for t in (dx, norm, stats, *trunk.grads.values(), *head.grads.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, norm = step(trunk, head, clip, made, old, ref, stats, 0.1)
    for _ in range(2):
        for t in (dx, norm, stats, *trunk.grads.values(), *head.grads.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (dx, norm, stats, *trunk.grads.values(), *head.grads.values())):
            assert torch.equal(a, b)


def test_the_example_runs():
    import math
    import recall_actions
    rewards, norms, stats = recall_actions.main(["--updates", "3", "--N", "32", "--T", "12", "--width", "64",
                                                 "--actions", "50"])
    assert all(math.isfinite(v) for v in rewards + norms + stats) and all(n > 0 for n in norms)
