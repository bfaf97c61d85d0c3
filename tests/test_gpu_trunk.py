"""RecurrentTrunk: a whole pre-norm residual recurrent trunk against 64-bit
autograd of its formulas, its acting step against its rollout, and the example.

fp32 bounds: each output passes about ten sums of up to 300 terms a block, each
off by 8 u (sqrt(n) + 8) of its magnitudes at most (u = 2^-24), with gradients
as much again: 2e-4 of the largest element is ten times their sum.  bf16: every
tensor between two operators is rounded once (2^-9); of the 7 tensors a block
forward and as many backward, in root mean square over two blocks about
sqrt(28) 2^-9 / sqrt(3) = 6e-3 of the norm; 3e-2 is allowed."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def build(T, N, D, H, F, dtype, act="gelu", seed=3):
    import torch
    from policy_rl_gb300.trunk import RecurrentTrunk
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = RecurrentTrunk(T, N, D, H, F, blocks=2, dtype=dtype, act=act, generator=g)
    for k, v in t.params.items():       # norms and biases away from their start
        if v.dim() == 1:
            v += 0.2 * torch.randn(v.shape, generator=g, device="cuda")
    t.load_params()
    made = dict(x=torch.randn(T, N, D, generator=g, device="cuda").to(t.dtype),
                dy=torch.randn(T, N, D, generator=g, device="cuda").to(t.dtype),
                done=(torch.rand(T, N, generator=g, device="cuda") < 0.05).float(),
                done0=(torch.rand(N, generator=g, device="cuda") < 0.3).float(),
                h0=torch.randn(2, N, H, generator=g, device="cuda"),
                dhT=torch.randn(2, N, H, generator=g, device="cuda"))
    return t, made


def reference(t, made):
    """Outputs and gradients in 64 bits by autograd, of the rounded weights."""
    import torch
    par = {k: (t._w[k] if k in t._w else v).double().clone().requires_grad_(True) for k, v in t.params.items()}
    x = made["x"].double().clone().requires_grad_(True)
    h0 = made["h0"].double().clone().requires_grad_(True)
    fn = {-1: lambda v: v, 0: torch.tanh, 1: torch.relu, 2: torch.nn.functional.silu,
          3: lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[t.act]
    y, hT = x, []
    for b in range(t.blocks):
        n = torch.nn.functional.layer_norm(y, (t.D,), par[b, "g1"], par[b, "c1"], t.eps)
        p = n @ par[b, "Wp"].T + par[b, "bp"]
        z, c = torch.sigmoid(p[..., :t.H]), p[..., t.H:]
        h, hs = h0[b], []
        for s in range(t.T):
            gone = made["done0"] if s == 0 else made["done"][s - 1]
            h = torch.where(gone[:, None] != 0, 0.0, h)
            h = (1 - z[s]) * h + z[s] * c[s]
            hs.append(h)
        hT.append(h)
        y = y + torch.stack(hs) @ par[b, "Wo"].T + par[b, "bo"]
        n = torch.nn.functional.layer_norm(y, (t.D,), par[b, "g2"], par[b, "c2"], t.eps)
        y = y + fn(n @ par[b, "W1"].T + par[b, "b1"]) @ par[b, "W2"].T + par[b, "b2"]
    hT = torch.stack(hT)
    ((y * made["dy"].double()).sum() + (hT * made["dhT"].double()).sum()).backward()
    return {"y": y.detach(), "hT": hT.detach(), "dx": x.grad, "dh0": h0.grad, **{k: v.grad for k, v in par.items()}}


def run(t, made):
    import torch
    hT, dh0 = torch.empty_like(made["h0"]), torch.empty_like(made["h0"])
    y = t.forward(made["x"], made["done"], made["done0"], made["h0"], hT).clone()
    dx = t.backward(made["dy"], made["dhT"], dh0)
    t.check()
    return {"y": y, "hT": hT, "dx": dx, "dh0": dh0, **t.grads}


SHAPES = [(1, 5, 24, 16, 40), (37, 9, 72, 33, 100), (200, 3, 64, 48, 136), (140, 20, 256, 128, 512)]


@pytest.mark.parametrize("T,N,D,H,F", SHAPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_trunk_in_fp32(T, N, D, H, F, act):
    import torch
    t, made = build(T, N, D, H, F, torch.float32, act)
    ref, got = reference(t, made), run(t, made)
    for k, r in ref.items():
        err = float((got[k].double() - r).abs().max() / r.abs().max())
        assert err <= 2e-4, (k, err)


@pytest.mark.parametrize("T,N,D,H,F", SHAPES)
def test_trunk_in_bf16(T, N, D, H, F):
    import torch
    t, made = build(T, N, D, H, F, torch.bfloat16)
    ref, got = reference(t, made), run(t, made)
    for k, r in ref.items():
        err = float((got[k].double() - r).norm() / r.norm())
        assert err <= 3e-2, (k, err)


def test_acting_steps_equal_the_rollout_in_fp32():
    import torch
    t, made = build(30, 6, 48, 32, 96, torch.float32)
    hT = torch.empty_like(made["h0"])
    y = t.forward(made["x"], made["done"], made["done0"], made["h0"], hT).clone()
    state = made["h0"].clone()
    for s in range(t.T):
        o = t.step(made["x"][s], state, made["done0"] if s == 0 else made["done"][s - 1])
        assert float((o - y[s]).abs().max()) <= 2e-4 * float(y.abs().max())
    assert float((state - hT).abs().max()) <= 2e-4 * float(hT.abs().max())


def test_trunk_on_another_stream_and_in_a_graph():
    import torch
    t, made = build(20, 6, 64, 32, 96, torch.bfloat16)
    want = {k: v.clone() for k, v in run(t, made).items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    hT, dh0 = torch.empty_like(made["h0"]), torch.empty_like(made["h0"])
    y = t.forward(made["x"], made["done"], made["done0"], made["h0"], hT, stream=side)
    dx = t.backward(made["dy"], made["dhT"], dh0, stream=side)
    side.synchronize()
    for k, v in {"y": y, "hT": hT, "dx": dx, "dh0": dh0, **t.grads}.items():
        assert torch.equal(v, want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = t.forward(made["x"], made["done"], made["done0"], made["h0"], hT)
        dx = t.backward(made["dy"], made["dhT"], dh0)
    for v in (y, hT, dx, dh0, *t.grads.values()):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k, v in {"y": y, "hT": hT, "dx": dx, "dh0": dh0, **t.grads}.items():
        assert torch.equal(v, want[k]), k


def test_example_learns_to_remember():
    import recurrent_trunk
    first, last, worst = recurrent_trunk.main(["--steps", "150", "--N", "64", "--T", "48", "--width", "128"])
    assert last < 0.7 * first       # a trunk without a state stays at the target's variance
    assert worst < 3e-2
