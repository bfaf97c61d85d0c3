"""Trains a recurrent trunk to remember, then acts with it one step at a time.

Each environment shows a vector on the first step of an episode and noise
after it; the target of every step is that first vector.  Only a state that is
carried, and cleared when an episode ends, can give it.

    python examples/recurrent_trunk.py [--steps 300] [--width 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from policy_rl_gb300.trunk import RecurrentTrunk  # noqa: E402


def rollout(T, N, D, gen, dtype, episode=24):
    """x, done, target: episodes of about `episode` steps, the first vector of
    each marked by its last column."""
    dev = "cuda"
    done = (torch.rand(T, N, generator=gen, device=dev) < 1 / episode).float()
    first = torch.cat([torch.ones(1, N, device=dev), done[:-1]]) > 0
    shown = torch.randn(T, N, D, generator=gen, device=dev)
    shown[..., -1] = torch.where(first, 3.0, 0.0)
    x = torch.where(first[..., None], shown, 0.3 * torch.randn(T, N, D, generator=gen, device=dev))
    # the step at which the running episode began
    began = torch.where(first, torch.arange(T, device=dev)[:, None].expand(T, N), 0).cummax(0).values
    target = torch.gather(shown, 0, began[..., None].expand(T, N, D))[..., :8]
    return x.to(dtype), done, target


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--T", type=int, default=64)
    ap.add_argument("--N", type=int, default=256)
    ap.add_argument("--lr", type=float, default=3e-3)
    args = ap.parse_args(argv)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    T, N, D = args.T, args.N, args.width
    trunk = RecurrentTrunk(T, N, D, hidden=D, inner=4 * D, blocks=2, generator=gen)
    names = list(trunk.params)
    opt = torch.optim.Adam([trunk.params[k].requires_grad_(False) for k in names], lr=args.lr)

    first = loss = None
    for i in range(args.steps):
        x, done, target = rollout(T, N, D, gen, trunk.dtype)
        y = trunk.forward(x, done)
        miss = y[..., :8].float() - target
        loss = float(miss.square().mean())
        first = first if first is not None else loss
        dy = torch.zeros_like(y)
        dy[..., :8] = miss * (2 / miss.numel())
        trunk.backward(dy)
        for k in names:
            trunk.params[k].grad = trunk.grads[k]
        opt.step()
        trunk.load_params()
        if i % 50 == 0 or i == args.steps - 1:
            print(f"step {i:4d}  mean square error {loss:.4f}", flush=True)
    trunk.check()

    # the same policy, one acting step at a time, replayed from a CUDA graph
    x, done, target = rollout(T, N, D, gen, trunk.dtype)
    y = trunk.forward(x, done).clone()
    state, xin, cleared = trunk.state(), torch.zeros_like(x[0]), torch.zeros(N, device="cuda")
    trunk.step(xin, state, cleared)     # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = trunk.step(xin, state, cleared)
    state.zero_()
    worst = 0.0
    for t in range(T):
        xin.copy_(x[t])
        cleared.copy_(done[t - 1] if t else torch.zeros_like(cleared))
        graph.replay()
        worst = max(worst, float((out.float() - y[t].float()).norm() / y[t].float().norm()))
    trunk.check()
    print(f"acting step by step: off by {worst:.2e} of the rollout's outputs at worst")
    return first, loss, worst


if __name__ == "__main__":
    main()
