"""Trains a gated recurrent trunk with a head over many actions to name what it saw.

Each environment shows one of V symbols on the first step of an episode and
noise after it.  Every step the policy names a symbol: reward 1 for the one
shown, of those that the step allows.  One update per rollout: act, the clipped
policy loss with a KL term towards the policy at the start, the gradients clipped
to one norm, Adam.

    python examples/recall_actions.py [--updates 60] [--actions 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import policy_rl_gb300 as P  # noqa: E402
from policy_rl_gb300.trunk import ActionHead, GradClip, RecurrentTrunk  # noqa: E402


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--updates", type=int, default=60)
    ap.add_argument("--actions", type=int, default=16)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--T", type=int, default=32)
    ap.add_argument("--N", type=int, default=128)
    ap.add_argument("--epochs", type=int, default=2)
    args = ap.parse_args(argv)
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    T, N, D, V = args.T, args.N, args.width, args.actions
    M = T * N
    trunk = RecurrentTrunk(T, N, D, hidden=D, inner=2 * D, blocks=1, act="silu", gated=True, generator=gen)
    head = ActionHead(M, D, V, generator=gen)
    clip = GradClip(trunk, head)
    parts = [(part, list(part.params)) for part in (trunk, head)]
    opt = torch.optim.Adam([part.params[k] for part, names in parts for k in names], lr=1e-3)
    symbols = torch.randn(V, D, generator=gen, device=dev)
    logp_old, logp_ref, stats = (torch.empty(n, device=dev) for n in (M, M, 8))
    norms, rewards = [], []
    start = None
    for i in range(args.updates):
        done = (torch.rand(T, N, generator=gen, device=dev) < 1 / 16).float()
        first = torch.cat([torch.ones(1, N, device=dev), done[:-1]]) > 0
        shown = torch.randint(0, V, (T, N), generator=gen, device=dev)
        began = torch.where(first, torch.arange(T, device=dev)[:, None].expand(T, N), 0).cummax(0).values
        target = torch.gather(shown, 0, began).reshape(M)
        noise = 0.3 * torch.randn(T, N, D, generator=gen, device=dev)
        x = torch.where(first[..., None], symbols[shown], noise).to(trunk.dtype)
        # half of the actions are allowed, the right one always
        mask = torch.rand(M, V, generator=gen, device=dev) < 0.5
        mask[torch.arange(M, device=dev), target] = True
        logits = head.logits(trunk.forward(x, done)).float().masked_fill(~mask, float("-inf"))
        u = torch.rand(M, V, generator=gen, device=dev).clamp_(1e-9, 1 - 1e-7)
        action = (logits - torch.log(-torch.log(u))).argmax(1).to(torch.int32)
        reward = (action == target).float()
        rewards.append(float(reward.mean()))
        adv = (reward - reward.mean()) / (reward.std() + 1e-8)
        y = trunk.forward(x, done)
        head.logp(y, action, logp_old, mask=mask)
        start = start or [{k: part.params[k].clone() for k in names} for part, names in parts]
        now = [{k: part.params[k].clone() for k in names} for part, names in parts]
        for (part, names), kept in zip(parts, start):
            for k in names:
                part.params[k].copy_(kept[k])
            part.load_params()
        head.logp(trunk.forward(x, done), action, logp_ref, mask=mask)
        for (part, names), kept in zip(parts, now):
            for k in names:
                part.params[k].copy_(kept[k])
            part.load_params()
        for _ in range(args.epochs):
            y = trunk.forward(x, done)
            dy = head.loss_grad(y, action, logp_old, adv, 1.0 / M, logp_ref=logp_ref, mask=mask, kl_coef=1e-4,
                                ent_coef=1e-3, stats=stats)
            trunk.backward(dy)
            norms.append(clip.clip(0.5).clone())
            for part, names in parts:
                for k in names:
                    part.params[k].grad = part.grads[k]
            opt.step()
            for part, _ in parts:
                part.load_params()
        if i % 10 == 0 or i == args.updates - 1:
            s = stats.tolist()
            print(f"update {i:3d}  reward {rewards[-1]:.4f}  loss {s[0]:+.4f}  kl {s[2]:.4f}  entropy {s[3]:.3f}  "
                  f"clipped {s[4]:.3f}  gradient norm {float(norms[-1]):.3f}", flush=True)
    trunk.check()
    head.check()
    return rewards, [float(n) for n in norms], stats.tolist()


if __name__ == "__main__":
    main()
