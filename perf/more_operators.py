"""What is measured of the operators that learn and act over many actions.

A recurrent trunk feeds a head over any number of actions and learns by the
clipped policy loss; these operators belong to that step:

  action log-probability  log softmax of a row of logits at the row's action, and the
                      row's entropy, over the actions that a mask leaves;
  policy loss         the clipped surrogate with a KL term towards a reference policy
                      and the entropy, and the loss's gradient with respect to every logit;
  gated linear        y = act(x Wg^T + bg) * (x Wu^T + bu), and the gradient of its
                      pre-activations from that of the layer behind it;
  gradient norm       the 2-norm over many tensors, and the tensors clipped to it.

listed() and draw() give cases, prepare() their inputs, run() one pass: in the
plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where `own` is true, through the framework's entry points.  exact() computes the
same outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# codes of the framework's activations
ACTS = {"none": -1, "tanh": 0, "relu": 1, "silu": 2, "gelu": 3}
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715
CLIP_LOW, CLIP_HIGH, KL, ENT = 0.2, 0.28, 0.05, 0.01


def listed():
    return [
        # 64 agents of one acting step, 9 buttons of which some are not allowed: the call's latency
        dict(name="logp_step", op="logp", M=64, V=9, dtype="f32", mask=True),
        # one token of a large vocabulary while acting
        dict(name="logp_token", op="logp", M=1, V=131072, dtype="bf16", mask=False),
        # a minibatch of 65,536 rows over 18 joint actions, some not allowed, fp32
        dict(name="loss_small_f32", op="loss", M=65536, V=18, dtype="f32", mask=True, ref=False, weight=False),
        # 8,192 tokens of a vocabulary of 32,768, everything in the loss
        dict(name="loss_vocab", op="loss", M=8192, V=32768, dtype="bf16", mask=False, ref=True, weight=True),
        # an odd number of tokens of an odd vocabulary, with allowed actions: rows off every boundary
        dict(name="loss_odd", op="loss", M=1001, V=50257, dtype="bf16", mask=True, ref=True, weight=False),
        # one acting step through a gated up-projection
        dict(name="gated_token", op="gated", M=1, K=512, N=2048, J=512, dtype="bf16", act="silu", train=False),
        # 33 agents through a wide one: the weights have to be streamed
        dict(name="gated_serve", op="gated", M=33, K=4096, N=4096, J=4096, dtype="bf16", act="silu", train=False),
        # a minibatch of 32,768 rows of the trunk, trained
        dict(name="gated_train", op="gated", M=32768, K=512, N=2048, J=512, dtype="bf16", act="silu", train=True),
        # odd rows and widths, trained
        dict(name="gated_odd", op="gated", M=10007, K=1397, N=1001, J=1397, dtype="bf16", act="gelu", train=True),
        # the same operator in the framework's fp32 mode
        dict(name="gated_f32", op="gated", M=4999, K=512, N=1365, J=512, dtype="f32", act="silu", train=True),
        # the gradients of a small trunk, 26 tensors: latency
        dict(name="clip_small", op="clip", n=26, total=100000, dtype="f32", sizes=1, max_norm=0.5),
        # 300 tensors of a large model, bf16 and fp32, odd sizes among them
        dict(name="clip_large", op="clip", n=300, total=500000000, dtype="mixed", sizes=2, max_norm=1.0),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logp", "loss", "loss", "gated", "gated", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("logp", "loss"):
        V = _size(rng, 2, 131072)
        if rng.random() < 0.5:
            V = max(8, V // 8 * 8)
        M = max(1, min(_size(rng, 1, 65536), int((130e6 if dtype == "f32" else 260e6) / V)))
        c = dict(op=op, M=M, V=V, dtype=dtype, mask=rng.random() < 0.4)
        if op == "loss":
            c |= dict(ref=rng.random() < 0.5, weight=rng.random() < 0.5)
        return c
    if op == "gated":
        top = 2048 if dtype == "f32" else 4096
        K, N, J = (_size(rng, 16, top) for _ in range(3))
        if rng.random() < 0.7:
            K, N, J = (max(16, v // 8 * 8) for v in (K, N, J))
        M = max(1, min(_size(rng, 1, 32768), int((3.5e9 if dtype == "f32" else 3.4e10) / (max(K, J) * N))))
        return dict(op=op, M=M, K=K, N=N, J=J, dtype=dtype, act=rng.choice(["tanh", "relu", "silu", "gelu"]),
                    train=rng.random() < 0.6)
    n = _size(rng, 1, 1000)
    return dict(op="clip", n=n, total=_size(rng, max(n, 1000), 400000000),
                dtype=rng.choice(["f32", "bf16", "mixed"]), sizes=rng.randrange(1 << 30),
                max_norm=rng.choice([0.5, 1.0, 1e6]))


def _tensor_sizes(c):
    """n sizes that add up to the total: a few matrices hold most of it, vectors of any length beside
    them, one tensor in ten of an odd size."""
    r = random.Random(c["sizes"])
    w = [math.exp(r.gauss(0, 2)) for _ in range(c["n"])]
    f = c["total"] / sum(w)
    out = [max(1, int(v * f)) for v in w]
    return [v if r.random() < 0.1 else max(1, v // 8 * 8) for v in out]


def _tensor_dtypes(c):
    kinds = {"f32": ["f32"], "bf16": ["bf16"], "mixed": ["bf16", "bf16", "f32"]}[c["dtype"]]
    return [kinds[i % len(kinds)] for i in range(c["n"])]


def _flat(sizes, kinds, new):
    """Buffers by type, and a piece of them for each tensor, on 8 elements: clipped gradients lie in one
    buffer of each type, as an optimizer or a collective takes them.  new(kind, n) makes one, of zeros."""
    room = {}
    at = []
    for n, d in zip(sizes, kinds):
        at.append(room.get(d, 0))
        room[d] = at[-1] + (n + 7) // 8 * 8
    flat = {d: new(d, n) for d, n in room.items()}
    return flat, [flat[d][o:o + n] for n, d, o in zip(sizes, kinds, at)]


# ---- inputs ---------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    f32 = torch.float32

    def normal(*shape, scale=1.0, shift=0.0, dtype=f32):
        return (torch.randn(*shape, generator=g, device=dev) * scale + shift).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def empty(*shape, dtype=f32):
        return torch.empty(*shape, device=dev, dtype=dtype)

    s = {"case": case}
    if case["op"] == "clip":
        # gradients of unlike scale from tensor to tensor
        sizes, kinds = _tensor_sizes(case), _tensor_dtypes(case)
        s["grads"] = [normal(n, scale=10.0 ** (-3 + k % 3), dtype=DTYPES[d])
                      for k, (n, d) in enumerate(zip(sizes, kinds))]
        s["flat"], s["out"] = _flat(sizes, kinds, lambda d, n: torch.zeros(n, dtype=DTYPES[d], device=dev))
        s["norm"] = empty(1)
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "gated":
        M, K, N, J = case["M"], case["K"], case["N"], case["J"]
        s["x"] = normal(M, K, dtype=dt)
        s["w"] = normal(2 * N, K, scale=1.0 / math.sqrt(K), dtype=dt)
        s["b"] = normal(2 * N, scale=0.1)
        s["y"] = empty(M, N, dtype=dt)
        if case["train"]:
            s["pre"] = empty(M, 2 * N, dtype=dt)
            s["dz"] = normal(M, J, dtype=dt)
            s["w2"] = normal(J, N, scale=1.0 / math.sqrt(N), dtype=dt)
            s["pre_in"] = normal(M, 2 * N, dtype=dt)     # what a forward pass has left
            s["dp"], s["y2"] = empty(M, 2 * N, dtype=dt), empty(M, N, dtype=dt)
        return s
    M, V = case["M"], case["V"]
    s["logits"] = normal(M, V, scale=2.0, dtype=dt)
    rows = torch.arange(M, device=dev)
    s["action"] = (uniform(M) * V).to(torch.int32).clamp_(max=V - 1)
    s["mask"] = None
    if case["mask"]:
        s["mask"] = uniform(M, V) < 0.7
        # the action was taken, so it was allowed; but for a row in 61, and one in 67 allows nothing
        s["mask"][rows, s["action"].long()] = rows % 61 != 60
        s["mask"][rows % 67 == 66] = False
    s["logp"], s["entropy"] = empty(M), empty(M)
    if case["op"] == "logp":
        return s
    s["action"][rows % 53 == 52] = -1        # rows that only fill the batch
    lp = _logp_plain(s)[0]
    lp = torch.where(torch.isfinite(lp), lp, torch.zeros_like(lp))
    # old log-probabilities on both sides of the clip and inside it, never next to its border
    off = torch.tensor([-0.5, -0.1, 0.0, 0.1, 0.5], device=dev)[rows % 5]
    s["old"] = lp - off - 0.06 * (uniform(M) - 0.5)
    s["adv"] = normal(M)
    s["ref"] = lp + normal(M, scale=0.3) if case["ref"] else None
    s["weight"] = (uniform(M) < 0.8).to(f32) if case["weight"] else None
    s["dlogits"], s["stats"] = empty(M, V, dtype=dt), empty(8)
    return s


# ---- the framework's calls --------------------------------------------------------
def _work(s, nbytes):
    """The workspace that a program keeps beside its buffers (zeroed once)."""
    if "work" not in s:
        s["work"] = torch.zeros(max(16, nbytes()), dtype=torch.uint8, device="cuda")
    return s["work"]


def _run_own(s):
    import policy_rl_gb300 as P
    c = s["case"]
    if c["op"] == "clip":
        # what a program keeps of its gradients: the list of their places
        if "list" not in s:
            s["list"], s["list_out"] = P.TensorList(s["grads"]), P.TensorList(s["out"])
        work = _work(s, lambda: P.ppo_grad_norm_workspace_bytes(s["list"]))
        P.ppo_clip_grad_norm(s["list"], c["max_norm"], s["norm"], out=s["list_out"], work=work)
        return {"norm": s["norm"], **s["flat"]}
    if c["op"] == "gated":
        work = _work(s, lambda: P.ppo_gated_linear_workspace_bytes(
            c["M"], c["N"], c["K"], s["x"].dtype, J=c["J"] if c["train"] else 0))
        P.ppo_gated_linear_forward(s["x"], s["w"], s["y"], bias=s["b"], act=ACTS[c["act"]], pre=s.get("pre"),
                                   work=work)
        if not c["train"]:
            return {"y": s["y"]}
        P.ppo_gated_linear_backward_data(s["dz"], s["w2"], s["pre_in"], s["dp"], act=ACTS[c["act"]], y=s["y2"],
                                         work=work)
        return {k: s[k] for k in ("y", "pre", "dp", "y2")}
    if c["op"] == "logp":
        P.ppo_action_logp(s["logits"], s["action"], logp=s["logp"], entropy=s["entropy"], mask=s["mask"])
        return {"logp": s["logp"], "entropy": s["entropy"]}
    work = _work(s, P.ppo_action_loss_workspace_bytes)
    P.ppo_action_loss_grad(s["logits"], s["action"], s["old"], s["adv"], s["dlogits"], 1.0 / c["M"],
                           logp_ref=s["ref"], weight=s["weight"], mask=s["mask"], clip_low=CLIP_LOW,
                           clip_high=CLIP_HIGH, kl_coef=KL if c["ref"] else 0.0, ent_coef=ENT, logp=s["logp"],
                           entropy=s["entropy"], stats=s["stats"], work=work)
    return {k: s[k] for k in ("dlogits", "logp", "entropy", "stats")}


# ---- the plain form -----------------------------------------------------------------
def _act(name, v):
    if name == "tanh":
        return torch.tanh(v)
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    return 0.5 * v * (1 + torch.tanh(GELU_C * (v + GELU_A * v * v * v)))


def _dact(name, v):
    if name == "tanh":
        return 1 - torch.tanh(v) ** 2
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        q = torch.sigmoid(v)
        return q * (1 + v * (1 - q))
    t = torch.tanh(GELU_C * (v + GELU_A * v * v * v))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * v * v)


def _logp_plain(s):
    """(log-probability of the row's action: 0 where it has none, -inf where the action is not allowed;
    entropy: 0 where nothing is allowed; log-probabilities; probabilities)."""
    l = s["logits"].float()
    if s["mask"] is not None:
        l = torch.where(s["mask"], l, torch.full_like(l, -math.inf))
    top = l.max(1, keepdim=True).values
    some = torch.isfinite(top)
    l = l - torch.where(some, top, torch.zeros_like(top))
    e = torch.exp(l)
    total = torch.where(some, e.sum(1, keepdim=True), torch.ones_like(top))
    lp, p = l - torch.log(total), e / total
    ent = -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(1)
    a = s["action"].long()
    at = lp.gather(1, a.clamp(min=0)[:, None])[:, 0]
    return torch.where(a < 0, torch.zeros_like(at), at), ent, lp, p


def _run_plain(s):
    c = s["case"]
    if c["op"] == "clip":
        norm = torch.sqrt(torch.stack([(t.float() * t.float()).sum() for t in s["grads"]]).sum())
        f = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0)
        flat, out = _flat([t.numel() for t in s["grads"]], _tensor_dtypes(c),
                          lambda d, n: torch.zeros(n, dtype=DTYPES[d], device=norm.device))
        for t, o in zip(s["grads"], out):
            o.copy_(t.float() * f)
        return {"norm": norm[None], **flat}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "gated":
        N = c["N"]
        pre = s["x"].float() @ s["w"].float().t() + s["b"]
        out = {"y": (_act(c["act"], pre[:, :N]) * pre[:, N:]).to(dt)}
        if c["train"]:
            g, u = s["pre_in"][:, :N].float(), s["pre_in"][:, N:].float()
            d = s["dz"].float() @ s["w2"].float()
            a = _act(c["act"], g)
            out |= {"pre": pre.to(dt), "dp": torch.cat([d * u * _dact(c["act"], g), d * a], 1).to(dt),
                    "y2": (a * u).to(dt)}
        return out
    if c["op"] == "logp":
        logp, ent, _, _ = _logp_plain(s)
        return {"logp": logp, "entropy": ent}
    logp, ent, lp, p = _logp_plain(s)
    act, kl_coef = s["action"], KL if c["ref"] else 0.0
    kept = (act >= 0) & torch.isfinite(logp)
    w = kept.float() / c["M"]
    if s["weight"] is not None:
        w = w * s["weight"]
    zero = torch.zeros_like(logp)
    x = torch.where(kept, logp - s["old"], zero)
    r = torch.exp(x)
    s1, s2 = r * s["adv"], torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH) * s["adv"]
    pg = -torch.minimum(s1, s2)
    d = torch.where(s1 <= s2, -s["adv"] * r, zero)
    kl = zero
    if s["ref"] is not None:
        y = torch.where(kept, s["ref"] - logp, zero)
        kl = torch.expm1(y) - y
        d = d - kl_coef * torch.expm1(y)
    hot = torch.arange(c["V"], device=p.device)[None] == act[:, None]
    inner = torch.where(p > 0, lp, torch.zeros_like(lp)) + ent[:, None]
    grad = d[:, None] * (hot.float() - p) + ENT * p * inner
    grad = torch.where(kept[:, None], w[:, None] * grad, torch.zeros_like(grad))
    if s["mask"] is not None:
        grad = torch.where(s["mask"], grad, torch.zeros_like(grad))
    clipped = ((r < 1 - CLIP_LOW) | (r > 1 + CLIP_HIGH)).float()
    terms = [pg + kl_coef * kl - ENT * ent, pg, kl, ent, clipped, torch.expm1(x) - x, torch.ones_like(x)]
    stats = [(w * t).sum() for t in terms] + [(~kept).float().sum()]
    return {"dlogits": grad.to(dt), "logp": logp, "entropy": ent, "stats": torch.stack(stats)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without -----------------------------------------------------
def work(case):
    if case["op"] == "clip":
        sizes, kinds = _tensor_sizes(case), _tensor_dtypes(case)
        return {"bytes": 2 * sum(n * (4 if d == "f32" else 2) for n, d in zip(sizes, kinds)) + 4,
                "flops": 3 * sum(sizes)}
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "gated":
        M, K, N, J = case["M"], case["K"], case["N"], case["J"]
        nbytes, flops = e * (M * K + 2 * N * K + M * N) + 8 * N, 4 * M * K * N
        if case["train"]:
            nbytes += e * (2 * M * N + M * J + J * N + 5 * M * N)
            flops += 2 * M * J * N
        return {"bytes": nbytes, "flops": flops}
    M, V = case["M"], case["V"]
    nbytes, flops = M * V * (e + (1 if case["mask"] else 0)) + 12 * M, 6 * M * V
    if case["op"] == "loss":
        nbytes += M * V * e + 4 * M * (2 + case["ref"] + case["weight"]) + 32
        flops += 6 * M * V
    return {"bytes": nbytes, "flops": flops}


# ---- the definitions in 64 bits ----------------------------------------------------------
def _gate64(name, v):
    """(value, derivative) of an activation, in 64 bits."""
    if name == "relu":
        return torch.where(v > 0, v, 0.0), torch.where(v > 0, 1.0, 0.0).double()
    if name == "tanh":
        e = torch.exp(-2 * v.abs())
        return torch.sign(v) * (1 - e) / (1 + e), 4 * e / (1 + e) ** 2
    # x * sigmoid(u(x)): u = x (silu), u = 2 sqrt(2/pi) (x + 0.044715 x^3) (gelu, tanh form)
    k = (1.0, 0.0) if name == "silu" else (2 * math.sqrt(2 / math.pi), 0.044715)
    u, du = k[0] * (v + k[1] * v ** 3), k[0] * (1 + 3 * k[1] * v ** 2)
    q = 1 / (1 + torch.exp(-u))
    return v * q, q + v * q * (1 - q) * du


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float((t.double() ** 2).sum()) for t in s["grads"])
        norm = math.sqrt(total)
        f = min(1.0, case["max_norm"] / (norm + 1e-6))
        flat, out = _flat([t.numel() for t in s["grads"]], _tensor_dtypes(case),
                          lambda d, n: torch.zeros(n, dtype=torch.float64, device="cuda"))
        for t, o in zip(s["grads"], out):
            o.copy_(t.double().mul_(f))
        return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), **flat}
    if case["op"] == "gated":
        N = case["N"]
        x, w = s["x"].double(), s["w"].double()
        gate = torch.einsum("mk,nk->mn", x, w[:N]) + s["b"][:N].double()
        up = torch.einsum("mk,nk->mn", x, w[N:]) + s["b"][N:].double()
        out = {"y": _gate64(case["act"], gate)[0] * up}
        if case["train"]:
            g, u = s["pre_in"].double().split(N, dim=1)
            a, da = _gate64(case["act"], g)
            d = torch.einsum("mj,jn->mn", s["dz"].double(), s["w2"].double())
            out |= {"pre": torch.cat([gate, up], 1), "dp": torch.cat([d * (u * da), d * a], 1), "y2": a * u}
        return out
    # row blocks: 64-bit copies of all logits would not fit beside the rest
    M, V = case["M"], case["V"]
    loss = case["op"] == "loss"
    logp = torch.empty(M, dtype=torch.float64, device="cuda")
    ent = torch.empty_like(logp)
    grad = torch.empty(M, V, dtype=torch.float64, device="cuda") if loss else None
    sums = torch.zeros(8, dtype=torch.float64, device="cuda")
    step = max(1, int(3e7) // V)
    for r0 in range(0, M, step):
        at = slice(r0, min(M, r0 + step))
        z = s["logits"][at].double()
        ok = torch.ones_like(z, dtype=torch.bool) if s["mask"] is None else s["mask"][at]
        z = z.masked_fill(~ok, -math.inf)
        empty = ~ok.any(1)
        lse = torch.logsumexp(z, 1).masked_fill(empty, 0.0)
        lp = z - lse[:, None]
        p = lp.exp()
        h = -(p * lp.masked_fill(~ok, 0.0)).sum(1)
        a = s["action"][at].long()
        la = lp.gather(1, a.clamp(min=0)[:, None]).squeeze(1).masked_fill(a < 0, 0.0)
        logp[at], ent[at] = la, h
        if not loss:
            continue
        kept = (a >= 0) & (la > -math.inf)
        adv = s["adv"][at].double()
        ratio = (la - s["old"][at].double()).masked_fill(~kept, 0.0).exp()
        lo, hi = 1 - CLIP_LOW, 1 + CLIP_HIGH
        # the surrogate's slope ends above 1 + high for good actions, below 1 - low for bad ones
        flat = torch.where(adv > 0, ratio > hi, ratio < lo) & (adv != 0)
        bound = torch.where(adv > 0, torch.full_like(adv, hi), torch.full_like(adv, lo))
        pg = -adv * torch.where(flat, bound, ratio)
        slope = torch.where(flat, torch.zeros_like(adv), -adv * ratio)
        kl = torch.zeros_like(adv)
        coef = 0.0
        if s["ref"] is not None:
            coef = KL
            y = (s["ref"][at].double() - la).masked_fill(~kept, 0.0)
            kl = y.exp() - y - 1
            slope = slope + coef * (1 - y.exp())
        w = kept.double() / M
        if s["weight"] is not None:
            w = w * s["weight"][at].double()
        gr = -slope[:, None] * p + ENT * p * (lp.masked_fill(~ok, 0.0) + h[:, None])
        gr.scatter_add_(1, a.clamp(min=0)[:, None], slope[:, None])
        grad[at] = (gr * w[:, None]).masked_fill(~kept[:, None], 0.0)
        out = (ratio < lo) | (ratio > hi)
        log_r = ratio.log()
        terms = [pg + coef * kl - ENT * h, pg, kl, h, out.double(), ratio - 1 - log_r, torch.ones_like(adv)]
        sums += torch.stack([(w * t).sum() for t in terms] + [(~kept).double().sum()])
    if not loss:
        return {"logp": logp, "entropy": ent}
    return {"dlogits": grad, "logp": logp, "entropy": ent, "stats": sums}
