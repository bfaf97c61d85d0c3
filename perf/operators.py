"""What is measured of the operators of a pre-norm residual recurrent policy.

The learner's policies are an MLP and a MinGRU.  A deeper recurrent trunk is a
stack of blocks  x -> x + Wo . scan(Wp . layernorm(x)),  x -> x + W2 . act(W1 .
layernorm(x)),  and these are its operators:

  layer norm          y = (x - mean) * rstd * gamma + beta, and its backward pass
                      with the sums of the gamma and beta gradients;
  gated linear scan   z = sigmoid(pz),  h_t = (1 - z_t) h_{t-1} + z_t ph_t  over the
                      steps of a rollout, the state cleared where an episode ended,
                      and its backward pass; one step of it when the policy acts;
  linear              y = act(x W^T + b) + residual, its data gradient with the
                      previous layer's act' and the residual's gradient, its
                      weight and bias gradients.

listed() and draw() give cases, prepare() their inputs, run() one pass: in the
plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where `own` is true, through the framework's entry points.  exact() computes the
same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
# codes of the framework's activations
ACTS = {"none": -1, "tanh": 0, "relu": 1, "silu": 2, "gelu": 3}
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # 64 agents of one acting step, width 512: the call's latency
        dict(name="ln_step", op="ln", M=64, D=512, dtype="bf16", train=False, dres=False),
        # a rollout of 128 steps x 2,048 environments, width 512, forward and backward, the
        # residual path's gradient added
        dict(name="ln_rollout", op="ln", M=262144, D=512, dtype="bf16", train=True, dres=True),
        # 48,000 raw observations of 1,397 numbers, normalised in fp32: odd rows
        dict(name="ln_obs_f32", op="ln", M=48000, D=1397, dtype="f32", train=True, dres=False),
        # one acting step of 2,048 environments, width 512, state carried
        dict(name="scan_step", op="scan", T=1, N=2048, H=512, dtype="bf16", train=False, done_p=0.004),
        # a rollout of 128 steps x 2,048 environments, width 256, forward and backward
        dict(name="scan_rollout", op="scan", T=128, N=2048, H=256, dtype="bf16", train=True, done_p=0.004),
        # one very long sequence, width 1,024: the time axis has to be split
        dict(name="scan_long", op="scan", T=65537, N=1, H=1024, dtype="bf16", train=True, done_p=0.0005),
        # an odd number of environments of odd width in fp32, long segments
        dict(name="scan_odd_f32", op="scan", T=1023, N=37, H=129, dtype="f32", train=True, done_p=0.01),
        # one token through an up-projection: latency
        dict(name="linear_token", op="linear", M=1, K=512, N=2048, dtype="bf16", act="gelu", pre=False,
             res=False, pact="none", dres=False, train=False),
        # 33 tokens through a wide layer with its residual: the weight has to be streamed
        dict(name="linear_serve", op="linear", M=33, K=4096, N=4096, dtype="bf16", act="none", pre=False,
             res=True, pact="none", dres=False, train=False),
        # the up-projection of a 32,768-row minibatch, trained
        dict(name="linear_up", op="linear", M=32768, K=512, N=2048, dtype="bf16", act="gelu", pre=True,
             res=False, pact="none", dres=False, train=True),
        # the down-projection of 65,536 rows with its residual, trained; the data gradient
        # continues through the up-projection's activation
        dict(name="linear_down", op="linear", M=65536, K=2048, N=512, dtype="bf16", act="none", pre=False,
             res=True, pact="gelu", dres=False, train=True),
        # fp32 weights and rows (the framework's fp32 mode), an odd number of rows and inputs
        dict(name="linear_f32", op="linear", M=4999, K=1397, N=512, dtype="f32", act="tanh", pre=True,
             res=True, pact="none", dres=True, train=True),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    return v - 1 if v == 3072 else v


def _capped(first, cap):
    return max(1, min(first, int(cap)))


def draw(rng):
    op = rng.choice(["ln", "scan", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.7
    if op == "ln":
        D = _size(rng, 16, 8192)
        if rng.random() < 0.6:
            D = max(16, D // 8 * 8)
        M = _capped(_size(rng, 1, 262144), (67e6 if dtype == "f32" else 134e6) / D)
        return dict(op="ln", M=M, D=D if D != 3072 else 3080, dtype=dtype, train=train,
                    dres=rng.random() < 0.5)
    if op == "scan":
        H = _size(rng, 16, 1024)
        if rng.random() < 0.6:
            H = max(16, H // 8 * 8)
        N = _size(rng, 1, 2048)
        T = _capped(_size(rng, 1, 65537), (33e6 if dtype == "f32" else 67e6) / (N * H))
        return dict(op="scan", T=T if T != 3072 else 3071, N=N, H=H, dtype=dtype, train=train,
                    done_p=rng.choice([0.0, 0.002, 0.03]))
    top = 2048 if dtype == "f32" else 4096
    K, N = _size(rng, 16, top), _size(rng, 16, top)
    if rng.random() < 0.7:
        K, N = max(16, K // 8 * 8), max(16, N // 8 * 8)
    K, N = (v if v != 3072 else 3080 for v in (K, N))
    M = _capped(_size(rng, 1, 32768), (4e9 if dtype == "f32" else 6.8e10) / (K * N))
    return dict(op="linear", M=M if M != 3072 else 3071, K=K, N=N, dtype=dtype,
                act=rng.choice(["none", "tanh", "relu", "silu", "gelu"]), pre=train and rng.random() < 0.5,
                res=rng.random() < 0.5, pact=rng.choice(["none", "tanh", "relu", "silu", "gelu"]),
                dres=rng.random() < 0.3, train=train)


# ---- inputs ---------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale + shift).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, device=dev, dtype=dtype)

    f32 = torch.float32
    s = {"case": case}
    if case["op"] == "ln":
        M, D = case["M"], case["D"]
        # the residual stream: rows of unlike scale, with a mean of their own
        s["x"] = (torch.randn(M, D, generator=g, device=dev) * torch.empty(M, 1, device=dev).uniform_(0.5, 4.0, generator=g)
                  + torch.randn(M, 1, generator=g, device=dev)).to(dt)
        s["gamma"] = normal(D, scale=0.2, shift=1.0, dtype=f32)
        s["beta"] = normal(D, scale=0.2, dtype=f32)
        s["y"] = empty(M, D)
        if case["train"]:
            s["dy"] = normal(M, D)
            s["dres"] = normal(M, D) if case["dres"] else None
            s["stats"] = empty(M, 2, dtype=f32)
            s["dx"], s["dgamma"], s["dbeta"] = empty(M, D), empty(D, dtype=f32), empty(D, dtype=f32)
        return s
    if case["op"] == "scan":
        T, N, H = case["T"], case["N"], case["H"]
        # gate pre-activations around a slow gate, candidates of unit scale
        s["p"] = torch.cat([normal(T, N, H, scale=1.5, shift=-2.0), normal(T, N, H)], dim=2)
        s["done"] = (torch.rand(T, N, generator=g, device=dev) < case["done_p"]).to(f32)
        s["done0"] = (torch.rand(N, generator=g, device=dev) < case["done_p"]).to(f32)
        s["h0"] = normal(N, H, dtype=f32)
        s["h"], s["hT"] = empty(T, N, H), empty(N, H, dtype=f32)
        if case["train"]:
            s["dh"], s["dhT"] = normal(T, N, H), normal(N, H, dtype=f32)
            s["carry"] = empty((T + 127) // 128, N, H, dtype=f32)  # the state that enters every 128th step
            s["dp"], s["dh0"] = empty(T, N, 2 * H), empty(N, H, dtype=f32)
        return s
    M, K, N = case["M"], case["K"], case["N"]
    s["x"] = normal(M, K)
    s["w"] = normal(N, K, scale=1.0 / math.sqrt(K))
    s["b"] = normal(N, scale=0.1, dtype=f32)
    s["res"] = normal(M, N) if case["res"] else None
    s["y"] = empty(M, N)
    s["pre"] = empty(M, N) if case["pre"] else None
    if case["train"]:
        s["dz"] = normal(M, N)
        s["ppre"] = normal(M, K) if case["pact"] != "none" else None
        s["dres"] = normal(M, K) if case["dres"] else None
        s["dx"], s["dw"], s["db"] = empty(M, K), empty(N, K, dtype=f32), empty(N, dtype=f32)
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
    if c["op"] == "ln":
        if not c["train"]:
            P.ppo_layernorm_forward(s["x"], s["gamma"], s["beta"], s["y"], eps=EPS)
            return {"y": s["y"]}
        work = _work(s, lambda: P.ppo_layernorm_backward_workspace_bytes(c["M"], c["D"]))
        P.ppo_layernorm_forward(s["x"], s["gamma"], s["beta"], s["y"], stats=s["stats"], eps=EPS)
        P.ppo_layernorm_backward(s["dy"], s["x"], s["gamma"], s["stats"], s["dx"], dgamma=s["dgamma"],
                                 dbeta=s["dbeta"], dres=s["dres"], work=work)
        return {k: s[k] for k in ("y", "stats", "dx", "dgamma", "dbeta")}
    if c["op"] == "scan":
        P.ppo_gated_scan_forward(s["p"], s["h"], h0=s["h0"], done=s["done"], done0=s["done0"], hT=s["hT"],
                                 carry=s.get("carry"))
        if not c["train"]:
            return {"h": s["h"], "hT": s["hT"]}
        P.ppo_gated_scan_backward(s["dh"], s["p"], s["carry"], s["dp"], done=s["done"], done0=s["done0"],
                                  dhT=s["dhT"], dh0=s["dh0"])
        return {k: s[k] for k in ("h", "hT", "dp", "dh0")}
    work = _work(s, lambda: P.ppo_linear_workspace_bytes(c["M"], c["N"], c["K"], s["x"].dtype))
    P.ppo_linear_forward(s["x"], s["w"], s["y"], bias=s["b"], act=ACTS[c["act"]], res=s["res"],
                         pre=s["pre"], work=work)
    out = {"y": s["y"]}
    if c["pre"]:
        out["pre"] = s["pre"]
    if c["train"]:
        P.ppo_linear_backward_data(s["dz"], s["w"], s["dx"], pre=s["ppre"], act=ACTS[c["pact"]],
                                   res=s["dres"], work=work)
        P.ppo_linear_backward_weight(s["dz"], s["x"], s["dw"], db=s["db"], work=work)
        out |= {k: s[k] for k in ("dx", "dw", "db")}
    return out


# ---- the plain form -----------------------------------------------------------------
def _act(name, v):
    if name == "tanh":
        return torch.tanh(v)
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1 + torch.tanh(GELU_C * (v + GELU_A * v * v * v)))
    return v


def _dact(name, v):
    if name == "tanh":
        return 1 - torch.tanh(v) ** 2
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        q = torch.sigmoid(v)
        return q * (1 + v * (1 - q))
    if name == "gelu":
        t = torch.tanh(GELU_C * (v + GELU_A * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * v * v)
    return torch.ones_like(v)


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 0 from h_{-1} = 0, by recursive doubling: log2(T) rounds,
    each of them over the whole array."""
    T, d = a.shape[0], 1
    while d < T:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _run_plain(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if c["op"] == "ln":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
        xh = xc * rstd
        out = {"y": (xh * s["gamma"] + s["beta"]).to(dt)}
        if c["train"]:
            dy = s["dy"].float()
            dxh = dy * s["gamma"]
            dx = rstd * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
            if s["dres"] is not None:
                dx = dx + s["dres"].float()
            out |= {"stats": torch.cat([mean, rstd], 1), "dx": dx.to(dt), "dgamma": (dy * xh).sum(0),
                    "dbeta": dy.sum(0)}
        return out
    if c["op"] == "scan":
        T, H = c["T"], c["H"]
        p = s["p"].float()
        z, cand = torch.sigmoid(p[..., :H]), p[..., H:]
        # the state that enters step t is cleared where the episode ended at step t - 1
        keep = 1 - torch.cat([s["done0"][None], s["done"][:-1]])[..., None]
        a = (1 - z) * keep
        b = z * cand
        b0 = b.clone()
        b0[0] += a[0] * s["h0"]
        h = _doubling(a, b0)
        out = {"h": h.to(dt), "hT": h[-1].clone()}
        if c["train"]:
            # dL/dh_t = dh_t + a_{t+1} dL/dh_{t+1}
            dh = torch.cat([s["dh"][:-1].float(), (s["dh"][-1].float() + s["dhT"])[None]])
            an = torch.cat([torch.zeros_like(a[:1]), a[1:].flip(0)])
            gr = _doubling(an, dh.flip(0)).flip(0)
            hp = torch.cat([s["h0"][None], h[:-1]]) * keep
            out["dp"] = torch.cat([gr * (cand - hp) * z * (1 - z), gr * z], 2).to(dt)
            out["dh0"] = gr[0] * a[0]
        return out
    x, w = s["x"].float(), s["w"].float()
    pre = x @ w.t() + s["b"]
    y = _act(c["act"], pre)
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(dt)}
    if c["pre"]:
        out["pre"] = pre.to(dt)
    if c["train"]:
        dz = s["dz"].float()
        dx = dz @ w
        if s["ppre"] is not None:
            dx = dx * _dact(c["pact"], s["ppre"].float())
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out |= {"dx": dx.to(dt), "dw": dz.t() @ x, "db": dz.sum(0)}
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without -----------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ln":
        n, D = case["M"] * case["D"], case["D"]
        nbytes, flops = 2 * n * e + 8 * D, 8 * n
        if case["train"]:
            nbytes += (3 + case["dres"]) * n * e + 16 * case["M"] + 12 * D
            flops += 14 * n
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "scan":
        n, ch = case["T"] * case["N"] * case["H"], case["N"] * case["H"]
        nbytes, flops = 3 * n * e + 8 * ch + 4 * case["T"] * case["N"], 8 * n
        if case["train"]:
            nbytes += 5 * n * e + 8 * ch + 4 * case["T"] * case["N"]
            flops += 16 * n
        return {"bytes": nbytes, "flops": flops}
    M, K, N = case["M"], case["K"], case["N"]
    nbytes = e * (M * K + N * K + M * N * (1 + case["res"] + case["pre"])) + 4 * N
    flops = 2 * M * K * N
    if case["train"]:
        nbytes += e * (2 * M * N + N * K + M * K * (2 + case["dres"] + (case["pact"] != "none"))) + 4 * N * K + 4 * N
        flops += 4 * M * K * N
    return {"bytes": nbytes, "flops": flops}


# ---- the definitions in 64 bits ----------------------------------------------------------
def _act64(name, v):
    """(value, derivative) of an activation, in 64 bits."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), torch.where(v > 0, 1.0, 0.0).double()
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
    if case["op"] == "ln":
        x, ga, be = (s[k].double() for k in ("x", "gamma", "beta"))
        D = x.shape[1]
        mu = x.sum(1) / D
        var = ((x - mu[:, None]) ** 2).sum(1) / D
        r = (var + EPS).rsqrt()
        xh = (x - mu[:, None]) * r[:, None]
        out = {"y": xh * ga + be}
        if case["train"]:
            dy = s["dy"].double()
            q = dy * ga
            # gradient of the row's output through x, its mean and its variance
            dvar = (q * (x - mu[:, None])).sum(1) * (-0.5) * r ** 3
            dmu = -r * q.sum(1)
            dx = q * r[:, None] + (2 * dvar / D)[:, None] * (x - mu[:, None]) + (dmu / D)[:, None]
            if s["dres"] is not None:
                dx += s["dres"].double()
            out |= {"stats": torch.stack([mu, r], 1), "dx": dx, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
        return out
    if case["op"] == "scan":
        T, N, H = case["T"], case["N"], case["H"]
        z = 1 / (1 + torch.exp(-s["p"][..., :H].double()))
        cand = s["p"][..., H:].double()
        gone = torch.cat([s["done0"][None], s["done"][:-1]]) != 0
        a = torch.where(gone[..., None], 0.0, 1 - z)
        b = z * cand
        h = torch.empty(T + 1, N, H, dtype=torch.float64, device=z.device)
        h[0] = s["h0"].double()
        for t in range(T):
            torch.addcmul(b[t], a[t], h[t], out=h[t + 1])
        out = {"h": h[1:], "hT": h[T].clone()}
        if case["train"]:
            g = s["dh"].double()
            g[T - 1] += s["dhT"].double()
            for t in range(T - 2, -1, -1):
                g[t].addcmul_(a[t + 1], g[t + 1])
            entering = torch.where(gone[..., None], 0.0, h[:-1])
            out["dp"] = torch.cat([g * (cand - entering) * z * (1 - z), g * z], 2)
            out["dh0"] = a[0] * g[0]
        return out
    x, w = s["x"].double(), s["w"].double()
    pre = torch.einsum("mk,nk->mn", x, w) + s["b"].double()
    y = _act64(case["act"], pre)[0]
    if s["res"] is not None:
        y = y + s["res"].double()
    out = {"y": y}
    if case["pre"]:
        out["pre"] = pre
    if case["train"]:
        dz = s["dz"].double()
        dx = torch.einsum("mn,nk->mk", dz, w)
        if s["ppre"] is not None:
            dx = dx * _act64(case["pact"], s["ppre"].double())[1]
        if s["dres"] is not None:
            dx = dx + s["dres"].double()
        out |= {"dx": dx, "dw": torch.einsum("mn,mk->nk", dz, x), "db": dz.sum(0)}
    return out
