"""A pre-norm residual recurrent trunk out of the trunk operators of ppo.h.

A block takes the residual stream x [T, N, D] of a rollout through a gated scan
(a MinGRU layer, H channels) and a two-layer perceptron (F wide):

    x <- x + Wo . scan(Wp . layernorm(x) + bp) + bo
    x <- x + W2 . act(W1 . layernorm(x) + b1) + b2

RecurrentTrunk holds the parameters, what the forward pass leaves for the
backward pass, and the workspaces, all allocated once: forward() and backward()
run whole rollouts, step() advances carried states by one acting step.  None of
them allocates or synchronises, so each can be captured in a CUDA graph, and
step() shares only the parameters with the other two, so that it may run on a
stream of its own between two load_params().
"""
import math

from . import (_abi, ppo_gated_scan_backward, ppo_gated_scan_forward, ppo_layernorm_backward,
               ppo_layernorm_backward_workspace_bytes, ppo_layernorm_forward,
               ppo_linear_backward_data, ppo_linear_backward_weight, ppo_linear_forward,
               ppo_linear_workspace_bytes, ppo_scan_blocks, ppo_work_status)

ACTIVATIONS = {"none": _abi.ACT_NONE, "tanh": _abi.ACT_TANH, "relu": _abi.ACT_RELU,
               "silu": _abi.ACT_SILU, "gelu": _abi.ACT_GELU}


class RecurrentTrunk:
    """`blocks` blocks for rollouts of T steps of N environments.

    params and grads map (block, name) to fp32 tensors: the layer norms' g1, c1,
    g2, c2 [D], the matrices Wp [2H, D], Wo [D, H], W1 [F, D], W2 [D, F] and
    their biases bp, bo, b1, b2.  The matrices enter the products in `dtype`:
    call load_params() after changing params.
    """

    def __init__(self, T, N, width, hidden, inner, blocks=1, dtype=None, act="gelu", eps=1e-5,
                 device="cuda", generator=None):
        import torch
        self.T, self.N, self.D, self.H, self.F, self.blocks = T, N, width, hidden, inner, blocks
        self.dtype = dtype or torch.bfloat16
        self.act, self.eps = ACTIVATIONS[act], eps
        D, H, F, M = width, hidden, inner, T * N
        f32 = dict(dtype=torch.float32, device=device)
        own = dict(dtype=self.dtype, device=device)
        shapes = {"Wp": (2 * H, D), "Wo": (D, H), "W1": (F, D), "W2": (D, F)}
        self.params, self.grads, self._w = {}, {}, {}
        for b in range(blocks):
            for name, (rows, cols) in shapes.items():
                scale = 1 / math.sqrt(cols) / (math.sqrt(2 * blocks) if name in ("Wo", "W2") else 1)
                self.params[b, name] = torch.randn(rows, cols, generator=generator, **f32) * scale
                self.params[b, "b" + name[1]] = torch.zeros(rows, **f32)
                self._w[b, name] = torch.empty(rows, cols, **own)
            # gates that start nearly closed remember
            self.params[b, "bp"][:H] = -2.0
            for k in "12":
                self.params[b, "g" + k] = torch.ones(D, **f32)
                self.params[b, "c" + k] = torch.zeros(D, **f32)
        self.grads = {k: torch.empty_like(v) for k, v in self.params.items()}
        self.load_params()

        self._kept = [dict(
            n1=torch.empty(M, D, **own), s1=torch.empty(M, 2, **f32),
            p=torch.empty(T, N, 2 * H, **own), h=torch.empty(T, N, H, **own),
            carry=torch.empty(ppo_scan_blocks(T), N, H, **f32), xm=torch.empty(M, D, **own),
            n2=torch.empty(M, D, **own), s2=torch.empty(M, 2, **f32), u=torch.empty(M, F, **own),
            a=torch.empty(M, F, **own), y=torch.empty(M, D, **own)) for _ in range(blocks)]
        self._du, self._dn = torch.empty(M, F, **own), torch.empty(M, D, **own)
        self._dh, self._dp = torch.empty(T, N, H, **own), torch.empty(T, N, 2 * H, **own)
        self._dxm, self._dx = torch.empty(M, D, **own), torch.empty(M, D, **own)
        # one acting step
        self._one = dict(n=torch.empty(N, D, **own), p=torch.empty(1, N, 2 * H, **own),
                         h=torch.empty(1, N, H, **own), xm=torch.empty(N, D, **own),
                         a=torch.empty(N, F, **own), y=torch.empty(N, D, **own))
        # acting may run on another stream than learning: a workspace each.  (dy, W2's
        # dz, may come in rows of any pitch: an odd one asks for most.)
        def workspace(rows):
            need = max(ppo_linear_workspace_bytes(rows, r, c, self.dtype, ldz=D | 1 if name == "W2" else 0)
                       for name, (r, c) in shapes.items())
            return torch.zeros(need, dtype=torch.uint8, device=device)

        self._work, self._act_work = workspace(M), workspace(N)
        self._ln_work = torch.empty(ppo_layernorm_backward_workspace_bytes(M, D), dtype=torch.uint8,
                                    device=device)
        self._in = None

    def load_params(self):
        """Rounds the matrices of params to the products' type."""
        for k, w in self._w.items():
            w.copy_(self.params[k])

    def state(self):
        """Carried states of the acting step, [blocks, N, H], all cleared."""
        import torch
        return torch.zeros(self.blocks, self.N, self.H, dtype=torch.float32,
                           device=self._work.device)

    def forward(self, x, done=None, done0=None, h0=None, hT=None, stream=None):
        """The last block's output [T, N, D] for x [T, N, D] (kept, not copied,
        until backward()).  done [T, N], done0 [N], h0 and hT [blocks, N, H] as
        in ppo_gated_scan_forward.  The result is the trunk's own buffer."""
        M, D = self.T * self.N, self.D
        P, W, work, st = self.params, self._w, self._work, stream
        self._in = (x.reshape(M, D), done, done0)
        x = self._in[0]
        for b, k in enumerate(self._kept):
            ppo_layernorm_forward(x, P[b, "g1"], P[b, "c1"], k["n1"], k["s1"], self.eps, st)
            ppo_linear_forward(k["n1"], W[b, "Wp"], k["p"].view(M, -1), P[b, "bp"], work=work, stream=st)
            ppo_gated_scan_forward(k["p"], k["h"], None if h0 is None else h0[b], done, done0,
                                   None if hT is None else hT[b], k["carry"], st)
            ppo_linear_forward(k["h"].view(M, -1), W[b, "Wo"], k["xm"], P[b, "bo"], res=x, work=work,
                               stream=st)
            ppo_layernorm_forward(k["xm"], P[b, "g2"], P[b, "c2"], k["n2"], k["s2"], self.eps, st)
            ppo_linear_forward(k["n2"], W[b, "W1"], k["a"], P[b, "b1"], self.act, pre=k["u"], work=work,
                               stream=st)
            ppo_linear_forward(k["a"], W[b, "W2"], k["y"], P[b, "b2"], res=k["xm"], work=work, stream=st)
            x = k["y"]
        return x.view(self.T, self.N, D)

    def backward(self, dy, dhT=None, dh0=None, stream=None):
        """Fills grads from dy [T, N, D], the gradient of forward()'s result, and
        dhT [blocks, N, H], that of hT; returns the gradient of x (the trunk's own
        buffer), and leaves that of h0 in dh0."""
        M, D = self.T * self.N, self.D
        P, W, G, work, st = self.params, self._w, self.grads, self._work, stream
        x0, done, done0 = self._in
        dy = dy.reshape(M, D)
        dp, dh = self._dp.view(M, -1), self._dh.view(M, -1)
        for b in reversed(range(self.blocks)):
            k = self._kept[b]
            x = x0 if b == 0 else self._kept[b - 1]["y"]
            ppo_linear_backward_weight(dy, k["a"], G[b, "W2"], G[b, "b2"], work=work, stream=st)
            ppo_linear_backward_data(dy, W[b, "W2"], self._du, k["u"], self.act, work=work, stream=st)
            ppo_linear_backward_weight(self._du, k["n2"], G[b, "W1"], G[b, "b1"], work=work, stream=st)
            ppo_linear_backward_data(self._du, W[b, "W1"], self._dn, work=work, stream=st)
            ppo_layernorm_backward(self._dn, k["xm"], P[b, "g2"], k["s2"], self._dxm, G[b, "g2"],
                                   G[b, "c2"], dy, self._ln_work, st)
            ppo_linear_backward_weight(self._dxm, k["h"].view(M, -1), G[b, "Wo"], G[b, "bo"], work=work,
                                       stream=st)
            ppo_linear_backward_data(self._dxm, W[b, "Wo"], dh, work=work, stream=st)
            ppo_gated_scan_backward(self._dh, k["p"], k["carry"], self._dp, done, done0,
                                    None if dhT is None else dhT[b], None if dh0 is None else dh0[b], st)
            ppo_linear_backward_weight(dp, k["n1"], G[b, "Wp"], G[b, "bp"], work=work, stream=st)
            ppo_linear_backward_data(dp, W[b, "Wp"], self._dn, work=work, stream=st)
            ppo_layernorm_backward(self._dn, x, P[b, "g1"], k["s1"], self._dx, G[b, "g1"], G[b, "c1"],
                                   self._dxm, self._ln_work, st)
            dy = self._dx
        return self._dx.view(self.T, self.N, D)

    def step(self, x, state, done=None, stream=None):
        """One acting step: the output [N, D] for x [N, D], the states [blocks, N,
        H] advanced in place (cleared first where done [N] is not 0).  The
        result is the trunk's own buffer."""
        P, W, o, work, st = self.params, self._w, self._one, self._act_work, stream
        for b in range(self.blocks):
            ppo_layernorm_forward(x, P[b, "g1"], P[b, "c1"], o["n"], None, self.eps, st)
            ppo_linear_forward(o["n"], W[b, "Wp"], o["p"][0], P[b, "bp"], work=work, stream=st)
            ppo_gated_scan_forward(o["p"], o["h"], state[b], None, done, state[b], None, st)
            ppo_linear_forward(o["h"][0], W[b, "Wo"], o["xm"], P[b, "bo"], res=x, work=work, stream=st)
            ppo_layernorm_forward(o["xm"], P[b, "g2"], P[b, "c2"], o["n"], None, self.eps, st)
            ppo_linear_forward(o["n"], W[b, "W1"], o["a"], P[b, "b1"], self.act, work=work, stream=st)
            ppo_linear_forward(o["a"], W[b, "W2"], o["y"], P[b, "b2"], res=o["xm"], work=work, stream=st)
            x = o["y"]
        return x

    def check(self, stream=None):
        """Synchronises the stream; raises PpoError if a bounded device wait of
        learning or acting gave up (on another stream: wait for that one first)."""
        failed = []
        for work in (self._work, self._act_work):
            try:
                ppo_work_status(work, stream)
            except RuntimeError as e:
                failed.append(e)
        if failed:
            raise failed[0]
