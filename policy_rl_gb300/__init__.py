"""GB300 (sm_103a) PPO learner step: Python binding of ``include/ppo.h``.

The functions here carry the C ABI's names and only marshal arguments: torch
tensors supply device memory (``data_ptr()``) and the current CUDA stream;
every step of the computation runs in the library's CUDA kernels.  There is
no CPU fallback -- without the built library (``policy_rl_gb300.build``) or
an sm_103a device every call raises.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

from . import _abi
from ._abi import PpoConfig, PpoError, RnnConfig

__all__ = [
    "PpoConfig", "PpoError", "Context", "make_config", "ppo_param_count", "ppo_gae",
    "ppo_gae_workspace_bytes", "ppo_gae_noalloc", "ppo_minibatch_perm", "ppo_perm_workspace_bytes",
    "ppo_segment_advantage", "ppo_segment_advantage_workspace_bytes",
    "ppo_minibatch_loss_grad_fresh", "ppo_policy_act", "ppo_muon_step", "RnnConfig",
    "make_rnn_config", "ppo_rnn_param_count", "ppo_rnn_workspace_bytes", "ppo_rnn_loss_grad",
    "ppo_create", "ppo_destroy", "ppo_buffers", "ppo_params_changed", "ppo_get_step",
    "ppo_minibatch_loss_grad", "ppo_adam_step", "ppo_update", "ppo_update_host",
    "ppo_update_host_async", "ppo_host_wait",
    "ppo_sync_status", "ppo_stage_name", "ppo_update_profile", "ppo_set_step_trace",
    "ppo_set_wait_limit", "ppo_set_collective", "TorchCollective", "RnnContext",
    "ppo_layernorm_forward", "ppo_layernorm_backward_workspace_bytes", "ppo_layernorm_backward",
    "ppo_gated_scan_forward", "ppo_gated_scan_backward", "ppo_scan_blocks",
    "ppo_linear_workspace_bytes", "ppo_linear_forward", "ppo_linear_backward_data",
    "ppo_linear_backward_weight", "ppo_work_status", "ppo_gated_linear_workspace_bytes",
    "ppo_gated_linear_forward", "ppo_gated_linear_backward_data", "ppo_action_logp",
    "ppo_action_loss_workspace_bytes", "ppo_action_loss_grad", "TensorList",
    "ppo_grad_norm_workspace_bytes", "ppo_grad_norm", "ppo_clip_grad_norm",
    "library_path",
]


def library_path() -> str:
    return _abi.LIB_PATH


def _lib():
    return _abi._lib or _abi.load()


def _ptr(t):
    """Device (or host) address of a tensor / numpy array, None for None."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return ctypes.c_void_p(t.data_ptr())
    if hasattr(t, "ctypes"):
        return ctypes.c_void_p(t.ctypes.data)
    return ctypes.c_void_p(int(t))


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_config(obs_dim, h1, h2, act=0, heads=(3, 2, 2), n_gauss=0, precision=1, clip=0.2,
                vf_coef=0.5, ent_coef=0.01, beta1=0.9, beta2=0.999, adam_eps=1e-8,
                max_grad_norm=0.5, max_batch=1, max_minibatch=1, max_epochs=1,
                persistent_minibatch=0, fused_mlp=0, fused_loss=0, adv_mode=0,
                vtrace_rho_clip=1.0, vtrace_c_clip=1.0, optimizer=0, muon_lr=0.02,
                muon_beta=0.95) -> PpoConfig:
    hn = (ctypes.c_int32 * _abi.MAX_HEADS)(*(list(heads) + [0] * (_abi.MAX_HEADS - len(heads))))
    return PpoConfig(obs_dim, h1, h2, act, len(heads), hn, n_gauss, precision, clip, vf_coef,
                     ent_coef, max_grad_norm, beta1, beta2, adam_eps, max_batch, max_minibatch,
                     max_epochs, persistent_minibatch, fused_mlp, fused_loss, adv_mode,
                     vtrace_rho_clip, vtrace_c_clip, optimizer, muon_lr, muon_beta)


def config_from_workload(w, max_batch=None, max_minibatch=None, max_epochs=None,
                         persistent_minibatch=0, fused_mlp=0, fused_loss=0, adv_mode=0,
                         vtrace_rho_clip=1.0, vtrace_c_clip=1.0, optimizer=0, muon_lr=0.02,
                         muon_beta=0.95) -> PpoConfig:
    B = w.T * w.N
    return make_config(w.obs_dim, w.h1, w.h2, w.act, tuple(w.heads), w.n_gauss,
                       1 if w.precision == "bf16" else 0, w.clip, w.vf_coef, w.ent_coef,
                       max_grad_norm=w.max_grad_norm, max_batch=max_batch or B,
                       max_minibatch=max_minibatch or B // w.minibatches,
                       max_epochs=max_epochs or w.epochs,
                       persistent_minibatch=persistent_minibatch,
                       fused_mlp=fused_mlp, fused_loss=fused_loss, adv_mode=adv_mode,
                       vtrace_rho_clip=vtrace_rho_clip, vtrace_c_clip=vtrace_c_clip,
                       optimizer=optimizer, muon_lr=muon_lr, muon_beta=muon_beta)


# ---- free functions -----------------------------------------------------------
def ppo_param_count(cfg: PpoConfig) -> int:
    n = ctypes.c_int64()
    _abi.check(_lib().ppo_param_count(ctypes.byref(cfg), ctypes.byref(n)), "ppo_param_count")
    return n.value


def ppo_gae_workspace_bytes(T: int, N: int) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_gae_workspace_bytes(T, N, ctypes.byref(n)), "ppo_gae_workspace_bytes")
    return n.value


def ppo_gae(rew, val, done, boot, gamma, lam, adv, ret, adv_norm=None, stats=None, work=None,
            stream=None) -> None:
    T, N = rew.shape
    wb = work.numel() * work.element_size() if work is not None else 0
    _abi.check(_lib().ppo_gae(_ptr(rew), _ptr(val), _ptr(done), _ptr(boot), T, N, gamma, lam,
                              _ptr(adv), _ptr(ret), _ptr(adv_norm), _ptr(stats), _ptr(work), wb,
                              _stream(stream)), "ppo_gae")


def ppo_gae_noalloc(rew, val, done, boot, gamma, lam, adv, ret, adv_norm=None, stats=None,
                    stream=None) -> None:
    """ppo_gae for callers that cannot allocate device memory (see ppo.h)."""
    T, N = rew.shape
    _abi.check(_lib().ppo_gae_noalloc(_ptr(rew), _ptr(val), _ptr(done), _ptr(boot), T, N, gamma,
                                      lam, _ptr(adv), _ptr(ret), _ptr(adv_norm), _ptr(stats),
                                      _stream(stream)), "ppo_gae_noalloc")


def ppo_segment_advantage_workspace_bytes() -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_segment_advantage_workspace_bytes(ctypes.byref(n)),
               "ppo_segment_advantage_workspace_bytes")
    return n.value


def ppo_segment_advantage(rew, done, boot, envs, val, ratio, gamma, lam, adv, ret,
                          rho_clip=1.0, c_clip=1.0, adv_norm=None, stats=None, work=None,
                          stream=None) -> None:
    """GAE / V-trace advantages of the environment segments ``envs`` (see ppo.h)."""
    T, N = rew.shape
    ns = envs.numel()
    wb = work.numel() * work.element_size() if work is not None else 0
    _abi.check(_lib().ppo_segment_advantage(
        _ptr(rew), _ptr(done), _ptr(boot), T, N, _ptr(envs), ns, _ptr(val), _ptr(ratio), gamma,
        lam, rho_clip, c_clip, _ptr(adv), _ptr(ret), _ptr(adv_norm), _ptr(stats), _ptr(work), wb,
        _stream(stream)), "ppo_segment_advantage")


def ppo_perm_workspace_bytes(B: int) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_perm_workspace_bytes(B, ctypes.byref(n)), "ppo_perm_workspace_bytes")
    return n.value


def ppo_minibatch_perm(seed, epoch, B, perm, work, stream=None) -> None:
    wb = work.numel() * work.element_size()
    _abi.check(_lib().ppo_minibatch_perm(seed & 0xFFFFFFFF, epoch, B, _ptr(perm), _ptr(work), wb,
                                         _stream(stream)), "ppo_minibatch_perm")


def make_rnn_config(obs_dim, hidden=128, layers=4, heads=(3, 2, 2), n_gauss=0, clip=0.2,
                    vf_coef=0.5, ent_coef=0.01, precision=0, max_grad_norm=0.5, beta1=0.9,
                    beta2=0.999, adam_eps=1e-8) -> RnnConfig:
    hn = (ctypes.c_int32 * _abi.MAX_HEADS)(*(list(heads) + [0] * (_abi.MAX_HEADS - len(heads))))
    return RnnConfig(obs_dim, hidden, layers, len(heads), hn, n_gauss, clip, vf_coef, ent_coef,
                     precision, max_grad_norm, beta1, beta2, adam_eps)


def ppo_rnn_param_count(cfg: RnnConfig) -> int:
    n = ctypes.c_int64()
    _abi.check(_lib().ppo_rnn_param_count(ctypes.byref(cfg), ctypes.byref(n)),
               "ppo_rnn_param_count")
    return n.value


def ppo_rnn_workspace_bytes(cfg: RnnConfig, T: int, ns: int) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_rnn_workspace_bytes(ctypes.byref(cfg), T, ns, ctypes.byref(n)),
               "ppo_rnn_workspace_bytes")
    return n.value


def ppo_rnn_loss_grad(cfg: RnnConfig, params, envs, obs, act_disc, act_cont, logp_old, adv, ret,
                      done, h0, grad, adv_stats=None, stats6=None, work=None, stream=None) -> None:
    """Loss and BPTT gradient of the recurrent policy over the segments envs (see ppo.h)."""
    T, N = done.shape
    wb = work.numel() * work.element_size() if work is not None else 0
    _abi.check(_lib().ppo_rnn_loss_grad(
        ctypes.byref(cfg), _ptr(params), T, N, _ptr(envs), envs.numel(), _ptr(obs),
        _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(adv), _ptr(ret), _ptr(adv_stats),
        _ptr(done), _ptr(h0), _ptr(grad), _ptr(stats6), _ptr(work), wb, _stream(stream)),
        "ppo_rnn_loss_grad")


class RnnContext:
    """Owns one ppo_rnn_ctx: the recurrent policy's parameters, gradient, Adam
    state and update workspaces (see ppo.h, ppo_rnn_update)."""

    def __init__(self, cfg: RnnConfig, init_params=None, max_T=1, max_N=1, max_epochs=1):
        import numpy as np
        self.cfg = cfg
        self.n_params = ppo_rnn_param_count(cfg)
        h = ctypes.c_void_p()
        ip = None if init_params is None else np.ascontiguousarray(init_params, np.float32)
        _abi.check(_lib().ppo_rnn_create(ctypes.byref(cfg), _ptr(ip), max_T, max_N, max_epochs,
                                         ctypes.byref(h)), "ppo_rnn_create")
        self.handle = h
        ps = [ctypes.c_void_p() for _ in range(4)]
        _abi.check(_lib().ppo_rnn_buffers(h, *[ctypes.byref(p) for p in ps]), "ppo_rnn_buffers")
        import torch
        self.params, self.grad, self.adam_m, self.adam_v = (
            torch.as_tensor(_DevArray(p.value, self.n_params), device="cuda") for p in ps)

    def update(self, obs, act_disc, act_cont, logp_old, val, rew, done, boot, h0, epochs,
               minibatches, gamma, lam, lr, seed, stats=None, stream=None):
        T, N = val.shape
        _abi.check(_lib().ppo_rnn_update(
            self.handle, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(val),
            _ptr(rew), _ptr(done), _ptr(boot), _ptr(h0), T, N, epochs, minibatches, gamma, lam,
            lr, seed & 0xFFFFFFFF, _ptr(stats), _stream(stream)), "ppo_rnn_update")

    def sync_status(self, stream=None):
        _abi.check(_lib().ppo_rnn_sync_status(self.handle, _stream(stream)),
                   "ppo_rnn_sync_status")

    def close(self):
        if self.handle is not None:
            _lib().ppo_rnn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- operators of a recurrent trunk ---------------------------------------------
# Matrices may be strided row by row (unit stride within a row); the other
# arguments are contiguous fp32.  Results go to the tensors the caller passes.
# A call on a few rows takes the GPU some 3 us, so these wrappers are written
# for little work per argument.
_F32 = None        # torch.float32 (torch is imported by the caller's tensors)
_I32S = _BYTES = ()
_DTYPES: dict = {}
_raw_stream = None
_current_gpu = None


def _bind_torch():
    global _F32, _I32S, _BYTES, _raw_stream, _current_gpu
    import torch
    _F32 = torch.float32
    _I32S, _BYTES = (torch.int32,), (torch.bool, torch.uint8)
    _DTYPES.update({torch.float32: _abi.DTYPE_F32, torch.bfloat16: _abi.DTYPE_BF16})
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _current_gpu = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _kind(t):
    """(dtype code, GPU index) of the argument that the others have to agree with."""
    if _F32 is None:
        _bind_torch()
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"dtype must be float32 or bfloat16, got {t.dtype}")
    gpu = t.get_device()
    if gpu < 0:
        raise ValueError(f"CUDA tensors are wanted, got one on {t.device}")
    if gpu != _current_gpu():
        raise ValueError(f"tensors are on cuda:{gpu}, the current device is cuda:{_current_gpu()}")
    return code, gpu


def _on(stream, gpu):
    """The stream's handle: the given one, or the current one of the GPU."""
    if stream is None:
        return _raw_stream(gpu)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _mat(t, dtype, gpu, shape, name):
    """(address, row pitch) of a matrix argument: the last dimension is a row,
    the others flatten to rows of one pitch."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != gpu:
        raise ValueError(f"{name}: a tensor {tuple(shape)} of {dtype} on cuda:{gpu} is wanted, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    st = t.stride()
    # (one row of each of [T, 1, W]: the pitch is the distance of the first dimension)
    pitch = st[0] if len(shape) == 3 and shape[1] == 1 else st[-2]
    if (st[-1] != 1 and shape[-1] > 1) or pitch < shape[-1] or (
            len(shape) == 3 and shape[0] > 1 and st[0] != shape[1] * pitch):
        raise ValueError(f"{name}: rows must be contiguous and of one pitch")
    return t.data_ptr(), pitch


def _vec(t, gpu, shape, name):
    """Address of a contiguous fp32 argument."""
    if t is None:
        return None
    if t.dtype is not _F32 or t.shape != shape or t.get_device() != gpu:
        raise ValueError(f"{name}: a tensor {tuple(shape)} of float32 on cuda:{gpu} is wanted, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    return t.data_ptr()


def _work_of(work, gpu):
    if work is None:
        return None, 0
    if work.get_device() != gpu or not work.is_contiguous():
        raise ValueError(f"work: a contiguous tensor on cuda:{gpu} is wanted")
    return work.data_ptr(), work.nbytes


def _check(status: int, what: str) -> None:
    if status:
        _abi.check(status, what)


def ppo_layernorm_forward(x, gamma, beta, y, stats=None, eps=1e-5, stream=None) -> None:
    """y = layer norm of the rows of x [M, D] (see ppo.h); gamma, beta fp32 [D]
    or None; stats fp32 [M, 2], kept for the backward pass."""
    code, gpu = _kind(x)
    dt = x.dtype
    M, D = shape = x.shape
    px, ldx = _mat(x, dt, gpu, shape, "x")
    py, ldy = _mat(y, dt, gpu, shape, "y")
    _check(_lib().ppo_layernorm_forward(
        code, px, ldx, M, D, _vec(gamma, gpu, (D,), "gamma"), _vec(beta, gpu, (D,), "beta"), eps, py,
        ldy, _vec(stats, gpu, (M, 2), "stats"), _on(stream, gpu)), "ppo_layernorm_forward")


def ppo_layernorm_backward_workspace_bytes(M: int, D: int) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_layernorm_backward_workspace_bytes(M, D, ctypes.byref(n)),
               "ppo_layernorm_backward_workspace_bytes")
    return n.value


def ppo_layernorm_backward(dy, x, gamma, stats, dx, dgamma=None, dbeta=None, dres=None, work=None,
                           stream=None) -> None:
    """dx (+ dres, the residual path's gradient), dgamma, dbeta of the layer norm (see ppo.h)."""
    code, gpu = _kind(x)
    dt = x.dtype
    M, D = shape = x.shape
    px, ldx = _mat(x, dt, gpu, shape, "x")
    pdy, lddy = _mat(dy, dt, gpu, shape, "dy")
    pr, ldr = _mat(dres, dt, gpu, shape, "dres")
    pdx, lddx = _mat(dx, dt, gpu, shape, "dx")
    pw, wb = _work_of(work, gpu)
    _check(_lib().ppo_layernorm_backward(
        code, pdy, lddy, px, ldx, M, D, _vec(gamma, gpu, (D,), "gamma"),
        _vec(stats, gpu, (M, 2), "stats"), pr, ldr, pdx, lddx, _vec(dgamma, gpu, (D,), "dgamma"),
        _vec(dbeta, gpu, (D,), "dbeta"), pw, wb, _on(stream, gpu)), "ppo_layernorm_backward")


def ppo_scan_blocks(T: int) -> int:
    """Rows of the gated scan's carry: the states entering every 128th step."""
    return -(-T // _abi.SCAN_BLOCK)


def ppo_gated_scan_forward(p, h, h0=None, done=None, done0=None, hT=None, carry=None,
                           stream=None) -> None:
    """h [T, N, H] from the pre-activations p [T, N, 2H] (see ppo.h); h0, hT
    fp32 [N, H], done fp32 [T, N], done0 fp32 [N], carry fp32
    [ppo_scan_blocks(T), N, H].  hT may be h0."""
    code, gpu = _kind(h)
    dt = h.dtype
    T, N, H = shape = h.shape
    pp, ldp = _mat(p, dt, gpu, (T, N, 2 * H), "p")
    ph, ldh = _mat(h, dt, gpu, shape, "h")
    _check(_lib().ppo_gated_scan_forward(
        code, pp, ldp, _vec(done, gpu, (T, N), "done"), _vec(done0, gpu, (N,), "done0"),
        _vec(h0, gpu, (N, H), "h0"), T, N, H, ph, ldh, _vec(hT, gpu, (N, H), "hT"),
        _vec(carry, gpu, (ppo_scan_blocks(T), N, H), "carry"), _on(stream, gpu)),
        "ppo_gated_scan_forward")


def ppo_gated_scan_backward(dh, p, carry, dp, done=None, done0=None, dhT=None, dh0=None,
                            stream=None) -> None:
    """dp [T, N, 2H] and dh0 from dh [T, N, H] and dhT (see ppo.h)."""
    code, gpu = _kind(dh)
    dt = dh.dtype
    T, N, H = shape = dh.shape
    pd, ldd = _mat(dh, dt, gpu, shape, "dh")
    pp, ldp = _mat(p, dt, gpu, (T, N, 2 * H), "p")
    po, ldo = _mat(dp, dt, gpu, (T, N, 2 * H), "dp")
    _check(_lib().ppo_gated_scan_backward(
        code, pd, ldd, pp, ldp, _vec(done, gpu, (T, N), "done"), _vec(done0, gpu, (N,), "done0"),
        _vec(carry, gpu, (ppo_scan_blocks(T), N, H), "carry"), _vec(dhT, gpu, (N, H), "dhT"), T, N, H, po,
        ldo, _vec(dh0, gpu, (N, H), "dh0"), _on(stream, gpu)), "ppo_gated_scan_backward")


def ppo_linear_workspace_bytes(M: int, N: int, K: int, dtype, ldx: int = 0, ldw: int = 0,
                               ldz: int = 0) -> int:
    """Bytes of workspace for the three products of x [M, K], w [N, K] and
    dz [M, N] (allocate it zeroed; pitches only where the rows are strided)."""
    if _F32 is None:
        _bind_torch()
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_linear_workspace_bytes(_DTYPES.get(dtype, -1), M, N, K, ldx, ldw,
                                                 ldz, ctypes.byref(n)),
               "ppo_linear_workspace_bytes")
    return n.value


def ppo_linear_forward(x, w, y, bias=None, act=_abi.ACT_NONE, res=None, pre=None, work=None,
                       stream=None) -> None:
    """y [M, N] = act(x w^T + bias) + res, x [M, K], w [N, K], bias fp32 [N];
    pre [M, N] takes the pre-activation (see ppo.h)."""
    code, gpu = _kind(x)
    dt = x.dtype
    M, K = x.shape
    N = w.shape[0]
    px, ldx = _mat(x, dt, gpu, (M, K), "x")
    pw, ldw = _mat(w, dt, gpu, (N, K), "w")
    pr, ldr = _mat(res, dt, gpu, (M, N), "res")
    py, ldy = _mat(y, dt, gpu, (M, N), "y")
    pp, ldp = _mat(pre, dt, gpu, (M, N), "pre")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_linear_forward(
        code, px, ldx, pw, ldw, _vec(bias, gpu, (N,), "bias"), act, pr, ldr, M, N, K, py, ldy, pp,
        ldp, pk, wb, _on(stream, gpu)), "ppo_linear_forward")


def ppo_linear_backward_data(dz, w, dx, pre=None, act=_abi.ACT_NONE, res=None, work=None,
                             stream=None) -> None:
    """dx [M, K] = (dz w) * act'(pre) + res; pre [M, K] is the pre-activation
    that the layer's input came from (see ppo.h)."""
    code, gpu = _kind(dz)
    dt = dz.dtype
    M, N = dz.shape
    K = w.shape[1]
    pd, ldd = _mat(dz, dt, gpu, (M, N), "dz")
    pw, ldw = _mat(w, dt, gpu, (N, K), "w")
    pp, ldp = _mat(pre, dt, gpu, (M, K), "pre")
    pr, ldr = _mat(res, dt, gpu, (M, K), "res")
    po, ldo = _mat(dx, dt, gpu, (M, K), "dx")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_linear_backward_data(
        code, pd, ldd, pw, ldw, pp, ldp, act, pr, ldr, M, N, K, po, ldo, pk, wb,
        _on(stream, gpu)), "ppo_linear_backward_data")


def ppo_linear_backward_weight(dz, x, dw, db=None, accumulate=False, work=None,
                               stream=None) -> None:
    """dw fp32 [N, K] = dz^T x and db fp32 [N] = column sums of dz, or their
    sums with what dw and db hold (see ppo.h)."""
    code, gpu = _kind(dz)
    dt = dz.dtype
    M, N = dz.shape
    K = x.shape[1]
    pd, ldd = _mat(dz, dt, gpu, (M, N), "dz")
    px, ldx = _mat(x, dt, gpu, (M, K), "x")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_linear_backward_weight(
        code, pd, ldd, px, ldx, M, N, K, _vec(dw, gpu, (N, K), "dw"), _vec(db, gpu, (N,), "db"),
        1 if accumulate else 0, pk, wb, _on(stream, gpu)), "ppo_linear_backward_weight")


def ppo_work_status(work, stream=None) -> None:
    """Synchronises the stream; raises PPO_ERR_TIMEOUT if a bounded device wait
    of a ppo_linear_* call on this workspace gave up."""
    _abi.check(_lib().ppo_work_status(_ptr(work), _stream(stream)), "ppo_work_status")


def ppo_gated_linear_workspace_bytes(M: int, N: int, K: int, dtype, J: int = 0, ldx: int = 0, ldw: int = 0,
                                     lddz: int = 0, ldw2: int = 0) -> int:
    """Bytes of workspace for a gated layer of x [M, K], w [2N, K] and, where J is
    not 0, its backward pass from dz [M, J] through w2 [J, N] (allocate it zeroed;
    pitches only where the rows are strided)."""
    if _F32 is None:
        _bind_torch()
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_gated_linear_workspace_bytes(_DTYPES.get(dtype, -1), M, N, K, J, ldx, ldw, lddz, ldw2,
                                                       ctypes.byref(n)), "ppo_gated_linear_workspace_bytes")
    return n.value


def ppo_gated_linear_forward(x, w, y, bias=None, act=_abi.ACT_SILU, pre=None, work=None, stream=None) -> None:
    """y [M, N] = act(gate) * up of x [M, K], the rows of w [2N, K] being the
    gate's and then the other projection's, bias fp32 [2N] likewise; pre [M, 2N]
    takes both (see ppo.h)."""
    code, gpu = _kind(x)
    dt = x.dtype
    M, K = x.shape
    N = y.shape[1]
    px, ldx = _mat(x, dt, gpu, (M, K), "x")
    pw, ldw = _mat(w, dt, gpu, (2 * N, K), "w")
    py, ldy = _mat(y, dt, gpu, (M, N), "y")
    pp, ldp = _mat(pre, dt, gpu, (M, 2 * N), "pre")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_gated_linear_forward(
        code, px, ldx, pw, ldw, _vec(bias, gpu, (2 * N,), "bias"), act, M, N, K, py, ldy, pp, ldp, pk, wb,
        _on(stream, gpu)), "ppo_gated_linear_forward")


def ppo_gated_linear_backward_data(dz, w2, pre, dp, act=_abi.ACT_SILU, y=None, work=None, stream=None) -> None:
    """dp [M, 2N], the gradient of pre [M, 2N], from dz [M, J] through w2 [J, N];
    y [M, N] takes the layer's output once more (see ppo.h).  dp may be pre."""
    code, gpu = _kind(dz)
    dt = dz.dtype
    M, J = dz.shape
    N = w2.shape[1]
    pd, ldd = _mat(dz, dt, gpu, (M, J), "dz")
    pw, ldw = _mat(w2, dt, gpu, (J, N), "w2")
    pp, ldp = _mat(pre, dt, gpu, (M, 2 * N), "pre")
    po, ldo = _mat(dp, dt, gpu, (M, 2 * N), "dp")
    py, ldy = _mat(y, dt, gpu, (M, N), "y")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_gated_linear_backward_data(
        code, pd, ldd, pw, ldw, pp, ldp, act, M, N, J, po, ldo, py, ldy, pk, wb, _on(stream, gpu)),
        "ppo_gated_linear_backward_data")


# ---- policy over any number of actions --------------------------------------------
def _of(t, dtypes, gpu, shape, name):
    """Address of a contiguous argument of one of the types."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != gpu or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor {tuple(shape)} of {dtypes[0]} on cuda:{gpu} is wanted, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")
    return t.data_ptr()


def _allowed(mask, gpu, shape):
    """(address, pitch) of a mask of bytes."""
    if mask is None:
        return None, 0
    if mask.dtype not in _BYTES:
        raise ValueError(f"mask: torch.bool or torch.uint8 is wanted, got {mask.dtype}")
    return _mat(mask, mask.dtype, gpu, shape, "mask")


def ppo_action_logp(logits, action, logp=None, entropy=None, mask=None, stream=None) -> None:
    """logp fp32 [M] of action int32 [M] and entropy fp32 [M] of the rows of
    logits [M, V], over the actions where mask [M, V] (bool) is set (see ppo.h)."""
    code, gpu = _kind(logits)
    M, V = shape = logits.shape
    pl, ld = _mat(logits, logits.dtype, gpu, shape, "logits")
    pm, ldm = _allowed(mask, gpu, shape)
    _check(_lib().ppo_action_logp(
        code, pl, ld, M, V, pm, ldm, _of(action, _I32S, gpu, (M,), "action"), _vec(logp, gpu, (M,), "logp"),
        _vec(entropy, gpu, (M,), "entropy"), _on(stream, gpu)), "ppo_action_logp")


def ppo_action_loss_workspace_bytes() -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_action_loss_workspace_bytes(ctypes.byref(n)), "ppo_action_loss_workspace_bytes")
    return n.value


def ppo_action_loss_grad(logits, action, logp_old, adv, dlogits, scale, logp_ref=None, weight=None, mask=None,
                         clip_low=0.2, clip_high=0.2, kl_coef=0.0, ent_coef=0.0, logp=None, entropy=None,
                         stats=None, work=None, stream=None) -> None:
    """dlogits [M, V], the gradient of the clipped policy loss with respect to
    logits [M, V], for action int32 [M] and logp_old, adv, logp_ref, weight fp32
    [M]; stats fp32 [8] takes the loss and its terms (see ppo.h).  dlogits may be
    logits."""
    code, gpu = _kind(logits)
    dt = logits.dtype
    M, V = shape = logits.shape
    row = (M,)
    pl, ld = _mat(logits, dt, gpu, shape, "logits")
    pm, ldm = _allowed(mask, gpu, shape)
    pd, ldd = _mat(dlogits, dt, gpu, shape, "dlogits")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_action_loss_grad(
        code, pl, ld, M, V, pm, ldm, _of(action, _I32S, gpu, row, "action"),
        _vec(logp_old, gpu, row, "logp_old"), _vec(adv, gpu, row, "adv"), _vec(logp_ref, gpu, row, "logp_ref"),
        _vec(weight, gpu, row, "weight"), scale, clip_low, clip_high, kl_coef, ent_coef, pd, ldd,
        _vec(logp, gpu, row, "logp"), _vec(entropy, gpu, row, "entropy"), _vec(stats, gpu, (8,), "stats"), pk, wb,
        _on(stream, gpu)), "ppo_action_loss_grad")


# ---- gradient norm of many tensors --------------------------------------------------
class TensorList:
    """The places of tensors on one GPU, as ppo_grad_norm and ppo_clip_grad_norm
    take them (contiguous, float32 or bfloat16).  It keeps the tensors alive; a
    program whose gradients stay where they are makes it once."""

    def __init__(self, tensors):
        if _F32 is None:
            _bind_torch()
        self.tensors = tuple(tensors)
        self.gpu = self.tensors[0].get_device() if self.tensors else -1
        self.array = (_abi.Tensor * max(1, len(self.tensors)))()
        for k, t in enumerate(self.tensors):
            code = _DTYPES.get(t.dtype)
            if code is None:
                raise ValueError(f"tensor {k}: float32 or bfloat16 is wanted, got {t.dtype}")
            if t.get_device() != self.gpu or self.gpu < 0:
                raise ValueError(f"tensor {k}: CUDA tensors of one GPU are wanted, got one on {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"tensor {k}: must be contiguous")
            self.array[k] = _abi.Tensor(t.data_ptr(), t.numel(), code, 0)

    def __len__(self):
        return len(self.tensors)


def _listed(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def ppo_grad_norm_workspace_bytes(tensors) -> int:
    """Bytes of workspace for a TensorList, a sequence of tensors or their number."""
    n = ctypes.c_size_t()
    _abi.check(_lib().ppo_grad_norm_workspace_bytes(tensors if isinstance(tensors, int) else len(tensors),
                                                    ctypes.byref(n)), "ppo_grad_norm_workspace_bytes")
    return n.value


def _list_gpu(norm, lists):
    """The GPU of a call on lists of tensors."""
    if _F32 is None:
        _bind_torch()
    gpu = norm.get_device()
    if gpu < 0 or gpu != _current_gpu():
        raise ValueError(f"norm is on {norm.device}, the current device is cuda:{_current_gpu()}")
    for t in lists:
        if len(t) and t.gpu != gpu:
            raise ValueError(f"the tensors are on cuda:{t.gpu}, norm is on cuda:{gpu}")
    return gpu


def ppo_grad_norm(tensors, norm, work=None, stream=None) -> None:
    """norm fp32 [1] = the 2-norm over all elements of the tensors (a TensorList or
    a sequence; see ppo.h)."""
    tensors = _listed(tensors)
    gpu = _list_gpu(norm, (tensors,))
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_grad_norm(tensors.array, len(tensors), _vec(norm, gpu, (1,), "norm"), pk, wb,
                                _on(stream, gpu)), "ppo_grad_norm")


def ppo_clip_grad_norm(tensors, max_norm, norm, out=None, work=None, stream=None) -> None:
    """Scales the tensors, or writes them scaled to out's, by min(1, max_norm /
    (norm + 1e-6)); norm fp32 [1] receives the norm before clipping (see ppo.h)."""
    tensors = _listed(tensors)
    out = None if out is None else _listed(out)
    gpu = _list_gpu(norm, (tensors,) if out is None else (tensors, out))
    if out is not None and len(out) != len(tensors):
        raise ValueError(f"out: {len(tensors)} tensors are wanted, got {len(out)}")
    pk, wb = _work_of(work, gpu)
    _check(_lib().ppo_clip_grad_norm(tensors.array, None if out is None else out.array, len(tensors), max_norm,
                                     _vec(norm, gpu, (1,), "norm"), pk, wb, _on(stream, gpu)),
           "ppo_clip_grad_norm")


# ---- context ------------------------------------------------------------------
def ppo_create(cfg: PpoConfig, init_params=None):
    h = ctypes.c_void_p()
    if init_params is not None:
        import numpy as np
        init_params = np.ascontiguousarray(init_params, dtype=np.float32)
    _abi.check(_lib().ppo_create(ctypes.byref(cfg), _ptr(init_params), ctypes.byref(h)),
               "ppo_create")
    return h


def ppo_destroy(ctx) -> None:
    _abi.check(_lib().ppo_destroy(ctx), "ppo_destroy")


class _DevArray:
    """Zero-copy view of library-owned device memory (CUDA array interface)."""

    def __init__(self, ptr: int, n: int, typestr: str = "<f4"):
        self.__cuda_array_interface__ = {"shape": (n,), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


def ppo_buffers(ctx, n_params: int):
    """Torch views (params, grad, adam_m, adam_v) of the context's buffers."""
    import torch
    ps = [ctypes.c_void_p() for _ in range(4)]
    _abi.check(_lib().ppo_buffers(ctx, *[ctypes.byref(p) for p in ps]), "ppo_buffers")
    return tuple(torch.as_tensor(_DevArray(p.value, n_params), device="cuda") for p in ps)


def ppo_params_changed(ctx, stream=None) -> None:
    _abi.check(_lib().ppo_params_changed(ctx, _stream(stream)), "ppo_params_changed")


def ppo_get_step(ctx) -> int:
    n = ctypes.c_int64()
    _abi.check(_lib().ppo_get_step(ctx, ctypes.byref(n)), "ppo_get_step")
    return n.value


def ppo_minibatch_loss_grad(ctx, obs, act_disc, act_cont, logp_old, adv, ret, idx,
                            adv_stats=None, stats6=None, stream=None) -> None:
    B = obs.shape[0]
    _abi.check(_lib().ppo_minibatch_loss_grad(
        ctx, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(adv), _ptr(ret),
        _ptr(idx), B, idx.numel(), _ptr(adv_stats), _ptr(stats6), _stream(stream)),
        "ppo_minibatch_loss_grad")


def ppo_minibatch_loss_grad_fresh(ctx, obs, act_disc, act_cont, logp_old, rew, done, boot, envs,
                                  adv_mode, gamma, lam, stats6=None, adv_out=None, ret_out=None,
                                  stream=None) -> None:
    T, N = rew.shape
    _abi.check(_lib().ppo_minibatch_loss_grad_fresh(
        ctx, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(rew), _ptr(done),
        _ptr(boot), T, N, _ptr(envs), envs.numel(), adv_mode, gamma, lam, _ptr(stats6),
        _ptr(adv_out), _ptr(ret_out), _stream(stream)), "ppo_minibatch_loss_grad_fresh")


def ppo_policy_act(ctx, obs, seed, draw0, act_disc, act_cont=None, logp=None, value=None,
                   stream=None) -> None:
    """Sampled actions, their log-probability and the value for the rows of obs."""
    _abi.check(_lib().ppo_policy_act(
        ctx, _ptr(obs), obs.shape[0], seed & 0xFFFFFFFF, int(draw0), _ptr(act_disc),
        _ptr(act_cont), _ptr(logp), _ptr(value), _stream(stream)), "ppo_policy_act")


def ppo_muon_step(ctx, lr, grad_norm=None, stream=None) -> None:
    _abi.check(_lib().ppo_muon_step(ctx, lr, _ptr(grad_norm), _stream(stream)), "ppo_muon_step")


def ppo_adam_step(ctx, lr, grad_norm=None, stream=None) -> None:
    _abi.check(_lib().ppo_adam_step(ctx, lr, _ptr(grad_norm), _stream(stream)), "ppo_adam_step")


def ppo_update(ctx, obs, act_disc, act_cont, logp_old, val, rew, done, boot, epochs,
               minibatches, gamma, lam, lr, seed, stats=None, stream=None) -> None:
    T, N = val.shape
    _abi.check(_lib().ppo_update(
        ctx, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(val), _ptr(rew),
        _ptr(done), _ptr(boot), T, N, epochs, minibatches, gamma, lam, lr, seed & 0xFFFFFFFF,
        _ptr(stats), _stream(stream)), "ppo_update")


def ppo_update_host(ctx, obs, act_disc, act_cont, logp_old, val, rew, done, boot, epochs,
                    minibatches, gamma, lam, lr, seed, stats=None, stream=None) -> None:
    T, N = val.shape
    _abi.check(_lib().ppo_update_host(
        ctx, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(val), _ptr(rew),
        _ptr(done), _ptr(boot), T, N, epochs, minibatches, gamma, lam, lr, seed & 0xFFFFFFFF,
        _ptr(stats), _stream(stream)), "ppo_update_host")


def ppo_update_host_async(ctx, obs, act_disc, act_cont, logp_old, val, rew, done, boot, epochs,
                          minibatches, gamma, lam, lr, seed, stats=None, stream=None) -> None:
    T, N = val.shape
    _abi.check(_lib().ppo_update_host_async(
        ctx, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(val), _ptr(rew),
        _ptr(done), _ptr(boot), T, N, epochs, minibatches, gamma, lam, lr, seed & 0xFFFFFFFF,
        _ptr(stats), _stream(stream)), "ppo_update_host_async")


def ppo_host_wait(ctx) -> None:
    _abi.check(_lib().ppo_host_wait(ctx), "ppo_host_wait")


def ppo_stage_name(stage: int) -> str:
    return _lib().ppo_stage_name(stage).decode()


def ppo_update_profile(ctx, obs, act_disc, act_cont, logp_old, val, rew, done, boot, epochs,
                       minibatches, gamma, lam, lr, seed, stats=None, stream=None):
    """One profiled update; returns {stage name: (total ms, launches)}."""
    T, N = val.shape
    ms = (ctypes.c_float * _abi.NUM_STAGES)()
    cnt = (ctypes.c_int32 * _abi.NUM_STAGES)()
    _abi.check(_lib().ppo_update_profile(
        ctx, _ptr(obs), _ptr(act_disc), _ptr(act_cont), _ptr(logp_old), _ptr(val), _ptr(rew),
        _ptr(done), _ptr(boot), T, N, epochs, minibatches, gamma, lam, lr, seed & 0xFFFFFFFF,
        _ptr(stats), ms, cnt, _stream(stream)), "ppo_update_profile")
    return {ppo_stage_name(i): (ms[i], cnt[i]) for i in range(_abi.NUM_STAGES) if cnt[i]}


def ppo_sync_status(ctx, stream=None) -> None:
    _abi.check(_lib().ppo_sync_status(ctx, _stream(stream)), "ppo_sync_status")


def ppo_set_collective(ctx, world: int, rank: int, fn=None, user=None) -> None:
    """Registers the collective of the data-parallel update (see ppo.h); fn is
    an _abi.COLLECTIVE_FN (e.g. TorchCollective(...).fn)."""
    cfn = fn if fn is not None else ctypes.cast(None, _abi.COLLECTIVE_FN)
    _abi.check(_lib().ppo_set_collective(ctx, world, rank, cfn, user), "ppo_set_collective")


class TorchCollective:
    """The library's collective over torch.distributed: an in-place sum
    all-reduce of fp32 buffers and an all-gather of fp64 buffers, issued on
    the stream the library passes (so that they are ordered with its
    kernels).  device: "cuda" (NCCL; buffers are device pointers) or "cpu"
    (gloo; host pointers).  Keep the object alive while the context uses it."""

    def __init__(self, group=None, device: str = "cuda"):
        self.group = group
        self.device = device
        self.fn = _abi.COLLECTIVE_FN(self._call)
        self.error = None

    def _view(self, ptr: int, n: int, fp64: bool):
        import torch
        if self.device == "cuda":
            return torch.as_tensor(_DevArray(ptr, n, "<f8" if fp64 else "<f4"), device="cuda")
        import numpy as np
        ct = ctypes.c_double if fp64 else ctypes.c_float
        return torch.from_numpy(np.ctypeslib.as_array((ct * n).from_address(ptr)))

    def _call(self, user, op, buf, count, stream):
        try:
            import contextlib
            import torch
            import torch.distributed as dist
            world = dist.get_world_size(self.group)
            rank = dist.get_rank(self.group)
            # the library's stream (the legacy default stream arrives as NULL)
            if self.device != "cuda":
                ctxm = contextlib.nullcontext()
            else:
                ctxm = torch.cuda.stream(torch.cuda.ExternalStream(stream) if stream
                                         else torch.cuda.default_stream())
            with ctxm:
                if op == _abi.COLL_ALLREDUCE_SUM_F32:
                    dist.all_reduce(self._view(buf, count, False), group=self.group)
                elif op == _abi.COLL_ALLGATHER_F64:
                    t = self._view(buf, world * count, True)
                    parts = list(t.split(count))
                    mine = parts[rank].clone()
                    dist.all_gather(parts, mine, group=self.group)
                else:
                    return 1
            return 0
        except Exception as e:   # reported to the library as a failed collective
            self.error = e
            return 1


def ppo_set_step_trace(ctx, trace=None, max_steps: int = 0) -> None:
    """Per-step copies of params, m, v and the gradient inside ppo_update (see ppo.h)."""
    _abi.check(_lib().ppo_set_step_trace(ctx, _ptr(trace), max_steps), "ppo_set_step_trace")


def ppo_set_wait_limit(ctx, limit_ns: int = 0) -> None:
    """Limit of the cooperative kernels' grid-barrier waits (0: the 2 s default)."""
    _abi.check(_lib().ppo_set_wait_limit(ctx, int(limit_ns)), "ppo_set_wait_limit")


class Context:
    """Owns one ppo_ctx (parameters, gradient, Adam state, workspaces)."""

    def __init__(self, cfg: PpoConfig, init_params=None):
        self.cfg = cfg
        self.n_params = ppo_param_count(cfg)
        self.handle = ppo_create(cfg, init_params)
        self.params, self.grad, self.adam_m, self.adam_v = ppo_buffers(self.handle, self.n_params)

    def close(self):
        if self.handle is not None:
            ppo_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def minibatch_loss_grad(self, *a, **k):
        return ppo_minibatch_loss_grad(self.handle, *a, **k)

    def minibatch_loss_grad_fresh(self, *a, **k):
        return ppo_minibatch_loss_grad_fresh(self.handle, *a, **k)

    def policy_act(self, *a, **k):
        return ppo_policy_act(self.handle, *a, **k)

    def muon_step(self, *a, **k):
        return ppo_muon_step(self.handle, *a, **k)

    def adam_step(self, *a, **k):
        return ppo_adam_step(self.handle, *a, **k)

    def update(self, *a, **k):
        return ppo_update(self.handle, *a, **k)

    def update_host(self, *a, **k):
        return ppo_update_host(self.handle, *a, **k)

    def update_host_async(self, *a, **k):
        return ppo_update_host_async(self.handle, *a, **k)

    def host_wait(self):
        return ppo_host_wait(self.handle)

    def update_profile(self, *a, **k):
        return ppo_update_profile(self.handle, *a, **k)

    def sync_status(self, stream=None):
        return ppo_sync_status(self.handle, stream)

    def params_changed(self, stream=None):
        return ppo_params_changed(self.handle, stream)

    def step(self) -> int:
        return ppo_get_step(self.handle)

    def set_step_trace(self, trace=None, max_steps: int = 0):
        return ppo_set_step_trace(self.handle, trace, max_steps)

    def set_wait_limit(self, limit_ns: int = 0):
        return ppo_set_wait_limit(self.handle, limit_ns)

    def set_collective(self, world: int, rank: int, collective=None):
        """Data-parallel update over `world` ranks (collective: a
        TorchCollective, or None with world == 1)."""
        self._collective = collective   # kept alive with the context
        return ppo_set_collective(self.handle, world, rank,
                                  collective.fn if collective is not None else None)
