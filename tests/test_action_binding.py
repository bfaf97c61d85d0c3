"""What the binding of the operators over many actions, gated layers and gradient
norms makes of its arguments, and what the library refuses before it needs a
device (CPU: tensors that say they are on a GPU, a library that records)."""
import ctypes

import pytest
import torch

import policy_rl_gb300 as P
from policy_rl_gb300 import _abi
from test_trunk_binding import OnGpu, lib, zeros  # noqa: F401


def typed(dtype, *shape, index=0):
    return OnGpu(torch.zeros(*shape, dtype=dtype), index)


M, N, K, J, V = 6, 4, 8, 5, 7


def calls(index):
    z = lambda *s: zeros(*s, index=index)
    i = lambda *s: typed(torch.int32, *s, index=index)
    b = lambda *s: typed(torch.bool, *s, index=index)
    return {
        "ppo_gated_linear_forward": dict(x=z(M, K), w=z(2 * N, K), y=z(M, N), bias=z(2 * N), pre=z(M, 2 * N),
                                         work=z(64)),
        "ppo_gated_linear_backward_data": dict(dz=z(M, J), w2=z(J, N), pre=z(M, 2 * N), dp=z(M, 2 * N), y=z(M, N),
                                               work=z(64)),
        "ppo_action_logp": dict(logits=z(M, V), action=i(M), logp=z(M), entropy=z(M), mask=b(M, V)),
        "ppo_action_loss_grad": dict(logits=z(M, V), action=i(M), logp_old=z(M), adv=z(M), dlogits=z(M, V),
                                     logp_ref=z(M), weight=z(M), mask=b(M, V), logp=z(M), entropy=z(M), stats=z(8),
                                     work=z(64)),
    }


def call(name, args):
    getattr(P, name)(**args, **({"scale": 1.0} if name == "ppo_action_loss_grad" else {}))


@pytest.mark.parametrize("name", list(calls(0)))
def test_tensors_of_two_devices_are_refused(lib, name):  # noqa: F811
    lib.gpu = 1
    call(name, calls(1)[name])
    assert len(lib.calls) == 1
    for k in calls(1)[name]:
        for other in (0, -1):
            with pytest.raises(ValueError):
                call(name, {**calls(1)[name], k: calls(other)[name][k]})
    lib.gpu = 0
    with pytest.raises(ValueError):
        call(name, calls(1)[name])
    assert len(lib.calls) == 1


@pytest.mark.parametrize("name", list(calls(0)))
def test_shapes_and_types_are_checked(lib, name):  # noqa: F811
    for k, t in calls(0)[name].items():
        if k in ("work", "logits", "x", "dz"):
            continue
        shape = list(t.shape)
        bad = [typed(torch.float64, *shape), typed(t.dtype, *(shape[:-1] + [shape[-1] + 1]))]
        if len(shape) == 2:
            bad.append(OnGpu(torch.zeros(shape[1], shape[0], dtype=t.dtype).t()))
        for v in bad:
            if k == "y" and v.shape != t.shape and name == "ppo_gated_linear_forward":
                continue            # y gives N: the others no longer fit it, which another loop turn checks
            with pytest.raises(ValueError):
                call(name, {**calls(0)[name], k: v})
    assert not lib.calls


def test_pitches_reach_the_library(lib):  # noqa: F811
    l, d = torch.zeros(M, 12)[:, :V], torch.zeros(M, 9)[:, :V]
    m = torch.zeros(M, 20, dtype=torch.bool)[:, :V]
    P.ppo_action_loss_grad(OnGpu(l), typed(torch.int32, M), zeros(M), zeros(M), OnGpu(d), 0.5, mask=OnGpu(m))
    (_, a), = lib.calls
    assert a[1:7] == (l.data_ptr(), 12, M, V, m.data_ptr(), 20) and a[17:19] == (d.data_ptr(), 9)


def test_lists_of_tensors(lib):  # noqa: F811
    ts = P.TensorList([zeros(3, 4), zeros(0), typed(torch.bfloat16, 5)])
    assert [(t.count, t.dtype) for t in ts.array] == [(12, 0), (0, 0), (5, 1)] and len(ts) == 3
    for bad in ([zeros(3), zeros(3, index=1)], [zeros(3, index=-1)], [typed(torch.float16, 3)],
                [OnGpu(torch.zeros(4, 4).t())]):
        with pytest.raises(ValueError):
            P.TensorList(bad)
    norm, work = zeros(1), zeros(64)
    P.ppo_clip_grad_norm(ts, 1.0, norm, work=work)
    P.ppo_grad_norm([zeros(3)], norm, work)
    assert [c[0] for c in lib.calls] == ["ppo_clip_grad_norm", "ppo_grad_norm"]
    for bad in (dict(norm=zeros(1, index=1)), dict(norm=zeros(2)), dict(out=[zeros(3)]), dict(work=zeros(64, index=1)),
                dict(tensors=[zeros(3, index=1)])):
        with pytest.raises(ValueError):
            P.ppo_clip_grad_norm(**{**dict(tensors=ts, max_norm=1.0, norm=norm, work=work), **bad})
    assert len(lib.calls) == 2


# ---- the library's own checks, before it looks for a device -------------------------
INVALID, ALIGN, CUDA, UNSUPPORTED = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from policy_rl_gb300 import build
    build.build()
    return _abi.load()


A16 = ctypes.c_void_p(1 << 20)


def at(n):
    return ctypes.c_void_p((1 << 20) + n)


def test_actions_refused(L):
    def loss(dtype=0, l=A16, ld=8, M=4, V=8, mask=None, ldm=0, a=A16, old=A16, adv=A16, ref=None, w=None, lo=0.2, hi=0.2,
             dl=at(1 << 16), lddl=8, stats=None, work=None, wb=0):
        return L.ppo_action_loss_grad(dtype, l, ld, M, V, mask, ldm, a, old, adv, ref, w, 1.0, lo, hi, 0.0, 0.0, dl, lddl,
                                      None, None, stats, work, wb, None)
    size = ctypes.c_size_t()
    assert L.ppo_action_loss_workspace_bytes(ctypes.byref(size)) == 0 and L.ppo_action_loss_workspace_bytes(None) == 1
    for bad in (dict(dtype=2), dict(l=None), dict(a=None), dict(old=None), dict(adv=None), dict(dl=None), dict(ld=7),
                dict(M=0), dict(V=0), dict(lddl=7), dict(lo=-1.0), dict(hi=float("nan")), dict(mask=A16, ldm=7),
                dict(dl=A16, lddl=9), dict(stats=A16), dict(stats=A16, work=A16, wb=size.value - 1)):
        assert loss(**bad) == INVALID, bad
    for bad in (dict(l=at(2)), dict(dl=at(1)), dict(a=at(2)), dict(old=at(1)), dict(adv=at(2)), dict(ref=at(2)),
                dict(w=at(1)), dict(stats=at(2), work=A16, wb=size.value),
                dict(stats=A16, work=at(8), wb=size.value)):
        assert loss(**bad) == ALIGN, bad
    assert loss(V=262145, ld=262145, lddl=262145) == UNSUPPORTED and loss(M=1 << 31) == UNSUPPORTED
    assert L.ppo_action_logp(0, A16, 8, 4, 8, None, 0, None, A16, None, None) == INVALID
    assert L.ppo_action_logp(1, at(1), 8, 4, 8, None, 0, A16, A16, None, None) == ALIGN
    assert L.ppo_action_logp(0, A16, 8, 4, 300000, None, 0, A16, A16, None, None) == INVALID


def test_gated_refused(L):
    size = ctypes.c_size_t()
    get = lambda *a: L.ppo_gated_linear_workspace_bytes(*a, 0, 0, 0, 0, ctypes.byref(size))
    assert get(1, 8, 16, 24, 32) == 0 and size.value > 0
    for bad in ((2, 8, 16, 24, 0), (1, 0, 16, 24, 0), (1, 8, 0, 24, 0), (1, 8, 16, 0, 0), (1, 8, 16, 24, -1),
                (1, 8, 1 << 28, 24, 0), (1, 1 << 29, 16, 24, 0)):
        assert get(*bad) == INVALID, bad
    need = size.value

    def fwd(dtype=1, x=A16, ldx=24, w=A16, ldw=24, act=2, M=8, N=16, K=24, y=A16, ldy=16, pre=None, ldp=0, work=A16,
            wb=1 << 30):
        return L.ppo_gated_linear_forward(dtype, x, ldx, w, ldw, None, act, M, N, K, y, ldy, pre, ldp, work, wb, None)

    def bwd(dtype=1, dz=A16, lddz=32, w=A16, ldw=16, pre=A16, ldp=32, act=2, M=8, N=16, J=32, dp=at(1 << 16), lddp=32, y=None,
            ldy=0, work=A16, wb=1 << 30):
        return L.ppo_gated_linear_backward_data(dtype, dz, lddz, w, ldw, pre, ldp, act, M, N, J, dp, lddp, y, ldy, work, wb,
                                                None)
    for bad in (dict(dtype=5), dict(x=None), dict(w=None), dict(y=None), dict(ldx=23), dict(ldw=8), dict(ldy=15), dict(act=4),
                dict(M=0), dict(pre=A16, ldp=31), dict(work=None), dict(wb=16)):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(x=at(8)), dict(w=at(2)), dict(y=at(4)), dict(pre=at(8), ldp=32), dict(work=at(8))):
        assert fwd(**bad) == ALIGN, bad
    for bad in (dict(dz=None), dict(w=None), dict(pre=None), dict(dp=None), dict(lddz=31), dict(ldw=15), dict(ldp=31),
                dict(lddp=31), dict(dp=A16, lddp=40), dict(y=A16, ldy=15), dict(wb=0)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(y=at(2), ldy=16) == ALIGN and need > 0


def test_gated_workspaces_hold_no_sums_that_stay_in_their_tiles(L):
    size = ctypes.c_size_t()
    for M, N, K in ((32768, 2048, 512), (1, 2048, 512), (8192, 4096, 4096)):
        assert L.ppo_gated_linear_workspace_bytes(1, M, N, K, 512, 0, 0, 0, 0, ctypes.byref(size)) == 0
        assert size.value < 1 << 20, (M, N, K, size.value)


def test_norms_refused(L):
    size = ctypes.c_size_t()
    for n in (-1, 1 << 20):
        assert L.ppo_grad_norm_workspace_bytes(n, ctypes.byref(size)) == INVALID
    assert L.ppo_grad_norm_workspace_bytes(4, ctypes.byref(size)) == 0
    T = _abi.Tensor

    def clip(ts, outs=None, n=None, max_norm=1.0, norm=A16, work=A16, wb=size.value):
        a = (T * max(1, len(ts)))(*ts)
        b = None if outs is None else (T * max(1, len(outs)))(*outs)
        return L.ppo_clip_grad_norm(a, b, len(ts) if n is None else n, max_norm, norm, work, wb, None)
    one, two = T(1 << 20, 16, 0, 0), T((1 << 20) + 64, 16, 0, 0)
    for bad in (dict(ts=[T(1 << 20, -1, 0, 0)]), dict(ts=[T(1 << 20, 1, 2, 0)]), dict(ts=[T(1 << 20, 1, 0, 1)]), dict(ts=[T(None, 1, 0, 0)]),
                dict(ts=[one], norm=None), dict(ts=[one], work=None), dict(ts=[one], wb=8), dict(ts=[one], n=-1),
                dict(ts=[one], max_norm=float("nan")), dict(ts=[one, one]), dict(ts=[one, T((1 << 20) + 60, 16, 0, 0)]),
                dict(ts=[two, one, T((1 << 20) + 126, 2, 1, 0)]),
                dict(ts=[one], outs=[T(1 << 22, 15, 0, 0)]), dict(ts=[one], outs=[T(1 << 22, 16, 1, 0)]),
                dict(ts=[one], outs=[T((1 << 20) + 4, 16, 0, 0)]), dict(ts=[one, two], outs=[two, T(1 << 22, 16, 0, 0)]),
                dict(ts=[one, two], outs=[T(1 << 22, 16, 0, 0), T(1 << 22, 16, 0, 0)])):
        assert clip(**bad) == INVALID, bad
    for bad in (dict(ts=[T((1 << 20) + 2, 1, 0, 0)]), dict(ts=[T((1 << 20) + 1, 1, 1, 0)]), dict(ts=[one], norm=at(2)),
                dict(ts=[one], work=at(8))):
        assert clip(**bad) == ALIGN, bad
    if not torch.cuda.is_available():      # allowed: adjacent tensors, an out that is its input, the same input twice
        assert clip([two, one]) == CUDA and clip([one, two], [one, two]) == CUDA
        assert clip([one, one], [T(1 << 22, 16, 0, 0), T(1 << 23, 16, 0, 0)]) == CUDA and clip([]) == CUDA
