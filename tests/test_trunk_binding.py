"""What the binding of the trunk operators makes of its tensors' shapes, strides
and devices (CPU: tensors that say they are on a GPU, and a library that
records its arguments)."""
import pytest
import torch

import policy_rl_gb300 as P
from policy_rl_gb300 import _abi


class OnGpu:
    """A CPU tensor that claims to be on GPU `index` (-1: on the CPU)."""

    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda, self.device = t, index, index >= 0, f"cuda:{index}"

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Recorder:
    def __init__(self):
        self.calls, self.gpu = [], 0

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(_abi, "_lib", r)
    P._bind_torch()
    monkeypatch.setattr(P, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(P, "_current_gpu", lambda: r.gpu)
    return r


def zeros(*shape, index=0):
    return OnGpu(torch.zeros(*shape), index)


@pytest.mark.parametrize("N,W,full", [(1, 8, 5), (3, 8, 3), (1, 1, 4)])
def test_pitch_of_rollout_views(lib, N, W, full):
    """The first N of `full` environments, as they lie."""
    T = 6
    p, h = torch.zeros(T, full, 2 * W)[:, :N], torch.zeros(T, full, W)[:, :N]
    P.ppo_gated_scan_forward(OnGpu(p), OnGpu(h))
    (name, a), = lib.calls
    assert name == "ppo_gated_scan_forward"
    assert a[1] == p.data_ptr() and a[9] == h.data_ptr() and a[6:9] == (T, N, W)
    rows = full if N == 1 else 1
    assert a[2] == rows * 2 * W and a[10] == rows * W


def test_views_without_one_pitch_are_refused(lib):
    base = torch.zeros(6, 5, 8)
    for bad in (base[:, :2], base[..., ::2], base[:, :1].expand(6, 2, 8), base[:1, :1].expand(6, 1, 8),
                torch.zeros(64).as_strided((6, 1, 8), (4, 8, 1))):
        h = OnGpu(bad)
        with pytest.raises(ValueError):
            P.ppo_gated_scan_forward(zeros(*bad.shape[:2], 2 * bad.shape[2]), h)
    assert not lib.calls


def calls():
    """Every operator with every tensor argument: (call, names), arguments by name."""
    T, N, H, M, D = 3, 2, 4, 6, 8
    m = lambda *s: dict(shape=s)
    return {
        "ppo_layernorm_forward": (dict(x=m(M, D), gamma=m(D), beta=m(D), y=m(M, D), stats=m(M, 2)), {}),
        "ppo_layernorm_backward": (dict(dy=m(M, D), x=m(M, D), gamma=m(D), stats=m(M, 2), dx=m(M, D), dgamma=m(D),
                                        dbeta=m(D), dres=m(M, D), work=m(64)), {}),
        "ppo_gated_scan_forward": (dict(p=m(T, N, 2 * H), h=m(T, N, H), h0=m(N, H), done=m(T, N), done0=m(N),
                                        hT=m(N, H), carry=m(1, N, H)), {}),
        "ppo_gated_scan_backward": (dict(dh=m(T, N, H), p=m(T, N, 2 * H), carry=m(1, N, H), dp=m(T, N, 2 * H),
                                         done=m(T, N), done0=m(N), dhT=m(N, H), dh0=m(N, H)), {}),
        "ppo_linear_forward": (dict(x=m(M, D), w=m(5, D), y=m(M, 5), bias=m(5), res=m(M, 5), pre=m(M, 5),
                                    work=m(64)), {}),
        "ppo_linear_backward_data": (dict(dz=m(M, 5), w=m(5, D), dx=m(M, D), pre=m(M, D), res=m(M, D), work=m(64)),
                                     dict(act=3)),
        "ppo_linear_backward_weight": (dict(dz=m(M, 5), x=m(M, D), dw=m(5, D), db=m(5), work=m(64)), {}),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_tensors_of_two_devices_are_refused(lib, name):
    tensors, other = calls()[name]
    given = {k: zeros(*v["shape"], index=1) for k, v in tensors.items()}
    lib.gpu = 1
    getattr(P, name)(**given, **other)          # all on one GPU, whichever
    assert len(lib.calls) == 1
    for k, v in tensors.items():
        for index in (0, -1):
            with pytest.raises(ValueError):
                getattr(P, name)(**{**given, k: zeros(*v["shape"], index=index)}, **other)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("name", list(calls()))
def test_another_device_than_the_current_one_is_refused(lib, name):
    """A launch goes to the current device: its kernel cannot read the other's memory."""
    tensors, other = calls()[name]
    lib.gpu = 0
    with pytest.raises(ValueError):
        getattr(P, name)(**{k: zeros(*v["shape"], index=1) for k, v in tensors.items()}, **other)
    assert not lib.calls
