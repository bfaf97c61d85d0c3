"""What the binding of the trunk operators makes of its tensors' shapes, strides
and devices (CPU: tensors that say they are on a GPU, and a library that
records its arguments)."""
import pytest
import torch

import policy_rl_gb300 as P
from policy_rl_gb300 import _abi


class OnGpu:
    """A CPU tensor that claims to be on GPU `index`."""

    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda, self.device = t, index, True, f"cuda:{index}"

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Recorder:
    def __init__(self):
        self.calls = []

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
