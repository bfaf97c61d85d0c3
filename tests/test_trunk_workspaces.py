"""Which workspaces RecurrentTrunk hands to its operators (CPU: recorded calls)."""
import pytest
import torch

from policy_rl_gb300 import trunk as trunk_module


@pytest.fixture
def made(monkeypatch):
    """A trunk on the CPU and the workspaces of each call, by name."""
    from policy_rl_gb300 import build
    build.build()
    used = []
    for name in ("ppo_linear_forward", "ppo_linear_backward_data", "ppo_linear_backward_weight"):
        monkeypatch.setattr(trunk_module, name, lambda *a, work=None, **k: used.append(work))
    monkeypatch.setattr(trunk_module, "ppo_layernorm_backward", lambda *a, **k: used.append(a[-2]))
    for name in ("ppo_layernorm_forward", "ppo_gated_scan_forward", "ppo_gated_scan_backward"):
        monkeypatch.setattr(trunk_module, name, lambda *a, **k: None)
    t = trunk_module.RecurrentTrunk(6, 4, 24, 16, 40, blocks=2, device="cpu")
    return t, used


def test_acting_and_learning_share_no_workspace(made):
    """step() may run on one stream while forward() or backward() runs on another."""
    t, used = made
    x = torch.zeros(6, 4, 24, dtype=t.dtype)
    t.forward(x)
    t.backward(x)
    learning = {w.data_ptr() for w in used}
    used.clear()
    t.step(x[0], t.state())
    acting = {w.data_ptr() for w in used}
    assert learning and acting and not learning & acting


def test_check_reads_every_status_word(made, monkeypatch):
    t, used = made
    read = []
    monkeypatch.setattr(trunk_module, "ppo_work_status", lambda work, stream=None: read.append(work.data_ptr()))
    t.forward(torch.zeros(6, 4, 24, dtype=t.dtype))
    t.step(torch.zeros(4, 24, dtype=t.dtype), t.state())
    t.check()
    assert {w.data_ptr() for w in used} <= set(read)


def test_check_goes_on_after_a_failure(made, monkeypatch):
    """The first error is raised after every status word was read (and cleared)."""
    t, _ = made
    read = []

    def status(work, stream=None):
        read.append(work.data_ptr())
        raise RuntimeError(f"wait gave up {len(read)}")
    monkeypatch.setattr(trunk_module, "ppo_work_status", status)
    with pytest.raises(RuntimeError, match="gave up 1"):
        t.check()
    assert len(read) == 2
