"""The head over many actions on rows of the trunk's output as they lie in a caller's buffer."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,V", [(70, 64, 33), (5, 24, 1001), (300, 33, 9), (1, 40, 7)])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_rows_of_any_pitch(M, D, V, pad, dtype):
    """x's rows may have any pitch: the results are those of the same rows without gaps."""
    import torch
    from policy_rl_gb300.trunk import ActionHead
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    head = ActionHead(M, D, V, dtype=dt, generator=g)
    x = torch.randn(M, D, generator=g, device="cuda").to(dt)
    wide = torch.full((M, D + pad), float("nan"), dtype=dt, device="cuda")[:, :D]
    wide.copy_(x)
    action = torch.randint(0, V, (M,), generator=g, device="cuda").to(torch.int32)
    adv = torch.randn(M, generator=g, device="cuda")
    got = []
    for rows in (x, wide):
        lp, st = torch.zeros(M, device="cuda"), torch.zeros(8, device="cuda")
        head.logp(rows, action, lp)
        dx = head.loss_grad(rows, action, lp, adv, 1.0 / M, ent_coef=0.01, stats=st)
        got.append([t.double().clone() for t in (lp, st, dx, head.grads["W"], head.grads["b"])])
        head.check()
    # sums of up to 64 terms (up to 300 in W's and b's gradients) in another order at most: one rounding of a
    # logit to bf16 (2^-7 between neighbours) may fall the other way, and reaches every result once
    for a, b in zip(*got):
        tol = (2.0 ** -6 if dtype == "bf16" else 2.0 ** -16)
        assert (a - b).abs().max() <= tol * a.abs().max() + 1e-12
