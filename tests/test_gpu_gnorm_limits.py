"""The gradient norm of very many large elements.

Bounds, u = 2^-24: 32 squares of a thread are summed in fp32 in four runs of 8 multiply-adds and
two levels (10 u at most); those sums and blocks' partial ones with compensation (2 u each), the
lanes and warps of a block over 8 levels (8 u), twice: for the partial sums and for their total.
30 u of the sum are 15 of the norm, and its own rounding makes 16."""
import numpy as np
import pytest

from test_gpu_gnorm import P, workspace  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NORM = 16 * U


@pytest.mark.parametrize("n,count", [(640, 1 << 25), (1280, 1 << 24), (33, 1 << 28)])
def test_large_elements_many_times_over(P, n, count):
    """A sum of squares past fp32's largest number, of squares that are not: its root is
    representable."""
    import torch
    t = torch.full((count,), 2.0 ** 47, dtype=torch.bfloat16, device="cuda")
    ts = P.TensorList([t] * n)
    norm, w = torch.zeros(1, device="cuda"), workspace(P, n)
    P.ppo_grad_norm(ts, norm, w)
    want = 2.0 ** 47 * float(n * count) ** 0.5
    assert abs(float(norm) - want) <= NORM * want, (float(norm), want)


def test_clip_of_large_elements(P):
    """The same where they are clipped: not a factor of 0."""
    import torch
    count, n, value = 15_500_000, 600, 1.375 * 2.0 ** 47
    if torch.cuda.mem_get_info()[0] < n * count * 2 + 2 ** 30:
        pytest.skip("needs 20 GB")
    src = torch.full((count,), value, dtype=torch.bfloat16, device="cuda")
    dst = torch.zeros(n, count, dtype=torch.bfloat16, device="cuda")
    norm, w = torch.zeros(1, device="cuda"), workspace(P, n)
    want = value * float(n * count) ** 0.5
    P.ppo_clip_grad_norm([src] * n, want / 4, norm, dst.unbind(0), w)
    assert abs(float(norm) - want) <= NORM * want
    assert all((d == value / 4).all() for d in dst)
