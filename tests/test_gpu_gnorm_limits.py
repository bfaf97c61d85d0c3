"""The gradient norm of very many tensors and very many large elements.

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


@pytest.mark.parametrize("n", [641, 50000, (1 << 20) - 1])
@pytest.mark.parametrize("value", [1.921875, 1.78125])
def test_very_many_tensors(P, n, value):
    """As many partial sums as there are blocks of all launches: a plain fp32 sum of them is off by
    277 u in the norm at n = 2^20 - 1."""
    import torch
    t = torch.full((1,), value, device="cuda")
    ts = P.TensorList([t] * n)
    norm, w = torch.zeros(1, device="cuda"), workspace(P, n)
    P.ppo_grad_norm(ts, norm, w)
    want = value * float(n) ** 0.5
    assert abs(float(norm) - want) <= NORM * want, (float(norm), want)


@pytest.mark.parametrize("n", [700, 5000, 40000])
def test_clip_of_very_many_tensors(P, n):
    """Many launches, in place and elsewhere, with NaN, infinities and squares past fp32's range in
    one of them, repeated and replayed."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    flat = torch.randn(n * 8, generator=g, device="cuda")
    ts = P.TensorList(flat.view(n, 8)[:, :5].unbind(0))
    x = flat.view(n, 8)[:, :5]
    norm, w = torch.zeros(1, device="cuda"), workspace(P, n)
    kept = flat.clone()
    for extra in (None, 1e25, float("inf"), float("nan")):
        flat.copy_(kept)
        if extra is not None:
            flat.view(n, 8)[n // 2, 3] = extra
        want = float((x.double() ** 2).sum().sqrt())
        f = 0.25 * want / (want + 1e-6)
        src = x.double().clone()
        P.ppo_clip_grad_norm(ts, 0.25 * want if want == want and want < 1e38 else 1.0, norm, None, w)
        if extra is None or extra == 1e25:
            assert abs(float(norm) - want) <= NORM * want
            assert ((x.double() - src * f).abs() <= (NORM + 6 * U) * (src * f).abs() + 2.0 ** -149).all()
        elif extra != extra:
            assert torch.isnan(norm).all() and torch.isnan(x).all()
        else:
            assert torch.isinf(norm).all() and int((x == 0).sum()) == x.numel() - 1
        assert torch.equal(flat.view(n, 8)[:, 5:], kept.view(n, 8)[:, 5:])
    flat.copy_(kept)
    dst = torch.full_like(flat, 7.0)
    outs = P.TensorList(dst.view(n, 8)[:, :5].unbind(0))
    P.ppo_clip_grad_norm(ts, 0.5, norm, outs, w)
    first = dst.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.ppo_clip_grad_norm(ts, 0.5, norm, outs, w)
    for _ in range(2):
        dst.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst, first)
