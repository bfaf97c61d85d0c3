"""The norm of many tensors and their clipping on the GPU.

Bounds: the sum of squares has only positive terms; pieces of up to 64 are
summed in fp32 (off by 64 u of themselves at most, u = 2^-24), the rest in 64 bits, and the
root halves that: the norm is off by 34 u with its own rounding.  The factor adds
three roundings, a product one, the result its type's."""
import numpy as np
import pytest

import _action_ref as A
from test_gpu_trunk_ops import tdt

pytestmark = pytest.mark.gpu
NORM = 34 * A.U


@pytest.fixture(scope="module")
def P():
    import policy_rl_gb300
    return policy_rl_gb300


def workspace(P, n):
    import torch
    return torch.empty(P.ppo_grad_norm_workspace_bytes(n), dtype=torch.uint8, device="cuda")


def norm64(ts):
    return float(np.sqrt(sum(float((t.double() ** 2).sum()) for t in ts)))


def tensors(sizes, seed, dtypes=("f32",), scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(tdt(dtypes[k % len(dtypes)]))
            for k, n in enumerate(sizes)]


def check(P, ts, max_norm, in_place=False):
    import torch
    n = norm64(ts)
    f = min(1.0, max_norm / (n + 1e-6)) if max_norm > 0 else 1.0
    ref = [t.double() * f for t in ts]
    norm, alone, work = torch.full((1,), 9.0, device="cuda"), torch.full((1,), 9.0, device="cuda"), workspace(P, len(ts))
    P.ppo_grad_norm(ts, alone, work)
    out = None if in_place else [torch.full_like(t, 7.0) for t in ts]
    P.ppo_clip_grad_norm(ts, max_norm, norm, out, work)
    assert torch.equal(norm, alone)
    assert abs(float(norm) - n) <= NORM * n, (float(norm), n)
    for r, o, t in zip(ref, ts if in_place else out, ts):
        half = A.HALF["bf16"] if t.dtype == torch.bfloat16 else A.HALF["f32"]
        bound = (NORM + 5 * A.U + half) * r.abs() + 2.0 ** -133 * (1 if half > A.U else 2.0 ** -16)
        assert ((o.double() - r).abs() <= bound).all()
    return norm


SIZES = [[1], [7], [8], [1000], [4096], [4097], [1, 2, 3, 4, 5], [0, 5, 0], [33, 0, 70001, 1, 128], [100003], [3000000],
         list(range(1, 200)), [17] * 700, [65537, 5] * 40, [2] * 1500 + [50000] * 3]


@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("k", range(len(SIZES)))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(P, k, dtypes, max_norm):
    check(P, tensors(SIZES[k], k, dtypes), max_norm)
    check(P, tensors(SIZES[k], k, dtypes), max_norm, in_place=True)


@pytest.mark.parametrize("max_norm", [0.0, -1.0, float("inf")])
def test_no_clip(P, max_norm):
    import torch
    ts = tensors([1000, 33], 1)
    out = [torch.zeros_like(t) for t in ts]
    P.ppo_clip_grad_norm(ts, max_norm, torch.zeros(1, device="cuda"), out, workspace(P, 2))
    assert all(torch.equal(a, b) for a, b in zip(ts, out))


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-15, 1e-8, 1e10, 1e18, 1e25, 1e33])
@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",)])
def test_scales(P, scale, dtypes):
    """Squares past fp32's range on both sides."""
    check(P, tensors([5000, 13], 2, dtypes, scale), scale)
    check(P, tensors([5000, 13], 2, dtypes, scale) + tensors([100], 3, dtypes, 1e-3), scale)


def test_empty_lists(P):
    import torch
    for ts in ([], tensors([0, 0], 1)):
        norm = torch.full((1,), 9.0, device="cuda")
        P.ppo_clip_grad_norm(ts, 1.0, norm, work=workspace(P, 0))
        assert float(norm) == 0
        norm.fill_(9.0)
        P.ppo_grad_norm(ts, norm, work=workspace(P, len(ts)))
        assert float(norm) == 0


def test_special_values(P):
    import torch
    for dt in ("f32", "bf16"):
        for bad, n_want in ((float("nan"), "nan"), (float("inf"), "inf"), (float("-inf"), "inf")):
            ts = tensors([5000, 300], 4, (dt,))
            ts[1][17] = bad
            out = [torch.zeros_like(t) for t in ts]
            norm = torch.zeros(1, device="cuda")
            P.ppo_clip_grad_norm(ts, 1.0, norm, out, workspace(P, 2))
            if n_want == "nan":
                assert torch.isnan(norm).all() and all(torch.isnan(o).all() for o in out)
            else:       # the factor is 0: 0 everywhere but at the infinity
                assert torch.isinf(norm).all() and (out[0] == 0).all() and torch.isnan(out[1][17])
                assert (out[1][:17] == 0).all() and (out[1][18:] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_places_inside_a_buffer(P, dt):
    """Tensors on their elements' alignment, inputs and outputs off by different amounts;
    what lies beside them is kept."""
    import torch
    for sizes in ([5, 1, 30, 9], [4099, 77, 8192], [20001]):
        src = tensors(sizes, 6, (dt,))
        for shift in range(4):
            buf, dst = (torch.full((sum(sizes) + 64,), v, dtype=tdt(dt), device="cuda") for v in (3.0, 5.0))
            at, ins, outs = 1 + shift, [], []
            for t in src:
                buf[at:at + t.numel()] = t
                ins.append(buf[at:at + t.numel()])
                outs.append(dst[at + 3:at + 3 + t.numel()])
                at += t.numel() + 1
            want = [torch.empty_like(t) for t in src]
            a, b = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
            P.ppo_clip_grad_norm(src, 0.7, a, want, workspace(P, len(src)))
            P.ppo_clip_grad_norm(ins, 0.7, b, outs, workspace(P, len(src)))
            assert abs(float(a) - float(b)) <= 2 * NORM * float(a)
            keep = torch.ones_like(dst, dtype=torch.bool)
            for w, o in zip(want, outs):
                half = A.HALF[dt]
                assert ((w.double() - o.double()).abs() <= (4 * NORM + 2 * half) * w.double().abs()).all()
                k = o.storage_offset()
                keep[k:k + o.numel()] = False
            assert (dst[keep] == 5.0).all()


def test_overlaps_are_refused(P):
    import torch
    buf = torch.ones(100, device="cuda")
    other = torch.ones(100, device="cuda")
    norm, w = torch.zeros(1, device="cuda"), workspace(P, 4)
    for ins, outs in (([buf, buf], None), ([buf[:50], buf[49:]], None), ([buf[40:], buf[:41]], None),
                      ([buf[:50], other[:50]], [other[10:60], buf[50:]]),          # an out inside another's input
                      ([buf[:50], other[:50]], [buf[1:51], other[:50]]),           # and in its own, moved
                      ([buf[:50], buf[50:]], [other[:50], other[40:90]])):
        with pytest.raises(P.PpoError):
            P.ppo_clip_grad_norm(ins, 1.0, norm, outs, w)
    # the same input twice, to different places; and an out that is its own input
    P.ppo_clip_grad_norm([buf, buf], 1.0, norm, [other, torch.empty_like(buf)], w)
    assert abs(float(norm) - 200 ** 0.5) < 1e-5
    P.ppo_clip_grad_norm([buf[:50], buf[50:]], 1.0, norm, [buf[:50], buf[50:]], w)
    assert abs(float(buf.norm()) - 1) < 1e-5
    P.ppo_grad_norm([buf, buf], norm, w)
    assert abs(float(norm) - 2 ** 0.5) < 1e-5


def test_refusals(P):
    import torch
    ts, norm, w = tensors([10, 20], 1), torch.zeros(1, device="cuda"), workspace(P, 2)
    for bad in (dict(work=None), dict(work=w[:16]), dict(max_norm=float("nan")), dict(work=w[4:]),
                dict(out=[ts[0]]), dict(out=[ts[1], ts[0]])):
        with pytest.raises((P.PpoError, ValueError)):
            P.ppo_clip_grad_norm(**{**dict(tensors=ts, max_norm=1.0, norm=norm, work=w), **bad})
    for bad in ([ts[0].half()], [ts[0].cpu()], [torch.ones(6, 6, device="cuda").t()[:3]]):
        with pytest.raises(ValueError):
            P.ppo_grad_norm(bad, norm, w)
    with pytest.raises(ValueError):
        P.ppo_grad_norm(ts, norm.double(), w)


def test_streams_graphs_and_determinism(P):
    import torch
    ts = P.TensorList(tensors([300000, 7, 65536, 123], 9, ("f32", "bf16")))
    outs = P.TensorList([torch.zeros_like(t) for t in ts.tensors])
    norm, w = torch.zeros(1, device="cuda"), workspace(P, 4)
    P.ppo_clip_grad_norm(ts, 0.3, norm, outs, w)
    torch.cuda.synchronize()
    want = [norm.clone()] + [t.clone() for t in outs.tensors]
    side = torch.cuda.Stream()
    P.ppo_clip_grad_norm(ts, 0.3, norm, outs, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [norm, *outs.tensors]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.ppo_clip_grad_norm(ts, 0.3, norm, outs, w)
    for _ in range(2):
        norm.zero_()
        for t in outs.tensors:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [norm, *outs.tensors]))


def test_past_32_bits(P):
    import torch
    n = (1 << 32) + 12345
    if torch.cuda.mem_get_info()[0] < 3 * n * 2:
        pytest.skip("needs 26 GB")
    t = torch.full((n,), 2.0 ** -16, dtype=torch.bfloat16, device="cuda")
    norm = torch.zeros(1, device="cuda")
    want = 2.0 ** -16 * float(n) ** 0.5
    P.ppo_clip_grad_norm([t], want / 2, norm, work=workspace(P, 1))
    assert abs(float(norm) - want) <= NORM * want
    assert (t[-5:] == 2.0 ** -17).all() and (t[:5] == 2.0 ** -17).all()
    assert (t[1 << 32:] == 2.0 ** -17).all()
