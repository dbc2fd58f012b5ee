"""Clipping of calls larger than the last cache takes, in every pair of types, and of so many tensors that the sums are joined once, on the
GPU."""
import math

import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _rand(n, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (1e-3 * torch.randn(n, generator=g, device="cuda")).to(dtype)


def _norm(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tensors,values", [(2100, 24577), (2016, 16385)])
def test_many_tensors(dtype, tensors, values):
    """More than 4096 partial sums: 224 tensors of four (three) pieces each make 512 workgroups a launch."""
    mx = _mx()
    flat = _rand(tensors * (values + 3), dtype, tensors)
    sizes = [values + k % 3 for k in range(tensors)]
    at, grads = 1, []
    for n in sizes:
        grads.append(flat[at:at + n])
        at += n + 1
    before = flat.clone()
    old = [before[t.storage_offset():t.storage_offset() + t.numel()] for t in grads]
    n = _norm(old)
    announce("clip many", tensors, values, dtype)
    sum_sq, norm = mx.grad_norm(grads)
    assert abs(float(sum_sq) - n * n) <= n * n * 2.0 ** -40 and abs(float(norm) - n) <= n * U * 1.0001
    outs = [torch.empty_like(t) for t in grads]
    assert torch.equal(mx.grad_scale(grads, sum_sq, n / 3, out=outs), norm) and torch.equal(flat, before)
    assert torch.equal(mx.grad_clip(grads, n / 3), norm)
    for g, o, t in zip(grads, outs, old):
        assert torch.equal(g, o)
        exact = t.double() * ((n / 3) / (n + 1e-6))
        # max_norm and eps in FP32, the factor, the product and the last rounding
        assert bool(((g.double() - exact).abs() <= exact.abs() * (3.02 * U + (2.0 ** -8 if dtype == BF else 0.0)) + 2.0 ** -149).all())
    # nothing between them
    at = torch.ones(flat.shape, dtype=torch.bool, device="cuda")
    for t in grads:
        at[t.storage_offset():t.storage_offset() + t.numel()] = False
    assert int(at.sum()) > tensors and torch.equal(flat[at], before[at])


@pytest.mark.parametrize("dtype,out", [(F32, BF), (F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("clip", [False, True])
def test_more_than_the_last_cache_takes(dtype, out, clip):
    mx = _mx()
    n = 60_000_017
    size = {BF: 2, F32: 4}
    assert n * (size[dtype] + size[out]) > 192 << 20
    flat, to = _rand(n + 3, dtype, 7), torch.full((n + 3,), 7.0, dtype=out, device="cuda")
    # odd sizes and offsets, a small one between large ones
    edges = [1, 25_000_002, 25_000_003, 25_008_195, 50_000_000, n + 2]
    cut = lambda t: [t[a:b] for a, b in zip(edges, edges[1:])]  # noqa: E731
    grads, outs = cut(flat), cut(to)
    announce("clip large", n, dtype, out, clip)
    if clip:
        norm = _norm(grads)
        top = float(torch.tensor(norm / 3))
        got = mx.grad_clip(grads, top, eps=0.0, out=outs)
        c = torch.tensor(top / norm, dtype=torch.float64).float().cuda()
        # the kernel's norm may be off by some 2^-50, and the factor with it by its rounding
        factors = [c, torch.nextafter(c, c * 2), torch.nextafter(c, c * 0)]
    else:
        norm = 2.0
        got = mx.grad_scale(grads, torch.tensor(4.0, dtype=torch.float64, device="cuda"), 0.7, eps=0.0, out=outs)
        factors = [torch.tensor(0.7).cuda() * 0.5]
    assert abs(float(got) - norm) <= norm * U * 1.0001
    assert any(all(torch.equal(o, (g.float() * c).to(out)) for g, o in zip(grads, outs)) for c in factors)
    assert to[0] == 7.0 and bool((to[n + 2:] == 7.0).all())
