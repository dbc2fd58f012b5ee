"""The Newton-Schulz update of matrices with a side of at most 64, which works in FP32 throughout, and on both sides of that border
what the two ways have in common."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_orthogonalize import COEFFS, _grad, _rel
from tests.test_gpu_orthogonalize_accuracy import spread

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _bound(g):
    """Three times the root mean square of two kinds of errors, added as squares.
    A and what is formed of it: what FP16 operands would give (spread), with roundings 2^13 times finer; a sum of up to l terms is
    rounded as often, independently: sqrt(l) of them; and those of an entry of A are relative to its row's and column's norms,
    not to itself: with s entries a row, sqrt(s).
    X itself, which is held in FP32 (with FP16 operands in 22 bits, where this is next to nothing): the start is rounded by 2^-24
    of its norm, and each step's sums of s terms by 2^-24 sqrt(s) of theirs, at most a |X|. Such an error lies in every
    direction, and where the values are small it grows by a in each step that follows: k steps before the end, a^k |X|. (One
    direction over noise: 3 x 5, 2^-24 3^0.5 a^5 / 0.7 = 7e-5; the first term alone is 1.5e-6.)"""
    few, many = min(g.shape), max(g.shape)
    formed = spread(g, 40 if few * many > 20000 else 200) * 2.0 ** -13 * (many * few) ** 0.5
    norms = [float(ref.newton_schulz(g, k, COEFFS, 1e-7).norm()) for k in range(6)]
    held = 2.0 ** -24 * few ** 0.5 * sum((COEFFS[0] ** (5 - k) * norms[k] / norms[5]) ** 2 for k in range(5)) ** 0.5
    return 3.0 * (formed ** 2 + held ** 2) ** 0.5


@pytest.mark.parametrize("m,n", [(1, 1), (1, 3), (2, 2), (3, 5), (7, 9), (16, 16), (19, 130), (20, 642), (33, 512), (33, 513), (64, 64), (64, 65),
                                 (64, 1000), (1, 20000), (18, 2048), (40, 17000)])
@pytest.mark.parametrize("kind", ["normal", "heavy", "strong", "one"])
def test_fp32_throughout(m, n, kind):
    """Wide and tall, from FP32 and bf16, to FP32 and bf16."""
    mx = _mx()
    g = _grad(m, n, kind, 5)
    if kind == "one":                              # one direction over noise of 1e-4
        r = torch.Generator().manual_seed(m + n)
        g = torch.randn(m, 1, generator=r) @ torch.randn(1, n, generator=r) + 1e-4 * torch.randn(m, n, generator=r)
    announce("orthogonalize thin", m, n, kind)
    for x in (g, g.to(BF), g.t().contiguous()):
        want = ref.newton_schulz(x, 5, COEFFS, 1e-7)
        got = mx.orthogonalize(x.cuda(), out_dtype=torch.float32)
        assert _rel(got, want) <= _bound(x.float())
        assert torch.equal(mx.orthogonalize(x.cuda()), got.to(BF))


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 7])
@pytest.mark.parametrize("m,n", [(5, 40), (300, 30), (60, 700)])
def test_steps_and_coefficients(steps, m, n):
    mx = _mx()
    for coeffs in (COEFFS, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (0.5, 0.0, 0.0)):
        g = _grad(m, n, "normal", steps)
        got = mx.orthogonalize(g.cuda(), steps=steps, coefficients=coeffs, out_dtype=torch.float32)
        assert _rel(got, ref.newton_schulz(g, steps, coeffs, 1e-7)) <= 2.0 ** -24 * 40 * (m * n) ** 0.5


@pytest.mark.parametrize("m,n", [(50, 700), (700, 50), (64, 64), (65, 200)])
def test_batches_strides_and_a_weight(m, n):
    """Each matrix of a batch as it is alone, bit for bit; onto a strided weight, whose other elements stay."""
    mx = _mx()
    big = torch.stack([_grad(m + 3, n + 5, k, 9) for k in ("normal", "heavy", "strong", "normal", "heavy")]).cuda()
    g = big[::2, 1:m + 1, 2:n + 2]
    announce("orthogonalize thin batch", m, n)
    got = mx.orthogonalize(g, out_dtype=torch.float32)
    for k in range(3):
        assert torch.equal(mx.orthogonalize(g[k], out_dtype=torch.float32), got[k])
        assert torch.equal(mx.orthogonalize(g[k].contiguous(), out_dtype=torch.float32), got[k])
    for dtype in (torch.float32, BF):
        w = torch.randn(3, m + 1, n + 3, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        old = w.clone()
        mx.orthogonalize(g, alpha=-0.02, beta=0.5, out=w[:, :m, :n])
        want = -0.02 * got.double() + 0.5 * old[:, :m, :n].double()
        # three roundings to FP32, each of at most the terms' size, and the result's
        tol = 2.0 ** -22 * (0.5 * old[:, :m, :n].double().abs() + 0.02 * got.double().abs())
        if dtype == BF:
            tol = tol + 2.0 ** -8 * want.abs()
        assert bool(((w[:, :m, :n].double() - want).abs() <= tol).all())
        assert torch.equal(w[:, m:], old[:, m:]) and torch.equal(w[:, :, n:], old[:, :, n:])


@pytest.mark.parametrize("m,n", [(1, 1), (40, 5000), (9, 30), (70, 90), (300, 200)])
def test_zeros_scales_and_nan(m, n):
    mx = _mx()
    announce("orthogonalize zeros, scales, NaN", m, n)
    assert not mx.orthogonalize(torch.zeros(m, n, device="cuda")).any()
    assert torch.isnan(mx.orthogonalize(torch.zeros(m, n, device="cuda"), eps=0.0)).all()
    g = _grad(m, n, "normal").clamp(-3, 3)
    g[g.abs() < 2.0 ** -10] = 0.25
    want = mx.orthogonalize(g.cuda(), eps=0.0)
    assert bool(torch.isfinite(want).all())
    for k in (-115, -60, 60, 126):
        assert torch.equal(mx.orthogonalize(torch.ldexp(g, torch.tensor(k)).cuda(), eps=0.0), want)
    for bad in (float("nan"), float("inf"), -float("inf")):
        two = torch.stack([g, g, g]).cuda()
        two[1, m // 2, n // 3] = bad
        got = mx.orthogonalize(two, eps=0.0)
        assert torch.equal(got[0], want) and torch.equal(got[2], want) and torch.isnan(got[1]).all()


def test_two_at_once_and_replayed():
    mx = _mx()
    a, b = _grad(30, 9000, "heavy").cuda(), _grad(5000, 64, "strong").cuda()
    wa, wb = mx.orthogonalize(a), mx.orthogonalize(b)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        ga, gb = mx.orthogonalize(a, stream=sides[0]), mx.orthogonalize(b, stream=sides[1])
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    held = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.orthogonalize(held)
    for k in range(4):
        held.copy_(_grad(30, 9000, "normal", k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.orthogonalize(held))
