"""The Newton-Schulz update on the GPU, against its steps in 64 bits."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu
COEFFS = (3.4445, -4.7750, 2.0315)
# The products' operands carry 11 bits (half a step: 2^-11 relative at most, 2^-12 in the root mean square),
# X 22. A step adds to X the errors of three operand roundings (X twice, in A and in the update, b A + c A A
# once), each weighted by |b x + c x x| <= 2.9 at squared singular values x; what small singular values
# pick up is relative to b A X, so to them, and grows with them; near 1 the step's slope is between -1.2
# and 1, so that errors do not grow there. Over five steps independent errors add up as squares:
# sqrt(15) * 2.9 * 2^-12 = 0.0027. A matrix of a few singular values averages nothing: then each of the
# five steps' errors may be 3 * 2.9 * 2^-11 and grow by 1.2 in each step after it.
OWN = 15 ** 0.5 * 2.9 * 2.0 ** -12
FEW = 3 * 2.9 * 2.0 ** -11 * sum(1.2 ** k for k in range(5))
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _grad(m, n, kind, seed=0):
    g = torch.Generator().manual_seed(seed + m * 31 + n)
    if kind == "normal":
        return torch.randn(m, n, generator=g)
    if kind == "heavy":
        return torch.randn(m, n, generator=g) / (torch.randn(3, m, n, generator=g).square().sum(0) / 3).sqrt() * 1e-3
    r = max(1, min(m, n) // 16)                    # a few strong directions over weak noise
    return torch.randn(m, r, generator=g) @ torch.randn(r, n, generator=g) + 0.1 * torch.randn(m, n, generator=g)


def _rel(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("m,n", [(1, 1), (1, 300), (300, 1), (16, 16), (19, 130), (128, 128), (129, 257), (500, 300), (256, 1100),
                                 (1500, 64)])
@pytest.mark.parametrize("kind", ["normal", "heavy", "strong"])
def test_against_the_steps(m, n, kind):
    mx = _mx()
    g = _grad(m, n, kind)
    want = ref.newton_schulz(g, 5, COEFFS, 1e-7)
    announce("orthogonalize", m, n, kind)
    got = mx.orthogonalize(g.cuda(), out_dtype=torch.float32)
    own = OWN if min(m, n) >= 16 else FEW
    assert _rel(got, want) <= own
    low = mx.orthogonalize(g.cuda())
    assert low.dtype == torch.bfloat16 and torch.equal(low, got.to(torch.bfloat16))
    gb = g.to(torch.bfloat16)
    assert _rel(mx.orthogonalize(gb.cuda()), ref.newton_schulz(gb, 5, COEFFS, 1e-7)) <= own + BF16


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 7])
def test_steps_and_coefficients(steps):
    mx = _mx()
    for coeffs in (COEFFS, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)):
        g = _grad(70, 200, "normal", steps)
        got = mx.orthogonalize(g.cuda(), steps=steps, coefficients=coeffs, out_dtype=torch.float32)
        want = ref.newton_schulz(g, steps, coeffs, 1e-7)
        assert _rel(got, want) <= max(OWN * max(1.0, (steps / 5) ** 0.5), 2.0 ** -21)


def test_batches_and_strides():
    mx = _mx()
    for m, n in ((60, 200), (300, 140)):
        big = torch.stack([_grad(m + 3, n + 5, k, 9) for k in ("normal", "heavy", "strong", "normal", "heavy")]).cuda()
        g = big[::2, 1:m + 1, 2:n + 2]
        announce("orthogonalize batch", m, n)
        got = mx.orthogonalize(g)
        for k in range(3):
            one = mx.orthogonalize(g[k])
            assert torch.equal(one, got[k])
            assert _rel(one, ref.newton_schulz(g[k].cpu(), 5, COEFFS, 1e-7)) <= OWN + BF16
        # onto a strided output: alpha and beta
        for dtype in (torch.float32, torch.bfloat16):
            w = torch.randn(3, m + 1, n + 3, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
            old = w.clone()
            mx.orthogonalize(g, alpha=-0.02, beta=0.5, out=w[:, :m, :n])
            x = mx.orthogonalize(g, out_dtype=torch.float32).double()
            want = (-0.02 * x + 0.5 * old[:, :m, :n].double())
            tol = 2.0 ** -22 * (want.abs() + 0.5 * old[:, :m, :n].double().abs() + 0.02 * x.abs())
            if dtype == torch.bfloat16:
                tol = tol + BF16 * want.abs()
            assert bool(((w[:, :m, :n].double() - want).abs() <= tol).all())
            assert torch.equal(w[:, m:], old[:, m:]) and torch.equal(w[:, :, n:], old[:, :, n:])


def test_zeros_scales_and_nan():
    mx = _mx()
    assert not mx.orthogonalize(torch.zeros(40, 50, device="cuda")).any()
    g = _grad(40, 50, "normal")
    want = mx.orthogonalize(g.cuda())
    # the scale of the gradient does not matter (powers of two: bit for bit), far outside FP32's squares too
    for k in (-60, 60):
        assert torch.equal(mx.orthogonalize((g * 2.0 ** k).cuda(), eps=0.0), mx.orthogonalize(g.cuda(), eps=0.0))
    assert mx.orthogonalize(torch.zeros(0, 5, device="cuda")).shape == (0, 5)
    two = torch.stack([g, g]).cuda()
    two[1, 3, 4] = float("nan")
    got = mx.orthogonalize(two)
    assert torch.equal(got[0], want) and torch.isnan(got[1]).all()
    one = torch.zeros(30, 40, device="cuda")        # a single entry: one singular value, 1
    one[7, 9] = 5.0
    assert _rel(mx.orthogonalize(one, out_dtype=torch.float32), ref.newton_schulz(one.cpu(), 5, COEFFS, 1e-7)) <= FEW


def test_large_tiles():
    """A shape with enough tiles for the 256 x 256 kernel, ragged on both sides, wide and tall."""
    mx = _mx()
    g = _grad(2900, 3001, "heavy").cuda()
    x = g.double() / (g.double().norm() + 1e-7)
    a, b, c = COEFFS
    for _ in range(5):
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    announce("orthogonalize large")
    assert _rel(mx.orthogonalize(g), x.cpu()) <= OWN + BF16
    assert _rel(mx.orthogonalize(g.t().contiguous()), x.t().cpu()) <= OWN + BF16


def test_other_stream_and_graph():
    mx = _mx()
    g = _grad(200, 300, "strong").cuda()
    want = mx.orthogonalize(g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mx.orthogonalize(g, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.orthogonalize(g)
    for k in range(3):
        g.copy_(_grad(200, 300, "heavy", k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.orthogonalize(g))
