"""How far the Newton-Schulz update with FP16 operands may be from its steps in 64 bits: the smallest sides that take them, whose
roundings average least, and one or a few strong directions over weak noise, where what the shifted polynomial adds to the
noise's directions grows."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_orthogonalize import COEFFS, OWN, _grad, _rel

pytestmark = pytest.mark.gpu
A, B, C = COEFFS
SHIFT = -(B + C)                 # of the last step; the one before takes a half of it, the others none
SHIFTS = [0.0, 0.0, 0.0, SHIFT / 2, SHIFT]
HALF = 2.0 ** -11                # half a step of the products' FP16 operands


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def spread(g, draws=200):
    """The root mean square of the relative error that roundings of FP16 operands make in five steps: the steps in 64 bits with
    every operand (X twice, A, b A + c A A + t; X itself is kept in 22 bits) off by a random part of half a step, in so many
    draws. A symmetric matrix is rounded once for both of its places."""
    r = torch.Generator().manual_seed(7)
    want = ref.newton_schulz(g, 5, COEFFS, 1e-7)
    x = g.double() if g.shape[0] <= g.shape[1] else g.double().t()
    want = want if g.shape[0] <= g.shape[1] else want.t()
    x = (x / (x.norm() + 1e-7)).expand(draws, *x.shape)
    some = lambda v: v * (1.0 + HALF * (2.0 * torch.rand(v.shape, generator=r, dtype=torch.float64) - 1.0))  # noqa: E731

    def both(v):
        v = some(v).tril()
        return v + v.tril(-1).transpose(1, 2)
    for t in SHIFTS:
        y = some(x)
        gram = both(y @ y.transpose(1, 2).contiguous())
        p = both(B * gram + C * (gram @ gram) + t * torch.eye(x.shape[1], dtype=torch.float64))
        x = (A - t) * x + p @ y
    return float(((x - want).square().sum((1, 2)).mean() / want.square().sum()).sqrt())


# One direction of singular value s near 1 over directions that are next to nothing: rounding X beside the shift t scatters
# t 2^-12 |X| (root mean square) over all of those, and they grow by a = 3.44 in each step that follows. The strong value
# goes 1 -> 0.70 -> 1.11 -> 0.72 -> 1.09 -> 0.70, so relative to the result the last two steps' roundings are 1.03 and 1.57 of
# 2^-12; they are independent, of each other and of the others (OWN).
STRONG = (OWN ** 2 + (SHIFT * 2.0 ** -12) ** 2 * ((1.03 * A / 2) ** 2 + 1.57 ** 2)) ** 0.5


@pytest.mark.parametrize("m,n", [(65, 65), (65, 1000), (300, 70), (90, 128), (128, 700)])
@pytest.mark.parametrize("kind", ["normal", "heavy", "strong"])
def test_smallest_sides(m, n, kind):
    """Within three times the root mean square: the roundings of a few numbers are bounded (the largest is 3 ** 0.5 times the
    root mean square of its range), and independent."""
    mx = _mx()
    announce("orthogonalize smallest sides", m, n, kind)
    for seed in range(3):
        g = _grad(m, n, kind, 1000 * seed)
        got = mx.orthogonalize(g.cuda(), out_dtype=torch.float32)
        assert _rel(got, ref.newton_schulz(g, 5, COEFFS, 1e-7)) <= 3.0 * spread(g, 20), seed


@pytest.mark.parametrize("m,n", [(65, 300), (300, 96), (128, 128), (256, 512), (500, 900), (1000, 1500)])
@pytest.mark.parametrize("noise", [1e-1, 1e-2, 1e-3, 1e-4, 1e-5, 0.0])
@pytest.mark.parametrize("few", [False, True])
def test_strong_directions_over_noise(m, n, noise, few):
    g = torch.Generator().manual_seed(m + n)
    r = max(1, min(m, n) // 16) if few else 1
    x = torch.randn(m, r, generator=g) @ torch.randn(r, n, generator=g) + noise * torch.randn(m, n, generator=g)
    announce("orthogonalize strong over noise", m, n, noise, few)
    want = ref.newton_schulz(x, 5, COEFFS, 1e-7)
    assert _rel(_mx().orthogonalize(x.cuda(), out_dtype=torch.float32), want) <= STRONG
