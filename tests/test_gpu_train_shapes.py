"""The training operators at shapes that take each way of working a product: tiles of three sizes, whole, split over the
contraction, and both in one launch."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.test_gpu_orthogonalize import BF16, COEFFS, OWN
from tests.test_gpu_xent import _check, _problem

pytestmark = pytest.mark.gpu
# rows, columns, contraction in stages of 128 bytes
SHAPES = [(16, 16, 1), (16, 16, 32), (1300, 1537, 1), (512, 4200, 40), (1537, 5000, 72), (1537, 5000, 1), (700, 4096, 152),
          (4096, 4200, 16)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


@pytest.mark.parametrize("M,N,stages", SHAPES)
def test_fp8_products_of_small_integers(M, N, stages):
    """Codes of 0, +-1, +-2 and scales of 1, 2 or 1/2: products are at most 16, and sums multiples of 1/4 below 2^19
    that FP32 holds exactly in any order; the 13 bits that a group of eight keeps do as well."""
    K = 128 * stages
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    codes = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device="cuda")
    values = torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0], dtype=torch.float64, device="cuda")

    def operand(outer):
        at = torch.randint(0, 5, (outer, K), generator=g, device="cuda")
        e = torch.randint(-1, 2, (outer, stages), generator=g, device="cuda")
        scales = torch.zeros(outer, (stages + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
        scales[:, :stages] = (127 + e).to(torch.uint8)
        factor = torch.where(e == 0, 1.0, torch.where(e > 0, 2.0, 0.5)).double()
        return codes[at], scales, values[at] * factor.repeat_interleave(128, dim=1)

    aq, as_, A = operand(M)
    bq, bs, B = operand(N)
    announce("fp8 gemm", M, N, K)
    want = A @ B.t().contiguous()
    assert torch.equal(_mx().fp8_gemm(aq, as_, bq, bs).double(), want)
    # on what is there, rounded once
    out = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    _mx().fp8_gemm(aq, as_, bq, bs, alpha=0.5, beta=3.0, out=out)
    assert torch.equal(out, (0.5 * want + 3.0).to(torch.bfloat16))


@pytest.mark.parametrize("T,V,stages", SHAPES)
def test_head(T, V, stages):
    announce("xent", T, 64 * stages, V)
    _check(*_problem(T, 64 * stages, V))


@pytest.mark.parametrize("batch,m,n", [(3, 16, 2048), (1, 2000, 3584), (1, 4608, 4096), (1, 4200, 6656), (1, 8192, 8192),
                                       (5, 700, 1100)])
def test_orthogonalize(batch, m, n):
    g = torch.randn(batch, m, n, generator=torch.Generator(device="cuda").manual_seed(m + n), device="cuda").to(torch.bfloat16)
    announce("orthogonalize", batch, m, n)
    got = _mx().orthogonalize(g)
    a, b, c = COEFFS
    for k in range(batch):
        x = g[k].double()
        x = x / (x.norm() + 1e-7)
        x = x.t().contiguous() if m > n else x
        for _ in range(5):
            A = x @ x.t().contiguous()
            x = a * x + (b * A + c * (A @ A)) @ x
        x = x.t() if m > n else x
        assert float((got[k].double() - x).norm() / x.norm()) <= OWN + BF16


def test_orthogonalize_at_the_ends_of_fp32():
    """Entries near FP32's largest and its smallest normal numbers: powers of two do not change the result."""
    g = torch.randn(40, 50, generator=torch.Generator().manual_seed(1)).clamp(-3, 3).cuda()
    g[g.abs() < 2.0 ** -10] = 0.25
    want = _mx().orthogonalize(g, eps=0.0)
    assert bool(torch.isfinite(want).all())
    # 24 bits below 2^-10 are still above the smallest subnormal, 2^-149; 3 * 2^126 is below the largest
    for k in (-115, 100, 126):
        announce("orthogonalize, scale 2^", k)
        assert torch.equal(_mx().orthogonalize(torch.ldexp(g.cpu(), torch.tensor(k)).cuda(), eps=0.0), want)


def test_small_losses_beside_large_logits():
    """A row whose target is far ahead: its loss is log(1 + (V - 1) exp(z - z_target)), however large the logits are that
    cancel in it. One product a logit, all exact: the loss is off by its own operations' roundings (an exponent of
    some 12, an exponential of 2^-22, a sum of 1 and little, a logarithm) alone, 2^-19 at most, where lse's rounding is 2^-17."""
    V, K = 600, 64
    x, w = torch.zeros(40, K), torch.zeros(V, K)
    target = torch.arange(40) * 13 % V
    gap = torch.arange(40) * 0.25 + 6.0
    big = 128.0
    x[:, 0], w[:, 0] = 1.0, big                      # z = 128 everywhere
    for t in range(40):                              # and 128 + gap at the target
        x[t, 1 + t % 60] = 1.0
    x[:, 0] = 1.0
    for t in range(40):
        w[target[t], 1 + t % 60] = gap[t]
    loss, lse = _mx().linear_xent_forward(x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda(), target.cuda())
    want = torch.log1p((V - 1) * torch.exp(-gap.double()))
    # 1 + s is added up in FP32, in an order of the kernel's: each addition to what holds the 1 already may be off by
    # 2^-24, and there are at most 16 in a lane, 2 across lanes, 3 across wavefronts, 10 across tiles: below 32 * 2^-24;
    # s is held to 16 * 2^-23 of itself, the logarithm to 2^-22 and its own 2^-23
    tol = 2.0 ** -22 + 2.0 ** -19 + want * 2.0 ** -18
    assert bool(((loss.cpu().double() - want).abs() <= tol).all())
    assert bool(((lse.cpu().double() - (big + gap.double() + want)).abs() <= tol + 2.0 ** -16).all())
