"""Clipping by factors below FP32's normal range, on the GPU, against 64 bits."""
import math

import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, U, assert_within, heavy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


# factors of 2^-125, on both sides of 2^-126, below FP32's smallest subnormal number 2^-149, and far below it
@pytest.mark.parametrize("exponent", [-125, -126.5, -128.3, -140.4, -150.5, -170.2])
def test_tiny_factors(exponent):
    mx = _mx()
    grads = [heavy((9001,), 1).clamp(-100, 100) * 2.0 ** 121, heavy((777,), 2).clamp(-100, 100).to(BF) * 2.0 ** 121, torch.full((5,), 3.0e38),
             torch.tensor([0.0, -0.0, 1.0, -2.0 ** -149, 2.0 ** 100])]
    assert all(bool(torch.isfinite(g).all()) for g in grads)
    n = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    top = float(torch.tensor(n * 2.0 ** exponent))               # as FP32 holds it
    announce("clip range", exponent, top)
    c = top / n
    for out_dtype in (None, F32, BF):
        work = [g.cuda() for g in grads]
        outs = None if out_dtype is None else [torch.full(g.shape, 7.0, dtype=out_dtype).cuda() for g in grads]
        norm = mx.grad_clip(work, top, eps=0.0, out=outs)
        # a norm beyond FP32 is infinite as a result, but counts as it is
        assert float(norm) == math.inf if n > 3.41e38 else abs(float(norm) - n) <= n * U * 1.0001
        for g, o in zip(grads, outs or work):
            exact = g.double() * c
            # the factor, the product, the last rounding; half a step each of the product's and of bf16's subnormal numbers
            assert_within(o, exact, exact.abs() * (2.01 * U + (2.0 ** -8 if o.dtype == BF else 0.0)) + 2.0 ** -150
                          + (2.0 ** -134 if o.dtype == BF else 2.0 ** -150))


def test_nothing_is_left_of_finite_values_under_an_infinite_norm():
    mx = _mx()
    g = torch.tensor([3.0e38, -math.inf, 1.0]).cuda()
    assert float(mx.grad_clip(g, 2.0 ** -149, eps=0.0)) == math.inf
    assert g.cpu().tolist()[0] == 0.0 and math.isnan(float(g[1])) and float(g[2]) == 0.0


def test_a_factor_that_rounds_to_a_power_of_two():
    """(1 - 2^-30) 2^-130 rounds to 2^-130: values in place are still scaled."""
    mx = _mx()
    g = torch.full((4,), 2.0 ** 126)
    sum_sq = torch.tensor(2.0 ** -20 / (1 - 2.0 ** -30), dtype=torch.float64).square() * 2.0 ** 260
    got = g.cuda()
    mx.grad_scale([got], sum_sq.cuda(), 2.0 ** -20, eps=0.0)
    assert bool((got == 2.0 ** -4).all())
