"""The gated activation's accuracy in FP32, over gates of every size: the header's bounds, which do not grow with the gate."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import F32, U, assert_within, gate_backward, gate_forward

pytestmark = pytest.mark.gpu

# In units of U = 2^-24, relative. The exponential: 2 of the hardware's (one last place), one for the sum that corrects its argument, and
# less than 0.1 for the square of that correction (below 2^-17): e 3.1. s = 1 / (1 + e): e's, half for 1 - s in the remainder of
# the Newton step, one for its last sum: 4.6. 1 - s = e s: e's error counts 1 / (1 + e) times, then half, one and one: 5.6.
# a = (g s) u and dup = da (g s): 4.6 and two products. dgate = da (u (s + (g s) (1 - s))): s 4.6 of s, (g s) (1 - s) 4.6 + 1 + 5.6 of itself, the sum one
# and the products two of both: 14.2 of |da u s| (1 + |g (1 - s)|).
A = 6.6 * U * 1.01
DGATE = 14.2 * U * 1.01


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


# s and 1 - s are above 2^-126 up to 87, and the products with these up and da in FP32's normal range
@pytest.mark.parametrize("low,high", [(-87.0, 87.0), (-20.0, 20.0), (-3.0, 3.0)])
def test_over_the_gates(low, high):
    mx = _mx()
    g = torch.Generator().manual_seed(int(high))
    gate = torch.linspace(low, high, 512 * 1000).reshape(512, 1000)
    up, da = (torch.where(torch.rand(gate.shape, generator=g) < 0.5, -1.0, 1.0) * (0.5 + torch.rand(gate.shape, generator=g)) for _ in range(2))
    announce("gate accuracy", low, high)
    exact = gate_forward(gate, up)
    assert_within(mx.swiglu_forward(gate.cuda(), up.cuda(), out_dtype=F32).a, exact, A * exact.abs(), "a")
    dg, du, basis = gate_backward(da, gate, up)
    o = mx.swiglu_backward(da.cuda(), gate.cuda(), up.cuda(), out_dtype=F32)
    assert_within(o.dgate, dg, DGATE * basis, "dgate")
    assert_within(o.dup, du, A * du.abs(), "dup")
