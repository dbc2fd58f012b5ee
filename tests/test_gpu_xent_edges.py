"""The head's gradients at the ends of FP32's range."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_xent import _problem, _tol

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _gradients(x, w, target, dloss, dlse=None):
    mx = _mx()
    X, W, Tg = x.cuda(), w.cuda(), target.cuda()
    lse = mx.linear_xent_forward(X, W, Tg)[1]
    dx, dw = mx.linear_xent_backward(dloss.cuda(), X, W, Tg, lse, dlse=None if dlse is None else dlse.cuda(),
                                     dx_dtype=torch.float32, dw_dtype=torch.float32)
    return dx.cpu(), dw.cpu()


@pytest.mark.parametrize("power", [126, 100, -100, -126])
@pytest.mark.parametrize("ex,ew", [(0, 0), (-20, 8), (60, -60)])
def test_row_gradients_at_the_ends_of_fp32(power, ex, ew):
    """Gradients that are finite (or normal) numbers come out, whatever the scales of G, X and W make of each other on
    the way."""
    T, K, V = 20, 64, 300
    x, w, target, _, _ = _problem(T, K, V)
    x, w, target = (x.float() * 2.0 ** ex).to(BF), (w.float() * 2.0 ** ew).to(BF), target.clamp(min=0)
    dloss = torch.full((T,), 2.0 ** power)
    announce("xent ends of fp32", power, ex, ew)
    dx, dw = _gradients(x, w, target, dloss)
    _, rlse, rdx, rdw, g, soft = ref.xent(x, w, target, -100, dloss, None)
    t = _tol(K, float((x.double().norm(dim=1)[:, None] * w.double().norm(dim=1)[None]).amax()))
    t += 2.0 ** -21 * (1.0 + float(rlse.abs().max()))
    # as in test_gpu_xent: G's half step and its exponent, 2^-39 of the largest of G, X and W, and FP32's rounding; then what
    # lies below FP32's normal numbers
    off = 2.0 ** -11 * g.abs() + 2.5 * t * soft + 2.0 ** -38 * 2.0 ** power
    half, tiny = 2.0 ** -24, 2.0 ** -126
    for got, want, tol in ((dx, rdx, 1.01 * (off @ w.double().abs()) + g.abs().sum(1, True) * 2.0 ** -39 * float(w.abs().max())),
                           (dw, rdw, 1.01 * (off.t() @ x.double().abs()) + g.abs().sum(0)[:, None] * 2.0 ** -39 * float(x.abs().max()))):
        held = want.abs() < 2.0 ** 127
        assert bool(((got.double() - want).abs() <= tol + half * want.abs() + tiny)[held].all())
