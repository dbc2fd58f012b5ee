"""The head's gradients at the ends of FP32's range, beside infinities in a row's gradient and in W, and of
confident rows with large logits."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_xent import _problem, _tol

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF, NAN = float("inf"), float("nan")


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


@pytest.mark.parametrize("bad", [dict(dloss=INF), dict(dloss=-INF), dict(dloss=NAN), dict(dlse=INF), dict(dlse=NAN),
                                 dict(dloss=INF, dlse=-INF), dict(dlse=3e38, dloss=3e38)])
@pytest.mark.parametrize("T,K,V", [(40, 64, 5000), (300, 96, 700)])
def test_an_infinite_row_gradient_leaves_the_other_rows(bad, T, K, V):
    """dX of the other rows is, bit for bit, what it is when the bad row has no gradient: the range that G is scaled to
    counts finite rows only. (Unscaled, G's entries of 1/8192 * 1e-4 would be nothing in FP16.)"""
    x, w, target, _, _ = _problem(T, K, V)
    dloss, dlse = torch.full((T,), 1.0 / 8192), torch.zeros(T)
    row = int((target != -100).nonzero()[T // 3, 0])
    dloss[row] = dlse[row] = 0.0
    announce("xent infinite row", bad, T, K, V)
    want, _ = _gradients(x, w, target, dloss, dlse)
    dloss[row], dlse[row] = bad.get("dloss", 0.0), bad.get("dlse", 0.0)
    dx, dw = _gradients(x, w, target, dloss, dlse)
    others = torch.arange(T) != row
    assert torch.equal(dx[others], want[others])
    assert not torch.isfinite(dx[row]).any() and not torch.isfinite(dw).any()


def test_the_largest_finite_row_gradients():
    """|dloss| + |dloss + dlse| beyond FP32's range where neither is: G is still scaled, and the result finite."""
    x, w, target, _, _ = _problem(20, 64, 300)
    target = target.clamp(min=0)
    top = 2.0 ** 127
    dloss, dlse = torch.full((20,), top), torch.zeros(20)
    x = (x.float() * 2.0 ** -40).to(BF)                   # every p is 1 / 300 to 2^-30
    announce("xent largest rows")
    dx, dw = _gradients(x, w, target, dloss, dlse)
    _, _, rdx, rdw, g, _ = ref.xent(x, w, target, -100, dloss, dlse)
    # G to half a step of FP16 and 2^-39 of the largest 2 top, p to 2^-20; FP32 sums of at most 300 terms
    off = (2.0 ** -11 + 2.0 ** -20) * g.abs() + 2.0 ** -38 * top
    assert bool(((dx.double() - rdx).abs() <= 1.01 * (off @ w.double().abs())).all())
    assert bool(((dw.double() - rdw).abs() <= 1.01 * (off.t() @ x.double().abs())).all())


@pytest.mark.parametrize("power", [-30, 0, 20, 40])
def test_a_mask_of_minus_infinity_in_w(power):
    """W[v][0] = -inf with X[t][0] = 1 masks word v out. The formula gives NaN in dX's column 0 (0 * inf) and the cut
    vocabulary's gradients everywhere else, at any magnitude of W's other entries: FP16 would take those below 2^-24 for
    nothing and those above 65504 for infinities, were they not scaled."""
    T, K, V, kept = 30, 64, 300, 100
    x, w, target, dloss, dlse = _problem(T, K, V, seed=power)
    target = torch.where(target >= 0, target % kept, target)
    x, w = (x.float() * 2.0 ** -power).to(BF), (w.float() * 2.0 ** power).to(BF)
    x[:, 0], w[:, 0] = 1.0, 0.0
    w[kept:, 0] = -INF
    announce("xent mask in w", power)
    dx, dw = _gradients(x, w, target, dloss, dlse)
    cut = w[:kept]
    rl, rlse, rdx, rdw, g, soft = ref.xent(x, cut, target, -100, dloss, dlse)
    t = _tol(K, float((x.double().norm(dim=1)[:, None] * cut.double().norm(dim=1)[None]).amax()))
    t += 2.0 ** -21 * (1.0 + float(rlse.abs().max()))
    g_top = float((dloss.abs() * 2 + dlse.abs()).max())
    off = 2.0 ** -11 * g.abs() + 2.5 * t * soft + 2.0 ** -39 * g_top
    half = 2.0 ** -24
    x_top, w_top = float(x.abs().max()), float(w[torch.isfinite(w)].abs().max())
    tol = (off @ cut.double().abs()) * 1.01 + g.abs().sum(1, True) * 2.0 ** -39 * w_top + half * rdx.abs()
    # the masked words' G is exactly 0, and 0 times their finite entries nothing
    assert torch.isnan(dx[:, 0]).all() and bool(((dx.double() - rdx).abs() <= tol)[:, 1:].all())
    tol = (off.t() @ x.double().abs()) * 1.01 + g.abs().sum(0)[:, None] * 2.0 ** -39 * x_top + half * rdw.abs()
    assert bool(((dw[:kept].double() - rdw).abs() <= tol).all()) and not dw[kept:].any()


@pytest.mark.parametrize("big", [0.0, 96.0, 128.0, 250.0, 1000.0, -40.0, -250.0])
def test_confident_rows_beside_large_logits(big):
    """Rows whose target leads by 28 or more, all logits shifted by `big`. One product of small integers a logit, all exact, so
    lse is the target's logit, rounded by less than (V - 1) exp(-gap) < 4.2e-10: G at the target, which is
    -(V - 1) exp(-gap) / (1 + ...) dloss, may be off by that much of dloss, and by nothing that grows with |lse|. Column
    1 + t of X is row t's alone, so dW[target(t)][1 + t] is G there."""
    T, K, V = 60, 64, 600
    x, w = torch.zeros(T, K), torch.zeros(V, K)
    rows = torch.arange(T)
    target = rows * 13 % V
    gap = 28.0 + rows % 30
    # big in two parts that bf16 holds exactly
    x[:, 0] = x[:, 61] = 1.0
    w[:, 0] = torch.tensor(big).to(BF).float()
    w[:, 61] = big - w[:, 0]
    x[rows, 1 + rows] = 1.0
    w[target, 1 + rows] = gap
    dloss = 0.5 + rows / 128.0
    announce("xent confident", big)
    _, dw = _gradients(x.to(BF), w.to(BF), target, dloss)
    at = dw[target, 1 + rows].double()
    rest = (V - 1) * torch.exp(-gap.double())
    want = -rest / (1.0 + rest) * dloss.double()
    assert bool(((at - want).abs() <= 1.01 * rest * dloss.double()).all())


def test_a_loss_of_more_tiles_than_a_grid():
    """2^21 - 1 tokens against 2^18 + 5 words: 2^23 tiles of 256 x 256, which the loss takes in two launches. Rows from all over
    the batch, their targets on both sides of the cut (column 261888), against the formula."""
    mx = _mx()
    T, K, V, cut = (1 << 21) - 1, 64, (1 << 18) + 5, 261888
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF)
    w = (torch.randn(V, K, generator=g, device="cuda") / 8).to(BF)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    rows = torch.cat([torch.arange(8), torch.tensor([255, 256, 1 << 20, T - 257, T - 2, T - 1]),
                      torch.randint(0, T, (50,), generator=torch.Generator().manual_seed(1))]).cuda()
    target[rows[::2]] = cut + torch.arange(rows[::2].numel(), device="cuda") % (V - cut)
    target[rows[1]], target[rows[3]], target[rows[5]] = cut - 1, 0, -100
    announce("xent of two launches")
    loss, lse = mx.linear_xent_forward(x, w, target)
    z = x[rows].double() @ w.double().t().contiguous()
    want = torch.logsumexp(z, dim=1)
    at = target[rows]
    wl = torch.where(at != -100, want - z[torch.arange(rows.numel(), device="cuda"), at.clamp(min=0)], 0.0)
    t = _tol(K, float(x[rows].double().norm(dim=1).max() * w.double().norm(dim=1).max())) + 2.0 ** -21 * (1.0 + float(want.abs().max()))
    assert float((lse[rows].double() - want).abs().max()) <= t and float((loss[rows].double() - wl).abs().max()) <= 2 * t
    assert bool(torch.isfinite(loss).all()) and bool((lse > 0).all())
