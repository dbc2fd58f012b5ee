"""Softmax cross entropy of a linear head on the GPU, against its formulas in 64 bits."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _problem(T, K, V, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + T + K + V)
    w = (torch.randn(V, K, generator=g) * scale / K ** 0.5).to(BF)
    target = torch.randint(0, V, (T,), generator=g)
    x = (torch.randn(T, K, generator=g) + 3.0 * torch.rand(T, 1, generator=g) * w[target].float() * K ** 0.5 / scale).to(BF)
    target[torch.rand(T, generator=g) < 0.15] = -100
    dloss = torch.rand(T, generator=g) / max(T, 1)
    dlse = 0.1 * torch.randn(T, generator=g) / max(T, 1)
    return x, w, target, dloss, dlse


def _tol(K, zmax):
    """Error of a logit: K products of bf16 numbers (exact in FP32) added up in FP32, and the exponent's base-2
    argument z log2(e), rounded once. All of |z| <= zmax; the sum of the |terms| of a logit is at most
    |x| |w|, taken as zmax by the caller."""
    return (K / 16 + 16) * 2.0 ** -23 * zmax


def _check(x, w, target, dloss, dlse, dtype=BF, **kw):
    mx = _mx()
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    X, W, Tg = x.cuda(), w.cuda(), target.cuda()
    loss, lse = mx.linear_xent_forward(X, W, Tg)
    rl, rlse, rdx, rdw, g, soft = ref.xent(x, w, target, -100, dloss, dlse)
    basis = (x.double().norm(dim=1)[:, None] * w.double().norm(dim=1)[None]).amax() if x.numel() else torch.tensor(1.0)
    t = _tol(x.shape[1], float(basis)) + 2.0 ** -21 * (1.0 + float(rlse.abs().max()))
    assert float((lse.cpu().double() - rlse).abs().max()) <= t
    assert float((loss.cpu().double() - rl).abs().max()) <= 2 * t
    assert (loss.cpu()[target == -100] == 0).all()
    dx, dw = mx.linear_xent_backward(dev(dloss), X, W, Tg, lse, dlse=dev(dlse), dx_dtype=dtype, dw_dtype=dtype, **kw)
    # each G is off by half a step of FP16; its first part, p (dloss + dlse), by 2 t relative before that
    # (the exponent z - lse is off by t + t), which the subtraction of dloss at the target leaves as it
    # is however small the difference (p -> 1); what lies 2^-28 below the largest of G, X or W is off by
    # 2^-39 of that; then the products' FP32 sums and the output's rounding
    dl = torch.zeros(1) if dloss is None else dloss.abs()
    dp = (dl if dlse is None else dl + dlse.abs())
    g_top, x_top, w_top = float((dl + dp).max()), float(x.abs().max()), float(w.abs().max())
    off = 2.0 ** -11 * g.abs() + 2.5 * t * soft + 2.0 ** -39 * g_top
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -126
    if dx is not None:
        tol = (off @ w.double().abs()) * 1.01 + g.abs().sum(1, True) * 2.0 ** -39 * w_top + half * rdx.abs() + tiny
        assert dx.dtype == dtype and bool(((dx.cpu().double() - rdx).abs() <= tol).all())
    if dw is not None:
        tol = (off.t() @ x.double().abs()) * 1.01 + g.abs().sum(0)[:, None] * 2.0 ** -39 * x_top + half * rdw.abs() + tiny
        assert dw.dtype == dtype and bool(((dw.cpu().double() - rdw).abs() <= tol).all())
    return loss, lse, dx, dw


@pytest.mark.parametrize("T,K,V", [(1, 32, 1), (1, 64, 2), (1, 512, 5000), (3, 33, 129), (31, 1, 7), (128, 512, 1000), (257, 96, 2051),
                                   (130, 1000, 515), (600, 64, 9000)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_against_the_formulas(T, K, V, dtype):
    announce("xent", T, K, V, dtype)
    _check(*_problem(T, K, V), dtype=dtype)


def test_many_pieces_of_the_vocabulary():
    """Enough tokens that the gradients are formed in several pieces, the last one ragged."""
    x, w, target, dloss, dlse = _problem(9000, 32, 31111)
    announce("xent pieces")
    mx = _mx()
    loss, lse = mx.linear_xent_forward(x.cuda(), w.cuda(), target.cuda())
    dx, dw = mx.linear_xent_backward(dloss.cuda(), x.cuda(), w.cuda(), target.cuda(), lse, dlse=dlse.cuda())
    rl, rlse, rdx, rdw, _, _ = ref.xent(x, w, target, -100, dloss, dlse)
    assert float((loss.cpu().double() - rl).abs().max()) < 1e-4 and float((lse.cpu().double() - rlse).abs().max()) < 1e-4
    # one rounding to bf16 and one, of G, to FP16
    assert float((dx.cpu().double() - rdx).norm() / rdx.norm()) < 2.0 ** -8 + 2.0 ** -11
    assert float((dw.cpu().double() - rdw).norm() / rdw.norm()) < 2.0 ** -8 + 2.0 ** -11


def test_gradients_alone_and_absent_row_gradients():
    x, w, target, dloss, dlse = _problem(77, 64, 400)
    full = _check(x, w, target, dloss, dlse)
    only_x = _check(x, w, target, dloss, dlse, need_dw=False)
    only_w = _check(x, w, target, dloss, dlse, need_dx=False)
    assert only_x[3] is None and torch.equal(only_x[2], full[2])
    assert only_w[2] is None and torch.equal(only_w[3], full[3])
    _check(x, w, target, dloss, None)
    _check(x, w, target, None, dlse)
    _, _, dx, dw = _check(x, w, target, None, None)
    assert not dx.any() and not dw.any()
    _check(x, w, target, dloss, -dloss)          # the probabilities' weight vanishes, the target's does not


def test_every_target_ignored():
    x, w, target, dloss, _ = _problem(50, 64, 300)
    target[:] = -100
    loss, lse, dx, dw = _check(x, w, target, dloss, None)
    assert not loss.any() and not dx.any() and not dw.any()


def test_nan_in_ignored_rows_and_bad_targets():
    mx = _mx()
    x, w, target, dloss, _ = _problem(40, 64, 300)
    keep = target != -100
    clean = mx.linear_xent_forward(x.cuda(), w.cuda(), target.cuda())
    g0 = mx.linear_xent_backward(dloss.cuda(), x.cuda(), w.cuda(), target.cuda(), clean[1])
    bad = x.clone()
    bad[~keep] = float("nan")
    loss, lse = mx.linear_xent_forward(bad.cuda(), w.cuda(), target.cuda())
    assert torch.equal(loss, clean[0]) and torch.isnan(lse.cpu()[~keep]).all() and torch.equal(lse.cpu()[keep], clean[1].cpu()[keep])
    g1 = mx.linear_xent_backward(dloss.cuda(), bad.cuda(), w.cuda(), target.cuda(), lse)
    assert torch.equal(g0[0], g1[0]) and torch.equal(g0[1], g1[1])
    # a target that is no index: NaN loss, no gradient; the other rows as before
    odd = target.clone()
    rows = keep.nonzero()[:3, 0]
    odd[rows] = torch.tensor([300, -1, 1 << 40])
    loss, lse = mx.linear_xent_forward(x.cuda(), w.cuda(), odd.cuda())
    assert torch.isnan(loss.cpu()).nonzero()[:, 0].tolist() == rows.tolist() and torch.equal(lse, clean[1])
    ign = target.clone()
    ign[rows] = -100
    a = mx.linear_xent_backward(dloss.cuda(), x.cuda(), w.cuda(), odd.cuda(), lse)
    b = mx.linear_xent_backward(dloss.cuda(), x.cuda(), w.cuda(), ign.cuda(), lse)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_magnitudes_far_from_one():
    """FP16 operands over bf16's range: X and W far larger and smaller than FP16 holds, and tiny row gradients."""
    for ex, ew, eg in ((20, -22, -30), (-40, 38, 0), (18, -18, 20), (-60, 60, -60)):
        x, w, target, dloss, dlse = _problem(70, 64, 300, seed=ex)
        announce("xent magnitudes", ex, ew, eg)
        _check((x.float() * 2.0 ** ex).to(BF), (w.float() * 2.0 ** ew).to(BF), target, dloss * 2.0 ** eg, dlse * 2.0 ** eg,
               dtype=torch.float32)


def test_infinite_logits():
    mx = _mx()
    x, w, target, dloss, _ = _problem(4, 32, 300)
    target[:] = torch.tensor([0, 1, 2, 3])
    x[:, 0] = torch.tensor([0.0, 1.0, 1.0, 1.0]).to(BF)
    w[:, 0] = 0.0
    w[100:, 0] = float("-inf")                    # rows 1 .. 3: most of the vocabulary masked out; row 0: 0 * inf
    announce("xent infinities")
    loss, lse = mx.linear_xent_forward(x.cuda(), w.cuda(), target.cuda())
    r = torch.logsumexp(x[1:].double() @ w[:100].double().t(), dim=1)
    assert torch.isnan(lse[0]) and float((lse[1:].cpu().double() - r).abs().max()) < 1e-5


def test_gradients_against_differences():
    """Along a random direction of X and of W, (loss(+h) - loss(-h)) / 2h from the operator's own losses in
    steps that bf16 holds exactly."""
    mx = _mx()
    g = torch.Generator().manual_seed(11)
    T, K, V = 64, 64, 200
    x = (torch.randint(-64, 65, (T, K), generator=g) / 64.0)
    w = (torch.randint(-32, 33, (V, K), generator=g) / 64.0)
    h = 2.0 ** -6                                  # a step of both grids: every shifted value has 7 bits or fewer
    target = torch.randint(0, V, (T,), generator=g).cuda()
    one = torch.ones(T, device="cuda")
    total = lambda a, b: float(mx.linear_xent_forward(a.to(BF).cuda(), b.to(BF).cuda(), target)[0].double().sum())  # noqa: E731
    lse = mx.linear_xent_forward(x.to(BF).cuda(), w.to(BF).cuda(), target)[1]
    dx, dw = mx.linear_xent_backward(one, x.to(BF).cuda(), w.to(BF).cuda(), target, lse, dx_dtype=torch.float32,
                                     dw_dtype=torch.float32)
    for grad, of in ((dx, "x"), (dw, "w")):
        d = torch.randint(0, 2, grad.shape, generator=g) * 2.0 - 1.0
        up = total(x + h * d, w) if of == "x" else total(x, w + h * d)
        dn = total(x - h * d, w) if of == "x" else total(x, w - h * d)
        slope = (up - dn) / (2 * h)
        want = float((grad.cpu().double() * d).sum())
        # third derivatives of T losses, each at most |dz|^3 h^2 with |dz| <= |d| |w| ~ 3, and G's rounding
        assert abs(slope - want) <= T * 27 * h * h / 6 + 2.0 ** -8 * float(grad.abs().sum())


def test_strided_inputs_other_stream_and_graph():
    mx = _mx()
    x, w, target, dloss, _ = _problem(200, 64, 700)
    wide = torch.zeros(200, 96, dtype=BF, device="cuda")
    wide[:, 8:72] = x.cuda()
    tall = torch.zeros(1400, 64, dtype=BF, device="cuda")
    tall[::2] = w.cuda()
    X, W, Tg, D = x.cuda(), w.cuda(), target.cuda(), dloss.cuda()
    loss, lse = mx.linear_xent_forward(X, W, Tg)
    grads = mx.linear_xent_backward(D, X, W, Tg, lse)
    l2, s2 = mx.linear_xent_forward(wide[:, 8:72], tall[::2], Tg)
    g2 = mx.linear_xent_backward(D, wide[:, 8:72], tall[::2], Tg, lse)
    assert torch.equal(loss, l2) and torch.equal(lse, s2) and torch.equal(grads[0], g2[0]) and torch.equal(grads[1], g2[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    l3, s3 = mx.linear_xent_forward(X, W, Tg, stream=side)
    g3 = mx.linear_xent_backward(D, X, W, Tg, s3, stream=side)
    side.synchronize()
    assert torch.equal(loss, l3) and torch.equal(grads[0], g3[0]) and torch.equal(grads[1], g3[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gl, gs = mx.linear_xent_forward(X, W, Tg)
        gdx, gdw = mx.linear_xent_backward(D, X, W, Tg, gs)
    for k in range(3):
        X.copy_(torch.randn(200, 64, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        el, es = mx.linear_xent_forward(X, W, Tg)
        edx, edw = mx.linear_xent_backward(D, X, W, Tg, es)
        assert torch.equal(gl, el) and torch.equal(gdx, edx) and torch.equal(gdw, edw)
