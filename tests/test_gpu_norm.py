"""RMS norm on the GPU, forward and backward, against the formulas in 64 bits; the 8-bit outputs bit for bit."""
import numpy as np
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, HALF, U, assert_within, check_axes, heavy, norm_grad, norm_rstd, norm_stream, norm_y32

pytestmark = pytest.mark.gpu
EPS = 1e-5
TYPES = [(BF, BF), (BF, F32), (F32, F32), (F32, BF)]        # branch, stream
# a single value, less than eight, ends inside eight and inside a block, every way of working a row, and rows too long for registers
SIZES = [(1, 1), (3, 7), (1, 4096), (5, 129), (130, 384), (2, 512), (7, 513), (129, 1000), (3, 1024), (2, 1100), (9, 2001), (3, 2056),
         (300, 256), (5, 4097), (2, 8200), (3, 9001), (3, 16384), (2, 16383), (12, 8), (2, 16390), (2, 33000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _data(rows, cols, branch, stream, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 31 + cols)
    x = torch.randn(rows, cols, generator=g).to(branch)
    r = (3 * torch.randn(rows, cols, generator=g)).to(stream)
    r[:, ::97] *= 50
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(BF)
    return x, r, w


def _check_forward(o, x, r, w, eps, axis, y_dtype):
    h = norm_stream(x, r)
    assert torch.equal(o.h.cpu(), h)
    rstd = norm_rstd(h, eps)
    assert_within(o.rstd, rstd, rstd * U * 1.0001, "rstd")
    y = norm_y32(h, o.rstd.cpu(), w)
    if y_dtype is not None:
        assert torch.equal(o.y.cpu(), y.to(y_dtype))
        # and against the formula: rstd, two products, and a last rounding
        exact = h.double() * rstd[:, None] * (1.0 if w is None else w.double())
        assert_within(o.y, exact, exact.abs() * (3.01 * U + (HALF[y_dtype] if y_dtype == BF else 0.0)) + 2.0 ** -149, "y")
    else:
        assert o.y is None
    check_axes(o, y, axis)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("branch,stream", TYPES)
def test_forward(rows, cols, branch, stream):
    mx = _mx()
    x, r, w = _data(rows, cols, branch, stream)
    announce("norm forward", rows, cols, branch, stream)
    for residual, weight, axis, y_dtype in ((r, w, "both", BF), (None, w.float(), 1, F32), (r, None, 0, None), (None, None, None, BF)):
        o = mx.rmsnorm_forward(x.cuda(), None if weight is None else weight.cuda(), None if residual is None else residual.cuda(), EPS,
                               axis=axis, y_dtype=y_dtype)
        _check_forward(o, x, residual, weight, EPS, axis, y_dtype)


@pytest.mark.parametrize("rows,cols", [(200, 384), (5, 2001), (3, 20000)])
def test_strides_alignment_and_in_place(rows, cols):
    mx = _mx()
    x, r, w = _data(rows, cols, BF, BF)
    announce("norm strides", rows, cols)
    wide = [torch.zeros(rows, cols + 13, dtype=BF).cuda() for _ in range(4)]
    views = [t[:, k:k + cols] for t, k in zip(wide, (1, 3, 5, 8))]
    views[0].copy_(x)
    views[1].copy_(r)
    wv = torch.zeros(cols + 1, dtype=BF).cuda()[1:]
    wv.copy_(w)
    base = mx.rmsnorm_forward(x.cuda(), w.cuda(), r.cuda(), EPS, axis="both")
    o = mx.rmsnorm_forward(views[0], wv, views[1], EPS, axis="both", h=views[2], y=views[3])
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b))  # noqa: E731
    nb = lambda o: (o.h, o.rstd, o.y, o.q1, o.s1[:, :(cols + 127) // 128], o.q0, o.s0[:, :(rows + 127) // 128])  # noqa: E731
    assert same(nb(base), nb(o)) and o.h is views[2] and o.y is views[3]
    for t, k in zip(wide[2:], (5, 8)):                          # nothing beside the rows
        assert not bool(t[:, :k].any()) and not bool(t[:, k + cols:].any())
    for target in (0, 1):                                       # h = x, h = residual
        xs, rs = views[0].clone(), views[1].clone()
        o = mx.rmsnorm_forward(xs, w.cuda(), rs, EPS, axis="both", h=(xs, rs)[target])
        assert same(nb(base), nb(o))
    # every second row of a matrix, and a single row whose stride says nothing
    tall = torch.zeros(2 * rows, cols, dtype=BF).cuda()
    tall[::2] = x.cuda()
    o, base = mx.rmsnorm_forward(tall[::2], w.cuda(), axis=1), mx.rmsnorm_forward(x.cuda(), w.cuda(), axis=1)
    assert torch.equal(o.y, base.y) and torch.equal(o.q1, base.q1)
    assert torch.equal(mx.rmsnorm_forward(tall[:1], w.cuda()).y, base.y[:1])


@pytest.mark.parametrize("cols", [300, 2048, 4096, 20000])
@pytest.mark.parametrize("branch,stream", [(BF, BF), (BF, F32), (F32, F32)])
def test_without_keeping_the_sum(cols, branch, stream):
    mx = _mx()
    x, r, w = _data(6, cols, branch, stream)
    full = mx.rmsnorm_forward(x.cuda(), w.cuda(), r.cuda(), EPS, axis=1)
    o = mx.rmsnorm_forward(x.cuda(), w.cuda(), r.cuda(), EPS, axis=1, need_h=False)
    assert o.h is None and torch.equal(o.y, full.y) and torch.equal(o.rstd, full.rstd) and torch.equal(o.q1, full.q1)
    nb = (cols + 127) // 128
    assert torch.equal(o.s1[:, :nb], full.s1[:, :nb])
    twice = x.cuda().clone()                                    # x + x in place
    o = mx.rmsnorm_forward(twice, w.cuda(), twice, EPS, h=twice)
    assert torch.equal(twice.cpu(), norm_stream(x, x)) and torch.equal(o.y, mx.rmsnorm_forward(twice, w.cuda(), eps=EPS).y)


@pytest.mark.parametrize("rows,cols", [(130, 700), (3, 4100), (2, 17000)])
def test_blocks_of_tiny_values_and_of_zeros(rows, cols):
    """Scale bytes of 0 (a block's maximum below 448 * 2^-127) beside ordinary ones, along both axes, and values below FP32's normal
    range."""
    mx = _mx()
    x, _, w = _data(rows, cols, F32, F32)
    w = w.float()
    for k, scale in ((0, 2.0 ** -119), (1, 0.0), (2, 2.0 ** -126), (3, 2.0 ** -135), (4, 2.0 ** 100)):
        w[128 * k:128 * k + 128] *= scale                       # whole blocks along the rows, and columns
        w[128 * k + 5] = 2.0 ** -130
    x[rows // 2] = 0.0
    announce("norm tiny", rows, cols)
    o = mx.rmsnorm_forward(x.cuda(), w.cuda(), eps=EPS, axis="both", y_dtype=F32)
    y = norm_y32(x, o.rstd.cpu(), w)
    assert torch.equal(o.y.cpu(), y)
    check_axes(o, y, "both")
    assert int((o.s1[:, :(cols + 127) // 128] == 0).sum()) > rows and bool((o.s0[:700, 0] == 0).any())


def test_single_outputs_of_the_library():
    """Each output alone, which the binding does not ask for: rstd, h, y."""
    mx = _mx()
    L = mx.layer_lib()
    for cols in (512, 4096, 20000):
        x, r, w = (t.cuda() for t in _data(5, cols, BF, BF))
        full = mx.rmsnorm_forward(x, w, r, EPS)
        h, y, rstd = torch.zeros_like(r), torch.zeros_like(x), torch.zeros(5, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream

        def call(h=None, rstd=None, y=None):
            at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
            return L.mxfp4_rmsnorm_forward(x.data_ptr(), 0, cols, r.data_ptr(), cols, 0, w.data_ptr(), 0, 5, cols, EPS, at(h), cols, at(rstd),
                                           at(y), 1, cols, None, 0, None, 0, None, 0, None, 0, stream)
        assert call(h=h) == 0 and torch.equal(h, full.h)
        assert call(rstd=rstd) == 0 and torch.equal(rstd, full.rstd)
        assert call(y=y) == 0 and torch.equal(y, full.y)


def test_no_rows():
    mx = _mx()
    x, w = torch.zeros(0, 300, dtype=BF).cuda(), torch.ones(300).cuda()
    o = mx.rmsnorm_forward(x, w, x, axis="both")
    assert o.y.shape == (0, 300) and o.q1.shape == (0, 384) and o.q0.shape == (300, 0)
    g = mx.rmsnorm_backward(x, x, o.rstd, w, dres=x, dweight=torch.full((300,), 7.0).cuda())
    assert g.dh.shape == (0, 300) and not bool(g.dweight.any())


@pytest.mark.parametrize("cols", [300, 4096, 17000])
def test_ends_of_the_range(cols):
    """Zeros, FP32's ends, infinities and NaN: each in its own row, the others as ever."""
    mx = _mx()
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(8, cols, generator=g)
    x[0] = 0.0
    x[1] *= 2.0 ** 110                # squares far beyond FP32
    x[2] *= 2.0 ** -120               # and far below it
    x[3, cols // 2] = float("inf")
    x[4, 1] = float("nan")
    x[5] = 3.0e38                     # the sum of squares of the largest values
    w = torch.ones(cols)
    announce("norm ends", cols)
    for eps in (0.0, EPS):
        o = mx.rmsnorm_forward(x.cuda(), w.cuda(), eps=eps, axis="both", y_dtype=F32)
        rstd = norm_rstd(x, eps)
        got = o.rstd.cpu().double()
        for i in (1, 2, 5, 6, 7) + ((0,) if eps else ()):
            # rstd of row 5 lies below FP32's normal range, where a rounding is 2^-150
            assert abs(float(got[i] - rstd[i])) <= float(rstd[i]) * U * 1.0001 + 2.0 ** -150, (eps, i)
            assert torch.equal(o.y[i].cpu(), norm_y32(x[i:i + 1], o.rstd[i:i + 1].cpu(), w)[0]), (eps, i)
        assert float(got[3]) == 0.0 and bool(torch.isnan(o.y[3, cols // 2])) and int((o.y[3] != 0).sum()) == 1
        assert bool(torch.isnan(o.y[4]).all()) and bool((o.s1[4, :(cols + 127) // 128] == 255).all()) and not bool(o.q1[4].any())
        assert int((o.s1[3] == 255)[:(cols + 127) // 128].sum()) == 1
        if not eps:
            assert bool(torch.isinf(o.rstd[0])) and bool(torch.isnan(o.y[0]).all())
        assert bool((o.s0[:, 0] == 255).all())                  # every column's block holds the row of NaN
        y = norm_y32(x[6:], o.rstd[6:].cpu(), w)
        o = mx.rmsnorm_forward(x[6:].cuda(), w.cuda(), eps=eps, axis="both")
        check_axes(o, y, "both")


@pytest.mark.parametrize("rows,cols", SIZES + [(2000, 512), (1500, 1000), (700, 2048)])
@pytest.mark.parametrize("branch,stream", TYPES)
def test_backward(rows, cols, branch, stream):
    mx = _mx()
    _, h, w = _data(rows, cols, branch, stream)
    dy, dres = heavy((rows, cols), rows + cols, 1e-3).to(branch), heavy((rows, cols), rows + cols + 1, 1e-3).to(stream)
    rstd = norm_rstd(h, EPS).float()
    announce("norm backward", rows, cols, branch, stream)
    for weight, res, wt in ((w, dres, F32), (w.float(), None, BF), (None, dres, F32)):
        got = mx.rmsnorm_backward(dy.cuda(), h.cuda(), rstd.cuda(), None if weight is None else weight.cuda(),
                                  None if res is None else res.cuda(), dweight_dtype=wt)
        dh, dw, tol, tol_w = norm_grad(dy, h, rstd, weight, res)
        assert got.dh.dtype == stream and got.dweight.dtype == wt
        assert_within(got.dh, dh, tol + HALF[stream] * (dh.abs() + tol) + 2.0 ** -149, "dh")
        assert_within(got.dweight, dw, tol_w + HALF[wt] * (dw.abs() + tol_w) + 2.0 ** -149, "dw")
        alone = mx.rmsnorm_backward(dy.cuda(), h.cuda(), rstd.cuda(), None if weight is None else weight.cuda(),
                                    None if res is None else res.cuda(), need_dweight=False)
        assert alone.dweight is None and torch.equal(alone.dh, got.dh)


def test_backward_strides_and_in_place():
    mx = _mx()
    for rows, cols in ((200, 384), (30, 2001), (3, 20000)):
        _, h, w = _data(rows, cols, BF, BF)
        dy, dres = heavy((rows, cols), 5, 1e-3).to(BF), heavy((rows, cols), 6, 1e-3).to(BF)
        rstd = norm_rstd(h, EPS).float().cuda()
        announce("norm backward strides", rows, cols)
        base = mx.rmsnorm_backward(dy.cuda(), h.cuda(), rstd, w.cuda(), dres.cuda())
        wide = [torch.zeros(rows, cols + 13, dtype=BF).cuda() for _ in range(4)]
        views = [t[:, k:k + cols] for t, k in zip(wide, (1, 3, 5, 8))]
        for v, t in zip(views, (dy, h, dres)):
            v.copy_(t)
        got = mx.rmsnorm_backward(views[0], views[1], rstd, w.cuda(), views[2], dh=views[3])
        assert torch.equal(got.dh, base.dh) and torch.equal(got.dweight, base.dweight)
        assert not bool(wide[3][:, :8].any()) and not bool(wide[3][:, 8 + cols:].any())
        d = dres.cuda()
        got = mx.rmsnorm_backward(dy.cuda(), h.cuda(), rstd, w.cuda(), d, dh=d)
        assert got.dh is d and torch.equal(d, base.dh) and torch.equal(got.dweight, base.dweight)


def test_backward_against_differences():
    """The gradients are those of the forward call: central differences of sum(y * c + h * e) in FP32."""
    mx = _mx()
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, res, w, c, e = r(6, 200), r(6, 200), 1 + 0.2 * r(200), r(6, 200), r(6, 200)

    def value(x, w):
        o = mx.rmsnorm_forward(x, w, res, EPS, y_dtype=F32)
        return float((o.y.double() * c.double() + o.h.double() * e.double()).sum())
    o = mx.rmsnorm_forward(x, w, res, EPS, y_dtype=F32)
    got = mx.rmsnorm_backward(c, o.h, o.rstd, w, dres=e)
    step = 2.0 ** -7
    for k in range(8):
        dx, dw = r(6, 200), r(200)
        slope = (value(x + step * dx, w + step * dw) - value(x - step * dx, w - step * dw)) / (2 * step)
        want = float((got.dh.double() * dx.double()).sum() + (got.dweight.double() * dw.double()).sum())
        # 1200 outputs of about one, each off by 2^-22 and divided by 2 step; the third derivative of a norm of 200 values along
        # such a direction, some tens, times step^2 / 6
        assert abs(slope - want) <= 1200 * 2.0 ** -22 / (2 * step) + 100 * step ** 2 / 6


def test_rows_of_one_call_do_not_depend_on_the_others():
    mx = _mx()
    x, r, w = _data(300, 1000, BF, BF)
    whole = mx.rmsnorm_forward(x.cuda(), w.cuda(), r.cuda(), EPS, axis=1)
    part = mx.rmsnorm_forward(x[37:41].cuda(), w.cuda(), r[37:41].cuda(), EPS, axis=1)
    for a, b in ((whole.h, part.h), (whole.rstd, part.rstd), (whole.y, part.y), (whole.q1, part.q1), (whole.s1[:, :8], part.s1[:, :8])):
        assert np.array_equal(a[37:41].cpu().float().numpy(), b.cpu().float().numpy())


def test_many_rows():
    """More rows than workgroups of one launch."""
    mx = _mx()
    rows = (1 << 22) + 5
    x = torch.randn(rows, 8, device="cuda").to(BF)
    announce("norm rows", rows)
    o = mx.rmsnorm_forward(x, eps=EPS, axis=1)
    h = x.double()
    rstd = (h.square().mean(dim=1) + EPS).rsqrt()
    assert bool(((o.rstd.double() - rstd).abs() <= rstd * U * 1.0001).all())
    assert torch.equal(o.y, (x.float() * o.rstd[:, None]).to(BF))
    g = mx.rmsnorm_backward(x, x, o.rstd)
    dw = (h * h * o.rstd.double()[:, None]).sum(dim=0)
    assert bool(((g.dweight.double() - dw).abs() <= U * (68 + rows / 64) * dw).all())


def test_many_rows_of_several_wavefronts():
    """A workgroup works several rows one after the other, each joined over its wavefronts."""
    mx = _mx()
    rows, cols = (1 << 20) + 3000, 1032
    x = torch.randn(rows, cols, device="cuda").to(BF)
    announce("norm rows", rows, cols)
    o = mx.rmsnorm_forward(x, eps=EPS, axis=1)
    for at in (0, 2990, (1 << 20) - 10, 1 << 20, rows - 20):     # rows of the first and of the second turn
        p = mx.rmsnorm_forward(x[at:at + 20], eps=EPS, axis=1)
        assert torch.equal(p.rstd, o.rstd[at:at + 20]) and torch.equal(p.y, o.y[at:at + 20]) and torch.equal(p.q1, o.q1[at:at + 20])
    n = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for part, to in zip(x.split(1 << 17), n.split(1 << 17)):
        to.copy_((part.double().square().mean(dim=1) + EPS).rsqrt())
    assert bool(((o.rstd.double() - n).abs() <= n * U * 1.0001).all())
