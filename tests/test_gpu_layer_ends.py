"""Infinities, NaN and rows of zeros in the gradients of the norm and of the gated activation, on the GPU: they are where the formulas in
FP32 have them, and the blocks of 8-bit codes that hold one have the scale 0xFF and zero codes."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, HALF, assert_within, check_axes, check_codes, norm_grad

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _same_kind(got, want, what):
    """NaN and infinities (with their signs) in the same places."""
    got, want = got.cpu().float(), want.float()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    at = torch.isinf(want)
    assert torch.equal(torch.isinf(got), at) and torch.equal(got[at], want[at]), what


# a whole tile, the matrix' ends, and both, with the bad values in either
@pytest.mark.parametrize("rows,cols", [(128, 128), (130, 300), (256, 384), (5, 7), (3, 260)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", ["gate", "up", "da"])
def test_gated_activation(rows, cols, dtype, which):
    mx = _mx()
    g = torch.Generator().manual_seed(rows + cols)
    t = {k: (torch.where(torch.rand(rows, cols, generator=g) < 0.5, -1.0, 1.0) * (0.25 + torch.rand(rows, cols, generator=g))).to(dtype)
         for k in ("gate", "up", "da")}
    for k, (i, j) in enumerate(((0, 0), (rows // 2, cols - 1), (rows - 1, cols // 2))):
        t[which][i, j] = (NAN, INF, -INF)[k]
    announce("gate ends", rows, cols, dtype, which)
    gate, up, da = (t[k].float() for k in ("gate", "up", "da"))
    s = 1 / (1 + torch.exp(-gate))
    dev = [t[k].cuda() for k in ("da", "gate", "up")]
    o = mx.swiglu_backward(*dev, axis="both", out_dtype=F32, joined=False)
    _same_kind(o.dgate, da * (up * (s * (1 + gate * (1 - s)))), "dgate")
    _same_kind(o.dup, da * (gate * s), "dup")
    check_axes(o.gate, o.dgate.cpu(), "both", "dgate")
    check_axes(o.up, o.dup.cpu(), "both", "dup")
    # the blocks of the bad values alone
    for codes, wide in ((o.gate, o.dgate.cpu()), (o.up, o.dup.cpu())):
        for s8, v in ((codes.s1, wide), (codes.s0, wide.t())):
            nb = (v.shape[1] + 127) // 128
            bad = torch.nn.functional.pad(~torch.isfinite(v), (0, nb * 128 - v.shape[1])).reshape(v.shape[0], nb, 128).any(dim=2)
            assert torch.equal(s8[:, :nb].cpu() == 255, bad)
    wide = torch.cat([o.dgate, o.dup], dim=1).cpu()
    j = mx.swiglu_backward(*dev, axis="both" if cols % 128 == 0 else 0)
    _same_kind(j.dgate, wide[:, :cols].to(BF), "joined dgate")
    check_codes(j.q0, j.s0, wide.t().contiguous(), "joined")
    if cols % 128 == 0:
        check_codes(j.q1, j.s1, wide, "joined")
    if which != "da":
        f = mx.swiglu_forward(*dev[1:], axis="both", out_dtype=F32)
        _same_kind(f.a, gate * s * up, "a")
        check_axes(f, f.a.cpu(), "both", "a")


def _norm_formula(dy, h, rstd, w, dres):
    """Product by product in FP32, as the kernels form them."""
    n = h.float() * rstd[:, None]
    u = dy.float() * w.float()
    mean = (u * n).mean(dim=1, keepdim=True)
    return (u - n * mean) * rstd[:, None] + dres.float(), (dy.float() * n).sum(dim=0)


@pytest.mark.parametrize("cols", [5, 40, 513, 1000, 2001, 4096, 8200, 16384, 16390])
@pytest.mark.parametrize("branch,stream", [(BF, BF), (BF, F32), (F32, F32)])
def test_norm(cols, branch, stream):
    mx = _mx()
    rows = 12
    g = torch.Generator().manual_seed(cols)
    r = lambda dtype: (torch.where(torch.rand(rows, cols, generator=g) < 0.5, -1.0, 1.0)  # noqa: E731
                       * (0.25 + torch.rand(rows, cols, generator=g))).to(dtype)
    dy, h, dres = r(branch), r(stream), r(stream)
    w = (0.5 + torch.rand(cols, generator=g)).to(BF)
    last = cols - 1
    h[1, 0], h[2, last], h[3, cols // 2] = NAN, INF, -INF
    h[4] = 0.0                                               # rstd is infinite
    dy[6, last], dy[7, 0], dy[8, cols // 2] = NAN, INF, -INF
    dres[9, 0], dres[10, last] = NAN, -INF
    announce("norm ends", cols, branch, stream)
    rstd = mx.rmsnorm_forward(h.cuda(), eps=0.0).rstd
    assert bool(torch.isnan(rstd[1])) and rstd[2:5].cpu().tolist() == [0.0, 0.0, INF]
    o = mx.rmsnorm_backward(dy.cuda(), h.cuda(), rstd, w.cuda(), dres=dres.cuda())
    dh, _ = _norm_formula(dy, h, rstd.cpu(), w, dres)
    _same_kind(o.dh, dh, "dh")
    # the rows without any are those of the formula, and so is dweight of those rows alone
    good = torch.tensor([0, 5, 11])
    want, dw, tol, tol_w = norm_grad(dy[good], h[good], rstd.cpu()[good], w, dres[good])
    assert_within(o.dh[good.cuda()], want, tol + (HALF[stream] * (want.abs() + tol) if stream == BF else 0.0), "dh")
    assert bool(torch.isnan(o.dweight).all())                # rows 1 and 4
    # a row with an infinity, or one in dy or dres, leaves the other columns of dweight as they are
    some = torch.tensor([0, 2, 3, 5, 6, 7, 8, 9, 10, 11])
    take = lambda t: t[some].contiguous().cuda()  # noqa: E731
    o = mx.rmsnorm_backward(take(dy), take(h), rstd[some.cuda()], w.cuda(), dres=take(dres))
    dh, dw = _norm_formula(dy[some], h[some], rstd.cpu()[some], w, dres[some])
    _same_kind(o.dh, dh, "dh")
    _same_kind(o.dweight, dw, "dweight")
    assert int(torch.isfinite(dw).sum()) >= cols - 3


@pytest.mark.parametrize("cols", [40, 1000, 4096, 16390])
@pytest.mark.parametrize("exponent", [-118, -60, 60, 118])
def test_norm_of_large_and_small_values(cols, exponent):
    """Streams near both ends of FP32's range: rstd is near the other one, and every product of the formula stays in it."""
    mx = _mx()
    rows = 5
    g = torch.Generator().manual_seed(cols + exponent)
    r = lambda: torch.where(torch.rand(rows, cols, generator=g) < 0.5, -1.0, 1.0) * (0.25 + torch.rand(rows, cols, generator=g))  # noqa: E731
    h, dy, dres = r() * 2.0 ** exponent, r(), r() * 2.0 ** -exponent
    w = (0.5 + torch.rand(cols, generator=g)).to(BF)
    rstd = mx.rmsnorm_forward(h.cuda(), eps=0.0).rstd
    announce("norm range", cols, exponent)
    o = mx.rmsnorm_backward(dy.cuda(), h.cuda(), rstd, w.cuda(), dres=dres.cuda())
    dh, dw, tol, tol_w = norm_grad(dy, h, rstd.cpu(), w, dres)
    assert_within(o.dh, dh, tol + 2.0 ** -149, "dh")
    assert_within(o.dweight, dw, tol_w, "dweight")
