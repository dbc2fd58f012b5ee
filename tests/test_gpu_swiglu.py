"""The gated activation on the GPU, forward and backward, against the formulas in 64 bits; the 8-bit outputs bit for bit."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, HALF, TINY, assert_within, check_axes, check_codes, gate_backward, gate_forward, heavy

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (1, 14336), (3, 7), (128, 128), (5, 129), (130, 384), (257, 1000), (129, 2001), (2, 256)]


def _own(gate):
    """The header's bound. exp(-g) = exp2(-g log2 e): the product is rounded by |g| log2(e) 2^-24 at most and log2(e) itself by 2^-26 of
    it, which is 1.25 |g| 2^-24 of the exponential (the derivative of exp2 is ln 2); its own 2^-23, the sum's 2^-24, the
    reciprocal's 2^-23 and three products make 8 * 2^-24 more: together less than 2^-20 (1 + |g| / 12)."""
    return 2.0 ** -20 * (1 + gate.double().abs() / 12)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _data(rows, cols, dtype, spread=2.0):
    g = torch.Generator().manual_seed(rows * 13 + cols)
    gate, up = spread * torch.randn(rows, cols, generator=g), torch.randn(rows, cols, generator=g)
    gate.view(-1)[::11] *= 20                        # far tails of the exponential
    return gate.to(dtype), up.to(dtype), heavy((rows, cols), rows + cols, 1e-3)


def _tol(exact, basis, dtype, factor, gate):
    """factor: what s is multiplied with. s below 2^-126 may be lost (exp(-|g|) counts as zero there), which the product makes
    2^-126 |factor|: with g = -90 and u = 2 that is 180 * 2^-126, of a value of 7e-38 = 8 * 2^-126 and less."""
    tol = _own(gate) * basis + TINY * (1 + factor.double().abs())
    return tol + (HALF[dtype] * (exact.abs() + tol) if dtype == BF else 0.0)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(rows, cols, dtype):
    mx = _mx()
    gate, up, _ = _data(rows, cols, dtype)
    announce("gate forward", rows, cols, dtype)
    exact = gate_forward(gate, up)
    for axis, out in ((None, BF), ("both", F32), (1, F32), (0, F32)):
        o = mx.swiglu_forward(gate.cuda(), up.cuda(), axis=axis, out_dtype=out)
        assert_within(o.a, exact, _tol(exact, exact.abs(), out, gate.double() * up.double(), gate), "a")
        if out == F32:
            check_axes(o, o.a.cpu(), axis)              # the codes are those of the FP32 values
            full = o
    o = mx.swiglu_forward(gate.cuda(), up.cuda(), axis="both", out_dtype=None)
    assert o.a is None
    check_axes(o, full.a.cpu(), "both")
    assert torch.equal(mx.swiglu_forward(gate.cuda(), up.cuda()).a, full.a.to(BF))


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,dtype_a", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_backward(rows, cols, dtype, dtype_a):
    mx = _mx()
    gate, up, da = _data(rows, cols, dtype)
    da = da.to(dtype_a)
    dg, du, basis = gate_backward(da, gate, up)
    dev = da.cuda(), gate.cuda(), up.cuda()
    announce("gate backward", rows, cols, dtype, dtype_a)
    o = mx.swiglu_backward(*dev, axis="both", out_dtype=F32, joined=False)
    assert_within(o.dgate, dg, _tol(dg, basis, F32, da.double() * up.double() * (1 + gate.double().abs()), gate), "dgate")
    assert_within(o.dup, du, _tol(du, du.abs(), F32, da.double() * gate.double(), gate), "dup")
    check_axes(o.gate, o.dgate.cpu(), "both", "dgate")
    check_axes(o.up, o.dup.cpu(), "both", "dup")
    wide = torch.cat([o.dgate, o.dup], dim=1).cpu()
    b = mx.swiglu_backward(*dev)
    assert torch.equal(b.dgate, o.dgate.to(BF)) and torch.equal(b.dup, o.dup.to(BF)) and b.q1 is None
    assert b.dgate.stride(0) == 2 * cols or rows == 1
    # as one operand of 2 F: columns with any F, rows with whole blocks
    j = mx.swiglu_backward(*dev, axis="both" if cols % 128 == 0 else 0, out_dtype=None)
    assert j.dgate is None
    check_codes(j.q0, j.s0, wide.t().contiguous(), "columns of both")
    if cols % 128 == 0:
        check_codes(j.q1, j.s1, wide, "rows of both")


def test_halves_strides_and_in_place():
    mx = _mx()
    for rows, cols in ((200, 384), (30, 1001)):
        gate, up, da = _data(rows, cols, BF)
        da = da.to(BF)
        announce("gate strides", rows, cols)
        base, grad = mx.swiglu_forward(gate.cuda(), up.cuda()), mx.swiglu_backward(da.cuda(), gate.cuda(), up.cuda())
        both = torch.cat([gate, up], dim=1).cuda()
        g, u = both[:, :cols], both[:, cols:]
        wide = torch.zeros(rows, cols + 9, dtype=BF).cuda()
        a = mx.swiglu_forward(g, u, a=wide[:, 3:3 + cols]).a
        assert torch.equal(a, base.a) and not bool(wide[:, :3].any()) and not bool(wide[:, 3 + cols:].any())
        off = torch.zeros(rows, cols + 1, dtype=BF).cuda()[:, 1:]
        off.copy_(da)
        got = mx.swiglu_backward(off, g, u)
        assert torch.equal(got.dgate, grad.dgate) and torch.equal(got.dup, grad.dup)
        d = both.clone()
        got = mx.swiglu_backward(off, d[:, :cols], d[:, cols:], dgate=d[:, :cols], dup=d[:, cols:])        # over gate and up
        assert torch.equal(got.dgate, grad.dgate) and torch.equal(d[:, cols:], grad.dup)
        d = both.clone()
        got = mx.swiglu_backward(off, d[:, :cols], d[:, cols:], dgate=off, dup=d[:, :cols])                 # over da and gate
        assert torch.equal(off, grad.dgate) and torch.equal(d[:, :cols], grad.dup)
        for k in (0, 1):
            d = both.clone()
            mx.swiglu_forward(d[:, :cols], d[:, cols:], a=(d[:, :cols], d[:, cols:])[k])
            assert torch.equal((d[:, :cols], d[:, cols:])[k], base.a)


@pytest.mark.parametrize("rows,cols", [(1, 3), (2, 8), (131, 9), (126, 135), (257, 1001)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_in_place_at_the_ends(rows, cols, dtype):
    """a over gate or up, where threads at the matrix' ends read values that others write."""
    mx = _mx()
    gate, up, _ = _data(rows, cols, dtype)
    announce("gate in place", rows, cols, dtype)
    base = mx.swiglu_forward(gate.cuda(), up.cuda(), axis="both", out_dtype=dtype)
    for k in (0, 1):
        at = gate.cuda(), up.cuda()
        o = mx.swiglu_forward(*at, axis="both", a=at[k])
        assert torch.equal(at[k], base.a) and torch.equal(o.q1, base.q1) and torch.equal(o.q0, base.q0)


@pytest.mark.parametrize("rows,cols", [(130, 256), (5, 300)])
def test_single_outputs_of_the_library(rows, cols):
    """Each gradient alone and each kind of codes of one of them, which the binding does not ask for."""
    mx = _mx()
    L = mx.layer_lib()
    gate, up, da = _data(rows, cols, BF)
    dev = da.to(BF).cuda(), gate.cuda(), up.cuda()
    full = mx.swiglu_backward(*dev, axis="both", joined=False)
    stream = torch.cuda.current_stream().cuda_stream
    lq1, ls1, lq0, ls0 = full.gate.q1.stride(0), full.gate.s1.stride(0), full.gate.q0.stride(0), full.gate.s0.stride(0)

    def call(dgate=None, dup=None, q1=(None, None), s1=(None, None), q0=(None, None), s0=(None, None)):
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        status = L.mxfp4_swiglu_backward(at(dev[0]), 0, cols, at(dev[1]), cols, at(dev[2]), cols, 0, rows, cols, at(dgate), cols, at(dup), cols,
                                         1, *map(at, q1), lq1, *map(at, s1), ls1, *map(at, q0), lq0, *map(at, s0), ls0, stream)
        assert status == 0
    new = lambda t: torch.full_like(t, 77)  # noqa: E731
    for name in ("dgate", "dup"):
        t = new(full.dgate)
        call(**{name: t})
        assert torch.equal(t, getattr(full, name))
    for k, want in enumerate((full.gate, full.up)):
        q, s = new(want.q1), new(want.s1)
        call(q1=(q, None) if k == 0 else (None, q), s1=(s, None) if k == 0 else (None, s))
        nb = (cols + 127) // 128
        assert torch.equal(q, want.q1) and torch.equal(s[:, :nb], want.s1[:, :nb]) and bool((s[:, nb:] == 77).all())
        q, s = new(want.q0), new(want.s0)
        call(q0=(q, None) if k == 0 else (None, q), s0=(s, None) if k == 0 else (None, s))
        nb = (rows + 127) // 128
        assert torch.equal(q, want.q0) and torch.equal(s[:, :nb], want.s0[:, :nb]) and bool((s[:, nb:] == 77).all())


@pytest.mark.parametrize("rows,cols", [(256, 384), (130, 700)])
def test_blocks_of_tiny_values_and_of_zeros(rows, cols):
    """Scale bytes of 0 beside ordinary ones, along both axes, in whole tiles and at the ends."""
    mx = _mx()
    gate, up, _ = _data(rows, cols, F32)
    gate = gate.clamp(min=-5)
    for k, scale in ((0, 2.0 ** -119), (1, 0.0), (2, 2.0 ** -126)):
        up[:, 128 * k:128 * k + 100] *= scale
    up[rows // 2], up[3, ::2] = 0.0, 2.0 ** -149
    announce("gate tiny", rows, cols)
    o = mx.swiglu_forward(gate.cuda(), up.cuda(), axis="both", out_dtype=F32)
    check_axes(o, o.a.cpu(), "both")
    exact = gate_forward(gate, up)
    assert_within(o.a, exact, _own(gate) * exact.abs() + 2.0 ** -149)
    assert bool((o.s0[:, 0] == 0).any()) and bool((o.s0[:, 0] > 0).any())


def test_empty():
    mx = _mx()
    for shape in ((0, 300), (5, 0)):
        z = torch.zeros(*shape, dtype=BF).cuda()
        o = mx.swiglu_forward(z, z, axis="both")
        assert o.a.shape == shape
        mx.swiglu_backward(z, z, z, axis="both", joined=False)
        d = mx.swiglu_backward(z, z, z, axis=0)
        assert d.q0.shape == (2 * shape[1], 0 if shape[0] == 0 else 128)
    z = torch.zeros(0, 256, dtype=BF).cuda()
    assert mx.swiglu_backward(z, z, z, axis="both").q1.shape == (0, 512)


def test_ends_of_the_range():
    """Gates from far below to far above zero, infinities and NaN."""
    mx = _mx()
    gate = torch.cat([torch.linspace(-130, 130, 2048), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 2e38, -2e38, 80.0, -80.0])])[None]
    up = torch.ones_like(gate) * 1.5
    exact = gate_forward(gate, up)
    announce("gate ends")
    o = mx.swiglu_forward(gate.cuda(), up.cuda(), out_dtype=F32)
    # exp(-|g|) that is lost at its end is below 2^-126: times |g u|
    lost = 2.0 ** -126 * (gate.double() * up.double()).abs()
    assert_within(o.a, exact, _own(gate) * exact.abs() + lost + 2.0 ** -149)
    da = torch.full_like(gate, 0.75)
    dg, du, basis = gate_backward(da, gate, up)
    b = mx.swiglu_backward(da.cuda(), gate.cuda(), up.cuda(), out_dtype=F32)
    assert_within(b.dgate, dg, _own(gate) * basis + lost + 2.0 ** -126 + 2.0 ** -149)
    assert_within(b.dup, du, _own(gate) * du.abs() + lost + 2.0 ** -149)
    inf, nan = float("inf"), float("nan")
    gate, up = torch.tensor([[inf, nan, 1.0, 1.0, 2.0]]), torch.tensor([[1.0, 1.0, inf, nan, 3.0]])
    a = mx.swiglu_forward(gate.cuda(), up.cuda(), axis="both", out_dtype=F32)
    assert float(a.a[0, 0]) == inf and float(a.a[0, 2]) == inf and bool(torch.isnan(a.a[0, 1])) and bool(torch.isnan(a.a[0, 3]))
    assert int(a.s1[0, 0]) == 255 and a.s0[:5, 0].cpu().tolist()[:4] == [255] * 4 and int(a.s0[4, 0]) != 255
    assert not bool(a.q1.any())


def test_backward_against_differences():
    mx = _mx()
    g = torch.Generator().manual_seed(3)
    r = lambda: torch.randn(40, 100, generator=g).cuda()  # noqa: E731
    gate, up, c = 2 * r(), r(), r()
    value = lambda p, q: float((mx.swiglu_forward(p, q, out_dtype=F32).a.double() * c.double()).sum())  # noqa: E731
    got = mx.swiglu_backward(c, gate, up, out_dtype=F32)
    step = 2.0 ** -7
    for _ in range(4):
        p, q = r(), r()
        slope = (value(gate + step * p, up + step * q) - value(gate - step * p, up - step * q)) / (2 * step)
        want = float((got.dgate.double() * p.double()).sum() + (got.dup.double() * q.double()).sum())
        # 4000 outputs of about two, each off by 2^-19 (in the root mean square far less), over 2 step; third
        # derivatives of silu are at most one half: 4000 random terms of that size, times step^2 / 6
        assert abs(slope - want) <= 4000 * 2.0 ** -19 / (2 * step) + 10 * 4000 ** 0.5 * step ** 2 / 6
