"""The gated activation's products over FP32's whole range, on the GPU: the header's bounds where its brackets and the results are in FP32's
normal range, and nowhere else."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import F32, U, gate_backward, gate_forward

pytestmark = pytest.mark.gpu
LOW, HIGH = 2.0 ** -125, 2.0 ** 127          # the normal range, less a factor of two for the roundings


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _normal(*parts):
    ok = torch.ones_like(parts[0], dtype=torch.bool)
    for p in parts:
        ok &= (p.abs() >= LOW) & (p.abs() <= HIGH)
    return ok


def _check(got, exact, tol, where, what):
    assert float(where.double().mean()) > 0.1, what
    off = (got.cpu().double() - exact).abs()
    bad = where & ~(off <= tol)
    assert not bool(bad.any()), "%s: %d outside, worst %.3g of its tolerance" % (what, int(bad.sum()), float((off / tol)[where].max()))


def test_bounds_where_the_header_gives_them():
    mx = _mx()
    g = torch.Generator().manual_seed(4)
    gates = torch.cat([torch.linspace(-86, 86, 345), torch.tensor([1e-30, -1e-30, 1e-20, -1e-3, -1.2784, 1.2784])])
    exponents = torch.arange(-124.0, 127.0, 10.0)
    pairs = torch.cartesian_prod(exponents, exponents)
    gate = gates[:, None].expand(-1, len(pairs)).contiguous()
    # magnitudes of one to two, times every pair of powers
    up, da = (torch.exp2(pairs[:, k]) * (1 + torch.rand(gate.shape, generator=g)) * torch.where(torch.rand(gate.shape, generator=g) < 0.5, -1.0, 1.0)
              for k in (0, 1))
    s, t = torch.sigmoid(gate.double()), torch.sigmoid(-gate.double())
    announce("gate range", *gate.shape)
    a = mx.swiglu_forward(gate.cuda(), up.cuda(), out_dtype=F32).a
    exact = gate_forward(gate, up)
    f = gate.double() * s
    _check(a, exact, 2.0 ** -21 * exact.abs(), _normal(f, exact), "a")
    dg, du, basis = gate_backward(da, gate, up)
    o = mx.swiglu_backward(da.cuda(), gate.cuda(), up.cuda(), out_dtype=F32)
    _check(o.dup, du, 2.0 ** -21 * du.abs(), _normal(f, du), "dup")
    slope = s * (1 + gate.double() * t)
    inner, both = up.double() * slope, da.double() * up.double()
    where = _normal(slope, inner, dg)
    _check(o.dgate, dg, 2.0 ** -20 * basis, where, "dgate")
    # among them products da up that FP32 does not hold
    assert int((where & (both.abs() > 2.0 ** 130)).sum()) > 1000 and bool(torch.isfinite(o.dgate.cpu()[where]).all())


def test_beyond_them():
    """Brackets that overflow, or are below the normal range, as the header's order of products has them."""
    mx = _mx()
    gate, up, da = torch.tensor([[2.0, -60.0, -60.0]]), torch.tensor([[3.3e38, 1e-18, 1e-25]]), torch.tensor([[1e-3, 1e10, 1e10]])
    o = mx.swiglu_backward(da.cuda(), gate.cuda(), up.cuda(), out_dtype=F32)
    got = o.dgate.cpu().double()[0]
    assert float(got[0]) == float("inf")
    # up s (1 + gate (1 - s)) is 59 * 8.8e-27 * up: 5e-43 and less are rounded to multiples of 2^-149, then multiplied by da
    dg, _, basis = gate_backward(da, gate, up)
    assert bool(((got - dg[0]).abs() <= 2.0 ** -20 * basis[0] + 2.0 ** -150 * da[0].double() * (1 + U))[1:].all())
