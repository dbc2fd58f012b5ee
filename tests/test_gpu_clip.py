"""The norm over many gradients and their clipping on the GPU, against 64 bits."""
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


def _grads(counts, dtypes, seed=0):
    return [heavy((n,), seed + k, 1e-3 * (1 + k % 3)).to(dtypes[k % len(dtypes)]) for k, n in enumerate(counts)]


def _norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


LISTS = [[1], [7], [8192], [8193, 1, 16384], [0, 5, 0, 3], [100000, 3, 20001, 1 << 20], [1 + 37 * k % 9000 for k in range(128)],
         [1 + 53 * k % 3000 for k in range(129)], [1 + 4099 * k % 25000 for k in range(161)], [8192 * (k % 3) + (k % 2) for k in range(230)], [5] * 700]


@pytest.mark.parametrize("counts", LISTS, ids=lambda c: "%d-%d" % (len(c), sum(c)))
@pytest.mark.parametrize("dtypes", [(BF,), (F32,), (BF, F32)])
@pytest.mark.parametrize("share", [0.5, 2.0])
def test_clip(counts, dtypes, share):
    mx = _mx()
    grads = _grads(counts, dtypes)
    n = _norm(grads)
    announce("clip", len(counts), sum(counts), dtypes, share)
    dev = [g.cuda() for g in grads]
    top = share * n
    c = min(1.0, top / (n + 1e-6))
    for out_dtype in (None, BF, F32):
        work = [g.clone() for g in dev]
        outs = None if out_dtype is None else [torch.full(g.shape, 7.0, dtype=out_dtype).cuda() for g in dev]
        norm = mx.grad_clip(work, top, out=outs)
        assert abs(float(norm) - n) <= n * U * 1.0001
        for g, w, o in zip(grads, work, outs or work):
            exact = g.double() * c
            # the factor, the product (the factor 1 is exact), and the last rounding
            assert_within(o, exact, exact.abs() * ((2.01 * U if c < 1.0 else 0.0) + (2.0 ** -8 if o.dtype == BF and c < 1.0 else 0.0)
                                                    + (2.0 ** -8 if o.dtype == BF and g.dtype == F32 else 0.0)) + 2.0 ** -149)
            assert outs is None or torch.equal(w.cpu(), g)
        # the halves give the same bits
        sum_sq, norm2 = mx.grad_norm(dev)
        assert torch.equal(norm2, norm) and abs(float(sum_sq) - n * n) <= n * n * 2.0 ** -40
        again = [g.clone() for g in dev]
        more = None if outs is None else [torch.empty_like(o) for o in outs]
        assert torch.equal(mx.grad_scale(again, sum_sq, top, out=more), norm)
        assert all(torch.equal(a, b) for a, b in zip(more or again, outs or work))


def test_sharded():
    """Ranks add up their sums of squares: the same factor as one call over all."""
    mx = _mx()
    grads = [g.cuda() for g in _grads([5000, 333, 20000, 7], (F32, BF))]
    parts = [grads[:1], grads[1:3], grads[3:]]
    total = sum(mx.grad_norm(p)[0] for p in parts)
    whole = [g.clone() for g in grads]
    norm = mx.grad_clip(whole, 0.01)
    for p in parts:
        assert abs(float(mx.grad_scale(p, total, 0.01)) - float(norm)) <= float(norm) * U
    for a, b in zip(grads, whole):
        assert_within(a, b.cpu(), b.cpu().double().abs() * (2 * U if a.dtype == F32 else 2.0 ** -7))


def test_views_and_orders():
    """Odd offsets inside one bucket (what lies between stays), transposed and permuted tensors."""
    mx = _mx()
    flat = heavy((5000,), 1).to(BF).cuda()
    want = flat.clone()
    views = [flat[1:8], flat[11:2060], flat[2060:2061], flat[2063:4990]]
    exact = [v.clone() for v in views]
    norm = mx.grad_clip(views, 0.25)
    n = _norm([v.cpu() for v in exact])
    assert abs(float(norm) - n) <= n * U * 1.0001
    at = torch.zeros(5000, dtype=torch.bool)
    for a, b in ((1, 8), (11, 2060), (2060, 2061), (2063, 4990)):
        at[a:b] = True
    assert torch.equal(flat.cpu()[~at], want.cpu()[~at]) and not torch.equal(flat, want)
    plain = [v.contiguous().clone() for v in exact]
    mx.grad_clip(plain, 0.25)
    assert all(torch.equal(a, b) for a, b in zip(views, plain))
    t = heavy((40, 60), 2).cuda()
    p = heavy((4, 5, 6), 3).cuda()
    a, b = t.t().clone(memory_format=torch.preserve_format), p.permute(2, 0, 1).clone(memory_format=torch.preserve_format)
    assert not a.is_contiguous() and not b.is_contiguous()
    mx.grad_clip([a, b], 1.0)
    c, d = t.clone(), p.clone()
    mx.grad_clip([c, d], 1.0)
    assert torch.equal(a, c.t()) and torch.equal(b, d.permute(2, 0, 1))
    out = torch.empty_like(a)
    mx.grad_clip([t.t()], 1.0, out=[out])
    c = t.clone()
    mx.grad_clip([c], 1.0)
    assert torch.equal(out, c.t())


def test_ends_of_the_range():
    mx = _mx()
    big, small = torch.full((1000,), 3.0e38), torch.full((1000,), 2.0 ** -140)
    for g in (big, small, torch.cat([big, small])):
        n = _norm([g])
        got = g.cuda()
        norm = mx.grad_clip([got], 1.0, eps=0.0)
        # a norm beyond FP32 is infinite as a result, but counts as it is
        assert float(norm) == math.inf if n > 3.4e38 else abs(float(norm) - n) <= n * U + 2.0 ** -150
        # the factor of 3e38 * sqrt(1000) lies below FP32's normal range, where a rounding is 2^-150
        c = min(1.0, 1.0 / n)
        assert_within(got, g.double() * c, g.double() * (c * 2.01 * U + (2.0 ** -150 if c < 1.0 else 0.0)) + 2.0 ** -149)
    bad = torch.tensor([1.0, math.inf, -2.0]).cuda()
    assert float(mx.grad_clip([bad], 1.0)) == math.inf
    assert bad.cpu().tolist()[0] == 0.0 and math.isnan(float(bad[1])) and float(bad[2]) == 0.0
    bad, other = torch.tensor([1.0, math.nan, -2.0]).cuda(), torch.ones(3, dtype=BF).cuda()
    assert math.isnan(float(mx.grad_clip([bad, other], 1.0))) and bool(torch.isnan(bad).all()) and bool(torch.isnan(other).all())
    zero = torch.zeros(5).cuda()
    assert float(mx.grad_clip([zero], 1.0, eps=0.0)) == 0.0 and not bool(zero.any())


def test_the_same_tensor_twice_is_refused():
    mx = _mx()
    g = torch.ones(100).cuda()
    with pytest.raises(mx.Mxfp4Error):
        mx.grad_clip([g, g], 1.0)
    with pytest.raises(mx.Mxfp4Error):
        mx.grad_clip([g, g[50:]], 1.0)
    with pytest.raises(mx.Mxfp4Error):
        mx.grad_clip([g[:50]], 1.0, out=[g[25:75]])
    assert bool((g == 1.0).all())


def test_no_write_where_nothing_is_clipped_and_results_repeat():
    mx = _mx()
    g = [t.cuda() for t in _grads([100000, 333], (F32,))]
    before = [t.clone() for t in g]
    norms = {float(mx.grad_clip(g, 1e6)) for _ in range(5)}
    assert len(norms) == 1 and all(torch.equal(a, b) for a, b in zip(g, before))


def test_many_values():
    """More pieces than workgroups, and a tensor of more than 2^31 bytes."""
    mx = _mx()
    g = torch.full(((1 << 30) + (1 << 20) + 3,), 2.0 ** -15, dtype=BF, device="cuda")
    g[-1] = 8.0
    announce("clip", g.numel())
    n = math.sqrt((g.numel() - 1) * 2.0 ** -30 + 64.0)
    assert abs(float(mx.grad_norm(g)[1]) - n) <= n * U * 1.0001
    norm = mx.grad_clip(g, n / 2, eps=0.0)
    assert abs(float(norm) - n) <= n * U * 1.0001
    assert bool((g[:-1] == 2.0 ** -16).all()) and float(g[-1]) == 4.0
