"""Calls of more than the last cache takes go past it, in kernels of their own: they give the bits that the same rows give in
calls of 1024 rows (whose results tests of their own hold to the formulas), at every way of working a row."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, U

pytestmark = pytest.mark.gpu
STEP = 1024                      # whole blocks along the columns


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _rand(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(dtype)


def _same_codes(o, part, at, rows, cols, q1, s1, q0, s0):
    """part's codes are those of rows at .. of o's."""
    n, nb = rows, (cols + 127) // 128
    assert torch.equal(part[0], q1[at:at + n]) and torch.equal(part[1][:, :nb], s1[at:at + n, :nb])
    wide = (n + 127) // 128
    assert torch.equal(part[2], q0[:, at:at + 128 * wide]) and torch.equal(part[3][:, :wide], s0[:, at // 128:at // 128 + wide])


@pytest.mark.parametrize("rows,cols,branch,stream", [(60001, 512, BF, BF), (30000, 1024, BF, BF), (15001, 2048, BF, F32), (6500, 4096, BF, BF),
                                                     (5100, 8192, F32, F32), (2300, 16384, F32, BF), (13000, 2056, BF, BF)])
def test_norm(rows, cols, branch, stream):
    mx = _mx()
    x, r = _rand(rows, cols, branch, 1), _rand(rows, cols, stream, 2, 3.0)
    w = 1 + _rand(1, cols, F32, 3, 0.2)[0]
    size = lambda t: 4 if t == F32 else 2  # noqa: E731
    assert rows * cols * (size(branch) + 2 * size(stream) + 2) > 192 << 20
    announce("norm large", rows, cols, branch, stream)
    o = mx.rmsnorm_forward(x, w, r, axis="both", y_dtype=None)
    grad = mx.rmsnorm_backward(x, o.h, o.rstd, w, dres=r)
    dw = torch.zeros(cols, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(dw)
    for at in range(0, rows, STEP):
        a, b = x[at:at + STEP], r[at:at + STEP]
        p = mx.rmsnorm_forward(a, w, b, axis="both", y_dtype=None)
        assert torch.equal(p.h, o.h[at:at + STEP]) and torch.equal(p.rstd, o.rstd[at:at + STEP])
        _same_codes(o, p[3:], at, a.shape[0], cols, *o[3:])
        assert torch.equal(mx.rmsnorm_backward(a, p.h, p.rstd, w, dres=b).dh, grad.dh[at:at + STEP])
        t = a.double() * p.h.double() * p.rstd.double()[:, None]
        dw += t.sum(dim=0)
        mass += t.abs().sum(dim=0)
    # two roundings for a product, one for each row that a thread adds, 64 to join them
    assert bool(((grad.dweight.double() - dw).abs() <= U * (68 + rows / 64) * mass).all())


@pytest.mark.parametrize("rows,cols,dtype,joined", [(4200, 8200, BF, True), (2700, 14336, BF, True), (5000, 5120, F32, False)])
def test_gate(rows, cols, dtype, joined):
    mx = _mx()
    if joined:
        both = _rand(rows, 2 * cols, dtype, 4, 1.5)
        gate, up = both[:, :cols], both[:, cols:]
    else:
        gate, up = _rand(rows, cols, dtype, 4, 1.5), _rand(rows, cols, dtype, 5)
    da = _rand(rows, cols, dtype, 6, 1e-3)
    assert rows * cols * (6 if dtype == BF else 10) > 192 << 20
    announce("gate large", rows, cols, dtype)
    o = mx.swiglu_forward(gate, up, axis="both")
    d = mx.swiglu_backward(da, gate, up, axis="both", joined=False)
    for at in range(0, rows, STEP):
        g, u = gate[at:at + STEP], up[at:at + STEP]
        p = mx.swiglu_forward(g, u, axis="both")
        assert torch.equal(p.a, o.a[at:at + STEP])
        _same_codes(o, p[1:], at, g.shape[0], cols, *o[1:])
        e = mx.swiglu_backward(da[at:at + STEP], g, u, axis="both", joined=False)
        assert torch.equal(e.dgate, d.dgate[at:at + STEP]) and torch.equal(e.dup, d.dup[at:at + STEP])
        _same_codes(d, e.gate, at, g.shape[0], cols, *d.gate)
        _same_codes(d, e.up, at, g.shape[0], cols, *d.up)


def test_offsets_beyond_32_bits():
    """Rows that start beyond 2^32 bytes, and values beyond 2^31: a narrow window of a wide matrix, and one tall matrix."""
    mx = _mx()
    wide = torch.zeros(300, 1 << 24, dtype=BF, device="cuda")            # 10 GB
    x = _rand(300, 384, BF, 7)
    view = wide[:, 5000:5384]
    view.copy_(x)
    announce("wide strides")
    a, b = mx.rmsnorm_forward(view, axis="both"), mx.rmsnorm_forward(x, axis="both")
    assert torch.equal(a.y, b.y) and torch.equal(a.q1, b.q1) and torch.equal(a.q0, b.q0)
    a, b = mx.swiglu_forward(view, view, axis="both"), mx.swiglu_forward(x, x, axis="both")
    assert torch.equal(a.a, b.a) and torch.equal(a.q1, b.q1) and torch.equal(a.q0, b.q0)
    rstd = mx.rmsnorm_forward(x).rstd
    grads = [mx.rmsnorm_backward(t, t, rstd, dres=t) for t in (view, x)]
    assert torch.equal(grads[0].dh, grads[1].dh) and torch.equal(grads[0].dweight, grads[1].dweight)
    out = wide[:, (1 << 24) - 384:]
    mx.swiglu_backward(view, view, view, dgate=out, dup=wide[:, 9000:9384])
    grad = mx.swiglu_backward(x, x, x)
    assert torch.equal(out, grad.dgate) and torch.equal(wide[:, 9000:9384], grad.dup)
    assert torch.equal(view, x) and not bool(wide[:, 9384:10000].any()) and not bool(wide[:, 4900:5000].any())
    del wide, view, out
    tall = torch.zeros((1 << 31) // 64 + 1000, 64, dtype=BF, device="cuda")
    tall[-700:] = _rand(700, 64, BF, 8)
    announce("tall")
    a, b = mx.rmsnorm_forward(tall, eps=1e-5, axis=1), mx.rmsnorm_forward(tall[-700:], eps=1e-5, axis=1)
    assert torch.equal(a.y[-700:], b.y) and torch.equal(a.q1[-700:], b.q1) and torch.equal(a.s1[-700:, :1], b.s1[:, :1])
    a, b = mx.swiglu_forward(tall, tall, axis="both"), mx.swiglu_forward(tall[-744:], tall[-744:], axis="both")
    assert torch.equal(a.a[-700:], b.a[-700:]) and torch.equal(a.q1[-700:], b.q1[-700:])
    first = tall.shape[0] - 744                                          # a whole number of blocks of 128 behind the start
    assert first % 128 == 0 and torch.equal(a.q0[:, first:], b.q0)
