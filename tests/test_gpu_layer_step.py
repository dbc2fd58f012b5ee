"""The operators between the products together with the products, as a step of a feed-forward block uses them: norm with the
residual's addition, fused gate-and-up product in 8 bits, gated activation, down product, the head's loss, all gradients, their
clipping and the update."""
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, HALF, U, assert_within, check_axes, gate_backward, gate_forward, norm_grad, norm_stream, norm_y32
from tests.test_gpu_fp8 import _bound

pytestmark = pytest.mark.gpu
T, K, F, V = 384, 256, 384, 700
EPS, LR, TOP = 1e-5, 0.02, 0.05


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _start(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    target = torch.randint(0, V, (T,), generator=g)
    target[::7] = -100
    return dict(x=r(T, K).to(BF), res=(2 * r(T, K)).to(BF), gain=(1 + 0.1 * r(K)).to(BF), last=(1 + 0.1 * r(K)).to(BF),
                w_gu=(r(2 * F, K) / K ** 0.5).to(BF), w_d=(r(K, F) / F ** 0.5).to(BF), head=(r(V, K) / K ** 0.5).to(BF), target=target)


def _nb(length):
    return (length + 127) // 128


def _step(s, stream=None):
    """One step on the tensors of s; the weights are updated in place. Everything it made on the way."""
    mx, o = _mx(), {}
    at = dict(stream=stream)
    n = mx.rmsnorm_forward(s["x"], s["gain"], s["res"], EPS, axis="both", y_dtype=None, **at)
    w1, s1, w0, s0 = mx.fp8_quantize(s["w_gu"], axis="both", block="tile", **at)
    gu = mx.fp8_gemm(n.q1, n.s1, w1, s1, out_dtype=BF, k=K, **at)
    a = mx.swiglu_forward(gu[:, :F], gu[:, F:], axis="both", out_dtype=None, **at)
    d1, t1, d0, t0 = mx.fp8_quantize(s["w_d"], axis="both", block="tile", **at)
    out = mx.fp8_gemm(a.q1, a.s1, d1, t1, out_dtype=BF, k=F, **at)
    f = mx.rmsnorm_forward(out, s["last"], n.h, EPS, **at)
    loss, lse = mx.linear_xent_forward(f.y, s["head"], s["target"], **at)
    valid = s["target"] != -100
    dloss = valid.float() / valid.sum()
    df, o["d_head"] = mx.linear_xent_backward(dloss, f.y, s["head"], s["target"], lse, dw_dtype=F32, **at)
    b = mx.rmsnorm_backward(df, f.h, f.rstd, s["last"], **at)
    o["d_last"] = b.dweight
    # the branch's gradient is the stream's
    y1, u1, y0, u0 = mx.fp8_quantize(b.dh, axis="both", **at)
    da = mx.fp8_gemm(y1, u1, d0, t0, out_dtype=BF, k=K, **at)
    o["d_wd"] = mx.fp8_gemm(y0, u0, a.q0, a.s0, k=T, **at)
    g = mx.swiglu_backward(da, gu[:, :F], gu[:, F:], axis="both", out_dtype=None, **at)
    dn = mx.fp8_gemm(g.q1, g.s1, w0, s0, out_dtype=BF, k=2 * F, **at)
    o["d_gu"] = mx.fp8_gemm(g.q0, g.s0, n.q0, n.s0, k=T, **at)
    c = mx.rmsnorm_backward(dn, n.h, n.rstd, s["gain"], dres=b.dh, **at)
    o["d_gain"] = c.dweight
    grads = [o["d_gu"], o["d_wd"], o["d_head"], o["d_gain"], o["d_last"]]
    o["raw"] = [t.clone() for t in grads]
    o["norm"] = mx.grad_clip(grads, TOP, **at)
    for w, d in ((s["w_gu"], "d_gu"), (s["w_d"], "d_wd")):
        mx.orthogonalize(o[d], alpha=-LR, beta=1.0, out=w, **at)
    # the gains' gradient steps: scaled into bf16 straight from the FP32 sums
    o["step"] = [torch.empty_like(s["gain"]), torch.empty_like(s["last"])]
    mx.grad_scale([o["d_gain"], o["d_last"]], torch.ones((), dtype=torch.float64, device=s["x"].device), 0.5, eps=0.0, out=o["step"], **at)
    o.update(h=n.h, rstd=n.rstd, gu=gu, out=out, y=f.y, h2=f.h, rstd2=f.rstd, loss=loss, lse=lse, df=df, dh2=b.dh, da=da, dn=dn, dx=c.dh,
             q1=n.q1, s1=n.s1[:, :_nb(K)], q0=n.q0, s0=n.s0[:, :_nb(T)], aq1=a.q1, as1=a.s1[:, :_nb(F)], aq0=a.q0, as0=a.s0[:, :_nb(T)],
             gq1=g.q1, gs1=g.s1[:, :_nb(2 * F)], gq0=g.q0, gs0=g.s0[:, :_nb(T)])
    return o


def _flat(o):
    return [t for k in sorted(o) for t in (o[k] if isinstance(o[k], list) else [o[k]])]


def _on_gpu(s):
    return {k: v.cuda() for k, v in s.items()}


def _values(q, s):
    return torch.from_numpy(ref.values(q.cpu().numpy(), s.cpu().numpy()))


def _codes_of(t, tile=False):
    return ref.values(*ref.quantize(t.cpu().double().numpy(), tile))


class _Eight:
    def __init__(self, o, p):
        self.q1, self.s1, self.q0, self.s0 = (o[p + k] for k in ("q1", "s1", "q0", "s0"))


def test_each_part_on_what_the_others_made():
    announce("layer step")
    before = _start()
    s = _on_gpu(before)
    o = {k: [t.cpu() for t in v] if isinstance(v, list) else v.cpu() for k, v in _step(s).items()}
    # the norm, its codes, and the products of them
    h = norm_stream(before["x"], before["res"])
    assert torch.equal(o["h"], h)
    check_axes(_Eight(o, ""), norm_y32(h, o["rstd"], before["gain"]), "both")

    def product(got, A, B, what):
        exact = torch.from_numpy(A @ B.T)
        tol = torch.from_numpy(1.01 * _bound(A, B))
        assert_within(got, exact, tol + HALF[got.dtype] * exact.abs(), what)
    A, W = _codes_of(norm_y32(h, o["rstd"], before["gain"])), _codes_of(before["w_gu"], True)
    product(o["gu"], A, W, "gate and up")
    # the activation: values of codes, which are within half a step (2^-4) of the formula's; a block's smallest codes have
    # steps of 2^-9 of its scale, a 448th of the block's maximum or less
    gate, up = o["gu"][:, :F], o["gu"][:, F:]
    exact = gate_forward(gate, up)
    got = _values(o["aq1"], o["as1"])
    top = exact.abs().reshape(T, -1, 128).amax(dim=2, keepdim=True).expand(-1, -1, 128).reshape(T, F)
    assert_within(got, exact, exact.abs() * (2.0 ** -4 + 2.0 ** -18) + top * 2.0 ** -10 / 224)
    product(o["out"], got.numpy(), _codes_of(before["w_d"], True), "down")
    f32 = norm_y32(o["h2"], o["rstd2"], before["last"])
    assert torch.equal(o["h2"], norm_stream(o["out"], h)) and torch.equal(o["y"], f32.to(BF))
    # gradients
    dh, dw, tol, tol_w = norm_grad(o["df"], o["h2"], o["rstd2"], before["last"], None)
    assert_within(o["dh2"], dh, tol + HALF[BF] * dh.abs(), "dh")
    assert_within(o["raw"][4], dw, tol_w + U * dw.abs(), "d_last")
    da, dg, du = o["da"], *gate_backward(o["da"], gate, up)[:2]
    exact = torch.cat([dg, du], dim=1)
    basis = torch.cat([gate_backward(da, gate, up)[2], du.abs()], dim=1)
    got = _values(o["gq1"], o["gs1"])
    top = exact.abs().reshape(T, -1, 128).amax(dim=2, keepdim=True).expand(-1, -1, 128).reshape(T, 2 * F)
    assert_within(got, exact, exact.abs() * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -19 * basis + top * 2.0 ** -10 / 224)
    product(o["raw"][0], _values(o["gq0"], o["gs0"]).numpy(), _values(o["q0"], o["s0"]).numpy(), "d_gu")
    dx, dw, tol, tol_w = norm_grad(o["dn"], h, o["rstd"], before["gain"], o["dh2"])
    assert_within(o["dx"], dx, tol + HALF[BF] * (dx.abs() + tol), "dx")
    assert_within(o["raw"][3], dw, tol_w + U * dw.abs(), "d_gain")
    # clipping
    n = sum(float(t.double().square().sum()) for t in o["raw"]) ** 0.5
    assert abs(float(o["norm"]) - n) <= n * U * 1.0001 and n > TOP
    for raw, d in zip(o["raw"], ("d_gu", "d_wd", "d_head", "d_gain", "d_last")):
        exact = raw.double() * (TOP / (n + 1e-6))
        assert_within(o[d], exact, exact.abs() * 2.01 * U + 2.0 ** -149, d)
    for d, step in zip(("d_gain", "d_last"), o["step"]):
        assert torch.equal(step, (o[d] * 0.5).to(BF))


def test_again_on_other_streams_at_once_and_replayed():
    """The same step gives the same bits: twice at once on two streams, and captured and replayed, each time from other
    weights, with eager steps between the replays."""
    announce("layer step: streams")
    s0 = _on_gpu(_start())
    o0 = _step(s0)
    a, b = _on_gpu(_start()), _on_gpu(_start())
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for side, s in zip(sides, (a, b)):
        with torch.cuda.stream(side):
            outs.append(_step(s))
    torch.cuda.synchronize()
    same = lambda p, q: all(torch.equal(x, y) for x, y in zip(_flat(p), _flat(q)))  # noqa: E731
    for s, o in ((a, outs[0]), (b, outs[1])):
        assert same(o, o0) and same(s, s0)
    announce("layer step: graph")
    held = _on_gpu(_start())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = _step(held)
    for seed in (0, 5, 6, 0):
        new = _start(seed)
        for k in held:
            held[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        eager = _on_gpu(new)
        o = _step(eager)
        assert same(made, o) and same(held, eager)


def test_a_stream_that_is_given():
    mx = _mx()
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(300, 256, generator=g).to(BF).cuda()
    torch.cuda.synchronize()
    o = mx.rmsnorm_forward(x, axis="both", stream=side)
    p = mx.swiglu_forward(x, x, axis="both", stream=side.cuda_stream)
    n = mx.grad_norm([x], stream=side)[1]
    side.synchronize()
    a, b, c = mx.rmsnorm_forward(x, axis="both"), mx.swiglu_forward(x, x, axis="both"), mx.grad_norm([x])[1]
    assert torch.equal(o.y, a.y) and torch.equal(o.q0, a.q0) and torch.equal(p.a, b.a) and torch.equal(p.q1, b.q1) and torch.equal(n, c)
