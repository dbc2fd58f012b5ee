"""The training operators together, as a step uses them: an FP8 layer, an MXFP4 layer, the head's loss and its gradients, the
layers' gradients, and the orthogonalized update of each weight."""
import numpy as np
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu
from tests.test_gpu_fp8 import _bound
from tests.test_gpu_orthogonalize import BF16, COEFFS, OWN

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, K, H, V = 384, 256, 320, 1111
LR = 0.02


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
    return dict(x=r(T, K).to(BF), w1=(r(H, K) / K ** 0.5).to(BF), w2=(r(H, H) / H ** 0.5).to(BF), w3=(r(V, H) / H ** 0.5).to(BF),
                target=target)


def _step(s, stream=None):
    """One step on the tensors of s; the weights are updated in place. Everything it made on the way."""
    mx = _mx()
    o = {}
    o["h1"] = mx.fp8_linear_fprop(s["x"], s["w1"], out_dtype=BF, stream=stream)
    o["h2"] = mx.linear_fprop(o["h1"], s["w2"], stream=stream).to(BF)
    o["loss"], o["lse"] = mx.linear_xent_forward(o["h2"], s["w3"], s["target"], stream=stream)
    o["dloss"] = (s["target"] != -100).float() / (s["target"] != -100).sum()
    o["dh2"], o["dw3"] = mx.linear_xent_backward(o["dloss"], o["h2"], s["w3"], s["target"], o["lse"], stream=stream)
    o["dh1"] = mx.linear_dgrad(o["dh2"], s["w2"], stream=stream).to(BF)
    o["dw2"] = mx.linear_wgrad(o["dh2"], o["h1"], stream=stream)
    o["dx"] = mx.fp8_linear_dgrad(o["dh1"], s["w1"], stream=stream)
    o["dw1"] = mx.fp8_linear_wgrad(o["dh1"], s["x"], stream=stream)
    for w, d in (("w1", "dw1"), ("w2", "dw2"), ("w3", "dw3")):
        mx.orthogonalize(o[d], alpha=-LR, beta=1.0, out=s[w], stream=stream)
    return o


def _on_gpu(s):
    return {k: v.cuda() for k, v in s.items()}


def _codes(t, axis=1, tile=False):
    t = t.cpu().double().numpy()
    return ref.values(*ref.quantize(np.ascontiguousarray(t if axis else t.T), tile))


def test_each_part_on_what_the_others_made():
    announce("train step")
    before = _start()
    s = _on_gpu(before)
    o = _step(s)
    cpu = {k: v.cpu() for k, v in o.items()}
    half = 2.0 ** -8                                 # a bf16 result's rounding

    def close(got, exact, tol):
        assert bool((np.abs(got.double().numpy() - exact) <= tol).all())

    A, B = _codes(before["x"]), _codes(before["w1"], tile=True)
    close(cpu["h1"], A @ B.T, 1.01 * _bound(A, B) + half * np.abs(A @ B.T))
    A, B = _codes(o["dh1"]), _codes(before["w1"], axis=0, tile=True)
    close(cpu["dx"], A @ B.T, _bound(A, B))
    A, B = _codes(o["dh1"], axis=0), _codes(before["x"], axis=0)
    close(cpu["dw1"], A @ B.T, _bound(A, B))
    loss, lse, dx, dw, g, _ = ref.xent(cpu["h2"], before["w3"], before["target"], -100, cpu["dloss"], None)
    # logits of some 1000 products each, well within 2^-14; G to 11 bits, then the outputs' rounding
    assert float((cpu["loss"].double() - loss).abs().max()) < 2.0 ** -14 and float((cpu["lse"].double() - lse).abs().max()) < 2.0 ** -14
    for got, want in ((cpu["dh2"], dx), (cpu["dw3"], dw)):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8 + 2.0 ** -11
    for w, d in (("w1", "dw1"), ("w2", "dw2"), ("w3", "dw3")):
        update = LR * ref.newton_schulz(cpu[d], 5, COEFFS, 1e-7)
        off = s[w].cpu().double() - (before[w].double() - update)
        # the update's own error, and one rounding of the new weight
        assert float(off.norm()) <= OWN * float(update.norm()) + BF16 * float(s[w].cpu().double().norm())


def test_again_on_another_stream_beside_one_and_replayed():
    """The same step gives the same bits: twice at once on two streams, and captured and replayed, each time from
    other weights."""
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
    for s, o in ((a, outs[0]), (b, outs[1])):
        assert all(torch.equal(o[k], o0[k]) for k in o0) and all(torch.equal(s[k], s0[k]) for k in s0)
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
        assert all(torch.equal(made[k], o[k]) for k in o) and all(torch.equal(held[k], eager[k]) for k in eager)
