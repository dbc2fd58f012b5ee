"""The binding of libmxfp4_layer without a GPU: what layer.py hands to the library, seen by a library that only records it,
and what it refuses by itself."""
import contextlib

import pytest
import torch

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class Recorder:
    """Stands in for the library: every call succeeds and is kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *sizes: 4096
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def recorded(monkeypatch):
    import mxfp4_block_scaled_h16_amd.layer as layer
    lib = Recorder()
    monkeypatch.setattr(layer, "layer_lib", lambda: lib)
    monkeypatch.setattr(layer, "_same_device", lambda **tensors: torch.device("cpu"))      # what a CPU tensor's check ends in
    monkeypatch.setattr(layer, "_on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(layer, "_current", lambda: 0)
    layer.rmsnorm_backward_workspace_bytes.cache_clear()
    yield layer, lib
    layer.rmsnorm_backward_workspace_bytes.cache_clear()


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_norm_outputs(recorded):
    layer, lib = recorded
    x, r, w = _z(5, 200), _z(5, 200, dtype=F32), _z(200)
    o = layer.rmsnorm_forward(x, w, residual=r, axis="both")
    assert o.h.dtype == F32 and o.y.dtype == BF and o.rstd.shape == (5,) and o.q1.shape == (5, 256) and o.q0.shape == (200, 128)
    assert o.s1.shape == (5, 16) and o.s0.shape == (200, 16)
    o = layer.rmsnorm_forward(x, w, y_dtype=None, axis=1)
    assert o.h is x and o.y is None and o.q0 is None
    assert layer.rmsnorm_forward(x, residual=r, need_h=False).h is None
    assert layer.rmsnorm_forward(x, residual=r, h=r).h is r
    g = layer.rmsnorm_backward(x, r, o.rstd, w, dres=r, dweight_dtype=BF)
    assert g.dh.dtype == F32 and g.dweight.dtype == BF
    assert layer.rmsnorm_backward(x, r, o.rstd, need_dweight=False).dweight is None
    assert len(lib.calls) == 6


def test_norm_refusals(recorded):
    layer, lib = recorded
    x, r, w = _z(5, 200), _z(5, 200, dtype=F32), _z(200)
    bad = [lambda: layer.rmsnorm_forward(x, h=r), lambda: layer.rmsnorm_forward(x, residual=r, h=x), lambda: layer.rmsnorm_forward(x, _z(199)),
           lambda: layer.rmsnorm_forward(x, _z(400)[::2]), lambda: layer.rmsnorm_forward(x, residual=_z(5, 201)),
           lambda: layer.rmsnorm_forward(x, axis=2), lambda: layer.rmsnorm_forward(x.t()), lambda: layer.rmsnorm_forward(x[0]),
           lambda: layer.rmsnorm_forward(x, residual=r, need_h=False, axis=0), lambda: layer.rmsnorm_forward(x, residual=r, need_h=False, h=r),
           lambda: layer.rmsnorm_forward(x, y_dtype=torch.float16), lambda: layer.rmsnorm_forward(x.half()),
           lambda: layer.rmsnorm_forward(x, w.half()), lambda: layer.rmsnorm_forward(x, y=_z(4, 200)),
           lambda: layer.rmsnorm_backward(x, r, _z(4, dtype=F32)), lambda: layer.rmsnorm_backward(x, r, _z(5)),
           lambda: layer.rmsnorm_backward(x, r, _z(5, dtype=F32), dres=x), lambda: layer.rmsnorm_backward(x, r, _z(5, dtype=F32), dh=x),
           lambda: layer.rmsnorm_backward(x, r, _z(5, dtype=F32), need_dweight=False, dweight=w),
           lambda: layer.rmsnorm_backward(x, r, _z(5, dtype=F32), workspace=_z(1, dtype=U8).expand(8192))]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    assert not lib.calls


def test_swiglu_outputs(recorded):
    layer, lib = recorded
    gu = _z(5, 512)
    g, u = gu[:, :256], gu[:, 256:]
    o = layer.swiglu_forward(g, u, axis="both", out_dtype=None)
    assert o.a is None and o.q1.shape == (5, 256) and o.q0.shape == (256, 128)
    assert lib.calls[-1][1][1] == 512                            # the halves' row stride
    d = layer.swiglu_backward(g, g, u, axis="both")
    assert d.q1.shape == (5, 512) and d.q0.shape == (512, 128) and d.dgate.data_ptr() + 512 == d.dup.data_ptr() and d.gate is None
    args = lib.calls[-1][1]
    at = args.index(d.q1.data_ptr())
    assert args[at:at + 6] == (d.q1.data_ptr(), d.q1.data_ptr() + 256, 512, d.s1.data_ptr(), d.s1.data_ptr() + 2, 16)
    assert args[at + 6:at + 12] == (d.q0.data_ptr(), d.q0.data_ptr() + 256 * 128, 128, d.s0.data_ptr(), d.s0.data_ptr() + 256 * 16, 16)
    d = layer.swiglu_backward(_z(5, 200), _z(5, 200), _z(5, 200), axis="both", joined=False, out_dtype=None)
    assert d.dgate is None and d.q1 is None and d.gate.q1.shape == (5, 256) and d.up.q0.shape == (200, 128)
    d = layer.swiglu_backward(g, g, u, dgate=g, dup=u)
    assert d.dgate is g and d.dup is u


def test_swiglu_refusals(recorded):
    layer, lib = recorded
    g, u = _z(5, 200), _z(5, 200)
    bad = [lambda: layer.swiglu_forward(g, u.float()), lambda: layer.swiglu_forward(g, _z(5, 201)), lambda: layer.swiglu_forward(g, u, axis="rows"),
           lambda: layer.swiglu_forward(g, u, out_dtype=torch.float16), lambda: layer.swiglu_forward(g.half(), u.half()),
           lambda: layer.swiglu_forward(g, u, a=_z(6, 200)), lambda: layer.swiglu_backward(g, g, u, axis=1),
           lambda: layer.swiglu_backward(g, g, u, dgate=g), lambda: layer.swiglu_backward(g, g, u, dgate=g, dup=u.float()),
           lambda: layer.swiglu_backward(_z(4, 200), g, u), lambda: layer.swiglu_backward(g, g, u.float())]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    assert not lib.calls


class OnDevice(torch.Tensor):
    """A tensor that says it lies on device 0, for checks that come before the library."""
    is_cuda = True

    def get_device(self):
        return 0


def _grad(*shape, dtype=F32):
    return _z(*shape, dtype=dtype).as_subclass(OnDevice)


def test_gradients_as_the_library_takes_them(recorded):
    layer, lib = recorded
    a, b, c = _grad(3, 5), _grad(7, dtype=BF), _grad(4, 6).t()
    _, items, n = layer._grads([a, b, c], None)
    assert n == 3 and list(items) == [a.data_ptr(), a.data_ptr(), 15, 1, b.data_ptr(), b.data_ptr(), 7, 1 << 32, c.data_ptr(), c.data_ptr(),
                                      24, 1]
    out = _grad(3, 5, dtype=BF)
    _, items, n = layer._grads(a, out)
    assert n == 1 and list(items) == [a.data_ptr(), out.data_ptr(), 15, 1 | 1 << 32]
    for t in (_grad(4, 6)[:, :3], _grad(8)[::2], _grad(1).expand(4), _grad(3, 1).expand(3, 4)):
        with pytest.raises(ValueError):
            layer._grads([t], None)
    _, items, n = layer._grads([a], [_grad(15)])                 # part of a flat buffer
    assert n == 1 and items[2] == 15
    for g, o in ((a, _grad(16)), (c, _grad(6, 4)), (c, _grad(24)), (a, _grad(5, 3).t())):
        with pytest.raises(ValueError):
            layer._grads([g], [o])
    for t in (_grad(4).half(), _grad(4).double()):
        with pytest.raises(TypeError):
            layer._grads([t], None)
    assert layer._dense(_grad(2, 3, 4).permute(2, 0, 1)) and layer._dense(_grad(5, 1, 3)[:, :, :]) and layer._dense(_grad(0, 3))
