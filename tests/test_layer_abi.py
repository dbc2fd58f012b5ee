"""libmxfp4_layer.so without a GPU: it loads, exports what include/mxfp4_layer.h declares, sizes its workspaces, and refuses
invalid calls before any HIP call (no call here reaches a launch)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxfp4_layer.h")
NULL, SHAPE, ARG, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
P = 1 << 12          # pointers that are never followed: every call fails its host-side checks
Q = 1 << 13
BIG = 1 << 62
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import mxfp4_block_scaled_h16_amd as mx
    return mx.layer_lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp4_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 10
    for name in names:
        assert hasattr(L, name), name
    version = re.search(r"MXFP4_LAYER_ABI_VERSION (\d+)", text)
    assert L.mxfp4_layer_abi_version() == int(version.group(1))


def test_package_exposes_them():
    import mxfp4_block_scaled_h16_amd as mx
    for name in ("rmsnorm_forward", "rmsnorm_backward", "swiglu_forward", "swiglu_backward", "grad_norm", "grad_scale", "grad_clip"):
        assert name in mx.__all__ and callable(getattr(mx, name))


def _norm(L, x=P, xt=0, ldx=200, r=P, ldr=200, st=0, w=P, wt=0, rows=64, cols=200, eps=1e-5, h=Q, ldh=200, rstd=P, y=P, yt=1, ldy=200,
          q1=None, ldq1=256, s1=P, lds1=2, q0=None, ldq0=128, s0=P, lds0=1):
    return L.mxfp4_rmsnorm_forward(x, xt, ldx, r, ldr, st, w, wt, rows, cols, eps, h, ldh, rstd, y, yt, ldy, q1, ldq1, s1, lds1, q0,
                                   ldq0, s0, lds0, None)


@pytest.mark.parametrize("want,change", [
    (ARG, dict(xt=2)), (ARG, dict(st=-1)), (ARG, dict(wt=3)), (ARG, dict(yt=2)), (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=0)),
    (SHAPE, dict(cols=(1 << 24) + 1)), (SHAPE, dict(rows=1 << 31)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=NAN)), (ARG, dict(eps=INF)),
    (ARG, dict(ldx=199)), (ARG, dict(ldr=199)), (ARG, dict(ldh=199)), (ARG, dict(ldy=199)), (ARG, dict(ldx=1 << 60)),
    (ARG, dict(r=None)), (NULL, dict(x=None)), (NULL, dict(q0=P, rstd=None)), (NULL, dict(q0=P, h=None)), (ALIGN, dict(x=P + 1)),
    (ALIGN, dict(x=P + 2, xt=1)), (ALIGN, dict(r=P + 1)), (ALIGN, dict(h=Q + 2, st=1)), (ALIGN, dict(rstd=P + 2)),
    (ALIGN, dict(y=P + 2, yt=0)), (ALIGN, dict(w=P + 1)), (ARG, dict(h=P, ldh=201)), (ARG, dict(x=Q, st=1)),
    (ARG, dict(x=Q, ldx=201)), (NULL, dict(q1=P, s1=None)), (ARG, dict(q1=P, ldq1=200)), (ALIGN, dict(q1=P + 8)),
    (ALIGN, dict(q1=P, ldq1=264)), (ARG, dict(q1=P, lds1=1)), (ARG, dict(q0=P, ldq0=64)), (ALIGN, dict(q0=P, ldq0=136)),
    (SHAPE, dict(q0=P, rows=1 << 30, cols=1 << 17, ldx=1 << 17, ldr=1 << 17, ldh=1 << 17, ldy=1 << 17)),
    (0, dict(rows=0, x=None)), (0, dict(r=None, h=None, rstd=None, y=None)),
])
def test_rmsnorm_forward_refusals(L, want, change):
    assert _norm(L, **change) == want


def _norm_grad(L, dy=P, dt=0, lddy=200, dres=P, lddr=200, h=P, ldh=200, st=0, w=P, wt=0, rstd=P, rows=64, cols=200, dh=Q, lddh=200,
               dw=P, dwt=0, ws=P, n=BIG):
    return L.mxfp4_rmsnorm_backward(dy, dt, lddy, dres, lddr, h, ldh, st, w, wt, rstd, rows, cols, dh, lddh, dw, dwt, ws, n, None)


@pytest.mark.parametrize("want,change", [
    (ARG, dict(dt=2)), (ARG, dict(st=2)), (ARG, dict(wt=2)), (ARG, dict(dwt=2)), (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=0)),
    (ARG, dict(lddy=199)), (ARG, dict(lddr=199)), (ARG, dict(ldh=199)), (ARG, dict(lddh=199)), (NULL, dict(dy=None)),
    (NULL, dict(h=None)), (NULL, dict(rstd=None)), (NULL, dict(dh=None)), (NULL, dict(ws=None)), (ALIGN, dict(dy=P + 1)),
    (ALIGN, dict(h=P + 2, st=1)), (ALIGN, dict(dh=Q + 1)), (ALIGN, dict(dres=P + 1)), (ALIGN, dict(rstd=P + 2)), (ALIGN, dict(w=P + 1)),
    (ALIGN, dict(dw=P + 2)), (ALIGN, dict(ws=P + 128)), (ARG, dict(dh=P, lddh=201)), (0, dict(rows=0, dw=None, dy=None)),
])
def test_rmsnorm_backward_refusals(L, want, change):
    assert _norm_grad(L, **change) == want


def test_rmsnorm_backward_workspace(L):
    f = L.mxfp4_rmsnorm_backward_workspace_bytes
    need = f(64, 200)
    assert need > 0 and _norm_grad(L, n=need - 1) == WORKSPACE
    assert f(0, 200) == 0 and f(-1, 200) == 0 and f(64, 0) == 0 and f(64, (1 << 24) + 1) == 0
    assert f(1 << 30, 4096) == f(1 << 20, 4096)                  # it does not grow with the rows
    assert f(8192, 4096) <= 16 << 20


def _gate(L, g=P, ldg=200, u=P, ldu=200, t=0, rows=64, cols=200, a=Q, at=1, lda=200, q1=None, ldq1=256, s1=P, lds1=2, q0=None, ldq0=128,
          s0=P, lds0=1):
    return L.mxfp4_swiglu_forward(g, ldg, u, ldu, t, rows, cols, a, at, lda, q1, ldq1, s1, lds1, q0, ldq0, s0, lds0, None)


@pytest.mark.parametrize("want,change", [
    (ARG, dict(t=2)), (ARG, dict(at=2)), (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=-1)), (SHAPE, dict(cols=1 << 31)),
    (SHAPE, dict(rows=1 << 30, cols=1 << 20)), (ARG, dict(ldg=199)), (ARG, dict(ldu=199)), (ARG, dict(lda=199)),
    (NULL, dict(g=None)), (NULL, dict(u=None)), (ALIGN, dict(g=P + 1)), (ALIGN, dict(u=P + 2, t=1)), (ALIGN, dict(a=Q + 2, at=0)),
    (ARG, dict(a=P, at=0)), (ARG, dict(a=P, lda=201)), (NULL, dict(q1=P, s1=None)), (ARG, dict(q0=P, lds0=0)),
    (ALIGN, dict(q0=P + 4)), (0, dict(rows=0, g=None)), (0, dict(cols=0, u=None)), (0, dict(a=None)),
])
def test_swiglu_forward_refusals(L, want, change):
    assert _gate(L, **change) == want


def _gate_grad(L, da=P, dt=0, ldda=200, g=P, ldg=200, u=P, ldu=200, t=0, rows=64, cols=200, dg=Q, lddg=200, du=2 * Q, lddu=200, ot=1,
               q1=(None, None), ldq1=256, s1=(P, P), lds1=2, q0=(None, None), ldq0=128, s0=(P, P), lds0=1):
    return L.mxfp4_swiglu_backward(da, dt, ldda, g, ldg, u, ldu, t, rows, cols, dg, lddg, du, lddu, ot, *q1, ldq1, *s1, lds1, *q0, ldq0,
                                   *s0, lds0, None)


@pytest.mark.parametrize("want,change", [
    (ARG, dict(dt=2)), (ARG, dict(t=-1)), (ARG, dict(ot=2)), (SHAPE, dict(rows=-1)), (SHAPE, dict(rows=1 << 30, cols=1 << 20)),
    (ARG, dict(ldda=1)), (ARG, dict(ldg=1)), (ARG, dict(ldu=1)), (ARG, dict(lddg=1)), (ARG, dict(lddu=1)), (NULL, dict(da=None)),
    (NULL, dict(g=None)), (NULL, dict(u=None)), (ALIGN, dict(da=P + 1)), (ALIGN, dict(dg=Q + 1)), (ALIGN, dict(du=Q + 2, ot=0)),
    (ARG, dict(dg=P, lddg=201)), (ARG, dict(dg=P, ot=0)), (ARG, dict(du=P, ot=0)), (ARG, dict(dg=Q, du=Q)),
    (NULL, dict(q1=(P, None), s1=(None, None))), (NULL, dict(q1=(None, P), s1=(P, None))), (ALIGN, dict(q0=(P, P + 8))),
    (ARG, dict(q0=(None, P), ldq0=64)), (0, dict(rows=0, da=None)), (0, dict(dg=None, du=None)),
])
def test_swiglu_backward_refusals(L, want, change):
    assert _gate_grad(L, **change) == want


class Grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


BF_IN, F32_IN, F32_OUT, BF_OUT = 0, 1, 0, 1


def _list(*items):
    a = (Grad * max(len(items), 1))()
    for k, (g, out, count, t, ot) in enumerate(items):
        a[k] = Grad(g, out, count, t, ot)
    return a


def _clip(L, items, n=None, top=1.0, eps=1e-6, ws=P, nbytes=BIG, norm=P):
    a = _list(*items)
    return L.mxfp4_grad_clip(ctypes.addressof(a), len(items) if n is None else n, top, eps, ws, nbytes, norm, None)


def _scale(L, items, sum_sq=P, top=1.0, eps=1e-6, norm=P):
    a = _list(*items)
    return L.mxfp4_grad_scale(ctypes.addressof(a), len(items), sum_sq, top, eps, norm, None)


A, B = 1 << 20, 1 << 24


@pytest.mark.parametrize("want,items", [
    (ARG, [(A, A, 10, 2, 0)]), (ARG, [(A, A, 10, 0, 2)]), (SHAPE, [(A, A, -1, 0, 1)]), (SHAPE, [(A, A, (1 << 37) + 1, 0, 1)]),
    (NULL, [(None, A, 10, 0, 1)]), (NULL, [(A, None, 10, 0, 1)]), (ALIGN, [(A + 1, B, 10, 0, 1)]), (ALIGN, [(A + 2, B, 10, 1, 0)]),
    (ALIGN, [(A, B + 2, 10, 0, 0)]),
    (ARG, [(A, A, 10, BF_IN, F32_OUT)]),                                                       # in place, another type
    (ARG, [(A, A, 10, BF_IN, BF_OUT)] * 2),                                                    # the same tensor twice
    (ARG, [(A, B, 10, BF_IN, BF_OUT)] * 2),                                                    # into the same output
    (ARG, [(A, A, 10, BF_IN, BF_OUT), (A + 18, A + 18, 10, BF_IN, BF_OUT)]),                    # an overlap by one value
    (ARG, [(A, A + 18, 10, BF_IN, BF_OUT)]), (ARG, [(A, A - 18, 10, BF_IN, BF_OUT)]),
    (ARG, [(A, B, 1000, F32_IN, F32_OUT), (B + 2000, 2 * B, 4, F32_IN, F32_OUT)]),               # an output inside another's input
    (ARG, [(A, B, 4, F32_IN, F32_OUT), (B - 2000, 2 * B, 1000, F32_IN, F32_OUT)]),
    (ARG, [(A, B, 4, F32_IN, F32_OUT), (A - 4000, 2 * B, 1000, F32_IN, F32_OUT), (2 * A, A - 16, 4, F32_IN, F32_OUT)]),
])
def test_grad_lists_refused(L, want, items):
    assert _clip(L, items) == want
    assert _scale(L, items) == want


def test_grad_refusals(L):
    ok = [(A, A, 10, BF_IN, BF_OUT), (A + 20, A + 20, 10, BF_IN, BF_OUT), (B, 2 * B, 7, F32_IN, BF_OUT), (None, None, 0, 0, 0)]
    for top in (0.0, -1.0, NAN, INF):
        assert _clip(L, ok, top=top) == ARG and _scale(L, ok, top=top) == ARG
    for eps in (-1.0, NAN, INF):
        assert _clip(L, ok, eps=eps) == ARG and _scale(L, ok, eps=eps) == ARG
    assert _clip(L, ok, ws=None) == NULL and _clip(L, ok, ws=P + 64) == ALIGN and _clip(L, ok, norm=P + 2) == ALIGN
    assert _scale(L, ok, sum_sq=None) == NULL and _scale(L, ok, sum_sq=P + 4) == ALIGN
    assert _clip(L, ok, n=-1) == SHAPE and _clip(L, ok, n=1 << 20) == SHAPE
    assert L.mxfp4_grad_clip(None, 1, 1.0, 0.0, P, BIG, P, None) == NULL
    a = _list(*ok)
    need = L.mxfp4_grad_norm_workspace_bytes(ctypes.addressof(a), 4)
    assert need > 0 and _clip(L, ok, nbytes=need - 1) == WORKSPACE
    at = ctypes.addressof(a)
    assert L.mxfp4_grad_norm(at, 4, P, need - 1, P, P, None) == WORKSPACE
    assert L.mxfp4_grad_norm(at, 4, None, need, P, P, None) == NULL
    assert L.mxfp4_grad_norm(at, 4, P, need, P + 4, P, None) == ALIGN and L.mxfp4_grad_norm(at, 4, P, need, P, P + 2, None) == ALIGN
    assert L.mxfp4_grad_norm(at, 4, P, need, None, None, None) == 0
    assert L.mxfp4_grad_norm_workspace_bytes(None, 4) == 0 and L.mxfp4_grad_norm_workspace_bytes(at, -1) == 0
    # nothing to do
    assert _clip(L, [], norm=None) == 0 and _scale(L, [(None, None, 0, 0, 0)], norm=None) == 0


def test_grad_workspace_is_small(L):
    """A few words a workgroup, whatever the tensors' sizes: at most 4 KB for each 128 of them."""
    f = L.mxfp4_grad_norm_workspace_bytes
    a = _list(*[(A, A, 1 << 37, 0, 1)] * 300)
    assert f(ctypes.addressof(a), 300) <= 3 * 4096 + 8
    assert f(ctypes.addressof(a), 1) <= 4096 + 8


def test_python_refusals():
    import torch
    import mxfp4_block_scaled_h16_amd as mx
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: mx.rmsnorm_forward(cpu), lambda: mx.rmsnorm_backward(cpu, cpu, torch.zeros(4)), lambda: mx.swiglu_forward(cpu, cpu),
                 lambda: mx.swiglu_backward(cpu, cpu, cpu), lambda: mx.grad_norm([cpu]), lambda: mx.grad_clip([cpu], 1.0),
                 lambda: mx.grad_scale([cpu], torch.zeros((), dtype=torch.float64), 1.0), lambda: mx.grad_clip([None], 1.0)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mx.grad_clip([], 1.0), lambda: mx.grad_clip([cpu], 1.0, out=[cpu, cpu])):
        with pytest.raises(ValueError):
            call()
