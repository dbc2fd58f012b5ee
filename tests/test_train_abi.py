"""libmxfp4_train.so without a GPU: it loads, exports what include/mxfp4_train.h declares, sizes its
workspaces, and refuses invalid calls before any HIP call (no call here reaches a launch)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxfp4_train.h")
NULL, SHAPE, ARG, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
P = 1 << 12          # a pointer that is never followed: every call fails its host-side checks
BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    import mxfp4_block_scaled_h16_amd as mx
    return mx.train_lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp4_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 14
    for name in names:
        assert hasattr(L, name), name
    assert L.mxfp4_train_abi_version() == 1


def test_package_exposes_them():
    import mxfp4_block_scaled_h16_amd as mx
    for name in ("fp8_quantize", "fp8_gemm", "fp8_linear_fprop", "fp8_linear_dgrad", "fp8_linear_wgrad", "linear_xent_forward",
                 "linear_xent_backward", "orthogonalize"):
        assert name in mx.__all__ and callable(getattr(mx, name))


def _quantize(L, x=P, dtype=0, rows=64, cols=200, ldx=200, block=0, q1=P, ldq1=256, s1=P, lds1=2, q0=None, ldq0=0, s0=None,
              lds0=0):
    return L.mxfp4_fp8_quantize(x, dtype, rows, cols, ldx, block, q1, ldq1, s1, lds1, q0, ldq0, s0, lds0, None)


@pytest.mark.parametrize("want,change", [
    (ARG, dict(dtype=2)), (ARG, dict(block=2)), (ARG, dict(block=-1)), (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=1 << 31)),
    (SHAPE, dict(rows=1 << 30, cols=1 << 30, ldx=1 << 30)), (ARG, dict(ldx=199)), (NULL, dict(x=None)), (NULL, dict(q1=None)),
    (NULL, dict(s1=None)), (ARG, dict(ldq1=200)), (ARG, dict(lds1=1)), (ALIGN, dict(ldq1=264)), (ALIGN, dict(q1=P + 8)),
    (ALIGN, dict(x=P + 1)), (ALIGN, dict(x=P + 2, dtype=1)), (ARG, dict(q0=P, ldq0=64, s0=P, lds0=1)),
    (NULL, dict(q0=P, ldq0=128, lds0=1)), (0, dict(rows=0, x=None, q1=None)), (0, dict(cols=0, ldx=1, x=None, q1=None)),
])
def test_fp8_quantize_refusals(L, want, change):
    assert _quantize(L, **change) == want


def _gemm(L, aq=P, lda=256, as_=P, ldas=16, bq=P, ldb=256, bs=P, ldbs=16, M=5, N=7, K=200, beta=0.0, c=P, c_dtype=0, ldc=7,
          ws=None, n=0):
    return L.mxfp4_fp8_gemm(aq, lda, as_, ldas, bq, ldb, bs, ldbs, M, N, K, 1.0, beta, c, c_dtype, ldc, ws, n, None)


@pytest.mark.parametrize("want,change", [
    (SHAPE, dict(M=-1)), (SHAPE, dict(N=1 << 31)), (SHAPE, dict(K=-5)), (ARG, dict(lda=200)), (ARG, dict(ldb=128)),
    (ARG, dict(ldas=1)), (ALIGN, dict(lda=264)), (ALIGN, dict(ldbs=24)), (ARG, dict(ldc=6)), (ARG, dict(c_dtype=2)),
    (NULL, dict(aq=None)), (NULL, dict(bs=None)), (NULL, dict(c=None)), (ALIGN, dict(aq=P + 8)), (ALIGN, dict(as_=P + 1)),
    (ALIGN, dict(c=P + 2)), (ALIGN, dict(c=P + 1, c_dtype=1)), (ALIGN, dict(ws=P + 16, n=100)), (ARG, dict(lda=1 << 24)),
    (0, dict(M=0, aq=None)), (0, dict(N=0, ldc=1, c=None)),
])
def test_fp8_gemm_refusals(L, want, change):
    assert _gemm(L, **change) == want


@pytest.mark.parametrize("name", ["fprop", "dgrad", "wgrad"])
def test_fp8_linear_refusals(L, name):
    f = getattr(L, "mxfp4_fp8_linear_" + name)
    call = lambda a=P, b=P, M=32, K=64, N=96, ws=P, n=BIG, out=P, t=0: f(a, b, M, K, N, ws, n, out, t, None)  # noqa: E731
    assert call(M=-1) == SHAPE and call(K=(1 << 23) + 1) == SHAPE
    assert call(t=5) == ARG
    assert call(a=None) == NULL and call(b=None) == NULL and call(ws=None) == NULL and call(out=None) == NULL
    assert call(a=P + 1) == ALIGN and call(out=P + 2) == ALIGN and call(ws=P + 128) == ALIGN
    need = L.mxfp4_fp8_linear_workspace_bytes({"fprop": 0, "dgrad": 1, "wgrad": 2}[name], 32, 64, 96)
    assert need > 0 and call(n=need - 1) == WORKSPACE
    assert call(N=0, M=0, a=None, b=None, out=None) == 0
    for sizes in ((0, 64, 32), (64, 0, 32), (64, 32, 0), (0, 0, 0)):     # an empty product of every pass
        assert all(L.mxfp4_fp8_linear_workspace_bytes(p, *sizes) < 1 << 20 for p in range(3))
    assert L.mxfp4_fp8_linear_workspace_bytes(7, 32, 64, 96) == 0 and L.mxfp4_fp8_linear_workspace_bytes(0, -1, 64, 96) == 0


def _forward(L, x=P, ldx=64, w=P, ldw=64, target=P, T=5, K=64, V=100, ignore=-100, ws=P, n=BIG, loss=P, lse=P):
    return L.mxfp4_linear_xent_forward(x, ldx, w, ldw, target, T, K, V, ignore, ws, n, loss, lse, None)


def _backward(L, dloss=P, dlse=None, x=P, ldx=64, w=P, ldw=64, target=P, lse=P, T=5, K=64, V=100, ws=P, n=BIG, dx=P, dxt=1, dw=P,
              dwt=0):
    return L.mxfp4_linear_xent_backward(dloss, dlse, x, ldx, w, ldw, target, lse, T, K, V, -100, ws, n, dx, dxt, dw, dwt, None)


@pytest.mark.parametrize("want,change", [
    (SHAPE, dict(T=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(V=0)), (SHAPE, dict(V=1 << 31)), (SHAPE, dict(T=1 << 21)),
    (ARG, dict(ldx=63)), (ARG, dict(ldw=63)), (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(target=None)),
    (NULL, dict(ws=None)), (ALIGN, dict(x=P + 2)), (ALIGN, dict(ldw=65)), (ALIGN, dict(target=P + 4)), (ALIGN, dict(ws=P + 64)),
    (ALIGN, dict(K=33, x=P + 1)),
])
def test_xent_refusals(L, want, change):
    assert _forward(L, **change) == want
    assert _backward(L, **change) == want


def test_xent_outputs_and_workspaces(L):
    assert _forward(L, loss=None) == NULL and _forward(L, lse=None) == NULL and _forward(L, lse=P + 2) == ALIGN
    assert _backward(L, lse=None) == NULL and _backward(L, dloss=P + 2) == ALIGN
    assert _backward(L, dxt=2) == ARG and _backward(L, dwt=-1) == ARG
    assert _backward(L, dx=P + 1) == ALIGN and _backward(L, dw=P + 2) == ALIGN
    assert _forward(L, T=0) == 0 and _backward(L, T=0, dw=None) == 0 and _backward(L, dx=None, dw=None) == 0
    f, b = L.mxfp4_linear_xent_forward_workspace_bytes, L.mxfp4_linear_xent_backward_workspace_bytes
    assert _forward(L, n=f(5, 64, 100) - 1) == WORKSPACE and _backward(L, n=b(5, 64, 100) - 1) == WORKSPACE
    assert f(0, 64, 100) == 0 and f(5, -1, 100) == 0 and b(5, 64, 1 << 40) == 0
    # the logits are not kept: far less than T x V numbers
    assert f(8192, 4096, 128256) < 8192 * 128256 * 2 // 8 and b(8192, 4096, 128256) < 8192 * 128256


def _ortho(L, g=P, dtype=1, batch=1, m=20, n=30, ldg=30, bg=600, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, alpha=1.0,
           beta=0.0, out=P, t=1, ldo=30, bo=600, ws=P, nbytes=BIG):
    return L.mxfp4_orthogonalize(g, dtype, batch, m, n, ldg, bg, steps, a, b, c, eps, alpha, beta, out, t, ldo, bo, ws, nbytes, None)


@pytest.mark.parametrize("want,change", [
    (ARG, dict(dtype=3)), (ARG, dict(t=2)), (SHAPE, dict(m=-1)), (SHAPE, dict(n=(1 << 20) + 1)), (SHAPE, dict(batch=65536)),
    (SHAPE, dict(batch=60000, m=1000, n=1000)), (ARG, dict(steps=-1)), (ARG, dict(steps=33)), (ARG, dict(a=float("nan"))),
    (ARG, dict(a=40.0)), (ARG, dict(b=50.0)), (ARG, dict(c=float("inf"))), (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))),
    (ARG, dict(ldg=29)), (ARG, dict(ldo=29)), (ARG, dict(batch=2, bg=599)), (ARG, dict(batch=2, bo=599)), (NULL, dict(g=None)),
    (NULL, dict(out=None)), (NULL, dict(ws=None)), (ALIGN, dict(g=P + 2)), (ALIGN, dict(out=P + 1)), (ALIGN, dict(ws=P + 8)),
    (WORKSPACE, dict(nbytes=1000)), (0, dict(m=0)), (0, dict(batch=0)), (0, dict(n=0, ldg=1, ldo=1)),
])
def test_orthogonalize_refusals(L, want, change):
    assert _ortho(L, **change) == want


def test_orthogonalize_workspace(L):
    f = L.mxfp4_orthogonalize_workspace_bytes
    assert f(1, 20, 30) > 0 and f(0, 20, 30) == 0 and f(1, -1, 30) == 0 and f(2, 20, 30) > f(1, 20, 30)


def test_python_refusals():
    import torch
    import mxfp4_block_scaled_h16_amd as mx
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        mx.fp8_quantize(cpu)
    with pytest.raises(ValueError):
        mx.fp8_quantize(cpu, axis=2)
    with pytest.raises(ValueError):
        mx.fp8_quantize(cpu, block="rows")
    with pytest.raises(TypeError):
        mx.fp8_linear_fprop(cpu, cpu)
    with pytest.raises(ValueError):
        mx.fp8_linear_fprop(cpu, torch.zeros(4, 65, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mx.linear_xent_forward(cpu, cpu, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        mx.orthogonalize(cpu)
