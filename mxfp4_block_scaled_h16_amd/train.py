"""The operators of ``libmxfp4_train.so`` (C ABI in ``include/mxfp4_train.h``): 8-bit linear products,
the loss of a linear head, and the orthogonalised update. Like the rest of the package this is a
thin ctypes binding: the library's HIP kernels do every step.

Tensors may lie on any gfx950 device: a call runs on the device of its first tensor, all tensors of a
call on the same one, on `stream` (a torch.cuda.Stream of that device, or its handle) or, by
default, on that device's current stream. Outputs and workspaces that the caller does not give are
allocated on that stream.
"""
import contextlib
import ctypes
import functools
import os

import torch  # imported first: the library binds to the HIP runtime torch has loaded

__all__ = [
    "fp8_quantize", "fp8_gemm", "fp8_gemm_workspace_bytes", "fp8_linear_fprop", "fp8_linear_dgrad", "fp8_linear_wgrad",
    "fp8_linear_workspace_bytes", "linear_xent_forward", "linear_xent_backward", "linear_xent_workspace_bytes",
    "orthogonalize", "orthogonalize_workspace_bytes", "train_lib", "train_library_path",
]

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4_train.so")
_FPROP, _DGRAD, _WGRAD = 0, 1, 2
_IN = {torch.bfloat16: 0, torch.float32: 1}
_OUT = {torch.float32: 0, torch.bfloat16: 1}
_lib = None


def train_library_path() -> str:
    return _LIB_PATH


def train_lib():
    """The loaded C library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError("%s is missing: build it with `python -m mxfp4_block_scaled_h16_amd.build` "
                          "(or __graft_entry__.build())" % _LIB_PATH)
    L = ctypes.CDLL(_LIB_PATH)
    i64, vp, ci, cf, cs = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.mxfp4_train_abi_version.argtypes, L.mxfp4_train_abi_version.restype = [], ci
    L.mxfp4_fp8_quantize.argtypes = [vp, ci, i64, i64, i64, ci, vp, i64, vp, i64, vp, i64, vp, i64, vp]
    L.mxfp4_fp8_gemm.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, cf, cf, vp, ci, i64, vp, cs, vp]
    for name in ("fprop", "dgrad", "wgrad"):
        f = getattr(L, "mxfp4_fp8_linear_" + name)
        f.argtypes, f.restype = [vp, vp, i64, i64, i64, vp, cs, vp, ci, vp], ci
    L.mxfp4_linear_xent_forward.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, cs, vp, vp, vp]
    L.mxfp4_linear_xent_backward.argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp, cs, vp, ci, vp, ci, vp]
    L.mxfp4_orthogonalize.argtypes = [vp, ci, i64, i64, i64, i64, i64, ci, cf, cf, cf, cf, cf, cf, vp, ci, i64, i64, vp, cs, vp]
    for name in ("fp8_quantize", "fp8_gemm", "linear_xent_forward", "linear_xent_backward", "orthogonalize"):
        getattr(L, "mxfp4_" + name).restype = ci
    for name, args in (("fp8_gemm", [i64] * 3), ("fp8_linear", [ci] + [i64] * 3), ("linear_xent_forward", [i64] * 3),
                       ("linear_xent_backward", [i64] * 3), ("orthogonalize", [i64] * 3)):
        f = getattr(L, "mxfp4_%s_workspace_bytes" % name)
        f.argtypes, f.restype = args, cs
    _lib = L
    return L


def _check(status, where):
    if status != 0:
        from . import Mxfp4Error
        raise Mxfp4Error(status, where)


def _same_device(**tensors):
    """The HIP device all the given tensors (None left out) lie on."""
    device = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("%s must be a tensor on a HIP device" % name)
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, device))
    return device


@contextlib.contextmanager
def _other(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device != device:
                raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
            with torch.cuda.stream(stream):
                yield


_here = contextlib.nullcontext()


def _on(device, stream):
    """Makes `device` and `stream` the current ones, so that allocations and launches go there."""
    if stream is None and torch.cuda.current_device() == device.index:
        return _here
    return _other(device, stream)


# the current stream's handle without a Stream object around it (a call costs a few microseconds of host
# time in all, which is what small products take on the GPU)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


@functools.lru_cache(maxsize=1024)
def _need(name, *sizes):
    """Workspace bytes of one operator at these sizes."""
    return int(getattr(train_lib(), "mxfp4_%s_workspace_bytes" % name)(*sizes))


def _room(workspace, need, device):
    """The workspace, allocated if there is none."""
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError("workspace is on %s, the tensors on %s" % (workspace.device, device))
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _bytes(t):
    return t.numel() * t.element_size()


def _rows(t, name, dtypes):
    """Check a 2-D tensor of unit column stride and one of `dtypes`; its row stride."""
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d).replace("torch.", "") for d in dtypes)))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    # the stride of a single row (or of none) says nothing
    return t.stride(0) if t.shape[0] > 1 and t.stride(0) > 0 else max(t.shape[1], 1) if t.shape[0] <= 1 else t.stride(0)


def _out(out, shape, dtype, device, name):
    """The output tensor: `out` checked, or a new one."""
    if out is None:
        if dtype not in _OUT:
            raise TypeError("%s must be float32 or bfloat16" % name)
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype not in _OUT:
        raise TypeError("%s must be float32 or bfloat16" % name)
    if tuple(out.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return out


# --------------------------------------------------------------------------- 8-bit products --
def _fp8_buffers(outer, L, q, s, device, name):
    lq, ls = (L + 127) // 128 * 128, ((L + 127) // 128 + 15) // 16 * 16
    if q is None:
        q = torch.empty((outer, lq), dtype=torch.uint8, device=device)
    if s is None:
        # whole 16 bytes a row; those behind the last block are never used
        s = torch.empty((outer, ls), dtype=torch.uint8, device=device)
    for t, width, what in ((q, lq, "codes"), (s, (L + 127) // 128, "scales")):
        if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[0] < outer or t.shape[1] < width or t.stride(1) != 1:
            raise ValueError("%s: %s must be uint8 [%d, >= %d] with unit column stride" % (name, what, outer, width))
    return q, s


def fp8_quantize(x, axis=1, block="row", q=None, scales=None, stream=None):
    """Quantize a 2-D bf16 / f32 device tensor to E4M3 with a power-of-two scale for each block of 128.

    axis 1: along the rows; axis 0: along the columns (the quantized transpose); axis "both": (q1, s1,
    q0, s0) from one read. block "row": 1 x 128 along the quantized axis; "tile": 128 x 128. Returns
    (q, scales), uint8: q [outer, round_up(L, 128)] (zero codes behind L), scales [outer, round_up(ceil(L
    / 128), 16)] (ceil(L / 128) of them written). `q` and `scales` may be given for axis 0 or 1."""
    if axis not in (0, 1, "both"):
        raise ValueError("axis must be 0, 1 or 'both'")
    if block not in ("row", "tile"):
        raise ValueError("block must be 'row' or 'tile'")
    if axis == "both" and (q is not None or scales is not None):
        raise ValueError("axis 'both' allocates its outputs")
    device = _same_device(x=x, q=q, scales=scales)
    ldx = _rows(x, "x", (torch.bfloat16, torch.float32))
    rows, cols = x.shape
    with _on(device, stream):
        q1 = s1 = q0 = s0 = None
        if axis != 0:
            q1, s1 = _fp8_buffers(rows, cols, q, scales, device, "axis 1")
        if axis != 1:
            q0, s0 = _fp8_buffers(cols, rows, q, scales, device, "axis 0")
        at = lambda t: (None, 0) if t is None else (t.data_ptr(), t.stride(0))  # noqa: E731
        _check(train_lib().mxfp4_fp8_quantize(x.data_ptr(), _IN[x.dtype], rows, cols, ldx, 1 if block == "tile" else 0,
                                              *at(q1), *at(s1), *at(q0), *at(s0), _current()), "mxfp4_fp8_quantize")
    return (q1, s1, q0, s0) if axis == "both" else (q1, s1) if axis == 1 else (q0, s0)


def fp8_gemm_workspace_bytes(M, N, K) -> int:
    return _need("fp8_gemm", int(M), int(N), int(K))


def fp8_gemm(aq, as_, bq, bs, alpha=1.0, beta=0.0, out=None, out_dtype=None, k=None, workspace="auto", stream=None):
    """out[m][n] = alpha * sum_k deq(A)[m][k] deq(B)[n][k] + beta * out (FP32, or bf16 rounded once), for
    operands of fp8_quantize. k: the operands' length, when it is not their whole row. workspace: "auto"
    (allocated when the product has use for one), None, or a device tensor."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a tensor")
    device = _same_device(aq=aq, as_=as_, bq=bq, bs=bs, out=out, workspace=None if isinstance(workspace, str) else workspace)
    for t, name in ((aq, "aq"), (as_, "as_"), (bq, "bq"), (bs, "bs")):
        if t.dtype != torch.uint8 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError("%s must be 2-D uint8 with unit column stride" % name)
    M, N = aq.shape[0], bq.shape[0]
    K = min(aq.shape[1], bq.shape[1]) if k is None else int(k)
    if k is None and aq.shape[1] != bq.shape[1]:
        raise ValueError("aq and bq disagree on the length (%d, %d)" % (aq.shape[1], bq.shape[1]))
    wide, blocks = (K + 127) // 128 * 128, (K + 127) // 128
    if K < 0 or aq.shape[1] < wide or bq.shape[1] < wide:
        raise ValueError("rows of %d codes hold no %d values in whole blocks" % (min(aq.shape[1], bq.shape[1]), K))
    if as_.shape[0] < M or bs.shape[0] < N:
        raise ValueError("fewer rows of scales than of codes")
    if min(as_.shape[1], bs.shape[1]) < (blocks + 15) // 16 * 16:
        raise ValueError("rows of scales must hold %d bytes (whole 16s)" % ((blocks + 15) // 16 * 16))
    if out is None and beta != 0.0:
        raise ValueError("beta != 0 needs an existing `out`")
    with _on(device, stream):
        out = _out(out, (M, N), out_dtype or torch.float32, device, "out")
        ldc = _rows(out, "out", tuple(_OUT))
        if isinstance(workspace, str):
            need = fp8_gemm_workspace_bytes(M, N, K)
            workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        elif workspace is not None:
            workspace = _room(workspace, 0, device)
        ws = (None, 0) if workspace is None else (workspace.data_ptr(), _bytes(workspace))
        _check(train_lib().mxfp4_fp8_gemm(aq.data_ptr(), aq.stride(0), as_.data_ptr(), as_.stride(0), bq.data_ptr(),
                                          bq.stride(0), bs.data_ptr(), bs.stride(0), M, N, K, float(alpha), float(beta),
                                          out.data_ptr(), _OUT[out.dtype], ldc, *ws, _current()), "mxfp4_fp8_gemm")
    return out


def fp8_linear_workspace_bytes(pass_, M, K, N) -> int:
    return _need("fp8_linear", int(pass_), int(M), int(K), int(N))


def _fp8_linear(name, pass_, a, b, M, K, N, shape, out, out_dtype, workspace, stream):
    device = _same_device(first=a, second=b, out=out, workspace=workspace)
    for t in (a, b):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise TypeError("linear operands must be contiguous bfloat16")
    with _on(device, stream):
        out = _out(out, shape, out_dtype or torch.float32, device, "out")
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        L = train_lib()
        ws = _room(workspace, _need("fp8_linear", pass_, M, K, N), device)
        _check(getattr(L, name)(a.data_ptr(), b.data_ptr(), M, K, N, ws.data_ptr(), _bytes(ws), out.data_ptr(),
                                _OUT[out.dtype], _current()), name)
    return out


def _two_matrices(a, b, na, nb, axis_a, axis_b, what):
    for t, n in ((a, na), (b, nb)):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError("%s must be a 2-D tensor" % n)
    if a.shape[axis_a] != b.shape[axis_b]:
        raise ValueError("%s and %s disagree on %s" % (na, nb, what))


def fp8_linear_fprop(x, w, out=None, out_dtype=None, workspace=None, stream=None):
    """Y[M,N] = X[M,K] W[N,K]^T in E4M3: X in 1 x 128 blocks along K, W in 128 x 128. FP32, or out_dtype bf16."""
    _two_matrices(x, w, "x", "w", 1, 1, "K")
    M, K = x.shape
    N = w.shape[0]
    return _fp8_linear("mxfp4_fp8_linear_fprop", _FPROP, x, w, M, K, N, (M, N), out, out_dtype, workspace, stream)


def fp8_linear_dgrad(dy, w, out=None, out_dtype=None, workspace=None, stream=None):
    """dX[M,K] = dY[M,N] W[N,K] in E4M3: dY in 1 x 128 blocks along N, W in 128 x 128 (the forward codes)."""
    _two_matrices(dy, w, "dy", "w", 1, 0, "N")
    M, N = dy.shape
    K = w.shape[1]
    return _fp8_linear("mxfp4_fp8_linear_dgrad", _DGRAD, dy, w, M, K, N, (M, K), out, out_dtype, workspace, stream)


def fp8_linear_wgrad(dy, x, out=None, out_dtype=None, workspace=None, stream=None):
    """dW[N,K] = dY[M,N]^T X[M,K] in E4M3: both in 1 x 128 blocks along the tokens M."""
    _two_matrices(dy, x, "dy", "x", 0, 0, "M")
    M, N = dy.shape
    K = x.shape[1]
    return _fp8_linear("mxfp4_fp8_linear_wgrad", _WGRAD, dy, x, M, K, N, (N, K), out, out_dtype, workspace, stream)


# ------------------------------------------------------------------------------- head loss ---
def linear_xent_workspace_bytes(T, K, V, backward=False) -> int:
    return _need("linear_xent_backward" if backward else "linear_xent_forward", int(T), int(K), int(V))


def _xent_operands(x, w, target):
    ldx, ldw = _rows(x, "x", (torch.bfloat16,)), _rows(w, "w", (torch.bfloat16,))
    if x.shape[1] != w.shape[1]:
        raise ValueError("x and w disagree on K")
    if target.dtype != torch.int64 or target.shape != x.shape[:1] or not target.is_contiguous():
        raise ValueError("target must be contiguous int64 [%d]" % x.shape[0])
    return ldx, ldw


def _per_row(t, T, name):
    if t is None:
        return None
    if t.dtype != torch.float32 or tuple(t.shape) != (T,) or not t.is_contiguous():
        raise ValueError("%s must be contiguous float32 [%d]" % (name, T))
    return t.data_ptr()


def linear_xent_forward(x, w, target, ignore_index=-100, workspace=None, stream=None):
    """Softmax cross entropy of the logits X[T,K] W[V,K]^T, which are not kept. Returns (loss, lse), FP32
    [T]: lse_t = log sum_v exp z_tv and loss_t = lse_t - z_t,target, 0 where target is ignore_index, NaN
    where it is no index. x and w bf16 of unit column stride; with K a multiple of 64 their rows have to start at
    multiples of 16 bytes, any other K is copied and needs no alignment."""
    device = _same_device(x=x, w=w, target=target, workspace=workspace)
    ldx, ldw = _xent_operands(x, w, target)
    (T, K), V = x.shape, w.shape[0]
    with _on(device, stream):
        L = train_lib()
        loss = torch.empty(T, dtype=torch.float32, device=device)
        lse = torch.empty(T, dtype=torch.float32, device=device)
        ws = _room(workspace, _need("linear_xent_forward", T, K, V), device)
        _check(L.mxfp4_linear_xent_forward(x.data_ptr(), ldx, w.data_ptr(), ldw, target.data_ptr(), T, K, V, int(ignore_index),
                                           ws.data_ptr(), _bytes(ws), loss.data_ptr(), lse.data_ptr(), _current()),
               "mxfp4_linear_xent_forward")
    return loss, lse


def linear_xent_backward(dloss, x, w, target, lse, dlse=None, ignore_index=-100, need_dx=True, need_dw=True,
                         dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16, dx=None, dw=None, workspace=None, stream=None):
    """Gradients (dX[T,K], dW[V,K]) of linear_xent_forward, from the gradients of each row's loss (dloss,
    FP32 [T] or None) and of each row's lse (dlse, likewise), and the forward call's lse. need_dx or need_dw
    false: None in that place. Outputs bf16 or FP32 (the products' operands are FP16 either way, scaled). x and w as in
    linear_xent_forward."""
    device = _same_device(x=x, w=w, target=target, lse=lse, dloss=dloss, dlse=dlse, dx=dx, dw=dw, workspace=workspace)
    ldx, ldw = _xent_operands(x, w, target)
    (T, K), V = x.shape, w.shape[0]
    if (dx is not None and not need_dx) or (dw is not None and not need_dw):
        raise ValueError("an output is given that is not needed")
    rows = [_per_row(t, T, n) for t, n in ((dloss, "dloss"), (dlse, "dlse"), (lse, "lse"))]
    with _on(device, stream):
        L = train_lib()
        dx = _out(dx, (T, K), dx_dtype, device, "dx") if need_dx else None
        dw = _out(dw, (V, K), dw_dtype, device, "dw") if need_dw else None
        for t, name in ((dx, "dx"), (dw, "dw")):
            if t is not None and not t.is_contiguous():
                raise ValueError("%s must be contiguous" % name)
        ws = _room(workspace, _need("linear_xent_backward", T, K, V), device)
        at = lambda t: (None, 0) if t is None else (t.data_ptr(), _OUT[t.dtype])  # noqa: E731
        _check(L.mxfp4_linear_xent_backward(rows[0], rows[1], x.data_ptr(), ldx, w.data_ptr(), ldw, target.data_ptr(), rows[2],
                                            T, K, V, int(ignore_index), ws.data_ptr(), _bytes(ws), *at(dx), *at(dw),
                                            _current()), "mxfp4_linear_xent_backward")
    return dx, dw


# --------------------------------------------------------------------------- Newton-Schulz ---
def orthogonalize_workspace_bytes(batch, m, n) -> int:
    return _need("orthogonalize", int(batch), int(m), int(n))


def orthogonalize(g, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, alpha=1.0, beta=0.0, out=None,
                  out_dtype=None, workspace=None, stream=None):
    """alpha * X + beta * out, X the Newton-Schulz orthogonalisation of a matrix g [m, n] (bf16 or f32) or of
    each matrix of g [batch, m, n]: X = g / (|g|_F + eps), then `steps` times A = X X^T, X <- a X + (b A +
    c A A) X. The result is bf16 unless `out` or out_dtype says float32; out must not overlap g. With
    beta != 0 the update goes straight onto a weight: orthogonalize(dw, alpha=-lr, beta=1.0, out=w)."""
    device = _same_device(g=g, out=out, workspace=workspace)
    if g.dtype not in _IN:
        raise TypeError("g must be bfloat16 or float32")
    if g.dim() not in (2, 3):
        raise ValueError("g must be [m, n] or [batch, m, n]")
    if out is None and beta != 0.0:
        raise ValueError("beta != 0 needs an existing `out`")
    a, b, c = coefficients
    with _on(device, stream):
        out = _out(out, tuple(g.shape), out_dtype or torch.bfloat16, device, "out")
        g3, o3 = (g, out) if g.dim() == 3 else (g[None], out[None])
        B, m, n = g3.shape
        strides = []
        for t, name in ((g3, "g"), (o3, "out")):
            if n > 1 and t.stride(2) != 1:
                raise ValueError("%s must have unit column stride" % name)
            row = t.stride(1) if m > 1 else max(n, 1)
            strides.append((row, t.stride(0) if B > 1 else m * row))
        L = train_lib()
        ws = _room(workspace, _need("orthogonalize", B, m, n), device)
        _check(L.mxfp4_orthogonalize(g.data_ptr(), _IN[g.dtype], B, m, n, *strides[0], int(steps), float(a), float(b), float(c),
                                     float(eps), float(alpha), float(beta), out.data_ptr(), _OUT[out.dtype], *strides[1],
                                     ws.data_ptr(), _bytes(ws), _current()), "mxfp4_orthogonalize")
    return out
