"""The operators of ``libmxfp4_layer.so`` (C ABI in ``include/mxfp4_layer.h``): what a training step does between its
products. RMS norm of a residual stream, the gated activation, both with 8-bit outputs for ``fp8_gemm``, their gradients,
and the norm and clipping of all gradients. Like the rest of the package this is a thin ctypes binding.

Tensors may lie on any gfx950 device: a call runs on the device of its first tensor, all tensors of a call on the same
one, on `stream` (a torch.cuda.Stream of that device, or its handle) or, by default, on that device's current
stream. Outputs and workspaces that the caller does not give are allocated on that stream. Matrices need unit column
stride, nothing else.

`axis` asks for 8-bit outputs, as fp8_quantize(block="row") would make them of the FP32 values: 1 along the
rows (q1, s1), 0 along the columns, the quantized transpose (q0, s0), "both", or None. q: uint8 [outer, round_up(L, 128)],
zero codes behind L; s: uint8 [outer, round_up(ceil(L / 128), 16)], ceil(L / 128) of them written.
"""
import array
import ctypes
import functools
import operator
import os
from typing import NamedTuple, Optional

import torch  # imported first: the library binds to the HIP runtime torch has loaded

from .train import _bytes, _check, _current, _on, _room, _rows, _same_device, _IN, _OUT

__all__ = [
    "rmsnorm_forward", "rmsnorm_backward", "rmsnorm_backward_workspace_bytes", "swiglu_forward", "swiglu_backward", "grad_norm",
    "grad_scale", "grad_clip", "grad_norm_workspace_bytes", "RmsNorm", "RmsNormGrad", "Swiglu", "SwigluGrad", "Codes", "layer_lib",
    "layer_library_path",
]

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4_layer.so")
_lib = None

_Tensor = Optional[torch.Tensor]


class Codes(NamedTuple):
    """8-bit outputs: along the rows, and along the columns."""
    q1: _Tensor = None
    s1: _Tensor = None
    q0: _Tensor = None
    s0: _Tensor = None


class RmsNorm(NamedTuple):
    h: _Tensor
    rstd: _Tensor
    y: _Tensor
    q1: _Tensor
    s1: _Tensor
    q0: _Tensor
    s0: _Tensor


class RmsNormGrad(NamedTuple):
    dh: torch.Tensor
    dweight: _Tensor


class Swiglu(NamedTuple):
    a: _Tensor
    q1: _Tensor
    s1: _Tensor
    q0: _Tensor
    s0: _Tensor


class SwigluGrad(NamedTuple):
    """joined: q1 .. s0 are those of [dgate | dup]; otherwise gate and up have each gradient's."""
    dgate: _Tensor
    dup: _Tensor
    q1: _Tensor = None
    s1: _Tensor = None
    q0: _Tensor = None
    s0: _Tensor = None
    gate: Optional[Codes] = None
    up: Optional[Codes] = None


def layer_library_path() -> str:
    return _LIB_PATH


def layer_lib():
    """The loaded C library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError("%s is missing: build it with `python -m mxfp4_block_scaled_h16_amd.build` "
                          "(or __graft_entry__.build())" % _LIB_PATH)
    L = ctypes.CDLL(_LIB_PATH)
    i64, vp, ci, cf, cs = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    matrix, typed, codes = [vp, i64], [vp, ci, i64], [vp, i64, vp, i64]
    L.mxfp4_layer_abi_version.argtypes, L.mxfp4_layer_abi_version.restype = [], ci
    L.mxfp4_rmsnorm_forward.argtypes = typed + matrix + [ci, vp, ci, i64, i64, cf] + matrix + [vp] + typed + codes + codes + [vp]
    L.mxfp4_rmsnorm_backward.argtypes = typed + matrix + matrix + [ci, vp, ci, vp, i64, i64] + matrix + [vp, ci, vp, cs, vp]
    L.mxfp4_swiglu_forward.argtypes = matrix + matrix + [ci, i64, i64] + typed + codes + codes + [vp]
    L.mxfp4_swiglu_backward.argtypes = typed + matrix + matrix + [ci, i64, i64] + matrix + matrix + [ci] + 2 * [vp, vp, i64, vp, vp, i64] + [vp]
    L.mxfp4_grad_norm.argtypes = [vp, i64, vp, cs, vp, vp, vp]
    L.mxfp4_grad_scale.argtypes = [vp, i64, vp, cf, cf, vp, vp]
    L.mxfp4_grad_clip.argtypes = [vp, i64, cf, cf, vp, cs, vp, vp]
    for name in ("rmsnorm_forward", "rmsnorm_backward", "swiglu_forward", "swiglu_backward", "grad_norm", "grad_scale", "grad_clip"):
        getattr(L, "mxfp4_" + name).restype = ci
    L.mxfp4_rmsnorm_backward_workspace_bytes.argtypes, L.mxfp4_rmsnorm_backward_workspace_bytes.restype = [i64, i64], cs
    L.mxfp4_grad_norm_workspace_bytes.argtypes, L.mxfp4_grad_norm_workspace_bytes.restype = [vp, i64], cs
    _lib = L
    return L


# A call's host time is what a small call takes in all: tensors are looked at once, with the cheapest question that settles the
# usual case (a contiguous matrix on the first tensor's device), and sizes are given to torch.empty one by one, which takes
# half the time of a tuple.
_FLOATS = (torch.bfloat16, torch.float32)
_U8 = torch.uint8
_empty = torch.empty


def _device(names, first, *others):
    """The HIP device that all these tensors (None left out) lie on."""
    try:
        index = first.get_device()
        if index >= 0:
            for t in others:
                if t is not None and t.get_device() != index:
                    break
            else:
                return first.device
    except AttributeError:
        pass
    names = names.split()
    if first is None:
        raise TypeError("%s must be a tensor on a HIP device" % names[0])
    return _same_device(**dict(zip(names, (first,) + others)))


def _ld(t, shape, dtypes, name):
    """Row stride of a matrix that has to be of this shape and one of these types."""
    if t.shape == shape and t.dtype in dtypes and t.is_contiguous():
        return shape[1] or 1
    ld = _rows(t, name, dtypes)
    if t.shape != shape:
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return ld


def _first(t, name, dtypes=_FLOATS):
    """Row stride of the matrix that gives a call its shape, one of these types."""
    if t.dim() == 2 and t.dtype in dtypes and t.is_contiguous():
        return t.shape[1] or 1
    return _rows(t, name, dtypes)


_AXES = {None: (False, False), 0: (False, True), 1: (True, False), "both": (True, True)}


def _axis(axis):
    """(along the rows, along the columns)"""
    try:
        return _AXES[axis]
    except (KeyError, TypeError):
        raise ValueError("axis must be None, 0, 1 or 'both'") from None


_NO_CODES = (None, 0, None, 0)


def _codes(outer, length, device):
    """New codes and scales of `outer` rows of this length (whole 16 bytes of scales, as fp8_gemm reads them), and those as the
    library takes them."""
    blocks = (length + 127) // 128
    ldq, lds = blocks * 128, (blocks + 15) // 16 * 16
    q, s = _empty(outer, ldq, dtype=_U8, device=device), _empty(outer, lds, dtype=_U8, device=device)
    return q, s, (q.data_ptr(), ldq, s.data_ptr(), lds)


def _vector(t, n, dtypes, name):
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d).replace("torch.", "") for d in dtypes)))
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous [%d]" % (name, n))
    return t.data_ptr()


def _float(dtype, name):
    if dtype not in _OUT:
        raise TypeError("%s must be float32 or bfloat16" % name)
    return dtype


# ------------------------------------------------------------------------------- RMS norm ----
def rmsnorm_forward(x, weight=None, residual=None, eps=1e-5, axis=None, y_dtype=torch.bfloat16, need_h=True, h=None, y=None,
                    stream=None):
    """RMS norm of x [T, K], or of h = x + residual (rounded to residual's type): y = h * rstd * weight with rstd = 1 / sqrt(mean
    h^2 + eps) per row. Returns RmsNorm(h, rstd, y, q1, s1, q0, s0): h (x itself without a residual; None with need_h
    false), rstd FP32 [T], y of y_dtype (None: not formed) and the 8-bit outputs that `axis` asks for.

    x, residual and weight [K] bf16 or f32 each. `h` may be given, also residual itself (or x, the types being the same), and is
    then updated in place; a y that is given overlaps no input. Codes along the columns need h."""
    device = _device("x weight residual h y", x, weight, residual, h, y)
    ldx = _first(x, "x")
    rows, cols = shape = x.shape
    along, across = _axis(axis)
    if residual is None:
        if h is not None:
            raise ValueError("h is an output of the addition: it needs a residual")
        sdtype, need_h, ldr = x.dtype, False, 0
    else:
        sdtype, ldr = residual.dtype, _ld(residual, shape, _FLOATS, "residual")
        if not need_h and (h is not None or across):
            raise ValueError("h is given but not needed" if h is not None else "codes along the columns need h")
    w = (None, 0) if weight is None else (_vector(weight, cols, _FLOATS, "weight"), _IN[weight.dtype])
    with _on(device, stream):
        if need_h and h is None:
            h, ldh = _empty(rows, cols, dtype=sdtype, device=device), cols
        else:
            ldh = 0 if h is None else _ld(h, shape, (sdtype,), "h")
        if y is not None:
            ldy = _ld(y, shape, _FLOATS, "y")
        elif y_dtype is not None:
            y, ldy = _empty(rows, cols, dtype=_float(y_dtype, "y_dtype"), device=device), cols
        rstd = _empty(rows, dtype=torch.float32, device=device)
        q1, s1, at1 = _codes(rows, cols, device) if along else (None, None, _NO_CODES)
        q0, s0, at0 = _codes(cols, rows, device) if across else (None, None, _NO_CODES)
        _check(layer_lib().mxfp4_rmsnorm_forward(
            x.data_ptr(), _IN[x.dtype], ldx, None if residual is None else residual.data_ptr(), ldr, _IN[sdtype], *w, rows, cols,
            eps, None if h is None else h.data_ptr(), ldh, rstd.data_ptr(), *((None, 0, 0) if y is None else (y.data_ptr(), _OUT[y.dtype], ldy)),
            *at1, *at0, _current()), "mxfp4_rmsnorm_forward")
    return RmsNorm(x if residual is None else h, rstd, y, q1, s1, q0, s0)


@functools.lru_cache(maxsize=1024)
def rmsnorm_backward_workspace_bytes(rows, cols) -> int:
    return int(layer_lib().mxfp4_rmsnorm_backward_workspace_bytes(rows, cols))


def rmsnorm_backward(dy, h, rstd, weight=None, dres=None, dh=None, need_dweight=True, dweight_dtype=torch.float32, dweight=None,
                     workspace=None, stream=None):
    """Gradients of rmsnorm_forward: RmsNormGrad(dh, dweight) from dy [T, K], the forward call's h and rstd, its weight, and dres,
    the gradient that arrives at h along the residual stream (None: none). dh, of h's type, is the gradient of both x and
    residual; it may be given, also dres itself. dweight FP32 or bf16 [K]; None with need_dweight false."""
    device = _device("dy h rstd weight dres dh dweight workspace", dy, h, rstd, weight, dres, dh, dweight, workspace)
    lddy = _first(dy, "dy")
    rows, cols = shape = dy.shape
    ldh, sdtype = _ld(h, shape, _FLOATS, "h"), h.dtype
    res = (None, 0) if dres is None else (dres.data_ptr(), _ld(dres, shape, (sdtype,), "dres"))
    r = _vector(rstd, rows, (torch.float32,), "rstd")
    w = (None, 0) if weight is None else (_vector(weight, cols, _FLOATS, "weight"), _IN[weight.dtype])
    if dweight is not None and not need_dweight:
        raise ValueError("dweight is given but not needed")
    with _on(device, stream):
        if dh is None:
            dh, lddh = _empty(rows, cols, dtype=sdtype, device=device), cols
        else:
            lddh = _ld(dh, shape, (sdtype,), "dh")
        dw = ws = (None, 0)
        if need_dweight:
            if dweight is None:
                dweight = _empty(cols, dtype=_float(dweight_dtype, "dweight_dtype"), device=device)
            dw = (_vector(dweight, cols, _FLOATS, "dweight"), _OUT[dweight.dtype])
            workspace = _room(workspace, rmsnorm_backward_workspace_bytes(rows, cols), device)
            ws = (workspace.data_ptr(), _bytes(workspace))
        _check(layer_lib().mxfp4_rmsnorm_backward(
            dy.data_ptr(), _IN[dy.dtype], lddy, *res, h.data_ptr(), ldh, _IN[sdtype], *w, r, rows, cols, dh.data_ptr(), lddh, *dw,
            *ws, _current()), "mxfp4_rmsnorm_backward")
    return RmsNormGrad(dh, dweight)


# ------------------------------------------------------------------------- gated activation --
def swiglu_forward(gate, up, axis=None, out_dtype=torch.bfloat16, a=None, stream=None):
    """a = silu(gate) * up of two matrices [T, F], bf16 or f32 alike (they may be the halves of one). Returns Swiglu(a, q1, s1,
    q0, s0): a of out_dtype (None: not formed) and the 8-bit outputs that `axis` asks for. `a` may be given, also gate or up."""
    device = _device("gate up a", gate, up, a)
    ldg = _first(gate, "gate")
    rows, cols = shape = gate.shape
    dtype = gate.dtype
    ldu = _ld(up, shape, (dtype,), "up")
    along, across = _axis(axis)
    with _on(device, stream):
        if a is not None:
            lda = _ld(a, shape, _FLOATS, "a")
        elif out_dtype is not None:
            a, lda = _empty(rows, cols, dtype=_float(out_dtype, "out_dtype"), device=device), cols or 1
        q1, s1, at1 = _codes(rows, cols, device) if along else (None, None, _NO_CODES)
        q0, s0, at0 = _codes(cols, rows, device) if across else (None, None, _NO_CODES)
        _check(layer_lib().mxfp4_swiglu_forward(
            gate.data_ptr(), ldg, up.data_ptr(), ldu, _IN[dtype], rows, cols, *((None, 0, 0) if a is None else (a.data_ptr(), _OUT[a.dtype], lda)),
            *at1, *at0, _current()), "mxfp4_swiglu_forward")
    return Swiglu(a, q1, s1, q0, s0)


def swiglu_backward(da, gate, up, axis=None, out_dtype=torch.bfloat16, joined=True, dgate=None, dup=None, stream=None):
    """Gradients of swiglu_forward from da [T, F]: SwigluGrad with dgate and dup of out_dtype (None: not formed) and the 8-bit
    outputs that `axis` asks for. joined: they are those of [dgate | dup], as one product of 2 F columns reads them (q1 [T, 2 F],
    F then a multiple of 128; q0 [2 F, T]), and dgate and dup the halves of one new matrix; otherwise .gate and .up have
    the Codes of each. dgate and dup may be given, also da, gate or up themselves."""
    device = _device("da gate up dgate dup", da, gate, up, dgate, dup)
    ldda = _first(da, "da")
    rows, cols = shape = da.shape
    dtype = gate.dtype
    ldg, ldu = _ld(gate, shape, _FLOATS, "gate"), _ld(up, shape, (dtype,), "up")
    along, across = _axis(axis)
    if (dgate is None) != (dup is None):
        raise ValueError("dgate and dup are given together")
    if dgate is not None and dgate.dtype != dup.dtype:
        raise TypeError("dgate and dup must be of one type")
    if joined and along and cols % 128:
        raise ValueError("joined codes along the rows need a multiple of 128 columns")
    with _on(device, stream):
        if dgate is not None:
            outs = (dgate.data_ptr(), _ld(dgate, shape, _FLOATS, "dgate"), dup.data_ptr(), _ld(dup, shape, _FLOATS, "dup"), _OUT[dgate.dtype])
        elif out_dtype is None:
            outs = (None, 0, None, 0, 0)
        else:
            _float(out_dtype, "out_dtype")
            if joined:
                both = _empty(rows, 2 * cols, dtype=out_dtype, device=device)
                dgate, dup, ld = both[:, :cols], both[:, cols:], 2 * cols or 1
            else:
                dgate, dup = (_empty(rows, cols, dtype=out_dtype, device=device) for _ in range(2))
                ld = cols or 1
            outs = (dgate.data_ptr(), ld, dup.data_ptr(), ld, _OUT[out_dtype])
        q1 = s1 = q0 = s0 = g = u = None
        at1 = at0 = (None, None, 0, None, None, 0)
        if joined:
            if along:
                q1, s1, (q, ldq, sc, lds) = _codes(rows, 2 * cols, device)
                at1 = (q, q + cols, ldq, sc, sc + cols // 128, lds)
            if across:
                q0, s0, (q, ldq, sc, lds) = _codes(2 * cols, rows, device)
                at0 = (q, q + cols * ldq, ldq, sc, sc + cols * lds, lds)
        else:
            none = (None, None, _NO_CODES)
            (gq1, gs1, g1), (uq1, us1, u1) = (_codes(rows, cols, device), _codes(rows, cols, device)) if along else (none, none)
            (gq0, gs0, g0), (uq0, us0, u0) = (_codes(cols, rows, device), _codes(cols, rows, device)) if across else (none, none)
            g, u = Codes(gq1, gs1, gq0, gs0), Codes(uq1, us1, uq0, us0)
            at1, at0 = (g1[0], u1[0], g1[1], g1[2], u1[2], g1[3]), (g0[0], u0[0], g0[1], g0[2], u0[2], g0[3])
        _check(layer_lib().mxfp4_swiglu_backward(
            da.data_ptr(), _IN[da.dtype], ldda, gate.data_ptr(), ldg, up.data_ptr(), ldu, _IN[dtype], rows, cols, *outs, *at1, *at0,
            _current()), "mxfp4_swiglu_backward")
    return SwigluGrad(dgate, dup, q1, s1, q0, s0, g, u)


# ------------------------------------------------------------------------- gradients' norm ---
def _dense(t):
    """Whether the values lie in memory without a gap or a repetition, in any order of the axes."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((st, sz) for sz, st in zip(t.shape, t.stride()) if sz != 1):
        if stride != want:
            return False
        want *= size
    return True


def _check_grad(g, o, index):
    if not isinstance(g, torch.Tensor) or not isinstance(o, torch.Tensor) or not g.is_cuda:
        raise TypeError("gradients and outputs must be tensors on a HIP device")
    if g.get_device() != index or o.get_device() != index:
        raise ValueError("gradients and outputs must be on one device")
    if g.dtype not in _IN or o.dtype not in _OUT:
        raise TypeError("gradients and outputs must be bfloat16 or float32")
    if not _dense(g):
        raise ValueError("gradients must be dense")
    if o is not g and (o.numel() != g.numel() if o.is_contiguous() and g.is_contiguous() else
                       o.shape != g.shape or o.stride() != g.stride()):
        raise ValueError("an output must have its gradient's shape and strides, or as many values where both are contiguous")


_T = torch.Tensor
_dtype = operator.attrgetter("dtype")
# types of a gradient and its output as the library's array holds them: two 32-bit words
_TYPES = {(g, o): _IN[g] | _OUT[o] << 32 for g in _IN for o in _OUT}


def _grads(grads, out):
    """The device, and the tensors as the library takes them."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    outs = grads if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    if len(outs) != len(grads):
        raise ValueError("%d outputs for %d gradients" % (len(outs), len(grads)))
    if not grads:
        raise ValueError("no gradients")
    if not isinstance(grads[0], torch.Tensor):
        raise TypeError("gradients must be tensors")
    index = grads[0].get_device()
    # one question to all tensors at a time, in half the time of a loop over them; where one is not as usual, each by itself
    try:
        usual = {index} == set(map(_T.get_device, grads)) and index >= 0 and all(map(_T.is_contiguous, grads))
        counts = list(map(_T.numel, grads))
        if usual and outs is not grads:
            usual = ({index} == set(map(_T.get_device, outs)) and all(map(_T.is_contiguous, outs))
                     and counts == list(map(_T.numel, outs)))
        types = list(map(_TYPES.get, zip(map(_dtype, grads), map(_dtype, outs))))
    except (AttributeError, TypeError):
        usual, types = False, [None]
    if not usual or None in types:
        for g, o in zip(grads, outs):
            _check_grad(g, o, index)
    items = array.array("q", bytes(32 * len(grads)))
    items[0::4] = array.array("q", list(map(_T.data_ptr, grads)))
    items[1::4] = items[0::4] if outs is grads else array.array("q", list(map(_T.data_ptr, outs)))
    items[2::4] = array.array("q", counts)
    items[3::4] = array.array("q", types)
    return grads[0].device, items, len(grads)


def grad_norm_workspace_bytes(grads) -> int:
    _, items, n = _grads(grads, None)
    return int(layer_lib().mxfp4_grad_norm_workspace_bytes(items.buffer_info()[0], n))


def grad_norm(grads, workspace=None, stream=None):
    """The norm over all values of the gradients (dense tensors, bf16 or f32 in any mixture) together. Returns (sum_sq, norm): the
    sum of squares, float64 [], which ranks that hold parts of the gradients add up, and its root, FP32 []."""
    device, items, n = _grads(grads, None)
    with _on(device, stream):
        L, at = layer_lib(), items.buffer_info()[0]
        ws = _room(workspace, L.mxfp4_grad_norm_workspace_bytes(at, n) if workspace is None else 0, device)
        sum_sq = torch.empty((), dtype=torch.float64, device=device)
        norm = torch.empty((), dtype=torch.float32, device=device)
        _check(L.mxfp4_grad_norm(at, n, ws.data_ptr(), _bytes(ws), sum_sq.data_ptr(), norm.data_ptr(), _current()), "mxfp4_grad_norm")
    return sum_sq, norm


def grad_scale(grads, sum_sq, max_norm, eps=1e-6, out=None, stream=None):
    """Multiplies the gradients by min(1, max_norm / (norm + eps)) with norm the root of sum_sq, float64 [] on their device: in
    place, or into `out` (bf16 or f32 tensors of the same shapes and strides; of contiguous ones also of other shapes, such as parts of
    a flat buffer). Returns norm, FP32 []."""
    device, items, n = _grads(grads, out)
    if not isinstance(sum_sq, torch.Tensor) or sum_sq.dtype != torch.float64 or sum_sq.numel() != 1 or sum_sq.device != device:
        raise ValueError("sum_sq must be one float64 on the gradients' device")
    with _on(device, stream):
        norm = torch.empty((), dtype=torch.float32, device=device)
        _check(layer_lib().mxfp4_grad_scale(items.buffer_info()[0], n, sum_sq.data_ptr(), float(max_norm), float(eps),
                                            norm.data_ptr(), _current()), "mxfp4_grad_scale")
    return norm


def grad_clip(grads, max_norm, eps=1e-6, out=None, workspace=None, stream=None):
    """grad_norm and grad_scale in one: scales the gradients so that their norm is at most max_norm, in place or into
    `out`, and returns the norm that they had, FP32 []. An infinite norm makes finite values 0, one that is NaN all values.
    max_norm and eps count as FP32 holds them, here and in grad_scale."""
    device, items, n = _grads(grads, out)
    with _on(device, stream):
        L, at = layer_lib(), items.buffer_info()[0]
        ws = _room(workspace, L.mxfp4_grad_norm_workspace_bytes(at, n) if workspace is None else 0, device)
        norm = torch.empty((), dtype=torch.float32, device=device)
        _check(L.mxfp4_grad_clip(at, n, float(max_norm), float(eps), ws.data_ptr(), _bytes(ws), norm.data_ptr(), _current()),
               "mxfp4_grad_clip")
    return norm
