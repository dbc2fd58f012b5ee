"""References of the operators between the products, in 64 bits on the CPU, from their formulas."""
import numpy as np
import torch

from tests import train_util as ref

U = 2.0 ** -24                   # a rounding to FP32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32


def heavy(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = torch.randn(*shape, generator=g)
    chi = sum(torch.randn(*shape, generator=g).square() for _ in range(3))
    return scale * n / (chi / 3.0).sqrt()


def quantize(x):
    """train_util.quantize for blocks along the rows, all blocks at once: (codes [R, L], scales [R, ceil(L / 128)])."""
    R, L = x.shape
    nb = (L + 127) // 128
    b = np.zeros((R, nb * 128))
    b[:, :L] = x
    b = b.reshape(R, nb, 128)
    bad = ~np.isfinite(b).all(axis=2)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=2))
    S = np.maximum(np.frexp(amax)[1] - 1 - 10 + 127, 0)             # frexp's exponent is one more than the logarithm's floor
    for _ in range(3):
        S = np.where(amax > 448.0 * np.exp2(S - 127.0), S + 1, S)
    S = np.where(amax == 0.0, 0, S)
    with np.errstate(invalid="ignore"):
        q = ref.e4m3_codes(np.where(bad[:, :, None], 0.0, b) * np.exp2(127.0 - S)[:, :, None])
    return q.reshape(R, -1)[:, :L], np.where(bad, 255, S).astype(np.uint8)


def check_codes(q, s, v, what=""):
    """Codes and scales bit for bit those of v (the FP32 values, [outer, L]), zero codes behind L."""
    rq, rs = quantize(v.double().numpy())
    L = v.shape[1]
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(s[:, :rs.shape[1]], rs), what
    assert np.array_equal(q[:, :L], rq), what
    assert q.shape[1] == (L + 127) // 128 * 128 and not q[:, L:].any(), what


def check_axes(o, v, axis, what=""):
    if axis in (1, "both"):
        check_codes(o.q1, o.s1, v, what)
    if axis in (0, "both"):
        check_codes(o.q0, o.s0, v.t().contiguous(), what)


def assert_within(got, exact, tol, what=""):
    got, exact, tol = got.cpu().double(), exact.double(), tol if isinstance(tol, torch.Tensor) else torch.tensor(tol)
    off = (got - exact).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), "%s: %d of %d outside, worst %.3g of its tolerance" % (
        what, int(bad.sum()), bad.numel(), float((off / tol.clamp(min=1e-300)).max()))


# ------------------------------------------------------------------------------- RMS norm ----
def norm_stream(x, r):
    """h: the sum rounded to the stream's type."""
    return x if r is None else (x.float() + r.float()).to(r.dtype)


def norm_rstd(h, eps):
    return 1.0 / torch.sqrt(h.double().square().mean(dim=1) + eps)


def norm_y32(h, rstd32, w):
    """y as FP32 gives it, product by product: (h rstd) w."""
    y = h.float() * rstd32[:, None]
    return y if w is None else y * w.float()


def norm_grad(dy, h, rstd, w, dres):
    """dh, dw in 64 bits, and the tolerances that FP32's roundings give them (without the last one)."""
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    rows, cols = dy.shape
    u = dy if w is None else dy * w.double()
    n = h * rstd
    mean = (u * n).mean(dim=1, keepdim=True)
    dh = rstd * (u - n * mean)
    if dres is not None:
        dh = dh + dres.double()
    dw = (dy * n).sum(dim=0)
    # u and n: one rounding each. The mean: three for a product of the sum, and the sum's own, at most one for each value that
    # a thread adds (16 of them, and one more for each 1024 columns of a long row), 6 in a wavefront and 16 behind it; its
    # division, n times it, the difference, the last product and sum
    spread = (u * n).abs().mean(dim=1, keepdim=True)
    tol = U * (rstd * (3 * u.abs() + 5 * (n * mean).abs() + n.abs() * (45 + cols / 1024) * spread) + 2 * dh.abs())
    # dw: two roundings for a product, one for each of the rows that a thread adds, 16 and 48 to join them
    tol_w = U * (68 + rows / 64) * (dy * n).abs().sum(dim=0)
    return dh, dw, tol, tol_w


# ------------------------------------------------------------------------- gated activation --
def gate_forward(g, u):
    g, u = g.double(), u.double()
    return g * torch.sigmoid(g) * u


def gate_backward(da, g, u):
    da, g, u = da.double(), g.double(), u.double()
    s, t = torch.sigmoid(g), torch.sigmoid(-g)
    return da * u * s * (1 + g * t), da * g * s, (da * u * s).abs() * (1 + (g * t).abs())


TINY = 2.0 ** -126               # what exp(-|g|) may lose at its end, and the products below FP32's normal range
