"""References of the training operators, in 64 bits on the CPU, from their formulas."""
import numpy as np
import torch


def e4m3_table():
    """The 256 values of the codes (OCP E4M3: bias 7, no infinities; 0x7F and 0xFF are NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 0x7F == 0x7F else (-x if c & 0x80 else x)
    return v


TABLE = e4m3_table()
POSITIVE = TABLE[:0x7F]          # ascending, 0 .. 448


def e4m3_codes(y):
    """Codes of y (|y| <= 448), nearest, ties to the even code, by search in the table."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    c = np.where(take_lo, lo, hi)
    return (c | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def quantize(x, tile=False):
    """(codes [R, L], scales [R, ceil(L / 128)]) of x (float64 holding bf16 / f32 values), blocks along the rows."""
    x = np.asarray(x, dtype=np.float64)
    R, L = x.shape
    nb = (L + 127) // 128
    q, s = np.zeros((R, L), np.uint8), np.zeros((R, nb), np.uint8)
    step = 128 if tile else 1
    for r in range(0, R, step):
        for b in range(nb):
            blk = x[r:r + step, 128 * b:128 * b + 128]
            if not np.isfinite(blk).all():
                s[r:r + step, b] = 255
                continue
            amax = np.abs(blk).max()
            S = 0
            if amax > 0:
                S = max(int(np.floor(np.log2(amax))) - 10 + 127, 0)
                while amax > 448.0 * 2.0 ** (S - 127):
                    S += 1
            s[r:r + step, b] = S
            q[r:r + step, 128 * b:128 * b + 128] = e4m3_codes(blk * 2.0 ** (127 - S))
    return q, s


def values(q, s):
    """The numbers that codes and scales (row-major, blocks of 128) stand for."""
    e = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127.0))
    return TABLE[q] * np.repeat(e, 128, axis=1)[:, :q.shape[1]]


def xent(x, w, target, ignore, dloss, dlse):
    """loss, lse, dx, dw, G and its first part |p (dloss + dlse)|, float64."""
    x, w = x.double(), w.double()
    T = x.shape[0]
    z = x @ w.t()
    lse = torch.logsumexp(z, dim=1)
    ok = target != ignore
    at = torch.where(ok, target, 0)
    loss = torch.where(ok, lse - z[torch.arange(T), at], 0.0)
    dl = torch.where(ok, dloss.double() if dloss is not None else torch.zeros(T, dtype=torch.float64), 0.0)
    dp = dl + (dlse.double() if dlse is not None else 0.0)
    p = torch.exp(z - lse[:, None])
    g = p * dp[:, None]
    g[torch.arange(T), at] -= dl
    return loss, lse, g @ w, g.t() @ x, g, (p * dp[:, None]).abs()


def newton_schulz(g, steps, coeffs, eps):
    """float64 [m, n] -> X."""
    a, b, c = coeffs
    x = g.double()
    x = x / (x.norm() + eps)
    flip = x.shape[0] > x.shape[1]
    if flip:
        x = x.t()
    for _ in range(steps):
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.t() if flip else x
