"""8-bit linear products on the GPU: codes and scales bit for bit, products against the 64-bit product
of the decoded operands."""
import numpy as np
import pytest
import torch

from tests import train_util as ref
from tests.gpu_util import announce, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _data(rows, cols, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if kind == "wide":        # magnitudes over 60 binades: subnormal codes and small scales
        x = x * torch.exp2(torch.randint(-30, 30, (rows, cols), generator=g).float())
    if kind == "tiny":        # block maxima below 448 * 2^-127: scale 0
        x = x * 2.0 ** -120
    if kind == "grid":        # ties and the border of the scale rule
        x = torch.randint(-480, 481, (rows, cols), generator=g).float() / 16.0
    return x


def _check_codes(q, s, x, tile):
    q, s = q.cpu().numpy(), s.cpu().numpy()
    rq, rs = ref.quantize(x, tile)
    L = x.shape[1]
    assert np.array_equal(s[:, :rs.shape[1]], rs)
    assert np.array_equal(q[:, :L], rq)
    assert not q[:, L:].any()                                   # zero codes behind the row


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (128, 1), (5, 129), (128, 128), (130, 383), (257, 1000), (64, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_codes_and_scales(rows, cols, dtype, block):
    mx = _mx()
    for kind in ("normal", "wide", "grid", "tiny"):
        x = _data(rows, cols, rows * 7 + cols, kind).to(dtype)
        if kind == "normal" and rows * cols > 4:
            x.view(-1)[::7] = 0.0
        if dtype == torch.float32 and kind == "tiny":
            x = x * 2.0 ** -8
        announce("fp8 quantize", rows, cols, dtype, block, kind)
        xd = x.cuda()
        q1, s1, q0, s0 = mx.fp8_quantize(xd, axis="both", block=block)
        _check_codes(q1, s1, x.double().numpy(), block == "tile")
        _check_codes(q0, s0, x.t().contiguous().double().numpy(), block == "tile")
        for axis, q, s in ((1, q1, s1), (0, q0, s0)):
            qa, sa = mx.fp8_quantize(xd, axis=axis, block=block)
            nb = ((cols if axis == 1 else rows) + 127) // 128
            assert torch.equal(qa, q) and torch.equal(sa[:, :nb], s[:, :nb])


def test_strided_and_misaligned_input():
    mx = _mx()
    for dtype in (torch.bfloat16, torch.float32):
        big = _data(140, 403, 3).to(dtype).cuda()
        for view in (big[:, 1:202], big[::2, 3:], big[3:4], big[:, :1]):
            announce("fp8 strided", tuple(view.shape), view.stride())
            q, s = mx.fp8_quantize(view)
            _check_codes(q, s, view.cpu().double().numpy(), False)


def test_blocks_with_nan_or_infinity():
    mx = _mx()
    x = _data(200, 300, 5)
    x[3, 5], x[130, 290], x[40, 130] = float("nan"), float("inf"), -float("inf")
    for block in ("row", "tile"):
        q1, s1, q0, s0 = mx.fp8_quantize(x.cuda(), axis="both", block=block)
        _check_codes(q1, s1, x.double().numpy(), block == "tile")
        _check_codes(q0, s0, x.t().contiguous().double().numpy(), block == "tile")
    # their products are NaN, the others are not
    q, s = mx.fp8_quantize(x.cuda())
    w, ws = mx.fp8_quantize(_data(17, 300, 6).cuda())
    c = mx.fp8_gemm(q, s, w, ws, k=300)
    assert torch.isnan(c).any(dim=1).nonzero()[:, 0].tolist() == [3, 40, 130]


def test_rows_behind_the_last_are_left_alone():
    mx = _mx()
    q = torch.full((8, 256), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((8, 16), 77, dtype=torch.uint8, device="cuda")
    mx.fp8_quantize(_data(5, 200, 1).cuda(), q=q, scales=s)
    assert (q[5:] == 77).all() and (s[5:] == 77).all() and (s[:, 2:] == 77).all()
    out = torch.full((6, 9), 7.0, device="cuda")
    mx.fp8_gemm(q[:5], s[:5], q[:5], s[:5], out=out[:5, :5], k=200)
    assert (out[5:] == 7.0).all() and (out[:, 5:] == 7.0).all() and (out[:5, :5] != 7.0).all()


# ------------------------------------------------------------------------------- products ----
def _random_operand(outer, L, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (outer, (L + 127) // 128 * 128), dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0
    q[:, L:] = 0
    s = rng.integers(117, 138, (outer, ((L + 127) // 128 + 15) // 16 * 16), dtype=np.uint8)
    return q, s


def _bound(A, B):
    """Elementwise bound of the product of the matrices A [M, K] and B [N, K] (values of codes times scales).

    The FP8 matrix cores add the products of eight consecutive k at a time and first cut each, toward
    zero, to multiples of 2^-13 of the largest one's power of two (pinned below): at most seven lose
    less than 2^-13 of the largest each. The sums of eight join the accumulator in FP32: K / 8 additions and
    one more for the last sum, each within a unit in the last place (2^-23) of the sum of the |terms|."""
    A, B = np.abs(A), np.abs(B)
    pad = -A.shape[1] % 8
    A, B = np.pad(A, ((0, 0), (0, pad))), np.pad(B, ((0, 0), (0, pad)))
    cut = np.zeros((A.shape[0], B.shape[0]))
    for k in range(0, A.shape[1], 8):
        top = np.zeros_like(cut)
        for j in range(8):
            np.maximum(top, np.outer(A[:, k + j], B[:, k + j]), out=top)
        cut += top
    return 7 * 2.0 ** -13 * cut + (A.shape[1] / 8 + 8) * 2.0 ** -23 * (A @ B.T)


def test_what_the_matrix_cores_keep():
    """A product of 1/2^k beside one of 1: in the same eight it is kept down to 2^-13 and cut below, further away
    it is kept as far as FP32 reaches."""
    mx = _mx()
    one = torch.zeros(1, 128)
    for far in (1, 7, 8, 127):
        for k, kept in ((13, True), (14, far >= 8), (20, far >= 8)):
            a, b = one.clone(), one.clone()
            a[0, 0] = b[0, 0] = 256.0               # scales 1, codes as they are
            a[0, far], b[0, far] = 2.0 ** (8 - k // 2), 2.0 ** (8 - (k - k // 2))
            (qa, sa), (qb, sb) = mx.fp8_quantize(a.cuda()), mx.fp8_quantize(b.cuda())
            got = float(mx.fp8_gemm(qa, sa, qb, sb)[0, 0])
            assert got == 65536.0 + (2.0 ** (16 - k) if kept else 0.0), (far, k)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 300, 128), (300, 1, 129), (17, 33, 64), (128, 128, 256), (129, 257, 2049),
                                   (256, 256, 4096), (311, 200, 5000), (2048, 4352, 48)])
def test_product_of_any_codes(M, N, K):
    mx = _mx()
    aq, as_ = _random_operand(M, K, 1)
    bq, bs = _random_operand(N, K, 2)
    A, B = ref.values(aq, as_[:, :(K + 127) // 128]), ref.values(bq, bs[:, :(K + 127) // 128])
    exact, bound = A @ B.T, _bound(A, B)
    dev = [torch.from_numpy(t).cuda() for t in (aq, as_, bq, bs)]
    announce("fp8 gemm", M, N, K)
    c = mx.fp8_gemm(*dev, k=K).cpu().numpy().astype(np.float64)
    assert bool((np.abs(c - exact) <= bound).all())
    # alpha, beta, bf16, a strided output, no workspace
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.randn(M, N + 3, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
        old = out.cpu().double().numpy()
        mx.fp8_gemm(*dev, k=K, alpha=0.25, beta=-2.0, out=out[:, :N], workspace=None)
        got = out.cpu().double().numpy()
        want = 0.25 * exact - 2.0 * old[:, :N]
        tol = 0.25 * bound + 2.0 ** -23 * (np.abs(0.25 * exact) + np.abs(2.0 * old[:, :N]))
        if dtype == torch.bfloat16:
            tol = tol * 1.01 + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
        assert bool((np.abs(got[:, :N] - want) <= tol).all())
        assert np.array_equal(got[:, N:], old[:, N:])
    # beta = 0 does not read the output
    out = torch.full((M, N), float("nan"), device="cuda")
    mx.fp8_gemm(*dev, k=K, out=out)
    assert np.array_equal(out.cpu().numpy().astype(np.float64), c)


@pytest.mark.parametrize("which", ["fprop", "dgrad", "wgrad"])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 512, 300), (256, 512, 256), (333, 200, 130), (1000, 130, 999), (0, 64, 32),
                                   (64, 0, 32)])
def test_linear_passes(which, M, K, N):
    mx = _mx()
    x = _data(M, K, 1).to(torch.bfloat16)
    w = (0.02 * _data(N, K, 2)).to(torch.bfloat16)
    dy = (1e-3 * _data(M, N, 3, "wide")).to(torch.bfloat16)
    d = lambda t: t.double().numpy()  # noqa: E731
    announce("fp8 linear", which, M, K, N)
    if which == "fprop":
        got = mx.fp8_linear_fprop(x.cuda(), w.cuda())
        A, B = ref.values(*ref.quantize(d(x))), ref.values(*ref.quantize(d(w), True))
    elif which == "dgrad":
        got = mx.fp8_linear_dgrad(dy.cuda(), w.cuda())
        A, B = ref.values(*ref.quantize(d(dy))), ref.values(*ref.quantize(d(w.t().contiguous()), True))
    else:
        got = mx.fp8_linear_wgrad(dy.cuda(), x.cuda())
        A, B = ref.values(*ref.quantize(d(dy.t().contiguous()))), ref.values(*ref.quantize(d(x.t().contiguous())))
    exact = A @ B.T
    assert got.shape == exact.shape and got.dtype == torch.float32
    assert bool((np.abs(got.cpu().double().numpy() - exact) <= _bound(A, B)).all())
    # the weight's codes are the same numbers along both axes
    if which == "dgrad" and K and N:
        q1, s1, q0, s0 = mx.fp8_quantize(w.cuda(), axis="both", block="tile")
        assert torch.equal(q1[:, :K], q0[:, :N].t())


def test_linear_in_bf16_on_another_stream_and_in_a_graph():
    mx = _mx()
    x, w = _data(300, 640, 1).to(torch.bfloat16).cuda(), _data(200, 640, 2).to(torch.bfloat16).cuda()
    want = mx.fp8_linear_fprop(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mx.fp8_linear_fprop(x, w, stream=side)
    low = mx.fp8_linear_fprop(x, w, out_dtype=torch.bfloat16, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(low, want.to(torch.bfloat16))
    ws = torch.empty(mx.fp8_linear_workspace_bytes(mx.FPROP, 300, 640, 200), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.fp8_linear_fprop(x, w, out=out, workspace=ws)
    for k in range(3):
        x.copy_(_data(300, 640, 10 + k))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.fp8_linear_fprop(x, w))
