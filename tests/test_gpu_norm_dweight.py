"""The norm's dweight over many rows, on the GPU, within what its own order of sums can lose: a workgroup's rows that are left out show,
and up to some 20000 rows a single one."""
import pytest
import torch

from tests.gpu_util import announce, require_gpu
from tests.layer_util import BF, F32, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _mx():
    import mxfp4_block_scaled_h16_amd as mx
    return mx


def _roundings(rows, cols):
    """Roundings that a term of dweight passes at most: h rstd and the multiply-add's sums, one for each of a thread's rows (512
    workgroups of 8, 4, 2 or 1 rows at a time), those of the row groups, then of 16 partial sums and of 32 shares."""
    at_once = 8 if cols <= 512 else 4 if cols <= 1024 else 2 if cols <= 2048 else 1
    groups = -(-rows // at_once)
    return 2 + -(-groups // 512) + at_once + 16 + 32


@pytest.mark.parametrize("rows,cols", [(1, 300), (512, 4096), (513, 4096), (1000, 2001), ((1 << 22) + 5, 8), (1000003, 60), (100003, 300), (60001, 1024), (20011, 2048),
                                       (9000, 4096), (5000, 8192), (3001, 16384), (2000, 20000)])
@pytest.mark.parametrize("branch,stream", [(BF, BF), (F32, F32)])
def test_every_row_counts(rows, cols, branch, stream):
    mx = _mx()
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    # terms of one sign, of which each is about one over the rows of the sum
    dy, h = (0.5 + torch.rand(rows, cols, generator=g, device="cuda") for _ in range(2))
    dy, h = dy.to(branch), h.to(stream)
    rstd = 0.5 + torch.rand(rows, generator=g, device="cuda")
    announce("norm dweight", rows, cols, branch, stream)
    got = mx.rmsnorm_backward(dy, h, rstd).dweight.double()
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 1 << 16):
        part = slice(at, at + (1 << 16))
        want += (dy[part].double() * h[part].double() * rstd[part].double()[:, None]).sum(dim=0)
    tol = U * _roundings(rows, cols) * 1.001
    off = float(((got - want).abs() / want).max())
    assert off <= tol, "%.3g of its tolerance" % (off / tol)
    # the smallest term is an eighth of the mean one: a workgroup's share of the rows shows, and of some 20000 rows one row
    assert tol < 0.1 / 512 and (rows > 20011 or tol < 0.1 / rows)
