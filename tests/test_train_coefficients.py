"""Which Newton-Schulz coefficients mxfp4_orthogonalize takes: those with which no singular value that starts in [0, 1] leaves the
bounds of include/mxfp4_train.h at any step (no GPU: accepted calls end at a workspace that is too small)."""
import numpy as np
import pytest

from tests.test_train_abi import ARG, WORKSPACE, L, _ortho  # noqa: F401  (L: a fixture)


def _accepted(L, steps, a, b, c):  # noqa: F811
    got = _ortho(L, steps=steps, a=a, b=b, c=c, nbytes=0)
    assert got in (ARG, WORKSPACE)
    return got == WORKSPACE


def _furthest(steps, a, b, c, starts=200001):
    """The largest |s| / 4 and |b x + c x x| / 32 on a fine grid of starting values."""
    s, most = np.linspace(0.0, 1.0, starts), 0.0
    for _ in range(steps):
        x = s * s
        p = b * x + c * x * x
        s = (a + p) * s
        most = max(most, np.abs(p).max() / 32.0, np.abs(s).max() / 4.0)
        s = np.clip(s, -1e6, 1e6)
    return most


@pytest.mark.parametrize("steps,a,b,c", [(5, 4.484556198120117, -13.70450496673584, 8.174581527709961),
                                         (5, -2.6081345081329346, 9.387134552001953, -5.6306257247924805),
                                         (5, 3.2855100631713867, -12.215631484985352, 8.161357879638672),
                                         (6, -1.1114431619644165, -1.6789993047714233, 1.4253063201904297)])
def test_values_between_the_even_ones(L, steps, a, b, c):  # noqa: F811
    """257 even starting values stay within the bounds, one between them gets beyond 64, where FP16 ends."""
    assert _furthest(steps, a, b, c, 257) <= 1.0 and 4.0 * _furthest(steps, a, b, c) > 64.0
    assert not _accepted(L, steps, a, b, c)


def test_the_usual_ones_and_the_ends_of_the_range(L):  # noqa: F811
    for steps in (0, 1, 5, 32):
        for coeffs in ((3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (0.0, 0.0, 0.0)):
            assert _accepted(L, steps, *coeffs)
    assert _accepted(L, 1, 4.0, 0.0, 0.0) and not _accepted(L, 1, 4.001, 0.0, 0.0) and not _accepted(L, 2, 4.0, 0.0, 0.0)
    assert _accepted(L, 0, 1e30, -1e30, 1e30) and not _accepted(L, 1, 1e38, -1e38, 1e38)
    # 32 at the middle, x = 1/2; within 4 there, and 0 at x = 1
    assert not _accepted(L, 1, 0.0, 128.5, -128.5)
    assert _accepted(L, 1, 3.0, 1e-30, -1e-38) and _accepted(L, 1, 1.0, 0.0, 3.0) and not _accepted(L, 1, 1.0, 0.0, 3.1)


def test_random_ones(L):  # noqa: F811
    rng = np.random.default_rng(4)
    seen = [0, 0]
    for _ in range(600):
        steps = int(rng.integers(1, 9))
        a, b, c = (float(np.float32(v)) for v in rng.uniform(-1.0, 1.0, 3) * rng.choice([1.0, 2.0, 4.0]) * [2.0, 4.0, 2.5])
        most = _furthest(steps, a, b, c)
        if 0.99 < most < 1.01:
            continue
        ok = _accepted(L, steps, a, b, c)
        # what the fine grid finds beyond the bounds is refused; the other way round it may miss a value
        assert ok == (most < 1.0) or not ok and _furthest(steps, a, b, c, 4000001) > 0.999, (steps, a, b, c, most)
        seen[ok] += 1
    assert min(seen) > 50
