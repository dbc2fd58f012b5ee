"""Which calls of libmxfp4_layer stream past the caches: those of more than the last cache takes, where that was measured to be faster. Its
host code, driven by tests/layer_kernels.c, which stands in for the HIP runtime (no GPU): a call streams if it launches other
kernels than the same one of few rows."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = 0, 1
WIDE, ROWS, BOTH = 0, 1, 3      # results: bf16 alone; codes along the rows; along both axes


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    import mxfp4_block_scaled_h16_amd as mx
    from mxfp4_block_scaled_h16_amd import build
    mx.layer_lib()
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(build.hipcc())))
    exe = str(tmp_path_factory.mktemp("layer_kernels") / "layer_kernels")
    here = os.path.dirname(build.LAYER_LIB)
    subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-I" + os.path.join(rocm, "include"),
                    os.path.join(ROOT, "tests", "layer_kernels.c"), build.LAYER_LIB, "-rdynamic", "-Wl,-rpath," + here,
                    "-Wl,-rpath," + os.path.join(rocm, "lib"), "-L" + os.path.join(rocm, "lib"), "-lamdhip64", "-o", exe], check=True)

    def calls(lines):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, line)) for line in lines) + "\n", capture_output=True, text=True,
                           timeout=60, check=True)
        out = [line.split() for line in r.stdout.splitlines()]
        assert len(out) == len(lines) and all(o[0] == "0" and len(o) > 1 for o in out)
        return [o[1:] for o in out]
    return calls


def _streams(kernels, name, rows, cols, pad, off, a, b, out):
    few, many = kernels([(name, n, cols, pad, off, a, b, out) for n in (256, rows)])
    assert len(few) == len(many)
    return [p != q for p, q in zip(few, many)]


@pytest.mark.parametrize("name", ["gate", "gategrad"])
@pytest.mark.parametrize("out", [WIDE, BOTH])
def test_gate(kernels, name, out):
    """All in bf16, and every row of every input at a multiple of 16 bytes."""
    for pad, off, want in ((0, 0, True), (8, 8, True), (16, 0, True), (1, 0, False), (4, 0, False), (0, 1, False), (8, 4, False), (7, 1, False)):
        assert _streams(kernels, name, 8192, 14336, pad, off, BF, BF, out) == [want], (pad, off)
    assert _streams(kernels, name, 8192, 14335, 1, 0, BF, BF, out) == [True]
    assert _streams(kernels, name, 8192, 14335, 0, 0, BF, BF, out) == [False]
    assert _streams(kernels, name, 1024, 14336, 0, 0, BF, BF, out) == [False]
    for a, b in ((F32, F32), (F32, BF), (BF, F32)):
        if name == "gategrad" or a == F32:
            assert _streams(kernels, name, 8192, 14336, 0, 0, a, b, out) == [False]


def test_norm(kernels):
    """x in bf16, and an FP32 stream only for codes along the columns; the kernel of those goes with the first one."""
    for pad, off in ((0, 0), (1, 1)):
        assert _streams(kernels, "norm", 16384, 4096, pad, off, BF, BF, WIDE) == [True]
        assert _streams(kernels, "norm", 16384, 4096, pad, off, BF, BF, ROWS) == [True]
        assert _streams(kernels, "norm", 16384, 4096, pad, off, BF, BF, BOTH) == [True, True]
        assert _streams(kernels, "norm", 16384, 4096, pad, off, BF, F32, BOTH) == [True, True]
        for a, b, out in ((BF, F32, WIDE), (BF, F32, ROWS), (F32, F32, WIDE), (F32, BF, ROWS)):
            assert _streams(kernels, "norm", 16384, 4096, pad, off, a, b, out) == [False]
        for b in (F32, BF):
            assert _streams(kernels, "norm", 16384, 4096, pad, off, F32, b, BOTH) == [False, False]
    assert _streams(kernels, "norm", 4096, 4096, 0, 0, BF, BF, BOTH) == [False, False]
    assert _streams(kernels, "norm", 16384, 4095, 1, 0, BF, BF, WIDE) == [False]


def test_norm_gradient(kernels):
    """The stream in bf16."""
    for pad, off in ((0, 0), (1, 1)):
        for dy in (BF, F32):
            assert _streams(kernels, "normgrad", 16384, 4096, pad, off, dy, BF, WIDE) == [True]
            assert _streams(kernels, "normgrad", 16384, 4096, pad, off, dy, F32, WIDE) == [False]
    assert _streams(kernels, "normgrad", 4096, 4096, 0, 0, BF, BF, WIDE) == [False]
