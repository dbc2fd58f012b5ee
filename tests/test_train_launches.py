"""What libmxfp4_train launches for the largest sizes that it takes, and that it refuses the others before it launches anything:
its host code, driven by tests/train_launches.c, which stands in for the HIP runtime (no GPU)."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, SHAPE = 0, 2
CARD = 288 * 1024 ** 3          # bytes of memory


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    import mxfp4_block_scaled_h16_amd as mx
    from mxfp4_block_scaled_h16_amd import build
    mx.train_lib()
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(build.hipcc())))
    exe = str(tmp_path_factory.mktemp("train_launches") / "train_launches")
    here = os.path.dirname(build.TRAIN_LIB)
    subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-I" + os.path.join(rocm, "include"),
                    os.path.join(ROOT, "tests", "train_launches.c"), build.TRAIN_LIB, "-rdynamic", "-Wl,-rpath," + here,
                    "-Wl,-rpath," + os.path.join(rocm, "lib"), "-L" + os.path.join(rocm, "lib"), "-lamdhip64", "-o", exe], check=True)

    def calls(lines):
        """(status, launches, launches beyond a grid, workspace bytes) of each 'name a b c'."""
        r = subprocess.run([exe], input="\n".join("%s %d %d %d" % line for line in lines) + "\n", capture_output=True, text=True,
                           timeout=120, check=True)
        out = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return out
    return calls


def _sound(line, got):
    status, launches, beyond, need = got
    if status == SHAPE:
        assert launches == 0 and need == 0, (line, got)
    else:
        assert status == OK and launches > 0 and beyond == 0, (line, got)


def test_ordinary_sizes(run):
    lines = [("quantize1", 8192, 4096, 0), ("quantize0", 8192, 4096, 0), ("gemm", 8192, 6144, 4096), ("fprop", 1111, 1000, 2001),
             ("wgrad", 8192, 14336, 4096), ("forward", 1537, 1000, 50257), ("backward", 8192, 4096, 128256),
             ("orthogonalize", 2, 1024, 4096)]
    for line, got in zip(lines, run(lines)):
        assert got[0] == OK and got[1] > 0 and got[2] == 0, (line, got)


@pytest.mark.parametrize("T,K,V", [((1 << 21) - 1, 64, 1 << 18), ((1 << 21) - 1, 64, 1 << 20), (1 << 20, 64, 1 << 21), (4096, 64, 1 << 29),
                                   (1, 1, (1 << 31) - 1), (300, 64, (1 << 31) - 1)])
def test_the_loss_of_more_tiles_than_a_grid(run, T, K, V):
    """The head's loss keeps no logits, so T and V may be large together: all of these fit the card's memory."""
    got = run([("forward", T, K, V)])[0]
    assert got[0] == OK and got[1] > 2 and got[2] == 0 and got[3] + 2 * (T + V) * K <= CARD


def test_products_and_quantizations_of_more_tiles_than_a_grid(run):
    big = (1 << 31) - 1
    lines = [("quantize0", big, 1, 0), ("quantize1", 1, big, 0), ("quantize1", (1 << 24) - 1 << 7, 1, 0), ("gemm", big, 1, 128),
             ("gemm", 1, big, 1), ("gemm", big, big, 1), ("fprop", 1 << 23, 1 << 23, 1 << 23), ("wgrad", 1, 1 << 23, 1 << 23),
             ("wgrad", 1 << 23, 1 << 23, 1), ("orthogonalize", 65535, 1, 32768), ("orthogonalize", 65535, 32768, 1),
             ("orthogonalize", 1, 1 << 20, 2048), ("orthogonalize", 65535, 181, 181)]
    for line, got in zip(lines, run(lines)):
        _sound(line, got)
    got = dict(zip(lines, run(lines)))
    assert got[("quantize1", (1 << 24) - 1 << 7, 1, 0)][0] == OK
    assert got[("quantize0", big, 1, 0)][0] == SHAPE and got[("gemm", big, 1, 128)][0] == SHAPE


def test_random_sizes(run):
    """Every accepted call's launches are launches; sizes over the whole documented ranges, operands that fit the card."""
    rng = random.Random(5)

    def size(top):
        return min(top, max(1, int(2.0 ** rng.uniform(0.0, top.bit_length()))))
    lines = []
    while len(lines) < 3000:
        name = rng.choice(["quantize1", "quantize0", "gemm", "fprop", "wgrad", "forward", "backward", "orthogonalize"])
        if name.startswith("quantize"):
            a, b, c = size((1 << 31) - 1), size((1 << 31) - 1), 0
            fits = a * b * 2
        elif name == "gemm":
            a, b, c = size((1 << 31) - 1), size((1 << 31) - 1), size((1 << 23) - 1)
            fits = 2 * a * b + (a + b) * c
        elif name in ("fprop", "wgrad"):
            a, b, c = (size(1 << 23) for _ in range(3))
            fits = 2 * (a * b + b * c + a * c)
        elif name == "orthogonalize":
            a, b, c = size(65535), size(1 << 20), size(1 << 20)
            if a * b * c > 1 << 31:
                continue
            fits = 4 * a * b * c
        else:
            a, b, c = size((1 << 21) - 1), size((1 << 21) - 1), size((1 << 31) - 1)
            fits = 2 * (a * b + b * c)
        if fits <= CARD:
            lines.append((name, a, b, c))
    for line, got in zip(lines, run(lines)):
        _sound(line, got)
