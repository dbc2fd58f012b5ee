"""What libmxfp4_train launches for the largest sizes that it takes: its host code, driven by tests/train_launches.c, which stands
in for the HIP runtime (no GPU)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK = 0
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
