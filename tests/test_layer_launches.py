"""What libmxfp4_layer launches for the largest sizes that it takes, and that it refuses the others before it launches anything:
its host code, driven by tests/layer_launches.c, which stands in for the HIP runtime (no GPU)."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, SHAPE = 0, 2
CARD = 288 * 1024 ** 3          # bytes of memory
ROWS, COLS = 1, 2               # codes along them


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    import mxfp4_block_scaled_h16_amd as mx
    from mxfp4_block_scaled_h16_amd import build
    mx.layer_lib()
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(build.hipcc())))
    exe = str(tmp_path_factory.mktemp("layer_launches") / "layer_launches")
    here = os.path.dirname(build.LAYER_LIB)
    subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-I" + os.path.join(rocm, "include"),
                    os.path.join(ROOT, "tests", "layer_launches.c"), build.LAYER_LIB, "-rdynamic", "-Wl,-rpath," + here,
                    "-Wl,-rpath," + os.path.join(rocm, "lib"), "-L" + os.path.join(rocm, "lib"), "-lamdhip64", "-o", exe], check=True)

    def calls(lines):
        """(status, launches, launches beyond a grid, workspace bytes) of each 'name a b c'."""
        r = subprocess.run([exe], input="\n".join("%s %d %d %d" % line for line in lines) + "\n", capture_output=True, text=True,
                           timeout=120, check=True)
        out = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return out
    return calls


def test_launches_of_ordinary_sizes(run):
    want = {("norm", 8192, 4096, ROWS): 1, ("norm", 8192, 4096, ROWS + COLS): 2, ("norm", 1, 100000, ROWS): 1, ("normgrad", 8192, 4096, 0): 2,
            ("normgrad", 0, 300, 0): 1, ("gate", 8192, 14336, ROWS + COLS): 1, ("gategrad", 8192, 14336, ROWS + COLS): 1,
            ("gate", 0, 300, ROWS): 0, ("clip", 1, 1000, 0): 2, ("clip", 160, 10, 0): 2, ("clip", 161, 10, 0): 3, ("clip", 224, 10, 0): 3, ("clip", 225, 10, 0): 4, ("clip", 0, 1, 0): 1,
            ("clip", 224 * 9, 1 << 24, 0): 9 + 1 + 13, ("scale", 321, 1000, 0): 3, ("scale", 0, 1, 0): 1, ("sum", 300, 1000, 0): 3, ("sum", 0, 1, 0): 1}
    for (line, launches), got in zip(want.items(), run(list(want))):
        assert got[:3] == (OK, launches, 0), (line, got)


def test_the_largest_sizes(run):
    big = (1 << 31) - 1
    fits = [("norm", big, 1, ROWS), ("norm", 1, 1 << 24, ROWS + COLS), ("norm", big, 1 << 24, ROWS), ("norm", ((1 << 23) - 1) * 128, 128, COLS),
            ("normgrad", big, 1 << 24, 0), ("normgrad", big, 1, 0), ("gate", ((1 << 23) - 1) * 128, 1, ROWS + COLS),
            ("gategrad", 1, ((1 << 23) - 1) * 128, ROWS + COLS), ("clip", 1, 1 << 37, 0), ("clip", 300, 1 << 37, 0), ("clip", (1 << 20) - 1, 1, 0)]
    for line, got in zip(fits, run(fits)):
        assert got[0] == OK and got[1] > 0 and got[2] == 0, (line, got)
    refused = [("norm", big, 128, COLS), ("norm", 1 << 31, 1, 0), ("norm", 1, (1 << 24) + 1, 0), ("normgrad", 1, (1 << 24) + 1, 0), ("gate", big, 128, 0),
               ("gate", (1 << 23) * 128 + 1, 128, ROWS), ("gategrad", 1, big, COLS), ("clip", 1, (1 << 37) + 1, 0), ("clip", 1 << 20, 1, 0)]
    for line, got in zip(refused, run(refused)):
        assert got == (SHAPE, 0, 0, 0), (line, got)


def test_random_sizes(run):
    """Every accepted call's launches are launches; sizes over the whole documented ranges, operands that fit the card."""
    rng = random.Random(7)

    def size(top):
        return min(top, max(1, int(2.0 ** rng.uniform(0.0, top.bit_length()))))
    lines = []
    while len(lines) < 3000:
        name = rng.choice(["norm", "normgrad", "gate", "gategrad", "clip"])
        a, b, c = size((1 << 31) - 1), size(1 << 24 if name.startswith("norm") else (1 << 31) - 1), rng.randrange(4)
        if name == "clip":
            a = size(5000)
        if a * b * 4 <= CARD and (c or not name.startswith("gate")):
            lines.append((name, a, b, c))
    for line, got in zip(lines, run(lines)):
        if got[0] == SHAPE:
            assert got[1] == 0 and got[3] == 0, (line, got)
        else:
            assert got[0] == OK and got[1] > 0 and got[2] == 0, (line, got)
