"""How the products of the vocabulary head are divided among pairs of SMs, on the CPU: every stage of
every tile once, parts of cut tiles inside the workspace and added by the join in order, whatever the
sizes, the number of counted rows and the number of SMs."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc needed to build")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOGITS, GRADIENT, INPUT, WEIGHT = range(4)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("hd") / "libhead_division_check.so"
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-shared", "-Xcompiler",
                    "-fPIC", "-I", os.path.join(ROOT, "zero_sharded_mixed_02_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "head_division_check.cu"), "-o",
                    str(out)], check=True, capture_output=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("pass_", [LOGITS, GRADIENT, INPUT, WEIGHT])
@pytest.mark.parametrize("counted,cols,columns", [
    (0, 1, 1), (1, 1, 1), (1, 64, 256), (64, 256, 1000), (255, 768, 50257), (256, 771, 32003), (257, 1600, 4096),
    (1023, 65, 1025), (8192, 1600, 50257), (8192, 4096, 32768), (65536, 128, 600), (1, 16384, 65536), (300, 16384, 300)])
@pytest.mark.parametrize("pairs", [1, 2, 7, 76, 80])
def test_every_stage_once(lib, pass_, counted, cols, columns, pairs):
    for band in (1, 3, 24, 1000):
        assert lib.head_check(pass_, counted, cols, columns, pairs, band) == 0


def test_every_stage_once_at_random(lib):
    rng = random.Random(5)
    for _ in range(400):
        counted, cols = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 13))
        columns, pairs = int(2 ** rng.uniform(0, 16)), rng.choice([1, 3, 70, 74, 76])
        for p in range(4):
            assert lib.head_check(p, counted, cols, columns, pairs, rng.choice([1, 5, 40])) == 0, (p, counted, cols, columns, pairs)
