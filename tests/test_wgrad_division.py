"""How zero_act_wgrad divides its work, on the CPU: every stage of every tile once, and every place
that sums are kept in inside the workspace that zero_act_wgrad_workspace() names, whatever the
number of stages, the gradient's type and the number of SMs."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc needed to build")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAGE = 64                       # tokens
BF16, FP32 = 1, 2


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("wd") / "libwgrad_division_check.so"
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-shared", "-Xcompiler",
                    "-fPIC", "-I", os.path.join(ROOT, "zero_sharded_mixed_02_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "wgrad_division_check.cu"), "-o",
                    str(out)], check=True, capture_output=True)
    so = ctypes.CDLL(str(out))
    i64, i32 = ctypes.c_int64, ctypes.c_int
    so.wgrad_reach.restype = ctypes.c_uint64
    so.wgrad_reach.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i32)]
    so.zero_act_wgrad_workspace.restype = ctypes.c_uint64
    so.zero_act_wgrad_workspace.argtypes = [i64, i64, i64]
    return so


def reach(lib, tokens, n, k, grad, pairs):
    stages, run = ctypes.c_int64(), ctypes.c_int()
    return lib.wgrad_reach(tokens, n, k, grad, pairs, ctypes.byref(stages), ctypes.byref(run)), stages.value, run.value


def up(a, b):
    return -(-a // b)


# one tile, a few, about a wave of 76 pairs, several waves
SIZES = [(64, 64), (776, 771), (1600, 1600), (2048, 2432), (6400, 1600), (4096, 4096), (25000, 300)]


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("grad", [BF16, FP32])
def test_sums_are_kept_inside_the_workspace(lib, n, k, grad):
    for stages in list(range(1, 41)) + [64, 129, 469, 1024, 1025, 3001]:
        for tokens in {max(1, STAGE * (stages - 1) + 1), STAGE * stages}:
            for pairs in (1, 7, 66, 74, 76, 80):
                used, covered, _ = reach(lib, tokens, n, k, grad, pairs)
                assert covered == up(n, 256) * up(k, 256) * stages, (tokens, pairs)
                # dy's copy comes after the slots: up to eight columns' worth of two bytes a token
                copy = up(tokens * up(n, 8) * 16, 256) * 256
                assert used + copy <= lib.zero_act_wgrad_workspace(tokens, n, k), (tokens, pairs)


def test_an_accumulator_adds_a_bounded_number_of_stages(lib):
    """12 stages for fp32 gradients (15 where there is one run), 1024 for 16-bit ones."""
    for n, k in SIZES:
        for stages in (1, 12, 13, 15, 16, 17, 469, 1024, 1025, 5000, 1 << 16):
            for pairs in (1, 76):
                most = {grad: reach(lib, STAGE * stages, n, k, grad, pairs)[2] for grad in (BF16, FP32)}
                assert most[FP32] <= (stages if stages < 16 else 12) and most[BF16] <= 1024, (stages, pairs, most)
