"""The bounded waits of the vocabulary head's products, made to run out: in a copy of the library's source whose
waits poll not once, every role gives up at its first wait, with copies in flight.  The calls have to end by
themselves, report ZERO_ETIMEOUT in the workspace's first word, give NaN where the sums are missing and nothing
elsewhere, and leave the context usable."""
import ctypes
import os
import subprocess
import time

import pytest

torch = pytest.importorskip("torch")
from test_gpu_head import BF16, FP16, KIND, Head, stream, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    out = tmp_path_factory.mktemp("hw") / "libhead_no_polls.so"
    csrc = os.path.join(ROOT, "zero_sharded_mixed_02_gb300", "csrc")
    # the limit of the waits for copies and products in flight at the end stays the library's
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-DZERO_HD_WAIT_LIMIT=0u",
                    "-shared", "-Xcompiler", "-fPIC", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                    *(os.path.join(csrc, f) for f in ("zero_head.cu", "zero_head_fp16.cu", "zero_head_bf16.cu")), "-o", str(out)],
                   check=True, capture_output=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("rows,cols,vocab,piece", [(40, 64, 300, 0), (700, 1600, 3000, 512), (3000, 136, 9000, 0)])
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("shift", [0, 1])
def test_calls_whose_waits_give_up(z, hasty, rows, cols, vocab, piece, dtype, shift):  # noqa: F811
    h = Head(z, rows, cols, vocab, dtype, piece=piece, shift=shift, ignored=[3])
    p = lambda v: ctypes.c_void_p(None if v is None else v.data_ptr())  # noqa: E731
    i64, f32 = ctypes.c_int64, ctypes.c_float
    loss, lse = torch.full((rows + 2,), 5.0, device="cuda"), torch.full((rows + 2,), 5.0, device="cuda")
    sums = torch.zeros(2, device="cuda")
    dx, dw = (torch.full((n, cols + 3), 5.0, dtype=KIND[dtype], device="cuda") for n in (rows, vocab))
    torch.cuda.synchronize()
    begin = time.monotonic()
    assert hasty.zero_ce_forward(ctypes.byref(h.head), p(h.x), i64(cols), p(h.w), i64(cols), p(h.labels), p(loss), p(lse), p(sums),
                                 p(h.work), ctypes.c_void_p(stream())) == z.ZERO_OK
    torch.cuda.synchronize()                                 # raises if a kernel did not end well
    assert int(h.work[:4].view(torch.int32)[0]) == z.ZERO_ETIMEOUT
    counted = torch.arange(rows, device="cuda") != 3
    for v in (loss, lse):
        assert bool(v[:rows][counted].isnan().all()) and float(v[3]) == 0.0 and bool((v[rows:] == 5.0).all())
    assert bool(sums[0].isnan())
    good = torch.zeros(rows, device="cuda")
    assert hasty.zero_ce_backward(ctypes.byref(h.head), p(h.x), i64(cols), p(h.w), i64(cols), p(h.labels), p(good), p(None), f32(1.0),
                                  p(None), p(dx), i64(cols + 3), p(dw), i64(cols + 3), 0, p(h.work),
                                  ctypes.c_void_p(stream())) == z.ZERO_OK
    torch.cuda.synchronize()
    assert time.monotonic() - begin < 30.0
    assert int(h.work[:4].view(torch.int32)[0]) == z.ZERO_ETIMEOUT
    assert bool(dw[:, :cols].isnan().all()) and bool(dx[counted][:, :cols].isnan().all()) and bool((dx[3, :cols] == 0).all())
    assert bool((dw[:, cols:] == 5.0).all()) and bool((dx[:, cols:] == 5.0).all())


def test_the_context_is_usable_afterwards(z, hasty):  # noqa: F811
    Head(z, 257, 200, 700, BF16).check()
