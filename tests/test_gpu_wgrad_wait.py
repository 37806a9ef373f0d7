"""The weight gradient's bounded waits, made to run out: in a copy of the library's source whose
waits poll not once, every role of the kernel gives up at its first wait, with copies in flight.
The call has to end by itself, report ZERO_ETIMEOUT in the workspace's first word, write NaN where
the sums are missing and nothing elsewhere, and leave the context usable."""
import ctypes
import os
import subprocess
import time

import numpy as np
import pytest

import act_reference as R
from test_gpu_act import env, kind, wgrad_case  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    out = tmp_path_factory.mktemp("ww") / "libwgrad_no_polls.so"
    csrc = os.path.join(ROOT, "zero_sharded_mixed_02_gb300", "csrc")
    # the limit of the waits for copies and products in flight at the end stays the library's
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-DZERO_WG_WAIT_LIMIT=0u",
                    "-shared", "-Xcompiler", "-fPIC", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                    os.path.join(csrc, "zero_wgrad.cu"), "-o", str(out)], check=True, capture_output=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("tokens,n,k", [(300, 300, 300), (20000, 64, 200), (130, 2500, 5000), (1500, 520, 520)])
@pytest.mark.parametrize("dtype,grad", [(R.BF16, R.BF16), (R.FP16, R.FP32)])
@pytest.mark.parametrize("affine", [False, True])
def test_a_call_whose_waits_give_up(env, hasty, tokens, n, k, dtype, grad, affine):  # noqa: F811
    torch, z = env
    t = kind(torch, dtype)
    dy, x = torch.randn(tokens, n, device="cuda").to(t), torch.randn(tokens, k, device="cuda").to(t)
    scale, shift = (torch.randn(k, device="cuda").to(t) for _ in range(2))
    ckpt = torch.empty(tokens, z.zero_act_row_bytes(k), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    z.zero_act_save(dtype, x, tokens, k, k, ckpt, s)
    dw = torch.full((n, k + 3), 5.0, dtype=kind(torch, grad), device="cuda")
    db = torch.full((n + 3,), 5.0, dtype=kind(torch, grad), device="cuda")
    work = torch.zeros(z.zero_act_wgrad_workspace(tokens, n, k), dtype=torch.uint8, device="cuda")
    p = lambda v: ctypes.c_void_p(v.data_ptr() if v is not None else None)  # noqa: E731
    i64 = ctypes.c_int64
    torch.cuda.synchronize()
    begin = time.monotonic()
    rc = hasty.zero_act_wgrad(dtype, p(dy), i64(tokens), i64(n), i64(n), p(ckpt), i64(k), p(scale if affine else None),
                              p(shift if affine else None), grad, p(dw), i64(k + 3), p(db), 0, p(work),
                              ctypes.c_void_p(s))
    torch.cuda.synchronize()                                 # raises if the kernel did not end well
    assert rc == z.ZERO_OK and time.monotonic() - begin < 30.0
    assert int(work[:4].view(torch.int32)[0]) == z.ZERO_ETIMEOUT
    assert bool(dw[:, :k].isnan().all()) and bool((dw[:, k:] == 5.0).all()) and bool((db[n:] == 5.0).all())
    # with the norm's bias and more than one column of tiles the sums of dy come from a pass of their own
    have = db[:n].float()
    if affine and k > 256:
        assert np.allclose(have.cpu().numpy(), dy.float().sum(0).cpu().numpy(), rtol=0.01, atol=0.01 * tokens ** 0.5)
    else:
        assert bool(have.isnan().all())


def test_the_context_is_usable_afterwards(env, hasty):  # noqa: F811
    wgrad_case(env, 1500, 520, 520, R.BF16, R.FP32)
