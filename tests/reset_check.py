"""Run as a program by tests/test_gpu_reset.py: the operators around residual blocks before and after
cudaDeviceReset, which destroys the process's context and with it what CUDA was told about the
library's kernels.  No torch, so that nothing else in the process holds on to the old context.
Prints OK, or what differs."""
import ctypes
import ctypes.util
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import zero_sharded_mixed_02_gb300 as z  # noqa: E402

BF16, FP32 = z.ZERO_BF16, z.ZERO_FP32


def runtime():
    for name in ("libcudart.so", "/usr/local/cuda/lib64/libcudart.so", ctypes.util.find_library("cudart")):
        try:
            return ctypes.CDLL(name)
        except (OSError, TypeError):
            pass
    print("no libcudart")
    sys.exit(77)


RT = runtime()


def check(rc, what):
    if rc:
        raise RuntimeError(f"{what}: CUDA error {rc}")


def device(a):
    """A device copy of a host array."""
    p = ctypes.c_void_p()
    check(RT.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(a.nbytes)), "cudaMalloc")
    check(RT.cudaMemcpy(p, a.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(a.nbytes), 1), "cudaMemcpy")
    return p.value


def host(p, like):
    out = np.empty_like(like)
    check(RT.cudaMemcpy(out.ctypes.data_as(ctypes.c_void_p), ctypes.c_void_p(p), ctypes.c_size_t(out.nbytes), 2), "cudaMemcpy")
    return out


def operators():
    """Weight gradient and both norm passes, on inputs of the same values each time."""
    rng = np.random.default_rng(0)
    t, n, d = 1100, 320, 4096

    def bf16(*shape):
        return (rng.standard_normal(shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    dy, h, y = bf16(t, n), bf16(t, d), bf16(t, d)
    rows16, rows8 = np.zeros((t, d), np.uint16), np.zeros((t, z.zero_act_row_bytes(d)), np.uint8)
    h_d, y_d, dy_d = device(h), device(y), device(dy)
    cx, cy, x, dh, db = device(rows8), device(rows8), device(rows16), device(rows16), device(rows16)
    st = device(np.zeros((t, 4), np.float32))
    dw, gw = np.zeros((n, d), np.float32), np.zeros(d, np.float32)
    dw_d, gw_d, g2_d = device(dw), device(gw), device(gw)
    w = device(np.full(d, 0x3F80, np.uint16))
    norm = z.norm(BF16, t, d, post=z.ZERO_NORM_LAYER, pre=z.ZERO_NORM_LAYER, post_w=w, pre_w=w, post_b=w, pre_b=w)
    work = device(np.zeros(z.zero_act_wgrad_workspace(t, n, d), np.uint8))
    work2 = device(np.zeros(z.zero_norm_workspace(norm), np.uint8))
    z.zero_norm_forward(norm, h_d, d, y_d, d, h_d, d, x, d, cy, cx, st)
    z.zero_norm_backward(norm, h_d, d, x, d, cy, cx, st, dh, d, db, d, FP32, dpost_w=gw_d, dpre_w=g2_d, work=work2)
    z.zero_act_wgrad(BF16, dy_d, t, n, n, cx, d, None, None, FP32, dw_d, d, None, 0, work)
    check(RT.cudaDeviceSynchronize(), "cudaDeviceSynchronize")
    return [host(x, rows16), host(dh, rows16), host(db, rows16), host(cx, rows8), host(gw_d, gw), host(g2_d, gw), host(dw_d, dw)]


if __name__ == "__main__":
    check(RT.cudaSetDevice(0), "cudaSetDevice")
    first = operators()
    for i in range(2):
        check(RT.cudaDeviceReset(), "cudaDeviceReset")
        again = operators()
        bad = [j for j, (a, b) in enumerate(zip(first, again)) if not np.array_equal(a, b)]
        if bad or not np.any(first[-1]):
            print("outputs differ after a reset:", bad)
            sys.exit(1)
    print("OK")
