"""Run as a program by tests/test_gpu_head_process.py.  `reset`: the vocabulary head's losses before and after
cudaDeviceReset, without torch, so that nothing else in the process holds on to the old context.  `capture`: their first
call of the process captured into a CUDA graph.  Prints OK, or what differs."""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))


def reset():
    from reset_check import BF16, RT, check, device, host, z

    def losses():
        rng = np.random.default_rng(0)
        n, d, v = 1300, 264, 3000
        x, w = ((rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16) for s in ((n, d), (v, d)))
        labels, rows = rng.integers(0, v, n).astype(np.int32), np.zeros(n, np.float32)
        head = z.head(BF16, n, d, v, piece=1024)
        x_d, w_d, y_d, loss, lse = device(x), device(w), device(labels), device(rows), device(rows)
        dx, dw, work = device(x), device(w), device(np.zeros(z.zero_head_workspace(head), np.uint8))
        z.zero_ce_forward(head, x_d, d, w_d, d, y_d, loss, lse, None, work)
        z.zero_ce_backward(head, x_d, d, w_d, d, y_d, lse, None, 1.0, None, dx, d, dw, d, 0, work)
        check(RT.cudaDeviceSynchronize(), "cudaDeviceSynchronize")
        return [host(loss, rows), host(lse, rows), host(dx, x), host(dw, w)]

    check(RT.cudaSetDevice(0), "cudaSetDevice")
    first = losses()
    for _ in range(2):
        check(RT.cudaDeviceReset(), "cudaDeviceReset")
        bad = [j for j, (a, b) in enumerate(zip(first, losses())) if not np.array_equal(a, b)]
        if bad or not np.all(np.isfinite(first[0])) or not np.any(first[-1]):
            print("outputs differ after a reset:", bad)
            sys.exit(1)


def capture():
    import torch
    import zero_sharded_mixed_02_gb300 as z
    z.lib()
    n, d, v = 300, 136, 5000
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, w = (torch.randn(s, d, generator=gen, device="cuda").bfloat16() for s in (n, v))
    labels = torch.randint(v, (n,), generator=gen, device="cuda").to(torch.int32)
    head = z.head(z.ZERO_BF16, n, d, v)
    work = torch.empty(z.zero_head_workspace(head), dtype=torch.uint8, device="cuda")
    loss, lse, dx, dw = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros_like(x), torch.zeros_like(w)

    def step():
        s = torch.cuda.current_stream().cuda_stream
        z.zero_ce_forward(head, x, d, w, d, labels, loss, lse, None, work, s)
        z.zero_ce_backward(head, x, d, w, d, labels, lse, None, 1.0, None, dx, d, dw, d, 0, work, s)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert not bool(loss.any())                              # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (loss, lse, dx, dw)]
    step()
    torch.cuda.synchronize()
    bad = [j for j, (a, b) in enumerate(zip(got, (loss, lse, dx, dw))) if not torch.equal(a, b)]
    if bad or not bool(got[0].isfinite().all()) or not bool(got[0].any()):
        print("outputs differ:", bad)
        sys.exit(1)


if __name__ == "__main__":
    {"reset": reset, "capture": capture}[sys.argv[1]]()
    print("OK")
