"""The weight gradient's sums in its workspace: nothing is written past the bytes that
zero_act_wgrad_workspace() names, at the numbers of tokens where a call begins to keep sums there."""
import pytest

import act_reference as R
from test_gpu_act import env, wgrad_case  # noqa: F401

pytestmark = pytest.mark.gpu


def guarded(torch, z, tokens, n, k):
    """A workspace at the head of a buffer 64 MB larger (more than all slots take), and the rest."""
    size = z.zero_act_wgrad_workspace(tokens, n, k)
    buf = torch.full((size + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    buf[:size] = 0
    return buf, buf[size:]


@pytest.mark.parametrize("tokens", [768, 769, 832, 896, 900, 960, 961])
@pytest.mark.parametrize("n,k,pad,shift,accumulate", [(776, 771, 0, 0, 0), (300, 520, 1, 1, 1), (1600, 520, 0, 0, 1),
                                                      (2500, 4000, 0, 0, 0), (25000, 300, 1, 0, 0)])
@pytest.mark.parametrize("grad", [R.BF16, R.FP32])
def test_nothing_past_the_workspace(env, tokens, n, k, pad, shift, accumulate, grad):  # noqa: F811
    torch, z = env
    work, rest = guarded(torch, z, tokens, n, k)
    wgrad_case(env, tokens, n, k, R.BF16, grad, pad=pad, shift=shift, dw_pad=pad, dw_shift=shift, accumulate=accumulate,
               work=work)
    assert bool((rest == 0xA5).all())


def test_a_very_long_token_axis_keeps_the_types_precision(env):  # noqa: F811
    """1 M tokens against a matrix of more whole tiles than the device takes at a time.  fp16's rounding
    alone is off by 2^-11 / sqrt(3) of the values' 2-norm at most.  The tensor cores' accumulators cut off
    up to 2^-23, on average 2^-24, of a sum at each step of 16 tokens; a sum of random terms grows with the
    root of the steps, which makes 2/3 of that a step, and an accumulator adds at most 65536 tokens."""
    torch, z = env
    tokens, n, k, rows, cols = 1 << 20, 2560, 2048, 64, 256
    gen = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.empty(tokens, n, dtype=torch.float16, device="cuda").normal_(0, 0.05, generator=gen)
    x = torch.empty(tokens, k, dtype=torch.float16, device="cuda").normal_(generator=gen)
    ckpt = torch.empty(tokens, z.zero_act_row_bytes(k), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    z.zero_act_save(R.FP16, x, tokens, k, k, ckpt, s)
    z.zero_act_load(R.FP16, ckpt, tokens, k, x, k, s)
    dw = torch.empty(n, k, dtype=torch.float16, device="cuda")
    work = torch.zeros(z.zero_act_wgrad_workspace(tokens, n, k), dtype=torch.uint8, device="cuda")
    z.zero_act_wgrad(R.FP16, dy, tokens, n, n, ckpt, k, None, None, R.FP16, dw, k, None, 0, work, s)
    want = dy[:, :rows].double().T @ x[:, :cols].double()
    rel = float((dw[:rows, :cols].double() - want).norm() / want.norm())
    assert rel <= 2.0 ** -11 / 3 ** 0.5 + 65536 / 16 * 2.0 ** -24 * 2 / 3, rel


def truncation(steps):
    """2-norm error of an accumulator that cuts a random sum off at each of so many steps of 16 tokens, at
    most: 2^-24 of the sum as it stands on average, which grows with the root of the steps."""
    return steps * 2.0 ** -24 * 2 / 3


@pytest.mark.parametrize("tokens,n,k", [(30011, 776, 771), (832, 1600, 520), (960, 2500, 4000), (7000, 2600, 2000), (20000, 64, 64)])
@pytest.mark.parametrize("dtype", [R.BF16, R.FP16])
def test_fp32_gradients_are_summed_in_short_runs(env, tokens, n, k, dtype):  # noqa: F811
    """At most 12 stages of four steps an accumulator (15 where there is one run), then rounded sums of the
    runs and parts, a walk of at most 2^-24 a sum.  Runs of 64 stages are off by 3.8e-6 at 30011 tokens."""
    torch, z = env
    t = torch.float16 if dtype == R.FP16 else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(tokens + n)
    dy = (0.05 * torch.randn(tokens, n, device="cuda", generator=gen)).to(t)
    x = torch.randn(tokens, k, device="cuda", generator=gen).to(t)
    s = torch.cuda.current_stream().cuda_stream
    ckpt = torch.empty(tokens, z.zero_act_row_bytes(k), dtype=torch.uint8, device="cuda")
    z.zero_act_save(dtype, x, tokens, k, k, ckpt, s)
    xq = torch.empty(tokens, k, device="cuda")
    z.zero_act_load(R.FP32, ckpt, tokens, k, xq, k, s)
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    work = torch.zeros(z.zero_act_wgrad_workspace(tokens, n, k), dtype=torch.uint8, device="cuda")
    z.zero_act_wgrad(dtype, dy, tokens, n, n, ckpt, k, None, None, R.FP32, dw, k, db, 0, work, s)
    stages = -(-tokens // 64)
    bound = truncation(4 * (12 if stages >= 16 else stages)) + (2 + stages / 12) ** 0.5 * 2.0 ** -24
    want = dy.double().T @ xq.double()
    assert float((dw.double() - want).norm() / want.norm()) <= bound
    # the sums of dy are rounded at every step, in runs as short and shorter
    want = dy.double().sum(0)
    assert float((db.double() - want).norm() / want.norm()) <= bound


@pytest.mark.parametrize("tokens,n,k", [(100, 300, 500), (700, 257, 300), (900, 300, 777), (5000, 300, 129)])
@pytest.mark.parametrize("dtype,grad", [(R.BF16, R.BF16), (R.FP16, R.FP32)])
@pytest.mark.parametrize("pad,shift,dw_pad,dw_shift", [(1, 1, 3, 1), (0, 0, 1, 0), (8, 0, 0, 3)])
def test_accumulation_into_rows_of_any_alignment(env, tokens, n, k, dtype, grad, pad, shift, dw_pad, dw_shift):  # noqa: F811
    wgrad_case(env, tokens, n, k, dtype, grad, pad=pad, shift=shift, affine=True, dw_pad=dw_pad, dw_shift=dw_shift,
               accumulate=1)
