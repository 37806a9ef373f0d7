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
