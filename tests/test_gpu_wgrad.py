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
