"""Rows of the losses over the vocabulary that take no part, against 64 bits (head_reference.py)."""
import math

import pytest

torch = pytest.importorskip("torch")
import head_reference as R  # noqa: E402
from test_gpu_head import BF16, FP16, Head, stream, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# ---- rows of no weight ------------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [300, 1500])                # one chunk of rows, several
@pytest.mark.parametrize("top,labels", [(0, True), (5, True), (5, False)])
@pytest.mark.parametrize("z_loss", [0.0, 0.01])
def test_rows_of_no_weight_whose_loss_is_not_finite(z, rows, top, labels, z_loss):  # noqa: F811
    """Their x is not finite when the forward pass runs, so their log-sum-exp is not either; others have a label
    past the vocabulary."""
    kw = dict(top=top, labels=labels, temperature=1.5, hard=0.5, soft=0.5) if top else {}
    h = Head(z, rows, 72, 500, BF16, z_loss=z_loss, **kw)
    clean, clean_lse = h.x.clone(), h.check_forward().clone()
    nan, inf, past = slice(10, 20), slice(20, 30), slice(30, 33)
    h.x[nan], h.x[inf] = math.nan, math.inf
    keep = None
    if labels:
        keep = h.labels.clone()
        h.labels[past] = 500
    lse = h.forward()[1]
    assert bool(lse[10:30].isnan().reshape(20, -1).any(1).all()) and (not labels or bool(lse[past].isnan().any()))
    lse = lse.clone()
    lse[25:30] = math.inf
    g = torch.rand(rows, device="cuda") + 0.5
    g[10:33] = 0.0
    g[15:20] = -0.0
    dx, dw = h.backward(lse, g, 3.0)
    h.x.copy_(clean)
    if labels:
        h.labels.copy_(keep)
    lse[10:33] = clean_lse[10:33]
    want_x, want_w, bound_x, bound_w = h.case().gradient(lse, g, 3.0)
    assert bool(bound_x.isfinite().all()) and bool(bound_w.isfinite().all())
    assert bool((dx[10:33] == 0).all())
    R.close(dx, want_x, bound_x, "dx")
    R.close(dw, want_w, bound_w, "dw")


# ---- no row that counts -----------------------------------------------------------------------------

@pytest.mark.parametrize("scale,divisor", [(math.inf, 1.0), (math.nan, 1.0), (1.0, math.nan), (1.0, 0.0), (1e38, 1e-30)])
@pytest.mark.parametrize("rows", [40, 2100])                 # 2100: where rows count, tiles are cut along them
def test_no_row_counts_and_the_factor_is_not_finite(z, scale, divisor, rows):  # noqa: F811
    """A sum over no rows is 0 whatever it is multiplied with."""
    h = Head(z, rows, 72, 3000, FP16, ignored=range(rows))
    lse = torch.zeros(rows, device="cuda")
    d = torch.tensor([divisor], device="cuda")
    dx, dw = h.backward(lse, None, scale, d)
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    before = torch.randn(3000, 72, device="cuda").half()
    assert torch.equal(h.backward(lse, None, scale, d, accumulate=before)[1], before)


@pytest.mark.parametrize("lddw", [1 << 30, 1 << 31])
def test_no_rows_and_rows_of_the_gradient_far_apart(z, lddw):  # noqa: F811
    h = z.head(BF16, 0, 64, 2)
    work = torch.empty(z.zero_head_workspace(h), dtype=torch.uint8, device="cuda")
    dw = torch.full((lddw + 72,), 3.0, dtype=torch.bfloat16, device="cuda")
    z.zero_ce_backward(h, None, 64, dw, 64, None, None, None, 1.0, None, None, 64, dw, lddw, 0, work, stream())
    for at in (0, lddw):
        assert bool((dw[at:at + 64] == 0).all())
    assert bool((dw[64:72] == 3.0).all()) and bool((dw[lddw - 8:lddw] == 3.0).all()) and bool((dw[lddw + 64:] == 3.0).all())


def test_no_rows_and_odd_places(z):  # noqa: F811
    for cols, ld, shift in ((1, 1, 0), (5, 9, 1), (8, 8, 0), (771, 773, 3), (4096, 4104, 0)):
        h = z.head(FP16, 0, cols, 1003)
        work = torch.empty(z.zero_head_workspace(h), dtype=torch.uint8, device="cuda")
        dw = torch.full((1003 * ld + shift + 8,), 3.0, dtype=torch.float16, device="cuda")
        z.zero_ce_backward(h, None, cols, dw, cols, None, None, None, 1.0, None, None, cols, dw[shift:], ld, 0, work, stream())
        inner = dw[shift:shift + 1003 * ld].view(1003, ld)
        assert bool((inner[:, :cols] == 0).all())
        inner[:, :cols] = 3.0
        assert bool((dw == 3.0).all())
