"""Rows of the losses over the vocabulary that take no part, against 64 bits (head_reference.py)."""
import math

import pytest

torch = pytest.importorskip("torch")
import head_reference as R  # noqa: E402
from test_gpu_head import BF16, Head, z  # noqa: E402, F401

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
