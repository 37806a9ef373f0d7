"""The losses over the vocabulary without a GPU: workspace sizes, invalid arguments refused before anything
touches CUDA, and the 64-bit reference gradients against differences."""
import math
import shutil

import pytest

torch = pytest.importorskip("torch")
import head_reference as R  # noqa: E402

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc needed to build")
P = 1 << 20                      # an address no refused call reads


@pytest.fixture(scope="module")
def z():
    from zero_sharded_mixed_02_gb300 import build
    build.build()
    import zero_sharded_mixed_02_gb300 as z
    z.lib()
    return z


def refused(z, call, *args, **kw):
    with pytest.raises(z.ZeroError) as e:
        call(*args, **kw)
    assert e.value.code == z.ZERO_EINVAL


def description(z, **kw):
    d = dict(dtype=1, rows=4, cols=64, vocab=100, top=3)
    d.update(kw)
    return z.head(d.pop("dtype"), d.pop("rows"), d.pop("cols"), d.pop("vocab"), **d)


FORWARD = dict(x=P, ldx=64, w=P, ldw=64, labels=P, loss=P, lse=P, sums=P, work=P)
BACKWARD = dict(x=P, ldx=64, w=P, ldw=64, labels=P, lse=P, row_grad=None, scale=1.0, divisor=None, dx=P, lddx=64, dw=P,
                lddw=64, accumulate=0, work=P)
TEACHER = dict(top_index=P, top_logit=P, ldt=3)


def both(z, head, forward, backward, teacher):
    """The four calls with these arguments, each of which has to be refused."""
    if forward is not None:
        refused(z, z.zero_ce_forward, head, **forward)
        refused(z, z.zero_distill_forward, head, **forward, **teacher)
    if backward is not None:
        refused(z, z.zero_ce_backward, head, **backward)
        refused(z, z.zero_distill_backward, head, **backward, **teacher)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=-1), dict(rows=-1), dict(rows=65537), dict(cols=0), dict(cols=16385), dict(vocab=0),
    dict(vocab=(1 << 24) + 1), dict(piece=-1), dict(top=-1), dict(top=257), dict(z_loss=math.nan), dict(z_loss=math.inf)])
def test_descriptions_refused(z, bad):
    h = description(z, **bad)
    both(z, h, {**FORWARD, "ldx": 1 << 16, "ldw": 1 << 16},
         {**BACKWARD, "ldx": 1 << 16, "ldw": 1 << 16, "lddx": 1 << 16, "lddw": 1 << 16}, {**TEACHER, "ldt": 300})
    assert z.zero_head_workspace(h) == 0


@pytest.mark.parametrize("bad", [
    dict(top_dtype=3), dict(top_dtype=-1), dict(hard=math.nan), dict(soft=math.inf), dict(temperature=0.0),
    dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=math.inf), dict(temperature=1e-39), dict(top=0)])
def test_descriptions_that_only_distillation_refuses(z, bad):
    h = description(z, **bad)
    refused(z, z.zero_distill_forward, h, **FORWARD, **TEACHER)
    refused(z, z.zero_distill_backward, h, **BACKWARD, **TEACHER)
    assert z.zero_head_workspace(h) > 0
    refused(z, z.zero_ce_forward, h, **{**FORWARD, "x": None})       # (for its x, not for the description)
    z.zero_ce_forward(description(z, rows=0, **bad), **{**FORWARD, "sums": None})


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=P + 1), dict(ldx=63), dict(ldx=(1 << 31) + 1), dict(w=None), dict(w=P + 1), dict(ldw=63),
    dict(ldw=(1 << 31) + 1), dict(labels=P + 2), dict(work=None), dict(work=P + 8), dict(lse=None), dict(lse=P + 2)])
def test_refused_by_either_pass(z, bad):
    both(z, description(z), {**FORWARD, **bad}, {**BACKWARD, **bad}, TEACHER)


@pytest.mark.parametrize("bad", [dict(loss=None), dict(loss=P + 2), dict(sums=P + 2)])
def test_forward_refusals(z, bad):
    both(z, description(z), {**FORWARD, **bad}, None, TEACHER)


@pytest.mark.parametrize("bad", [
    dict(dx=None, dw=None), dict(dx=P + 1), dict(dw=P + 1), dict(lddx=63), dict(lddw=63), dict(lddx=(1 << 31) + 1),
    dict(lddw=(1 << 31) + 1), dict(row_grad=P + 2), dict(divisor=P + 1)])
def test_backward_refusals(z, bad):
    both(z, description(z), None, {**BACKWARD, **bad}, TEACHER)


def test_cross_entropy_needs_labels(z):
    refused(z, z.zero_ce_forward, description(z), **{**FORWARD, "labels": None})
    refused(z, z.zero_ce_backward, description(z), **{**BACKWARD, "labels": None})


@pytest.mark.parametrize("bad", [dict(top_index=None), dict(top_logit=None), dict(ldt=2), dict(ldt=(1 << 31) + 1),
                                 dict(top_index=P + 2), dict(top_logit=P + 2)])
def test_teacher_refusals(z, bad):
    t = {**TEACHER, **bad}
    refused(z, z.zero_distill_forward, description(z), **FORWARD, **t)
    refused(z, z.zero_distill_backward, description(z), **BACKWARD, **t)
    refused(z, z.zero_distill_forward, description(z, top=0), **FORWARD, **TEACHER)
    refused(z, z.zero_distill_backward, description(z, top=0), **BACKWARD, **TEACHER)


def test_no_description(z):
    assert z.lib().zero_head_workspace(None) == 0
    assert z.lib().zero_ce_forward(None, P, 64, P, 64, P, P, P, P, P, None) == z.ZERO_EINVAL


def test_workspace_grows_with_a_piece(z):
    small = z.zero_head_workspace(description(z, rows=8192, cols=1600, vocab=50257, piece=1024))
    large = z.zero_head_workspace(description(z, rows=8192, cols=1600, vocab=50257))
    assert 0 < small < large < 4 << 30
    # a piece of any length is cut where the vocabulary ends
    assert z.zero_head_workspace(description(z, piece=1 << 40)) == z.zero_head_workspace(description(z, piece=256))
    for rows in (0, 1, 65536):
        assert z.zero_head_workspace(description(z, rows=rows)) > 0


# ---- the reference against differences ---------------------------------------------------------------

def reference_case(distill, labels, temperature=1.7, z_loss=0.01):
    gen = torch.Generator().manual_seed(3)
    x, w = torch.randn(5, 4, generator=gen, dtype=torch.float64), torch.randn(9, 4, generator=gen, dtype=torch.float64)
    kw = dict(z_loss=z_loss, hard=0.6, soft=0.9, temperature=temperature)
    if labels:
        kw["labels"] = torch.tensor([3, -100, 8, 0, 3], dtype=torch.int32)
    if distill:
        kw["index"] = torch.tensor([[1, 3, -1], [2, 2, 4], [-1, -1, -1], [8, 0, 8], [5, 6, 7]], dtype=torch.int32)
        kw["logit"] = torch.randn(5, 3, generator=gen, dtype=torch.float64)
        kw["logit"][4, 1] = -math.inf
    return x, w, kw


@pytest.mark.parametrize("distill,labels", [(False, True), (True, True), (True, False)])
def test_reference_gradients_against_differences(distill, labels, monkeypatch):
    monkeypatch.setitem(R.EPS, torch.float64, 0.0)
    x, w, kw = reference_case(distill, labels)
    g = torch.tensor([0.5, 2.0, -1.0, 3.0, 1.0], dtype=torch.float64)
    total = lambda x, w: float((R.Case(x, w, **kw).forward()[0] * g).sum()) * 7.0 / 4.0  # noqa: E731
    c = R.Case(x, w, **kw)
    dx, dw, _, _ = c.gradient(c.forward()[1], g, 7.0, torch.tensor(4.0))
    for v, d in ((x, dx), (w, dw)):
        for at in range(v.numel()):
            h = 1e-5
            plus, minus = v.clone(), v.clone()
            plus.view(-1)[at] += h
            minus.view(-1)[at] -= h
            pair = lambda u: (u, w) if v is x else (x, u)  # noqa: E731
            assert abs((total(*pair(plus)) - total(*pair(minus))) / (2 * h) - float(d.reshape(-1)[at])) < 1e-7


def test_reference_against_autograd_and_torch():
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(6, 5, generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn(11, 5, generator=gen, dtype=torch.float64, requires_grad=True)
    y = torch.tensor([1, -100, 10, 0, 4, 4], dtype=torch.int32)
    want = torch.nn.functional.cross_entropy(x @ w.T, y.long(), reduction="none")
    got = R.Case(x.detach(), w.detach(), y).forward()[0]
    assert torch.allclose(want.detach(), got, rtol=1e-12, atol=1e-12)
