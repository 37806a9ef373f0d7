"""Rows of the losses over the vocabulary that take no part, rows whose weights lie far apart, and targets that
share a column, against 64 bits (head_reference.py)."""
import math

import pytest

torch = pytest.importorskip("torch")
import head_reference as R  # noqa: E402
from test_gpu_head import BF16, FP16, KIND, Head, stream, z  # noqa: E402, F401

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


# ---- weights far apart ------------------------------------------------------------------------------

def apart(z, dtype, groups, times, kw, size=1.0):  # noqa: F811
    """Rows and tokens in groups that have nothing to do with each other's softmax: token j of group k has 12 in column k, and
    so have the group's rows, so that another group's logits lie 144 lower."""
    tokens, each = 8, 4 * times
    h = Head(z, groups * each, 32 + groups, groups * tokens, dtype, **kw)
    gen = torch.Generator(device="cuda").manual_seed(7)
    of_row, of_token = (torch.arange(groups, device="cuda").repeat_interleave(n) for n in (each, tokens))
    h.w.copy_(torch.randn(h.w.shape, generator=gen, device="cuda") * 0.2)
    h.w[:, :groups] = 12.0 / size * torch.nn.functional.one_hot(of_token, groups).to(KIND[dtype])
    h.x.copy_(torch.randn(h.x.shape, generator=gen, device="cuda") * size)
    h.x[:, :groups] = 12.0 * size * torch.nn.functional.one_hot(of_row, groups).to(KIND[dtype])
    if h.labels is not None:
        h.labels.copy_(of_row * tokens + torch.randint(tokens, of_row.shape, generator=gen, device="cuda"))
    if h.top:
        h.index.copy_(of_row[:, None] * tokens + torch.randint(tokens, h.index.shape, generator=gen, device="cuda"))
    return h, of_row, of_token


@pytest.mark.parametrize("times", [1, 30])                   # up to 1024 rows, more
@pytest.mark.parametrize("kw", [{}, dict(top=3, temperature=2.0, hard=0.5, soft=0.25)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -9, 2.0 ** 10])    # of x
def test_fp16_weights_far_apart(z, times, kw, size):  # noqa: F811
    """Weights of 1 to 2^-24, a group of tokens each, whose gradients are all fp16's numbers or far from overflow.  Per
    element of dw, before its own rounding: dz's rounding (half a step, and half of its smallest number, 2^-39 of its row's
    power of two), what its logits' errors change of the probabilities, 2^-20 of the targets' weights, and the sums
    (2^-22 a step of 16 rows, 2^-20 for what follows).  And x's: where B_i is the bound of row i's dz (2 g_i of a cross
    entropy) and 2^R the largest power of two of a B_i times that of the largest |x_ik|, x times its row's power of two
    2^e <= B_i is kept below 2^16 in steps of 2^-24 at most, so that dz x is off by no more than |dz_ij| 2^(R - 40 - e)."""
    groups = 13
    h, of_row, _ = apart(z, FP16, groups, times, kw, size)
    lse = h.check_forward()
    g = torch.exp2(-2.0 * of_row.float())
    scale = 2.0 ** 9 / size / times
    _, dw = h.backward(lse, g, scale)
    _, want, _, _ = h.case().gradient(lse, g, scale)
    assert float(want.abs().max()) < 65504.0
    c, kept, eps = h.case(), lse.double(), R.EPS[torch.float16]
    (x, logits), t = c.logits(), c.temperature
    p = c.hard * (logits - (kept[:, 1:] if h.top else kept[:, None])).exp()
    weight = torch.zeros_like(p).scatter_add(1, h.labels.long()[:, None], torch.full_like(p[:, :1], c.hard))
    if h.top:
        q, at, _ = c.teacher()
        p = p + c.soft * t * (logits / t - kept[:, :1]).exp()
        weight.scatter_add_(1, at, c.soft * t * q)
    gd = g.double()[:, None]
    most = 2.0 * (c.hard + (c.soft * t if h.top else 0.0)) * gd                     # B
    e = torch.floor(torch.log2(most))
    reach = (e[:, 0] + torch.floor(torch.log2(x.abs().max(1).values))).max()
    dz = gd * (p - weight)
    off = c.logit_error(x, logits, run=1 << 30)[:, None] * 2 / min(t, 1.0)
    each = eps * dz.abs() + torch.exp2(e - 39) + gd * (p * off + 2.0 ** -20 * weight)
    sums = -(-h.rows // 16) * 2.0 ** -22 + 2.0 ** -20
    bound = each.T @ x.abs() + sums * (dz.abs().T @ x.abs()) + (dz.abs() * torch.exp2(reach - 40 - e)).sum(0)[:, None]
    R.close(dw, want, scale * bound, "dw")


def test_fp16_one_row_far_above_the_others(z):  # noqa: F811
    """Of 300 rows one has 2^20 times the others' weight and almost no loss: the others' tokens keep their gradients."""
    h, of_row, of_token = apart(z, FP16, 2, 75, {})
    h.labels[0] = 0
    h.w[0] *= 2.0                                            # token 0 is certain for group 0
    lse = h.check_forward()
    g = torch.ones(h.rows, device="cuda")
    g[0] = 2.0 ** 20
    g[1:h.rows // 2] = 0.0
    dx, dw = h.backward(lse, g, 16.0)
    want_x, want_w, bound_x, _ = h.case().gradient(lse, g, 16.0)
    R.close(dx, want_x, bound_x, "dx")
    mine = of_token == 1
    off = float((dw.double() - want_w)[mine].norm() / want_w[mine].norm())
    assert off < 2.0 ** -10, off


def test_fp16_rows_of_zeros_and_of_one_element(z):  # noqa: F811
    """The largest weight belongs to a row of zeros; other rows hold fp16's smallest and largest numbers alone."""
    h = Head(z, 70, 40, 60, FP16)
    h.x[3] = 0.0
    h.x[5], h.x[6] = 0.0, 0.0
    h.x[5, 7], h.x[6, 9] = 2.0 ** -24, 65504.0
    lse = h.check_forward()
    g = torch.full((70,), 2.0 ** -20, device="cuda")
    g[3] = 2.0 ** 100
    g[6] = 2.0 ** -30
    dx, dw = h.backward(lse, g, 16.0)
    keep = g.clone()
    keep[3] = 2.0 ** -20                                     # its x is 0 and so is its part of dw
    _, want_w, _, bound_w = h.case().gradient(lse, keep, 16.0)
    R.close(dw, want_w, bound_w, "dw")
    assert bool((dw[:, 9] != 0).any())


@pytest.mark.parametrize("rows", [60, 1500])
def test_fp16_weights_equal_bits_and_captured(z, rows):  # noqa: F811
    """Whatever the workspace holds, and in a graph; dw alone, and dx alone, whose rows are not lifted."""
    h = Head(z, rows, 136, 3000, FP16, ignored=range(0, rows, 5), piece=1024)
    lse = h.check_forward()
    g = torch.exp2(-20.0 * torch.rand(rows, device="cuda"))
    first = h.check_backward(lse, row_grad=g, scale=64.0)
    for _ in range(5):
        h.space[:h.work.numel()].random_(0, 256)
        assert all(torch.equal(a, b) for a, b in zip(first, h.backward(lse, g, 64.0)))
    for want in ((True, False), (False, True)):
        h.space[:h.work.numel()].random_(0, 256)
        one = h.backward(lse, g, 64.0, want=want)
        assert all(torch.equal(a, b) for a, b, w in zip(first, one, want) if w)
    dx, dw = torch.zeros_like(h.x), torch.zeros_like(h.w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_ce_backward(h.head, h.x, 136, h.w, 136, h.labels, lse, g, 64.0, None, dx, 136, dw, 136, 0, h.work, stream())
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])


# ---- what dx gets back of dz's rounding ------------------------------------------------------------

def gradient_of_inputs(h, lse, rows):
    """dx of these rows in the 2-norm: its own rounding, and of dz's what the heavy columns leave (those with a quarter of
    the row's weight or more), eps / sqrt(3) of it in the mean square.  A tenth for chance.  The rows' weights put what the
    targets get of dz, some -1, just above a power of two, where rounding it costs most."""
    g = 1.02 + 0.2 * torch.rand(h.rows, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    dx, _ = h.backward(lse, g, 64.0)
    c = h.case()
    want, _, _, _ = c.gradient(lse, g, 64.0)
    (x, logits), t = c.logits(), c.temperature
    kept, weight = lse.double(), torch.zeros_like(logits)
    dz = torch.zeros_like(logits)
    q, at, has = c.teacher()
    weight.scatter_add_(1, at, c.soft * t * q)
    dz += c.soft * t * (logits / t - kept[:, :1]).exp() * has[:, None]
    if h.labels is not None:
        weight.scatter_add_(1, h.labels.long()[:, None], torch.full_like(logits[:, :1], c.hard))
        dz += c.hard * (logits - kept[:, 1:]).exp()
    dz = (dz - weight) * g.double()[:, None]
    heavy = weight >= weight.sum(1, keepdim=True) * 0.25
    rho = float((dz * ~heavy)[rows].square().sum() / dz[rows].square().sum())
    off = lambda got: float((got.double() - want)[rows].norm() / want[rows].norm())  # noqa: E731
    assert rho < 0.3
    eps = R.EPS[KIND[h.dtype]]
    assert off(dx) < 1.1 * math.sqrt(off(want.to(KIND[h.dtype])) ** 2 + rho * eps ** 2 / 3), (off(dx), rho)


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_rows_of_which_the_teacher_kept_nothing(z, dtype):  # noqa: F811
    """All of their weight is the label's; others have some absent entries."""
    h = Head(z, 600, 512, 2000, dtype, spread=1.0, top=6, temperature=2.0, hard=0.5, soft=0.5)
    h.index[:300] = -1
    h.index[300:400, 3:] = -1
    h.logit[:300], h.logit[300:400, 3:] = math.nan, -math.inf
    lse = h.check_forward()
    gradient_of_inputs(h, lse, slice(0, 300))


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_a_light_label_on_a_heavy_entry(z, dtype):  # noqa: F811
    h = Head(z, 600, 512, 2000, dtype, spread=1.0, top=6, temperature=2.0, hard=0.1, soft=0.45)
    h.logit[:, 2] += 12.0
    h.labels.copy_(h.index[:, 2])
    gradient_of_inputs(h, h.check_forward(), slice(None))


@pytest.mark.parametrize("labels", [False, True])
def test_entries_of_one_column_that_are_light_alone(z, labels):  # noqa: F811
    """Of nine equal entries five are one column, which has more than half of the weight; the others none has a quarter of."""
    h = Head(z, 600, 512, 2000, BF16, spread=1.0, top=9, temperature=1.0, labels=labels, hard=0.1, soft=1.0)
    h.logit[:] = 4.0
    h.index[:, 4:9] = h.index[:, 4:5]
    gradient_of_inputs(h, h.check_forward(), slice(None))


# ---- captured after work that is not a kernel of the same stream --------------------------------------

@pytest.mark.parametrize("rows", [16, 300, 1300])
@pytest.mark.parametrize("before", ["nothing", "copy", "clear", "two streams"])
def test_captured_behind_other_work(z, rows, before):  # noqa: F811
    """The first kernel of few rows' calls may begin early; behind whatever a graph holds it waits for all of it."""
    h = Head(z, rows, 136, 1500, BF16)
    source = h.x.clone()
    want_loss, want_lse, _ = h.forward()
    want = h.backward(want_lse)
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    dx, dw = torch.zeros_like(h.x), torch.zeros_like(h.w)
    other = torch.cuda.Stream()
    big = torch.zeros(1 << 26, device="cuda")

    def step():
        if before == "copy":
            h.x.copy_(source)
        elif before == "clear":
            big.add_(1.0)
            h.x.zero_()
            h.x.add_(source)
            loss.zero_()
        elif before == "two streams":
            mine = torch.cuda.current_stream()
            other.wait_stream(mine)
            h.x.zero_()
            with torch.cuda.stream(other):
                big.add_(1.0)
                h.w.mul_(1.0)
            h.x.add_(source)
            mine.wait_stream(other)
        z.zero_ce_forward(h.head, h.x, 136, h.w, 136, h.labels, loss, lse, None, h.work, stream())
        z.zero_ce_backward(h.head, h.x, 136, h.w, 136, h.labels, lse, None, 1.0, None, dx, 136, dw, 136, 0, h.work, stream())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (loss, lse, dx, dw):
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((loss, lse, dx, dw), (want_loss, want_lse, *want)):
            assert torch.equal(a, b)
