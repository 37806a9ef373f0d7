"""The losses over the vocabulary on the GPU against 64 bits (head_reference.py), at the sizes, strides and masks
where they can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")
import head_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu
FP16, BF16, FP32 = 0, 1, 2
KIND = {FP16: torch.float16, BF16: torch.bfloat16, FP32: torch.float32}
GUARD = 77                       # bytes around and between what a call may write


@pytest.fixture(scope="module")
def z():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zero_sharded_mixed_02_gb300 as z
    z.lib()
    return z


def stream():
    return torch.cuda.current_stream().cuda_stream


def matrix(rows, cols, dtype, pad=0, shift=0, fill=0.0):
    """A [rows][cols] view `shift` elements into a buffer whose rows are cols + pad apart, and the buffer."""
    buf = torch.full((rows * (cols + pad) + shift + 8,), fill, dtype=KIND[dtype], device="cuda")
    return buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


class Head:
    """A case and its calls."""

    def __init__(self, z, rows, cols, vocab, dtype=BF16, seed=0, ignored=None, top=0, top_dtype=FP32, labels=True, pad=0, shift=0,
                 spread=2.0, **kw):
        self.z, self.rows, self.cols, self.vocab, self.dtype = z, rows, cols, vocab, dtype
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.ld = cols + pad
        self.x, self.x_buf = matrix(rows, cols, dtype, pad, shift)
        self.w, self.w_buf = matrix(vocab, cols, dtype, pad, shift)
        self.w.copy_(rand(vocab, cols) * (spread / math.sqrt(cols)))
        self.labels = self.index = self.logit = None
        y = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        self.x.copy_(rand(rows, cols) + 2.0 * self.w[y].float())
        if labels:
            self.labels = y.to(torch.int32)
            if ignored is not None:
                self.labels[torch.as_tensor(ignored, device="cuda", dtype=torch.long)] = -100
        if top:
            self.index = torch.randint(vocab, (rows, top), generator=gen, device="cuda").to(torch.int32)
            self.logit = (rand(rows, top) * 2 + 5).to(KIND[top_dtype])
        head_kw = {k: kw[k] for k in ("z_loss", "hard", "soft", "temperature") if k in kw}
        self.args = head_kw
        self.head = z.head(dtype, rows, cols, vocab, piece=kw.get("piece", 0), top=top, top_dtype=top_dtype, **head_kw)
        need = z.zero_head_workspace(self.head)
        assert need > 0
        self.space = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        self.work = self.space[:need]
        self.top = top

    def case(self):
        return R.Case(self.x, self.w, self.labels, self.index, self.logit, **self.args)

    def teacher(self):
        return (self.index, self.logit, self.top) if self.top else ()

    def forward(self, sums=True):
        loss = torch.full((self.rows + 2,), 9.0, device="cuda")
        lse = torch.full(((self.rows + 2), 2) if self.top else (self.rows + 2,), 9.0, device="cuda")
        s = torch.full((3,), 9.0, device="cuda")
        call = self.z.zero_distill_forward if self.top else self.z.zero_ce_forward
        call(self.head, self.x, self.ld, self.w, self.ld, *self.teacher(), self.labels, loss, lse, s if sums else None,
             self.work, stream())
        torch.cuda.synchronize()
        assert bool((loss[self.rows:] == 9).all()) and bool((lse[self.rows:] == 9).all()) and float(s[2]) == 9.0
        self.untouched()
        return loss[:self.rows], lse[:self.rows], s[:2]

    def untouched(self):
        assert int(self.work[:4].view(torch.int32)[0]) == 0
        assert bool((self.space[self.work.numel():] == 0xA5).all()), "written past the workspace"

    def backward(self, lse, row_grad=None, scale=1.0, divisor=None, pad=0, shift=0, want=(True, True), accumulate=None, dx=None):
        if dx is None:
            dx, dx_buf = matrix(self.rows, self.cols, self.dtype, pad, shift, fill=7.0)
        else:
            dx_buf = None
        dw, dw_buf = matrix(self.vocab, self.cols, self.dtype, pad, shift, fill=7.0)
        if accumulate is not None:
            dw.copy_(accumulate)
        call = self.z.zero_distill_backward if self.top else self.z.zero_ce_backward
        call(self.head, self.x, self.ld, self.w, self.ld, *self.teacher(), self.labels, lse, row_grad, scale, divisor,
             dx if want[0] else None, dx.stride(0) if self.rows > 1 else self.cols + pad, dw if want[1] else None, self.cols + pad,
             0 if accumulate is None else 1, self.work, stream())
        torch.cuda.synchronize()
        self.untouched()
        for buf, rows, wanted in ((dx_buf, self.rows, want[0]), (dw_buf, self.vocab, want[1])):
            if buf is None:
                continue
            rest = buf.clone()
            if wanted:
                rest[shift:shift + rows * (self.cols + pad)].view(rows, self.cols + pad)[:, :self.cols] = 7.0
            assert bool((rest == 7.0).all()), "written outside the result"
        return dx, dw

    def check_forward(self):
        loss, lse, sums = self.forward()
        want, want_lse, want_sums, bound = self.case().forward()
        R.close(loss, want, bound, "loss")
        R.close(lse, want_lse, self.case().lse_bound(), "lse")
        if not bool(torch.isnan(want).any()):
            # the losses themselves are added exactly enough: their bounds, and the result's rounding
            assert abs(float(sums[0]) - float(want_sums[0])) <= float(bound.sum()) + 2.0 ** -22 * float(want.abs().sum()) + 1e-30
        assert float(sums[1]) == float(want_sums[1])
        return lse

    def check_backward(self, lse, row_grad=None, scale=1.0, divisor=None, **kw):
        dx, dw = self.backward(lse, row_grad, scale, divisor, **kw)
        want_x, want_w, bound_x, bound_w = self.case().gradient(lse, row_grad, scale, divisor)
        if kw.get("want", (True, True))[0]:
            R.close(dx, want_x, bound_x, "dx")
        if kw.get("want", (True, True))[1]:
            if kw.get("accumulate") is not None:
                want_w = want_w + kw["accumulate"].double()
            R.close(dw, want_w, bound_w, "dw")
        return dx, dw

    def check(self, **kw):
        return self.check_backward(self.check_forward(), **kw)


SIZES = [(1, 1, 1), (1, 8, 2), (2, 64, 255), (31, 63, 256), (64, 65, 257), (64, 256, 1000), (255, 128, 513), (257, 200, 700),
         (300, 771, 1003), (513, 832, 300), (1025, 320, 2000), (40, 2312, 515), (700, 1600, 4099), (2100, 96, 96)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_cross_entropy(z, rows, cols, vocab, dtype):
    Head(z, rows, cols, vocab, dtype).check(scale=64.0 if dtype == FP16 else 1.0)


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("top,temperature,labels", [(1, 1.0, False), (5, 2.0, True), (40, 1.0, True)])
def test_distillation(z, rows, cols, vocab, top, temperature, labels):
    dtype = (rows + top) % 2
    Head(z, rows, cols, vocab, dtype, top=top, temperature=temperature, labels=labels, hard=0.4, soft=0.7,
         top_dtype=(rows + cols) % 3).check(scale=64.0 if dtype == FP16 else 1.0)


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (8, 8), (3, 5), (8, 4)])
@pytest.mark.parametrize("out", [(0, 0), (0, 1), (5, 0), (8, 8)])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_strides_and_alignment(z, pad, shift, out, dtype):
    Head(z, 130, 200, 600, dtype, pad=pad, shift=shift).check(scale=64.0, pad=out[0], shift=out[1])


@pytest.mark.parametrize("cols", [1, 31, 193, 196, 199, 1479])
@pytest.mark.parametrize("rows", [64, 1100])
def test_columns_that_end_inside_a_vector(z, cols, rows):
    """Aligned rows whose last 16 bytes hold more than the row: what is there is neither used nor written."""
    pad = -cols % 8
    h = Head(z, rows, cols, 300, BF16, pad=pad, top=3, hard=0.5, soft=0.5)
    for buf, n in ((h.x_buf, rows), (h.w_buf, 300)):
        buf[:n * h.ld].view(n, h.ld)[:, cols:] = math.nan
    h.check(pad=pad)
    before = torch.randn(300, cols, device="cuda").bfloat16()
    h.check_backward(h.forward()[1], pad=pad, accumulate=before)


@pytest.mark.parametrize("piece", [1, 256, 512, 700, 1 << 20])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("top", [0, 7])
def test_pieces_of_the_vocabulary(z, piece, shift, top):
    kw = dict(top=top, temperature=2.0, hard=0.5, soft=0.5) if top else {}
    h = Head(z, 300, 136, 1500, BF16, piece=piece, shift=shift, **kw)
    h.check()


@pytest.mark.parametrize("ignored", [[0], [299], range(0, 300, 2), range(10, 290), range(1, 300), range(300)])
@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_rows_without_a_label_are_not_read(z, ignored, top, dtype):
    kw = dict(top=top, temperature=1.5, hard=0.5, soft=0.5) if top else {}
    h = Head(z, 300, 72, 500, dtype, ignored=list(ignored), **kw)
    at = torch.tensor(list(ignored), device="cuda")
    h.x[at] = math.nan
    h.x[at[::2]] = math.inf
    if top:
        h.logit[at] = math.nan
        h.index[at[::2]] = 1 << 30
    lse = h.check_forward()
    dx, dw = h.check_backward(lse, scale=32.0)
    assert bool((dx[at] == 0).all()) and bool(dw.isfinite().all())
    before = torch.randn(500, 72, device="cuda").to(KIND[dtype])
    h.check_backward(lse, accumulate=before)


def test_labels_past_the_vocabulary_give_nan(z):
    for top in (0, 3):
        for bad in (1000, 1023, 5000, 2 ** 31 - 1):
            h = Head(z, 270, 64, 1000, BF16, top=top, **(dict(hard=0.5, soft=0.5) if top else {}))
            h.labels[77] = bad
            lse = h.check_forward()
            assert int(torch.isnan(lse.reshape(270, -1)[:, 0]).sum()) == 1
            dx, dw = h.check_backward(lse)
            assert bool(dw.isnan().all()) and bool(dx[77].isnan().all()) and bool(dx[:77].isfinite().all())


def test_entries_past_the_vocabulary_give_nan(z):
    h = Head(z, 100, 64, 1000, BF16, top=4, labels=False)
    h.index[50, 2] = 1000
    lse = h.check_forward()
    assert bool(lse[50, 0].isnan())
    h.check_backward(lse)


def test_non_finite_rows_that_count_give_nan_in_their_row(z):
    h = Head(z, 100, 64, 1000, BF16)
    h.x[3, 5] = math.nan
    loss, lse, _ = h.forward()
    assert bool(loss[3].isnan()) and int(loss.isnan().sum()) == 1
    dx, dw = h.backward(lse)
    assert bool(dx[3].isnan().all()) and bool(dx[:3].isfinite().all()) and bool(dw.isnan().all())


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("top", [0, 5])
def test_row_weights_scale_and_divisor(z, dtype, top):
    kw = dict(top=top, temperature=0.7, hard=0.3, soft=0.6) if top else {}
    h = Head(z, 400, 136, 700, dtype, ignored=[5, 6, 399], z_loss=0.01, **kw)
    lse = h.check_forward()
    g = torch.randn(400, device="cuda")
    g[10:40] = 0.0                                   # no gradient, not read
    g[40:80] *= 1e-4
    g[80:90] *= 300.0
    keep = h.x.clone()
    h.x[10:40] = math.nan
    h2 = h.case()
    dx, dw = h.backward(lse, g, 3.0, torch.tensor([17.0], device="cuda"))
    h.x.copy_(keep)
    want_x, want_w, bound_x, bound_w = h.case().gradient(lse, g, 3.0, torch.tensor(17.0))
    R.close(dx, want_x, bound_x, "dx")
    R.close(dw, want_w, bound_w, "dw")
    assert h2.x is h.x
    # a mean over no rows
    dx, dw = h.backward(lse, g, 3.0, torch.zeros(1, device="cuda"))
    assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-20, 1e20, 2.0 ** 100])
def test_scales_of_any_size(z, scale):
    """bf16 has fp32's range: a scale moves the results, not their precision."""
    h = Head(z, 100, 64, 300, BF16)
    h.check(scale=scale)
    h = Head(z, 100, 64, 300, BF16)
    lse = h.check_forward()
    h.check_backward(lse, row_grad=torch.rand(100, device="cuda") + 0.5, scale=scale)


def test_fp16_gradients_keep_their_precision_at_small_scales(z):
    """Tiny row weights and probabilities far below fp16's smallest number."""
    h = Head(z, 200, 64, 3000, FP16, spread=6.0)
    lse = h.check_forward()
    h.check_backward(lse, row_grad=torch.full((200,), 1e-12, device="cuda"), scale=1e13)
    h.check_backward(lse, scale=2.0 ** 15)


@pytest.mark.parametrize("want", [(True, False), (False, True)])
def test_one_gradient_alone(z, want):
    h = Head(z, 200, 136, 700, BF16)
    lse = h.check_forward()
    both = h.backward(lse)
    one = h.check_backward(lse, want=want)
    for a, b, wanted in zip(both, one, want):
        assert torch.equal(a, b) if wanted else bool((b == 7.0).all())


@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (3, 7)])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_accumulation(z, dtype, shift, pad):
    for rows in (70, 1300):                              # whole tiles, and tiles cut along the rows
        h = Head(z, rows, 200, 300, dtype)
        before = torch.randn(300, 200, device="cuda").to(KIND[dtype])
        h.check_backward(h.check_forward(), accumulate=before, shift=shift, pad=pad)


def test_input_gradient_in_place(z):
    for shift, pad in ((0, 0), (1, 3)):
        h = Head(z, 300, 136, 700, BF16, ignored=[0, 7, 100], shift=shift, pad=pad)
        lse = h.check_forward()
        dx, dw = h.backward(lse)
        _, dw2 = h.backward(lse, dx=h.x)
        assert torch.equal(h.x, dx) and torch.equal(dw, dw2)


def test_few_columns_of_tiles_cut_along_a_long_vocabulary(z):
    """dx of few rows: parts of the vocabulary joined; dw of many rows: parts of the rows."""
    Head(z, 40, 72, 30000, BF16).check()
    Head(z, 9000, 72, 130, FP16).check(scale=64.0)
    Head(z, 600, 392, 20000, BF16, piece=4096).check()


@pytest.mark.parametrize("top", [2, 33, 128, 256])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 4.0])
def test_teachers(z, top, temperature):
    """Absent entries, rows without any, repeated indices, lowest values and -inf."""
    for labels in (False, True):
        h = Head(z, 140, 96, 900, BF16, top=top, temperature=temperature, labels=labels, hard=0.25, soft=0.75)
        h.index[:, 1] = h.index[:, 0]                    # the same index twice
        h.index[3] = 5                                   # all one index
        h.index[10:20, ::2] = -1
        h.logit[10:20, ::2] = math.nan                   # absent: not read
        h.index[20] = -1                                 # nothing kept
        h.logit[21] = -math.inf
        h.logit[22, 0] = -math.inf
        h.logit[23] = torch.finfo(torch.float32).min
        h.logit[24, 1:] = torch.finfo(torch.float32).min
        h.logit[25, 0] = 300.0                           # all of the probability
        h.index[26] = torch.arange(top, device="cuda")   # neighbours: one tile
        h.index[27] = 899
        lse = h.check_forward()
        dx, _ = h.check_backward(lse)
        if not labels:
            assert bool((lse[20:22] == 0).all()) and bool((dx[20:22] == 0).all())


def test_a_dense_teacher(z):
    """Every token an entry: the plain divergence between two softmaxes."""
    h = Head(z, 64, 64, 200, BF16, top=200, temperature=2.0, labels=False)
    h.index.copy_(torch.argsort(torch.rand(64, 200, device="cuda"), 1))
    h.check()
    z_ = h.x.double() @ h.w.double().T
    t = torch.empty(64, 200, device="cuda", dtype=torch.float64).scatter_(1, h.index.long(), h.logit.double())
    want = 4.0 * torch.nn.functional.kl_div((z_ / 2).log_softmax(1), (t / 2).softmax(1), reduction="none").sum(1)
    loss = h.forward()[0]
    assert torch.allclose(loss.double(), want, rtol=0, atol=1e-4)


def test_a_label_is_a_teacher_of_one_entry(z):
    h = Head(z, 300, 136, 700, BF16)
    loss, lse, _ = h.forward()
    grads = h.backward(lse)
    t = Head(z, 300, 136, 700, BF16, top=1, labels=False)
    t.index[:, 0] = h.labels
    loss_t, lse_t, _ = t.forward()
    assert torch.equal(loss, loss_t) and torch.equal(lse, lse_t[:, 0])
    for a, b in zip(grads, t.backward(lse_t)):
        assert torch.equal(a, b)


def test_precision_of_the_loss(z):
    """Long rows: sums of at most 48 steps of 16 columns on the tensor cores, each step at random inputs
    off by about 1.6e-8 of the sum: 7.7e-7 with the fp32 additions of the runs (2^-24 each, sqrt(6)
    of them: 1.5e-7) below 1e-6 of the logits; log-sum-exp averages its terms and adds no more than
    its own rounding, 2^-23 of about 10."""
    h = Head(z, 500, 4096, 5000, BF16)
    loss, lse, _ = h.forward()
    want, want_lse, _, _ = h.case().forward()
    size = float(h.case().logits()[1].square().mean().sqrt())
    assert float((lse.double() - want_lse).square().mean().sqrt()) < 1e-6 * size + 2.0 ** -23 * 16
    assert float((loss.double() - want).square().mean().sqrt()) < 3e-6 * size + 2.0 ** -22 * 16


@pytest.mark.parametrize("top", [0, 20])
def test_equal_calls_give_equal_bits(z, top):
    kw = dict(top=top, temperature=2.0, hard=0.5, soft=0.5) if top else {}
    h = Head(z, 1500, 264, 6000, BF16, ignored=range(0, 1500, 7), piece=2048, **kw)
    first = h.forward()
    grads = h.backward(first[1])
    for _ in range(20):
        h.space[:h.work.numel()].random_(0, 256)         # whatever the workspace holds
        for a, b in zip(first, h.forward()):
            assert torch.equal(a, b)
        for a, b in zip(grads, h.backward(first[1])):
            assert torch.equal(a, b)


def test_two_streams_at_once(z):
    heads = [Head(z, 700, 264, 5000, BF16, seed=s) for s in (0, 1)]
    want = []
    for h in heads:
        loss, lse, _ = h.forward()
        want.append((loss, lse, *h.backward(lse)))
    streams = [torch.cuda.Stream() for _ in heads]
    outs = []
    for h in heads:
        outs.append((torch.empty(700, device="cuda"), torch.empty(700, device="cuda"),
                     torch.empty(700, 264, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(5000, 264, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for h, s, (loss, lse, dx, dw) in zip(heads, streams, outs):
            z.zero_ce_forward(h.head, h.x, 264, h.w, 264, h.labels, loss, lse, None, h.work, s.cuda_stream)
            z.zero_ce_backward(h.head, h.x, 264, h.w, 264, h.labels, lse, None, 1.0, None, dx, 264, dw, 264, 0, h.work,
                               s.cuda_stream)
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        for a, b in zip(got, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("top", [0, 9])
def test_captured_and_replayed(z, top):
    """A training step's loss and gradients in a CUDA graph, replayed on other inputs."""
    kw = dict(top=top, temperature=2.0, hard=0.5, soft=0.5) if top else {}
    h = Head(z, 300, 136, 1500, BF16, piece=512, **kw)
    other = Head(z, 300, 136, 1500, BF16, seed=9, ignored=range(50, 120), piece=512, **kw)
    loss, sums = torch.zeros(300, device="cuda"), torch.zeros(2, device="cuda")
    lse = torch.zeros((300, 2) if top else (300,), device="cuda")
    dx, dw = torch.zeros_like(h.x), torch.zeros_like(h.w)
    fwd = z.zero_distill_forward if top else z.zero_ce_forward
    bwd = z.zero_distill_backward if top else z.zero_ce_backward

    def step():
        fwd(h.head, h.x, 136, h.w, 136, *h.teacher(), h.labels, loss, lse, sums, h.work, stream())
        bwd(h.head, h.x, 136, h.w, 136, *h.teacher(), h.labels, lse, None, 1.0, sums[1:], dx, 136, dw, 136, 0, h.work, stream())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in (other, h):
        saved = [t.clone() for t in (new.x, new.w, new.labels)] + ([new.index.clone(), new.logit.clone()] if top else [])
        want_loss, want_lse, want_sums = new.forward()
        want = new.backward(want_lse, divisor=want_sums[1:])
        mine = [h.x, h.w, h.labels] + ([h.index, h.logit] if top else [])
        keep = [t.clone() for t in mine]
        for a, b in zip(mine, saved):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want_loss) and torch.equal(lse, want_lse) and torch.equal(sums, want_sums)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        for a, b in zip(mine, keep):
            a.copy_(b)


def test_no_rows(z):
    h = z.head(BF16, 0, 64, 100)
    work = torch.empty(z.zero_head_workspace(h), dtype=torch.uint8, device="cuda")
    w, dw = torch.randn(100, 64, device="cuda").bfloat16(), torch.full((100, 64), 3.0, device="cuda").bfloat16()
    sums = torch.full((2,), 5.0, device="cuda")
    z.zero_ce_forward(h, None, 64, w, 64, None, None, None, sums, work, stream())
    z.zero_ce_backward(h, None, 64, w, 64, None, None, None, 1.0, None, None, 64, dw, 64, 1, work, stream())
    assert bool((sums == 0).all()) and bool((dw == 3.0).all())
    z.zero_ce_backward(h, None, 64, w, 64, None, None, None, 1.0, None, None, 64, dw, 64, 0, work, stream())
    assert bool((dw == 0).all())
    z.zero_distill_forward(z.head(BF16, 0, 64, 100, top=2), None, 64, w, 64, None, None, 2, None, None, None, sums, work, stream())


def test_gradients_go_into_a_step(z):
    """Norm, loss and their gradients into a rank's gradient row at unaligned places, and one optimizer step."""
    rows, d, vocab, nd = 260, 72, 501, 2
    shapes = [(3,), (d,), (vocab, d)]                    # the head's weights begin at an odd element
    psi = sum(math.prod(s) for s in shapes)
    plan = z.zero_plan_create(psi, nd, 2, FP16, shapes, z.hparams(lr=1e-2, loss_scale=1024.0, dynamic_scale=1))
    _, padded, _, ws = z.zero_plan_layout(plan)
    new = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    grads, master, m, v = new(nd, padded, t=torch.float16), new(padded), new(padded), new(padded)
    params, step_work = new(padded, t=torch.float16), new(max(ws, 16), t=torch.uint8)
    master[:psi].normal_(generator=torch.Generator(device="cuda").manual_seed(1)).mul_(0.2)
    master[3:3 + d] = 1.0
    params.copy_(master)
    norm_w, w = params[3:3 + d], params[3 + d:psi]
    norm = z.norm(FP16, rows, d, pre=z.ZERO_NORM_RMS, pre_w=norm_w)
    head = z.head(FP16, rows, d, vocab)
    work, norm_work = new(z.zero_head_workspace(head), t=torch.uint8), new(z.zero_norm_workspace(norm), t=torch.uint8)
    x, dx, dh = (new(rows, d, t=torch.float16) for _ in range(3))
    ckpt, stats = new(rows, z.zero_act_row_bytes(d), t=torch.uint8), new(rows, 4)
    loss, lse, sums, s = new(rows), new(rows), new(2), stream()
    for rank in range(nd):
        gen = torch.Generator(device="cuda").manual_seed(5 + rank)
        h = torch.randn(rows, d, generator=gen, device="cuda").half()
        labels = torch.randint(vocab, (rows,), generator=gen, device="cuda").to(torch.int32)
        labels[::9] = -1
        z.zero_norm_forward(norm, h, d, None, 0, None, 0, x, d, None, ckpt, stats, s)
        z.zero_ce_forward(head, x, d, w, d, labels, loss, lse, sums, work, s)
        z.zero_ce_backward(head, x, d, w, d, labels, lse, None, 1024.0, sums[1:], dx, d, grads[rank, 3 + d:], d, 0, work, s)
        z.zero_norm_backward(norm, None, d, dx, d, None, ckpt, stats, dh, d, None, d, FP16, dpre_w=grads[rank, 3:],
                             work=norm_work, stream=s)
        case = R.Case(x, w.view(vocab, d), labels)
        R.close(loss, *[case.forward()[i] for i in (0, 3)], "loss")
        want_x, want_w, bound_x, bound_w = case.gradient(lse, None, 1024.0, sums[1])
        R.close(dx, want_x, bound_x, "dx")
        R.close(grads[rank, 3 + d:psi].view(vocab, d), want_w, bound_w, "dw")
        assert bool((grads[rank, :3] == 0).all()) and bool((grads[rank, psi:] == 0).all())
    before = params.clone()
    z.zero_step(plan, grads, master, m, v, params, step_work, s)
    assert z.zero_step_result(plan)["skipped"] == 0 and not torch.equal(before, params)
    z.zero_plan_destroy(plan)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("top", [0, 6])
def test_precision_of_the_gradients(z, dtype, top):
    """In the 2-norm over many rows: a result's own rounding (e0), and of dz's (its relative error is spread over at most
    half a step, eps / sqrt(3) in the mean square) for dw all of it, for dx what the heavy targets leave, whose
    share of dz's square is 1 - rho; rows of w and x are independent, so squares add.  A tenth for chance."""
    kw = dict(top=top, temperature=1.0, hard=0.5, soft=0.5) if top else {}
    h = Head(z, 600, 512, 2000, dtype, spread=3.0, **kw)
    lse = h.check_forward()
    dx, dw = h.backward(lse, scale=64.0)
    c = h.case()
    want_x, want_w, _, _ = c.gradient(lse, None, 64.0)
    x, logits = c.logits()
    heavy = torch.zeros_like(logits)
    weight = heavy.clone()
    if top:
        q, at, _ = c.teacher()
        weight.scatter_add_(1, at, 0.5 * q)
        dz = 0.5 * (logits - lse[:, :1].double()).exp() + 0.5 * (logits - lse[:, 1:].double()).exp()
    else:
        dz = (logits - lse[:, None].double()).exp()
    weight.scatter_add_(1, h.labels.long()[:, None], torch.full_like(logits[:, :1], 0.5 if top else 1.0))
    dz = dz - weight
    heavy = weight >= weight.sum(1, keepdim=True) / 4
    rho = float((dz * ~heavy).square().sum() / dz.square().sum())
    assert 0.001 < rho < 0.9
    eps = R.EPS[KIND[dtype]]
    off = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
    for got, want, share in ((dx, want_x, rho), (dw, want_w, 1.0)):
        e0 = off(want.to(KIND[dtype]), want)
        assert off(got, want) < 1.1 * math.sqrt(e0 ** 2 + share * eps ** 2 / 3)


def test_teachers_entries_with_a_stride(z):
    h = Head(z, 70, 64, 500, BF16, top=5, labels=False)
    loss, lse, _ = h.forward()
    wide_i, wide_l = torch.full((70, 9), 499, dtype=torch.int32, device="cuda"), torch.full((70, 9), math.nan, device="cuda")
    wide_i[:, :5], wide_l[:, :5] = h.index, h.logit
    out, out_lse = torch.empty(70, device="cuda"), torch.empty(70, 2, device="cuda")
    z.zero_distill_forward(h.head, h.x, 64, h.w, 64, wide_i, wide_l, 9, None, out, out_lse, None, h.work, stream())
    assert torch.equal(out, loss) and torch.equal(out_lse, lse)


def test_weights_of_the_parts(z):
    """Either part switched off, and negative weights."""
    for hard, soft in ((0.0, 1.0), (1.0, 0.0), (0.0, 0.0), (-0.5, 0.7), (2.0, 30.0)):
        h = Head(z, 130, 72, 400, BF16, top=4, temperature=1.5, hard=hard, soft=soft)
        h.check()


def test_largest_sizes_of_one_kind(z):
    """A row of 16384 columns, a vocabulary of 200003 in many pieces, 65536 rows."""
    Head(z, 3, 16384, 70, BF16).check()
    Head(z, 5, 16, 200003, BF16, piece=3000).check()
    h = Head(z, 65536, 16, 40, BF16, ignored=range(0, 65536, 3))
    lse = h.check_forward()
    h.check_backward(lse, row_grad=torch.rand(65536, device="cuda"))
