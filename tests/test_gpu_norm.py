"""The norms around a block on the GPU, forward and backward, against a plain 64-bit
implementation.

Tolerances.  A sum of n fp32 terms taken in a tree of depth at most L loses at most L 2^-24 of
the terms' magnitudes; here L <= 64 for the sums over a row (at most 32 elements in a thread, 5
shuffles, 16 warps, and the operations around them).  K = 2^-18 covers 64 such roundings; output
types add their own rounding.  Sums over rows: a block adds its rows one after another, then the
blocks are added: at most rows + 64 roundings."""
import numpy as np
import pytest

import act_reference as R
from test_gpu_act import TINY, U, activations, device_matrix, env, kind, stream  # noqa: F401

pytestmark = pytest.mark.gpu
K = 2.0 ** -18
EPS = 1e-5


def weights(torch, rng, p, dtype, shift=0):
    """Random weights for the norms of p, on the device (shift elements into their allocation), and
    in 64 bits in p; returns the device tensors."""
    groups = 1 if p["group"] == 0 or p["rows"] == 0 else -(-p["rows"] // p["group"])
    dev = {}
    for w, on, shape, mean in (("post_w", p["post"], (p["cols"],), 1.0), ("post_b", p["post"] and p["bias"], (p["cols"],), 0.0),
                               ("pre_w", p["pre"], (p["cols"],), 1.0), ("pre_b", p["pre"] and p["bias"], (p["cols"],), 0.0),
                               ("gate", p["has_gate"], (groups, p["cols"]), 0.5)):
        dev[w] = p[w] = None
        if on:
            n = int(np.prod(shape))
            t = torch.empty(n + shift, dtype=kind(torch, dtype), device="cuda")[shift:].view(shape)
            t.copy_(torch.from_numpy(mean + 0.3 * rng.standard_normal(shape)))
            dev[w], p[w] = t, t.double().cpu().numpy()
    return dev


def params(rows, cols, post, pre, group=0, alpha=0.7, bias=True, has_gate=True):
    return dict(rows=rows, cols=cols, post=post, pre=pre, group=group, alpha=alpha, bias=bias,
                has_gate=has_gate, eps=EPS)


def describe(z, p, dtype, res, dev):
    return z.norm(dtype, p["rows"], p["cols"], res_dtype=res, post=p["post"], pre=p["pre"], eps=EPS,
                  alpha=p["alpha"], group_rows=p["group"], **dev)


def rounded(got, want, mag, dtype, k=K):
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(got))
    tol = U[dtype] * np.abs(want) + TINY[dtype] + k * mag
    assert np.all(np.abs(got - want)[fine] <= tol[fine]), np.max((np.abs(got - want) / (tol + 1e-300))[fine])


def checkpointed(got, want, mag, dtype, cols):
    """A checkpoint of values known up to K mag: the exponents of some value in that range, and codes
    within half a step (and that range) of the value."""
    rows = len(want)
    e = R.exponents(got, cols)
    lo, hi = (R.exponents(R.quantize(np.abs(want) + s * K * mag, dtype), cols) for s in (-1, 1))
    assert np.all((e >= np.minimum(lo, hi)) & (e <= np.maximum(lo, hi)))
    unit = np.repeat(np.ldexp(1.0, e - 127), 32, axis=1)[:, :cols]
    assert np.all(np.abs(R.values(got, cols) - want) <= 0.5 * unit + K * mag)
    wide = R.wide_of(cols)
    assert not got[:, cols:wide].any() and not got[:, wide + wide // 32:].any()


def run_forward(env, p, dtype, res, pad=0, shift=0, with_y=True, ckpt=True, in_place=False, seed=0, edit=None):
    torch, z = env
    rows, cols = p["rows"], p["cols"]
    rng = np.random.default_rng(seed + rows + 3 * cols + 7 * p["post"] + 11 * p["pre"])
    dev = weights(torch, rng, p, dtype, shift)
    h, y = activations(rng, rows, cols, 2.0) + 0.3, activations(rng, rows, cols, 0.7) - 0.2
    if edit:
        edit(h, y)
    kh, ph, ld, hv, hview = device_matrix(torch, h, res, pad, shift)
    ky, py, _, yv, _ = device_matrix(torch, y, dtype, pad, shift)
    ko, po, _, _, oview = device_matrix(torch, np.zeros((rows, cols)), res, pad, shift)
    kx, px, _, _, xview = device_matrix(torch, np.zeros((rows, cols)), dtype, pad, shift)
    if in_place:
        po, oview = ph, hview
    cy = torch.full((rows, R.row_bytes(cols)), 0xA5, dtype=torch.uint8, device="cuda") if ckpt and with_y else None
    cx = torch.full((rows, R.row_bytes(cols)), 0xA5, dtype=torch.uint8, device="cuda") if ckpt and p["pre"] else None
    stats = torch.full((rows, 4), 9.0, device="cuda") if ckpt else None
    z.zero_norm_forward(describe(z, p, dtype, res, dev), ph, ld, py if with_y else None, ld, po, ld,
                        px if p["pre"] else None, ld, cy, cx, stats, stream(torch))
    torch.cuda.synchronize()
    f = R.forward(hv, yv if with_y else None, p)
    # magnitudes: a mean is off by K mean|v|, a reciprocal deviation by K of itself (and what the
    # mean's error adds), a normalised value by both
    _, m2, r2 = R.normalise(yv, p["post"], EPS)
    my = np.abs(yv) * r2[:, None] + (np.abs(yv).mean(1) * r2)[:, None]
    mz = my * np.abs(R.one(p["post_w"], 1.0)) + np.abs(R.one(p["post_b"], 0.0))
    mh = np.abs(hv)
    if with_y:
        mh = mh + abs(p["alpha"]) * np.abs(R.gate_rows(p["gate"], rows, p["group"])) * mz
    rounded(oview.double().cpu().numpy(), f["h"], mh, res)
    r1 = f["stats"][:, 3:4]
    mx = (mh + mh.mean(1, keepdims=True)) * r1 + np.abs(f["xh"]) * (mh * r1).max(1, keepdims=True)
    if p["pre"]:
        mo = mx * np.abs(R.one(p["pre_w"], 1.0)) + np.abs(R.one(p["pre_b"], 0.0))
        rounded(xview.double().cpu().numpy(), f["x"], mo, dtype)
    if ckpt:
        s = stats.double().cpu().numpy()
        mag = np.stack([np.abs(yv).mean(1), r2 * my.max(1), mh.mean(1), r1[:, 0] * (1 + (mh * r1).max(1))], 1)
        if not with_y:
            mag[:, :2] = 0
        mag = np.nan_to_num(mag)                    # what a NaN row still fixes (a mean of 0) is exact
        fine = np.isfinite(f["stats"])
        assert np.array_equal(fine, np.isfinite(s))
        assert np.all((np.abs(s - f["stats"]) <= K * (mag + np.abs(f["stats"])))[fine])
        if not edit:
            if with_y:
                checkpointed(cy.cpu().numpy(), f["yh"], my, dtype, cols)
            if p["pre"]:
                checkpointed(cx.cpu().numpy(), f["xh"], mx, dtype, cols)
    return f, oview, xview, cy, cx, stats


KINDS = [(R.RMS, R.RMS), (R.LAYER, R.LAYER), (R.NONE, R.RMS), (R.NONE, R.LAYER), (R.RMS, R.NONE), (R.LAYER, R.NONE),
         (R.NONE, R.NONE)]
SIZES = [(1, 1), (1, 1600), (3, 33), (5, 64), (2, 771), (40, 768), (7, 4096), (3, 4097), (2, 8200), (2, 16384), (700, 96)]


@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("rows,cols", [(5, 64), (17, 1600), (3, 4097)])
@pytest.mark.parametrize("dtype,res", [(R.BF16, R.BF16), (R.FP16, R.FP32)])
def test_forward_kinds(env, post, pre, rows, cols, dtype, res):  # noqa: F811
    run_forward(env, params(rows, cols, post, pre, group=2), dtype, res)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,res", [(R.BF16, R.FP32), (R.FP16, R.FP16), (R.BF16, R.BF16)])
def test_forward_sizes(env, rows, cols, dtype, res):  # noqa: F811
    run_forward(env, params(rows, cols, R.RMS, R.RMS, bias=False), dtype, res)
    run_forward(env, params(rows, cols, R.LAYER, R.LAYER, group=1), dtype, res, ckpt=False)


@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (8, 8), (3, 4)])
@pytest.mark.parametrize("res", [R.BF16, R.FP32])
def test_forward_strides(env, pad, shift, res):  # noqa: F811
    run_forward(env, params(21, 200, R.RMS, R.LAYER, group=4), R.BF16, res, pad, shift)


def test_forward_without_a_block(env):  # noqa: F811
    run_forward(env, params(9, 320, R.NONE, R.RMS, has_gate=False), R.BF16, R.FP32, with_y=False)


def test_forward_in_place(env):  # noqa: F811
    run_forward(env, params(300, 256, R.RMS, R.RMS, group=100), R.BF16, R.BF16, in_place=True)


def test_forward_rows_of_zeros_and_non_finite_rows(env):  # noqa: F811
    """Zero rows normalise to zero; a NaN or an infinity stays in its row."""
    torch, z = env

    def edit(h, y):
        h[1] = y[1] = 0.0
        y[3, 7] = np.nan
        h[5, 9] = np.nan
    p = params(8, 96, R.RMS, R.RMS, bias=False)
    f, o, x, cy, cx, stats = run_forward(env, p, R.BF16, R.FP32, edit=edit)
    assert not x[1].any() and not R.values(cx.cpu().numpy()[1:2], 96).any()
    assert np.isnan(R.values(cy.cpu().numpy()[3:4], 96)).all() and np.isnan(R.values(cx.cpu().numpy()[5:6], 96)).all()


def run_backward(env, p, dtype, res, grad, pad=0, shift=0, with_dh=True, in_place=False, accumulate=0, seed=0,
                 want=("dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b"), with_block=True):
    torch, z = env
    rows, cols = p["rows"], p["cols"]
    rng = np.random.default_rng(seed + rows + 5 * cols + 7 * p["post"] + 11 * p["pre"])
    dev = weights(torch, rng, p, dtype, shift)
    h, y = activations(rng, rows, cols, 2.0) + 0.3, activations(rng, rows, cols, 0.7) - 0.2
    yh, m2, r2 = R.normalise(y, p["post"], EPS) if rows else (y, np.zeros(0), np.zeros(0))
    xh, m1, r1 = R.normalise(h, p["pre"], EPS) if rows else (h, np.zeros(0), np.zeros(0))
    qy, qx = R.quantize(yh, dtype), R.quantize(xh, dtype)
    stats = np.stack([m2, r2, m1, r1], 1).astype(np.float32)
    dho = rng.standard_normal((rows, cols)) * 0.1
    dx = rng.standard_normal((rows, cols)) * 0.2
    kd, pd, ld, dhov, dview = device_matrix(torch, dho, res, pad, shift)
    kx, px, _, dxv, _ = device_matrix(torch, dx, dtype, pad, shift)
    ko, po, _, _, oview = device_matrix(torch, np.zeros((rows, cols)), res, pad, shift)
    ky, py, _, _, yview = device_matrix(torch, np.zeros((rows, cols)), dtype, pad, shift)
    if in_place:
        po, oview = pd, dview
    cy = torch.from_numpy(qy).cuda() if with_block else None
    cx = torch.from_numpy(qx).cuda() if p["pre"] else None
    st = torch.from_numpy(stats).cuda()
    groups = 1 if p["group"] == 0 or rows == 0 else -(-rows // p["group"])
    grads, old = {}, {}
    for name in want:
        on = {"dgate": with_block, "dpost_w": p["post"], "dpost_b": p["post"]}.get(name, p["pre"])
        shape = (groups, cols) if name == "dgate" else (cols,)
        grads[name] = None
        if on:
            t = torch.empty(int(np.prod(shape)) + shift, dtype=kind(torch, grad), device="cuda")[shift:].view(shape)
            t.copy_(torch.from_numpy(rng.standard_normal(shape)))
            grads[name], old[name] = t, t.double().cpu().numpy()
    n = describe(z, p, dtype, res, dev)
    work = torch.full((z.zero_norm_workspace(n),), 0xFF, dtype=torch.uint8, device="cuda")
    z.zero_norm_backward(n, pd if with_dh else None, ld, px if p["pre"] else None, ld, cy, cx, st, po, ld,
                         py if with_block else None, ld, grad, accumulate=accumulate, work=work,
                         stream=stream(torch), **grads)
    torch.cuda.synchronize()
    ref, mag = R.backward(dhov if with_dh else None, dxv, R.values(qy, cols) if with_block else None,
                          R.values(qx, cols), stats.astype(np.float64), p)
    rounded(oview.double().cpu().numpy(), ref["dh"], mag["dh"], res)
    if with_block:
        rounded(yview.double().cpu().numpy(), ref["dy"], mag["dy"], dtype)
    for name, t in grads.items():
        if t is not None:
            w = ref[name].reshape(t.shape) + (old[name] if accumulate else 0.0)
            m = mag[name].reshape(t.shape) + (np.abs(w) if accumulate else 0.0)
            rounded(t.double().cpu().numpy(), w, m, grad, K + (rows + 64) * 2.0 ** -24)
    return grads


@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("rows,cols", [(5, 64), (37, 1600), (3, 4097)])
@pytest.mark.parametrize("dtype,res,grad", [(R.BF16, R.BF16, R.BF16), (R.FP16, R.FP32, R.FP32)])
def test_backward_kinds(env, post, pre, rows, cols, dtype, res, grad):  # noqa: F811
    run_backward(env, params(rows, cols, post, pre, group=2), dtype, res, grad)


@pytest.mark.parametrize("rows,cols", SIZES + [(2500, 320), (5000, 64)])
@pytest.mark.parametrize("dtype,res,grad", [(R.BF16, R.FP32, R.BF16), (R.FP16, R.FP16, R.FP32)])
def test_backward_sizes(env, rows, cols, dtype, res, grad):  # noqa: F811
    run_backward(env, params(rows, cols, R.RMS, R.RMS, bias=False), dtype, res, grad)
    run_backward(env, params(rows, cols, R.LAYER, R.LAYER), dtype, res, grad)


@pytest.mark.parametrize("group", [1, 2, 7, 64, 999, 1000, 5000])
@pytest.mark.parametrize("bias", [False, True])
def test_backward_gate_groups(env, group, bias):  # noqa: F811
    """Groups smaller and larger than a block's rows, ending inside and at its ends."""
    run_backward(env, params(1000, 96, R.RMS, R.RMS, group=group, bias=bias), R.BF16, R.FP32, R.FP32)


@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (8, 8), (3, 4)])
@pytest.mark.parametrize("res", [R.BF16, R.FP32])
def test_backward_strides(env, pad, shift, res):  # noqa: F811
    run_backward(env, params(21, 200, R.RMS, R.LAYER, group=4), R.BF16, res, R.BF16, pad, shift)


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 9), (5, 249), (11, 250), (700, 255), (3, 4081), (40, 4088), (9, 4090), (3, 4096), (2, 8177),
                                       (2, 8190), (2000, 33)])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (0, 5), (7, 7)])
@pytest.mark.parametrize("dtype,res,post,pre,bias", [(R.BF16, R.BF16, 1, 1, False), (R.FP16, R.FP32, 2, 2, True),
                                                     (R.FP16, R.FP16, 0, 2, True), (R.BF16, R.FP32, 0, 1, False),
                                                     (R.BF16, R.BF16, 1, 1, True), (R.FP16, R.FP32, 1, 0, True),
                                                     (R.FP16, R.FP16, 1, 0, False), (R.BF16, R.FP32, 0, 1, True)])
def test_backward_rows_of_any_alignment(env, rows, cols, pad, shift, dtype, res, post, pre, bias):  # noqa: F811
    """Rows whose words and chunks do not coincide: every shift, rows of one warp, rows that fill
    the threads, and the matrices' first and last words."""
    run_backward(env, params(rows, cols, post, pre, group=3, bias=bias), dtype, res, R.FP32, pad=pad, shift=shift,
                 in_place=rows == 40)


@pytest.mark.parametrize("rows,cols", [(7, 64), (700, 1600), (30, 4096), (9, 8192)])
@pytest.mark.parametrize("post,pre,bias", [(1, 1, True), (0, 1, True), (1, 0, True), (1, 0, False)])
@pytest.mark.parametrize("res", [R.BF16, R.FP32])
def test_backward_aligned_rows_of_other_kinds(env, rows, cols, post, pre, bias, res):  # noqa: F811
    run_backward(env, params(rows, cols, post, pre, group=4, bias=bias), R.BF16, res, R.FP32)


@pytest.mark.parametrize("accumulate", [0, 1])
def test_backward_accumulates(env, accumulate):  # noqa: F811
    run_backward(env, params(90, 160, R.LAYER, R.RMS, group=40), R.FP16, R.FP16, R.FP16, accumulate=accumulate)


def test_backward_without_an_incoming_stream_gradient_and_in_place(env):  # noqa: F811
    run_backward(env, params(30, 128, R.RMS, R.RMS), R.BF16, R.FP32, R.FP32, with_dh=False)
    run_backward(env, params(300, 128, R.RMS, R.RMS), R.BF16, R.BF16, R.FP32, in_place=True)


def test_backward_without_a_block(env):  # noqa: F811
    run_backward(env, params(30, 128, R.NONE, R.RMS, has_gate=False), R.BF16, R.FP32, R.FP32, with_block=False,
                 want=("dpre_w", "dpre_b"))


@pytest.mark.parametrize("want", [("dpre_w",), ("dpost_w",), ("dgate",), ("dpost_b", "dpre_b"), ()])
def test_backward_gives_what_is_asked_for(env, want):  # noqa: F811
    run_backward(env, params(50, 96, R.LAYER, R.LAYER, group=20), R.BF16, R.FP32, R.FP32, want=want)


def test_backward_without_rows(env):  # noqa: F811
    for accumulate in (0, 1):
        run_backward(env, params(0, 96, R.RMS, R.RMS), R.BF16, R.FP32, R.FP32, accumulate=accumulate)


def test_backward_is_deterministic(env):  # noqa: F811
    torch, z = env
    p = params(3000, 1600, R.RMS, R.RMS, group=700)
    a = run_backward(env, dict(p), R.BF16, R.BF16, R.FP32)
    b = run_backward(env, dict(p), R.BF16, R.BF16, R.FP32)
    assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


def test_forward_and_backward_against_differences(env):  # noqa: F811
    """The slope of sum(h' A + x B) along random directions, by central differences of the 64-bit
    forward pass, against the GPU's gradients from the GPU's own checkpoints.  A checkpoint's values
    are off by at most half a step, 2^-6 of their block's largest (the step is at most 2^-6 of it and
    half of that is 2^-7; 2^-6 leaves room for the products of two such errors)."""
    torch, z = env
    rng = np.random.default_rng(77)
    p = params(40, 128, R.RMS, R.RMS, group=16, bias=True)
    dev = weights(torch, rng, p, R.BF16)
    rows, cols = 40, 128
    kh, ph, ld, hv, _ = device_matrix(torch, rng.standard_normal((rows, cols)), R.FP32)
    ky, py, _, yv, _ = device_matrix(torch, rng.standard_normal((rows, cols)), R.BF16)
    ka, pa, _, av, _ = device_matrix(torch, rng.standard_normal((rows, cols)), R.FP32)
    kb, pb, _, bv, _ = device_matrix(torch, rng.standard_normal((rows, cols)), R.BF16)
    n = describe(z, p, R.BF16, R.FP32, dev)
    ho = torch.empty(rows, cols, device="cuda")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    cy, cx = (torch.empty(rows, R.row_bytes(cols), dtype=torch.uint8, device="cuda") for _ in range(2))
    st = torch.empty(rows, 4, device="cuda")
    z.zero_norm_forward(n, ph, ld, py, ld, ho, cols, x, cols, cy, cx, st, stream(torch))
    dh = torch.empty(rows, cols, device="cuda")
    dy = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = {k: torch.empty(p[k[1:]].shape, device="cuda") for k in ("dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b")}
    work = torch.empty(z.zero_norm_workspace(n), dtype=torch.uint8, device="cuda")
    z.zero_norm_backward(n, pa, ld, pb, ld, cy, cx, st, dh, cols, dy, cols, R.FP32, work=work,
                         stream=stream(torch), **g)
    torch.cuda.synchronize()
    got = {"h": dh, "y": dy, **{k[1:]: v for k, v in g.items()}}
    t = {"h": hv, "y": yv, **{k: p[k] for k in ("post_w", "post_b", "gate", "pre_w", "pre_b")}}

    def loss(t):
        f = R.forward(t["h"], t["y"], {**p, **{k: v for k, v in t.items() if k not in ("h", "y")}})
        return (f["h"] * av).sum() + (f["x"] * bv).sum()
    f = R.forward(hv, yv, p)
    _, mag = R.backward(av, bv, f["yh"], f["xh"], f["stats"], p)
    for name, v in t.items():
        m = mag["d" + name]
        for _ in range(3):
            u = rng.choice([-1.0, 1.0], v.shape)
            slope = (loss({**t, name: v + 1e-5 * u}) - loss({**t, name: v - 1e-5 * u})) / 2e-5
            have = (got[name].double().cpu().numpy().reshape(v.shape) * u).sum()
            # each term off by 2^-6 of its magnitude (times the largest |normalised| value, below 5), in
            # random directions: five standard deviations
            assert abs(slope - have) <= 5 * 2.0 ** -6 * 5 * np.sqrt((m.reshape(v.shape) ** 2).sum()) + 1e-6, name


@pytest.mark.parametrize("pad", [0, 1])
def test_rows_past_32_bits(env, pad):  # noqa: F811
    """2.3 G elements: the last rows of both passes against a call on those rows alone."""
    torch, z = env
    rows, cols, last = 140000, 16384 - 8, 3
    ld = cols + pad
    new = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    h, y, x = new(rows, ld), new(rows, ld), new(rows, ld)
    h[-last:].normal_(), y[-last:].normal_()
    size = z.zero_act_row_bytes(cols)
    cy, cx = new(rows, size, dtype=torch.uint8), new(rows, size, dtype=torch.uint8)
    st = new(rows, 4, dtype=torch.float32)

    def forward(n, h, y, x, cy, cx, st):
        z.zero_norm_forward(z.norm(R.BF16, n, cols, post=R.RMS, pre=R.RMS), h.data_ptr(), ld, y.data_ptr(), ld, h.data_ptr(), ld,
                            x.data_ptr(), ld, cy.data_ptr(), cx.data_ptr(), st.data_ptr(), stream(torch))

    tail = [t[-last:].clone() for t in (h, y, x, cy, cx, st)]
    forward(rows, h, y, x, cy, cx, st)
    forward(last, *tail)
    for a, b in zip((h, y, x, cy, cx, st), tail):
        assert torch.equal(a[-last:], b)

    def backward(n, dh, dx, cy, cx, st, dy):
        norm = z.norm(R.BF16, n, cols, post=R.RMS, pre=R.RMS)
        z.zero_norm_backward(norm, dh.data_ptr(), ld, dx.data_ptr(), ld, cy.data_ptr(), cx.data_ptr(), st.data_ptr(), dh.data_ptr(), ld,
                             dy.data_ptr(), ld, R.BF16, stream=stream(torch))

    tail = [t[-last:].clone() for t in (h, x, cy, cx, st, y)]
    backward(rows, h, x, cy, cx, st, y)
    backward(last, *tail)
    for a, b in zip((h, x, cy, cx, st, y), tail):
        assert torch.equal(a[-last:], b)
