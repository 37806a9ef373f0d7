"""8-bit activation checkpoints on the GPU against a plain 64-bit implementation:
codes, exponents and values bit for bit; weight gradients within the bound that
their output type and fp32 sums allow."""
import numpy as np
import pytest

import act_reference as R

pytestmark = pytest.mark.gpu
U = {R.FP16: 2.0 ** -11, R.BF16: 2.0 ** -8, R.FP32: 2.0 ** -24}     # unit roundoff (bf16: 8 bits)
TINY = {R.FP16: 2.0 ** -25, R.BF16: 2.0 ** -134, R.FP32: 2.0 ** -150}   # half the smallest subnormal


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_sharded_mixed_02_gb300 import build
    build.build()
    import zero_sharded_mixed_02_gb300 as z
    z.lib()
    return torch, z


def kind(torch, dtype):
    return (torch.float16, torch.bfloat16, torch.float32)[dtype]


def device_matrix(torch, x, dtype, pad=0, shift=0):
    """x as a device matrix of the type whose rows are cols + pad apart, starting `shift`
    elements into its allocation; returns (tensor to keep, pointer, ld, the rounded values)."""
    rows, cols = x.shape
    ld = cols + pad
    buf = torch.full((rows * ld + shift + 8,), 77.0, dtype=kind(torch, dtype), device="cuda")
    view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(torch.from_numpy(np.asarray(x)).cuda())
    return buf, view.data_ptr(), ld, view.double().cpu().numpy(), view


def activations(rng, rows, cols, sigma=1.0):
    x = rng.standard_normal((rows, cols)) * sigma
    return x * np.where(rng.random(cols) < 0.02, 20.0, 1.0)


def stream(torch):
    return torch.cuda.current_stream().cuda_stream


def save(torch, z, ptr, dtype, rows, cols, ld):
    ckpt = torch.full((rows, R.row_bytes(cols)), 0xA5, dtype=torch.uint8, device="cuda")
    z.zero_act_save(dtype, ptr, rows, cols, ld, ckpt, stream(torch))
    return ckpt


# ---- save and load ------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols,pad,shift", [
    (1, 1, 0, 0), (1, 7, 0, 1), (3, 31, 1, 0), (2, 32, 0, 0), (5, 33, 3, 0), (1, 768, 0, 0), (7, 771, 2, 1),
    (64, 1600, 0, 0), (33, 1600, 8, 8), (1, 16385, 0, 0), (257, 4096, 0, 0), (4099, 96, 0, 0)])
@pytest.mark.parametrize("dtype", [R.FP16, R.BF16, R.FP32])
def test_save_and_load_bitwise(env, rows, cols, pad, shift, dtype):
    torch, z = env
    rng = np.random.default_rng(rows * 31 + cols)
    x = activations(rng, rows, cols) * 10.0 ** rng.uniform(-3, 2, (rows, 1))
    if cols > 64:
        x[:, 32:64] = 0.0                                       # a block of zeros
    keep, ptr, ld, xv, _ = device_matrix(torch, x, dtype, pad, shift)
    ckpt = save(torch, z, ptr, dtype, rows, cols, ld)
    want = R.quantize(xv, dtype)
    got = ckpt.cpu().numpy()
    assert np.array_equal(got, want)
    out = torch.full((rows * ld + shift + 8,), 55.0, dtype=kind(torch, dtype), device="cuda")
    view = out[shift:shift + rows * ld].view(rows, ld)
    z.zero_act_load(dtype, ckpt, rows, cols, view.data_ptr(), ld, stream(torch))
    assert np.array_equal(view[:, :cols].double().cpu().numpy(), R.values(want, cols))
    assert bool((view[:, cols:] == 55.0).all()) and bool((out[:shift] == 55.0).all())   # nothing else written


@pytest.mark.parametrize("dtype", [R.FP16, R.BF16, R.FP32])
def test_save_at_the_types_edges(env, dtype):
    """Largest values (where the exponent is cut and codes are clamped), subnormals, exact ties,
    blocks whose largest value sits on either side of 127 * 2^e, infinities and NaN."""
    torch, z = env
    t = kind(torch, dtype)
    big, small = torch.finfo(t).max, torch.finfo(t).tiny
    ulp = {R.FP16: 2.0 ** -10, R.BF16: 2.0 ** -7, R.FP32: 2.0 ** -23}[dtype]
    rng = np.random.default_rng(5)
    rows = []
    for top in (big, -big, big * (1 - ulp), small, small * ulp, small * ulp * 3, 127.0 * 2.0 ** -6,
                127.0 * 2.0 ** -6 * (1 + ulp), 127.0 * 2.0 ** -6 * (1 - ulp), 1.0, -2.0):
        r = rng.uniform(-1, 1, 64) * abs(top)
        r[17], r[40] = top, -top
        rows.append(r)
    ties = (rng.integers(-126, 126, 64) + 0.5) * 0.25
    ties[[3, 50]] = 127 * 0.25
    rows.append(ties)
    for bad in (np.inf, -np.inf, np.nan):
        r = rng.standard_normal(64)
        r[9] = bad                                              # the first block alone
        rows.append(r)
    x = np.stack(rows)
    keep, ptr, ld, xv, _ = device_matrix(torch, x, dtype)
    ckpt = save(torch, z, ptr, dtype, len(x), 64, ld)
    want = R.quantize(xv, dtype)
    assert np.array_equal(ckpt.cpu().numpy(), want)
    out = torch.empty(len(x), 64, dtype=t, device="cuda")
    z.zero_act_load(dtype, ckpt, len(x), 64, out, 64, stream(torch))
    got = out.double().cpu().numpy()
    assert np.array_equal(got, R.values(want, 64), equal_nan=True)
    assert np.isnan(got[-3:, :32]).all() and np.isfinite(got[-3:, 32:]).all()


def test_load_in_another_type_rounds(env):
    """A bf16 checkpoint read as fp16 and as fp32: the values rounded to the type asked for."""
    torch, z = env
    rng = np.random.default_rng(8)
    x = rng.standard_normal((16, 256)) * 10.0 ** rng.uniform(-9, 6, (16, 1))
    keep, ptr, ld, xv, _ = device_matrix(torch, x, R.BF16)
    ckpt = save(torch, z, ptr, R.BF16, 16, 256, ld)
    v = torch.from_numpy(R.values(R.quantize(xv, R.BF16), 256))
    for dtype in (R.FP16, R.FP32):
        out = torch.empty(16, 256, dtype=kind(torch, dtype), device="cuda")
        z.zero_act_load(dtype, ckpt, 16, 256, out, 256, stream(torch))
        assert torch.equal(out.cpu(), v.float().to(kind(torch, dtype)))


def test_rows_of_a_checkpoint_are_a_checkpoint(env):
    torch, z = env
    rng = np.random.default_rng(3)
    keep, ptr, ld, xv, _ = device_matrix(torch, rng.standard_normal((50, 100)), R.BF16)
    ckpt = save(torch, z, ptr, R.BF16, 50, 100, ld)
    out = torch.empty(7, 100, dtype=torch.bfloat16, device="cuda")
    z.zero_act_load(R.BF16, ckpt[20:27], 7, 100, out, 100, stream(torch))
    assert np.array_equal(out.double().cpu().numpy(), R.values(R.quantize(xv[20:27], R.BF16), 100))


def test_save_and_load_on_another_stream(env):
    torch, z = env
    rng = np.random.default_rng(4)
    keep, ptr, ld, xv, view = device_matrix(torch, rng.standard_normal((300, 640)), R.FP16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ckpt = save(torch, z, ptr, R.FP16, 300, 640, ld)
        out = torch.empty(300, 640, dtype=torch.float16, device="cuda")
        z.zero_act_load(R.FP16, ckpt, 300, 640, out, 640, side.cuda_stream)
    side.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), R.values(R.quantize(xv, R.FP16), 640))


# ---- the weight gradient ------------------------------------------------------------

def wgrad_case(env, tokens, n, k, dtype, grad, pad=0, shift=0, affine=False, bias=True, dw_pad=0, dw_shift=0,
               accumulate=0, work=None, seed=0, edit=None):
    """Runs one weight gradient and checks it; returns (dw, db, work)."""
    torch, z = env
    rng = np.random.default_rng(seed + tokens + 7 * n + 13 * k)
    dy = rng.standard_normal((tokens, n)) * 0.05
    x = activations(rng, tokens, k)
    if edit:
        edit(dy, x)
    kdy, pdy, ldy, dyv, _ = device_matrix(torch, dy, dtype, pad, shift)
    kx, px, ldx, xv, _ = device_matrix(torch, x, dtype)
    ckpt = save(torch, z, px, dtype, tokens, k, ldx) if tokens else None
    xq = R.values(R.quantize(xv, dtype), k) if tokens else np.zeros((0, k))
    cs = sh = None
    csv, shv = np.ones(k), np.zeros(k)
    if affine:
        cs = torch.from_numpy(1 + 0.3 * rng.standard_normal(k)).to(kind(torch, dtype)).cuda()
        sh = torch.from_numpy(0.3 * rng.standard_normal(k)).to(kind(torch, dtype)).cuda()
        csv, shv = cs.double().cpu().numpy(), sh.double().cpu().numpy()
    ldw = k + dw_pad
    dw = torch.from_numpy(rng.standard_normal(n * ldw + dw_shift + 8)).to(kind(torch, grad)).cuda()
    db = torch.from_numpy(rng.standard_normal(n)).to(kind(torch, grad)).cuda() if bias else None
    dw0, db0 = dw.double().cpu().numpy(), db.double().cpu().numpy() if bias else None
    if work is None:
        work = torch.zeros(z.zero_act_wgrad_workspace(tokens, n, k), dtype=torch.uint8, device="cuda")
    z.zero_act_wgrad(dtype, pdy, tokens, n, ldy, ckpt, k, cs, sh, grad, dw[dw_shift:].data_ptr(), ldw, db,
                     accumulate, work, stream(torch))
    torch.cuda.synchronize()
    assert int(work[:4].view(torch.int32)[0]) == 0
    place = slice(dw_shift, dw_shift + n * ldw)
    got = dw.double().cpu().numpy()
    inside = got[place].reshape(n, ldw)[:, :k]
    outside = np.ones(got.size, bool)
    outside[place].reshape(n, ldw)[:, :k] = False
    assert np.array_equal(got[outside], dw0[outside])            # nothing else written
    old = dw0[place].reshape(n, ldw)[:, :k] if accumulate else 0.0
    s = dyv.sum(0)
    want = (dyv.T @ xq) * csv + s[:, None] * shv + old
    with np.errstate(invalid="ignore"):
        mag = (np.abs(dyv).T @ np.abs(xq)) * np.abs(csv) + np.abs(dyv).sum(0)[:, None] * np.abs(shv)
    # one rounding to the type; fp32 sums whose every step may lose a unit in the last place
    # (the tensor cores truncate): at most (tokens + 8) 2^-23 of the magnitudes summed
    def near(got, want, mag):
        fine = np.isfinite(want)
        assert np.array_equal(fine, np.isfinite(got))
        tol = U[grad] * np.abs(want) + TINY[grad] + (tokens + 8) * 2.0 ** -23 * (mag + np.abs(want))
        assert np.all(np.abs(got - want)[fine] <= tol[fine])
        # errors of many roundings do not all point one way: their 2-norm against the result's
        w = want[fine]
        if w.size and np.linalg.norm(w):
            rel = np.linalg.norm((got - want)[fine]) / np.linalg.norm(w)
            assert rel <= U[grad] + max(tokens, 64) * 2.0 ** -24, rel
    near(inside, want, mag)
    if bias:
        near(db.double().cpu().numpy(), s + (db0 if accumulate else 0.0), np.abs(dyv).sum(0))
    return dw, db, work


SIZES = [(1, 1, 1), (1, 8, 8), (1, 300, 500), (2, 16, 32), (63, 64, 64), (64, 128, 128), (65, 130, 129),
         (16, 768, 768), (127, 256, 256), (129, 257, 255), (200, 100, 40), (1000, 776, 771), (512, 1600, 520)]


@pytest.mark.parametrize("tokens,n,k", SIZES)
@pytest.mark.parametrize("dtype,grad", [(R.BF16, R.BF16), (R.FP16, R.FP16), (R.BF16, R.FP32), (R.FP16, R.FP32)])
def test_wgrad(env, tokens, n, k, dtype, grad):
    wgrad_case(env, tokens, n, k, dtype, grad)


@pytest.mark.parametrize("tokens,n,k", [(100, 136, 264), (333, 520, 96), (1, 40, 72), (700, 300, 300)])
@pytest.mark.parametrize("dtype", [R.BF16, R.FP16])
@pytest.mark.parametrize("pad,shift,dw_pad,dw_shift", [(1, 0, 0, 0), (0, 1, 3, 1), (8, 8, 8, 8), (3, 2, 0, 1)])
def test_wgrad_strides_and_alignment(env, tokens, n, k, dtype, pad, shift, dw_pad, dw_shift):
    wgrad_case(env, tokens, n, k, dtype, dtype, pad, shift, dw_pad=dw_pad, dw_shift=dw_shift)


@pytest.mark.parametrize("tokens,n,k", [(1, 24, 40), (300, 264, 776), (4100, 128, 256)])
@pytest.mark.parametrize("dtype,grad", [(R.BF16, R.BF16), (R.FP16, R.FP32)])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_wgrad_with_the_norms_weight_and_bias(env, tokens, n, k, dtype, grad, accumulate):
    wgrad_case(env, tokens, n, k, dtype, grad, affine=True, accumulate=accumulate)
    wgrad_case(env, tokens, n, k, dtype, grad, affine=True, bias=False, accumulate=accumulate)


@pytest.mark.parametrize("tokens,n,k", [(20000, 64, 64), (30011, 776, 771), (9000, 8, 2000), (12345, 300, 32)])
@pytest.mark.parametrize("grad", [R.BF16, R.FP32])
def test_wgrad_long_token_axis(env, tokens, n, k, grad):
    wgrad_case(env, tokens, n, k, R.BF16, grad)


def test_wgrad_without_tokens(env):
    torch, z = env
    for accumulate in (0, 1):
        wgrad_case(env, 0, 40, 72, R.BF16, R.BF16, accumulate=accumulate)


def test_wgrad_workspace_serves_calls_of_other_sizes(env):
    """One workspace, zeroed once, for a sequence of calls that split their work differently; and
    equal inputs give equal bits."""
    torch, z = env
    sizes = [(20000, 64, 64), (64, 900, 1100), (3000, 520, 520), (1, 8, 8), (20000, 64, 64), (3000, 520, 520)]
    work = torch.zeros(max(z.zero_act_wgrad_workspace(*s) for s in sizes), dtype=torch.uint8, device="cuda")
    seen = {}
    for s in sizes:
        dw, db, _ = wgrad_case(env, *s, R.BF16, R.FP32, work=work)
        if s in seen:
            assert torch.equal(seen[s][0], dw) and torch.equal(seen[s][1], db)
        seen[s] = (dw, db)


@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64, 65])
@pytest.mark.parametrize("n,k,pad,shift", [(64, 128, 0, 0), (130, 257, 1, 1), (1, 33, 3, 1), (768, 768, 0, 0)])
@pytest.mark.parametrize("dtype,grad,accumulate", [(R.BF16, R.BF16, 0), (R.FP16, R.FP32, 1), (R.FP16, R.FP16, 1)])
def test_wgrad_of_few_tokens(env, tokens, n, k, pad, shift, dtype, grad, accumulate):
    wgrad_case(env, tokens, n, k, dtype, grad, pad=pad, shift=shift, affine=tokens % 2 == 1, dw_pad=pad, dw_shift=shift,
               accumulate=accumulate)


@pytest.mark.parametrize("tokens,n,k,grad,affine", [(300, 4200, 5200, R.BF16, False), (130, 5000, 6272, R.BF16, True),
                                                    (1020, 2500, 9000, R.FP32, False)])
def test_wgrad_of_many_tiles(env, tokens, n, k, grad, affine):
    """More tiles than the device takes at a time, so that buffers stay full while a tile is written
    out and the next one's operands wait."""
    wgrad_case(env, tokens, n, k, R.BF16, grad, affine=affine)


@pytest.mark.parametrize("tokens,n,k,grad", [(30011, 776, 771, R.FP32), (8192, 1024, 1024, R.BF16), (700, 40, 100, R.BF16)])
def test_wgrad_gives_equal_bits_over_many_calls(env, tokens, n, k, grad):
    """Loads that land in another order must not be taken for one another: the same call, with other
    work on the stream between some of them, gives the same bits each time."""
    torch, z = env
    dw, db, work = wgrad_case(env, tokens, n, k, R.BF16, grad)
    rng = np.random.default_rng(tokens + 7 * n + 13 * k)
    dy = torch.from_numpy(rng.standard_normal((tokens, n)) * 0.05).to(torch.bfloat16).cuda()
    x = torch.from_numpy(activations(rng, tokens, k)).to(torch.bfloat16).cuda()
    ckpt = save(torch, z, x.data_ptr(), R.BF16, tokens, k, k)
    first, other = None, torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    for i in range(400):
        dw, db = (torch.empty(n, k, device="cuda", dtype=kind(torch, grad)), torch.empty(n, device="cuda", dtype=kind(torch, grad)))
        if i % 3 == 0:
            other.fill_(i & 127)                                 # the operands leave the cache
        z.zero_act_wgrad(R.BF16, dy, tokens, n, n, ckpt, k, None, None, grad, dw, k, db, 0, work, stream(torch))
        if first is None:
            first = (dw, db)
        assert torch.equal(first[0], dw) and torch.equal(first[1], db), i
    assert int(work[:4].view(torch.int32)[0]) == 0


@pytest.mark.parametrize("what", ["dy", "x"])
def test_wgrad_carries_non_finite_values(env, what):
    """An infinity or NaN in dy reaches its column's gradients; in x, its block's: what the step's
    overflow flag looks for."""
    def edit(dy, x):
        if what == "dy":
            dy[70, 5] = np.nan
        else:
            x[70, 40] = np.inf
    torch, z = env
    dw, db, _ = wgrad_case(env, 150, 64, 96, R.BF16, R.FP32, bias=True, edit=edit)
    got = np.isfinite(dw[:64 * 96].view(64, 96).cpu().numpy())
    if what == "dy":
        assert not got[5].any() and got[:5].all() and got[6:].all()
    else:
        assert not got[:, 32:64].any() and got[:, :32].all() and got[:, 64:].all()


def test_wgrad_fp16_refuses_no_exponent_silently(env):
    """A checkpoint saved as bf16 with values beyond fp16's range, used with fp16 dy, reads as NaN."""
    torch, z = env
    x = torch.ones(64, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 32:] = 1e6
    ckpt = save(torch, z, x.data_ptr(), R.BF16, 64, 64, 64)
    dy = torch.ones(64, 64, dtype=torch.float16, device="cuda")
    dw = torch.zeros(64, 64, device="cuda")
    work = torch.zeros(z.zero_act_wgrad_workspace(64, 64, 64), dtype=torch.uint8, device="cuda")
    z.zero_act_wgrad(R.FP16, dy, 64, 64, 64, ckpt, 64, None, None, R.FP32, dw, 64, None, 0, work, stream(torch))
    got = dw.cpu().numpy()
    assert np.all(got[:, :32] == 64.0) and np.isnan(got[:, 32:]).all()


def test_wgrad_against_differences(env):
    """sum(dY * (x W^T)) is linear in W: its slope along any direction is the gradient's, up to the
    gradient's own rounding."""
    torch, z = env
    rng = np.random.default_rng(2)
    tokens, n, k = 96, 72, 136
    kdy, pdy, ldy, dyv, _ = device_matrix(torch, rng.standard_normal((tokens, n)), R.BF16)
    kx, px, ldx, xv, _ = device_matrix(torch, rng.standard_normal((tokens, k)), R.BF16)
    ckpt = save(torch, z, px, R.BF16, tokens, k, ldx)
    xq = R.values(R.quantize(xv, R.BF16), k)
    dw = torch.empty(n, k, device="cuda")
    work = torch.zeros(z.zero_act_wgrad_workspace(tokens, n, k), dtype=torch.uint8, device="cuda")
    z.zero_act_wgrad(R.BF16, pdy, tokens, n, ldy, ckpt, k, None, None, R.FP32, dw, k, None, 0, work, stream(torch))
    got = dw.double().cpu().numpy()
    w = rng.standard_normal((n, k))
    for _ in range(4):
        u = rng.standard_normal((n, k))
        slope = ((dyv * (xq @ (w + u).T)).sum() - (dyv * (xq @ (w - u).T)).sum()) / 2
        room = (tokens + 8) * 2.0 ** -23 * ((np.abs(dyv).T @ np.abs(xq)) * np.abs(u)).sum()
        assert abs(slope - (got * u).sum()) <= room


# ---- offsets past 32 bits -------------------------------------------------------------

def test_checkpoints_past_32_bits(env):
    """4.6 G elements: rows at both ends against the same rows alone."""
    torch, z = env
    rows, cols = 70001, 65536
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:3].normal_(), x[-3:].normal_()
    ckpt = save(torch, z, x.data_ptr(), R.BF16, rows, cols, cols)
    for part in (slice(0, 3), slice(rows - 3, rows)):
        alone = save(torch, z, x[part].data_ptr(), R.BF16, 3, cols, cols)
        assert torch.equal(ckpt[part], alone)
    assert not ckpt[3:6, :cols].any()
    out = torch.full((rows, cols + 1), 7.0, dtype=torch.bfloat16, device="cuda")          # unaligned rows
    z.zero_act_load(R.BF16, ckpt, rows, cols, out, cols + 1, stream(torch))
    want = torch.empty(3, cols, dtype=torch.bfloat16, device="cuda")
    z.zero_act_load(R.BF16, ckpt[-3:], 3, cols, want, cols, stream(torch))
    assert torch.equal(out[-3:, :cols], want) and bool((out[-5:, cols] == 7.0).all()) and not out[3:6, :cols].any()
    again = save(torch, z, out.data_ptr(), R.BF16, rows, cols, cols + 1)
    assert torch.equal(again[-3:], ckpt[-3:])


@pytest.mark.parametrize("shift", [0, 1])
def test_wgrad_past_32_bits(env, shift):
    """dy of 2.2 G elements, zero but for its first and last tokens."""
    torch, z = env
    tokens, n, k = (1 << 21) + 5, 1040, 40
    rng = np.random.default_rng(1)
    store = torch.zeros(tokens * n + 8, dtype=torch.bfloat16, device="cuda")
    dy = store[shift:shift + tokens * n].view(tokens, n)
    x = torch.randn(tokens, k, device="cuda").to(torch.bfloat16)
    ckpt = save(torch, z, x.data_ptr(), R.BF16, tokens, k, k)
    pick = [0, 1, 70, tokens - 66, tokens - 2, tokens - 1]
    for t in pick:
        dy[t] = torch.from_numpy(rng.standard_normal(n)).to(torch.bfloat16).cuda()
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    work = torch.zeros(z.zero_act_wgrad_workspace(tokens, n, k), dtype=torch.uint8, device="cuda")
    z.zero_act_wgrad(R.BF16, dy.data_ptr(), tokens, n, n, ckpt, k, None, None, R.FP32, dw, k, db, 0, work, stream(torch))
    assert int(work[:4].view(torch.int32)[0]) == 0
    xq = R.values(ckpt[pick].cpu().numpy(), k)
    d = dy[pick].double().cpu().numpy()
    # six terms and zeros: a few units in the last place of the magnitudes
    assert np.all(np.abs(dw.double().cpu().numpy() - d.T @ xq) <= 2.0 ** -20 * (np.abs(d).T @ np.abs(xq)) + 1e-30)
    assert np.all(np.abs(db.double().cpu().numpy() - d.sum(0)) <= 2.0 ** -20 * np.abs(d).sum(0) + 1e-30)
