"""The 8-bit activation checkpoint and block-norm entry points without a GPU: the
checkpoint layout, the workspace sizes, and invalid arguments refused before
anything touches CUDA; and the 64-bit reference gradients against differences."""
import shutil

import numpy as np
import pytest

import act_reference as R

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


@pytest.mark.parametrize("cols", [1, 31, 32, 33, 64, 768, 992, 993, 1600, 4096, 14336, 1 << 24])
def test_row_bytes(z, cols):
    assert z.zero_act_row_bytes(cols) == R.row_bytes(cols)


def test_row_bytes_invalid(z):
    assert [z.zero_act_row_bytes(c) for c in (0, -1, (1 << 24) + 1)] == [0, 0, 0]


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(ld=63),
    dict(cols=(1 << 24) + 1, ld=1 << 25), dict(x=None), dict(x=P + 1), dict(ckpt=None), dict(ckpt=P + 8),
    dict(dtype=2, x=P + 2)])
def test_save_and_load_refusals(z, bad):
    a = dict(dtype=1, x=P, rows=4, cols=64, ld=64, ckpt=P)
    a.update(bad)
    refused(z, z.zero_act_save, a["dtype"], a["x"], a["rows"], a["cols"], a["ld"], a["ckpt"])
    refused(z, z.zero_act_load, a["dtype"], a["ckpt"], a["rows"], a["cols"], a["x"], a["ld"])


def test_no_rows_is_accepted(z):
    z.zero_act_save(1, None, 0, 64, 64, None)
    z.zero_act_load(1, None, 0, 64, None, 64)
    z.zero_norm_forward(z.norm(1, 0, 64), None, 64, None, 64, None, 64, None, 64)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(grad=0), dict(grad=3), dict(tokens=-1), dict(tokens=1 << 31), dict(n=0),
    dict(n=(1 << 24) + 1, ldy=1 << 25), dict(k=0), dict(ldy=63), dict(ldw=31), dict(dy=None),
    dict(dy=P + 1), dict(ckpt=None), dict(ckpt=P + 8), dict(dw=None), dict(dw=P + 1),
    dict(grad=2, dw=P + 2), dict(db=P + 1), dict(scale=P + 1), dict(shift=P + 1), dict(work=None),
    dict(work=P + 8)])
def test_wgrad_refusals(z, bad):
    a = dict(dtype=1, dy=P, tokens=8, n=64, ldy=64, ckpt=P, k=32, scale=None, shift=None, grad=1, dw=P,
             ldw=32, db=None, work=P)
    a.update(bad)
    refused(z, z.zero_act_wgrad, a["dtype"], a["dy"], a["tokens"], a["n"], a["ldy"], a["ckpt"], a["k"],
            a["scale"], a["shift"], a["grad"], a["dw"], a["ldw"], a["db"], 0, a["work"])


def test_wgrad_workspace(z):
    assert z.zero_act_wgrad_workspace(8192, 6400, 1600) >= 16
    for bad in ((-1, 64, 64), (8, 0, 64), (8, 64, 0), (1 << 31, 64, 64)):
        assert z.zero_act_wgrad_workspace(*bad) == 0


DESCRIPTIONS = [
    dict(dtype=2), dict(res_dtype=0), dict(res_dtype=3), dict(post=3), dict(pre=-1), dict(rows=-1),
    dict(cols=0), dict(cols=16385), dict(group_rows=-1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(alpha=float("inf")), dict(post=0), dict(pre=0), dict(pre_w=P + 1), dict(gate=P + 1)]


def description(z, **kw):
    d = dict(dtype=1, rows=4, cols=64, post=1, pre=1, post_w=P, pre_w=P)
    d.update(kw)
    return z.norm(d.pop("dtype"), d.pop("rows"), d.pop("cols"), **d)


@pytest.mark.parametrize("bad", DESCRIPTIONS)
def test_norm_descriptions_refused(z, bad):
    n = description(z, **bad)
    refused(z, z.zero_norm_forward, n, P, 1 << 16, P, 1 << 16, P, 1 << 16, P, 1 << 16)
    refused(z, z.zero_norm_backward, n, P, 1 << 16, P, 1 << 16, P, P, P, P, 1 << 16, P, 1 << 16, 1, work=P)
    assert z.zero_norm_workspace(n) == 0


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(h=P + 1), dict(ldh=63), dict(y=None), dict(ldy=63), dict(h_out=None), dict(x=None),
    dict(ldx=1), dict(ckpt_y=P + 4), dict(ckpt_x=P + 4), dict(stats=P + 4)])
def test_norm_forward_refusals(z, bad):
    a = dict(h=P, ldh=64, y=P, ldy=64, h_out=P, ldho=64, x=P, ldx=64, ckpt_y=None, ckpt_x=None, stats=None)
    a.update(bad)
    refused(z, z.zero_norm_forward, description(z), *a.values())


def test_norm_forward_without_a_block_refuses_its_parts(z):
    for kw in (dict(post=1, post_w=None), dict(post=0, post_w=None, gate=P)):
        refused(z, z.zero_norm_forward, description(z, **kw), P, 64, None, 0, None, 0, P, 64)
    refused(z, z.zero_norm_forward, description(z, post=0, post_w=None), P, 64, None, 0, None, 0, P, 64, P)
    refused(z, z.zero_norm_forward, description(z, pre=0, pre_w=None), P, 64, P, 64, P, 64, P, 64)


@pytest.mark.parametrize("bad", [
    dict(dh_out=P + 1), dict(dx=None), dict(ckpt_x=None), dict(ckpt_y=None), dict(stats=None),
    dict(stats=P + 4), dict(dh=None, dy=None), dict(dy=None), dict(lddx=1), dict(lddh=1), dict(lddy=1),
    dict(grad=0), dict(grad=3), dict(work=None), dict(work=P + 8), dict(dpre_w=P + 1),
    dict(grad=2, dgate=P + 2)])
def test_norm_backward_refusals(z, bad):
    a = dict(dh_out=P, lddho=64, dx=P, lddx=64, ckpt_y=P, ckpt_x=P, stats=P, dh=P, lddh=64, dy=P, lddy=64,
             grad=1, dpost_w=P, dpost_b=None, dgate=P, dpre_w=P, dpre_b=None, accumulate=0, work=P)
    a.update(bad)
    refused(z, z.zero_norm_backward, description(z), *a.values())


def test_norm_backward_refuses_gradients_of_absent_norms(z):
    a = [P, 64, P, 64, P, P, P, P, 64, P, 64, 1]
    refused(z, z.zero_norm_backward, description(z, post=0, post_w=None), *a, dpost_w=P, work=P)
    no_pre = [P, 64, None, 64, P, None, P, P, 64, P, 64, 1]
    refused(z, z.zero_norm_backward, description(z, pre=0, pre_w=None), *no_pre, dpre_b=P, work=P)


# ---- the 64-bit reference itself --------------------------------------------------------

@pytest.mark.parametrize("post,pre", [(R.RMS, R.RMS), (R.LAYER, R.LAYER), (R.NONE, R.LAYER), (R.RMS, R.NONE)])
@pytest.mark.parametrize("group", [0, 3])
def test_reference_gradients_against_differences(post, pre, group):
    """Central differences of sum(h' A + x B) in every input, in 64 bits: the step 1e-6 leaves
    a truncation error of about 1e-12 and a rounding error of about 1e-16 / 1e-6 = 1e-10 relative
    to the sum of the terms' magnitudes."""
    rng = np.random.default_rng(post * 10 + pre + group)
    rows, cols = 7, 12
    groups = 1 if group == 0 else -(-rows // group)
    t = {"h": rng.standard_normal((rows, cols)), "y": rng.standard_normal((rows, cols)),
         "gate": 0.5 + rng.random((groups, cols))}
    for w, on in (("post_w", post), ("post_b", post), ("pre_w", pre), ("pre_b", pre)):
        t[w] = rng.standard_normal(cols) if on else None
    a, b = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))

    def params(t):
        return dict(post=post, pre=pre, eps=1e-5, alpha=0.7, group=group, cols=cols, **{
            k: t[k] for k in ("post_w", "post_b", "gate", "pre_w", "pre_b")})

    def loss(t):
        f = R.forward(t["h"], t["y"], params(t))
        return (f["h"] * a).sum() + ((f["x"] * b).sum() if pre else 0.0)

    f = R.forward(t["h"], t["y"], params(t))
    got, _ = R.backward(a, b if pre else None, f["yh"], f["xh"], f["stats"], params(t))
    got["dh_in"] = got.pop("dh")
    names = {"h": "dh_in", "y": "dy"}
    for name, v in t.items():
        if v is None:
            continue
        grad = got[names.get(name, "d" + name)]
        for _ in range(4):
            u = rng.standard_normal(v.shape)
            up, down = dict(t), dict(t)
            up[name], down[name] = v + 1e-6 * u, v - 1e-6 * u
            slope = (loss(up) - loss(down)) / 2e-6
            assert abs(slope - (grad * u).sum()) < 1e-7 * (1 + np.abs(a).sum() + np.abs(b).sum())
