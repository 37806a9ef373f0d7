"""Plain 64-bit implementations of the 8-bit activation checkpoint and of the norms
around a block, for the tests.  numpy only; shares nothing with the library."""
import numpy as np

FP16, BF16, FP32 = 0, 1, 2
LIMITS = {FP16: (-24, 9), BF16: (-126, 121), FP32: (-126, 121)}
NONE, RMS, LAYER = 0, 1, 2


def wide_of(cols):
    return -(-cols // 32) * 32


def row_bytes(cols):
    return -(-(wide_of(cols) * 33 // 32) // 32) * 32


def quantize(x, dtype):
    """64-bit rows -> the checkpoint's bytes [rows, row_bytes]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    wide = wide_of(cols)
    blocks = np.zeros((rows, wide))
    blocks[:, :cols] = x
    blocks = blocks.reshape(rows, wide // 32, 32)
    top = np.abs(blocks).max(-1)
    bad = ~np.isfinite(top)
    lo, hi = LIMITS[dtype]
    # smallest e with top <= 127 * 2^e: top / 127 compared exactly through integers
    m, p = np.frexp(np.where(bad, 1.0, top))                 # top = m 2^p, m in [1/2, 1)
    e = np.where(m * 128 <= 127, p - 7, p - 6)               # 127 * 2^(p - 7) = (127/128) 2^p
    e = np.clip(np.where(top == 0, lo, e), lo, hi)
    with np.errstate(invalid="ignore", over="ignore"):
        codes = np.clip(np.rint(np.ldexp(blocks, -e[..., None])), -127, 127)
    codes = np.where(bad[..., None], 0, codes)
    out = np.zeros((rows, row_bytes(cols)), np.uint8)
    out[:, :wide] = codes.reshape(rows, wide).astype(np.int8).view(np.uint8)
    out[:, wide:wide + wide // 32] = np.where(bad, 255, e + 127).astype(np.uint8)
    return out


def values(ckpt, cols):
    """The checkpoint's bytes -> 64-bit values."""
    wide = wide_of(cols)
    codes = ckpt[:, :wide].view(np.int8).astype(np.float64)
    e = ckpt[:, wide:wide + wide // 32].astype(np.int64)
    unit = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    return (codes * np.repeat(unit, 32, axis=1))[:, :cols]


def exponents(ckpt, cols):
    wide = wide_of(cols)
    return ckpt[:, wide:wide + wide // 32].astype(np.int64)


def normalise(v, kind, eps):
    """(normalised rows, mean, 1/deviation), in 64 bits."""
    n = v.shape[0]
    if kind == NONE:
        return v, np.zeros(n), np.ones(n)
    mean = v.mean(1) if kind == LAYER else np.zeros(n)
    d = v - mean[:, None]
    r = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * r[:, None], mean, r


def one(v, other):
    return other if v is None else np.asarray(v, np.float64)


def gate_rows(gate, rows, group):
    if gate is None:
        return np.ones((1, 1))
    if group == 0:
        return gate
    return gate[np.arange(rows) // group]


def forward(h, y, p):
    """p: dict of post, pre, eps, alpha, group, post_w, post_b, gate, pre_w, pre_b.
    Returns dict h, x, yh, xh, stats."""
    if y is None:
        out, yh = h, None
        mu2, r2 = np.zeros(len(h)), np.ones(len(h))
    else:
        yh, mu2, r2 = normalise(y, p["post"], p["eps"])
        z = yh * one(p["post_w"], 1.0) + one(p["post_b"], 0.0)
        out = h + p["alpha"] * gate_rows(p["gate"], len(h), p["group"]) * z
    xh, mu1, r1 = normalise(out, p["pre"], p["eps"])
    x = xh * one(p["pre_w"], 1.0) + one(p["pre_b"], 0.0) if p["pre"] != NONE else None
    return {"h": out, "x": x, "yh": yh, "xh": xh, "stats": np.stack([mu2, r2, mu1, r1], 1)}


def group_sums(v, group):
    if group == 0 or len(v) == 0:
        return v.sum(0, keepdims=True)
    return np.add.reduceat(v, np.arange(0, len(v), group), axis=0)


def backward(dh_out, dx, yh, xh, stats, p):
    """Gradients, and for each an array of the magnitudes its rounding errors scale with."""
    rows = len(stats)
    d = np.zeros((rows, p["cols"])) if dh_out is None else dh_out
    mag = np.abs(d)
    out, big = {}, {}
    r2, r1 = stats[:, 1:2], stats[:, 3:4]
    if p["pre"] != NONE:
        g = dx * one(p["pre_w"], 1.0)
        m0 = g.mean(1, keepdims=True) if p["pre"] == LAYER else 0.0
        a0 = np.abs(g).mean(1, keepdims=True) if p["pre"] == LAYER else 0.0
        d = d + r1 * (g - m0 - xh * (g * xh).mean(1, keepdims=True))
        mag = mag + r1 * (np.abs(g) + a0 + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
        out["dpre_w"], out["dpre_b"] = (dx * xh).sum(0), dx.sum(0)
        big["dpre_w"], big["dpre_b"] = np.abs(dx * xh).sum(0), np.abs(dx).sum(0)
    out["dh"], big["dh"] = d, mag
    if yh is None:
        yh = np.zeros((rows, p["cols"]))
    g2 = p["alpha"] * gate_rows(p["gate"], rows, p["group"])
    w2 = one(p["post_w"], 1.0)
    z = yh * w2 + one(p["post_b"], 0.0)
    az = np.abs(yh * w2) + np.abs(one(p["post_b"], 0.0))
    out["dgate"] = group_sums(p["alpha"] * d * z, p["group"])
    big["dgate"] = group_sums(abs(p["alpha"]) * mag * az, p["group"])
    dz, mz = g2 * d, np.abs(g2) * mag
    dy, my = dz, mz
    if p["post"] != NONE:
        out["dpost_w"], out["dpost_b"] = (dz * yh).sum(0), dz.sum(0)
        big["dpost_w"], big["dpost_b"] = (mz * np.abs(yh)).sum(0), mz.sum(0)
        g, mg = dz * w2, mz * np.abs(w2)
        m0 = g.mean(1, keepdims=True) if p["post"] == LAYER else 0.0
        a0 = mg.mean(1, keepdims=True) if p["post"] == LAYER else 0.0
        dy = r2 * (g - m0 - yh * (g * yh).mean(1, keepdims=True))
        my = r2 * (mg + a0 + np.abs(yh) * (mg * np.abs(yh)).mean(1, keepdims=True))
    out["dy"], big["dy"] = dy, my
    return out, big
