"""The activation-checkpoint and block-norm operators: cases, inputs, plain forms and exact values.

Operators (the C entry points of include/zero_b200.h, through the Python binding):

  act_save       x -> an 8-bit checkpoint, and back to the values it stands for
  act_load       an 8-bit checkpoint -> 16-bit values
  act_wgrad      a linear layer's weight (and bias) gradient from dy and the 8-bit checkpoint of its input
  norm_forward   the norm after a block, its gate and residual scale, the residual sum and the norm before the
                 next block, with the 8-bit checkpoints and statistics that the backward pass reads
  norm_backward  its gradients

``own`` False computes the plain form (elementary torch operations in 32 bits, rounded once at the end);
``own`` True calls the library.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
CODE = {"fp16": 0, "bf16": 1, "fp32": 2}
LIMITS = {"fp16": (103, 136), "bf16": (1, 248), "fp32": (1, 248)}   # biased block exponents
NORM = {"none": 0, "rms": 1, "layer": 2}
EPS = 1e-5


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # one micro-batch of a small model's block input, kept for the backward pass
        {"name": "save_small", "op": "act_save", "dtype": "bf16", "rows": 512, "cols": 768, "pad": 0},
        # a 16 x 1024 token batch's feed-forward activations of the 1.5B list (h = 1600, ffn = 6400)
        {"name": "save_large", "op": "act_save", "dtype": "fp16", "rows": 16384, "cols": 6400, "pad": 0},
        # odd sizes: a ragged last batch, rows whose stride is no multiple of a vector
        {"name": "load_odd", "op": "act_load", "dtype": "fp16", "rows": 3001, "cols": 771, "pad": 2},
        # the feed-forward activations of the 8B list (ffn = 14336)
        {"name": "load_large", "op": "act_load", "dtype": "bf16", "rows": 8192, "cols": 14336, "pad": 0},
        # the smallest: a handful of tokens (the last, nearly empty micro-batch), bias gradient too
        {"name": "wgrad_small", "op": "act_wgrad", "dtype": "bf16", "tokens": 16, "n": 768, "k": 768,
         "pad": 0, "affine": False, "bias": True, "grad": "bf16"},
        # the 1.5B list's first feed-forward matrix over 8 x 1024 tokens, its input checkpointed as the
        # normalised row (the norm's weight and bias enter the gradient)
        {"name": "wgrad_ordinary", "op": "act_wgrad", "dtype": "bf16", "tokens": 8192, "n": 6400, "k": 1600,
         "pad": 0, "affine": True, "bias": True, "grad": "bf16"},
        # a long, ragged token axis against a small matrix (the work has to be split over tokens),
        # fp32 gradient for accumulation outside
        {"name": "wgrad_long", "op": "act_wgrad", "dtype": "fp16", "tokens": 30011, "n": 776, "k": 771,
         "pad": 0, "affine": False, "bias": False, "grad": "fp32"},
        # the 8B list's down projection over 16 x 1024 tokens
        {"name": "wgrad_large", "op": "act_wgrad", "dtype": "bf16", "tokens": 16384, "n": 4096, "k": 14336,
         "pad": 0, "affine": False, "bias": False, "grad": "bf16"},
        # a single token through a trained block boundary: no checkpoint, latency counts
        {"name": "forward_token", "op": "norm_forward", "dtype": "bf16", "res": "bf16", "rows": 1, "cols": 1600,
         "pad": 0, "post": "rms", "pre": "rms", "bias": False, "group": 0, "alpha": 0.5, "ckpt": False},
        # 16 x 1024 tokens of the 8B list, norms on both sides, one gate per sequence, fp32 residual stream
        {"name": "forward_large", "op": "norm_forward", "dtype": "bf16", "res": "fp32", "rows": 16384,
         "cols": 4096, "pad": 0, "post": "rms", "pre": "rms", "bias": False, "group": 1024, "alpha": 0.7,
         "ckpt": True},
        # odd sizes: layer norms with biases, ragged rows and groups, unaligned strides
        {"name": "backward_odd", "op": "norm_backward", "dtype": "fp16", "res": "fp16", "rows": 2047,
         "cols": 1601, "pad": 0, "post": "layer", "pre": "layer", "bias": True, "group": 300, "alpha": 1.0,
         "grad": "fp32"},
        # 16 x 1024 tokens of the 8B list's width
        {"name": "backward_large", "op": "norm_backward", "dtype": "bf16", "res": "fp32", "rows": 16384,
         "cols": 4096, "pad": 0, "post": "rms", "pre": "rms", "bias": False, "group": 1024, "alpha": 0.7,
         "grad": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _shape(rng, most_rows, lo, hi, most):
    cols = _log_int(rng, lo, hi)
    if rng.random() < 0.6:
        cols = max(lo, cols // 64 * 64)
    rows = _log_int(rng, 1, max(1, min(most_rows, most // cols)))
    return rows, cols


def draw(rng):
    op = rng.choice(["act_save", "act_load", "act_wgrad", "act_wgrad", "norm_forward", "norm_backward"])
    dtype = rng.choice(["fp16", "bf16"])
    pad = rng.choice([0, 0, 0, 1, 8, 64])
    if op in ("act_save", "act_load"):
        rows, cols = _shape(rng, 65536, 32, 16384, 16384 * 6400)
        return {"op": op, "dtype": rng.choice(["fp16", "bf16", "bf16", "fp32"]), "rows": rows, "cols": cols,
                "pad": pad}
    if op == "act_wgrad":
        n, k = _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            n, k = n // 64 * 64, k // 64 * 64
        most = 16384 * 4096 * 14336 // (n * k)
        return {"op": op, "dtype": dtype, "tokens": _log_int(rng, 1, max(1, min(65536, most))), "n": n, "k": k,
                "pad": pad, "affine": rng.random() < 0.4, "bias": rng.random() < 0.4,
                "grad": rng.choice([dtype, dtype, "fp32"])}
    rows, cols = _shape(rng, 32768, 64, 8192, 16384 * 4096)
    post, pre = rng.choice([("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("none", "layer"),
                            ("rms", "none")])
    c = {"op": op, "dtype": dtype, "res": rng.choice([dtype, "fp32"]), "rows": rows, "cols": cols, "pad": pad,
         "post": post, "pre": pre, "bias": rng.random() < 0.5, "group": rng.choice([-1, 0, 1024, 300]),
         "alpha": rng.choice([1.0, 0.5, 0.1])}
    if op == "norm_forward":
        c["ckpt"] = rng.random() < 0.7
    else:
        c["grad"] = rng.choice([dtype, "fp32"])
    return c


# ---- the checkpoint format in plain operations ------------------------------------------------------

def _row_bytes(cols):
    c = -(-cols // 32) * 32
    return -(-(c + c // 32) // 32) * 32


def _quantize(x, dtype):
    """fp32 [rows, cols] -> (codes as fp32 [rows, blocks, 32], biased exponents int32 [rows, blocks, 1])."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)
    amax = x.abs().amax(-1, keepdim=True)
    bits = amax.view(torch.int32)
    lo, hi = LIMITS[dtype]
    e = ((bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000).int()).clamp(lo, hi)
    bad = ~torch.isfinite(amax)
    step = ((254 - e) << 23).view(torch.float32)
    codes = torch.where(bad, torch.zeros_like(x), torch.round(x * step).clamp(-127, 127))
    return codes, torch.where(bad, torch.full_like(e, 255), e)


def _values(codes, e, cols):
    """The values that codes and exponents stand for, in fp32."""
    v = codes * (e << 23).view(torch.float32)
    return torch.where(e == 255, torch.full_like(v, math.nan), v).reshape(v.shape[0], -1)[:, :cols]


def _pack(x, dtype):
    """fp32 [rows, cols] -> the checkpoint's bytes."""
    rows, cols = x.shape
    codes, e = _quantize(x, dtype)
    out = torch.zeros(rows, _row_bytes(cols), dtype=torch.uint8, device=x.device)
    c = codes.shape[1] * 32
    out[:, :c] = codes.reshape(rows, c).to(torch.int8).view(torch.uint8)
    out[:, c:c + c // 32] = e[:, :, 0].to(torch.uint8)
    return out


def _unpack(ckpt, cols):
    """The checkpoint's bytes -> the values in fp32."""
    c = -(-cols // 32) * 32
    codes = ckpt[:, :c].view(torch.int8).float().reshape(ckpt.shape[0], -1, 32)
    return _values(codes, ckpt[:, c:c + c // 32].int().unsqueeze(-1), cols)


# ---- inputs -----------------------------------------------------------------------------------------

def _normal(gen, rows, cols, sigma=1.0):
    return torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float32) * sigma


def _activation(gen, rows, cols, sigma=1.0):
    """Normal activations with a few channels far larger than the rest."""
    big = 1.0 + 19.0 * (torch.rand(cols, generator=gen, device="cuda") < 0.004).float()
    return _normal(gen, rows, cols, sigma).mul_(big)


def _strided(x, dtype, pad):
    """A [rows, cols] view of a buffer whose rows are cols + pad apart."""
    out = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=DT[dtype], device=x.device)[:, :x.shape[1]]
    out.copy_(x)
    return out


def _empty(rows, cols, dtype, pad=0):
    return torch.empty(rows, cols + pad, dtype=DT[dtype], device="cuda")[:, :cols]


def _groups(c):
    return 1 if c["group"] <= 0 else -(-c["rows"] // c["group"])


def _norm_weights(c, gen):
    def w(mean):
        return (mean + 0.2 * _normal(gen, 1, c["cols"])[0]).to(DT[c["dtype"]])
    s = {"post_w": w(1.0) if c["post"] != "none" else None, "pre_w": w(1.0) if c["pre"] != "none" else None}
    s["post_b"] = w(0.0) if c["post"] != "none" and c["bias"] else None
    s["pre_b"] = w(0.0) if c["pre"] != "none" and c["bias"] else None
    s["gate"] = (None if c["group"] < 0 else
                 (0.5 + 0.3 * _normal(gen, _groups(c), c["cols"])).to(DT[c["dtype"]]))
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "act_save":
        s["x"] = _strided(_activation(gen, c["rows"], c["cols"]), c["dtype"], c["pad"])
        s["ckpt"] = torch.empty(c["rows"], _row_bytes(c["cols"]), dtype=torch.uint8, device="cuda")
        s["out"] = _empty(c["rows"], c["cols"], c["dtype"])
    elif c["op"] == "act_load":
        x = _activation(gen, c["rows"], c["cols"]).to(DT[c["dtype"]])
        s["ckpt"] = _pack(x.float(), c["dtype"])
        s["out"] = _empty(c["rows"], c["cols"], c["dtype"], c["pad"])
    elif c["op"] == "act_wgrad":
        s["dy"] = _strided(_normal(gen, c["tokens"], c["n"], 0.01), c["dtype"], c["pad"])
        s["ckpt"] = _pack(_activation(gen, c["tokens"], c["k"]).to(DT[c["dtype"]]).float(), c["dtype"])
        s["scale"] = s["shift"] = None
        if c["affine"]:
            s["scale"] = (1.0 + 0.2 * _normal(gen, 1, c["k"])[0]).to(DT[c["dtype"]])
            s["shift"] = (0.2 * _normal(gen, 1, c["k"])[0]).to(DT[c["dtype"]])
        s["dw"] = _empty(c["n"], c["k"], c["grad"])
        s["db"] = torch.empty(c["n"], dtype=DT[c["grad"]], device="cuda") if c["bias"] else None
    elif c["op"] == "norm_forward":
        s["h"] = _strided(_activation(gen, c["rows"], c["cols"], 2.0), c["res"], c["pad"])
        s["y"] = _strided(_activation(gen, c["rows"], c["cols"], 0.7), c["dtype"], c["pad"])
        s.update(_norm_weights(c, gen))
        s["h_out"] = _empty(c["rows"], c["cols"], c["res"], c["pad"])
        s["x"] = _empty(c["rows"], c["cols"], c["dtype"], c["pad"]) if c["pre"] != "none" else None
        s["stats"] = s["ckpt_y"] = s["ckpt_x"] = s["yq"] = s["xq"] = None
        if c["ckpt"]:
            def raw():
                return torch.empty(c["rows"], _row_bytes(c["cols"]), dtype=torch.uint8, device="cuda")
            s["stats"] = torch.empty(c["rows"], 4, device="cuda")
            s["ckpt_y"], s["yq"] = raw(), _empty(c["rows"], c["cols"], c["dtype"])
            if c["pre"] != "none":
                s["ckpt_x"], s["xq"] = raw(), _empty(c["rows"], c["cols"], c["dtype"])
    else:
        h = _activation(gen, c["rows"], c["cols"], 2.0)
        y = _activation(gen, c["rows"], c["cols"], 0.7)
        yh, mu2, r2 = _normalise(y, c["post"])
        xh, mu1, r1 = _normalise(h, c["pre"])
        s["stats"] = torch.cat([mu2, r2, mu1, r1], 1)
        s["ckpt_y"] = _pack(yh, c["dtype"])
        s["ckpt_x"] = _pack(xh, c["dtype"]) if c["pre"] != "none" else None
        s["dh_out"] = _strided(_normal(gen, c["rows"], c["cols"], 0.01), c["res"], c["pad"])
        s["dx"] = (_strided(_normal(gen, c["rows"], c["cols"], 0.02), c["dtype"], c["pad"])
                   if c["pre"] != "none" else None)
        s.update(_norm_weights(c, gen))
        s["dh"] = _empty(c["rows"], c["cols"], c["res"], c["pad"])
        s["dy"] = _empty(c["rows"], c["cols"], c["dtype"], c["pad"])
        for w in ("post_w", "post_b", "pre_w", "pre_b", "gate"):
            s["d" + w] = None if s[w] is None else torch.empty(s[w].shape, dtype=DT[c["grad"]], device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------------------------------

def _normalise(v, kind):
    """(normalised rows, mean [rows, 1], reciprocal deviation [rows, 1]) of fp32 rows."""
    one, zero = torch.ones_like(v[:, :1]), torch.zeros_like(v[:, :1])
    if kind == "none":
        return v, zero, one
    mu = v.mean(1, keepdim=True) if kind == "layer" else zero
    d = v - mu
    r = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * r, mu, r


def _gate_rows(s, c):
    """The gate of each row, fp32 [rows or 1, cols]; 1.0 without a gate."""
    if s["gate"] is None:
        return 1.0
    g = s["gate"].float()
    if g.shape[0] == 1:
        return g
    return g[torch.arange(c["rows"], device="cuda") // c["group"]]


def _affine(v, w, b):
    v = v if w is None else v * w.float()
    return v if b is None else v + b.float()


def _per_group(v, c):
    """Sums over the rows of each group: [groups, cols]."""
    if c["group"] <= 0:
        return v.sum(0, keepdim=True)
    v = torch.nn.functional.pad(v, (0, 0, 0, _groups(c) * c["group"] - c["rows"]))
    return v.reshape(_groups(c), c["group"], -1).sum(1)


def _plain(s):
    c = s["case"]
    if c["op"] == "act_save":
        return _values(*_quantize(s["x"].float(), c["dtype"]), c["cols"]).to(DT[c["dtype"]])
    if c["op"] == "act_load":
        return _unpack(s["ckpt"], c["cols"]).to(DT[c["dtype"]])
    if c["op"] == "act_wgrad":
        dy = s["dy"].float()
        dw, db = dy.t() @ _unpack(s["ckpt"], c["k"]), dy.sum(0)
        if s["scale"] is not None:
            dw = dw * s["scale"].float() + db[:, None] * s["shift"].float()
        return {"dw": dw.to(DT[c["grad"]]), "db": db.to(DT[c["grad"]]) if c["bias"] else None}
    if c["op"] == "norm_forward":
        yh, mu2, r2 = _normalise(s["y"].float(), c["post"])
        h = s["h"].float() + c["alpha"] * (_gate_rows(s, c) * _affine(yh, s["post_w"], s["post_b"]))
        xh, mu1, r1 = _normalise(h, c["pre"])
        out = {"h": h.to(DT[c["res"]]), "x": None, "stats": None, "yq": None, "xq": None}
        if c["pre"] != "none":
            out["x"] = _affine(xh, s["pre_w"], s["pre_b"]).to(DT[c["dtype"]])
        if c["ckpt"]:
            out["stats"] = torch.cat([mu2, r2, mu1, r1], 1)
            out["yq"] = _values(*_quantize(yh, c["dtype"]), c["cols"]).to(DT[c["dtype"]])
            if c["pre"] != "none":
                out["xq"] = _values(*_quantize(xh, c["dtype"]), c["cols"]).to(DT[c["dtype"]])
        return out
    r2, r1 = s["stats"][:, 1:2], s["stats"][:, 3:4]
    d = s["dh_out"].float()
    out = dict.fromkeys(("dh", "dy", "dpost_w", "dpost_b", "dpre_w", "dpre_b", "dgate"))
    if c["pre"] != "none":
        dx, xh = s["dx"].float(), _unpack(s["ckpt_x"], c["cols"])
        g = dx * s["pre_w"].float()
        m = g.mean(1, keepdim=True) if c["pre"] == "layer" else 0.0
        d = d + r1 * (g - m - xh * (g * xh).mean(1, keepdim=True))
        out["dpre_w"] = (dx * xh).sum(0)
        out["dpre_b"] = dx.sum(0) if s["pre_b"] is not None else None
    yh = _unpack(s["ckpt_y"], c["cols"])
    dz = c["alpha"] * (_gate_rows(s, c) * d)
    if s["gate"] is not None:
        out["dgate"] = _per_group(c["alpha"] * (d * _affine(yh, s["post_w"], s["post_b"])), c)
    dy = dz
    if c["post"] != "none":
        out["dpost_w"] = (dz * yh).sum(0)
        out["dpost_b"] = dz.sum(0) if s["post_b"] is not None else None
        g = dz * s["post_w"].float()
        m = g.mean(1, keepdim=True) if c["post"] == "layer" else 0.0
        dy = r2 * (g - m - yh * (g * yh).mean(1, keepdim=True))
    out = {k: None if v is None else v.to(DT[c["grad"]]) for k, v in out.items()}
    out["dh"], out["dy"] = d.to(DT[c["res"]]), dy.to(DT[c["dtype"]])
    return out


# ---- the library's calls ----------------------------------------------------------------------------

def _norm_handle(z, s, c):
    """The description of a block boundary, which a program makes once and keeps."""
    if "norm" not in s:
        s["norm"] = z.norm(CODE[c["dtype"]], c["rows"], c["cols"], res_dtype=CODE[c["res"]],
                           post=NORM[c["post"]], pre=NORM[c["pre"]], eps=EPS, alpha=c["alpha"],
                           group_rows=max(0, c["group"]), post_w=s["post_w"], post_b=s["post_b"],
                           gate=s["gate"], pre_w=s["pre_w"], pre_b=s["pre_b"])
    return s["norm"]


def _call(s):
    import zero_sharded_mixed_02_gb300 as z
    c = s["case"]
    stream = torch.cuda.current_stream().cuda_stream
    if c["op"] == "act_save":
        z.zero_act_save(CODE[c["dtype"]], s["x"], c["rows"], c["cols"], c["cols"] + c["pad"], s["ckpt"], stream)
        z.zero_act_load(CODE[c["dtype"]], s["ckpt"], c["rows"], c["cols"], s["out"], c["cols"], stream)
        return s["out"]
    if c["op"] == "act_load":
        z.zero_act_load(CODE[c["dtype"]], s["ckpt"], c["rows"], c["cols"], s["out"], c["cols"] + c["pad"], stream)
        return s["out"]
    if c["op"] == "act_wgrad":
        if "work" not in s:   # kept by the program from step to step
            s["work"] = torch.zeros(z.zero_act_wgrad_workspace(c["tokens"], c["n"], c["k"]), dtype=torch.uint8,
                                    device="cuda")
        z.zero_act_wgrad(CODE[c["dtype"]], s["dy"], c["tokens"], c["n"], c["n"] + c["pad"], s["ckpt"], c["k"],
                         s["scale"], s["shift"], CODE[c["grad"]], s["dw"], c["k"], s["db"], 0, s["work"], stream)
        return {"dw": s["dw"], "db": s["db"]}
    ld = c["cols"] + c["pad"]
    if c["op"] == "norm_forward":
        z.zero_norm_forward(_norm_handle(z, s, c), s["h"], ld, s["y"], ld, s["h_out"], ld, s["x"], ld,
                            s["ckpt_y"], s["ckpt_x"], s["stats"], stream)
        for ckpt, out in ((s["ckpt_y"], s["yq"]), (s["ckpt_x"], s["xq"])):
            if ckpt is not None:
                z.zero_act_load(CODE[c["dtype"]], ckpt, c["rows"], c["cols"], out, c["cols"], stream)
        return {"h": s["h_out"], "x": s["x"], "stats": s["stats"], "yq": s["yq"], "xq": s["xq"]}
    norm = _norm_handle(z, s, c)
    if "work" not in s:
        s["work"] = torch.empty(z.zero_norm_workspace(norm), dtype=torch.uint8, device="cuda")
    z.zero_norm_backward(norm, s["dh_out"], ld, s["dx"], ld, s["ckpt_y"], s["ckpt_x"], s["stats"], s["dh"], ld,
                         s["dy"], ld, CODE[c["grad"]], s["dpost_w"], s["dpost_b"], s["dgate"], s["dpre_w"],
                         s["dpre_b"], 0, s["work"], stream)
    return {k: s[k] for k in ("dh", "dy", "dpost_w", "dpost_b", "dpre_w", "dpre_b", "dgate")}


def run(state):
    return _call(state) if own else _plain(state)


# ---- work -------------------------------------------------------------------------------------------

def _size(dtype):
    return 4 if dtype == "fp32" else 2


def work(case):
    c = case
    if c["op"] in ("act_save", "act_load"):
        n = c["rows"] * c["cols"]
        once = n * (1 + 1 / 32) + n * _size(c["dtype"])
        return {"bytes": once * (2 if c["op"] == "act_save" else 1), "flops": 2 * n}
    if c["op"] == "act_wgrad":
        t, n, k = c["tokens"], c["n"], c["k"]
        side = (4 * k if c["affine"] else 0) + (n * _size(c["grad"]) if c["bias"] else 0)
        return {"bytes": 2 * t * n + t * k * (1 + 1 / 32) + n * k * _size(c["grad"]) + side,
                "flops": 2 * t * n * k}
    n, d = c["rows"] * c["cols"], c["cols"]
    q, r = n * (1 + 1 / 32), _size(c["res"])
    pre, post = c["pre"] != "none", c["post"] != "none"
    weights = d * ((1 + c["bias"]) * (pre + post) + (0 if c["group"] < 0 else _groups(c)))
    if c["op"] == "norm_forward":
        b = 2 * r * n + 2 * n + (2 * n if pre else 0) + 2 * weights
        if c["ckpt"]:       # written, and read back to the values that are returned
            b += (2 * q + 2 * n) * (1 + pre) + 16 * c["rows"]
        return {"bytes": b, "flops": 12 * n}
    b = 2 * r * n + 2 * n + q + (2 * n + q if pre else 0) + 16 * c["rows"] + weights * (2 + _size(c["grad"]))
    return {"bytes": b, "flops": 24 * n}


# ---- exact values, from the definitions in 64 bits --------------------------------------------------

def _power_of_two(e):
    """2^e in 64 bits from its bits: a power function may be off by an ulp, which would break ties."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantize(v, dtype):
    """64-bit rows -> the 64-bit values that their checkpoint stands for: per 32 columns the smallest power of
    two 2^e with max|v| <= 127 * 2^e (e kept in the type's range), and the nearest multiples of it, ties to
    even, at most 127 of them."""
    rows, cols = v.shape
    lo, hi = LIMITS[dtype]
    blocks = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=v.device)
    blocks[:, :cols] = v
    blocks = blocks.view(rows, -1, 32)
    top = blocks.abs().max(dim=2, keepdim=True).values
    m, p = torch.frexp(top / 127.0)                      # top / 127 = m 2^p, m in [1/2, 1)
    e = torch.where(m == 0.5, p - 1, p)
    e = torch.where(top == 0, torch.full_like(e, lo - 127), e).clamp(lo - 127, hi - 127)
    unit = _power_of_two(e)
    q = torch.clamp(torch.round(blocks / unit), -127, 127) * unit
    q = torch.where(torch.isfinite(top), q, torch.full_like(q, math.nan))
    return q.view(rows, -1)[:, :cols]


def _exact_read(ckpt, cols):
    """The checkpoint's bytes -> 64-bit values."""
    wide = -(-cols // 32) * 32
    raw = ckpt[:, :wide].to(torch.int64)
    raw = torch.where(raw > 127, raw - 256, raw).double()
    e = ckpt[:, wide:wide + wide // 32].to(torch.int64)
    unit = _power_of_two(e - 127)
    unit = torch.where(e == 255, torch.full_like(unit, math.nan), unit)
    return (raw * unit.repeat_interleave(32, dim=1))[:, :cols]


def _exact_stats(v, kind):
    d = v.shape[1]
    if kind == "none":
        return torch.zeros(v.shape[0], dtype=torch.float64, device=v.device), torch.ones(
            v.shape[0], dtype=torch.float64, device=v.device)
    mean = v.sum(1) / d if kind == "layer" else torch.zeros(v.shape[0], dtype=torch.float64, device=v.device)
    second = (v * v).sum(1) / d - mean * mean
    return mean, (second + EPS) ** -0.5


def _or(v, other):
    return other if v is None else v.double()


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "act_save":
        return _exact_quantize(s["x"].double(), c["dtype"])
    if c["op"] == "act_load":
        return _exact_read(s["ckpt"], c["cols"])
    if c["op"] == "act_wgrad":
        x = _exact_read(s["ckpt"], c["k"])
        if c["affine"]:
            x = x * s["scale"].double() + s["shift"].double()
        dy = s["dy"].double()
        return {"dw": torch.einsum("tn,tk->nk", dy, x), "db": dy.sum(0) if c["bias"] else None}
    rows, cols = c["rows"], c["cols"]
    owner = torch.zeros(rows, dtype=torch.int64, device="cuda")
    if c["group"] > 0:
        owner = torch.arange(rows, device="cuda").div(c["group"], rounding_mode="floor")
    gate = torch.ones(1, 1, dtype=torch.float64, device="cuda") if s["gate"] is None else s["gate"].double()[owner]
    w2, b2, w1, b1 = _or(s["post_w"], 1.0), _or(s["post_b"], 0.0), _or(s["pre_w"], 1.0), _or(s["pre_b"], 0.0)
    if c["op"] == "norm_forward":
        y = s["y"].double()
        mu2, r2 = _exact_stats(y, c["post"])
        yh = (y - mu2[:, None]) * r2[:, None]
        h = s["h"].double() + c["alpha"] * gate * (yh * w2 + b2)
        mu1, r1 = _exact_stats(h, c["pre"])
        xh = (h - mu1[:, None]) * r1[:, None]
        pre = c["pre"] != "none"
        return {"h": h, "x": xh * w1 + b1 if pre else None,
                "stats": torch.stack([mu2, r2, mu1, r1], 1) if c["ckpt"] else None,
                "yq": _exact_quantize(yh, c["dtype"]) if c["ckpt"] else None,
                "xq": _exact_quantize(xh, c["dtype"]) if c["ckpt"] and pre else None}
    total = s["dh_out"].double()
    out = {}
    if c["pre"] != "none":
        # through x = w1 xh + b1, xh = (h - mean) r: the projections of the gradient on 1 and on xh go out
        xh, dx = _exact_read(s["ckpt_x"], cols), s["dx"].double()
        up = dx * w1
        back = up - xh * ((up * xh).sum(1, keepdim=True) / cols)
        if c["pre"] == "layer":
            back = back - up.sum(1, keepdim=True) / cols
        total = total + back * s["stats"][:, 3:4].double()
        out["dpre_w"] = torch.einsum("rc,rc->c", dx, xh)
        out["dpre_b"] = dx.sum(0) if s["pre_b"] is not None else None
    yh = _exact_read(s["ckpt_y"], cols)
    through = total * gate * c["alpha"]
    if s["gate"] is not None:
        per_row = total * (yh * w2 + b2) * c["alpha"]
        out["dgate"] = torch.zeros(_groups(c), cols, dtype=torch.float64, device="cuda").index_add_(0, owner, per_row)
    dy = through
    if c["post"] != "none":
        out["dpost_w"] = torch.einsum("rc,rc->c", through, yh)
        out["dpost_b"] = through.sum(0) if s["post_b"] is not None else None
        up = through * w2
        dy = up - yh * ((up * yh).sum(1, keepdim=True) / cols)
        if c["post"] == "layer":
            dy = dy - up.sum(1, keepdim=True) / cols
        dy = dy * s["stats"][:, 1:2].double()
    return {"dh": total, "dy": dy, **out}
