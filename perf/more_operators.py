"""The vocabulary head's losses: cases, inputs, plain forms and exact values.

Operators (the C entry points of include/zero_b200.h, through the Python binding); the logits x w^T are never
kept:

  ce_forward        softmax cross entropy over the vocabulary: loss and log-sum-exp of each row, their sum and number
  ce_backward       its gradients of x and w
  distill_forward   divergence of the softmax at a temperature from a teacher's top logits, with the cross
                    entropy of labels where there are some
  distill_backward  its gradients of x and w

``own`` False computes the plain form (elementary torch operations in 32 bits, rounded once at the end);
``own`` True calls the library.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
CODE = {"fp16": 0, "bf16": 1, "fp32": 2}


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # the last, nearly empty micro-batch against the small model's head: the weights are read once
        {"name": "ce_forward_few", "op": "ce_forward", "dtype": "bf16", "rows": 16, "cols": 768, "vocab": 50257,
         "pad": 0, "ignored": 0.0, "z_loss": 0.0},
        # odd sizes: a ragged batch with padding tokens, rows that no vector load can take
        {"name": "ce_forward_odd", "op": "ce_forward", "dtype": "fp16", "rows": 1999, "cols": 771, "vocab": 32003,
         "pad": 0, "ignored": 0.2, "z_loss": 1e-4},
        # 8 x 1024 tokens through the 8B list's head
        {"name": "ce_forward_large", "op": "ce_forward", "dtype": "bf16", "rows": 8192, "cols": 4096,
         "vocab": 128256, "pad": 0, "ignored": 0.0, "z_loss": 0.0},
        # the smallest: a toy vocabulary, where only latency counts
        {"name": "ce_backward_small", "op": "ce_backward", "dtype": "bf16", "rows": 64, "cols": 256, "vocab": 1000,
         "pad": 0, "ignored": 0.0, "z_loss": 0.0, "weights": False},
        # 8 x 1024 tokens through the 1.5B list's head, a quarter of them prompts without a loss
        {"name": "ce_backward_ordinary", "op": "ce_backward", "dtype": "bf16", "rows": 8192, "cols": 1600,
         "vocab": 50257, "pad": 0, "ignored": 0.25, "z_loss": 0.0, "weights": False},
        # odd sizes, weighted tokens, scaled fp16 gradients, a z-loss
        {"name": "ce_backward_odd", "op": "ce_backward", "dtype": "fp16", "rows": 1023, "cols": 771, "vocab": 32003,
         "pad": 3, "ignored": 0.1, "z_loss": 1e-4, "weights": True},
        # 4 x 1024 tokens through the 8B list's head
        {"name": "ce_backward_large", "op": "ce_backward", "dtype": "bf16", "rows": 4096, "cols": 4096,
         "vocab": 128256, "pad": 0, "ignored": 0.0, "z_loss": 0.0, "weights": False},
        # a few tokens of an online teacher with sixteen logits each, no labels
        {"name": "distill_forward_few", "op": "distill_forward", "dtype": "fp16", "rows": 33, "cols": 768,
         "vocab": 50257, "pad": 0, "top": 16, "top_dtype": "fp16", "temperature": 1.0, "labels": False,
         "ignored": 0.0},
        # 4 x 1024 tokens of a stored teacher's 64 logits, softened, mixed with the labels' loss
        {"name": "distill_forward_ordinary", "op": "distill_forward", "dtype": "bf16", "rows": 4096, "cols": 1600,
         "vocab": 50257, "pad": 0, "top": 64, "top_dtype": "bf16", "temperature": 2.0, "labels": True,
         "ignored": 0.1},
        # odd sizes, few teacher logits, weighted tokens
        {"name": "distill_backward_odd", "op": "distill_backward", "dtype": "fp16", "rows": 777, "cols": 520,
         "vocab": 32003, "pad": 8, "top": 9, "top_dtype": "fp32", "temperature": 1.5, "labels": False,
         "ignored": 0.0, "weights": True},
        # 2 x 1024 tokens through the 8B list's head, softened and mixed with the labels' loss
        {"name": "distill_backward_large", "op": "distill_backward", "dtype": "bf16", "rows": 2048, "cols": 4096,
         "vocab": 128256, "pad": 0, "top": 32, "top_dtype": "bf16", "temperature": 2.0, "labels": True,
         "ignored": 0.1, "weights": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce_forward", "ce_backward", "distill_forward", "distill_backward"])
    cols, vocab = _log_int(rng, 64, 4096), _log_int(rng, 500, 131072)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    if rng.random() < 0.3:
        vocab = max(512, vocab // 128 * 128)
    most = (4096 if "backward" in op else 8192) * 4096 * 128256 // (cols * vocab)
    c = {"op": op, "dtype": rng.choice(["fp16", "bf16", "bf16"]), "rows": _log_int(rng, 1, min(16384, most)),
         "cols": cols, "vocab": vocab, "pad": rng.choice([0, 0, 0, 1, 8, 64]),
         "ignored": rng.choice([0.0, 0.0, 0.1, 0.6])}
    if op.startswith("ce"):
        c["z_loss"] = rng.choice([0.0, 0.0, 1e-4])
    else:
        c.update(top=_log_int(rng, 1, 128), top_dtype=rng.choice(["fp16", "bf16", "fp32"]),
                 temperature=rng.choice([1.0, 1.0, 2.0, 0.7]), labels=rng.random() < 0.5)
        if not c["labels"]:
            c["ignored"] = 0.0
    if "backward" in op:
        c["weights"] = rng.random() < 0.4
    return c


# ---- inputs -----------------------------------------------------------------------------------------

HARD, SOFT = 0.5, 0.5                   # weights of the labels' and the teacher's part, where both are there


def _parts(c):
    """(weight of the labels' part, of the teacher's, z-loss, temperature)."""
    if c["op"].startswith("ce"):
        return 1.0, 0.0, c["z_loss"], 1.0
    return (HARD, SOFT, 0.0, c["temperature"]) if c["labels"] else (0.0, 1.0, 0.0, c["temperature"])


def _strided(x, dtype, pad):
    """A [rows, cols] view of a buffer whose rows are cols + pad apart."""
    out = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=DT[dtype], device=x.device)[:, :x.shape[1]]
    out.copy_(x)
    return out


def _tokens(gen, rows, n, vocab):
    """Token numbers with the frequencies of text: density 1 / number."""
    u = torch.rand(rows, n, generator=gen, device="cuda", dtype=torch.float64)
    return ((vocab + 1.0) ** u).floor().long().sub_(1).clamp_(0, vocab - 1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows, d, vocab, back = c["rows"], c["cols"], c["vocab"], "backward" in c["op"]
    w = torch.randn(vocab, d, generator=gen, device="cuda") * (2.0 / math.sqrt(d))
    labels = _tokens(gen, rows, 1, vocab)[:, 0]
    # a normalised row that leans towards its label, as a model in training gives
    x = torch.randn(rows, d, generator=gen, device="cuda") + w[labels] * (
        4.0 * torch.rand(rows, 1, generator=gen, device="cuda"))
    s = {"case": c, "x": _strided(x, c["dtype"], c["pad"]), "w": _strided(w, c["dtype"], c["pad"])}
    del w, x
    distill = c["op"].startswith("distill")
    s["labels"] = s["index"] = s["logit"] = None
    if not distill or c["labels"]:
        none = torch.rand(rows, generator=gen, device="cuda") < c["ignored"]
        s["labels"] = torch.where(none, torch.full_like(labels, -100), labels).to(torch.int32)
    if distill:
        # a teacher's kept logits, largest first; fewer than `top` where it kept only the likely ones
        index = torch.cat([labels[:, None], _tokens(gen, rows, c["top"] - 1, vocab)], 1).sort(1).values
        twice = torch.zeros_like(index, dtype=torch.bool)
        twice[:, 1:] = index[:, 1:] == index[:, :-1]
        s["index"] = torch.where(twice, torch.full_like(index, -1), index).to(torch.int32).contiguous()
        logit = torch.randn(rows, c["top"], generator=gen, device="cuda") * 2.0 + 12.0
        logit += 3.0 * (index == labels[:, None])
        order = logit.argsort(1, descending=True)
        s["index"] = s["index"].gather(1, order).contiguous()
        s["logit"] = logit.gather(1, order).to(DT[c["top_dtype"]]).contiguous()
    if back:
        s["lse"] = _stats(s)[0]                          # kept from the forward pass
        s["weight"] = (0.5 + torch.rand(rows, generator=gen, device="cuda")) if c["weights"] else None
        counted = rows if s["labels"] is None else (s["labels"] >= 0).sum()
        s["divisor"] = torch.ones(1, device="cuda") * counted
        s["scale"] = 16384.0 if c["dtype"] == "fp16" else 1.0
        s["dx"] = torch.empty(rows, d + c["pad"], dtype=DT[c["dtype"]], device="cuda")[:, :d]
        s["dw"] = torch.empty(vocab, d, dtype=DT[c["dtype"]], device="cuda")
    else:
        s["loss"] = torch.empty(rows, device="cuda")
        s["lse"] = torch.empty((rows, 2) if distill else (rows,), device="cuda")
        s["sums"] = torch.empty(2, device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------------------------------

def _log_sum_exp(v):
    m = v.max(1, keepdim=True).values
    return m[:, 0] + torch.exp(v - m).sum(1).log()


def _counted(s):
    """Rows that take part, as a column of truth values."""
    if s["labels"] is not None:
        return s["labels"] >= 0
    return (s["index"] >= 0).any(1)


def _teacher(s, t):
    """(the entries' probabilities, 0 where there is none; their places)."""
    there = s["index"] >= 0
    v = torch.where(there, s["logit"].float() / t, torch.full_like(s["logit"], -math.inf, dtype=torch.float32))
    e = torch.exp(v - v.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True), s["index"].clamp(min=0).long()


def _stats(s):
    """(log-sum-exps as the forward pass returns them, the logits in fp32)."""
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    keep = _counted(s)
    if c["op"].startswith("ce"):
        return torch.where(keep, _log_sum_exp(z), torch.zeros_like(z[:, 0])), z
    soft = _log_sum_exp(z / c["temperature"])
    hard = _log_sum_exp(z) if c["labels"] else torch.zeros_like(soft)
    return torch.where(keep[:, None], torch.stack([soft, hard], 1), torch.zeros_like(z[:, :2])), z


def _plain_forward(s):
    c = s["case"]
    hard, soft, z_loss, t = _parts(c)
    lse, z = _stats(s)
    keep = _counted(s)
    loss = torch.zeros_like(z[:, 0])
    if s["labels"] is not None:
        top = lse if lse.dim() == 1 else lse[:, 1]
        loss = hard * (top - z.gather(1, s["labels"].clamp(min=0).long()[:, None])[:, 0] + z_loss * top * top)
    if s["index"] is not None:
        q, at = _teacher(s, t)
        log_q = torch.where(q > 0, q, torch.ones_like(q)).log()
        loss = loss + soft * t * t * (q * (log_q - z.gather(1, at) / t + lse[:, :1])).sum(1)
    loss = torch.where(keep, loss, torch.zeros_like(loss))
    return {"loss": loss, "lse": lse, "sums": torch.stack([loss.sum(), keep.sum().float()])}


def _plain_backward(s):
    c = s["case"]
    hard, soft, z_loss, t = _parts(c)
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    g = (s["scale"] / s["divisor"]) * _counted(s).float()
    if s["weight"] is not None:
        g = g * s["weight"]
    d = torch.zeros_like(z)
    if s["labels"] is not None:
        lse = s["lse"] if s["lse"].dim() == 1 else s["lse"][:, 1]
        d += torch.exp(z - lse[:, None]) * (hard * (1.0 + 2.0 * z_loss * lse))[:, None]
        d.scatter_add_(1, s["labels"].clamp(min=0).long()[:, None], torch.full_like(z[:, :1], -hard))
    if s["index"] is not None:
        q, at = _teacher(s, t)
        d += torch.exp(z / t - s["lse"][:, :1]) * (soft * t)
        d.scatter_add_(1, at, q * (-soft * t))
    d *= g[:, None]
    return {"dx": (d @ w).to(DT[c["dtype"]]), "dw": (d.t() @ x).to(DT[c["dtype"]])}


# ---- the library's calls ----------------------------------------------------------------------------

def _call(s):
    import zero_sharded_mixed_02_gb300 as z
    c = s["case"]
    stream = torch.cuda.current_stream().cuda_stream
    if "head" not in s:             # kept by the program from step to step
        hard, soft, z_loss, t = _parts(c)
        s["head"] = z.head(CODE[c["dtype"]], c["rows"], c["cols"], c["vocab"], z_loss=z_loss, hard=hard, soft=soft,
                           temperature=t, top=c.get("top", 0), top_dtype=CODE[c.get("top_dtype", "fp32")])
        s["work"] = torch.empty(z.zero_head_workspace(s["head"]), dtype=torch.uint8, device="cuda")
    head, ld, work = s["head"], c["cols"] + c["pad"], s["work"]
    teacher = (s["index"], s["logit"], c["top"]) if c["op"].startswith("distill") else ()
    if "forward" in c["op"]:
        call = z.zero_distill_forward if teacher else z.zero_ce_forward
        call(head, s["x"], ld, s["w"], ld, *teacher, s["labels"], s["loss"], s["lse"], s["sums"], work, stream)
        return {"loss": s["loss"], "lse": s["lse"], "sums": s["sums"]}
    call = z.zero_distill_backward if teacher else z.zero_ce_backward
    call(head, s["x"], ld, s["w"], ld, *teacher, s["labels"], s["lse"], s["weight"], s["scale"], s["divisor"],
         s["dx"], ld, s["dw"], c["cols"], 0, work, stream)
    return {"dx": s["dx"], "dw": s["dw"]}


def run(state):
    if own:
        return _call(state)
    return _plain_forward(state) if "forward" in state["case"]["op"] else _plain_backward(state)


# ---- work -------------------------------------------------------------------------------------------

def work(case):
    """Rows without a loss need no product; the backward pass needs the logits again."""
    c = case
    rows, d, vocab = c["rows"], c["cols"], c["vocab"]
    product = 2 * round(rows * (1.0 - c["ignored"])) * d * vocab
    side = rows * (4 * (c["op"].startswith("ce") or c["labels"]))
    if c["op"].startswith("distill"):
        side += rows * c["top"] * (4 + (4 if c["top_dtype"] == "fp32" else 2))
    stats = 4 * rows * (2 if c["op"].startswith("distill") else 1)
    once = 2 * d * (rows + vocab)
    if "forward" in c["op"]:
        return {"bytes": once + side + stats + 4 * rows + 8, "flops": product}
    return {"bytes": 2 * once + side + stats + (4 * rows if c["weights"] else 0), "flops": 3 * product}


# ---- exact values, from the definitions in 64 bits --------------------------------------------------

def _softmax64(v):
    v = v - v.amax(dim=1, keepdim=True)
    p = v.exp()
    return p.div_(p.sum(dim=1, keepdim=True))


def exact(case, seed):
    c = case
    rows, d, vocab = c["rows"], c["cols"], c["vocab"]
    products = 3 if "backward" in c["op"] else 1
    if products * 2.0 * rows * d * vocab > 18e12:        # at about 1.2e12 a second in 64 bits
        return None
    s = prepare(case, seed)
    hard, soft, z_loss, t = _parts(c)
    x, w = s["x"].double(), s["w"].double()
    z = torch.einsum("rd,vd->rv", x, w)
    labels = None if s["labels"] is None else s["labels"].long()
    counts = torch.ones(rows, dtype=torch.bool, device="cuda") if labels is None else labels >= 0
    entries = []                                         # (row, column, teacher's probability)
    if s["index"] is not None:
        here = s["index"] >= 0
        v = s["logit"].double() / t
        q = _softmax64(v.masked_fill(~here, -math.inf))
        row, k = here.nonzero(as_tuple=True)
        entries = (row, s["index"][row, k].long(), q[row, k])
    if "forward" in c["op"]:
        lse = torch.logsumexp(z, dim=1)
        out = torch.zeros(rows, dtype=torch.float64, device="cuda")
        if labels is not None:
            own_logit = z[torch.arange(rows, device="cuda"), labels.clamp(min=0)]
            out += hard * ((lse - own_logit) + z_loss * lse.square())
        stats = lse
        if entries:
            lse_t = torch.logsumexp(z / t, dim=1)
            row, col, q = entries
            log_p = z[row, col] / t - lse_t[row]
            out.index_add_(0, row, soft * t * t * (torch.xlogy(q, q) - q * log_p))
            stats = torch.stack([lse_t, lse if labels is not None else torch.zeros_like(lse)], dim=1)
            stats = stats * counts[:, None]
        else:
            stats = stats * counts
        out = out * counts
        return {"loss": out, "lse": stats, "sums": torch.stack([out.sum(), counts.sum().double()])}
    kept = s["lse"].double()
    g = torch.zeros_like(z)
    if labels is not None:
        lse = kept if kept.dim() == 1 else kept[:, 1]
        g += hard * (1.0 + 2.0 * z_loss * lse[:, None]) * (z - lse[:, None]).exp()
        g[torch.arange(rows, device="cuda"), labels.clamp(min=0)] -= hard
    if entries:
        row, col, q = entries
        g += soft * t * (z / t - kept[:, :1]).exp()
        g.index_put_((row, col), -soft * t * q, accumulate=True)
    each = s["scale"] / s["divisor"].double() * counts.double()
    if s["weight"] is not None:
        each = each * s["weight"].double()
    g = g * each[:, None]
    return {"dx": torch.einsum("rv,vd->rd", g, w), "dw": torch.einsum("rv,rd->vd", g, x)}
