"""Trains a small stack of residual feed-forward blocks with 8-bit activation checkpoints.

Every block is x = norm(h), a = tanh(x W1' + b1), y = a W2' + b2, h += gate * norm(y).  The
forward pass keeps, per block, the normalised rows around it and a in 8 bits, and four numbers
a row; h itself is overwritten in place.  The backward pass reads the checkpoints where they
are used, writes every gradient to its place in the rank's row of flat gradients, and one
zero_step takes all ranks' rows to the new weights.  The products with the weights themselves
(forward, and the gradients of activations) are plain torch ones.

    python examples/residual_blocks.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_02_gb300 as z  # noqa: E402

HALF, FP16 = torch.float16, z.ZERO_FP16


class ResidualBlocks:
    """`blocks` blocks of width d and inner width f; `ranks` batches of `tokens` rows a step."""

    def __init__(self, d, f, blocks, tokens, ranks=2, seed=0, **hparams):
        self.d, self.f, self.blocks, self.tokens, self.ranks = d, f, blocks, tokens, ranks
        # boundary i stands before block i; the last one feeds the loss
        named = []
        for i in range(blocks + 1):
            if i:
                named += [(f"post_w{i}", (d,)), (f"gate{i}", (d,))]
            named += [(f"pre_w{i}", (d,)), (f"pre_b{i}", (d,))]
            if i < blocks:
                named += [(f"w1_{i}", (f, d)), (f"b1_{i}", (f,)), (f"w2_{i}", (d, f)), (f"b2_{i}", (d,))]
        self.place, psi = {}, 0
        for name, shape in named:
            self.place[name] = (psi, shape)
            psi += math.prod(shape)
        hp = z.hparams(**{**dict(lr=3e-3, loss_scale=65536.0, dynamic_scale=1, clip_norm=1.0), **hparams})
        self.plan = z.zero_plan_create(psi, ranks, 2, FP16, [s for _, s in named], hp)
        _, padded, _, step_bytes = z.zero_plan_layout(self.plan)
        new = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
        self.grads = new(ranks, padded, dtype=HALF)
        self.master, self.m, self.v = new(padded), new(padded), new(padded)
        self.params = new(padded, dtype=HALF)
        self.step_work = new(max(step_bytes, 16), dtype=torch.uint8)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for name, (at, shape) in self.place.items():
            w = self.master[at:at + math.prod(shape)].view(shape)
            if len(shape) == 2:
                w.normal_(generator=gen).mul_(shape[1] ** -0.5)
            elif name.startswith(("pre_w", "post_w")):
                w.fill_(1.0)
            elif name.startswith("gate"):
                w.fill_(0.5)
        self.params.copy_(self.master)
        # what a batch keeps for its backward pass
        keep = lambda cols: new(tokens, z.zero_act_row_bytes(cols), dtype=torch.uint8)  # noqa: E731
        self.ckpt_x = [keep(d) for _ in range(blocks + 1)]
        self.ckpt_y = [None] + [keep(d) for _ in range(blocks)]
        self.ckpt_a = [keep(f) for _ in range(blocks)]
        self.stats = [new(tokens, 4) for _ in range(blocks + 1)]
        self.norms = [z.norm(FP16, tokens, d, res_dtype=z.ZERO_FP32, pre=z.ZERO_NORM_LAYER, pre_w=self.weight(f"pre_w{i}"),
                             pre_b=self.weight(f"pre_b{i}"),
                             **(dict(post=z.ZERO_NORM_RMS, post_w=self.weight(f"post_w{i}"), gate=self.weight(f"gate{i}"))
                                if i else {})) for i in range(blocks + 1)]
        self.norm_work = new(max(z.zero_norm_workspace(n) for n in self.norms), dtype=torch.uint8)
        self.wgrad_work = new(max(z.zero_act_wgrad_workspace(tokens, f, d), z.zero_act_wgrad_workspace(tokens, d, f)),
                              dtype=torch.uint8)

    def weight(self, name):
        at, shape = self.place[name]
        return self.params[at:at + math.prod(shape)].view(shape)

    def grad(self, rank, name):
        at, shape = self.place[name]
        return self.grads[rank, at:at + math.prod(shape)].view(shape)

    def kept_bytes(self):
        """Bytes that a batch's forward pass leaves for its backward pass."""
        return sum(t.numel() * t.element_size() for t in self.ckpt_x + self.ckpt_y[1:] + self.ckpt_a + self.stats)

    def forward(self, h):
        """The last boundary's rows from h [tokens][d] fp32, which is overwritten."""
        d, f, t, s = self.d, self.f, self.tokens, torch.cuda.current_stream().cuda_stream
        x, y = torch.empty(t, d, dtype=HALF, device="cuda"), None
        for i, norm in enumerate(self.norms):
            z.zero_norm_forward(norm, h, d, y, d, h, d, x, d, self.ckpt_y[i], self.ckpt_x[i], self.stats[i], s)
            if i < self.blocks:
                a = torch.addmm(self.weight(f"b1_{i}"), x, self.weight(f"w1_{i}").T).tanh_()
                z.zero_act_save(FP16, a, t, f, f, self.ckpt_a[i], s)
                y = torch.addmm(self.weight(f"b2_{i}"), a, self.weight(f"w2_{i}").T)
        return x

    def backward(self, dx, rank):
        """All weights' gradients, into the rank's row, from the last boundary's; returns h's."""
        d, f, t, s = self.d, self.f, self.tokens, torch.cuda.current_stream().cuda_stream
        dh = torch.empty(t, d, device="cuda")
        dy = torch.empty(t, d, dtype=HALF, device="cuda")
        a = torch.empty(t, f, dtype=HALF, device="cuda")
        for i in range(self.blocks, -1, -1):
            later = dh if i < self.blocks else None         # nothing uses h after the last boundary
            g = lambda name: self.grad(rank, name)  # noqa: E731
            z.zero_norm_backward(self.norms[i], later, d, dx, d, self.ckpt_y[i], self.ckpt_x[i], self.stats[i], dh, d,
                                 dy if i else None, d, FP16, dpost_w=g(f"post_w{i}") if i else None,
                                 dgate=g(f"gate{i}") if i else None, dpre_w=g(f"pre_w{i}"), dpre_b=g(f"pre_b{i}"),
                                 work=self.norm_work, stream=s)
            if i == 0:
                return dh
            b = i - 1                                       # the block before this boundary
            z.zero_act_wgrad(FP16, dy, t, d, d, self.ckpt_a[b], f, None, None, FP16, g(f"w2_{b}"), f, g(f"b2_{b}"), 0,
                             self.wgrad_work, s)
            z.zero_act_load(FP16, self.ckpt_a[b], t, f, a, f, s)
            du = (dy @ self.weight(f"w2_{b}")).mul_(1 - a * a)
            # the checkpoint is the normalised row: the norm's weight and bias make it the layer's input
            z.zero_act_wgrad(FP16, du, t, f, f, self.ckpt_x[b], d, self.weight(f"pre_w{b}"), self.weight(f"pre_b{b}"), FP16,
                             g(f"w1_{b}"), d, g(f"b1_{b}"), 0, self.wgrad_work, s)
            dx = du @ self.weight(f"w1_{b}")

    def step(self, batches, targets):
        """One optimizer step from a batch and its targets a rank; (mean loss, the step's result)."""
        scale = z.zero_step_result(self.plan)["loss_scale"]
        loss = 0.0
        for rank in range(self.ranks):
            off = self.forward(batches[rank].clone()).float() - targets[rank]
            loss += off.square().mean() / (2 * self.ranks)
            self.backward((off * (scale / off.numel())).to(HALF), rank)
        z.zero_step(self.plan, self.grads, self.master, self.m, self.v, self.params, self.step_work,
                    torch.cuda.current_stream().cuda_stream)
        return float(loss), z.zero_step_result(self.plan)

    def close(self):
        z.zero_plan_destroy(self.plan)


def train(steps=60, d=256, f=1024, blocks=3, tokens=1000, ranks=2, seed=0):
    """Fits the stack to a fixed random map; the losses."""
    net = ResidualBlocks(d, f, blocks, tokens, ranks, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn(d, d, generator=gen, device="cuda") * (2.0 / math.sqrt(d))
    losses = []
    for _ in range(steps):
        batches = [torch.randn(tokens, d, generator=gen, device="cuda") for _ in range(ranks)]
        loss, _ = net.step(batches, [torch.tanh(b @ teacher) for b in batches])
        losses.append(loss)
    kept = net.kept_bytes()
    net.close()
    return losses, kept


if __name__ == "__main__":
    losses, kept = train()
    for i in range(0, len(losses), 10):
        print(f"step {i:3d}  loss {losses[i]:.4f}")
    print(f"last loss {losses[-1]:.4f}; kept for the backward pass: {kept / 2**20:.1f} MiB a batch")
