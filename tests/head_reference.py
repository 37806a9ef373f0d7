"""The losses over the vocabulary and their gradients in 64 bits (torch), from the definitions in
include/zero_b200.h, with bounds of what the library's roundings can change.

Bounds, per row i: with A_i = max_j sum_k |x_ik w_jk|, a logit of `cols` columns is off by at most
steps * 2^-22 * A_i, a step being the tensor cores' 16 columns: an accumulator and the step's products
are each cut off at no more than one unit in the last place of the larger (2^-23 of it, twice), and a
loss adds at most 48 such steps at a time, then runs of them rounded in fp32 (below one step each).
exp2's argument and result, sums of exponentials and logarithms add a few units in the last place of
fp32: 2^-19 (1 + max|z|)."""
import math

import torch

EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step


class Case:
    """Inputs of a head; values as the library gets them."""

    def __init__(self, x, w, labels=None, index=None, logit=None, z_loss=0.0, hard=1.0, soft=1.0, temperature=1.0):
        self.x, self.w, self.labels, self.index, self.logit = x, w, labels, index, logit
        self.distill = index is not None
        self.z_loss, self.temperature = z_loss, temperature if self.distill else 1.0
        self.hard, self.soft = (hard, soft) if self.distill else (1.0, 0.0)

    def counted(self):
        if self.labels is not None:
            return self.labels >= 0
        return ((self.index >= 0) & (self.logit.double() != -math.inf)).any(1)

    def bad(self):
        """Counted rows with a label or entry past the vocabulary."""
        vocab, b = self.w.shape[0], torch.zeros(self.x.shape[0], dtype=torch.bool, device=self.x.device)
        if self.labels is not None:
            b |= self.labels >= vocab
        if self.distill:
            b |= ((self.index >= vocab) & (self.logit.double() != -math.inf)).any(1)
        return b & self.counted()

    def logits(self):
        """z of the counted rows, 0 elsewhere."""
        x = torch.where(self.counted()[:, None], self.x.double(), torch.zeros((), dtype=torch.float64, device=self.x.device))
        return x, x @ self.w.double().T

    def teacher(self):
        """(q, its places, rows that have any)."""
        there = (self.index >= 0) & (self.logit.double() != -math.inf)
        t = torch.where(there, self.logit.double() / self.temperature, torch.full_like(self.logit.double(), -math.inf))
        has = there.any(1)
        t = t - torch.where(has, t.max(1).values, torch.zeros_like(t[:, 0]))[:, None]
        e = torch.where(there, t.exp(), torch.zeros_like(t))
        q = e / torch.where(has, e.sum(1), torch.ones_like(e[:, 0]))[:, None]
        return q, self.index.clamp(0, self.w.shape[0] - 1).long(), has

    def forward(self):
        """(loss, lse as the library lays it out, sums, bound of loss and lse per row)."""
        keep, (x, z), t = self.counted(), self.logits(), self.temperature
        lse = torch.logsumexp(z, 1)
        soft_lse = torch.logsumexp(z / t, 1)
        loss = torch.zeros_like(lse)
        if self.labels is not None:
            y = self.labels.clamp(0, z.shape[1] - 1).long()
            loss = self.hard * (lse - z.gather(1, y[:, None])[:, 0] + self.z_loss * lse * lse)
        off = self.logit_error(x, z, run=48)
        scale = abs(self.hard) * (2 + 2 * abs(self.z_loss) * lse.abs())
        if self.distill:
            q, at, has = self.teacher()
            kl = torch.where(q > 0, q * (q.clamp(min=1e-300).log() - z.gather(1, at) / t + soft_lse[:, None]), torch.zeros_like(q))
            loss = loss + self.soft * t * t * kl.sum(1)
            scale = scale + abs(self.soft) * t * t * 4 / min(t, 1.0)
        nan = torch.full_like(loss, math.nan)
        zero = torch.zeros_like(loss)
        fix = lambda v: torch.where(keep, torch.where(self.bad(), nan, v), zero)  # noqa: E731
        loss = fix(loss)
        out = fix(lse)
        if self.distill:
            out = torch.stack([fix(soft_lse), fix(lse) if self.labels is not None else zero], 1)
        # sums of the teacher's entries and of the loss's parts: 2^-18 of what they add
        size = (scale * (1 + lse.abs() + soft_lse.abs() + z.abs().max(1).values))
        return loss, out, torch.stack([loss.sum(), keep.sum().double()]), scale * off + size * 2.0 ** -18

    def lse_bound(self):
        """A log-sum-exp moves by no more than its logits do (by the softmax's mean of it), at a temperature T by 1/T of
        that; its sums, exponentials and logarithm add 2^-18 of 1 and itself."""
        x, z = self.logits()
        t = self.temperature
        off = self.logit_error(x, z, run=48)
        soft = off / t + 2.0 ** -18 * (1 + torch.logsumexp(z / t, 1).abs())
        hard = off + 2.0 ** -18 * (1 + torch.logsumexp(z, 1).abs())
        return torch.stack([soft, hard], 1) if self.distill else hard

    def logit_error(self, x, z, run):
        top = (x.abs() @ self.w.double().abs().T).max(1).values
        steps = min(run, -(-x.shape[1] // 16)) + x.shape[1] / 768
        return steps * 2.0 ** -22 * top + 2.0 ** -19 * (1 + z.abs().max(1).values)

    def gradient(self, lse, row_grad=None, scale=1.0, divisor=None):
        """(dx, dw, bounds of both before the results' own rounding), from the lse that is kept."""
        keep, (x, z), t = self.counted(), self.logits(), self.temperature
        g = torch.full_like(z[:, 0], scale)
        if row_grad is not None:
            g = g * row_grad.double()
        if divisor is not None:
            g = torch.zeros_like(g) if float(divisor) == 0 else g / float(divisor)
        g = torch.where(keep, g, torch.zeros_like(g))
        kept = lse.double()
        dz, size = torch.zeros_like(z), torch.zeros_like(z)
        if self.labels is not None:
            l = kept[:, 1] if self.distill else kept
            p = (z - l[:, None]).exp() * (self.hard * (1 + 2 * self.z_loss * l))[:, None]
            y = self.labels.clamp(0, z.shape[1] - 1).long()[:, None]
            dz, size = dz + p, size + p.abs()
            dz = dz.scatter_add(1, y, torch.full_like(z[:, :1], -self.hard))
            size = size.scatter_add(1, y, torch.full_like(z[:, :1], abs(self.hard)))
        if self.distill:
            q, at, has = self.teacher()
            p = self.soft * t * (z / t - kept[:, :1]).exp() * has[:, None]
            dz, size = dz + p, size + p.abs()
            dz = dz.scatter_add(1, at, -self.soft * t * q)
            size = size.scatter_add(1, at, abs(self.soft) * t * q)
        live = g != 0
        zero = torch.zeros_like(z)
        dz = torch.where(live[:, None], dz * g[:, None], zero)
        size = torch.where(live[:, None], size * g.abs()[:, None], zero)
        dz = torch.where((self.bad() & live)[:, None], torch.full_like(z, math.nan), dz)
        x = torch.where(live[:, None], x, torch.zeros_like(x))
        w, half = self.w.double(), EPS[self.x.dtype]
        # dz: its own rounding; what the logits' errors change; and for fp16 half its smallest number,
        # 2^-25, over the 2^14 and the power of two (at most the sum of the row's sizes) that it is kept at
        off = self.logit_error(x, z, run=1 << 30) * 2 / min(t, 1.0)
        each = half * dz.abs() + size * off[:, None]
        if self.x.dtype == torch.float16:
            each = each + 2.0 ** -37 * size.sum(1, keepdim=True)
        # probabilities below fp32's normal numbers (2^-126) are 0
        each = each + 2.0 ** -126 * size.sum(1, keepdim=True)
        steps_x, steps_w = -(-z.shape[1] // 16), -(-z.shape[0] // 16)
        dx, dw = dz @ w, dz.T @ x
        a, b = dz.abs() @ w.abs(), dz.abs().T @ x.abs()
        # x of a row of small scale is multiplied by its power of two over the largest row's: exact, but
        # for fp16's smallest number (half of it, 2^-25, times what it is multiplied with)
        low = 0.0
        if self.x.dtype == torch.float16:
            total = size.sum(1, keepdim=True)
            low = 2.0 ** -24 * float(total.max()) * (size / total.clamp(min=1e-300)).sum(0)[:, None]
        bound_x = each @ w.abs() + (min(steps_x, 4096) * 2.0 ** -22 + 2.0 ** -20) * a
        bound_w = each.T @ x.abs() + (steps_w * 2.0 ** -22 + 2.0 ** -20) * b + low
        return dx, dw, bound_x, bound_w


def close(got, want, bound, what=""):
    """got (a 16-bit or fp32 result) is want to its own rounding and the bound; NaN where want is."""
    g = got.double()
    assert bool((torch.isnan(want) == torch.isnan(g)).all()), f"{what}: NaN in other places"
    half = EPS[got.dtype]
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134 if got.dtype == torch.bfloat16 else 2.0 ** -149
    lim = bound * (1 + 2 * half) + half * want.abs() + tiny
    bad = torch.where(torch.isnan(want), torch.zeros_like(g), (g - want).abs()) > lim
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, largest "
                                 f"{float(((g - want).abs() / lim)[bad].max())} of the bound")
