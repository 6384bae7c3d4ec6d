"""Plain 64-bit implementations of the root-mean-square norm and of rows in 8
bits, with bounds on what fp32 arithmetic and one rounding at the end may
differ by (conventions and `check` of root_reference).

u = 2^-24.  A row's sum of squares goes through at most 32 additions in a
thread, 5 + 5 + 1 between lanes and warps, each term with one rounding: off by
43 u of itself (all terms positive); the mean, eps and the square root's
reciprocal (approximation and one Newton step: 4 u) leave rstd within
(44 + 2) / 2 + 4 < 28 u.  An output is s rstd w: 28 u and three roundings.
"""
from __future__ import annotations

import numpy as np
import torch

from root_reference import F64, U

BLOCK = 128
RSTD = 28 * U


def pack(x):
    """(codes uint8, scales float32) of fp32 rows, by the definition: value by value
    the nearest of the 127 magnitudes that e4m3 has, ties to the even code; NaN is 127."""
    x = np.asarray(x, dtype=np.float32)
    n, d = x.shape
    blocks = (d + BLOCK - 1) // BLOCK
    codes = np.zeros((n, d), dtype=np.uint8)
    scales = np.zeros((n, blocks), dtype=np.float32)
    grid = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                     for e in range(16) for m in range(8)][:127])
    for b in range(blocks):
        part = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        mag = np.where(np.isfinite(part), np.abs(part), 0.0)
        top = mag.max(1)
        scale = np.full(n, 2.0 ** -126)
        while True:                          # the smallest that is enough
            more = top > 448.0 * scale
            if not more.any():
                break
            scale[more] *= 2.0
        q = mag / scale[:, None]
        # no code stands for 2^128
        most = np.where(scale == 2.0 ** 120, 240.0, 448.0)[:, None]
        q = np.minimum(q, most)
        hi = np.clip(np.searchsorted(grid, q), 0, 126)
        lo = np.maximum(hi - 1, 0)
        below, above = q - grid[lo], grid[hi] - q
        k = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
        k = np.where(np.isfinite(part), k, 127)
        sign = (np.signbit(part) & np.isfinite(part)).astype(np.uint8) << 7
        codes[:, b * BLOCK:(b + 1) * BLOCK] = k.astype(np.uint8) | sign
        scales[:, b] = scale
    return codes, scales


def unpack(codes, scales):
    """float64 values of rows in 8 bits (codes uint8, scales float32 arrays)."""
    codes, scales = np.asarray(codes), np.asarray(scales, dtype=np.float64)
    e, m = (codes >> 3) & 15, (codes & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((codes & 127) == 127, np.nan, v)
    v = np.where(codes >> 7 == 1, -v, v)
    return v * np.repeat(scales, BLOCK, axis=1)[:, :codes.shape[1]]


def eight_bound(y, bound):
    """How far a value in 8 bits may be from y (float64 rows) when the fp32 value that was
    rounded is within `bound` of it: half a step of 4 bits (the block's largest value,
    itself off by its bound, sets the scale, so the smallest step may be twice as long)."""
    n, d = y.shape
    out = torch.zeros_like(y)
    for a in range(0, d, BLOCK):
        part, off = y[:, a:a + BLOCK].abs(), bound[:, a:a + BLOCK]
        top = (part + off).amax(1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -117) / 448.0)) + 1e-9)
        scale = torch.maximum(scale, torch.full_like(scale, 2.0 ** -126))
        out[:, a:a + BLOCK] = torch.maximum((part + off) * 2.0 ** -4, scale * 2.0 ** -10) + off
    return out


def rms_norm(total, weight, eps):
    """(out, its bound, rstd, its bound) of fp32 rows `total` (float64 tensor)."""
    x = total
    w = torch.ones(x.shape[1], dtype=F64) if weight is None else weight.cpu().to(F64)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    rstd = 1.0 / torch.sqrt(x.square().mean(1) + eps)
    y = x * rstd[:, None] * w
    return y, (RSTD + 3 * U) * y.abs(), rstd, RSTD * rstd


def rms_norm_grad(grad_out, total, weight, rstd, grad_total):
    """(grad_x, bound), (grad_weight, bound), (out, bound): the rows and rstd as given.
    The row's sum of g xh goes through 32 + 11 additions, g and xh are rounded once each;
    the weight's gradient is a sum over the rows, of at most n additions in a group, 8
    between groups and 160 between CTAs."""
    x, dy, r = total, grad_out.cpu().to(F64), rstd.cpu().to(F64)[:, None]
    n, d = x.shape
    w = torch.ones(d, dtype=F64) if weight is None else weight.cpu().to(F64)
    xh, g = x * r, dy * w
    m = (g * xh).sum(1, keepdim=True) / d
    off = 48 * U * (g * xh).abs().sum(1, keepdim=True) / d
    dx = r * (g - xh * m)
    bound = r * (xh.abs() * off + 4 * U * (g.abs() + (xh * m).abs()))
    if grad_total is not None:
        t = grad_total.cpu().to(F64)
        dx = dx + t
        bound = bound + U * dx.abs()
    dw = (dy * xh).sum(0)
    dw_bound = (n + 168 + 3) * U * (dy * xh).abs().sum(0)
    return (dx, bound), (dw, dw_bound), (xh * w, 3 * U * (xh * w).abs())


# ------------------------------------------------- cross entropy of the head ----
#
# A product of d bf16 pairs is summed on the tensor cores 16 pairs at a time; each step
# adds them to the running sum in fp32, off by at most 2 units of 2^-23 of the magnitudes
# added so far: (d / 16 + 1) 2^-22 sum|h w| in all (`chain`).  Exponentials are off by 4 u
# and 3 u |x| of themselves, their sums go through at most 256 + 32 additions, so lse and
# loss are off by the logits' bound (the loss twice) and 300 u, and by their own rounding.
# dz is rounded to bf16 (2^-8 of itself).

def chain(n):
    return (n / 16 + 1) * 2.0 ** -22


def head_logits(hidden, table):
    """(z, bound) in 64 bits, where the tensors are."""
    h, w = hidden.to(F64), table.to(F64)
    return h @ w.t(), chain(h.shape[1]) * (h.abs() @ w.abs().t())


def head_loss(hidden, table, labels):
    """(loss, bound), (lse, bound); 0 where the label is outside the vocabulary."""
    vocab = table.shape[0]
    live = (labels >= 0) & (labels < vocab)
    z, off = head_logits(hidden[live], table)
    lse = torch.logsumexp(z, 1)
    at = labels[live].long()[:, None]
    loss = lse - z.gather(1, at)[:, 0]
    off = off.amax(1)
    out = torch.zeros((4, labels.numel()), dtype=F64, device=hidden.device)
    out[0, live], out[1, live] = loss, 2 * off + 300 * U + 2 * U * loss.abs()
    out[2, live], out[3, live] = lse, off + 300 * U + 2 * U * lse.abs()
    return (out[0], out[1]), (out[2], out[3])


def head_loss_grad(hidden, table, labels, lse, grad_loss, old=None):
    """(grad_hidden, bound, bound of its 2-norm), the same for the table (added to old)."""
    vocab = table.shape[0]
    live = (labels >= 0) & (labels < vocab) & (grad_loss != 0)
    h, w, g = hidden[live].to(F64), table.to(F64), grad_loss[live].to(F64)[:, None]
    z, off = head_logits(hidden[live], table)
    x = z - lse[live].to(F64)[:, None]
    p = torch.exp(x)
    p_off = p * (off + 6 * U + 3 * U * (x.abs() + lse[live].to(F64).abs()[:, None]))
    dz = p.scatter_add(1, labels[live].long()[:, None], torch.full_like(p[:, :1], -1.0)) * g
    # to bf16 (below the normal numbers: flushed or rounded by 2^-134)
    dz_off = (p_off + 2 * U * (p + dz.abs())) * g.abs() + 2.0 ** -8 * dz.abs() + 2.0 ** -126
    dh, dw = dz @ w, dz.t() @ h
    n = h.shape[0]
    dh_off = dz_off @ w.abs() + (chain(vocab) + 80 * U) * (dz.abs() @ w.abs())
    dw_off = dz_off.t() @ h.abs() + (chain(n) + 2 * U) * (dz.abs().t() @ h.abs())
    norm = lambda t: float(torch.linalg.vector_norm(t))     # noqa: E731
    # ||E W||_F <= ||E||_F ||W||_2, and the result's own rounding
    wide = lambda t: float(torch.linalg.matrix_norm(t, 2)) if t.numel() else 0.0   # noqa: E731
    dh_norm = norm(dz_off) * wide(w) + norm(dh) * 2.0 ** -8
    dw_norm = norm(dz_off) * wide(h) + norm(dw) * 2.0 ** -8
    full = torch.zeros(hidden.shape, dtype=F64, device=hidden.device)
    full_off = torch.zeros_like(full)
    full[live], full_off[live] = dh, dh_off
    if old is not None:
        dw = dw + old.to(F64)
        dw_off = dw_off + 2 * U * dw.abs()
        dw_norm += norm(dw) * 2.0 ** -8
    return (full, full_off, dh_norm), (dw, dw_off, dw_norm)
