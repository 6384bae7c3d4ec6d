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
