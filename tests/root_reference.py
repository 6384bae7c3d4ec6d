"""Plain 64-bit implementations of the operators around the root unit, with
bounds on what fp32 arithmetic and one rounding at the end may differ by.

u = 2^-24 is half an fp32 ulp.  The bounds are those of the fp32 value; where
it is stored in bf16, what is stored must lie between the roundings of the
two ends (rounding is monotone), which needs no tolerance of its own.
First-order bounds: a sum of n terms over chains of c additions is off by at
most c u sum|terms|; a product or difference of two adds u of itself; an
exponential exp(x) computed in fp32 is off by 4 u plus 3 u |x| of itself (x
is a rounded difference times a rounded constant).
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
F64 = torch.float64


TINY = 2.0 ** -126        # results below the normal numbers may be flushed


def check(got, ref, bound, what):
    """got within bound of ref (bf16: between the roundings of ref +- bound);
    NaN and infinities where ref has them."""
    dtype = got.dtype
    bound = torch.as_tensor(bound, dtype=F64).expand(ref.shape).reshape(-1)
    got, ref = got.detach().cpu().to(F64).reshape(-1), ref.reshape(-1)
    special = ~torch.isfinite(ref)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    if dtype == torch.bfloat16:
        near = (got >= (ref - bound).to(dtype).to(F64)) & (got <= (ref + bound).to(dtype).to(F64))
    else:
        near = (got - ref).abs() <= bound
    ok = torch.where(special, same, near)
    if not bool(ok.all()):
        i = int((~ok).nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ref.numel()} values off; first at "
                             f"{i}: got {got[i]!r}, ref {ref[i]!r}, bound {bound[i]!r}")


# ----------------------------------------------------------- token table ----

def embedding(ids, weight, scale):
    w = weight.cpu().to(F64)
    ids = ids.cpu().reshape(-1).long()
    inside = (ids >= 0) & (ids < w.shape[0])
    y = w[torch.where(inside, ids, 0)] * float(torch.tensor(scale, dtype=torch.float32))
    y[~inside] = 0.0
    return y, 2 * U * y.abs()


def embedding_grad(ids, grad_out, shape, scale, old=None):
    dy = grad_out.cpu().to(F64).reshape(-1, shape[1])
    ids = ids.cpu().reshape(-1).long()
    inside = ((ids >= 0) & (ids < shape[0])).nonzero()[:, 0]
    scale = float(torch.tensor(scale, dtype=torch.float32))
    g, mag, count = (torch.zeros(shape, dtype=F64), torch.zeros(shape, dtype=F64),
                     torch.zeros(shape[0], dtype=F64))
    g.index_add_(0, ids[inside], dy[inside] * scale)
    mag.index_add_(0, ids[inside], dy[inside].abs() * abs(scale))
    count.index_add_(0, ids[inside], torch.ones(len(inside), dtype=F64))
    if old is not None:
        old = old.cpu().to(F64)
        g, mag = g + old, mag + old.abs()
    # any order of the tokens: a chain of at most `count` additions
    return g, (count[:, None] + 3) * U * mag


# ------------------------------------------------------------ layer norm ----

# additions one after another in a row's sum: 32 in a thread, 5 in a warp, 5
# over the warps, and room for the products' roundings
CHAIN = 64


def layer_norm(x, weight, bias, eps):
    x = x.cpu().to(F64)
    d = x.shape[1]
    w = torch.ones(d, dtype=F64) if weight is None else weight.cpu().to(F64)
    b = torch.zeros(d, dtype=F64) if bias is None else bias.cpu().to(F64)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    y = xh * w + b
    d_mean = CHAIN * U * x.abs().mean(1, keepdim=True)
    r_rstd = CHAIN * U + (d_mean * rstd) ** 2
    d_y = w.abs() * (rstd * (d_mean + 2 * U * (x - mean).abs()) + (r_rstd + 4 * U) * xh.abs()) \
        + 2 * U * (y.abs() + b.abs())
    return dict(out=y, mean=mean[:, 0], rstd=rstd[:, 0], d_out=d_y, d_mean=d_mean[:, 0],
                d_rstd=(r_rstd * rstd)[:, 0])


def layer_norm_grad(grad_out, x, weight, mean, rstd, ctas):
    x, dy = x.cpu().to(F64), grad_out.cpu().to(F64)
    n, d = x.shape
    w = torch.ones(d, dtype=F64) if weight is None else weight.cpu().to(F64)
    mu, r = mean.cpu().to(F64)[:, None], rstd.cpu().to(F64)[:, None]
    xh = (x - mu) * r
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    d_x = (CHAIN + 16) * U * r * (g.abs() + g.abs().mean(1, keepdim=True)
                                  + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    # a column: the rows of a warp or block, 8 warps, the CTAs in 16 strands
    chain = -(-n // ctas) + 8 + -(-ctas // 16) + 16 + 4
    return dict(grad_x=dx, d_x=d_x, grad_weight=(dy * xh).sum(0), grad_bias=dy.sum(0),
                d_weight=chain * U * (dy * xh).abs().sum(0), d_bias=chain * U * dy.abs().sum(0))


# ----------------------------------------------------------- distillation ----

def distill(logits, ids, teacher, weights, tau):
    """Loss and gradient with their bounds (of fp32 results)."""
    z, t = logits.cpu().to(F64), teacher.cpu().to(F64)
    ids = ids.cpu().long().reshape(z.shape[0], -1)
    n, vocab = z.shape
    t = t.reshape(ids.shape)
    w = torch.ones(n, dtype=F64) if weights is None else weights.cpu().to(F64)
    inside = (ids >= 0) & (ids < vocab)
    t = torch.where(inside, t / tau, float("-inf"))
    some = (t > float("-inf")).any(1)
    live = some & (w != 0)
    x = z / tau
    top = x.amax(1, keepdim=True)
    logq = torch.log_softmax(x, 1)
    p = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)
    logp = torch.where(p > 0, torch.log(p), 0.0)
    at = torch.where(inside, ids, 0)
    lq = torch.gather(logq, 1, at)
    kl = torch.where(p > 0, p * (logp - lq), 0.0).sum(1)
    loss = torch.where(live, w * tau * tau * kl, 0.0)
    q = torch.exp(logq)
    P = torch.zeros_like(q).scatter_add_(1, at, torch.where(inside, p, 0.0))
    grad = torch.where(live[:, None], (q - P) * (tau * w)[:, None], 0.0)

    # bounds.  A term of the sum of exponentials is off by its exponential and
    # by one more for every time the maximum of its thread grew (at most once
    # a vector of 4, over 128 threads or more) or two sums were joined.
    away = torch.nan_to_num((x - top).abs(), nan=0.0, posinf=0.0)
    joins = vocab / 512 + 32
    r_sum = U * (4 * (q * away).sum(1, keepdim=True) + 8 * joins)
    r_q = U * (4 * away + 8) + r_sum
    r_p = U * (8 * torch.nan_to_num((t - t.amax(1, keepdim=True)).abs(), nan=0.0, posinf=0.0)
               + ids.shape[1] / 16 + 32)
    far = torch.gather(away, 1, at)
    d_kl = (p * (r_p * ((logp - lq).abs() + 1) + U * 8 * (logp.abs() + far + 1))).sum(1) \
        + r_sum[:, 0] + U * (8 + ids.shape[1] / 16) * \
        (p * (logp.abs() + far + (logq.amax(1, keepdim=True)).abs())).sum(1)
    d_loss = w.abs() * tau * tau * torch.nan_to_num(d_kl) + TINY
    r_P = torch.where(inside, r_p, 0.0).amax(1, keepdim=True)
    d_grad = (tau * w.abs())[:, None] * (q * r_q + P * (r_P + 4 * U) + 4 * U * (q + P)) + TINY
    return dict(loss=loss, grad=grad, d_loss=d_loss, d_grad=torch.nan_to_num(d_grad), live=live)
