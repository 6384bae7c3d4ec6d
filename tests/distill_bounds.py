"""The distillation loss and its gradient in 64 bits, on the inputs' device,
with bounds that are finite wherever the value is.

u = 2^-24.  An exponential of a difference x from the largest of its row,
computed in fp32, is off by 4 u (of the function) plus 4 u |x| (the constant,
the difference and the product are each rounded once) of itself.  A sum of
exponentials adds u a step of its chain and 4 u for every move to a larger
maximum; both are counted as one step of 8 u a 512 elements and 32 at the end.
An error of p_k counts with p_k: an entry of weight zero adds none, however far
from the others its logit lies.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126        # exponentials below the normal numbers may be flushed
F64 = torch.float64


def distill(logits, ids, teacher, weights, tau):
    z = logits.to(F64)
    n, vocab = z.shape
    ids = ids.reshape(n, -1).long()
    top = ids.shape[1]
    w = torch.ones(n, dtype=F64, device=z.device) if weights is None else weights.to(F64)
    inside = (ids >= 0) & (ids < vocab)
    at = torch.where(inside, ids, 0)
    t = torch.where(inside, teacher.reshape(n, top).to(F64) / tau, float("-inf"))
    t_top = t.amax(1, keepdim=True)
    live = (t_top[:, 0] > float("-inf")) & (w != 0)
    t_far = torch.where(t > float("-inf"), t_top - t, 0.0)
    p = torch.where(t > float("-inf"), torch.exp(-t_far), 0.0)
    p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    has = p > 0
    logp = torch.where(has, torch.log(torch.where(has, p, 1.0)), 0.0)

    x = z / tau
    x = x - x.amax(1, keepdim=True)               # differences: 0 and below
    log_sum = torch.log(torch.exp(x).sum(1, keepdim=True))
    q = torch.exp(x - log_sum)
    far = torch.where(torch.isfinite(x), -x, 0.0)
    lq = torch.gather(x, 1, at) - log_sum
    kl = torch.where(has, p * (logp - lq), 0.0)
    loss = torch.where(live, w * tau * tau * kl.sum(1), 0.0)

    def by_id(values):
        return torch.zeros_like(q).scatter_add_(1, at, torch.where(inside, values, 0.0))

    P = by_id(p)
    scale = (tau * w.abs())[:, None]
    grad = torch.where(live[:, None], (q - P) * (tau * w)[:, None], 0.0)

    r_sum = U * (4 * (q * far).sum(1, keepdim=True) + 8 * (vocab / 512 + 32))
    r_q = U * (4 * far + 8) + r_sum
    r_p = U * (4 * t_far + 4 * (p * t_far).sum(1, keepdim=True) + top / 16 + 40)
    size = torch.where(has, logp.abs() + lq.abs(), 0.0)
    d_kl = torch.where(has, p * (r_p * (size + 1) + 8 * U * (size + t_far + 1)), 0.0).sum(1) \
        + r_sum[:, 0] + U * (8 + top / 16) * (p * size).sum(1)
    d_loss = torch.where(live, w.abs() * tau * tau * d_kl, 0.0) + 8 * TINY
    d_grad = torch.where(
        live[:, None],
        scale * (q * r_q + by_id(p * r_p) + U * (4 + by_id(torch.ones_like(p))) * (q + P)), 0.0) \
        + 8 * TINY * (1 + scale)
    assert bool((torch.isfinite(d_loss) | ~torch.isfinite(loss)).all())
    assert bool((torch.isfinite(d_grad) | ~torch.isfinite(grad)).all())
    return dict(loss=loss, grad=grad, d_loss=d_loss, d_grad=d_grad, live=live)


def check(got, ref, bound, what):
    """got within bound of ref; in bf16, between the roundings of ref +- bound."""
    got64 = got.to(F64)
    if got.dtype == torch.bfloat16:
        ok = (got64 >= (ref - bound).to(got.dtype).to(F64)) & \
             (got64 <= (ref + bound).to(got.dtype).to(F64))
    else:
        ok = (got64 - ref).abs() <= bound
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        i = tuple(int(k) for k in bad[0])
        raise AssertionError(
            f"{what}: {len(bad)} of {ref.numel()} values off, rows {sorted(set(bad[:, 0].tolist()))[:12]}; "
            f"first at {i}: got {float(got[i])!r}, ref {float(ref[i])!r}, bound {float(bound[i])!r}")
