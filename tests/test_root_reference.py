"""The 64-bit formulas of the operators around the root unit against plain
differences of their forward passes, and the layer norm's and the loss's
against torch's own in 64 bits.  CPU only."""
import pytest
import torch

import root_reference as R


def _differences(f, x, v, h):
    """Central difference of f along v; off by h^2 / 6 of the third derivative."""
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("n,d", [(1, 1), (3, 8), (5, 33)])
def test_layer_norm_gradient_is_the_difference_quotient(n, d):
    g = torch.Generator().manual_seed(n * 100 + d)
    x, dy, v = (torch.randn((n, d), generator=g, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(d, generator=g, dtype=torch.float64) for _ in range(2))
    eps = 0.5      # keeps the third derivative small where a row is constant

    def f(x, w=w, b=b):
        return float((R.layer_norm(x, w, b, eps)["out"] * dy).sum())

    fwd = R.layer_norm(x, w, b, eps)
    ref = R.layer_norm_grad(dy, x, w, fwd["mean"], fwd["rstd"], 1)
    h = 1e-4
    assert abs(_differences(f, x, v, h) - float((ref["grad_x"] * v).sum())) < 1e-5
    vw = torch.randn(d, generator=g, dtype=torch.float64)
    assert abs(_differences(lambda t: f(x, w=t), w, vw, h)
               - float((ref["grad_weight"] * vw).sum())) < 1e-8
    assert abs(_differences(lambda t: f(x, b=t), b, vw, h)
               - float((ref["grad_bias"] * vw).sum())) < 1e-8
    torch.testing.assert_close(fwd["out"], torch.nn.functional.layer_norm(x, (d,), w, b, eps))


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_distillation_gradient_is_the_difference_quotient(tau):
    g = torch.Generator().manual_seed(7)
    n, vocab, top = 6, 19, 5
    z, v = (torch.randn((n, vocab), generator=g, dtype=torch.float64) for _ in range(2))
    ids = torch.randint(0, vocab, (n, top), generator=g)
    ids[1, 3:] = -1                                # a short row
    ids[2, :] = -1                                 # no entry
    ids[3, 1] = ids[3, 0]                          # equal ids
    ids[4, 2] = vocab                              # out of range
    t = torch.randn((n, top), generator=g, dtype=torch.float64)
    t[5, 1] = float("-inf")
    w = torch.rand(n, generator=g, dtype=torch.float64)
    w[0] = 0.0
    ref = R.distill(z, ids, t, w, tau)
    assert float(ref["loss"][0]) == 0.0 and float(ref["loss"][2]) == 0.0
    assert not ref["grad"][0].any() and not ref["grad"][2].any()

    def f(z):
        return float(R.distill(z, ids, t, w, tau)["loss"].sum())

    assert abs(_differences(f, z, v, 1e-4) - float((ref["grad"] * v).sum())) < 1e-6


def test_distillation_loss_is_the_divergence():
    g = torch.Generator().manual_seed(8)
    z = torch.randn((4, 11), generator=g, dtype=torch.float64)
    ids = torch.stack([torch.randperm(11, generator=g) for _ in range(4)])
    t = torch.randn((4, 11), generator=g, dtype=torch.float64)
    full = torch.zeros_like(t).scatter_(1, ids, t)
    kl = torch.nn.functional.kl_div(torch.log_softmax(z / 2, 1), torch.log_softmax(full / 2, 1),
                                    reduction="none", log_target=True).sum(1) * 4
    torch.testing.assert_close(R.distill(z, ids, t, None, 2.0)["loss"], kl)


def test_table_gradient_is_the_transposed_lookup():
    g = torch.Generator().manual_seed(9)
    w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((7, 5), (20, 5)))
    ids = torch.randint(-2, 9, (20,), generator=g)
    y, _ = R.embedding(ids, w, 1.5)
    dw, _ = R.embedding_grad(ids, dy, (7, 5), 1.5)
    assert abs(float((y * dy).sum()) - float((w * dw).sum())) < 1e-12
