"""Gradients of the head's loss at logits of any size: what counts is how far a logit is
from the row's log of the sum of exponentials, and fp32 holds that difference."""
import math

import pytest
import torch

import layer_reference as L
import root_reference as R

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


def _grad(h, w, y, lse, gl):
    n, vocab, d = h.shape[0], *w.shape
    size = zf.zero_head_loss_grad_workspace_bytes(n, vocab, d)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    zf.zero_head_loss_grad(h, w, y, lse, gl, dh, dw, False, ws, size)
    return dh, dw


# A single product makes a logit, so that it is exact.
@pytest.mark.parametrize("size", [3.0, 300.0, 1e4, 1e6, 1e9, 1e15, 1e30])
@pytest.mark.parametrize("n", [6, 300])
def test_gradients_of_logits_of_any_size(n, size):
    """z - lse is rounded once (u of itself; exact where it is small), its multiple of log2 e
    and the constant once each, the exponential is off by 4 u: p within (4 |x| + 8) u of
    itself.  dz: bf16 (2^-8 of itself); the products' sums: L.chain."""
    vocab, d = 1000, 64
    g = torch.Generator().manual_seed(n)
    h = torch.zeros((n, d))
    h[:, 0] = size ** 0.5 * (1 + torch.arange(n) % 7 / 8.0)
    h[::2, 0] *= -1.0
    h[:, 1:] = torch.randn((n, d - 1), generator=g) * 2.0
    h = h.to(BF16)
    w = torch.zeros((vocab, d))
    w[:, 0] = size ** 0.5
    some = torch.arange(vocab) % 3 == 0
    w[some, 1 + torch.arange(vocab)[some] % (d - 1)] = 0.5       # z of one more product
    w = w.to(BF16)
    # where fp32 cannot hold both products' sum, one is enough
    if size > 300.0:
        w[:, 1:] = 0.0
    z = (h.double() @ w.double().t()).float().double()
    assert torch.equal(z, h.double() @ w.double().t()) or size <= 300.0
    lse = torch.logsumexp(z, 1).float()
    y = torch.arange(n) * 3 % vocab
    gl = torch.rand(n, generator=g) + 0.5
    args = h.cuda(), w.cuda(), y.cuda(), lse.cuda(), gl.cuda()
    dh, dw = _grad(*args)
    h, w, y, lse, gl = (a.cpu() for a in args)
    x = h.double() @ w.double().t() - lse.double()[:, None]
    p = torch.exp(x)
    g64 = gl.double()[:, None]
    dz = p.scatter_add(1, y[:, None], torch.full((n, 1), -1.0, dtype=F64)) * g64
    z_off = L.chain(d) * (h.double().abs() @ w.double().abs().t()) if size <= 300.0 else 0.0
    off = (p * (z_off + (4 * x.abs() + 8) * U) + 2 * U * (p + 1.0)) * g64 + 2.0 ** -8 * dz.abs()
    for got, a, a_off, b, what in ((dh, dz, off, w.double(), "grad_hidden"),
                                   (dw, dz.t(), off.t(), h.double(), "grad_table")):
        bound = a_off @ b.abs() + (L.chain(2 * a.shape[1]) + 80 * U) * (a.abs() @ b.abs())
        R.check(got, a @ b, bound, what)


@pytest.mark.parametrize("size", [1e4, 1e6, 1e9])
@pytest.mark.parametrize("n", [3, 200])
def test_a_token_sure_of_its_label_has_no_gradient(n, size):
    """All of the probability at the label, lse the label's logit: nothing is left."""
    vocab, d = 500, 64
    h, w = torch.zeros((n, d), dtype=BF16), torch.zeros((vocab, d), dtype=BF16)
    h[:, 0] = (size ** 0.5 * (1 + torch.arange(n) % 128 / 128.0)).to(BF16)
    y = torch.full((n,), 77)
    w[77, 0] = math.sqrt(size)
    z = h[:, 0].double() * float(w[77, 0])
    lse = z.float()
    assert torch.equal(lse.double(), z)
    dh, dw = _grad(h.cuda(), w.cuda(), y.cuda(), lse.cuda(), torch.ones(n, device="cuda"))
    assert bool((dh == 0.0).all()) and bool((dw == 0.0).all())
