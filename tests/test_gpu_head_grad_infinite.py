"""Gradients of the head's loss with rows of the table that no token reaches."""
import pytest
import torch

import layer_reference as L

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


@pytest.mark.parametrize("n", [1, 40, 128, 130, 300, 512])
def test_rows_at_minus_infinity_get_a_gradient_of_zeros(n):
    """Every token has a logit of minus infinity at them, so a probability of 0: 0 times the
    hidden states, whatever stands in a tile beside the tokens.  The others' gradients are what
    they are without such rows.  (The hidden states' gradient is NaN: 0 times infinity.)"""
    g = torch.Generator().manual_seed(n)
    vocab, d = 700, 64
    h, w = torch.randn((n, d), generator=g) * 0.5, torch.randn((vocab, d), generator=g) * 0.25
    h[:, 0] = 1.0
    gone = torch.arange(vocab) % 5 == 0
    w[gone, 0] = float("-inf")
    y = 1 + 5 * (torch.arange(n) % 100)
    h, w, y = h.to(BF16).cuda(), w.to(BF16).cuda(), y.cuda()
    size = max(zf.zero_head_loss_workspace_bytes(n, vocab, d),
               zf.zero_head_loss_grad_workspace_bytes(n, vocab, d))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    dw = torch.full_like(w, 3.0)
    gl = torch.rand(n, generator=g).cuda() + 0.5
    zf.zero_head_loss_grad(h, w, y, lse, gl, None, dw, False, ws, size)
    assert bool((dw[gone.cuda()] == 0.0).all())
    rest = ~gone.cuda()
    at = torch.cumsum(rest, 0) - 1
    _, (want, off, _) = L.head_loss_grad(h, w[rest].contiguous(), at[y], lse, gl)
    got = dw[rest].to(F64)
    assert bool(((got - want).abs() <= off + 2.0 ** -8 * want.abs()).all())
