"""The head's loss and gradients with a workspace of just what a table that is read in
place needs."""
import pytest
import torch

import layer_reference as L
import root_reference as R

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


@pytest.mark.parametrize("n,vocab,d", [(1, 9000, 1024), (33, 50257, 64), (300, 2048, 768),
                                       (8192, 50257, 64), (130, 70000, 256), (9000, 600, 96)])
def test_within_the_workspace_of_a_table_read_in_place(n, vocab, d):
    g = torch.Generator().manual_seed(n + vocab)
    h = (torch.randn((n, d), generator=g) * (8.0 / d ** 0.5)).to(BF16).cuda()
    w = torch.empty((vocab, d), dtype=BF16, device="cuda")
    w.copy_(torch.randn((1000, d), generator=g).repeat((vocab + 999) // 1000, 1)[:vocab] * 0.25)
    y = torch.randint(0, vocab, (n,), generator=g).cuda()
    size = zf.zero_head_loss_in_place_workspace_bytes(n, vocab, d)
    ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    assert bool((ws[size:] == 0xFF).all())
    (ref, off), (ref_lse, lse_off) = L.head_loss(h, w, y)
    R.check(loss, ref.cpu(), off.cpu(), "loss")
    R.check(lse, ref_lse.cpu(), lse_off.cpu(), "lse")
    size = zf.zero_head_loss_grad_in_place_workspace_bytes(n, vocab, d)
    ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    gl = torch.full((n,), 1.0 / n, device="cuda")
    zf.zero_head_loss_grad(h, w, y, lse, gl, dh, dw, False, ws, size)
    assert bool((ws[size:] == 0xFF).all())
    for got, (want, off, norm), what in zip((dh, dw), L.head_loss_grad(h, w, y, lse, gl),
                                            ("grad_hidden", "grad_table")):
        R.check(got, want.cpu(), off.cpu(), what)
        assert float(torch.linalg.vector_norm(got.to(F64) - want)) <= norm
    # more workspace changes nothing
    more = zf.zero_head_loss_grad_workspace_bytes(n, vocab, d)
    ws = torch.full((more,), 0xFF, dtype=torch.uint8, device="cuda")
    dh2, dw2 = torch.empty_like(h), torch.empty_like(w)
    zf.zero_head_loss_grad(h, w, y, lse, gl, dh2, dw2, False, ws, more)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2)
