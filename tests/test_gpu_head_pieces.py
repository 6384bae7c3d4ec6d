"""The head's loss and gradients in pieces of the vocabulary: a table off the 16-byte grid
whose copy is more than a piece holds, labels in every piece and at their borders, and
gradients that are added to, on and off the grid."""
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


def _at(shape, offset):
    n = shape[0] * shape[1]
    return torch.empty(offset + n, dtype=BF16, device="cuda")[offset:].view(shape)


def _inputs(n, vocab, d, offset):
    g = torch.Generator(device="cuda").manual_seed(n + vocab)
    h = (torch.randn((n, d), generator=g, device="cuda") * (8.0 / d ** 0.5)).to(BF16)
    w = _at((vocab, d), offset)
    for a in range(0, vocab, 1 << 14):
        part = w[a:a + (1 << 14)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * 0.25)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    y[torch.rand(n, generator=g, device="cuda") < 0.1] = -100
    return g, h, w, y


@pytest.mark.parametrize("n,vocab,d,edges", [
    (40, 75000, 3600, (37631, 37632)), (300, 160000, 3600, (53503, 53504, 107007, 107008)),
    (300, 75000, 4104, (25087, 25088, 50175, 50176))])
def test_loss_in_pieces(n, vocab, d, edges):
    """Copies of 547 MB (two pieces), 1.2 GB and 620 MB; `edges` are about where pieces end."""
    _, h, w, y = _inputs(n, vocab, d, 5)
    y[:4] = torch.tensor([0, vocab - 1, vocab // 2, vocab // 3], device="cuda")
    y[4:4 + len(edges)] = torch.tensor(edges, device="cuda")
    y[9], y[10] = vocab, -1
    size = zf.zero_head_loss_workspace_bytes(n, vocab, d)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.full((2, n), 7.0, device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    assert bool((ws[size:] == 0xFF).all())
    (want, off), (want_lse, lse_off) = L.head_loss(h, w, y)
    R.check(loss, want.cpu(), off.cpu(), "loss")
    R.check(lse, want_lse.cpu(), lse_off.cpu(), "lse")
    again = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, again[0], again[1], ws, size)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("grad_offset", [0, 5, 8])
@pytest.mark.parametrize("n,vocab,d,offset", [(8192, 50257, 64, 0), (8000, 40000, 100, 3),
                                              (50, 80000, 3600, 5)])
def test_gradients_in_pieces(n, vocab, d, offset, grad_offset, accumulate):
    g, h, w, y = _inputs(n, vocab, d, offset)
    size = max(zf.zero_head_loss_workspace_bytes(n, vocab, d),
               zf.zero_head_loss_grad_workspace_bytes(n, vocab, d))
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    gl = torch.rand(n, generator=g, device="cuda") / n
    dh, dw = torch.empty_like(h), _at((vocab, d), grad_offset)
    dw.copy_(torch.randn((1, d), generator=g, device="cuda") * 1e-4)
    old = dw.clone() if accumulate else None
    zf.zero_head_loss_grad(h, w, y, lse, gl, dh, dw, accumulate, ws, size)
    assert bool((ws[size:] == 0xFF).all())
    live = (y >= 0) & (y < vocab)
    hl, wl, gg = h[live].to(F64), w.to(F64), gl[live].to(F64)[:, None]
    z, off = L.head_logits(h[live], w)
    x = z - lse[live].to(F64)[:, None]
    p = torch.exp(x)
    # the bounds of layer_reference: fp32's exponent and exponential, dz in bf16
    p_off = p * (off + 6 * R.U + 3 * R.U * (x.abs() + lse[live].to(F64).abs()[:, None]))
    dz = p.clone().scatter_add(1, y[live][:, None], torch.full_like(p[:, :1], -1.0)) * gg
    dz_off = (p_off + 2 * R.U * (p + dz.abs())) * gg + 2.0 ** -8 * dz.abs() + 2.0 ** -126
    for got, a, a_off, b, before, what in ((dh[live], dz, dz_off, wl, None, "grad_hidden"),
                                           (dw, dz.t(), dz_off.t(), hl, old, "grad_table")):
        want = a @ b
        bound = a_off @ b.abs() + (L.chain(2 * a.shape[1]) + 80 * R.U) * (a.abs() @ b.abs())
        if before is not None:
            want = want + before.to(F64)
            bound = bound + 2 * R.U * want.abs()
        got, low, high = got.to(F64), (want - bound).to(BF16).to(F64), (want + bound).to(BF16).to(F64)
        assert bool(((got >= low) & (got <= high)).all()), what
        # as far as their own rounding and dz's leave them in the 2-norm: 2^-9 each and more
        norm = torch.linalg.vector_norm
        assert float(norm(got - want)) <= 2.0 ** -8 * float(norm(want)), what
    assert bool((dh[~live] == 0.0).all())
