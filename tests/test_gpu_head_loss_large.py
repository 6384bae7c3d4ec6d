"""The head's loss at logits of any size that fp32 holds."""
import math

import pytest
import torch

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


def _loss(h, w, y):
    n, vocab, d = h.shape[0], *w.shape
    size = zf.zero_head_loss_workspace_bytes(n, vocab, d)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((2, n), 7.0, device="cuda")
    zf.zero_head_loss(h.to(BF16).cuda(), w.to(BF16).cuda(), y.cuda(), out[0], out[1], ws, size)
    return out.to(F64).cpu()


SIZES = [2.0 ** e for e in (10, 24, 31, 32, 33, 40, 60, 90, 120)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("n", [2, 40, 130, 300])
def test_equal_logits(n, size):
    """log(vocab) and lse = z + log(vocab).  z is one product; a row's sum has no rounding
    larger than 300 2^-24 of itself, each exponential is of 0, the logarithm is within 2 ulp
    (2^-21 below 16), and lse is rounded once."""
    vocab, d = 12288, 64
    h, w = torch.zeros((n, d)), torch.zeros((vocab, d))
    h[:, 0] = 2.0 ** (round(math.log2(size)) // 2) * (1 + torch.arange(n) % 128 / 128.0)
    h[::2, 0] *= -1.0
    w[:, 0] = 2.0 ** (round(math.log2(size)) - round(math.log2(size)) // 2)
    loss, lse = _loss(h, w, torch.arange(n) * 37)
    z = h[:, 0].double() * w[0, 0].double()
    off = 300 * 2.0 ** -24 + 2.0 ** -20
    assert float((loss - math.log(vocab)).abs().max()) <= off
    assert bool(((lse - z - math.log(vocab)).abs() <= off + 2.0 ** -23 * z.abs()).all())


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("n", [2, 40, 130, 300])
def test_labels_below_the_largest_logit(n, size):
    """Half of the table is at z, the label far below it: the loss is the difference and the
    logarithm of half the vocabulary, rounded once."""
    vocab, d = 4000, 64
    h, w = torch.zeros((n, d)), torch.zeros((vocab, d))
    h[:, 0] = 2.0 ** (round(math.log2(size)) // 2)
    w[::2, 0] = 2.0 ** (round(math.log2(size)) - round(math.log2(size)) // 2)
    w[1::2, 0] = -0.75 * w[0, 0]
    loss, lse = _loss(h, w, 1 + 2 * (torch.arange(n) * 37 % 2000))
    want = 1.75 * size + math.log(vocab / 2)
    assert bool(((loss - want).abs() <= 2.0 ** -23 * want).all())
    assert bool(((lse - size - math.log(vocab / 2)).abs() <= 2.0 ** -23 * size + 2e-5).all())
