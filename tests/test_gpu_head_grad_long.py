"""Long sums of the head's loss and its gradients: tensor memory cuts its sums off instead
of rounding them, so what is summed there in one go has to end before that counts."""
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


def _workspace(n, vocab, d):
    size = max(zf.zero_head_loss_workspace_bytes(n, vocab, d),
               zf.zero_head_loss_grad_workspace_bytes(n, vocab, d))
    return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"), size


def _sure(n, d, z):
    """Tokens whose label has a logit of about z, a sum of products of one sign; the other
    rows of the table are zeros."""
    g = torch.Generator().manual_seed(n + d)
    h = (torch.rand((n, d), generator=g) + 0.5).to(BF16).cuda()
    w = torch.zeros((40, d), dtype=BF16, device="cuda")
    w[11] = ((torch.rand(d, generator=g) + 0.5) * (z / d)).to(BF16).cuda()
    y = torch.full((n,), 11, device="cuda")
    return h, w, y


@pytest.mark.parametrize("d", [1536, 1544, 4096, 8192])
@pytest.mark.parametrize("n", [1, 20, 50, 200, 300])
def test_the_gradients_logits_are_the_losss(n, d):
    """Where a token's label has all of the probability, the loss's lse is the label's logit
    itself; the gradient is zero, as it finds the same logit."""
    h, w, y = _sure(n, d, 300.0)
    ws, size = _workspace(n, 40, d)
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    zf.zero_head_loss_grad(h, w, y, lse, torch.ones(n, device="cuda"), dh, dw, False, ws, size)
    assert bool((dh == 0.0).all()) and bool((dw == 0.0).all())


@pytest.mark.parametrize("d", [4096, 8192])
def test_the_gradients_logits_are_sums_of_short_parts(d):
    """dz of a sure token is exp(z - lse) - 1, and shows how far the kernel's z is off.  A
    step of 16 products cuts off half a unit of the sum so far, 2^-24 of it at most, in the
    mean.  In parts of 1536 columns, whose sums grow evenly, those are 48 such losses of a
    part's whole sum, so 48 2^-24 z; the additions of the parts are rounded.  In one go they
    would be 128 losses of half a unit between 2^-25 and 2^-24 of z at 4096 columns: 64 2^-24 z
    and more.  A mean over 300 tokens whose dz has bf16's rounding (2^-9 of it)."""
    n = 300
    h, w, y = _sure(n, d, 300.0)
    z = h.to(F64) @ w[11].to(F64)
    lse = z.float()
    ws, size = _workspace(n, 40, d)
    dh = torch.empty_like(h)
    zf.zero_head_loss_grad(h, w, y, lse, torch.ones(n, device="cuda"), dh, None, False, ws, size)
    dz = (dh.to(F64) @ w[11].to(F64)) / w[11].to(F64).square().sum()
    want = torch.exp(z - lse.to(F64)) - 1.0
    off = float((dz - want).mean().abs() / z.mean())
    assert off <= 56 * 2.0 ** -24, f"off by {off * 2.0 ** 24} 2^-24"


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,d,offset", [(1 << 21, 64, 0), (70000, 600, 0), (70001, 77, 5)])
def test_sums_over_many_tokens_of_one_sign(n, d, offset, accumulate):
    """Equal logits of 32 rows and one label: dz is 2^-5 and 2^-5 - 1, bf16 values, so the
    table's gradient is a sum of h.  Each element is bf16 (2^-8 of itself); a step of 16
    tokens cuts off two units of 2^-23 of the sum so far at most, so parts of 65536, whose sums
    grow evenly, end 4096 / 2 2^-22 = 2^-11 low at most, and exponentials are off by 2^-22.  The
    columns' sums are spread over an octave, where roundings average out, to 2^-11 in the mean
    of 64 of them."""
    g = torch.Generator(device="cuda").manual_seed(d)
    vocab = 32
    spread = 1.0 + torch.arange(d, device="cuda") % 64 / 64.0
    h = torch.empty((n, d), dtype=BF16, device="cuda")
    h.copy_((torch.rand((n, d), generator=g, device="cuda") + 0.5) * spread)
    w = torch.zeros(offset + vocab * d, dtype=BF16, device="cuda")[offset:].view(vocab, d)
    y = torch.full((n,), 5, device="cuda")
    ws, size = _workspace(n, vocab, d)
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    dw = torch.full((offset + vocab * d,), 3.0, dtype=BF16, device="cuda")[offset:].view(vocab, d)
    zf.zero_head_loss_grad(h, w, y, lse, torch.full((n,), 1.0 / 1024, device="cuda"), None, dw,
                           accumulate, ws, size)
    total = torch.zeros(d, dtype=F64, device="cuda")
    for a in range(0, n, 1 << 18):
        total += h[a:a + (1 << 18)].to(F64).sum(0)
    for v, p in ((5, 2.0 ** -5 - 1.0), (0, 2.0 ** -5), (31, 2.0 ** -5)):
        want = total * p / 1024 + (3.0 if accumulate else 0.0)
        off = (dw[v].to(F64) - want) / want.abs()
        assert float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20
        assert abs(float(off.mean())) <= 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -20


@pytest.mark.parametrize("n", [3, 200])
def test_sums_over_a_long_vocabulary(n):
    """No hidden states: every row of the table counts 1 / vocab in the gradient, as a sum of
    262144 values of one sign.  dz is bf16 (2^-18 is one of its values; minus one, 1), the
    result is (2^-8), and sums end 2^-11 low at most (as above)."""
    vocab, d = 1 << 18, 8192
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.empty((vocab, d), dtype=BF16, device="cuda")
    mean = torch.zeros(d, dtype=F64, device="cuda")
    for a in range(0, vocab, 1 << 14):
        w[a:a + (1 << 14)] = (torch.rand((1 << 14, d), generator=g, device="cuda") + 0.5).to(BF16)
        mean += w[a:a + (1 << 14)].to(F64).sum(0) / vocab
    h = torch.zeros((n, d), dtype=BF16, device="cuda")
    y = torch.arange(n, device="cuda") * 977
    ws, size = _workspace(n, vocab, d)
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    dh = torch.empty_like(h)
    zf.zero_head_loss_grad(h, w, y, lse, torch.ones(n, device="cuda"), dh, None, False, ws, size)
    own = w[y].to(F64)
    want = mean - own
    off = (dh.to(F64) - want).abs()
    assert bool((off <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * mean + 2.0 ** -20 * own).all())


@pytest.mark.parametrize("n", [20, 50, 200, 300])
def test_the_losss_logits_are_sums_of_short_parts(n):
    """The same of the loss, in the mean over tokens whose label's logit is 0: it is the other
    logit itself."""
    d = 4096
    h, w, y = _sure(n, d, 300.0)
    z = h.to(F64) @ w[11].to(F64)
    ws, size = _workspace(n, 40, d)
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, torch.full_like(y, 3), loss, lse, ws, size)
    off = float((loss.to(F64) - z).mean().abs() / z.mean())
    assert off <= 56 * 2.0 ** -24, f"off by {off * 2.0 ** 24} 2^-24"
