"""Gradients of the head's loss where few tokens are live, next to their own rounding:
so few terms average nothing, and the bf16 operand of the products has to keep more
digits than one bf16 value holds."""
import pytest
import torch

import layer_reference as L

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


def _case(seed, n, live, vocab, d, offset):
    """Live tokens spread over the n, logits spread by 2, some labels of large logits."""
    g = torch.Generator().manual_seed(1000 * n + 10 * live + seed)
    flat = torch.zeros(offset + vocab * d, dtype=BF16, device="cuda")
    w = flat[offset:].view(vocab, d)
    w.copy_(torch.randn((vocab, d), generator=g) * 0.25)
    y = torch.full((n,), -100)
    at = torch.randperm(n, generator=g)[:live]
    y[at] = torch.randint(0, vocab, (live,), generator=g)
    h = torch.randn((n, d), generator=g) * (8.0 / d ** 0.5)
    near = w[y[at].cuda()].cpu().float()
    h[at] += near / near.square().sum(1, keepdim=True) * torch.rand((live, 1), generator=g) * 9.0
    gl = torch.rand(n, generator=g) + 0.5
    return h.to(BF16).cuda(), w, y.cuda(), gl.cuda()


def _grads(h, w, y, gl, old=None):
    (n, d), vocab = h.shape, w.shape[0]
    size = max(zf.zero_head_loss_workspace_bytes(n, vocab, d),
               zf.zero_head_loss_grad_workspace_bytes(n, vocab, d))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty((2, n), device="cuda")
    zf.zero_head_loss(h, w, y, loss, lse, ws, size)
    dh = torch.empty_like(h)
    flat = torch.zeros(w.storage_offset() + w.numel(), dtype=BF16, device="cuda")
    dw = flat[w.storage_offset():].view(w.shape)
    if old is not None:
        dw.copy_(old)
    zf.zero_head_loss_grad(h, w, y, lse, gl, dh, dw, old is not None, ws, size)
    return lse, dh, dw


def _exact(h, w, y, lse, gl):
    """The gradients, and how far (2-norm) a sum of products of dz in two bf16 parts may be
    off them before its rounding: 2^-16 of a dz from the rest's rounding, the logits' sums
    (L.chain), p's exponent and exponential (8 u and 3 u |x|), and the products' own sums."""
    live = (y >= 0) & (y < w.shape[0])
    hl, wl, g = h[live].to(F64), w.to(F64), gl[live].to(F64)[:, None]
    z, off = L.head_logits(h[live], w)
    x = z - lse[live].to(F64)[:, None]
    p = torch.exp(x)
    dz = p.scatter_add(1, y[live][:, None], torch.full_like(p[:, :1], -1.0)) * g
    dz_off = (p * (off + 8 * U + 3 * U * (x.abs() + lse[live].to(F64).abs()[:, None])) + 2 * U) \
        * g + 2.0 ** -16 * dz.abs()
    norm = lambda t: float(torch.linalg.vector_norm(t))                  # noqa: E731
    wide = lambda t: float(torch.linalg.matrix_norm(t, 2))               # noqa: E731
    out = []
    for a, b, of in ((dz, wl, wl), (dz.t(), hl, hl)):
        sums = norm((L.chain(2 * a.shape[1]) + 80 * U) * (a.abs() @ b.abs()))
        out.append((a @ b, norm(dz_off) * wide(of) + sums))
    full = torch.zeros(h.shape, dtype=F64, device=h.device)
    full[live] = out[0][0]
    return (full, out[0][1]), out[1]


def _near(got, want, off, what):
    """Rounded to nearest after an error of `off` (2-norm): bf16(x + e) is no farther from x
    than bf16(x) is, and 2 |e|."""
    norm = torch.linalg.vector_norm
    own = float(norm(want.to(BF16).to(F64) - want))
    far = float(norm(got.to(F64) - want))
    assert far <= own + 2 * off, f"{what}: {far / float(norm(want))} of itself off, " \
        f"{own / float(norm(want))} by rounding, {off / float(norm(want))} before it"


@pytest.mark.parametrize("offset", [0, 5])
@pytest.mark.parametrize("n,live,vocab,d", [
    (1, 1, 5003, 256), (2, 2, 3001, 72), (5, 3, 777, 64), (64, 64, 5003, 256), (65, 65, 1000, 257),
    (127, 127, 2000, 136), (128, 128, 4099, 256), (600, 100, 1000, 200), (9000, 1, 600, 96),
    (9000, 128, 600, 96), (257, 7, 50257, 768)])
def test_gradients_of_few_live_tokens_are_off_by_their_own_rounding(n, live, vocab, d, offset):
    for seed in range(4 if n < 8 else 1):
        h, w, y, gl = _case(seed, n, live, vocab, d, offset)
        old = (torch.randn(w.shape, device="cuda") * 0.01).to(BF16) if seed % 2 else None
        lse, dh, dw = _grads(h, w, y, gl, old)
        (eh, h_off), (ew, w_off) = _exact(h, w, y, lse, gl)
        _near(dh, eh, h_off, "grad_hidden")
        if old is not None:
            ew = ew + old.to(F64)
            w_off += 2 * U * float(torch.linalg.vector_norm(ew))
        _near(dw, ew, w_off, "grad_table")
        again = _grads(h, w, y, gl, old)
        assert torch.equal(again[1], dh) and torch.equal(again[2], dw)
