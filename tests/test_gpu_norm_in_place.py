"""The norm's gradient in place of any of its inputs gives the bits that it gives beside
them, and so does the forward pass, where the arrays beside them are laid out alike (the
sums' order goes by strides)."""
import pytest
import torch

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


def _rows(n, d, pad, dtype, g):
    t = torch.zeros((n, d + pad), dtype=dtype, device="cuda")[:, :d]
    return t.copy_(torch.randn((n, d), generator=g))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (700, 64, 0), (333, 257, 3), (400, 4096, 0),
                                     (400, 4001, 0), (9, 8200, 8), (170, 16384, 0),
                                     (5, 16383, 1)])
def test_gradient_in_place_of_each_input(n, d, pad, dtype):
    g = torch.Generator().manual_seed(n + d)
    total, dy, dt = (_rows(n, d, pad, dtype, g) for _ in range(3))
    w = (torch.rand(d, generator=g) + 0.5).to(dtype).cuda()
    rstd = torch.empty(n, device="cuda")
    zf.zero_rms_norm(total, None, w, 1e-5, None, None, rstd)
    size = zf.zero_rms_norm_grad_workspace_bytes(n, d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want, again = (_rows(n, d, pad, dtype, g) for _ in range(2))
    want_w = torch.empty_like(w)
    zf.zero_rms_norm_grad(dy, total, w, rstd, want, want_w, dt, again, ws, size)
    for which in range(3):
        a = [t.new_zeros((n, d + pad))[:, :d].copy_(t) for t in (dy, total, dt)]
        dw, out = torch.empty_like(w), _rows(n, d, pad, dtype, g)
        zf.zero_rms_norm_grad(a[0], a[1], w, rstd, a[which], dw, a[2], out, ws, size)
        assert torch.equal(a[which], want) and torch.equal(dw, want_w), which
        assert torch.equal(out, again)
        for i, t in enumerate((dy, total, dt)):
            assert i == which or torch.equal(a[i], t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d,pad", [(700, 64, 0), (333, 257, 3), (400, 4096, 0), (170, 16384, 0)])
def test_forward_in_place(n, d, pad, dtype):
    g = torch.Generator().manual_seed(n + d)
    x, residual = (_rows(n, d, pad, dtype, g) for _ in range(2))
    out, total = (_rows(n, d, pad, dtype, g) for _ in range(2))
    zf.zero_rms_norm(x, residual, None, 1e-5, out, total)
    for out_at, total_at in ((0, None), (None, 0), (None, 1), (0, 1)):
        a = [t.new_zeros((n, d + pad))[:, :d].copy_(t) for t in (x, residual)]
        o = _rows(n, d, pad, dtype, g) if out_at is None else a[out_at]
        t = _rows(n, d, pad, dtype, g) if total_at is None else a[total_at]
        zf.zero_rms_norm(a[0], a[1], None, 1e-5, o, t)
        assert torch.equal(o, out) and torch.equal(t, total)
