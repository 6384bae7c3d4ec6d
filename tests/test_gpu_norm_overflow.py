"""Rows whose sum of squares is beyond fp32."""
import pytest
import torch

import layer_reference as L
import root_reference as R

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d", [(7, 64), (300, 1501), (40, 4096), (9, 8200), (5, 16384),
                                 (5, 16383)])
def test_rms_norm_of_rows_whose_squares_overflow(n, d, dtype):
    """Row by row values about 2^56 ... 2^126 (every third row an ordinary one), a single
    large value, the residual's share of it.  rstd times 2^-72 is as exact as any, and the
    product is rounded where it is below the normal numbers (2^-150), as are s rstd (then
    times w, at most 1.5) and its product by w: 2.5 2^-150 < 2^-148 in all."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn((n, d), generator=g)
    size = torch.exp2(torch.randint(56, 124, (n,), generator=g).float())
    size[::3] = 1.0
    x = (x * size[:, None]).to(dtype)
    x[1] = torch.randn(d, generator=g).to(dtype)
    x[1, d // 2] = 3.0e38
    residual = (torch.randn((n, d), generator=g) * size[:, None]).to(dtype)
    residual[1] = 0.0
    w = (torch.rand(d, generator=g) + 0.5).to(dtype)
    dy = torch.randn((n, d), generator=g).to(dtype)
    xg, rg, wg, dyg = (t.cuda() for t in (x, residual, w, dy))
    total = (xg.float() + rg.float())
    assert bool(torch.isfinite(total).all())
    out, kept = torch.empty_like(xg), torch.empty_like(xg)
    rstd = torch.empty(n, device="cuda")
    zf.zero_rms_norm(xg, rg, wg, 1e-5, out, kept, rstd)
    y, y_off, r, r_off = L.rms_norm(total.cpu().to(F64), w, 1e-5)
    R.check(rstd, r, r_off + 2.0 ** -149, "rstd")
    R.check(out, y, y_off + total.cpu().to(F64).abs() * 2.0 ** -148 + 2.0 ** -148, "out")
    dx, dw = torch.empty_like(xg), torch.empty_like(wg)
    size = zf.zero_rms_norm_grad_workspace_bytes(n, d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    zf.zero_rms_norm_grad(dyg, kept, wg, rstd, dx, dw, None, None, ws, size)
    (ex, x_off), (ew, w_off), _ = L.rms_norm_grad(dyg, kept.cpu().to(F64), w, rstd, None)
    # (below the normal numbers: a unit of 2^-149, of bf16 2^-133)
    R.check(dx, ex, x_off + 2.0 ** -132, "grad_x")
    R.check(dw, ew, w_off, "grad_weight")


@pytest.mark.parametrize("d", [64, 1501, 4096])
def test_layer_norm_of_rows_whose_variance_overflows(d):
    """1 / sqrt of infinity is 0, so the row is the bias; the other rows are what they are."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn((6, d), generator=g)
    x[::2] *= 1e30
    w, b = torch.rand(d, generator=g) + 0.5, torch.randn(d, generator=g)
    out, mean, rstd = torch.empty((6, d), device="cuda"), *torch.empty((2, 6), device="cuda")
    zf.zero_layer_norm(x.cuda(), w.cuda(), b.cuda(), 1e-5, out, mean, rstd)
    assert bool((rstd[::2] == 0.0).all()) and torch.equal(out[::2].cpu(), b.expand(3, d))
    want = torch.nn.functional.layer_norm(x[1::2].double(), (d,), w.double(), b.double(), 1e-5)
    assert float((out[1::2].cpu() - want).abs().max()) <= 1e-4
