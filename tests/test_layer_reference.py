"""The plain implementations of layer_reference.py against other ones: rows in
8 bits against PyTorch's e4m3, the norm and its gradient against autograd."""
import numpy as np
import torch

import layer_reference as L

F64 = torch.float64


def test_pack_is_torchs_rounding():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((40, 300), generator=g) * torch.exp(4 * torch.randn((40, 300), generator=g))
    codes, scales = L.pack(x.numpy())
    for a in range(0, 300, 128):
        part = x[:, a:a + 128]
        s = torch.from_numpy(scales[:, a // 128:a // 128 + 1])
        top = part.abs().amax(1, keepdim=True)
        assert bool((top <= 448 * s).all()) and bool((top > 224 * s).all())
        want = (part / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes[:, a:a + 128], want)
        back = torch.from_numpy(want).view(torch.float8_e4m3fn).to(F64) * s
        assert np.array_equal(L.unpack(codes, scales)[:, a:a + 128], back.numpy())


def test_every_code_is_its_own_rounding():
    codes = np.arange(256, dtype=np.uint8)
    values = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    full = np.concatenate([[448.0], values])[None, :128].astype(np.float32)
    got, scale = L.pack(full)
    assert scale[0, 0] == 1.0 and np.array_equal(got[0, 1:], codes[:127])
    assert np.array_equal(np.nan_to_num(L.unpack(codes[None], np.ones((1, 2)))[0], nan=7.0),
                          np.nan_to_num(values.astype(np.float64), nan=7.0))


def test_norm_is_autograds():
    g = torch.Generator().manual_seed(6)
    x, dy, t = (torch.randn((5, 77), generator=g, dtype=F64) for _ in range(3))
    w = torch.randn(77, generator=g, dtype=F64)
    x.requires_grad_()
    w.requires_grad_()
    eps = float(torch.tensor(1e-5))
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * w
    (y * dy).sum().add((x * t).sum()).backward()
    out, _, rstd, _ = L.rms_norm(x.detach(), w.detach(), 1e-5)
    (dx, _), (dw, _), (again, _) = L.rms_norm_grad(dy, x.detach(), w.detach(), rstd, t)
    for a, b in ((out, y), (again, y), (dx, x.grad), (dw, w.grad)):
        assert torch.allclose(a, b.detach(), rtol=1e-12, atol=1e-12)


def test_head_loss_is_autograds():
    g = torch.Generator().manual_seed(7)
    h = torch.randn((9, 24), generator=g).bfloat16().to(F64).requires_grad_()
    w = (torch.randn((50, 24), generator=g) * 0.3).bfloat16().to(F64).requires_grad_()
    y = torch.tensor([3, -100, 49, 0, 50, 7, 7, 8, 1])
    gl = torch.rand(9, generator=g)
    gl[5] = 0.0
    each = torch.nn.functional.cross_entropy(h @ w.t(), torch.where(y < 50, y, -100),
                                             reduction="none", ignore_index=-100)
    (each * gl).sum().backward()
    (loss, _), (lse, _) = L.head_loss(h.detach(), w.detach(), y)
    assert torch.allclose(loss, each.detach(), rtol=1e-12, atol=1e-12)
    # the reference takes the rows' fp32 lse; here in full, through a 64-bit tensor
    (dh, _, _), (dw, _, _) = L.head_loss_grad(h.detach(), w.detach(), y, lse, gl)
    assert torch.allclose(dh, h.grad, rtol=1e-12, atol=1e-12)
    assert torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-12)
