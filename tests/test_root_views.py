"""Tensors of more than two dimensions as rows of one stride: which views the
binding takes, and on the GPU what the operators make of them."""
import pytest
import torch

import distill_bounds as D

import fsdp_sharded_mixed_flatten_gb300 as zf
from fsdp_sharded_mixed_flatten_gb300.root_ops import _rows


def _t(*shape):
    return torch.arange(torch.Size(shape).numel(), dtype=torch.float32).view(shape)


@pytest.mark.parametrize("view,n,stride", [
    (_t(4, 5, 6), 20, 6), (_t(2, 3, 4, 5), 24, 5),
    (_t(4, 5, 6)[:, -1:], 4, 30),                  # the last token of each sequence
    (_t(4, 5, 6)[:, :1, :4], 4, 30), (_t(4, 5, 6)[1:2], 5, 6), (_t(4, 5, 6)[::2, 2:3], 2, 60),
    (_t(7, 9)[:, :8].unsqueeze(1), 7, 9), (_t(7, 9)[:, :8].unsqueeze(0), 7, 9),
    (_t(7, 9)[:, :8].unflatten(0, (7, 1, 1)), 7, 9), (_t(6, 9)[:, :8].unflatten(0, (2, 1, 3)), 6, 9),
    (_t(4, 5, 6)[2:3, 3:4], 1, 6), (_t(4, 5, 6)[:, :0], 0, 6), (_t(4, 0, 6), 0, 6),
    (_t(0, 5, 6)[:, :3], 0, 6), (_t(1, 1, 6), 1, 6),
])
def test_rows_of_one_stride(view, n, stride):
    got_n, d, got = _rows(view, "x", "f")
    assert (got_n, d) == (n, view.shape[-1])
    assert got == stride if n > 1 else got >= d
    if n > 1:                                      # the rows that these numbers name
        flat = torch.as_strided(view, (n, d), (got, 1))
        assert torch.equal(flat, view.reshape(n, d))


@pytest.mark.parametrize("view", [
    _t(4, 5, 6)[:, :3], _t(4, 5, 6).transpose(0, 1), _t(4, 5, 6)[:, ::2], _t(2, 5, 3, 6)[:, :, :2],
    _t(4, 6, 5).transpose(1, 2), _t(3, 1, 6).expand(3, 4, 6),
])
def test_other_views_are_refused(view):
    with pytest.raises(zf.ZeroError) as ei:
        _rows(view, "x", "f")
    assert ei.value.code == -3


@pytest.mark.gpu
def test_last_tokens_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    g = torch.Generator(device="cuda").manual_seed(4)
    b, s, d, vocab, top = 5, 7, 40, 33, 3
    x = torch.randn((b, s, d), generator=g, device="cuda")
    before, last = x.clone(), x[:, -1:]
    w, bias = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    want, got = torch.empty((b, d), device="cuda"), torch.empty((b, 1, d), device="cuda")
    zf.zero_layer_norm(last.reshape(b, d).clone(), w, bias, 1e-5, want)
    zf.zero_layer_norm(last, w, bias, 1e-5, got)
    assert torch.equal(got[:, 0], want)
    zf.zero_layer_norm(last, w, bias, 1e-5, last)                 # in place, in the buffer
    assert torch.equal(x[:, -1], want) and torch.equal(x[:, :-1], before[:, :-1])
    table = torch.randn((vocab, d), generator=g, device="cuda")
    ids = torch.randint(0, vocab, (b, 1), generator=g, device="cuda")
    zf.zero_embedding(ids, table, last)
    assert torch.equal(x[:, -1], table[ids[:, 0]]) and torch.equal(x[:, :-1], before[:, :-1])
    z = torch.randn((b, s, vocab), generator=g, device="cuda")
    tid = torch.randint(0, vocab, (b, top), generator=g, device="cuda", dtype=torch.int32)
    t = torch.randn((b, top), generator=g, device="cuda")
    loss = torch.empty(b, device="cuda")
    ref = D.distill(z[:, -1], tid, t, None, 2.0)
    zf.zero_distill_loss_grad(z[:, -1:], tid, t, None, 2.0, loss, z[:, -1:])
    D.check(loss, ref["loss"], ref["d_loss"], "loss")
    D.check(z[:, -1], ref["grad"], ref["d_grad"], "grad_logits")
