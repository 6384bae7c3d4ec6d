"""Operators of a decoder layer's norm and of the head: the root-mean-square
norm with the residual's addition, rows in 8 bits, and the softmax cross
entropy over the vocabulary without the logits in memory.

The same function names as in include/zero_flat.h, and the conventions of
``root_ops``: torch CUDA tensors, matrices with contiguous rows of any stride,
the current stream of the tensors' device unless another is given, ZeroError
for what does not fit together.

Rows in 8 bits are a pair (codes, scales): codes of torch.float8_e4m3fn (or
torch.uint8), rows of the matrix's width and of any stride; scales fp32,
contiguous (rows, ceil(width / 128)).
"""
from __future__ import annotations

import ctypes

import torch

from .root_ops import (_ELEM, _F32, _IDS, _INVALID, _SIZE, _bytes, _here, _on, _ptr, _refuse,
                       _rows, _table, _vector, _workspace)
from .zero import _check, load

ZERO_EIGHT_BLOCK = 128
ZERO_MAX_HEAD_TOKENS = 1 << 22
ZERO_MAX_HEAD_VOCAB = 1 << 22
ZERO_MAX_HEAD_DIM = 32768

_BF16 = {torch.bfloat16: 2}
_CODES = {torch.float8_e4m3fn: 1, torch.uint8: 1}


def _packed(pair, n: int, d: int, name: str, func: str, device: int):
    """(codes, row stride, scales) as addresses of an optional pair."""
    if pair is None:
        return None, 0, None
    if isinstance(pair, torch.Tensor) or len(pair) != 2:
        _refuse(_INVALID, func, f"{name}: a pair (codes, scales) is needed")
    codes, scales = pair
    m, e, stride = _rows(codes, f"{name}'s codes", func)
    if (m, e) != (n, d):
        _refuse(_SIZE, func, f"{name}: codes {tuple(codes.shape)} do not hold {n} rows of {d}")
    _bytes(codes, _CODES, f"{name}'s codes", func, device)
    blocks = (d + ZERO_EIGHT_BLOCK - 1) // ZERO_EIGHT_BLOCK
    _vector(scales, n * blocks, _F32, f"{name}'s scales", func, device)
    return codes.data_ptr(), stride, scales.data_ptr()


def _like(t, n: int, d: int, dtype, name: str, func: str, device: int):
    """(address, row stride) of an optional matrix of n rows of d."""
    if t is None:
        return None, 0
    m, e, stride = _rows(t, name, func)
    if (m, e) != (n, d):
        _refuse(_SIZE, func, f"{name} {tuple(t.shape)} does not hold {n} rows of {d}")
    if t.dtype != dtype:
        _refuse(_INVALID, func, f"{name} is of type {t.dtype}, not {dtype}")
    if t.get_device() != device or device < 0:
        _here(t, name, func, device)
    return t.data_ptr(), stride


def zero_pack_rows(x, packed, stream=None):
    """Rows of x (bf16 or fp32) in 8 bits: packed = (codes, scales) is written."""
    f, dev = "zero_pack_rows", x.get_device()
    n, d, stride = _rows(x, "x", f)
    codes, codes_stride, scales = _packed(packed, n, d, "packed", f, dev)
    _check(load().zero_pack_rows(x.data_ptr(), _bytes(x, _ELEM, "x", f, dev), n, d, stride, codes,
                                 codes_stride, scales, _on(dev, stream)), f)


def zero_unpack_rows(packed, out, stream=None):
    """What rows in 8 bits stand for: out (bf16 or fp32) = code * scale."""
    f, dev = "zero_unpack_rows", out.get_device()
    n, d, stride = _rows(out, "out", f)
    codes, codes_stride, scales = _packed(packed, n, d, "packed", f, dev)
    _check(load().zero_unpack_rows(codes, codes_stride, scales, n, d, out.data_ptr(),
                                   _bytes(out, _ELEM, "out", f, dev), stride, _on(dev, stream)), f)


def zero_rms_norm(x, residual, weight, eps: float, out=None, total=None, rstd=None,
                  packed_out=None, packed_total=None, stream=None):
    """total = x + residual; out = total * rstd * weight over the last dimension.

    residual: of x's shape and type, or None; weight: (dim,) or None (ones);
    out, total: of x's shape and type, or None (total may be x or residual, out
    may be x); rstd: fp32, one value per row, or None; packed_out, packed_total:
    (codes, scales) for out and total in 8 bits, or None."""
    f, dev = "zero_rms_norm", x.get_device()
    n, d, x_stride = _rows(x, "x", f)
    xb = _bytes(x, _ELEM, "x", f, dev)
    res, res_stride = _like(residual, n, d, x.dtype, "residual", f, dev)
    o, o_stride = _like(out, n, d, x.dtype, "out", f, dev)
    t, t_stride = _like(total, n, d, x.dtype, "total", f, dev)
    wb = _vector(weight, d, _ELEM, "weight", f, dev)
    _vector(rstd, n, _F32, "rstd", f, dev)
    _check(load().zero_rms_norm(x.data_ptr(), res, xb, n, d, x_stride, res_stride, _ptr(weight),
                                wb or 4, eps, o, o_stride, t, t_stride,
                                *_packed(packed_out, n, d, "packed_out", f, dev),
                                *_packed(packed_total, n, d, "packed_total", f, dev), _ptr(rstd),
                                _on(dev, stream)), f)


def zero_rms_norm_grad_workspace_bytes(n_rows: int, dim: int) -> int:
    out = ctypes.c_int64(0)
    f = "zero_rms_norm_grad_workspace_bytes"
    _check(load().zero_rms_norm_grad_workspace_bytes(n_rows, dim, ctypes.byref(out)), f)
    return int(out.value)


def zero_rms_norm_grad(grad_out, total, weight, rstd, grad_x, grad_weight=None, grad_total=None,
                       out=None, workspace=None, workspace_bytes: int = 0, stream=None):
    """Gradients of zero_rms_norm from its total and rstd.

    total: the rows, or a pair (codes, scales) that holds them in 8 bits;
    grad_total: the gradient that reaches total from elsewhere, added to
    grad_x, or None; grad_x may be grad_out, total or grad_total; grad_weight:
    (dim,) of the weight's type, or None; out: the norm's output once more, or
    None; workspace: device buffer of at least
    zero_rms_norm_grad_workspace_bytes(rows, dim) bytes (None without
    grad_weight)."""
    f, dev = "zero_rms_norm_grad", grad_out.get_device()
    n, d, g_stride = _rows(grad_out, "grad_out", f)
    gb = _bytes(grad_out, _ELEM, "grad_out", f, dev)
    if isinstance(total, torch.Tensor):
        t, t_stride = _like(total, n, d, grad_out.dtype, "total", f, dev)
        eight = (None, 0, None)
    else:
        t, t_stride = None, 0
        eight = _packed(total, n, d, "total", f, dev)
    gt, gt_stride = _like(grad_total, n, d, grad_out.dtype, "grad_total", f, dev)
    if grad_x is None:
        _refuse(_INVALID, f, "grad_x is needed")
    gx, gx_stride = _like(grad_x, n, d, grad_out.dtype, "grad_x", f, dev)
    o, o_stride = _like(out, n, d, grad_out.dtype, "out", f, dev)
    sizes = {b for b in (_vector(weight, d, _ELEM, "weight", f, dev),
                         _vector(grad_weight, d, _ELEM, "grad_weight", f, dev)) if b}
    if len(sizes) > 1:
        _refuse(_INVALID, f, "weight and grad_weight are of different types")
    _vector(rstd, n, _F32, "rstd", f, dev)
    _check(load().zero_rms_norm_grad(
        grad_out.data_ptr(), t, *eight, gb, n, d, g_stride, t_stride, _ptr(weight),
        sizes.pop() if sizes else 4, _ptr(rstd), gt, gt_stride, gx, gx_stride, _ptr(grad_weight),
        o, o_stride, _workspace(workspace, workspace_bytes, f, dev), workspace_bytes,
        _on(dev, stream)), f)


def _head_workspace(f: str, n_tokens: int, vocab: int, dim: int) -> int:
    out = ctypes.c_int64(0)
    _check(getattr(load(), f)(n_tokens, vocab, dim, ctypes.byref(out)), f)
    return int(out.value)


def zero_head_loss_workspace_bytes(n_tokens: int, vocab: int, dim: int) -> int:
    """Bytes that zero_head_loss of up to n_tokens tokens needs, wherever the table lies."""
    return _head_workspace("zero_head_loss_workspace_bytes", n_tokens, vocab, dim)


def zero_head_loss_grad_workspace_bytes(n_tokens: int, vocab: int, dim: int) -> int:
    """Bytes that zero_head_loss_grad of up to n_tokens tokens needs, wherever the table lies."""
    return _head_workspace("zero_head_loss_grad_workspace_bytes", n_tokens, vocab, dim)


def zero_head_loss_in_place_workspace_bytes(n_tokens: int, vocab: int, dim: int) -> int:
    """The same of a table on a 16-byte boundary, dim a multiple of 8: without a copy of it."""
    return _head_workspace("zero_head_loss_in_place_workspace_bytes", n_tokens, vocab, dim)


def zero_head_loss_grad_in_place_workspace_bytes(n_tokens: int, vocab: int, dim: int) -> int:
    """The same of a table on a 16-byte boundary, dim a multiple of 8: without a copy of it."""
    return _head_workspace("zero_head_loss_grad_in_place_workspace_bytes", n_tokens, vocab, dim)


def _head(hidden, table, labels, func: str, device: int):
    """(tokens, dim, hidden's row stride, vocab, bytes of a label)."""
    n, d, stride = _rows(hidden, "hidden", func)
    vocab, dim = _table(table, "table", func)
    if d != dim:
        _refuse(_SIZE, func, f"hidden {tuple(hidden.shape)} and table {tuple(table.shape)} are "
                "of different widths")
    _bytes(hidden, _BF16, "hidden", func, device)
    _bytes(table, _BF16, "table", func, device)
    return n, d, stride, vocab, _vector(labels, n, _IDS, "labels", func, device)


def zero_head_loss(hidden, table, labels, loss, lse=None, workspace=None,
                   workspace_bytes: int = 0, stream=None):
    """Softmax cross entropy of the head, without the logits in memory:
    loss = lse - z[label], lse = log sum exp z, z = hidden table^T; 0 for
    tokens whose label is outside [0, vocab).

    hidden (rows of dim) and table (vocab, dim): bf16; labels: int32 or int64,
    one per row; loss, lse: fp32, one value per row (lse or None); workspace:
    device buffer of at least zero_head_loss_workspace_bytes(rows, vocab, dim)
    bytes."""
    f, dev = "zero_head_loss", hidden.get_device()
    n, d, stride, vocab, lb = _head(hidden, table, labels, f, dev)
    _vector(loss, n, _F32, "loss", f, dev)
    _vector(lse, n, _F32, "lse", f, dev)
    _check(load().zero_head_loss(hidden.data_ptr(), n, d, stride, table.data_ptr(), vocab,
                                 _ptr(labels), lb, _ptr(loss), _ptr(lse),
                                 _workspace(workspace, workspace_bytes, f, dev), workspace_bytes,
                                 _on(dev, stream)), f)


def zero_head_loss_grad(hidden, table, labels, lse, grad_loss, grad_hidden=None, grad_table=None,
                        accumulate: bool = False, workspace=None, workspace_bytes: int = 0,
                        stream=None):
    """Gradients of zero_head_loss from its lse and each token's gradient of
    the loss (fp32; 0 for tokens that do not count).

    grad_hidden: of hidden's shape, bf16 (may be hidden), or None; grad_table:
    (vocab, dim), bf16, or None; with accumulate it is added to; workspace:
    device buffer of at least zero_head_loss_grad_workspace_bytes(rows, vocab,
    dim) bytes."""
    f, dev = "zero_head_loss_grad", hidden.get_device()
    n, d, stride, vocab, lb = _head(hidden, table, labels, f, dev)
    _vector(lse, n, _F32, "lse", f, dev)
    _vector(grad_loss, n, _F32, "grad_loss", f, dev)
    gh, gh_stride = _like(grad_hidden, n, d, torch.bfloat16, "grad_hidden", f, dev)
    if grad_table is not None:
        if tuple(_table(grad_table, "grad_table", f)) != (vocab, d):
            _refuse(_SIZE, f, f"grad_table {tuple(grad_table.shape)} is not of the table's shape "
                    f"{(vocab, d)}")
        _bytes(grad_table, _BF16, "grad_table", f, dev)
    _check(load().zero_head_loss_grad(
        hidden.data_ptr(), n, d, stride, table.data_ptr(), vocab, _ptr(labels), lb,
        _ptr(lse), _ptr(grad_loss), gh, gh_stride, _ptr(grad_table), 1 if accumulate else 0,
        _workspace(workspace, workspace_bytes, f, dev), workspace_bytes, _on(dev, stream)), f)
