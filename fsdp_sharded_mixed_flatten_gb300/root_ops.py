"""Operators around the root unit: token table, layer norm, distillation loss.

The same function names as in include/zero_flat.h.  Unlike the sharded step,
whose buffers may be raw addresses, these take torch CUDA tensors: sizes,
types and row strides are read from them and passed on; what does not fit
together is refused here with the library's codes (ZeroError), the rest by
the library.  A parameter or gradient may be a view into a flat buffer at any
element.  Matrices need contiguous rows, of any stride; tensors of more than
two dimensions, one stride over all leading ones.  Calls run on the given stream, by
default torch's current one of the tensors' device, which must be the current
device and the same for all of them.
"""
from __future__ import annotations

import ctypes

import torch

from .zero import ZeroError, _check, load

ZERO_MAX_NORM_DIM = 16384
ZERO_MAX_TEACHER = 1024

_INVALID, _SIZE = -1, -3
_ELEM = {torch.bfloat16: 2, torch.float32: 4}
_IDS = {torch.int32: 4, torch.int64: 8}
_I32 = {torch.int32: 4}
_F32 = {torch.float32: 4}
# the raw handle without building a Stream object, which costs as much as a call
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _refuse(code: int, func: str, message: str):
    raise ZeroError(code, message, func)


def _here(t: torch.Tensor, name: str, func: str, device: int):
    """The kernels reach a tensor only on the call's GPU, `device`.  (Called only
    where a comparison beforehand leaves a doubt: small calls are host-bound.)"""
    if t.get_device() != device or not t.is_cuda:
        _refuse(_INVALID, func, f"{name} is on {t.device}: all tensors of a call have to be on "
                "one GPU")


def _bytes(t: torch.Tensor, types, name: str, func: str, device: int) -> int:
    b = types.get(t.dtype)
    if b is None:
        _refuse(_INVALID, func, f"{name}: type {t.dtype} is not one of "
                + ", ".join(str(k) for k in types))
    if t.get_device() != device or device < 0:
        _here(t, name, func, device)
    return b


def _vector(t, n: int, types, name: str, func: str, device: int) -> int:
    """Element size of an optional contiguous vector of n values (0 if None)."""
    if t is None:
        return 0
    if t.numel() != n or not t.is_contiguous():
        _refuse(_SIZE, func, f"{name}: {n} contiguous values are needed, got shape "
                f"{tuple(t.shape)}, strides {t.stride()}")
    return _bytes(t, types, name, func, device)


def _workspace(t, nbytes: int, func: str, device: int):
    """Address of an optional workspace that holds the stated bytes."""
    if t is None:
        return None
    if t.numel() * t.element_size() < nbytes or not t.is_contiguous():
        _refuse(_SIZE, func, f"workspace of shape {tuple(t.shape)}, {t.dtype}, does not hold the "
                f"stated {nbytes} contiguous bytes")
    if t.get_device() != device or device < 0:
        _here(t, "workspace", func, device)
    return t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t: torch.Tensor, name: str, func: str):
    """(rows, columns, row stride) of a matrix with contiguous rows."""
    if t.dim() == 2:
        (n, d), (stride, inner) = t.shape, t.stride()
    elif t.dim() == 1:
        n, d, stride, inner = 1, t.shape[0], t.shape[0], t.stride(0)
    elif t.dim() == 0:
        _refuse(_SIZE, func, f"{name} has no dimensions")
    else:
        d, inner = t.shape[-1], t.stride(-1)
        n = t.numel() // d if d else 0
        stride, step = t.stride(-2), 0          # of the rows, and of the next dimension
        if n > 1:
            for size, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
                if size == 1:                   # its stride is of no account
                    continue
                if step == 0:
                    stride = step = s
                if s != step or s == 0:
                    _refuse(_SIZE, func, f"{name}: leading dimensions {tuple(t.shape)} with "
                            f"strides {t.stride()} are not rows of one stride")
                step *= size
    if inner != 1 and d > 1:
        _refuse(_SIZE, func, f"{name}: rows are not contiguous (strides {t.stride()})")
    # the stride of a single row is of no account
    return n, d, stride if n > 1 else max(stride, d)


def _table(t: torch.Tensor, name: str, func: str):
    if t.dim() != 2 or not t.is_contiguous():
        _refuse(_SIZE, func, f"{name}: a contiguous (vocab, dim) table is needed, got shape "
                f"{tuple(t.shape)}, strides {t.stride()}")
    return t.shape


def _on(device: int, stream) -> int:
    if stream is None:
        return _current_stream(device)
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def zero_embedding(ids, weight, out, scale: float = 1.0, stream=None):
    """out[t] = scale * weight[ids[t]]; 0 for ids outside the table.

    ids: int32 or int64, contiguous, any shape; weight: (vocab, dim); out:
    rows of dim, one per id."""
    f, dev = "zero_embedding", out.get_device()
    vocab, dim = _table(weight, "weight", f)
    n, d, stride = _rows(out, "out", f)
    if d != dim or n != ids.numel():
        _refuse(_SIZE, f, f"out {tuple(out.shape)} does not hold {ids.numel()} rows of {dim}")
    _check(load().zero_embedding(ids.data_ptr(), _vector(ids, n, _IDS, "ids", f, dev), n,
                                 weight.data_ptr(), _bytes(weight, _ELEM, "weight", f, dev), vocab,
                                 dim, scale, out.data_ptr(), _bytes(out, _ELEM, "out", f, dev),
                                 stride, _on(dev, stream)), f)


def zero_embedding_grad_workspace_bytes(n_tokens: int, vocab: int, dim: int) -> int:
    out = ctypes.c_int64(0)
    f = "zero_embedding_grad_workspace_bytes"
    _check(load().zero_embedding_grad_workspace_bytes(n_tokens, vocab, dim, ctypes.byref(out)), f)
    return int(out.value)


def zero_embedding_grad(ids, grad_out, grad_weight, scale: float = 1.0, accumulate: bool = False,
                        workspace=None, workspace_bytes: int = 0, stream=None):
    """grad_weight[v] = scale * sum of grad_out[t] over the tokens with id v
    (every row is written), or, with accumulate, that added to grad_weight
    (rows without a token are not touched).

    workspace: device buffer of at least
    zero_embedding_grad_workspace_bytes(tokens, vocab, dim) bytes."""
    f, dev = "zero_embedding_grad", grad_weight.get_device()
    vocab, dim = _table(grad_weight, "grad_weight", f)
    n, d, stride = _rows(grad_out, "grad_out", f)
    if d != dim or n != ids.numel():
        _refuse(_SIZE, f, f"grad_out {tuple(grad_out.shape)} does not hold {ids.numel()} rows "
                f"of {dim}")
    _check(load().zero_embedding_grad(
        ids.data_ptr(), _vector(ids, n, _IDS, "ids", f, dev), n, grad_out.data_ptr(),
        _bytes(grad_out, _ELEM, "grad_out", f, dev), stride, scale, grad_weight.data_ptr(),
        _bytes(grad_weight, _ELEM, "grad_weight", f, dev), vocab, dim, 1 if accumulate else 0,
        _workspace(workspace, workspace_bytes, f, dev), workspace_bytes, _on(dev, stream)), f)


def zero_layer_norm(x, weight, bias, eps: float, out, mean=None, rstd=None, stream=None):
    """out = (x - mean) * rstd * weight + bias over the last dimension.

    weight, bias: (dim,) of one type, or None (ones, zeros); mean, rstd: fp32,
    one value per row, or None; out may be x."""
    f, dev = "zero_layer_norm", x.get_device()
    n, d, x_stride = _rows(x, "x", f)
    m, e, out_stride = _rows(out, "out", f)
    if (m, e) != (n, d) or out.dtype != x.dtype:
        _refuse(_SIZE, f, f"out {tuple(out.shape)} {out.dtype} is not x {tuple(x.shape)} {x.dtype}")
    if out.get_device() != dev or dev < 0:
        _here(out, "out", f, dev)
    wb = _vector(weight, d, _ELEM, "weight", f, dev)
    bb = _vector(bias, d, _ELEM, "bias", f, dev)
    if wb and bb and wb != bb:
        _refuse(_INVALID, f, "weight and bias are of different types")
    _vector(mean, n, _F32, "mean", f, dev)
    _vector(rstd, n, _F32, "rstd", f, dev)
    _check(load().zero_layer_norm(x.data_ptr(), _bytes(x, _ELEM, "x", f, dev), n, d, x_stride,
                                  _ptr(weight), _ptr(bias), wb or bb or 4, eps, out.data_ptr(),
                                  out_stride, _ptr(mean), _ptr(rstd), _on(dev, stream)), f)


def zero_layer_norm_grad_workspace_bytes(n_rows: int, dim: int) -> int:
    out = ctypes.c_int64(0)
    f = "zero_layer_norm_grad_workspace_bytes"
    _check(load().zero_layer_norm_grad_workspace_bytes(n_rows, dim, ctypes.byref(out)), f)
    return int(out.value)


def zero_layer_norm_grad(grad_out, x, weight, mean, rstd, grad_x, grad_weight=None,
                         grad_bias=None, workspace=None, workspace_bytes: int = 0, stream=None):
    """Gradients of zero_layer_norm from its mean and rstd.

    grad_x may be grad_out or x; grad_weight, grad_bias: (dim,) of the
    weight's type, or None; workspace: device buffer of at least
    zero_layer_norm_grad_workspace_bytes(rows, dim) bytes."""
    f, dev = "zero_layer_norm_grad", x.get_device()
    n, d, x_stride = _rows(x, "x", f)
    my, ey, grad_out_stride = _rows(grad_out, "grad_out", f)
    mx, ex, grad_x_stride = _rows(grad_x, "grad_x", f)
    if (my, ey) != (n, d) or (mx, ex) != (n, d):
        _refuse(_SIZE, f, f"grad_out {tuple(grad_out.shape)} and grad_x {tuple(grad_x.shape)} "
                f"are not of x's shape {tuple(x.shape)}")
    if grad_out.dtype != x.dtype or grad_x.dtype != x.dtype:
        _refuse(_INVALID, f, "grad_out, x and grad_x are of different types")
    if grad_out.get_device() != dev or dev < 0:
        _here(grad_out, "grad_out", f, dev)
    if grad_x.get_device() != dev or dev < 0:
        _here(grad_x, "grad_x", f, dev)
    sizes = {b for b in (_vector(weight, d, _ELEM, "weight", f, dev),
                         _vector(grad_weight, d, _ELEM, "grad_weight", f, dev),
                         _vector(grad_bias, d, _ELEM, "grad_bias", f, dev)) if b}
    if len(sizes) > 1:
        _refuse(_INVALID, f, "weight, grad_weight and grad_bias are of different types")
    _vector(mean, n, _F32, "mean", f, dev)
    _vector(rstd, n, _F32, "rstd", f, dev)
    _check(load().zero_layer_norm_grad(
        grad_out.data_ptr(), x.data_ptr(), _bytes(x, _ELEM, "x", f, dev), n, d, grad_out_stride,
        x_stride, _ptr(weight), sizes.pop() if sizes else 4, _ptr(mean), _ptr(rstd),
        grad_x.data_ptr(), grad_x_stride, _ptr(grad_weight), _ptr(grad_bias),
        _workspace(workspace, workspace_bytes, f, dev), workspace_bytes, _on(dev, stream)), f)


def _teacher(ids, teacher, n: int, func: str, device: int):
    if ids.shape != teacher.shape or ids.dim() == 0 or not ids.is_contiguous() or \
            not teacher.is_contiguous():
        _refuse(_SIZE, func, f"teacher_ids {tuple(ids.shape)} and teacher_logits "
                f"{tuple(teacher.shape)} are not contiguous arrays of one shape")
    top = ids.shape[-1]
    if ids.numel() != n * top:
        _refuse(_SIZE, func, f"teacher_ids {tuple(ids.shape)}: {n} rows are needed")
    _bytes(ids, _I32, "teacher_ids", func, device)
    return top, _bytes(teacher, _ELEM, "teacher_logits", func, device)


def zero_distill_loss(logits, teacher_ids, teacher_logits, weights, temperature: float, loss,
                      stream=None):
    """Per-row distillation loss from the teacher's top entries:
    loss = weight * T^2 * sum_k p_k (log p_k - log q[id_k]), p the softmax of
    the entries / T, q that of the whole row / T.

    teacher_ids (int32) and teacher_logits: (rows, top); entries with an id
    outside [0, vocab) are absent; weights: fp32 (rows,) or None; loss: fp32
    (rows,)."""
    f, dev = "zero_distill_loss", logits.get_device()
    n, vocab, stride = _rows(logits, "logits", f)
    top, tb = _teacher(teacher_ids, teacher_logits, n, f, dev)
    _vector(weights, n, _F32, "weights", f, dev)
    _vector(loss, n, _F32, "loss", f, dev)
    _check(load().zero_distill_loss(
        logits.data_ptr(), _bytes(logits, _ELEM, "logits", f, dev), n, vocab, stride,
        teacher_ids.data_ptr(), teacher_logits.data_ptr(), tb, top, _ptr(weights), temperature,
        _ptr(loss), _on(dev, stream)), f)


def zero_distill_loss_grad(logits, teacher_ids, teacher_logits, weights, temperature: float, loss,
                           grad_logits, stream=None):
    """zero_distill_loss and its gradient with respect to the logits, in one
    call; grad_logits may be logits."""
    f, dev = "zero_distill_loss_grad", logits.get_device()
    n, vocab, stride = _rows(logits, "logits", f)
    m, v, grad_stride = _rows(grad_logits, "grad_logits", f)
    if (m, v) != (n, vocab):
        _refuse(_SIZE, f, f"grad_logits {tuple(grad_logits.shape)} is not of logits' shape "
                f"{tuple(logits.shape)}")
    if grad_logits.dtype != logits.dtype:
        _refuse(_INVALID, f, "grad_logits is not of logits' type")
    if grad_logits.get_device() != dev or dev < 0:
        _here(grad_logits, "grad_logits", f, dev)
    top, tb = _teacher(teacher_ids, teacher_logits, n, f, dev)
    _vector(weights, n, _F32, "weights", f, dev)
    _vector(loss, n, _F32, "loss", f, dev)
    _check(load().zero_distill_loss_grad(
        logits.data_ptr(), _bytes(logits, _ELEM, "logits", f, dev), n, vocab, stride,
        teacher_ids.data_ptr(), teacher_logits.data_ptr(), tb, top, _ptr(weights), temperature,
        _ptr(loss), _ptr(grad_logits), grad_stride, _on(dev, stream)), f)
