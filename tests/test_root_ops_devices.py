"""What the binding refuses because a tensor is not where it has to be: on the
host, on another GPU than the rest, or a workspace shorter than its stated
bytes.  Nothing is launched."""
import pytest
import torch

import fsdp_sharded_mixed_flatten_gb300 as zf

INVALID, SIZE = -1, -3
F32, I32 = torch.float32, torch.int32


class _Gpu0(torch.Tensor):
    """A CPU tensor that says it is on a GPU: these checks come before any use."""
    INDEX = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.INDEX


class _Gpu1(_Gpu0):
    INDEX = 1


@pytest.fixture(autouse=True)
def _nothing_runs(monkeypatch):
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")


def _t(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Gpu0)


def _calls():
    """Every call with its tensors by name, which fit but for what a test changes."""
    x, y, dx, vec, stat = _t(6, 4), _t(6, 4), _t(6, 4), _t(4), _t(6)
    ids, w, out, ws = _t(6, dtype=I32), _t(10, 4), _t(6, 4), _t(1 << 20, dtype=torch.uint8)
    z, tid, t, loss = _t(6, 30), _t(6, 3, dtype=I32), _t(6, 3), _t(6)
    return {
        "embedding": (lambda ids, weight, out: zf.zero_embedding(ids, weight, out, stream=0),
                      dict(ids=ids, weight=w, out=out)),
        "embedding_grad": (lambda ids, grad_out, grad_weight, workspace: zf.zero_embedding_grad(
            ids, grad_out, grad_weight, 1.0, False, workspace, 1 << 20, stream=0),
            dict(ids=ids, grad_out=out, grad_weight=w, workspace=ws)),
        "layer_norm": (lambda x, weight, bias, out, mean, rstd: zf.zero_layer_norm(
            x, weight, bias, 1e-5, out, mean, rstd, stream=0),
            dict(x=x, weight=vec, bias=vec, out=y, mean=stat, rstd=stat)),
        "layer_norm_grad": (lambda grad_out, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                            workspace: zf.zero_layer_norm_grad(
                                grad_out, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                                workspace, 1 << 20, stream=0),
                            dict(grad_out=y, x=x, weight=vec, mean=stat, rstd=stat, grad_x=dx,
                                 grad_weight=vec, grad_bias=vec, workspace=ws)),
        "distill_loss": (lambda logits, ids, teacher, weights, loss: zf.zero_distill_loss(
            logits, ids, teacher, weights, 1.0, loss, stream=0),
            dict(logits=z, ids=tid, teacher=t, weights=stat, loss=loss)),
        "distill_loss_grad": (lambda logits, ids, teacher, weights, loss, grad_logits:
                              zf.zero_distill_loss_grad(logits, ids, teacher, weights, 1.0, loss,
                                                        grad_logits, stream=0),
                              dict(logits=z, ids=tid, teacher=t, weights=stat, loss=loss,
                                   grad_logits=_t(6, 30))),
    }


def _code(call, tensors):
    with pytest.raises(zf.ZeroError) as ei:
        call(**tensors)
    return ei.value.code


EVERY = [(c, name) for c, (_, tensors) in _calls().items() for name in tensors]


@pytest.mark.parametrize("call", sorted(_calls()))
def test_what_fits_reaches_the_launch(call):
    fn, tensors = _calls()[call]
    assert _code(fn, tensors) == -4


@pytest.mark.parametrize("call,name", EVERY)
def test_a_host_tensor_is_refused(call, name):
    fn, tensors = _calls()[call]
    tensors[name] = torch.zeros(tensors[name].shape, dtype=tensors[name].dtype)
    assert _code(fn, tensors) == INVALID


@pytest.mark.parametrize("call,name", EVERY)
def test_a_tensor_of_another_gpu_is_refused(call, name):
    fn, tensors = _calls()[call]
    t = tensors[name]
    tensors[name] = torch.zeros(t.shape, dtype=t.dtype).as_subclass(_Gpu1)
    assert _code(fn, tensors) == INVALID


@pytest.mark.parametrize("call", ["embedding_grad", "layer_norm_grad"])
def test_a_short_workspace_is_refused(call):
    fn, tensors = _calls()[call]
    for ws in (_t((1 << 20) - 1, dtype=torch.uint8), _t(1 << 21, dtype=torch.uint8)[::2],
               _t((1 << 18) - 1)):
        assert _code(fn, dict(tensors, workspace=ws)) == SIZE
    assert _code(fn, dict(tensors, workspace=_t(1 << 18))) == -4      # by its bytes
