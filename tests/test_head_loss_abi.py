"""What the head's cross entropy refuses, before anything is launched: the C ABI's
own checks with fake addresses that are never dereferenced, and the binding's
checks of shapes, types and places."""
import ctypes

import pytest
import torch

import fsdp_sharded_mixed_flatten_gb300 as zf

A = [0x100000 * (i + 1) for i in range(12)]       # fake, aligned addresses
INVALID, MISALIGNED, SIZE = -1, -2, -3
TOKENS, VOCAB, DIM = zf.ZERO_MAX_HEAD_TOKENS, zf.ZERO_MAX_HEAD_VOCAB, zf.ZERO_MAX_HEAD_DIM


@pytest.fixture(scope="module")
def lib():
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    return zf.load()


def _loss(lib, **o):
    a = dict(h=A[0], n=4, d=16, hs=16, w=A[1], v=50, y=A[2], yb=8, loss=A[3], lse=A[4], ws=A[5],
             wsb=1 << 40)
    a.update(o)
    return lib.zero_head_loss(a["h"], a["n"], a["d"], a["hs"], a["w"], a["v"], a["y"], a["yb"],
                              a["loss"], a["lse"], a["ws"], a["wsb"], None)


def _grad(lib, **o):
    a = dict(h=A[0], n=4, d=16, hs=16, w=A[1], v=50, y=A[2], yb=8, lse=A[3], gl=A[4], dh=A[5],
             dhs=16, dw=A[6], acc=0, ws=A[7], wsb=1 << 40)
    a.update(o)
    return lib.zero_head_loss_grad(a["h"], a["n"], a["d"], a["hs"], a["w"], a["v"], a["y"],
                                   a["yb"], a["lse"], a["gl"], a["dh"], a["dhs"], a["dw"],
                                   a["acc"], a["ws"], a["wsb"], None)


BOTH = [(dict(h=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
        (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(v=0), INVALID), (dict(yb=2), INVALID),
        (dict(hs=15), SIZE), (dict(n=TOKENS + 1), SIZE), (dict(v=VOCAB + 1), SIZE),
        (dict(d=DIM + 1, hs=DIM + 1), SIZE), (dict(hs=2 ** 62), SIZE),
        (dict(h=A[0] + 1), MISALIGNED), (dict(w=A[1] + 1), MISALIGNED),
        (dict(y=A[2] + 4), MISALIGNED), (dict(ws=None), INVALID), (dict(ws=A[5] + 8), MISALIGNED),
        (dict(wsb=1000), SIZE)]


@pytest.mark.parametrize("call,over,code", [(_loss, *b) for b in BOTH] + [(_grad, *b) for b in BOTH] + [
    (_loss, dict(loss=None), INVALID), (_loss, dict(loss=A[3] + 2), MISALIGNED),
    (_loss, dict(lse=A[4] + 2), MISALIGNED),
    (_grad, dict(lse=None), INVALID), (_grad, dict(gl=None), INVALID),
    (_grad, dict(gl=A[4] + 1), MISALIGNED), (_grad, dict(dhs=15), SIZE),
    (_grad, dict(dh=A[0], dhs=24), SIZE), (_grad, dict(dw=A[1]), INVALID),
    (_grad, dict(dw=A[6] + 1), MISALIGNED), (_grad, dict(acc=2), INVALID),
])
def test_refused_by_the_library(lib, call, over, code):
    assert call(lib, **over) == code, zf.zero_last_error()
    assert zf.zero_last_error() != ""


def test_workspaces(lib):
    for n, v, d in ((1, 1, 1), (100, 50257, 768), (8192, 131072, 4096), (TOKENS, 1000, 64)):
        some = zf.zero_head_loss_workspace_bytes(n, v, d)
        assert some >= 2 * n * d + 8 * n * ((v + 255) // 256)
        assert zf.zero_head_loss_grad_workspace_bytes(n, v, d) >= 2 * n * d + 4 * n * d
    # the logits' gradient is held in pieces: 2 GB in one
    assert zf.zero_head_loss_grad_workspace_bytes(8192, 131072, 4096) < 3 << 29
    out = ctypes.c_int64(0)
    for f in (lib.zero_head_loss_workspace_bytes, lib.zero_head_loss_grad_workspace_bytes):
        assert f(1, 8, 8, None) == INVALID
        assert f(1, 0, 8, ctypes.byref(out)) == INVALID
        assert f(1, 8, DIM + 1, ctypes.byref(out)) == SIZE


def test_nothing_to_do_is_done(lib):
    assert _loss(lib, n=0, h=None, y=None, loss=None, ws=None) == 0
    assert _grad(lib, dh=None, dw=None, ws=None) == 0
    assert _grad(lib, n=0, acc=1, ws=None) == 0


def test_injected_failure(lib, monkeypatch):
    for call, label in ((_loss, "head loss launch"), (_grad, "head rows launch")):
        monkeypatch.setenv("ZERO_INJECT_FAILURE", label)
        assert call(lib) == -4
        assert "injected failure" in zf.zero_last_error()


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


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Gpu0)


def _b(*shape):
    return _t(*shape, dtype=torch.bfloat16)


def _tensors(back):
    t = dict(hidden=_b(6, 16), table=_b(50, 16), labels=_t(6, dtype=torch.int64))
    if back:
        return dict(t, lse=_t(6), grad_loss=_t(6), grad_hidden=_b(6, 16), grad_table=_b(50, 16),
                    workspace=_t(1 << 22, dtype=torch.uint8))
    return dict(t, loss=_t(6), lse=_t(6), workspace=_t(1 << 22, dtype=torch.uint8))


CALLS = [(zf.zero_head_loss, False), (zf.zero_head_loss_grad, True)]


@pytest.mark.parametrize("fn,back", CALLS)
def test_refused_by_the_binding(lib, monkeypatch, fn, back):
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")
    wrong = [("hidden", _b(5, 16), SIZE), ("hidden", _b(6, 15), SIZE), ("hidden", _t(6, 16), INVALID),
             ("hidden", _b(16, 6).t(), SIZE), ("table", _t(50, 16), INVALID),
             ("table", _b(50, 32)[:, :16], SIZE), ("table", _b(800), SIZE),
             ("labels", _t(6), INVALID), ("labels", _t(12, dtype=torch.int64)[::2], SIZE),
             ("lse", _t(5), SIZE), ("lse", _t(6).double(), INVALID),
             ("workspace", _t(100, dtype=torch.uint8), SIZE)]
    if back:
        wrong += [("grad_loss", _t(5), SIZE), ("grad_loss", _b(6), INVALID),
                  ("grad_hidden", _b(6, 15), SIZE), ("grad_hidden", _t(6, 16), INVALID),
                  ("grad_table", _b(49, 16), SIZE), ("grad_table", _t(50, 16), INVALID)]
    else:
        wrong += [("loss", _t(5), SIZE), ("loss", _b(6), INVALID)]
    for name, t, code in wrong:
        with pytest.raises(zf.ZeroError) as ei:
            fn(**dict(_tensors(back), **{name: t}), workspace_bytes=1 << 22, stream=0)
        assert ei.value.code == code, (name, ei.value)


@pytest.mark.parametrize("elsewhere", [torch.Tensor, _Gpu1])
@pytest.mark.parametrize("fn,back", CALLS)
def test_tensors_elsewhere_are_refused(lib, monkeypatch, fn, back, elsewhere):
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")
    with pytest.raises(zf.ZeroError) as ei:
        fn(**_tensors(back), workspace_bytes=1 << 22, stream=0)
    assert ei.value.code == -4, ei.value                 # all well: only the launch is refused
    for name, t in _tensors(back).items():
        moved = t.as_subclass(torch.Tensor)
        if elsewhere is not torch.Tensor:
            moved = moved.as_subclass(elsewhere)
        with pytest.raises(zf.ZeroError) as ei:
            fn(**dict(_tensors(back), **{name: moved}), workspace_bytes=1 << 22, stream=0)
        assert ei.value.code == INVALID and "on one GPU" in str(ei.value), (name, ei.value)
