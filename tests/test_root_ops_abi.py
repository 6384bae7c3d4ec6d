"""What the operators around the root unit refuse, before anything is
launched: the C ABI's own checks with fake addresses that are never
dereferenced, and the binding's checks of shapes and types."""
import ctypes

import pytest
import torch

import fsdp_sharded_mixed_flatten_gb300 as zf

A = [0x100000 * (i + 1) for i in range(12)]       # fake, aligned addresses


@pytest.fixture(scope="module")
def lib():
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    return zf.load()


def _embed(lib, **o):
    a = dict(ids=A[0], idb=4, n=10, w=A[1], wb=2, v=50, d=8, scale=1.0, out=A[2], ob=2, s=8)
    a.update(o)
    return lib.zero_embedding(a["ids"], a["idb"], a["n"], a["w"], a["wb"], a["v"], a["d"],
                              a["scale"], a["out"], a["ob"], a["s"], None)


def _embed_grad(lib, **o):
    a = dict(ids=A[0], idb=4, n=10, g=A[1], gb=2, s=8, scale=1.0, w=A[2], wb=2, v=50, d=8, acc=0,
             ws=A[3], wsb=1 << 30)
    a.update(o)
    return lib.zero_embedding_grad(a["ids"], a["idb"], a["n"], a["g"], a["gb"], a["s"], a["scale"],
                                   a["w"], a["wb"], a["v"], a["d"], a["acc"], a["ws"], a["wsb"],
                                   None)


def _norm(lib, **o):
    a = dict(x=A[0], b=2, n=4, d=16, xs=16, w=A[1], bias=A[2], pb=2, eps=1e-5, out=A[3], os=16,
             mean=A[4], rstd=A[5])
    a.update(o)
    return lib.zero_layer_norm(a["x"], a["b"], a["n"], a["d"], a["xs"], a["w"], a["bias"], a["pb"],
                               a["eps"], a["out"], a["os"], a["mean"], a["rstd"], None)


def _norm_grad(lib, **o):
    a = dict(g=A[0], x=A[1], b=2, n=4, d=16, gs=16, xs=16, w=A[2], pb=2, mean=A[3], rstd=A[4],
             dx=A[5], dxs=16, dw=A[6], db=A[7], ws=A[8], wsb=1 << 30)
    a.update(o)
    return lib.zero_layer_norm_grad(a["g"], a["x"], a["b"], a["n"], a["d"], a["gs"], a["xs"],
                                    a["w"], a["pb"], a["mean"], a["rstd"], a["dx"], a["dxs"],
                                    a["dw"], a["db"], a["ws"], a["wsb"], None)


def _distill(lib, **o):
    a = dict(z=A[0], b=2, n=4, v=100, s=100, ids=A[1], t=A[2], tb=4, k=8, w=A[3], tau=1.0,
             loss=A[4], dz=A[5], ds=100)
    a.update(o)
    return lib.zero_distill_loss_grad(a["z"], a["b"], a["n"], a["v"], a["s"], a["ids"], a["t"],
                                      a["tb"], a["k"], a["w"], a["tau"], a["loss"], a["dz"],
                                      a["ds"], None)


INVALID, MISALIGNED, SIZE = -1, -2, -3
MANY = 20_000                     # tokens whose gradient needs a workspace
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("call,over,code", [
    (_embed, dict(ids=None), INVALID), (_embed, dict(w=None), INVALID),
    (_embed, dict(out=None), INVALID), (_embed, dict(idb=2), INVALID),
    (_embed, dict(wb=1), INVALID), (_embed, dict(ob=8), INVALID), (_embed, dict(n=-1), INVALID),
    (_embed, dict(v=0), INVALID), (_embed, dict(d=0), INVALID), (_embed, dict(scale=NAN), INVALID),
    (_embed, dict(s=7), SIZE), (_embed, dict(v=2 ** 31), SIZE), (_embed, dict(n=2 ** 31), SIZE),
    (_embed, dict(ids=A[0] + 2), MISALIGNED), (_embed, dict(w=A[1] + 1), MISALIGNED),
    (_embed, dict(idb=8, ids=A[0] + 4), MISALIGNED),
    (_embed, dict(ob=4, out=A[2] + 2), MISALIGNED), (_embed, dict(s=2 ** 62), SIZE),
    (_embed_grad, dict(g=None), INVALID), (_embed_grad, dict(w=None), INVALID),
    (_embed_grad, dict(acc=2), INVALID), (_embed_grad, dict(n=MANY, ws=None), INVALID),
    (_embed_grad, dict(n=MANY, ws=A[3] + 8), MISALIGNED), (_embed_grad, dict(n=MANY, wsb=16), SIZE),
    (_embed_grad, dict(s=4), SIZE), (_embed_grad, dict(scale=INF), INVALID),
    (_embed_grad, dict(d=2 ** 28, s=2 ** 28), SIZE),
    (_norm, dict(x=None), INVALID), (_norm, dict(out=None), INVALID), (_norm, dict(d=0), INVALID),
    (_norm, dict(n=-2), INVALID), (_norm, dict(b=8), INVALID), (_norm, dict(pb=3), INVALID),
    (_norm, dict(eps=-1.0), INVALID), (_norm, dict(eps=NAN), INVALID),
    (_norm, dict(d=16385, xs=16385, os=16385), SIZE), (_norm, dict(xs=15), SIZE),
    (_norm, dict(os=15), SIZE), (_norm, dict(w=A[1] + 1), MISALIGNED),
    (_norm, dict(mean=A[4] + 2), MISALIGNED),
    (_norm_grad, dict(g=None), INVALID), (_norm_grad, dict(mean=None), INVALID),
    (_norm_grad, dict(rstd=None), INVALID), (_norm_grad, dict(dx=None), INVALID),
    (_norm_grad, dict(ws=None), INVALID), (_norm_grad, dict(wsb=0), SIZE),
    (_norm_grad, dict(ws=A[8] + 4), MISALIGNED), (_norm_grad, dict(dxs=3), SIZE),
    (_norm_grad, dict(pb=4, dw=A[6] + 2), MISALIGNED),
    (_distill, dict(z=None), INVALID), (_distill, dict(ids=None), INVALID),
    (_distill, dict(t=None), INVALID), (_distill, dict(loss=None), INVALID),
    (_distill, dict(dz=None), INVALID), (_distill, dict(v=0), INVALID),
    (_distill, dict(k=0), INVALID), (_distill, dict(k=1025), SIZE), (_distill, dict(tau=0.0), INVALID),
    (_distill, dict(tau=-1.0), INVALID), (_distill, dict(tau=NAN), INVALID),
    (_distill, dict(tau=INF), INVALID), (_distill, dict(tau=1e-45), INVALID),
    (_distill, dict(tau=1e30), INVALID), (_distill, dict(s=99), SIZE), (_distill, dict(ds=99), SIZE),
    (_distill, dict(dz=A[0], ds=104), SIZE), (_distill, dict(w=A[3] + 2), MISALIGNED),
    (_distill, dict(tb=2, b=3), INVALID), (_distill, dict(b=4, z=A[0] + 2), MISALIGNED),
])
def test_refused_by_the_library(lib, call, over, code):
    assert call(lib, **over) == code, zf.zero_last_error()
    assert zf.zero_last_error() != ""


def test_workspace_sizes(lib):
    for d in (1, 255, 256, 257, 4096):
        for n in (16385, MANY, 2 ** 20):
            assert zf.zero_embedding_grad_workspace_bytes(n, 1000, d) >= 16 * n + n // 16 * d * 4
        for n in (0, 1, 4096):        # few tokens take one launch without
            assert zf.zero_embedding_grad_workspace_bytes(n, 1000, d) == 0
    out = ctypes.c_int64(0)
    assert lib.zero_embedding_grad_workspace_bytes(1, 0, 8, ctypes.byref(out)) == INVALID
    assert lib.zero_embedding_grad_workspace_bytes(1, 8, 8, None) == INVALID
    assert lib.zero_layer_norm_grad_workspace_bytes(1, 16385, ctypes.byref(out)) == SIZE
    assert lib.zero_layer_norm_grad_workspace_bytes(-1, 8, ctypes.byref(out)) == INVALID


def test_injected_failure(lib, monkeypatch):
    for call, label in ((_embed, "embedding launch"), (_embed_grad, "embedding gradient launch"),
                        (_norm, "layer norm launch"), (_norm_grad, "layer norm gradient launch"),
                        (_distill, "distillation loss")):
        monkeypatch.setenv("ZERO_INJECT_FAILURE", label)
        assert call(lib) == -4
        assert label in zf.zero_last_error() and "injected failure" in zf.zero_last_error()


class _Cuda(torch.Tensor):
    """A CPU tensor that says it is on the GPU: the shape checks come first."""
    @property
    def is_cuda(self):
        return True


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)


def _refused(code, fn, *args, **kw):
    with pytest.raises(zf.ZeroError) as ei:
        fn(*args, stream=0, **kw)
    assert ei.value.code == code, ei.value


def test_refused_by_the_binding(lib):
    ids = _t(6, dtype=torch.int32)
    w, out = _t(10, 4), _t(6, 4)
    _refused(SIZE, zf.zero_embedding, ids, w, _t(5, 4))
    _refused(SIZE, zf.zero_embedding, ids, w, _t(6, 3))
    _refused(SIZE, zf.zero_embedding, ids, _t(10, 8)[:, :4], out)
    _refused(SIZE, zf.zero_embedding, ids, w, _t(4, 6).t())
    _refused(SIZE, zf.zero_embedding, _t(12, dtype=torch.int32)[::2], w, out)
    _refused(INVALID, zf.zero_embedding, _t(6), w, out)
    _refused(INVALID, zf.zero_embedding, ids, _t(10, 4, dtype=torch.float16), out)
    _refused(INVALID, zf.zero_embedding, ids, w, torch.zeros(6, 4))        # not on the GPU
    _refused(SIZE, zf.zero_embedding_grad, ids, _t(5, 4), w)
    many = _t(MANY, dtype=torch.int32)
    _refused(INVALID, zf.zero_embedding_grad, many, _t(MANY, 4), w)         # no workspace
    x, stat, vec = _t(6, 4), _t(6), _t(4)
    _refused(SIZE, zf.zero_layer_norm, x, vec, vec, 1e-5, _t(6, 5))
    _refused(SIZE, zf.zero_layer_norm, x, _t(5), vec, 1e-5, x)
    _refused(SIZE, zf.zero_layer_norm, x, vec, vec, 1e-5, x, _t(5), stat)
    _refused(INVALID, zf.zero_layer_norm, x, vec, _t(4, dtype=torch.bfloat16), 1e-5, x)
    _refused(INVALID, zf.zero_layer_norm, x, vec, vec, 1e-5, x, stat.double(), stat)
    _refused(SIZE, zf.zero_layer_norm, _t(2, 5, 3, 4).transpose(1, 2), vec, vec, 1e-5, x)
    _refused(SIZE, zf.zero_layer_norm_grad, x, _t(6, 5), None, stat, stat, x)
    _refused(INVALID, zf.zero_layer_norm_grad, x, _t(6, 4, dtype=torch.bfloat16), None, stat, stat,
             x)
    _refused(INVALID, zf.zero_layer_norm_grad, x, x, vec, stat, stat, x,
             _t(4, dtype=torch.bfloat16))
    z, k, t = _t(6, 30), _t(6, 3, dtype=torch.int32), _t(6, 3)
    _refused(SIZE, zf.zero_distill_loss, z, k, _t(6, 4), None, 1.0, stat)
    _refused(SIZE, zf.zero_distill_loss, z, _t(5, 3, dtype=torch.int32), _t(5, 3), None, 1.0, stat)
    _refused(INVALID, zf.zero_distill_loss, z, k.long(), t, None, 1.0, stat)
    _refused(SIZE, zf.zero_distill_loss, z, k, t, _t(5), 1.0, stat)
    _refused(INVALID, zf.zero_distill_loss, z, k, t, None, 0.0, stat)
    _refused(SIZE, zf.zero_distill_loss_grad, z, k, t, None, 1.0, stat, _t(6, 29))
    _refused(INVALID, zf.zero_distill_loss_grad, z, k, t, None, 1.0, stat,
             _t(6, 30, dtype=torch.bfloat16))
