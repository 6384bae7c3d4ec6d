"""What the root-mean-square norm and the rows in 8 bits refuse, before anything
is launched: the C ABI's own checks with fake addresses that are never
dereferenced, and the binding's checks of shapes and types."""
import ctypes

import pytest
import torch

import fsdp_sharded_mixed_flatten_gb300 as zf

A = [0x100000 * (i + 1) for i in range(16)]       # fake, aligned addresses
INVALID, MISALIGNED, SIZE = -1, -2, -3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    return zf.load()


def _pack(lib, **o):
    a = dict(x=A[0], b=2, n=4, d=200, xs=200, c=A[1], cs=200, s=A[2])
    a.update(o)
    return lib.zero_pack_rows(a["x"], a["b"], a["n"], a["d"], a["xs"], a["c"], a["cs"], a["s"],
                              None)


def _unpack(lib, **o):
    a = dict(x=A[0], b=2, n=4, d=200, xs=200, c=A[1], cs=200, s=A[2])
    a.update(o)
    return lib.zero_unpack_rows(a["c"], a["cs"], a["s"], a["n"], a["d"], a["x"], a["b"], a["xs"],
                                None)


def _norm(lib, **o):
    a = dict(x=A[0], r=A[1], b=2, n=4, d=16, xs=16, rs=16, w=A[2], pb=2, eps=1e-5, o=A[3], os=16,
             t=A[4], ts=16, o8=A[5], o8s=16, o8c=A[6], t8=A[7], t8s=16, t8c=A[8], rstd=A[9])
    a.update(o)
    return lib.zero_rms_norm(a["x"], a["r"], a["b"], a["n"], a["d"], a["xs"], a["rs"], a["w"],
                             a["pb"], a["eps"], a["o"], a["os"], a["t"], a["ts"], a["o8"],
                             a["o8s"], a["o8c"], a["t8"], a["t8s"], a["t8c"], a["rstd"], None)


def _norm_grad(lib, **o):
    a = dict(g=A[0], t=A[1], t8=None, t8s=16, t8c=None, b=2, n=4, d=16, gs=16, ts=16, w=A[2],
             pb=2, rstd=A[3], gt=A[4], gts=16, dx=A[5], dxs=16, dw=A[6], o=A[7], os=16, ws=A[8],
             wsb=1 << 30)
    a.update(o)
    return lib.zero_rms_norm_grad(a["g"], a["t"], a["t8"], a["t8s"], a["t8c"], a["b"], a["n"],
                                  a["d"], a["gs"], a["ts"], a["w"], a["pb"], a["rstd"], a["gt"],
                                  a["gts"], a["dx"], a["dxs"], a["dw"], a["o"], a["os"], a["ws"],
                                  a["wsb"], None)


@pytest.mark.parametrize("call,over,code", [
    (_pack, dict(x=None), INVALID), (_pack, dict(c=None), INVALID), (_pack, dict(s=None), INVALID),
    (_pack, dict(b=1), INVALID), (_pack, dict(n=-1), INVALID), (_pack, dict(d=0), INVALID),
    (_pack, dict(xs=199), SIZE), (_pack, dict(cs=199), SIZE), (_pack, dict(x=A[0] + 1), MISALIGNED),
    (_pack, dict(s=A[2] + 2), MISALIGNED), (_pack, dict(n=2 ** 31), SIZE),
    (_pack, dict(n=2 ** 30, d=4096, xs=4096, cs=4096), SIZE), (_pack, dict(xs=2 ** 62), SIZE),
    (_unpack, dict(x=None), INVALID), (_unpack, dict(c=None), INVALID),
    (_unpack, dict(s=None), INVALID), (_unpack, dict(b=3), INVALID), (_unpack, dict(d=-1), INVALID),
    (_unpack, dict(xs=4), SIZE), (_unpack, dict(cs=4), SIZE),
    (_unpack, dict(b=4, x=A[0] + 2), MISALIGNED),
    (_norm, dict(x=None), INVALID), (_norm, dict(d=0), INVALID), (_norm, dict(n=-2), INVALID),
    (_norm, dict(b=8), INVALID), (_norm, dict(pb=3), INVALID), (_norm, dict(eps=-1.0), INVALID),
    (_norm, dict(eps=NAN), INVALID), (_norm, dict(eps=INF), INVALID), (_norm, dict(xs=15), SIZE),
    (_norm, dict(rs=15), SIZE), (_norm, dict(os=15), SIZE), (_norm, dict(ts=15), SIZE),
    (_norm, dict(o8s=15), SIZE), (_norm, dict(t8s=15), SIZE), (_norm, dict(o8c=None), INVALID),
    (_norm, dict(o8=None), INVALID), (_norm, dict(t8c=None), INVALID),
    (_norm, dict(t8=None), INVALID), (_norm, dict(t8c=A[8] + 1), MISALIGNED),
    (_norm, dict(o=A[4]), INVALID), (_norm, dict(o=A[1]), INVALID),
    (_norm, dict(t=A[0], ts=24), SIZE), (_norm, dict(t=A[1], rs=24), SIZE),
    (_norm, dict(o=A[0], os=24), SIZE), (_norm, dict(w=A[2] + 1), MISALIGNED),
    (_norm, dict(rstd=A[9] + 2), MISALIGNED), (_norm, dict(r=A[1] + 1), MISALIGNED),
    (_norm, dict(d=16385, xs=16385, rs=16385, os=16385, ts=16385, o8s=16385, t8s=16385), SIZE),
    (_norm_grad, dict(g=None), INVALID), (_norm_grad, dict(t=None), INVALID),
    (_norm_grad, dict(t8=A[9], t8c=A[10]), INVALID), (_norm_grad, dict(rstd=None), INVALID),
    (_norm_grad, dict(t=None, t8=A[9]), INVALID), (_norm_grad, dict(dx=None), INVALID),
    (_norm_grad, dict(t=None, t8=A[9], t8c=A[10], t8s=3), SIZE),
    (_norm_grad, dict(ws=None), INVALID), (_norm_grad, dict(ws=A[8] + 4), MISALIGNED),
    (_norm_grad, dict(wsb=0), SIZE), (_norm_grad, dict(gs=3), SIZE), (_norm_grad, dict(dxs=3), SIZE),
    (_norm_grad, dict(gts=3), SIZE), (_norm_grad, dict(os=3), SIZE),
    (_norm_grad, dict(dx=A[0], dxs=24), SIZE), (_norm_grad, dict(dx=A[1], dxs=24), SIZE),
    (_norm_grad, dict(dx=A[4], dxs=24), SIZE), (_norm_grad, dict(o=A[5]), INVALID),
    (_norm_grad, dict(o=A[0]), INVALID), (_norm_grad, dict(o=A[1]), INVALID),
    (_norm_grad, dict(pb=4, dw=A[6] + 2), MISALIGNED),
])
def test_refused_by_the_library(lib, call, over, code):
    assert call(lib, **over) == code, zf.zero_last_error()
    assert zf.zero_last_error() != ""


def test_workspace_sizes(lib):
    for n in (0, 1, 1000, 2 ** 20):
        for d in (1, 257, 4096, 16384):
            assert zf.zero_rms_norm_grad_workspace_bytes(n, d) >= 4 * d
    out = ctypes.c_int64(0)
    assert lib.zero_rms_norm_grad_workspace_bytes(1, 16385, ctypes.byref(out)) == SIZE
    assert lib.zero_rms_norm_grad_workspace_bytes(-1, 8, ctypes.byref(out)) == INVALID
    assert lib.zero_rms_norm_grad_workspace_bytes(1, 8, None) == INVALID


def test_injected_failure(lib, monkeypatch):
    for call, label in ((_pack, "row packing launch"), (_unpack, "row unpacking launch"),
                        (_norm, "rms norm launch"), (_norm_grad, "rms norm gradient launch")):
        monkeypatch.setenv("ZERO_INJECT_FAILURE", label)
        assert call(lib) == -4
        assert label in zf.zero_last_error() and "injected failure" in zf.zero_last_error()


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


def _eight(n, d, dtype=torch.uint8):
    return (_t(n, d, dtype=dtype), _t(n, (d + 127) // 128))


def _refused(code, fn, *args, **kw):
    with pytest.raises(zf.ZeroError) as ei:
        fn(*args, stream=0, **kw)
    assert ei.value.code == code, ei.value


def test_refused_by_the_binding(lib, monkeypatch):
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")
    x, y, vec, stat, p = _t(6, 130), _t(6, 130), _t(130), _t(6), _eight(6, 130)
    _refused(SIZE, zf.zero_pack_rows, x, _eight(5, 130))
    _refused(SIZE, zf.zero_pack_rows, x, _eight(6, 131))
    _refused(SIZE, zf.zero_pack_rows, x, (p[0], _t(6, 1)))
    _refused(SIZE, zf.zero_pack_rows, x, (p[0], _t(2, 6).t()))
    _refused(INVALID, zf.zero_pack_rows, x, (p[0].float(), p[1]))
    _refused(INVALID, zf.zero_pack_rows, x, (p[0], p[1].double()))
    _refused(INVALID, zf.zero_pack_rows, x, p[0])
    _refused(INVALID, zf.zero_pack_rows, x.half(), p)
    _refused(INVALID, zf.zero_unpack_rows, p, x.double())
    _refused(SIZE, zf.zero_unpack_rows, p, _t(6, 129))
    _refused(SIZE, zf.zero_rms_norm, x, None, _t(129), 1e-5, y)
    _refused(SIZE, zf.zero_rms_norm, x, _t(5, 130), vec, 1e-5, y)
    _refused(INVALID, zf.zero_rms_norm, x, y.bfloat16(), vec, 1e-5, y)
    _refused(INVALID, zf.zero_rms_norm, x, None, vec.half(), 1e-5, y)
    _refused(INVALID, zf.zero_rms_norm, x, None, vec, 1e-5, y.bfloat16())
    _refused(SIZE, zf.zero_rms_norm, x, None, vec, 1e-5, y, None, _t(5))
    _refused(SIZE, zf.zero_rms_norm, x, None, vec, 1e-5, _t(130, 6).t())
    _refused(INVALID, zf.zero_rms_norm_grad, x, None, vec, stat, y)
    _refused(SIZE, zf.zero_rms_norm_grad, x, _eight(6, 129), vec, stat, y)
    _refused(SIZE, zf.zero_rms_norm_grad, x, _t(6, 129), vec, stat, y)
    _refused(INVALID, zf.zero_rms_norm_grad, x, y, vec, stat, None)
    _refused(INVALID, zf.zero_rms_norm_grad, x, y, vec, stat, y, vec.bfloat16())
    _refused(INVALID, zf.zero_rms_norm_grad, x, y, vec, stat, y, vec)       # no workspace
    _refused(SIZE, zf.zero_rms_norm_grad, x, y, vec, stat, y, vec, None, None, _t(4), 1 << 20)


@pytest.mark.parametrize("elsewhere", [torch.Tensor, _Gpu1])
def test_tensors_elsewhere_are_refused(lib, monkeypatch, elsewhere):
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")
    codes, scales = _eight(6, 130)
    pack = dict(x=_t(6, 130), codes=codes, scales=scales)
    norm = dict(x=_t(6, 130), residual=_t(6, 130), weight=_t(130), out=_t(6, 130),
                total=_t(6, 130), rstd=_t(6), codes=codes, scales=scales)
    grad = dict(grad_out=_t(6, 130), total=_t(6, 130), weight=_t(130), rstd=_t(6),
                grad_x=_t(6, 130), grad_weight=_t(130), grad_total=_t(6, 130), out=_t(6, 130),
                workspace=_t(1 << 20, dtype=torch.uint8))
    calls = [
        (lambda x, codes, scales: zf.zero_pack_rows(x, (codes, scales), stream=0), pack),
        (lambda x, codes, scales: zf.zero_unpack_rows((codes, scales), x, stream=0), pack),
        (lambda codes, scales, x, residual, weight, out, total, rstd: zf.zero_rms_norm(
            x, residual, weight, 1e-5, out, total, rstd, (codes, scales), (codes, scales),
            stream=0), norm),
        (lambda **k: zf.zero_rms_norm_grad(**k, workspace_bytes=1 << 20, stream=0), grad),
        (lambda codes, scales, total, **k: zf.zero_rms_norm_grad(
            total=(codes, scales), **k, workspace_bytes=1 << 20, stream=0),
         dict(grad, codes=codes, scales=scales)),
    ]
    for call, tensors in calls:
        with pytest.raises(zf.ZeroError) as ei:
            call(**tensors)
        assert ei.value.code == -4, ei.value             # all well: only the launch is refused
        for name in tensors:
            if name == "total" and "codes" in tensors and "grad_out" in tensors:
                continue
            moved = dict(tensors)
            moved[name] = tensors[name].as_subclass(torch.Tensor)
            if elsewhere is not torch.Tensor:
                moved[name] = moved[name].as_subclass(elsewhere)
            with pytest.raises(zf.ZeroError) as ei:
                call(**moved)
            assert ei.value.code == INVALID and "on one GPU" in str(ei.value), (name, ei.value)
