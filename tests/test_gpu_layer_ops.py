"""The root-mean-square norm and rows in 8 bits against plain 64-bit
implementations (layer_reference.py, whose bounds are derived there): every
type, odd and ragged sizes, strides and alignments, lengths of zero and one,
results in place, values at the ends of the types' ranges."""
import numpy as np
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


def _gen(*key):
    from fsdp_sharded_mixed_flatten_gb300.synthetic import seed_for
    return torch.Generator().manual_seed(seed_for("layer-ops", *key))


class Guarded:
    """A matrix of n rows in a wider buffer at an element offset, with a sentinel
    everywhere else."""

    def __init__(self, n, d, dtype, pad=0, offset=0, fill=None):
        self.bytes = torch.full(((offset + n * (d + pad) + 64) * dtype.itemsize,), 0x5A,
                                dtype=torch.uint8, device="cuda")
        base = self.bytes.view(dtype)
        self.t = base[offset:offset + n * (d + pad)].view(n, d + pad)[:, :d]
        if fill is not None:
            self.t.copy_(fill)
        mask = torch.zeros(base.shape, dtype=torch.bool, device="cuda")
        mask[offset:offset + n * (d + pad)].view(n, d + pad)[:, :d] = True
        self.outside = ~mask.repeat_interleave(dtype.itemsize)

    def check_guard(self, what):
        assert bool((self.bytes[self.outside] == 0x5A).all()), f"{what}: wrote outside its rows"


class Packed:
    def __init__(self, n, d, pad=0, offset=0):
        self.codes = Guarded(n, d, torch.uint8, pad, offset)
        self.scales = Guarded(n, (d + 127) // 128, F32, 0, offset)
        self.pair = (self.codes.t, self.scales.t)

    def numpy(self):
        return self.codes.t.cpu().numpy(), self.scales.t.cpu().numpy()

    def check(self, x, what):
        """Holds the rows of x (fp32 values), bit for bit."""
        codes, scales = L.pack(x)
        got_codes, got_scales = self.numpy()
        assert np.array_equal(got_scales, scales), f"{what}: scales"
        assert np.array_equal(got_codes, codes), f"{what}: codes"
        self.check_guard(what)

    def check_guard(self, what):
        self.codes.check_guard(what)
        self.scales.check_guard(what)


def _f32(t):
    return t.detach().cpu().float().numpy()


# rows, columns, pad columns, element offset
SHAPES = [(1, 1, 0, 0), (3, 7, 1, 1), (5, 127, 0, 0), (4, 128, 0, 0), (9, 129, 7, 0), (2, 256, 8, 8),
          (33, 770, 0, 0), (17, 1501, 3, 5), (8, 4096, 0, 0), (6, 4097, 0, 0), (5, 8192, 16, 16),
          (4, 9000, 0, 3), (3, 16384, 0, 0), (2, 16383, 1, 0)]


# ---------------------------------------------------------- rows in 8 bits ----

@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n,d,pad,offset", SHAPES + [(2, 20000, 0, 0), (700, 385, 0, 0)])
def test_pack_and_unpack(n, d, pad, offset, act):
    g = _gen("pack", n, d)
    size = torch.exp(torch.randn((n, (d + 15) // 16), generator=g) * 3).repeat_interleave(16, 1)
    x = Guarded(n, d, act, pad, offset, torch.randn((n, d), generator=g) * size[:, :d])
    p = Packed(n, d, pad, offset)
    zf.zero_pack_rows(x.t, p.pair)
    p.check(_f32(x.t), "packed")
    ref = torch.from_numpy(L.unpack(*p.numpy()))
    for out_type in (BF16, F32):
        out = Guarded(n, d, out_type, pad, offset)
        zf.zero_unpack_rows(p.pair, out.t)
        R.check(out.t, ref, 0.0, "unpacked")           # no rounding in either type
        out.check_guard("unpacked")
    big = (_f32(x.t).astype(np.float64), ref.numpy())
    step = np.repeat(p.numpy()[1].astype(np.float64), 128, 1)[:, :d] * 2.0 ** -10
    assert np.all(np.abs(big[0] - big[1]) <= np.maximum(np.abs(big[0]) * 2.0 ** -4, step))


@pytest.mark.parametrize("d", [130, 256])           # single elements, whole words
def test_pack_at_the_ends_of_the_range(d):
    inf, nan, most, low = float("inf"), float("nan"), 3.4028234663852886e38, 2.0 ** -149
    x = torch.zeros((12, d))
    x[0, :3] = torch.tensor([inf, -inf, nan])
    x[1, :3] = torch.tensor([inf, 3.0, nan])
    x[2, :4] = torch.tensor([most, -most, 1.0, 2.0 ** 127 * 1.76])
    x[3, :4] = torch.tensor([low, -low, 2.0 ** -126, 2.0 ** -135])
    x[4, :2] = torch.tensor([448.0, 1.0])           # the largest code itself
    x[5, :2] = torch.tensor([448.0001, 1.0])        # the next scale
    x[6, :2] = torch.tensor([-0.0, 0.0])
    x[7, :6] = torch.tensor([256.0, 1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10])  # ties
    x[8, :2] = torch.tensor([2.0 ** -118, 2.0 ** -117])
    x[9, 127:130] = torch.tensor([100.0, 7.0, nan])     # across the border of two blocks
    x[10, :2] = torch.tensor([2.0 ** 127 * 1.75, 1.0])
    x[11] = torch.full((d,), -3.3895313892515355e38)    # bf16's lowest
    p = Packed(12, d)
    zf.zero_pack_rows(x.cuda(), p.pair)
    p.check(x.numpy(), "packed")
    out = torch.empty((12, d), device="cuda")
    zf.zero_unpack_rows(p.pair, out)
    R.check(out, torch.from_numpy(L.unpack(*p.numpy())), 0.0, "unpacked")
    got = out.cpu()
    assert torch.isnan(got[0, :3]).all() and torch.isnan(got[1, [0, 2]]).all() and got[1, 1] == 3.0
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[10:]).all()


def test_every_code_unpacks():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(2, 1).cuda()
    scales = torch.tensor([[1.0, 0.5], [3.0, 2.0 ** -120]], device="cuda")    # any fp32 scale
    out = torch.empty((2, 256), device="cuda")
    zf.zero_unpack_rows((codes.view(torch.float8_e4m3fn), scales), out)
    ref = torch.from_numpy(L.unpack(codes.cpu().numpy(), scales.cpu().numpy()))
    R.check(out, ref, 0.0, "unpacked")


def test_unpack_beyond_32_bit_elements():
    n, d = 70_000, 32_768                                  # 2.3 G values
    codes = torch.full((n, d), 0x38, dtype=torch.uint8, device="cuda")          # 1.0
    scales = torch.ones((n, d // 128), device="cuda")
    scales[-1, -1] = 4.0
    out = torch.empty((n, d), dtype=BF16, device="cuda")
    zf.zero_unpack_rows((codes, scales), out)
    assert bool((out[-1, -128:] == 4.0).all()) and bool((out[-1, :-128] == 1.0).all())
    assert bool((out[n // 2] == 1.0).all())
    out[-2, 5] = -300.0
    codes.zero_()
    zf.zero_pack_rows(out, (codes, scales))
    back = torch.empty((3, d), dtype=BF16, device="cuda")
    zf.zero_unpack_rows((codes[-3:], scales[-3:]), back)
    assert bool((back[1, 5] == -288.0) | (back[1, 5] == -320.0) | (back[1, 5] == -304.0))
    assert bool((back[2, -128:] == 4.0).all()) and bool((back[0] == 1.0).all())


# -------------------------------------------------------------------- norm ----

def _stream(g, n, d, act):
    size = torch.rand((n, 1), generator=g) * 2 + 0.5
    return (torch.randn((n, d), generator=g) * size).to(act)


def _weight(g, d, param, offset):
    if param is None:
        return None
    flat = torch.zeros(offset + d, dtype=param, device="cuda")
    flat[offset:] = (torch.randn(d, generator=g) * 0.2 + 1.0).to(param).cuda()
    return flat[offset:]


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("param", [BF16, F32, None])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("n,d,pad,offset", SHAPES)
def test_rms_norm(n, d, pad, offset, with_residual, act, param):
    g = _gen("norm", n, d)
    x = Guarded(n, d, act, pad, offset, _stream(g, n, d, act))
    res = Guarded(n, d, act, pad, offset, _stream(g, n, d, act)) if with_residual else None
    w = _weight(g, d, param, offset)
    out, total = Guarded(n, d, act, pad, offset), Guarded(n, d, act, pad, offset)
    p_out, p_total = Packed(n, d, pad, offset), Packed(n, d, pad, offset)
    rstd = torch.zeros(n, device="cuda")
    zf.zero_rms_norm(x.t, res.t if res else None, w, 1e-5, out.t, total.t, rstd, p_out.pair,
                     p_total.pair)
    s = x.t.cpu().float()
    if res:
        s = s + res.t.cpu().float()                    # one fp32 rounding, as in the kernel
    R.check(total.t, s.to(F64), 0.0, "total")
    y, bound, r, r_bound = L.rms_norm(s.to(F64), w, 1e-5)
    R.check(out.t, y, bound, "out")
    R.check(rstd, r, r_bound, "rstd")
    p_total.check(s.numpy(), "total in 8 bits")
    if act == F32:
        p_out.check(_f32(out.t), "out in 8 bits")      # of the very values
    else:
        got = torch.from_numpy(L.unpack(*p_out.numpy()))
        assert bool(((got - y).abs() <= L.eight_bound(y, bound)).all()), "out in 8 bits"
    for m, what in ((out, "out"), (total, "total"), (p_out, "out8"), (p_total, "total8")):
        m.check_guard(what)


@pytest.mark.parametrize("act", [BF16, F32])
def test_rms_norm_of_some_results(act):
    """Each result alone is what it is among all."""
    n, d = 37, 1000
    g = _gen("some", n, d)
    x, res = _stream(g, n, d, act).cuda(), _stream(g, n, d, act).cuda()
    w = _weight(g, d, BF16, 0)

    def fresh():
        return dict(out=torch.zeros((n, d), dtype=act, device="cuda"),
                    total=torch.zeros((n, d), dtype=act, device="cuda"),
                    rstd=torch.zeros(n, device="cuda"), packed_out=Packed(n, d).pair,
                    packed_total=Packed(n, d).pair)

    everything = fresh()
    zf.zero_rms_norm(x, res, w, 1e-6, **everything)
    for name, got in fresh().items():
        zf.zero_rms_norm(x, res, w, 1e-6, **{name: got})
        want = everything[name]
        for a, b in zip(got if isinstance(got, tuple) else (got,),
                        want if isinstance(want, tuple) else (want,)):
            assert torch.equal(a, b), name
    for place in ("x", "residual"):                    # total in place, as a residual stream is
        xs, rs = x.clone(), res.clone()
        got = fresh()
        got["total"] = xs if place == "x" else rs
        zf.zero_rms_norm(xs, rs, w, 1e-6, **got)
        assert torch.equal(got["total"], everything["total"]), place
        assert torch.equal(got["out"], everything["out"]), place
    xs, got = x.clone(), fresh()
    zf.zero_rms_norm(xs, res, w, 1e-6, xs, got["total"])
    assert torch.equal(xs, everything["out"]) and torch.equal(got["total"], everything["total"])


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("param", [BF16, F32, None])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("n,d,pad,offset", SHAPES)
def test_rms_norm_grad(n, d, pad, offset, eight, act, param):
    g = _gen("norm-grad", n, d)
    x = Guarded(n, d, act, pad, offset, _stream(g, n, d, act))
    w = _weight(g, d, param, offset)
    dy = Guarded(n, d, act, pad, offset, _stream(g, n, d, act) * 0.01)
    through = Guarded(n, d, act, pad, offset, _stream(g, n, d, act) * 0.01) if n % 2 else None
    dx, again = Guarded(n, d, act, pad, offset), Guarded(n, d, act, pad, offset)
    rstd = torch.zeros(n, device="cuda")
    p = Packed(n, d, pad, offset)
    zf.zero_rms_norm(x.t, None, w, 1e-5, rstd=rstd, packed_total=p.pair)
    dw = Guarded(1, d, param or F32, 0, offset)
    nbytes = zf.zero_rms_norm_grad_workspace_bytes(n, d)
    ws = torch.full((nbytes + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    zf.zero_rms_norm_grad(dy.t, p.pair if eight else x.t, w, rstd, dx.t, dw.t[0],
                          through.t if through else None, again.t, ws, nbytes)
    s = torch.from_numpy(L.unpack(*p.numpy())) if eight else x.t.cpu().to(F64)
    ref_x, ref_w, ref_out = L.rms_norm_grad(dy.t, s, w, rstd, through.t if through else None)
    R.check(dx.t, *ref_x, "grad_x")
    R.check(dw.t[0], *ref_w, "grad_weight")
    R.check(again.t, *ref_out, "out again")
    assert bool((ws[nbytes:] == 0xA5).all()), "wrote past the workspace"
    for m, what in ((dx, "grad_x"), (dw, "grad_weight"), (again, "out again")):
        m.check_guard(what)
    # without the other results, in place
    rows = dy.t.clone() if pad == 0 else dy.t
    zf.zero_rms_norm_grad(rows, p.pair if eight else x.t, w, rstd, rows, None,
                          through.t if through else None)
    assert torch.equal(rows, dx.t)


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n,d", [(3000, 768), (2001, 1501), (1999, 4096), (20000, 96), (800, 9000),
                                 (700, 16384)])
def test_rms_norm_of_many_rows(n, d, act):
    g = _gen("many", n, d)
    x, dy = _stream(g, n, d, act).cuda(), (_stream(g, n, d, act) * 0.01).cuda()
    w = _weight(g, d, BF16, 1)
    out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    rstd = torch.zeros(n, device="cuda")
    zf.zero_rms_norm(x, None, w, 1e-5, out, rstd=rstd)
    y, bound, r, r_bound = L.rms_norm(x.cpu().to(F64), w, 1e-5)
    R.check(out, y, bound, "out")
    R.check(rstd, r, r_bound, "rstd")
    nbytes = zf.zero_rms_norm_grad_workspace_bytes(n, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    zf.zero_rms_norm_grad(dy, x, w, rstd, dx, dw, workspace=ws, workspace_bytes=nbytes)
    ref_x, ref_w, _ = L.rms_norm_grad(dy, x.cpu().to(F64), w, rstd, None)
    R.check(dx, *ref_x, "grad_x")
    R.check(dw, *ref_w, "grad_weight")
    first = dx.clone(), dw.clone()
    zf.zero_rms_norm_grad(dy, x, w, rstd, dx, dw, workspace=ws, workspace_bytes=nbytes)
    assert torch.equal(first[0], dx) and torch.equal(first[1], dw), "bits differ from run to run"


def test_rms_norm_gradient_is_the_difference_quotient():
    """d/dx and d/dw of sum(out * c) + sum(total * e), by central differences of the
    64-bit norm."""
    n, d, h = 3, 33, 1e-6
    g = _gen("difference")
    x, c, e = (torch.randn((n, d), generator=g) for _ in range(3))
    w = torch.randn(d, generator=g)

    def value(xs, ws):
        y = L.rms_norm(xs, ws, 1e-3)[0]
        return float((y * c.to(F64)).sum() + (xs * e.to(F64)).sum())

    rstd = torch.zeros(n, device="cuda")
    zf.zero_rms_norm(x.cuda(), None, w.cuda(), 1e-3, rstd=rstd)
    dx, dw = torch.empty((n, d), device="cuda"), torch.empty(d, device="cuda")
    nbytes = zf.zero_rms_norm_grad_workspace_bytes(n, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    zf.zero_rms_norm_grad(c.cuda(), x.cuda(), w.cuda(), rstd, dx, dw, e.cuda(), None, ws, nbytes)
    # the quotient of values of about 100 is off by 1e-14 * 100 / h = 1e-6 and by h^2; the
    # gradient of values of at most 10 by some 50 u of them, 3e-5
    for i, j in ((0, 0), (1, 17), (2, 32)):
        up, down = x.to(F64), x.to(F64)
        up, down = up.clone(), down.clone()
        up[i, j] += h
        down[i, j] -= h
        q = (value(up, w.to(F64)) - value(down, w.to(F64))) / (2 * h)
        assert abs(q - float(dx[i, j])) <= 5e-5
    for j in (0, 20):
        up, down = w.to(F64).clone(), w.to(F64).clone()
        up[j] += h
        down[j] -= h
        q = (value(x.to(F64), up) - value(x.to(F64), down)) / (2 * h)
        assert abs(q - float(dw[j])) <= 5e-5


def test_rms_norm_of_no_rows():
    x = torch.empty((0, 64), device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    zf.zero_rms_norm(x, x, None, 1e-5, x, None, torch.empty(0, device="cuda"),
                     (torch.empty((0, 64), dtype=torch.uint8, device="cuda"),
                      torch.empty((0, 1), device="cuda")))
    nbytes = zf.zero_rms_norm_grad_workspace_bytes(0, 64)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    zf.zero_rms_norm_grad(x, x, None, torch.empty(0, device="cuda"), torch.empty_like(x), dw,
                          workspace=ws, workspace_bytes=nbytes)
    assert bool((dw == 0).all())
    zf.zero_pack_rows(x, (torch.empty((0, 64), dtype=torch.uint8, device="cuda"),
                          torch.empty((0, 1), device="cuda")))


def test_rms_norm_of_zeros_and_of_nan():
    x = torch.ones((4, 300), device="cuda")
    x[1] = 0.0
    x[2, 7] = float("nan")
    out, rstd = torch.empty_like(x), torch.zeros(4, device="cuda")
    zf.zero_rms_norm(x, None, None, 1e-5, out, rstd=rstd)
    y = L.rms_norm(x.cpu().to(F64), None, 1e-5)
    R.check(out, *y[:2], "out")                        # NaN stays in its row
    assert bool((out[1] == 0).all()) and bool(torch.isnan(out[2]).all())


def _mixed_calls(stream=None):
    """The norm, its checkpoint and its gradient, as a training step runs them."""
    g = _gen("mixed")
    n, d = 300, 1504
    x, res = _stream(g, n, d, BF16).cuda(), _stream(g, n, d, BF16).cuda()
    w, dy = _weight(g, d, BF16, 0), (_stream(g, n, d, BF16) * 0.01).cuda()
    total, out, dx, again = (torch.zeros_like(x) for _ in range(4))
    rstd, dw, p = torch.zeros(n, device="cuda"), torch.zeros_like(w), Packed(n, d)
    nbytes = zf.zero_rms_norm_grad_workspace_bytes(n, d)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def call():
        zf.zero_rms_norm(x, res, w, 1e-5, out, total, rstd, None, p.pair, stream=stream)
        zf.zero_rms_norm_grad(dy, p.pair, w, rstd, dx, dw, total, again, ws, nbytes,
                              stream=stream)
        zf.zero_unpack_rows(p.pair, total, stream=stream)
    return call, (total, out, rstd, dx, dw, again, *p.pair)


def test_streams_give_the_same_bits():
    call, ref = _mixed_calls()
    call()
    side = torch.cuda.Stream()
    call2, got = _mixed_calls(side)
    call2()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_capture_into_a_graph():
    call, ref = _mixed_calls()
    call()
    torch.cuda.synchronize()
    call2, got = _mixed_calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call2()
    for t in got:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("label", ["rms norm launch", "rms norm gradient launch",
                                   "rms norm gradient reduction launch", "row unpacking launch"])
def test_injected_failure_is_reported_and_a_retry_is_clean(monkeypatch, label):
    call, got = _mixed_calls()
    call()
    want = [t.clone() for t in got]
    monkeypatch.setenv("ZERO_INJECT_FAILURE", label)
    with pytest.raises(zf.ZeroError, match="injected failure"):
        call()
    monkeypatch.delenv("ZERO_INJECT_FAILURE")
    call()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
