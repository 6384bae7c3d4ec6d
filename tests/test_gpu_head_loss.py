"""The head's softmax cross entropy and its gradients against plain 64-bit
implementations (layer_reference.py, whose bounds are derived there): odd and
ragged sizes, strides and alignments, one and no tokens, labels that leave
nothing, NaN in tokens that do not count, several pieces of the vocabulary."""
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


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert zf.zero_device_status(clear=True) == 0


def _gen(*key):
    from fsdp_sharded_mixed_flatten_gb300.synthetic import seed_for
    return torch.Generator().manual_seed(seed_for("head-loss", *key))


def _rows(n, d, pad, offset, fill=None):
    """n rows of d in a wider buffer at an element offset, and the buffer, of NaN bits."""
    base = torch.full((offset + n * (d + pad) + 64,), 0x7FC1, dtype=torch.int16, device="cuda")
    t = base.view(BF16)[offset:offset + n * (d + pad)].view(n, d + pad)[:, :d]
    if fill is not None:
        t.copy_(fill)
    return t, base


def _outside(t, base):
    """Nothing but t's own elements has been written."""
    mask = torch.ones(base.shape, dtype=torch.bool, device="cuda")
    n, d = t.shape
    if n * d:
        torch.as_strided(mask, (n, d), t.stride(), t.storage_offset()).fill_(False)
    return bool((base[mask] == 0x7FC1).all())


def _labels(g, n, vocab, kind):
    y = torch.randint(0, vocab, (n,), generator=g)
    if kind == "some":
        y[torch.rand(n, generator=g) < 0.4] = -100
        y[torch.rand(n, generator=g) < 0.1] = vocab
    elif kind == "none":
        y[:] = -1
    elif kind == "last":
        y[:] = -100
        y[-1] = vocab - 1
    elif kind == "one":
        y[:] = 0
    return y


def _workspace(nbytes):
    ws = torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN everywhere
    return ws


def _inputs(key, n, vocab, d, pad, offset, kind, label_type=torch.int64):
    g = _gen(*key, n, vocab, d, kind)
    h, _ = _rows(n, d, pad, offset, torch.randn((n, d), generator=g) * (8.0 / d ** 0.5))
    w, _ = _rows(vocab, d, 0, offset, torch.randn((vocab, d), generator=g) * 0.25)
    y = _labels(g, n, vocab, kind)
    dead = (y < 0) | (y >= vocab)
    h[dead.cuda()] = float("nan")                  # what does not count reaches nothing
    return g, h, w.reshape(vocab, d), y.to(label_type).cuda()


def _loss(h, w, y, lse=True):
    n, vocab, d = h.shape[0], *w.shape
    nbytes = zf.zero_head_loss_workspace_bytes(n, vocab, d)
    ws = _workspace(nbytes)
    out = torch.full((2, n), 7.0, device="cuda")
    zf.zero_head_loss(h, w, y, out[0], out[1] if lse else None, ws, nbytes)
    assert bool((ws[nbytes:] == 0xFF).all()), "wrote past the workspace"
    return out


def _grad(h, w, y, lse, gl, dh, dw, accumulate=False):
    n, vocab, d = h.shape[0], *w.shape
    nbytes = zf.zero_head_loss_grad_workspace_bytes(n, vocab, d)
    ws = _workspace(nbytes)
    zf.zero_head_loss_grad(h, w, y, lse, gl, dh, dw, accumulate, ws, nbytes)
    assert bool((ws[nbytes:] == 0xFF).all()), "wrote past the workspace"


def _near(got, ref, bound, norm, what):
    R.check(got, ref.cpu(), bound.cpu(), what)
    off = float(torch.linalg.vector_norm(got.to(F64) - ref.to(got.device)))
    assert off <= norm, f"{what}: 2-norm off by {off}, at most {norm}"


# tokens, vocabulary, width, pad columns, element offset
SIZES = [(1, 1, 1, 0, 0), (1, 256, 64, 0, 0), (2, 3, 8, 0, 0), (5, 257, 63, 1, 1),
         (127, 1000, 65, 0, 8), (128, 512, 128, 8, 0), (129, 255, 257, 0, 0), (256, 4099, 256, 0, 0),
         (257, 1000, 770, 2, 37), (300, 2048, 768, 0, 0), (700, 513, 72, 0, 3), (64, 50257, 96, 0, 0),
         (33, 5003, 1504, 0, 16)]


@pytest.mark.parametrize("kind", ["all", "some", "none", "last", "one"])
@pytest.mark.parametrize("n,vocab,d,pad,offset", SIZES)
def test_head_loss(n, vocab, d, pad, offset, kind):
    label_type = torch.int32 if n % 2 else torch.int64
    _, h, w, y = _inputs(("loss",), n, vocab, d, pad, offset, kind, label_type)
    out = _loss(h, w, y)
    loss, lse = L.head_loss(h, w, y)
    R.check(out[0], *(t.cpu() for t in loss), "loss")
    R.check(out[1], *(t.cpu() for t in lse), "lse")
    alone = _loss(h, w, y, lse=False)
    assert torch.equal(alone[0], out[0]) and bool((alone[1] == 7.0).all())


# Few tokens in place: one row of the table and one more than the even shares, a share that
# ends inside a tile, columns summed in parts, tokens on both sides of a half, strided rows.
@pytest.mark.parametrize("kind", ["all", "some", "last"])
@pytest.mark.parametrize("n,vocab,d,pad", [
    (1, 1, 8, 0), (1, 17, 64, 8), (2, 15, 72, 0), (3, 127, 1528, 0), (7, 129, 1544, 24),
    (31, 2432, 128, 0), (32, 2433, 136, 0), (32, 33000, 64, 0), (33, 19457, 776, 8),
    (63, 22000, 1600, 0), (64, 40009, 200, 0), (64, 1000, 4104, 0), (65, 1000, 200, 0)])
def test_head_loss_of_few_tokens(n, vocab, d, pad, kind):
    _, h, w, y = _inputs(("few",), n, vocab, d, pad, 0, kind)
    out = _loss(h, w, y)
    loss, lse = L.head_loss(h, w, y)
    R.check(out[0], *(t.cpu() for t in loss), "loss")
    R.check(out[1], *(t.cpu() for t in lse), "lse")
    assert torch.equal(_loss(h, w, y), out)


def test_head_loss_of_few_tokens_with_infinite_logits():
    """Rows of the table that a token reaches at minus infinity leave the sum, one at plus
    infinity or NaN takes its own token's loss and no other's."""
    g = _gen("few", "infinite")
    h, w = torch.zeros((40, 64)), torch.randn((3000, 64), generator=g) * 0.25
    h[:, 0] = 1.0
    h[:, 1:8] = torch.randn((40, 7), generator=g)
    w[100:900, 0] = float("-inf")
    w[2500:, 0] = float("-inf")
    h[3, 5] = float("nan")
    h[37, 0] = -1.0
    y = torch.full((40,), 2000)
    h, w, y = h.to(BF16).cuda(), w.to(BF16).cuda(), y.cuda()
    out = _loss(h, w, y)
    live = torch.ones(3000, dtype=torch.bool)
    live[100:900] = False
    live[2500:] = False
    keep = [i for i in range(40) if i not in (3, 37)]
    few_y = torch.full((38,), int(live[:2000].sum()), device="cuda")
    loss, lse = L.head_loss(h[keep].contiguous(), w[live.cuda()].contiguous(), few_y)
    R.check(out[0][keep], *(t.cpu() for t in loss), "loss")
    R.check(out[1][keep], *(t.cpu() for t in lse), "lse")
    assert bool(out[0][[3, 37]].isnan().all())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["all", "some", "none", "last", "one"])
@pytest.mark.parametrize("n,vocab,d,pad,offset", SIZES)
def test_head_loss_grad(n, vocab, d, pad, offset, kind, accumulate):
    g, h, w, y = _inputs(("grad",), n, vocab, d, pad, offset, kind)
    lse = _loss(h, w, y)[1]
    gl = torch.rand(n, generator=g) * 2 - 0.5
    gl[torch.rand(n, generator=g) < 0.1] = 0.0
    gl = gl.cuda()
    h[(gl == 0)] = float("inf")
    dh, dh_base = _rows(n, d, pad, offset, torch.full((n, d), 3.0))
    old = torch.randn((vocab, d), generator=g)
    dw, dw_base = _rows(vocab, d, 0, offset, old)
    before = dw.clone() if accumulate else None
    _grad(h, w, y, lse, gl, dh, dw.reshape(vocab, d), accumulate)
    ref_h, ref_w = L.head_loss_grad(h, w, y, lse, gl, before)
    _near(dh, *ref_h, "grad_hidden")
    _near(dw, *ref_w, "grad_table")
    assert _outside(dh, dh_base) and _outside(dw, dw_base)
    # one gradient alone is what it is with the other; in place of the hidden states
    dw1 = before.clone() if accumulate else torch.empty_like(dw)
    _grad(h, w, y, lse, gl, None, dw1, accumulate)
    assert torch.equal(dw1, dw)
    _grad(h, w, y, lse, gl, h, None)
    assert torch.equal(h, dh)


@pytest.mark.parametrize("n,vocab,d,pad,offset", [(8192, 50257, 64, 0, 0), (8000, 33000, 100, 4, 5),
                                                  (3000, 12345, 768, 0, 0)])
def test_head_loss_in_pieces(n, vocab, d, pad, offset):
    """More of the logits' gradient than the workspace holds, many rows; the
    same bits from run to run."""
    g, h, w, y = _inputs(("pieces",), n, vocab, d, pad, offset, "some")
    out = _loss(h, w, y)
    loss, lse = L.head_loss(h, w, y)
    R.check(out[0], *(t.cpu() for t in loss), "loss")
    R.check(out[1], *(t.cpu() for t in lse), "lse")
    gl = torch.full((n,), 1.0 / n, device="cuda")
    dh, dh_base = _rows(n, d, pad, offset)
    dw, dw_base = _rows(vocab, d, 0, offset)
    _grad(h, w, y, out[1], gl, dh, dw.reshape(vocab, d))
    ref_h, ref_w = L.head_loss_grad(h, w, y, out[1], gl)
    _near(dh, *ref_h, "grad_hidden")
    _near(dw, *ref_w, "grad_table")
    assert _outside(dh, dh_base) and _outside(dw, dw_base)
    again = torch.empty_like(dw), torch.empty((n, d), dtype=BF16, device="cuda")
    _grad(h, w, y, out[1], gl, again[1], again[0])
    assert torch.equal(again[0], dw) and torch.equal(again[1], dh), "bits differ from run to run"
    assert torch.equal(_loss(h, w, y), out)


def test_head_loss_gradient_is_the_difference_quotient():
    """d sum(g loss) / dh and dW by central differences of the 64-bit loss.  The
    gradients are bf16: 2^-8 of themselves, and 2^-8 sum |dz w| from dz (the bounds
    of layer_reference); the quotient's own error is about 1e-9."""
    n, vocab, d, step = 7, 301, 40, 1e-5
    g, h, w, y = _inputs(("difference",), n, vocab, d, 0, 0, "all")
    lse = _loss(h, w, y)[1]
    gl = torch.rand(n, generator=g).cuda()
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    _grad(h, w, y, lse, gl, dh, dw)
    (_, h_off, _), (_, w_off, _) = L.head_loss_grad(h, w, y, lse, gl)

    def value(hh, ww):
        return float((torch.nn.functional.cross_entropy(hh @ ww.t(), y, reduction="none")
                      * gl.to(F64)).sum())

    for which, got, off in ((0, dh, h_off), (1, dw, w_off)):
        for i, j in ((0, 0), (3, 17), (6, 39), (int(y[2]) if which else 2, 5)):
            args = [[h.to(F64), w.to(F64)] for _ in range(2)]
            for sign, a in zip((1, -1), args):
                a[which] = a[which].clone()
                a[which][i, j] += sign * step
            q = (value(*args[0]) - value(*args[1])) / (2 * step)
            assert abs(q - float(got[i, j])) <= float(off[i, j]) + 2.0 ** -8 * abs(q) + 1e-8


def test_head_loss_of_large_and_equal_logits():
    """Logits of +-2000 keep their differences; a row of equal ones is log(vocab)."""
    vocab, d = 1000, 64
    h = torch.zeros((4, d), dtype=BF16, device="cuda")
    w = torch.zeros((vocab, d), dtype=BF16, device="cuda")
    w[:, 0] = 1.0
    w[5, 1] = 1.0
    h[0, 0], h[1, 0], h[2, 0] = 2000.0, -2000.0, 0.0
    h[0, 1] = h[1, 1] = 8.0
    h[3, 1] = 1000.0
    y = torch.tensor([5, 6, 7, 5], device="cuda")
    out = _loss(h, w, y)
    loss, lse = L.head_loss(h, w, y)
    R.check(out[0], *(t.cpu() for t in loss), "loss")
    R.check(out[1], *(t.cpu() for t in lse), "lse")
    # the other 999 exponentials are 0 and the label's is 1, off by at most 2 units of 2^-23
    assert 0.0 <= float(out[0, 3]) <= 2.0 ** -22


@pytest.mark.parametrize("n", [4, 32, 40, 300])
def test_head_loss_of_equal_logits_of_any_size(n):
    """Equal logits up to 5.6e7, each one product that fp32 holds: log(vocab).  Their
    multiples of log2 e are rounded by up to 4 there, which the sum makes up for.  Off by
    the sum's additions (at most 300 one after another, 2^-24 each), an exponential's error
    (2^-22), the logarithm's (below 16: an ulp of 2^-20) and the roundings of the result's
    parts (2^-20 in all): below 2^-15."""
    vocab, d = 12288, 64
    h = torch.zeros((n, d), dtype=BF16, device="cuda")
    w = torch.zeros((vocab, d), dtype=BF16, device="cuda")
    i = torch.arange(n, device="cuda")
    h[:, 0] = ((128 + i % 128) * 2.0 ** (i % 4 * 3 - 2)).to(BF16)       # up to 32640
    h[::2, 0] *= -1.0
    w[:, 0] = 1696.0
    y = torch.arange(n, device="cuda") * 37
    out = _loss(h, w, y)
    off = (out[0].to(F64) - torch.log(torch.tensor(float(vocab), dtype=F64))).abs()
    assert float(off.max()) <= 2.0 ** -15


def test_head_loss_of_nan_stays_in_its_row():
    g, h, w, y = _inputs(("nan",), 300, 700, 64, 0, 0, "all")
    clean = _loss(h, w, y)
    h[7, 3] = float("nan")
    out = _loss(h, w, y)
    assert bool(torch.isnan(out[:, 7]).all())
    keep = torch.arange(300, device="cuda") != 7
    assert torch.equal(out[:, keep], clean[:, keep])
    gl = torch.ones(300, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    _grad(h, w, y, out[1], gl, dh, dw)
    assert bool(torch.isnan(dh[7]).all()) and bool(torch.isfinite(dh[keep]).all())


def test_head_loss_of_no_tokens():
    w = torch.ones((300, 64), dtype=BF16, device="cuda")
    h = torch.empty((0, 64), dtype=BF16, device="cuda")
    y, e = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    zf.zero_head_loss(h, w, y, e, e)
    dw = torch.full((300, 64), 3.0, dtype=BF16, device="cuda")
    _grad(h, w, y, e, e, h, dw, accumulate=True)
    assert bool((dw == 3.0).all())
    _grad(h, w, y, e, e, h, dw)
    assert bool((dw == 0.0).all())


@pytest.mark.parametrize("n", [1, 12, 9000])
def test_gradients_of_alike_losses_keep_their_size(n):
    """Equal logits and one gradient of the loss, halfway between two of bf16 and of either
    sign: softmax minus one is off by 2^-12 at most, and nothing else is rounded before the
    result (2^-8 of it); 9000 terms' sum is off by 2^-10 of it more at most."""
    vocab, d, size = 4096, 96, 0.5 + 2.0 ** -9
    g = _gen("alike", n)
    h = (torch.rand((n, d), generator=g) + 1.0).to(BF16).cuda()
    w = torch.zeros((vocab, d), dtype=BF16, device="cuda")
    y = torch.full((n,), 17, device="cuda")
    lse = _loss(h, w, y)[1]
    gl = torch.full((n,), -size if n == 12 else size, device="cuda")
    if n > 1:
        gl[1] = float("nan")
        y[1] = -1
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    _grad(h, w, y, lse, gl, dh, dw)
    keep = (y >= 0).to(F64)[:, None]
    total = (h.to(F64) * keep).sum(0) * gl[0].to(F64)
    for row, want in ((17, total * (1.0 / vocab - 1.0)), (5, total / vocab)):
        off = ((dw[row].to(F64) - want) / want).abs()
        assert float(off.max()) <= 2.0 ** -8 + 2.0 ** -12 + 2.0 ** -10
    assert bool((dh == 0.0).all())


def _mixed_calls(stream=None, key="mixed"):
    g, h, w, y = _inputs((key,), 500, 3001, 136, 0, 0, "some")
    n, vocab, d = 500, 3001, 136
    gl = torch.rand(n, generator=g).cuda()
    out = torch.zeros((2, n), device="cuda")
    dh, dw = torch.zeros((n, d), dtype=BF16, device="cuda"), torch.zeros_like(w)
    size = max(zf.zero_head_loss_workspace_bytes(n, vocab, d),
               zf.zero_head_loss_grad_workspace_bytes(n, vocab, d))
    ws = _workspace(size)
    torch.cuda.synchronize()

    def call():
        zf.zero_head_loss(h, w, y, out[0], out[1], ws, size, stream=stream)
        zf.zero_head_loss_grad(h, w, y, out[1], gl, dh, dw, False, ws, size, stream=stream)
    return call, (out, dh, dw)


def _few_calls(stream, n):
    g, h, w, y = _inputs(("few at once",), n, 20011, 264, 0, 0, "some")
    out, size = torch.zeros((2, n), device="cuda"), zf.zero_head_loss_workspace_bytes(n, 20011, 264)
    ws = _workspace(size)
    torch.cuda.synchronize()
    return lambda: zf.zero_head_loss(h, w, y, out[0], out[1], ws, size, stream=stream), out


def test_few_tokens_on_streams_at_once_and_captured():
    refs = {}
    for n in (20, 50):
        call, refs[n] = _few_calls(None, n)
        call()
    torch.cuda.synchronize()
    calls = [(_few_calls(torch.cuda.Stream(), n), n) for n in (20, 50, 20)]
    for _ in range(3):
        for (call, _), _ in calls:
            call()
    torch.cuda.synchronize()
    for (_, out), n in calls:
        assert torch.equal(out, refs[n])
    some = [_few_calls(None, n) for n in (20, 50)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _ in some + some:
            call()
    for _, out in some:
        out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for (_, out), n in zip(some, (20, 50)):
        assert torch.equal(out, refs[n])


def test_streams_at_once_give_the_same_bits():
    call, ref = _mixed_calls()
    call()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    calls = [_mixed_calls(s) for s in sides]
    for _ in range(3):
        for c, _ in calls:
            c()
    torch.cuda.synchronize()
    for _, got in calls:
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


@pytest.mark.parametrize("label", ["head rows", "head gather", "head loss launch", "head join",
                                   "head logits' gradient", "head gradients launch",
                                   "head gradient rows"])
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
