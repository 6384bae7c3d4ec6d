"""The operators around the root unit against plain 64-bit implementations
(root_reference.py, whose bounds are derived there): every type, odd and
ragged sizes, strides and alignments, lengths of zero and one, masks that
leave nothing, values at the ends of the types' ranges."""
import numpy as np
import pytest
import torch

import root_reference as R

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


def _gen(*key):
    from fsdp_sharded_mixed_flatten_gb300.synthetic import seed_for
    return torch.Generator().manual_seed(seed_for("root-ops", *key))


class Guarded:
    """A matrix of n rows in a wider buffer at an element offset, with a
    sentinel everywhere else."""

    def __init__(self, n, d, dtype, pad=0, offset=0, fill=None):
        self.sentinel = 1536.0                 # exact in bf16
        self.base = torch.full((offset + n * (d + pad) + 64,), self.sentinel, dtype=dtype,
                               device="cuda")
        self.t = self.base[offset:offset + n * (d + pad)].view(n, d + pad)[:, :d]
        if fill is not None:
            self.t.copy_(fill)
        elif n * d:
            self.t.fill_(-7.0)                 # stale values

    def check_guard(self, what):
        keep = self.base.clone()
        n, d = self.t.shape
        inside = torch.zeros_like(self.base, dtype=torch.bool)
        if n * d:
            torch.as_strided(inside, (n, d), self.t.stride(), self.t.storage_offset()).fill_(True)
        assert bool((keep[~inside] == self.sentinel).all()), f"{what}: wrote outside its rows"


def _bits(t):
    t = t.contiguous()
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32).cpu()


# ----------------------------------------------------------- token table ----

TABLES = [
    # tokens, vocab, dim, pad columns, flat offset
    (1, 1, 1, 0, 0), (1, 50257, 768, 0, 0), (7, 5, 3, 1, 1), (33, 11, 257, 0, 3),
    (129, 4096, 520, 8, 8), (1000, 300, 64, 0, 0), (2049, 1000, 770, 2, 5), (4096, 50257, 256, 0, 0),
    # beyond the bucket launch's tokens: sorted
    (16385, 1000, 40, 0, 0), (20011, 50257, 73, 1, 3), (33000, 7, 264, 0, 0),
]


def _ids(g, n, vocab, kind):
    """hot: most tokens alike; tail: some out of range; one: all the same."""
    ids = torch.randint(0, vocab, (n,), generator=g)
    if kind == "hot":
        ids[torch.rand(n, generator=g) < 0.7] = vocab // 2
    elif kind == "tail":
        ids[torch.rand(n, generator=g) < 0.2] = -1
        ids[torch.rand(n, generator=g) < 0.1] = vocab
        ids[torch.rand(n, generator=g) < 0.1] = 2 ** 31 - 1
    elif kind == "one":
        ids[:] = vocab - 1
    elif kind == "none":
        ids[:] = -5
    return ids


@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,vocab,dim,pad,offset", TABLES)
def test_embedding(n, vocab, dim, pad, offset, types, id_type):
    g = _gen("embedding", n, vocab, dim)
    w = Guarded(vocab, dim, types[0], 0, offset, torch.randn((vocab, dim), generator=g))
    ids = _ids(g, n, vocab, "tail").to(id_type).cuda()
    if id_type == torch.int64 and n > 2:
        ids[1] = 2 ** 32              # its low half is a valid id
    out = Guarded(n, dim, types[1], pad, offset)
    zf.zero_embedding(ids, w.t, out.t, 27.75)
    ref, bound = R.embedding(ids, w.t, 27.75)
    R.check(out.t, ref, bound, "out")
    out.check_guard("out")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["uniform", "hot", "tail", "one", "none"])
@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,vocab,dim,pad,offset", TABLES)
def test_embedding_grad(n, vocab, dim, pad, offset, types, kind, accumulate):
    g = _gen("embedding-grad", n, vocab, dim, kind)
    ids = _ids(g, n, vocab, kind).to(torch.int32).cuda()
    dy = Guarded(n, dim, types[0], pad, 0, torch.randn((n, dim), generator=g) * 0.01)
    old = torch.randn((vocab, dim), generator=g) * 0.01
    dw = Guarded(vocab, dim, types[1], 0, offset, old if accumulate else None)
    before = dw.t.clone()
    nbytes = zf.zero_embedding_grad_workspace_bytes(n, vocab, dim)
    ws = torch.full((nbytes + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    zf.zero_embedding_grad(ids, dy.t, dw.t, 0.5, accumulate, ws, nbytes)
    ref, bound = R.embedding_grad(ids, dy.t, (vocab, dim), 0.5, before if accumulate else None)
    R.check(dw.t, ref, bound, "grad_weight")
    dw.check_guard("grad_weight")
    assert bool((ws[nbytes:] == 0xA5).all()), "wrote past the workspace"
    if accumulate:
        used = torch.zeros(vocab, dtype=torch.bool)
        used[ids.cpu().long()[(ids.cpu() >= 0) & (ids.cpu() < vocab)]] = True
        assert torch.equal(_bits(dw.t)[~used], _bits(before)[~used]), "touched an unused row"


def test_embedding_grad_of_ignored_tokens_is_not_read():
    """NaN and infinities in the rows of ids out of range stay out."""
    dy = torch.full((40, 24), float("nan"), device="cuda")
    dy[5] = 1.0
    dy[6] = float("inf")
    ids = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    ids[5] = 3
    dw = torch.empty((9, 24), device="cuda")
    nbytes = zf.zero_embedding_grad_workspace_bytes(40, 9, 24)
    zf.zero_embedding_grad(ids, dy, dw, 2.0, False, torch.empty(nbytes, dtype=torch.uint8,
                                                               device="cuda"), nbytes)
    ref = torch.zeros((9, 24))
    ref[3] = 2.0
    assert torch.equal(dw.cpu(), ref)


@pytest.mark.parametrize("n", [5000, 70001])
def test_embedding_grad_repeats_bit_for_bit(n):
    """Long runs over many chunks are joined in chunk order, whoever is last."""
    g = _gen("embedding-repeat", n)
    ids = torch.where(torch.rand(n, generator=g) < 0.5, 17, torch.randint(0, 200, (n,), generator=g))
    ids = ids.cuda()
    dy = torch.randn((n, 264), generator=g).to(BF16).cuda()
    nbytes = zf.zero_embedding_grad_workspace_bytes(n, 200, 264)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(20):
        dw = torch.empty((200, 264), device="cuda")
        zf.zero_embedding_grad(ids, dy, dw, 1.0, False, ws, nbytes)
        if first is None:
            first = dw
            ref, bound = R.embedding_grad(ids, dy, (200, 264), 1.0)
            R.check(dw, ref, bound, "grad_weight")
        assert torch.equal(_bits(dw), _bits(first))


@pytest.mark.parametrize("label", ["embedding gradient sort", "embedding gradient sum"])
def test_embedding_grad_failure_and_retry(monkeypatch, label):
    ids = torch.randint(0, 500, (18000,), generator=_gen("retry")).cuda()
    dy = torch.randn((18000, 48), generator=_gen("retry-dy")).cuda()
    nbytes = zf.zero_embedding_grad_workspace_bytes(18000, 500, 48)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    dw = [torch.zeros((500, 48), device="cuda") for _ in range(2)]
    zf.zero_embedding_grad(ids, dy, dw[0], 1.0, True, ws, nbytes)
    monkeypatch.setenv("ZERO_INJECT_FAILURE", label)
    with pytest.raises(zf.ZeroError) as ei:
        zf.zero_embedding_grad(ids, dy, dw[1], 1.0, True, ws, nbytes)
    assert ei.value.code == -4 and label in str(ei.value)
    assert not dw[1].any()
    monkeypatch.delenv("ZERO_INJECT_FAILURE")
    zf.zero_embedding_grad(ids, dy, dw[1], 1.0, True, ws, nbytes)
    assert torch.equal(dw[0], dw[1])


def test_embedding_of_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones((5, 6), device="cuda")
    none = torch.empty((0, 6), device="cuda")
    zf.zero_embedding(ids, w, none)
    zf.zero_embedding_grad(ids, none, w, 1.0, True)
    assert bool((w == 1).all())
    zf.zero_embedding_grad(ids, none, w, 1.0, False)
    assert bool((w == 0).all())


def test_table_beyond_32_bit_elements():
    """Rows whose first element lies past 2^31 elements."""
    vocab, dim = 600_000, 4096                 # 2.46e9 elements, 4.9 GB
    w = torch.zeros((vocab, dim), dtype=BF16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, 524_289, vocab - 1], device="cuda")
    w[ids] = torch.randn((4, dim), generator=_gen("far")).to(BF16).cuda()
    out = torch.empty((4, dim), dtype=BF16, device="cuda")
    zf.zero_embedding(ids, w, out, 1.0)
    assert torch.equal(_bits(out), _bits(w[ids]))
    dy = torch.randn((4, dim), generator=_gen("far-dy")).to(BF16).cuda()
    w.fill_(3.0)
    nbytes = zf.zero_embedding_grad_workspace_bytes(4, vocab, dim)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    zf.zero_embedding_grad(ids, dy, w, 1.0, False, ws, nbytes)
    f = dy.float()
    assert torch.equal(_bits(w[vocab - 1]), _bits((f[0] + f[3]).to(BF16)))
    assert torch.equal(_bits(w[524_289]), _bits(dy[2]))
    assert torch.equal(_bits(w[0]), _bits(dy[1]))
    w[ids] = 0
    assert int(torch.count_nonzero(w)) == 0


# ------------------------------------------------------------ layer norm ----

NORMS = [
    # rows, dim, pad columns, flat offset
    (1, 1, 0, 0), (3, 2, 0, 1), (5, 31, 1, 0), (1, 256, 0, 0), (17, 264, 8, 0), (9, 500, 3, 3),
    (300, 768, 0, 64), (33, 770, 0, 0), (8, 1024, 0, 0), (13, 1032, 0, 0), (257, 1501, 3, 3),
    (6, 4096, 0, 0), (3, 8192, 8, 8), (2, 12289, 0, 0), (5, 16384, 0, 0),
]


def _norm_inputs(n, dim, act, param, pad, offset):
    g = _gen("norm", n, dim)
    x = torch.randn((n, dim), generator=g) * (0.5 + torch.rand((n, 1), generator=g) * 3) \
        + torch.randn((n, 1), generator=g)
    x = Guarded(n, dim, act, pad, 0, x)
    w = Guarded(1, dim, param, 0, offset, 1 + 0.2 * torch.randn((1, dim), generator=g))
    b = Guarded(1, dim, param, 0, offset, torch.randn((1, dim), generator=g))
    dy = Guarded(n, dim, act, pad, 0, torch.randn((n, dim), generator=g) * 0.1)
    return x, w, b, dy


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("param", [BF16, F32, None])
@pytest.mark.parametrize("n,dim,pad,offset", NORMS)
def test_layer_norm(n, dim, pad, offset, act, param):
    x, w, b, _ = _norm_inputs(n, dim, act, param or F32, pad, offset)
    weight, bias = (w.t[0], b.t[0]) if param else (None, None)
    out = Guarded(n, dim, act, pad, 0)
    mean, rstd = (torch.empty(n, device="cuda") for _ in range(2))
    zf.zero_layer_norm(x.t, weight, bias, 1e-5, out.t, mean, rstd)
    ref = R.layer_norm(x.t, weight, bias, 1e-5)
    R.check(mean, ref["mean"], ref["d_mean"], "mean")
    R.check(rstd, ref["rstd"], ref["d_rstd"] + 4 * R.U * ref["rstd"], "rstd")
    R.check(out.t, ref["out"], ref["d_out"], "out")
    out.check_guard("out")
    # in place, and without the statistics
    again = out.t.clone()
    zf.zero_layer_norm(x.t, weight, bias, 1e-5, x.t)
    assert torch.equal(_bits(x.t), _bits(again))
    x.check_guard("x")


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("param", [BF16, F32])
@pytest.mark.parametrize("n,dim,pad,offset", NORMS)
def test_layer_norm_grad(n, dim, pad, offset, act, param):
    x, w, _, dy = _norm_inputs(n, dim, act, param, pad, offset)
    xd = x.t.double()
    mu = xd.mean(1)
    mean = mu.float()
    rstd = torch.rsqrt((xd - mu[:, None]).square().mean(1) + 1e-5).float()
    dx = Guarded(n, dim, act, pad, 0)
    dw, db = Guarded(1, dim, param, 0, offset), Guarded(1, dim, param, 0, offset)
    nbytes = zf.zero_layer_norm_grad_workspace_bytes(n, dim)
    ws = torch.full((nbytes + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    zf.zero_layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, dx.t, dw.t[0], db.t[0], ws, nbytes)
    ref = R.layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, max(1, nbytes // (8 * dim)))
    R.check(dx.t, ref["grad_x"], ref["d_x"], "grad_x")
    R.check(dw.t, ref["grad_weight"], ref["d_weight"],
            "grad_weight")
    R.check(db.t, ref["grad_bias"], ref["d_bias"],
            "grad_bias")
    for b in (dx, dw, db):
        b.check_guard("gradient")
    assert bool((ws[nbytes:] == 0xA5).all()), "wrote past the workspace"
    # in place of grad_out, without the parameters' gradients: the same bits
    again = dx.t.clone()
    zf.zero_layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, dy.t, None, None, ws, nbytes)
    assert torch.equal(_bits(dy.t), _bits(again))
    dy.check_guard("grad_out")


@pytest.mark.parametrize("n,dim", [(3000, 768), (2000, 1501), (999, 4096), (20000, 96)])
def test_layer_norm_grad_of_many_rows(n, dim):
    x, w, _, dy = _norm_inputs(n, dim, BF16, F32, 0, 0)
    xd = x.t.double()
    mean = xd.mean(1).float()
    rstd = torch.rsqrt(xd.var(1, unbiased=False) + 1e-5).float()
    nbytes = zf.zero_layer_norm_grad_workspace_bytes(n, dim)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    ref = R.layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, max(1, nbytes // (8 * dim)))
    first = None
    for _ in range(3):
        dx, dw, db = torch.empty_like(x.t), *(torch.empty(dim, device="cuda") for _ in range(2))
        zf.zero_layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, dx, dw, db, ws, nbytes)
        if first is None:
            first = (dx, dw, db)
            R.check(dx, ref["grad_x"], ref["d_x"], "grad_x")
            R.check(dw, ref["grad_weight"], ref["d_weight"], "grad_weight")
            R.check(db, ref["grad_bias"], ref["d_bias"], "grad_bias")
        for a, b in zip(first, (dx, dw, db)):
            assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n,dim", [(500, 9000), (350, 16384)])
def test_layer_norm_grad_of_wide_rows(n, dim, act):
    """Several rows a CTA where a thread holds the most columns; in place."""
    x, w, _, dy = _norm_inputs(n, dim, act, F32, 0, 0)
    xd = x.t.double()
    mean = xd.mean(1).float()
    rstd = torch.rsqrt(xd.var(1, unbiased=False) + 1e-5).float()
    nbytes = zf.zero_layer_norm_grad_workspace_bytes(n, dim)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    ref = R.layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, max(1, nbytes // (8 * dim)))
    dx = Guarded(n, dim, act, 0, 0)
    dw, db = (torch.empty(dim, device="cuda") for _ in range(2))
    zf.zero_layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, dx.t, dw, db, ws, nbytes)
    R.check(dx.t, ref["grad_x"], ref["d_x"], "grad_x")
    R.check(dw, ref["grad_weight"], ref["d_weight"], "grad_weight")
    R.check(db, ref["grad_bias"], ref["d_bias"], "grad_bias")
    dx.check_guard("grad_x")
    zf.zero_layer_norm_grad(dy.t, x.t, w.t[0], mean, rstd, x.t, None, None, ws, nbytes)
    assert torch.equal(_bits(x.t), _bits(dx.t))


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n,dim", [(2, 3), (700, 33), (900, 1501), (7, 2049), (900, 4001),
                                   (400, 8190), (3, 9001)])
def test_layer_norm_of_rows_off_the_16_byte_grid(n, dim, act):
    """Every matrix at a start and a stride of its own; in place; the same bits
    from call to call."""
    g = _gen("off the grid", n, dim)
    x = Guarded(n, dim, act, 1, 1, torch.randn((n, dim), generator=g) * 2 + 0.5)
    dy = Guarded(n, dim, act, 3, 2, torch.randn((n, dim), generator=g) * 0.1)
    out, dx = Guarded(n, dim, act, 2, 3), Guarded(n, dim, act, 4, 5)
    w, b = (torch.randn(dim, generator=g).to(act).cuda() for _ in range(2))
    mean, rstd = (torch.empty(n, device="cuda") for _ in range(2))
    zf.zero_layer_norm(x.t, w, b, 1e-5, out.t, mean, rstd)
    ref = R.layer_norm(x.t, w, b, 1e-5)
    R.check(out.t, ref["out"], ref["d_out"], "out")
    out.check_guard("out")
    nbytes = zf.zero_layer_norm_grad_workspace_bytes(n, dim)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(w)
    zf.zero_layer_norm_grad(dy.t, x.t, w, mean, rstd, dx.t, dw, db, ws, nbytes)
    ref = R.layer_norm_grad(dy.t, x.t, w, mean, rstd, max(1, nbytes // (8 * dim)))
    R.check(dx.t, ref["grad_x"], ref["d_x"], "grad_x")
    R.check(dw, ref["grad_weight"], ref["d_weight"], "grad_weight")
    R.check(db, ref["grad_bias"], ref["d_bias"], "grad_bias")
    dx.check_guard("grad_x")
    again, dw2, db2 = dx.t.clone(), torch.empty_like(w), torch.empty_like(w)
    zf.zero_layer_norm_grad(dy.t, x.t, w, mean, rstd, dy.t, dw2, db2, ws, nbytes)
    for p, q in ((dy.t, again), (dw2, dw), (db2, db)):
        assert torch.equal(_bits(p), _bits(q))
    dy.check_guard("grad_out")
    again = out.t.clone()
    zf.zero_layer_norm(x.t, w, b, 1e-5, x.t)
    assert torch.equal(_bits(x.t), _bits(again))
    x.check_guard("x")


def test_layer_norm_of_no_rows():
    none = torch.empty((0, 12), device="cuda")
    stat = torch.empty(0, device="cuda")
    zf.zero_layer_norm(none, None, None, 1e-5, none, stat, stat)
    dw, db = (torch.full((12,), 5.0, device="cuda") for _ in range(2))
    nbytes = zf.zero_layer_norm_grad_workspace_bytes(0, 12)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    zf.zero_layer_norm_grad(none, none, None, stat, stat, none, dw, db, ws, nbytes)
    assert not dw.any() and not db.any()


def test_layer_norm_of_a_constant_row_and_of_nan():
    x = torch.full((3, 40), 2.0, device="cuda")
    x[1, 7] = float("nan")
    out = torch.empty_like(x)
    b = torch.arange(40, device="cuda", dtype=F32)
    zf.zero_layer_norm(x, None, b, 1e-5, out)
    assert torch.equal(out[0], b) and torch.equal(out[2], b)
    assert bool(torch.isnan(out[1]).all())


# ----------------------------------------------------------- distillation ----

LOSSES = [
    # rows, vocab, top, pad columns, flat offset
    (1, 1, 1, 0, 0), (4, 2, 3, 0, 1), (3, 7, 5, 1, 0), (5, 31, 4, 0, 3), (2, 1000, 64, 8, 8),
    (6, 1001, 33, 0, 0), (7, 4099, 17, 3, 1), (3, 50257, 64, 0, 0), (2, 50257, 1, 0, 5),
    (1, 131072, 128, 0, 0), (5, 65536, 1024, 0, 0), (2, 131073, 40, 0, 1), (1, 300007, 8, 0, 0),
]


def _distill_inputs(n, vocab, top, pad, offset, dtype, teacher, key=()):
    g = _gen("distill", n, vocab, top, *key)
    z = Guarded(n, vocab, dtype, pad, offset, torch.randn((n, vocab), generator=g) * 3)
    ids = torch.randint(0, vocab, (n, top), generator=g, dtype=torch.int32)
    gone = torch.rand((n, top), generator=g) < 0.1
    ids[gone] = -1
    t = (torch.randn((n, top), generator=g) * 2).to(teacher).cuda()
    w = (torch.rand(n, generator=g) + 0.1).cuda()
    return z, ids.cuda(), t, w


def _run_distill(z, ids, t, w, tau, pad=0, offset=0):
    """Loss alone, loss with gradient, and the same in place."""
    n, vocab = z.shape
    alone, loss = (torch.full((n,), -1.0, device="cuda") for _ in range(2))
    zf.zero_distill_loss(z, ids, t, w, tau, alone)
    dz = Guarded(n, vocab, z.dtype, pad, offset)
    zf.zero_distill_loss_grad(z, ids, t, w, tau, loss, dz.t)
    dz.check_guard("grad_logits")
    return alone, loss, dz.t


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.5])
@pytest.mark.parametrize("dtype,teacher", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,vocab,top,pad,offset", LOSSES)
def test_distill(n, vocab, top, pad, offset, dtype, teacher, tau):
    z, ids, t, w = _distill_inputs(n, vocab, top, pad, offset, dtype, teacher)
    ref = R.distill(z.t, ids, t, w, tau)
    # the gradient at another alignment than the logits', and at the same one
    for gpad, goff in ((pad, offset), (pad + 1, offset + 1)):
        alone, loss, dz = _run_distill(z.t, ids, t, w, tau, gpad, goff)
        R.check(alone, ref["loss"], ref["d_loss"], "loss alone")
        R.check(loss, ref["loss"], ref["d_loss"], "loss")
        R.check(dz, ref["grad"], ref["d_grad"], "grad_logits")
    _, _, same = _run_distill(z.t, ids, t, w, tau, pad, offset)
    loss = torch.empty(n, device="cuda")
    zf.zero_distill_loss_grad(z.t, ids, t, w, tau, loss, z.t)
    assert torch.equal(_bits(z.t), _bits(same)), "in place differs"
    z.check_guard("logits")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [24, 100, 300])
@pytest.mark.parametrize("vocab", [1000, 16001, 50257])
def test_distill_many_rows(vocab, top, dtype):
    """More rows than the GPU holds at once, in every CTA shape; masked rows
    among them, rows with equal ids; repeats bit for bit."""
    n = 700
    z, ids, t, w = _distill_inputs(n, vocab, top, 0, 0, dtype, dtype, ("many",))
    w[::3] = 0.0
    w[5:60] = 0.0
    ids[7] = -1
    ref = R.distill(z.t, ids, t, w, 2.0)
    runs = [_run_distill(z.t, ids, t, w, 2.0) for _ in range(3)]
    alone, loss, dz = runs[0]
    R.check(alone, ref["loss"], ref["d_loss"], "loss alone")
    R.check(loss, ref["loss"], ref["d_loss"], "loss")
    R.check(dz, ref["grad"], ref["d_grad"], "grad_logits")
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("vocab,top", [(4000, 128), (20000, 130), (50257, 200)])
def test_distill_equal_ids_among_many(vocab, top):
    """Rows with more entries than are compared one by one: all distinct, two of
    one id at the ends, every id twice, one id only."""
    n = 640
    z, ids, t, w = _distill_inputs(n, vocab, top, 0, 0, BF16, F32, ("equal",))
    ids[:] = torch.arange(top, dtype=torch.int32, device="cuda") * 29 \
        + torch.arange(n, dtype=torch.int32, device="cuda")[:, None] % 97
    ids %= vocab
    ids[1::4, -1] = ids[1::4, 0]
    ids[2::4, 1::2] = ids[2::4, 0::2]
    ids[3::4] = ids[3::4, :1]
    ref = R.distill(z.t, ids, t, w, 1.0)
    _, loss, dz = _run_distill(z.t, ids, t, w, 1.0)
    R.check(loss, ref["loss"], ref["d_loss"], "loss")
    R.check(dz, ref["grad"], ref["d_grad"], "grad_logits")


def test_distill_teacher_at_the_ends_of_its_range():
    """Teacher logits of the type's lowest value only (a row of equal ones), far
    beyond the exponents' range, and one entry at +-inf."""
    n, vocab, top = 5, 3000, 8
    z, ids, t, w = _distill_inputs(n, vocab, top, 0, 0, F32, F32, ("teacher",))
    ids[:] = torch.arange(top, dtype=torch.int32, device="cuda") * 11
    t[0] = torch.finfo(F32).min
    t[1] = torch.arange(top, device="cuda") * 1e30
    t[2, 1:] = torch.finfo(F32).min
    t[3] = 1e31
    t[4, 2] = float("-inf")
    ref = R.distill(z.t, ids, t, w, 0.5)
    alone, loss, dz = _run_distill(z.t, ids, t, w, 0.5)
    R.check(alone, ref["loss"], ref["d_loss"], "alone")
    R.check(loss, ref["loss"], ref["d_loss"], "loss")
    R.check(dz, ref["grad"], ref["d_grad"], "grad")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [40, 5003, 131077])
def test_distill_masks(dtype, vocab):
    """Masked logits (-inf and the type's lowest value), masked rows holding
    NaN, rows without entries, equal ids, teacher entries of -inf."""
    n, top = 8, 6
    z, ids, t, w = _distill_inputs(n, vocab, top, 0, 0, dtype, F32, ("masks",))
    ids[:] = torch.arange(top, dtype=torch.int32, device="cuda") * 3
    low = torch.finfo(dtype).min
    z.t[0, 20:] = float("-inf")
    z.t[1, 20:] = low
    z.t[2] = low                                   # a row of equal logits
    z.t[3] = float("nan")
    w[3] = 0.0
    z.t[4] = float("inf")
    ids[4] = -1                                    # no entry: nothing leaks
    ids[5] = 9                                     # one id six times
    t[6, 2:] = float("-inf")
    t[7] = float("-inf")                           # no entry left
    ref = R.distill(z.t, ids, t, w, 1.5)
    for i in (3, 4, 7):
        ref["loss"][i], ref["grad"][i] = 0.0, 0.0
    # the row of equal logits: log(vocab) against the teacher's entropy
    ref_q = 1.0 / vocab
    p = torch.softmax(t[2].double().cpu() / 1.5, 0)
    ref["loss"][2] = float(w[2]) * 2.25 * float((p * (p.log() - np.log(ref_q))).sum())
    ref["grad"][2] = ref_q * 1.5 * float(w[2])
    ref["grad"][2, ids[2].cpu().long()] -= p * 1.5 * float(w[2])
    alone, loss, dz = _run_distill(z.t, ids, t, w, 1.5)
    R.check(alone, ref["loss"], torch.nan_to_num(ref["d_loss"]) + 1e-6 * ref["loss"].abs(), "alone")
    R.check(loss, ref["loss"], torch.nan_to_num(ref["d_loss"]) + 1e-6 * ref["loss"].abs(), "loss")
    R.check(dz, ref["grad"], ref["d_grad"] + 1e-6 * ref["grad"].abs(), "grad")
    for i in (3, 4, 7):
        assert float(loss[i]) == 0.0 and not dz[i].any()


def test_distill_non_finite_rows():
    """What a live row holds shows: NaN anywhere and +inf make the row NaN; an
    entry the student rules out makes the loss infinite."""
    z = torch.zeros((3, 600), device="cuda")
    z[0, 500] = float("nan")
    z[1, 500] = float("inf")
    z[2, 4] = float("-inf")
    ids = torch.tensor([[4, 7]] * 3, dtype=torch.int32, device="cuda")
    t = torch.zeros((3, 2), device="cuda")
    alone, loss, dz = _run_distill(z, ids, t, None, 1.0)
    for got in (alone, loss):
        assert bool(torch.isnan(got[:2]).all()) and float(got[2]) == float("inf")
    assert bool(torch.isnan(dz[0]).all()) and bool(torch.isnan(dz[1]).all())
    assert bool(torch.isfinite(dz[2]).all()) and float(dz[2, 4]) == -0.5


def test_distill_of_no_rows():
    z = torch.empty((0, 50), device="cuda")
    ids = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    t = torch.empty((0, 4), device="cuda")
    zf.zero_distill_loss_grad(z, ids, t, None, 1.0, torch.empty(0, device="cuda"), z)


def test_distill_logits_beyond_32_bit_elements():
    n, vocab = 40_000, 65_536                      # 2.6e9 elements
    z = torch.zeros((n, vocab), dtype=BF16, device="cuda")
    ids = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    t = torch.zeros((n, 1), device="cuda")
    w = torch.zeros(n, device="cuda")
    w[n - 1] = 1.0
    z[n - 1, 0] = 1.0
    z[:n - 1, 0] = float("nan")
    loss = torch.empty(n, device="cuda")
    zf.zero_distill_loss_grad(z, ids, t, w, 1.0, loss, z)
    ref = np.log(np.e + vocab - 1) - 1.0
    assert abs(float(loss[n - 1]) - ref) < 1e-5 and not loss[:n - 1].any()
    assert not z[:n - 1].any()
    assert abs(float(z[n - 1, 0]) - (np.e / (np.e + vocab - 1) - 1)) < 2.0 ** -8


@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_gradient_is_the_difference_quotient(tau):
    """fp32 losses of z +- h v, summed in 64 bits, against the kernel's
    gradient along v: off by h^2 / 6 times a third derivative of at most
    2 max|v|^3 w / tau a row, and by the rounding of the losses over h."""
    n, vocab = 5, 700
    z, ids, t, w = _distill_inputs(n, vocab, 12, 0, 0, F32, F32, ("quotient",))
    v = torch.randn((n, vocab), generator=_gen("direction"))
    v = (v / v.abs().max()).cuda()
    loss = [torch.empty(n, device="cuda") for _ in range(3)]
    dz = torch.empty_like(z.t)
    h = 2.0 ** -5
    zf.zero_distill_loss_grad(z.t, ids, t, w, tau, loss[0], dz)
    zf.zero_distill_loss((z.t + h * v).contiguous(), ids, t, w, tau, loss[1])
    zf.zero_distill_loss((z.t - h * v).contiguous(), ids, t, w, tau, loss[2])
    got = float((dz.double() * v.double()).sum())
    want = float((loss[1].double() - loss[2].double()).sum()) / (2 * h)
    ref = R.distill(z.t, ids, t, w, tau)
    # the shifted inputs are rounded too: half an ulp of |z| < 16 times |dz|
    bound = float(w.sum()) / tau * 2 * h * h / 6 + float(ref["d_loss"].sum()) / h + \
        float(ref["grad"].abs().sum()) * 16 * R.U / h
    assert abs(got - want) <= bound, (got, want, bound)


# ----------------------------------------------------- streams and graphs ----

def _mixed_calls(stream=None):
    """A closure running all eight calls on its own buffers, and its results."""
    g = _gen("mixed")
    n, vocab, dim, top = 96, 1003, 264, 8
    ids = torch.randint(0, vocab, (n,), generator=g).cuda()
    w = torch.randn((vocab, dim), generator=g).to(BF16).cuda()
    lw, lb = (torch.randn(dim, generator=g).to(BF16).cuda() for _ in range(2))
    x, y, dx = (torch.zeros((n, dim), dtype=BF16, device="cuda") for _ in range(3))
    mean, rstd, loss, alone = (torch.zeros(n, device="cuda") for _ in range(4))
    z = torch.randn((n, vocab), generator=g).to(BF16).cuda()
    dz = torch.zeros_like(z)
    tid = torch.randint(0, vocab, (n, top), generator=g, dtype=torch.int32).cuda()
    t = torch.randn((n, top), generator=g).cuda()
    dw = torch.zeros((vocab, dim), dtype=BF16, device="cuda")
    dlw, dlb = (torch.zeros(dim, dtype=BF16, device="cuda") for _ in range(2))
    b1 = zf.zero_embedding_grad_workspace_bytes(n, vocab, dim)
    b2 = zf.zero_layer_norm_grad_workspace_bytes(n, dim)
    ws1, ws2 = (torch.empty(b, dtype=torch.uint8, device="cuda") for b in (b1, b2))

    def call():
        zf.zero_embedding(ids, w, x, 2.0, stream=stream)
        zf.zero_layer_norm(x, lw, lb, 1e-5, y, mean, rstd, stream=stream)
        zf.zero_distill_loss(z, tid, t, None, 2.0, alone, stream=stream)
        zf.zero_distill_loss_grad(z, tid, t, None, 2.0, loss, dz, stream=stream)
        zf.zero_layer_norm_grad(y, x, lw, mean, rstd, dx, dlw, dlb, ws2, b2, stream=stream)
        zf.zero_embedding_grad(ids, dx, dw, 2.0, False, ws1, b1, stream=stream)
        zf.zero_embedding_grad(ids, dx, dw, 2.0, True, ws1, b1, stream=stream)

    return call, [x, y, mean, rstd, alone, loss, dz, dx, dlw, dlb, dw]


def test_streams_give_the_same_bits():
    ref_call, ref = _mixed_calls()
    ref_call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s if i < 2 else torch.cuda.current_stream()):
            call, out = _mixed_calls(s if i == 2 else None)
        torch.cuda.synchronize()
        runs.append((s, call, out))
    for _ in range(5):
        for i, (s, call, _) in enumerate(runs):
            with torch.cuda.stream(s if i < 2 else torch.cuda.current_stream()):
                call()
    torch.cuda.synchronize()
    for _, _, out in runs:
        for a, b in zip(ref, out):
            assert torch.equal(_bits(a), _bits(b))
    assert zf.zero_device_status() == zf.zero.ZERO_DEVICE_OK


def test_capture_into_a_graph():
    ref_call, ref = _mixed_calls()
    ref_call()
    call, out = _mixed_calls()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for o in out:
        o.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, out):
        assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("label", ["embedding gradient launch", "layer norm gradient launch",
                                   "layer norm gradient reduction",
                                   "distillation loss and gradient"])
def test_injected_failure_is_reported_and_a_retry_is_clean(monkeypatch, label):
    ref_call, ref = _mixed_calls()
    ref_call()
    call, out = _mixed_calls()
    monkeypatch.setenv("ZERO_INJECT_FAILURE", label)
    with pytest.raises(zf.ZeroError) as ei:
        call()
    assert ei.value.code == -4 and label in str(ei.value)
    monkeypatch.delenv("ZERO_INJECT_FAILURE")
    call()
    torch.cuda.synchronize()
    for a, b in zip(ref, out):
        assert torch.equal(_bits(a), _bits(b))
