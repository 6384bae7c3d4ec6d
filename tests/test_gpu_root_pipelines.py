"""Several rows of work one after another in the kernels around the root unit:
rows copied ahead, slots used again, results in place of inputs still to come,
sorts of three passes, sums over many groups of columns."""
import pytest
import torch

import distill_bounds as D
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
    return torch.Generator(device="cuda").manual_seed(seed_for("root-pipelines", *key))


# more than two rows for every group of threads that 152 SMs hold
NORMS = [(4001, 768), (9001, 96), (2001, 2048), (1501, 4096), (901, 8192), (401, 16384)]


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n,dim", NORMS)
def test_layer_norm_on_the_grid(n, dim, act):
    g = _gen("norm", n, dim)
    x = (torch.randn((n, dim), generator=g, device="cuda") * 2
         + torch.randn((n, 1), generator=g, device="cuda")).to(act)
    dy = (torch.randn((n, dim), generator=g, device="cuda") * 0.1).to(act)
    w, b = (torch.randn(dim, generator=g, device="cuda").to(act) for _ in range(2))
    out, dx, dw, db = (torch.empty_like(t) for t in (x, x, w, b))
    mean, rstd = (torch.empty(n, device="cuda") for _ in range(2))
    zf.zero_layer_norm(x, w, b, 1e-5, out, mean, rstd)
    ref = R.layer_norm(x, w, b, 1e-5)
    R.check(mean, ref["mean"], ref["d_mean"], "mean")
    R.check(rstd, ref["rstd"], ref["d_rstd"] + 4 * R.U * ref["rstd"], "rstd")
    R.check(out, ref["out"], ref["d_out"], "out")
    nbytes = zf.zero_layer_norm_grad_workspace_bytes(n, dim)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    zf.zero_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, ws, nbytes)
    ref = R.layer_norm_grad(dy, x, w, mean, rstd, max(1, nbytes // (8 * dim)))
    R.check(dx, ref["grad_x"], ref["d_x"], "grad_x")
    R.check(dw, ref["grad_weight"], ref["d_weight"], "grad_weight")
    R.check(db, ref["grad_bias"], ref["d_bias"], "grad_bias")
    # in place of either input, and of x forward: the same bits
    dw2, db2, dy2 = torch.empty_like(w), torch.empty_like(b), dy.clone()
    zf.zero_layer_norm_grad(dy2, x, w, mean, rstd, dy2, dw2, db2, ws, nbytes)
    assert torch.equal(dy2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    x2 = x.clone()
    zf.zero_layer_norm_grad(dy, x2, w, mean, rstd, x2, None, None, ws, nbytes)
    assert torch.equal(x2, dx)
    zf.zero_layer_norm(x, w, b, 1e-5, x)
    assert torch.equal(x, out)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("n,vocab,dim", [(20011, 300007, 24),      # three passes of the sort
                                         (17001, 2 ** 18, 16),     # the least vocabulary of three
                                         (17001, 801, 600),        # three groups of columns
                                         (16500, 401, 2104)])      # nine, in two blocks
def test_table_gradient_by_sorted_tokens(n, vocab, dim, types, accumulate):
    g = _gen("table", n, vocab, dim)
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    hot = torch.rand(n, generator=g, device="cuda")
    ids[hot < 0.2] = vocab - 1                         # runs over many chunks
    ids[hot > 0.95] = vocab                            # no row
    dy = (torch.randn((n, dim), generator=g, device="cuda") * 0.01).to(types[0])
    old = (torch.randn((vocab, dim), generator=g, device="cuda") * 0.01).to(types[1])
    nbytes = zf.zero_embedding_grad_workspace_bytes(n, vocab, dim)
    assert nbytes > 0
    ws = torch.full((nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
    dw = old.clone()
    zf.zero_embedding_grad(ids, dy, dw, 0.5, accumulate, ws, nbytes)
    ref, bound = R.embedding_grad(ids, dy, (vocab, dim), 0.5, old if accumulate else None)
    R.check(dw, ref, bound, "grad_weight")
    again = old.clone()
    zf.zero_embedding_grad(ids, dy, again, 0.5, accumulate, ws, nbytes)
    assert torch.equal(again, dw)


# rows, vocab, top of bf16 (in fp32 half the vocabulary), more rows than CTAs of
# 4, 8 and 16 warps; rows beyond shared memory; ids found equal by hashing
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab,top", [(4001, 3001, 24), (2001, 16001, 24), (901, 40009, 24),
                                         (901, 50257, 70), (451, 70001, 24), (3001, 4001, 200)])
def test_distillation_in_place(n, vocab, top, dtype):
    vocab = vocab if dtype == BF16 else (vocab + 1) // 2
    g = _gen("in place", n, vocab, top)
    z = (torch.randn((n, vocab), generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, vocab, (n, top), generator=g, device="cuda", dtype=torch.int32)
    t = torch.randn((n, top), generator=g, device="cuda") * 2
    w = torch.rand(n, generator=g, device="cuda") + 0.1
    w[::7] = 0.0
    ids[3::11] = -1
    ref = D.distill(z, ids, t, w, 1.5)
    loss, again = (torch.empty(n, device="cuda") for _ in range(2))
    dz = torch.full_like(z, -7.0)
    zf.zero_distill_loss_grad(z, ids, t, w, 1.5, loss, dz)
    D.check(loss, ref["loss"], ref["d_loss"], "loss")
    D.check(dz, ref["grad"], ref["d_grad"], "grad_logits")
    del ref
    zf.zero_distill_loss_grad(z, ids, t, w, 1.5, again, z)
    assert torch.equal(again, loss) and torch.equal(z, dz)
