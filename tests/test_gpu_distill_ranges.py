"""The distillation loss where logits are spread over the types' ranges:
mask values that are finite, rows far from zero, in every shape of CTA."""
import pytest
import torch

import distill_bounds as D

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
    return torch.Generator(device="cuda").manual_seed(seed_for("distill-ranges", *key))


def _inputs(n, vocab, top, dtype, teacher, *key):
    g = _gen(n, vocab, top, *key)
    z = (torch.randn((n, vocab), generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, vocab, (n, top), generator=g, device="cuda", dtype=torch.int32)
    t = (torch.randn((n, top), generator=g, device="cuda") * 2).to(teacher)
    w = torch.rand(n, generator=g, device="cuda") + 0.1
    return z, ids, t, w


def _compare(z, ids, t, w, tau):
    """Loss alone, loss with gradient, and in place, against 64 bits."""
    n = z.shape[0]
    ref = D.distill(z, ids, t, w, tau)
    alone, loss, again = (torch.full((n,), -1.0, device="cuda") for _ in range(3))
    zf.zero_distill_loss(z, ids, t, w, tau, alone)
    dz = torch.full_like(z, -7.0)
    zf.zero_distill_loss_grad(z, ids, t, w, tau, loss, dz)
    D.check(alone, ref["loss"], ref["d_loss"], "loss alone")
    D.check(loss, ref["loss"], ref["d_loss"], "loss")
    D.check(dz, ref["grad"], ref["d_grad"], "grad_logits")
    zf.zero_distill_loss_grad(z, ids, t, w, tau, again, z)
    assert torch.equal(again, loss) and torch.equal(z, dz), "in place differs"


# rows, vocab, top of bf16 (in fp32 half the vocabulary): CTAs of 4, 8 and 16
# warps, few rows in clusters, rows beyond shared memory, ids found equal by hashing
SHAPES = [(320, 3001, 24), (320, 16001, 24), (100, 50257, 24), (6, 50257, 24), (9, 131077, 100),
          (78, 70001, 24), (320, 4001, 200)]
MASKS = [-1e9, -1e10, -1e12, -1e20, -1e30]


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.37])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab,top", SHAPES)
def test_finite_masks(n, vocab, top, dtype, tau):
    """Row i: mask value i % 5 in a prefix of the row, in all but a few columns,
    in every other column or in the whole row; large positive logits."""
    vocab = vocab if dtype == BF16 else (vocab + 1) // 2
    z, ids, t, w = _inputs(n, vocab, top, dtype, F32, "masks")
    for i in range(n):
        m, kind = MASKS[i % 5], i // 5 % 6
        if kind == 0:
            z[i, :vocab // 2] = m
        elif kind == 1:
            keep = z[i, vocab - 5:].clone()
            z[i] = m
            z[i, vocab - 5:] = keep
        elif kind == 2:
            z[i, i % 2::2] = m
        elif kind == 3:
            z[i] = m
        elif kind == 4:
            z[i] = -m
        else:
            z[i, ids[i, :2].long()] = 3e10
    _compare(z, ids, t, w, tau)


@pytest.mark.parametrize("mask", MASKS + [3e10, 2.0 ** 22, -2.0 ** 22, -2.0 ** 31])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab,top", [(3, 50257, 24), (4, 4001, 70)])
def test_every_row_masked_alike(n, vocab, top, dtype, mask):
    """Whole rows at one value, and a prefix of it: few rows, every mask."""
    z, ids, t, w = _inputs(n, vocab, top, dtype, dtype, "alike")
    z[0] = mask
    z[1:, :vocab - 900] = mask
    _compare(z, ids, t, w, 1.0)


@pytest.mark.parametrize("level", [0.0, 30.0, -700.0, 5e3, -5e3, 3e5, -2e6, 1e8, -1e12])
@pytest.mark.parametrize("teacher", [BF16, F32])
@pytest.mark.parametrize("n,vocab,top", [(5, 3001, 24), (320, 4001, 200), (6, 50257, 70)])
def test_teacher_far_from_zero(n, vocab, top, teacher, level):
    """A teacher's logits that share a level, as unnormalised ones may: only
    their differences count."""
    z, ids, t, w = _inputs(n, vocab, top, F32, F32, "level")
    t = (t + level).to(teacher)
    _compare(z, ids, t, w, 0.7)


def test_teacher_of_widely_spread_entries():
    """Entries that lie 1e30 apart, and one among entries of the type's lowest
    value: the largest takes all, and nothing else is off."""
    z, ids, t, w = _inputs(4, 3001, 8, F32, F32, "spread")
    ids[:] = torch.arange(8, dtype=torch.int32, device="cuda") * 11
    t[0] = torch.arange(8, device="cuda") * 1e30
    t[1, 1:] = torch.finfo(F32).min
    t[2, ::2] = -1e9
    t[3, 3:] = -1e20
    _compare(z, ids, t, w, 0.5)


@pytest.mark.parametrize("tau", [1e-22, 1e-18, 1e-8, 1e-3, 1e4, 1e15])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_temperatures_far_from_one(dtype, tau):
    """Loss and gradient scale with the temperature, whose square may be too
    small for fp32."""
    z, ids, t, w = _inputs(6, 3001, 24, dtype, F32, "temperature")
    _compare(z, ids, t, w, tau)
