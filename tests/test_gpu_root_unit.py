"""The root unit's forward and backward pass (examples/distill_root_unit.py)
against autograd in 64 bits on the same parameters and tokens, and a short
training run whose loss falls."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location(
        "distill_root_unit", os.path.join(ROOT, "examples", "distill_root_unit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("vocab,context,dim", [(503, 16, 64), (777, 24, 50)])
def test_gradients_against_autograd(ex, vocab, context, dim):
    """Relative 2-norm errors: every tensor between the operators is bf16 (8
    bits, half an ulp is 2^-8 of a value), and about ten such roundings lie
    between the parameters and a gradient, so 10 * 2^-8 = 0.04 bounds their sum
    if none is amplified; the norm divides by a standard deviation near one."""
    tokens, top, tau = 3 * context, 5, 1.5
    root = ex.RootUnit(vocab, context, dim, 2, seed=3)
    b = ex.Buffers(root, tokens)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    pos = torch.arange(context, device="cuda", dtype=torch.int32).repeat(3)
    tid = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:top]
                       for _ in range(tokens)]).to(torch.int32)
    t = torch.randn((tokens, top), generator=g, device="cuda")
    w = torch.rand(tokens, generator=g, device="cuda")
    w[::context] = 0.0
    ex.rank_pass(root, 1, b, ids, pos, tid, t, w, tau)
    got = root.views(root.unit.grads[1])

    p = {k: v.double().requires_grad_() for k, v in root.views(root.unit.params[0]).items()}
    x = p["wte"][ids] * dim ** 0.5 + p["wpe"][pos.long()]
    y = torch.nn.functional.layer_norm(x, (dim,), p["ln_w"], p["ln_b"], ex.EPS)
    logq = torch.log_softmax(y @ p["wte"].t() / tau, 1)
    pt = torch.softmax(t.double() / tau, 1)
    kl = (pt * (pt.log() - torch.gather(logq, 1, tid.long()))).sum(1)
    loss = w.double() * tau * tau * kl
    loss.sum().backward()
    assert float((b.loss.double() - loss.detach()).norm() / loss.detach().norm()) < 0.04
    for name, want in p.items():
        err = float((got[name].double() - want.grad).norm() / want.grad.norm())
        assert err < 0.04, (name, err)
    # the other rank's gradient is untouched
    assert not root.unit.grads[0].any()


def test_training_lowers_the_loss(ex):
    losses = ex.train(12, n_ranks=3, vocab=1009, context=32, dim=128, sequences=4)
    assert all(l == l for l in losses) and losses[-1] < losses[0], losses
