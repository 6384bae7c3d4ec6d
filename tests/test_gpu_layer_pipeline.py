"""The norm, its checkpoint in 8 bits, the head's loss and their gradients one
after another, into ranks' flat gradients, and the sharded step on them: a
model's last norm and its head, against autograd in 64 bits."""
import pytest
import torch

import layer_reference as L

import fsdp_sharded_mixed_flatten_gb300 as zf
from fsdp_sharded_mixed_flatten_gb300.buffers import FlatUnit
from fsdp_sharded_mixed_flatten_gb300.synthetic import ADAMW_DEFAULTS

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


class Head:
    """A unit of the head's table and the last norm's weight, and one rank's pass."""

    def __init__(self, vocab, dim, n_ranks, tokens):
        self.vocab, self.dim, self.tokens = vocab, dim, tokens
        self.unit = FlatUnit([vocab * dim, dim], n_ranks)
        g = torch.Generator().manual_seed(11)
        flat = torch.zeros(self.unit.P_pad)
        flat[:vocab * dim] = torch.randn(vocab * dim, generator=g) * 0.05
        flat[vocab * dim:vocab * dim + dim] = 1.0 + 0.1 * torch.randn(dim, generator=g)
        self.unit.set_master_flat(flat.cuda())
        self.unit.params[0].copy_(flat.cuda())
        rows = lambda: torch.zeros((tokens, dim), dtype=BF16, device="cuda")     # noqa: E731
        self.total, self.h, self.dh, self.again = rows(), rows(), rows(), rows()
        self.rstd, self.loss, self.lse = (torch.zeros(tokens, device="cuda") for _ in range(3))
        self.kept = (torch.zeros((tokens, dim), dtype=torch.float8_e4m3fn, device="cuda"),
                     torch.zeros((tokens, (dim + 127) // 128), device="cuda"))
        self.bytes = max(zf.zero_head_loss_workspace_bytes(tokens, vocab, dim),
                         zf.zero_head_loss_grad_workspace_bytes(tokens, vocab, dim),
                         zf.zero_rms_norm_grad_workspace_bytes(tokens, dim))
        self.ws = torch.empty(self.bytes, dtype=torch.uint8, device="cuda")

    def views(self, flat):
        n = self.vocab * self.dim
        return flat[:n].view(self.vocab, self.dim), flat[n:n + self.dim]

    def rank_pass(self, rank, x, residual, labels, grad_loss, grad_total, accumulate=False):
        table, weight = self.views(self.unit.params[0])
        d_table, d_weight = self.views(self.unit.grads[rank])
        zf.zero_rms_norm(x, residual, weight, EPS, self.h, self.total, self.rstd, None, self.kept)
        zf.zero_head_loss(self.h, table, labels, self.loss, self.lse, self.ws, self.bytes)
        zf.zero_head_loss_grad(self.h, table, labels, self.lse, grad_loss, self.dh, d_table,
                               accumulate, self.ws, self.bytes)
        # the norm's input comes from the 8 bits; the gradient in place of dh
        zf.zero_rms_norm_grad(self.dh, self.kept, weight, self.rstd, self.dh, d_weight, grad_total,
                              self.again, self.ws, self.bytes)


def _inputs(key, tokens, dim, vocab):
    g = torch.Generator().manual_seed(key)
    x, residual = (torch.randn((tokens, dim), generator=g).to(BF16).cuda() for _ in range(2))
    through = (torch.randn((tokens, dim), generator=g) * 1e-3).to(BF16).cuda()
    labels = torch.randint(0, vocab, (tokens,), generator=g)
    labels[torch.rand(tokens, generator=g) < 0.25] = -100
    grad_loss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    return x, residual, labels.cuda(), grad_loss, through


def _close(got, want, roundings, what):
    """Relative 2-norm error: `roundings` bf16 roundings (2^-8 of a value at most) lie on the
    way, and none is amplified (the norm divides by about 1.4)."""
    err = float((got.double() - want).norm() / want.norm())
    assert err <= roundings * 2.0 ** -8, (what, err)


@pytest.mark.parametrize("vocab,dim,tokens", [(1009, 64, 96), (5003, 200, 300), (777, 130, 50)])
def test_pass_against_autograd(vocab, dim, tokens):
    head = Head(vocab, dim, 2, tokens)
    x, residual, labels, grad_loss, through = _inputs(1, tokens, dim, vocab)
    head.rank_pass(1, x, residual, labels, grad_loss, through)
    table, weight = (p.double() for p in head.views(head.unit.params[0]))
    s = (x.float() + residual.float()).double()
    # autograd through the norm at the values that the checkpoint holds
    kept = torch.from_numpy(L.unpack(head.kept[0].view(torch.uint8).cpu().numpy(),
                                     head.kept[1].cpu().numpy())).cuda()
    assert bool(((kept - s).abs() <= L.eight_bound(s.cpu(), 0 * s.cpu()).cuda()).all())
    table.requires_grad_()
    h = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * weight
    _close(head.total, s, 1, "total")
    _close(head.h, h, 1, "h")
    h = h.requires_grad_()
    each = torch.nn.functional.cross_entropy(h @ table.t(), labels, reduction="none",
                                             ignore_index=-100)
    (each * grad_loss.double()).sum().backward()
    _close(head.loss, each.detach(), 2, "loss")
    d_table, d_weight = head.views(head.unit.grads[1])
    _close(d_table, table.grad, 4, "table")              # h, dz, itself; h again in z
    k, w = kept.clone(), weight.clone()
    r = head.rstd.double()[:, None]
    (dx, _), (dw, _), (again, _) = L.rms_norm_grad(h.grad.cpu(), k.cpu(), w.cpu(), head.rstd,
                                                   through)
    _close(head.dh, dx.cuda(), 6, "x")
    _close(d_weight, dw.cuda(), 6, "weight")
    _close(head.again, again.cuda(), 1, "h again")
    assert float((r * k * w - head.h.double()).abs().max()) < 1.0     # (the same numbers at all)
    assert not head.unit.grads[0].any()


def test_ranks_gradients_and_the_step():
    """Two ranks, two micro-batches each in place of one another (accumulate), one step: the
    parameters are AdamW's first step on the mean of the ranks' gradients."""
    vocab, dim, tokens, lr = 1009, 72, 80, 1e-3
    head = Head(vocab, dim, 2, tokens)
    before = head.unit.master.reshape(-1)[:vocab * dim + dim].double().clone()
    for rank in range(2):
        for micro in range(2):
            x, residual, labels, grad_loss, through = _inputs(10 * rank + micro, tokens, dim, vocab)
            head.rank_pass(rank, x, residual, labels, grad_loss, through, accumulate=micro > 0)
    n = vocab * dim + dim
    g = (head.unit.grads[0][:n].double() + head.unit.grads[1][:n].double()) / 2
    u = head.unit
    zf.zero_step(u.grad_rows(), *u.state_rows(), None, 1, 1, u.param_rows(), u.layout,
                 dict(ADAMW_DEFAULTS, lr=lr, step=1))
    hp = ADAMW_DEFAULTS
    want = before * (1 - lr * hp["weight_decay"]) - lr * g / (g.abs() + hp["eps"])
    # the master is the step's fp32 result to 1e-6 of itself and 1e-7 (the step's own bound)
    got = u.master.reshape(-1)[:n].double()
    assert bool(((got - want).abs() <= 1e-6 * want.abs() + 2e-7).all())


def test_a_captured_step_replays():
    """The whole pass in a graph, its labels changed between replays (other live tokens)."""
    vocab, dim, tokens = 1009, 64, 96
    head = Head(vocab, dim, 1, tokens)
    x, residual, labels, grad_loss, through = _inputs(3, tokens, dim, vocab)
    other = _inputs(4, tokens, dim, vocab)[2]
    results = []
    for y in (labels, other):
        head.rank_pass(0, x, residual, y, grad_loss, through)
        results.append([t.clone() for t in (head.loss, head.dh, head.unit.grads[0])])
    y = labels.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        head.rank_pass(0, x, residual, y, grad_loss, through)
    for which, want in ((other, results[1]), (labels, results[0])):
        y.copy_(which)
        head.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((head.loss, head.dh, head.unit.grads[0]), want):
            assert torch.equal(a, b)
