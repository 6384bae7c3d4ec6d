"""Train the root unit of a language model (token table tied with the head,
position table, final layer norm) against a teacher's top logits, over several
logical data-parallel ranks in one GPU.

Each rank runs forward and backward on its own tokens: lookup, layer norm, the
head's product, the distillation loss with its gradient, and back.  Parameters
are read from the unit's gathered flat buffer and gradients written straight
into the rank's flat gradient, at the tensors' offsets; one zero_step then
averages the ranks' gradients, updates the sharded fp32 state and gathers the
new parameters.

    python examples/distill_root_unit.py [--steps 20] [--ranks 4]

The teacher's entries are synthetic: a fixed random table of the next token's
logits, of which the best few per token are stored.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fsdp_sharded_mixed_flatten_gb300 as zf  # noqa: E402
from fsdp_sharded_mixed_flatten_gb300.buffers import FlatUnit  # noqa: E402
from fsdp_sharded_mixed_flatten_gb300.synthetic import ADAMW_DEFAULTS  # noqa: E402

EPS = 1e-5


class RootUnit:
    """The unit's flat buffers, and views of its four tensors in them."""

    def __init__(self, vocab: int, context: int, dim: int, n_ranks: int, seed: int = 0):
        self.vocab, self.context, self.dim, self.n_ranks = vocab, context, dim, n_ranks
        self.shapes = {"wte": (vocab, dim), "wpe": (context, dim), "ln_w": (dim,), "ln_b": (dim,)}
        numels = [torch.Size(s).numel() for s in self.shapes.values()]
        self.unit = FlatUnit(numels, n_ranks)
        g = torch.Generator().manual_seed(seed)
        flat = torch.zeros(self.unit.P_pad)
        for (name, shape), off, n in zip(self.shapes.items(), self.unit.offsets, numels):
            flat[off:off + n] = 1.0 if name == "ln_w" else 0.0 if name == "ln_b" else \
                0.02 * torch.randn(n, generator=g)
        self.unit.set_master_flat(flat.cuda())
        self.unit.params[0].copy_(flat.cuda())

    def views(self, flat: torch.Tensor):
        """The unit's tensors in a flat buffer (parameters or a rank's gradient)."""
        out = {}
        for (name, shape), off in zip(self.shapes.items(), self.unit.offsets):
            out[name] = flat[off:off + torch.Size(shape).numel()].view(shape)
        return out

    def step(self, t: int, lr: float):
        u = self.unit
        zf.zero_step(u.grad_rows(), *u.state_rows(), None, 1, 1, u.param_rows(), u.layout,
                     dict(ADAMW_DEFAULTS, lr=lr, step=t))


class Buffers:
    """What one rank's pass needs besides the unit, kept over the steps."""

    def __init__(self, root: RootUnit, tokens: int):
        d, dev = root.dim, "cuda"
        rows = dict(device=dev, dtype=torch.bfloat16)
        self.tok, self.pos, self.x, self.y, self.dy, self.dx = (
            torch.empty((tokens, d), **rows) for _ in range(6))
        self.logits = torch.empty((tokens, root.vocab), **rows)
        self.mean, self.rstd, self.loss = (torch.empty(tokens, device=dev) for _ in range(3))
        self.bytes = max(
            zf.zero_embedding_grad_workspace_bytes(tokens, root.vocab, d),
            zf.zero_embedding_grad_workspace_bytes(tokens, root.context, d),
            zf.zero_layer_norm_grad_workspace_bytes(tokens, d), 16)
        self.workspace = torch.empty(self.bytes, device=dev, dtype=torch.uint8)


def rank_pass(root: RootUnit, rank: int, b: Buffers, ids, positions, teacher_ids, teacher_logits,
              weights, temperature: float):
    """Forward and backward of one rank: fills its flat gradient, and b.loss."""
    p = root.views(root.unit.params[0])
    g = root.views(root.unit.grads[rank])
    scale = root.dim ** 0.5
    zf.zero_embedding(ids, p["wte"], b.tok, scale)
    zf.zero_embedding(positions, p["wpe"], b.pos)
    torch.add(b.tok, b.pos, out=b.x)
    zf.zero_layer_norm(b.x, p["ln_w"], p["ln_b"], EPS, b.y, b.mean, b.rstd)
    torch.mm(b.y, p["wte"].t(), out=b.logits)
    # the loss, and its gradient in place of the logits
    zf.zero_distill_loss_grad(b.logits, teacher_ids, teacher_logits, weights, temperature, b.loss,
                              b.logits)
    torch.mm(b.logits, p["wte"], out=b.dy)
    torch.mm(b.logits.t(), b.y, out=g["wte"])             # the head's part of the tied table
    zf.zero_layer_norm_grad(b.dy, b.x, p["ln_w"], b.mean, b.rstd, b.dx, g["ln_w"], g["ln_b"],
                            b.workspace, b.bytes)
    zf.zero_embedding_grad(ids, b.dx, g["wte"], scale, True, b.workspace, b.bytes)
    zf.zero_embedding_grad(positions, b.dx, g["wpe"], 1.0, False, b.workspace, b.bytes)


def train(steps: int, n_ranks: int = 4, vocab: int = 5003, context: int = 128, dim: int = 256,
          sequences: int = 4, top: int = 16, temperature: float = 2.0, lr: float = 1e-3,
          seed: int = 0):
    """Mean loss per token of every step."""
    root = RootUnit(vocab, context, dim, n_ranks, seed)
    tokens = sequences * context
    b = Buffers(root, tokens)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    positions = torch.arange(context, device="cuda", dtype=torch.int32).repeat(sequences)
    best = torch.randint(0, vocab, (vocab, top), generator=g, device="cuda", dtype=torch.int32)
    level = torch.rand((vocab, top), generator=g, device="cuda").mul_(6.0)
    losses = []
    for t in range(1, steps + 1):
        total = torch.zeros((), device="cuda")
        for r in range(n_ranks):
            ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
            weights = torch.full((tokens,), 1.0 / tokens, device="cuda")
            weights[::context] = 0.0                      # a first token has no target
            rank_pass(root, r, b, ids, positions, best[ids], level[ids], weights, temperature)
            total += b.loss.sum() / n_ranks
        root.step(t, lr)
        losses.append(total)
    return [float(x) for x in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    for t, loss in enumerate(train(a.steps, a.ranks), 1):
        print(f"step {t:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
