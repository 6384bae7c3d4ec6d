"""What is measured of the operators of a decoder layer's norm and of the model's head:
the root-mean-square norm with the residual's addition, forward and backward, with its
results in 8 bits where wanted; activation checkpoints in 8 bits; and the softmax cross
entropy of the head in pieces of the vocabulary, without keeping the logits, with its
gradients.

Each case is one pass as a training program makes it.  `run` computes it in its plain
form (elementary torch operations in 32 bits), or, where `own` is true, through the
library's entry points.

8 bits: a row is cut into blocks of 128 columns, the last one shorter.  A block's scale
is the smallest power of two, at least 2^-126, that brings its largest magnitude to at
most 448; its values divided by the scale are rounded to e4m3.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------- cases ------

def listed():
    return [
        # One decoding step of a small batch at a Llama-3-8B layer's width, the residual
        # stream updated in place; latency is all that counts.
        dict(name="rms_norm_4x4096", op="norm", tokens=4, dim=4096, dtype="bf16", residual=True,
             pad_cols=0, offset=0),
        # Two sequences of 8192 tokens through such a layer.
        dict(name="rms_norm_16384x4096", op="norm", tokens=16384, dim=4096, dtype="bf16",
             residual=True, pad_cols=0, offset=0),
        # Odd width, rows of a wider fp32 buffer, the weight at an odd place of its flat
        # buffer; the result in 8 bits, restored for the weights' gradients.
        dict(name="rms_norm8_f32_5003x1501", op="norm8", tokens=5003, dim=1501, dtype="f32",
             residual=False, pad_cols=3, offset=37),
        # The backward pass of one sequence of 8192 tokens.
        dict(name="rms_norm_grad_8192x4096", op="norm_grad", tokens=8192, dim=4096, dtype="bf16",
             residual=True, pad_cols=0, offset=64),
        # Two sequences forward with the norm's input kept in 8 bits alone, and backward
        # from it, the norm's output made again for the weights' gradients.
        dict(name="rms_step8_16384x4096", op="step8", tokens=16384, dim=4096, dtype="bf16",
             residual=True, pad_cols=0, offset=0),
        # A feed-forward's activations of two sequences, saved and restored.
        dict(name="checkpoint_16384x14336", op="checkpoint", tokens=16384, dim=14336,
             dtype="bf16", pad_cols=0),
        # A ragged batch of odd width in fp32.
        dict(name="checkpoint_f32_1021x770", op="checkpoint", tokens=1021, dim=770, dtype="f32",
             pad_cols=1),
        # Validation of a few sequences' last tokens on GPT-2-small's table.
        dict(name="head_loss_32x50257x768", op="loss", tokens=32, vocab=50257, dim=768,
             masked=0.0, offset=0, pad_cols=0, accumulate=False),
        # Validation of a long batch, a third of it prompts without a label.
        dict(name="head_loss_8192x131072x4096", op="loss", tokens=8192, vocab=131072, dim=4096,
             masked=0.33, offset=0, pad_cols=0, accumulate=False),
        # A ragged batch with an odd vocabulary, a width that is no multiple of 8 and
        # the table at an odd place of its flat buffer.
        dict(name="head_grad_1021x32003x770", op="loss_grad", tokens=1021, vocab=32003, dim=770,
             masked=0.2, offset=37, pad_cols=2, accumulate=False),
        # GPT-2-small, 8 sequences of 1024 tokens, added to what earlier micro-batches left.
        dict(name="head_grad_8192x50257x768", op="loss_grad", tokens=8192, vocab=50257, dim=768,
             masked=0.0, offset=0, pad_cols=0, accumulate=True),
        # The largest: 8192 tokens, 131072 rows of width 4096.
        dict(name="head_grad_8192x131072x4096", op="loss_grad", tokens=8192, vocab=131072,
             dim=4096, masked=0.0, offset=0, pad_cols=0, accumulate=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm8", "norm_grad", "step8", "checkpoint", "loss",
                     "loss", "loss_grad", "loss_grad", "loss_grad"])
    if op.startswith("loss"):
        vocab = _log_int(rng, 1000, 131072)
        dim = _log_int(rng, 64, 4096)
        # mostly whole vectors, as models have them; sometimes any width
        dim = dim if rng.random() < 0.25 else (dim + 7) // 8 * 8
        return dict(op=op, vocab=vocab, dim=dim,
                    tokens=_log_int(rng, 1, min(8192, 2 ** 40 // (vocab * dim))),
                    masked=rng.choice([0.0, round(rng.uniform(0.0, 0.9), 3)]),
                    offset=rng.choice([0, 0, 8 * rng.randrange(1, 100), rng.randrange(1, 100)]),
                    pad_cols=rng.choice([0, 0, 8, rng.randrange(1, 20)]),
                    accumulate=op == "loss_grad" and rng.random() < 0.5)
    wide = op == "checkpoint"
    dim = _log_int(rng, 64, 16384 if wide else 8192)
    dim = dim if rng.random() < 0.3 else (dim + 7) // 8 * 8
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), dim=dim,
             tokens=_log_int(rng, 1, min(65536, 2 ** 26 // dim)),
             pad_cols=rng.choice([0, 0, 8, rng.randrange(1, 20)]))
    if not wide:
        c["residual"] = rng.random() < 0.7
        c["offset"] = rng.choice([0, 0, rng.randrange(1, 100)])
    return c


# -------------------------------------------------------------- inputs ------

def _rows(n, cols, pad_cols, dtype):
    """(n, cols) rows of an (n, cols + pad_cols) buffer, zeroed."""
    return torch.zeros((n, cols + pad_cols), device="cuda", dtype=dtype)[:, :cols]


def _flat(shape, offset, dtype):
    """A tensor at element `offset` of a flat buffer, zeroed."""
    n = math.prod(shape)
    return torch.zeros(offset + n, device="cuda", dtype=dtype)[offset:].view(shape)


def _blocks(dim):
    return (dim + BLOCK - 1) // BLOCK


def _packed(n, dim):
    return (torch.zeros((n, dim), device="cuda", dtype=torch.float8_e4m3fn),
            torch.zeros((n, _blocks(dim)), device="cuda"))


def _scratch(s, nbytes):
    s["scratch"] = torch.empty(nbytes, device="cuda", dtype=torch.uint8)
    s["scratch_bytes"] = nbytes


def _stream(g, n, d):
    """Values of a residual stream: rows of different sizes, some columns far larger."""
    size = torch.rand((n, 1), generator=g, device="cuda").mul_(2.0).add_(0.5)
    column = torch.rand(d, generator=g, device="cuda")
    column = torch.where(column < 0.005, 20.0, 1.0)
    return torch.randn((n, d), generator=g, device="cuda").mul_(size).mul_(column)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T, d = case["op"], case["tokens"], case["dim"]
    s = dict(case)
    if op.startswith("loss"):
        bf16, V = torch.bfloat16, case["vocab"]
        W = _flat((V, d), case["offset"], bf16)
        step = max(1, (1 << 28) // d)
        for a in range(0, V, step):
            b = min(V, a + step)
            W[a:b].copy_(torch.randn((b - a, d), generator=g, device="cuda").mul_(0.02))
        labels = torch.randint(0, V, (T,), generator=g, device="cuda")
        # logits spread by 2, and about 6 more at the label: some tokens are easy
        sure = torch.rand((T, 1), generator=g, device="cuda").mul_(12.0)
        near = W[labels].float()
        near.mul_(sure / near.square().sum(1, keepdim=True))
        h = torch.randn((T, d), generator=g, device="cuda").mul_(100.0 / math.sqrt(d)).add_(near)
        s["hidden"] = _rows(T, d, case["pad_cols"], bf16)
        s["hidden"].copy_(h)
        s["table"] = W
        if case["masked"]:
            out = torch.rand(T, generator=g, device="cuda") < case["masked"]
            labels = torch.where(out, torch.full_like(labels, -100), labels)
        s["labels"] = labels
        s["loss"] = torch.zeros(T, device="cuda")
        s["lse"] = torch.zeros(T, device="cuda")
        if op == "loss_grad":
            # the forward pass has left the rows' log of the sum of exponentials
            part = max(1, (1 << 28) // V)
            Wf = W.float()
            for a in range(0, T, part):
                b = min(T, a + part)
                s["lse"][a:b] = torch.logsumexp(s["hidden"][a:b].float() @ Wf.t(), 1)
            del Wf
            live = int((labels >= 0).sum())
            s["grad_loss"] = torch.full((T,), 1.0 / max(live, 1), device="cuda")
            s["grad_hidden"] = _rows(T, d, case["pad_cols"], bf16)
            s["grad_table"] = _flat((V, d), case["offset"], bf16)
            if case["accumulate"]:
                s["grad_table"].copy_(
                    torch.randn((V, d), generator=g, device="cuda").mul_(1e-5))
        _scratch(s, (1280 << 20) + 32 * (T + 256) * (d + 64))
        return s
    dt = _DTYPES[case["dtype"]]
    s["x"] = _rows(T, d, case["pad_cols"], dt)
    s["x"].copy_(_stream(g, T, d))
    if op == "checkpoint":
        s["packed"] = _packed(T, d)
        s["restored"] = _rows(T, d, case["pad_cols"], dt)
        return s
    s["weight"] = _flat((d,), case["offset"], dt)
    s["weight"].copy_(torch.randn(d, generator=g, device="cuda").mul_(0.1).add_(1.0))
    s["residual_in"] = None
    if case["residual"] and op != "norm_grad":
        s["residual_in"] = _rows(T, d, case["pad_cols"], dt)
        s["residual_in"].copy_(_stream(g, T, d))
    s["total"] = _rows(T, d, case["pad_cols"], dt) if case["residual"] else None
    s["out"] = _rows(T, d, case["pad_cols"], dt)
    s["rstd"] = torch.zeros(T, device="cuda")
    if op in ("norm8", "step8"):
        s["packed"] = _packed(T, d)
        s["restored"] = torch.zeros((T, d), device="cuda", dtype=torch.bfloat16)
    if op in ("norm_grad", "step8"):
        s["grad_out"] = _rows(T, d, case["pad_cols"], dt)
        s["grad_out"].copy_(torch.randn((T, d), generator=g, device="cuda").mul_(1e-2))
        s["grad_total"] = None
        if case["residual"]:
            s["grad_total"] = _rows(T, d, case["pad_cols"], dt)
            s["grad_total"].copy_(torch.randn((T, d), generator=g, device="cuda").mul_(1e-2))
        s["grad_x"] = _rows(T, d, case["pad_cols"], dt)
        s["again"] = _rows(T, d, case["pad_cols"], dt)
        s["grad_weight"] = _flat((d,), case["offset"], dt)
        _scratch(s, (64 << 20) + 8192 * d)
    if op == "norm_grad":
        s["rstd"].copy_(torch.rsqrt(s["x"].double().square().mean(1) + EPS))
    return s


# ----------------------------------------------------------- plain forms ----

def _plain_in_8_bits(x):
    """What x (fp32) is after a way through 8 bits."""
    n, d = x.shape
    b = torch.zeros((n, _blocks(d) * BLOCK), device=x.device)
    b[:, :d] = x
    b = b.view(n, -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))
    scale = torch.ldexp(torch.ones_like(m),
                        torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=-126))
    q = (b / scale).to(torch.float8_e4m3fn).float() * scale
    return q.reshape(n, -1)[:, :d]


def _plain_norm(s):
    x = s["x"].float()
    if s["residual_in"] is not None:
        x = x + s["residual_in"].float()
    rstd = 1.0 / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + EPS)
    y = x * rstd * s["weight"].float()
    return x, rstd, y


def _plain_norm_grad(s, x, rstd):
    dy, d = s["grad_out"].float(), s["dim"]
    xh = x * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - xh * ((g * xh).sum(1, keepdim=True) / d))
    if s["grad_total"] is not None:
        dx = dx + s["grad_total"].float()
    dt = s["x"].dtype
    return {"grad_x": dx.to(dt), "grad_weight": (dy * xh).sum(0).to(dt)}


def _plain_loss(s, with_grad):
    h, W, labels = s["hidden"].float(), s["table"].float(), s["labels"]
    V = W.shape[0]
    live = (labels >= 0) & (labels < V)
    at = torch.where(live, labels, 0)[:, None]
    z = h @ W.t()
    if not with_grad:
        top = z.amax(1, keepdim=True)
        lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
        loss = torch.where(live, lse - torch.gather(z, 1, at)[:, 0], 0.0)
        return {"loss": loss, "lse": torch.where(live, lse, 0.0)}
    p = torch.exp(z.sub_(s["lse"][:, None]))
    p.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
    dz = torch.where(live[:, None], p * s["grad_loss"][:, None], 0.0)
    dW = dz.t() @ h
    if s["accumulate"]:
        dW += s["grad_table"]
        s["grad_table"].copy_(dW)
    return {"grad_hidden": (dz @ W).to(torch.bfloat16), "grad_table": dW.to(torch.bfloat16)}


def _plain(s):
    op, dt = s["op"], None if s["op"].startswith("loss") else s["x"].dtype
    if dt is None:
        return _plain_loss(s, op == "loss_grad")
    if op == "checkpoint":
        return _plain_in_8_bits(s["x"].float()).to(dt)
    if op == "norm_grad":
        return _plain_norm_grad(s, s["x"].float(), s["rstd"][:, None])
    x, rstd, y = _plain_norm(s)
    out = {"out": y.to(dt), "rstd": rstd[:, 0]}
    if s["residual"]:
        out["total"] = x.to(dt)
    if op == "norm8":
        out["restored"] = _plain_in_8_bits(y).to(torch.bfloat16)
    if op == "step8":
        kept = _plain_in_8_bits(x)
        out.update(_plain_norm_grad(s, kept, rstd))
        out["again"] = (kept * rstd * s["weight"].float()).to(dt)
    return out


# ----------------------------------------------------------------- pass -----

def run(s):
    if not own:
        return _plain(s)
    import fsdp_sharded_mixed_flatten_gb300 as zf
    op = s["op"]
    if op == "loss":
        zf.zero_head_loss(s["hidden"], s["table"], s["labels"], s["loss"], s["lse"],
                          s["scratch"], s["scratch_bytes"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "loss_grad":
        zf.zero_head_loss_grad(s["hidden"], s["table"], s["labels"], s["lse"], s["grad_loss"],
                               s["grad_hidden"], s["grad_table"], s["accumulate"], s["scratch"],
                               s["scratch_bytes"])
        return {"grad_hidden": s["grad_hidden"], "grad_table": s["grad_table"]}
    if op == "checkpoint":
        zf.zero_pack_rows(s["x"], s["packed"])
        zf.zero_unpack_rows(s["packed"], s["restored"])
        return s["restored"]
    if op == "norm_grad":
        zf.zero_rms_norm_grad(s["grad_out"], s["x"], s["weight"], s["rstd"], s["grad_x"],
                              s["grad_weight"], s["grad_total"], None, s["scratch"],
                              s["scratch_bytes"])
        return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"]}
    out = {"out": s["out"], "rstd": s["rstd"]}
    if s["residual"]:
        out["total"] = s["total"]
    packed_out = s["packed"] if op == "norm8" else None
    packed_total = s["packed"] if op == "step8" else None
    zf.zero_rms_norm(s["x"], s["residual_in"], s["weight"], EPS, s["out"], s["total"], s["rstd"],
                     packed_out, packed_total)
    if op == "norm8":
        zf.zero_unpack_rows(s["packed"], s["restored"])
        out["restored"] = s["restored"]
    if op == "step8":
        zf.zero_rms_norm_grad(s["grad_out"], s["packed"], s["weight"], s["rstd"], s["grad_x"],
                              s["grad_weight"], s["grad_total"], s["again"], s["scratch"],
                              s["scratch_bytes"])
        out.update(grad_x=s["grad_x"], grad_weight=s["grad_weight"], again=s["again"])
    return out


# ---------------------------------------------------------------- work ------

def work(case):
    op, T, d = case["op"], case["tokens"], case["dim"]
    if op.startswith("loss"):
        V, live = case["vocab"], T * (1.0 - case["masked"])
        if op == "loss":
            return {"bytes": 2 * (live * d + V * d) + 16 * T, "flops": 2 * live * V * d}
        return {"bytes": 2 * (live * d + T * d + (3 if case["accumulate"] else 2) * V * d) + 16 * T,
                "flops": 6 * live * V * d}
    b, n = _BYTES[case["dtype"]], T * d
    eight = n + 4 * T * _blocks(d)
    if op == "checkpoint":
        return {"bytes": 2 * b * n + 2 * eight, "flops": 4 * n}
    r = 1 if case["residual"] else 0
    forward = (2 + 2 * r) * b * n + b * d + 4 * T
    if op == "norm":
        return {"bytes": forward, "flops": 5 * n}
    if op == "norm8":
        return {"bytes": forward + 2 * eight + 2 * n, "flops": 9 * n}
    backward = (2 + r) * b * n + 2 * b * d + 4 * T
    if op == "norm_grad":
        return {"bytes": backward + b * n, "flops": 10 * n}
    return {"bytes": forward + backward + 2 * eight + b * n, "flops": 21 * n}


# --------------------------------------------------------------- exact ------

def _exact_8_bits(x):
    """Rounding to 4 significant bits, none smaller than 2^-9 of the block's scale."""
    n, d = x.shape
    y = torch.empty_like(x)
    for a in range(0, d, BLOCK):
        part = x[:, a:a + BLOCK]
        top = part.abs().max(1, keepdim=True).values
        k = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0)
        # the logarithm may be off where the quotient is next to a power of two
        k = torch.where(top > 448.0 * torch.exp2(k), k + 1, k)
        k = torch.where((top <= 448.0 * torch.exp2(k - 1)) & (k > -126), k - 1, k)
        v = part / torch.exp2(k)
        step = torch.exp2((torch.frexp(v).exponent - 4).clamp(min=-9).double())
        y[:, a:a + BLOCK] = torch.round(v / step) * step * torch.exp2(k)
    return y


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    op, f64, d, T = case["op"], torch.float64, case["dim"], case["tokens"]
    if op.startswith("loss"):
        if T * case["vocab"] * d > (1.5e12 if op == "loss_grad" else 5e12):
            return None             # the products would take minutes
        s = prepare(case, seed)
        V, W, h = case["vocab"], s["table"].to(f64), s["hidden"].to(f64)
        loss, lse = torch.zeros(T, dtype=f64, device="cuda"), torch.zeros(T, dtype=f64, device="cuda")
        dh = torch.zeros((T, d), dtype=f64, device="cuda")
        dW = torch.zeros((V, d), dtype=f64, device="cuda")
        known = ((s["labels"] >= 0) & (s["labels"] < V)).nonzero()[:, 0]
        step = max(1, (1 << 27) // V)
        for a in range(0, len(known), step):
            rows = known[a:a + step]
            z = torch.mm(h[rows], W.T)
            y = torch.nn.functional.one_hot(s["labels"][rows], V).to(f64)
            if op == "loss":
                lse[rows] = torch.logsumexp(z, 1)
                loss[rows] = -(torch.log_softmax(z, 1) * y).sum(1)
            else:
                # the rows' normalisation is an input
                dz = (torch.exp(z - s["lse"][rows].to(f64)[:, None]) - y) \
                    * s["grad_loss"][rows].to(f64)[:, None]
                dh[rows] = torch.mm(dz, W)
                dW.addmm_(dz.T, h[rows])
        if op == "loss":
            return {"loss": loss, "lse": lse}
        if case["accumulate"]:
            dW += s["grad_table"].to(f64)
        return {"grad_hidden": dh, "grad_table": dW}
    s = prepare(case, seed)
    x = s["x"].to(f64)
    if op == "checkpoint":
        return _exact_8_bits(x)
    w, out = s["weight"].to(f64), {}
    if op != "norm_grad":
        if s["residual_in"] is not None:
            x = x + s["residual_in"].to(f64)
        # the sums of the residual's addition are fp32 values
        x = x.float().to(f64)
        r = (torch.linalg.vector_norm(x, dim=1) ** 2 / d + EPS) ** -0.5
        y = torch.einsum("td,t,d->td", x, r, w)
        out = {"out": y, "rstd": r}
        if case["residual"]:
            out["total"] = x
        if op == "norm8":
            out["restored"] = _exact_8_bits(y)
        if op != "step8":
            return out
        x = _exact_8_bits(x)
        out["again"] = torch.einsum("td,t,d->td", x, r, w)
    else:
        r = s["rstd"].to(f64)
    # dx as the Jacobian of x * rstd applied to dy * w
    dy = s["grad_out"].to(f64)
    along = torch.einsum("td,d,td->t", dy, w, x) * r ** 3 / d
    dx = torch.einsum("td,d,t->td", dy, w, r) - x * along[:, None]
    if s["grad_total"] is not None:
        dx += s["grad_total"].to(f64)
    out["grad_x"], out["grad_weight"] = dx, torch.einsum("td,td,t->d", dy, x, r)
    return out
