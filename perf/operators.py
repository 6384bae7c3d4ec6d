"""What is measured of the operators around the root unit of a sharded language
model: the token table's lookup and gradient, layer norm forward and backward,
and the distillation loss over the vocabulary with its gradient.

Each case is one call as a training program makes it.  `run` computes it in
its plain form (elementary torch operations in 32 bits), or, where `own` is
true, through the library's entry points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-5
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------- cases ------

def listed():
    return [
        # One decoding step of a small batch: the lookup of 32 single tokens in
        # a 50257-token table of width 4096; latency is all that counts.
        dict(name="lookup_tokens_32x4096", op="embed", tokens=32, vocab=50257, dim=4096,
             dtype="bf16", scale=64.0, pad=0.0, offset=0, accumulate=False),
        # The tied table of GPT-2-small: the head's product has already written
        # the table's gradient, 8 sequences of 1024 tokens add theirs.
        dict(name="table_grad_tied_8192x768", op="embed_grad", tokens=8192, vocab=50257, dim=768,
             dtype="bf16", scale=1.0, pad=0.0, offset=0, accumulate=True),
        # A ragged batch with padded places, odd sizes, fp32, and the gradient
        # at an odd place of a flat buffer.
        dict(name="table_grad_f32_4099x770", op="embed_grad", tokens=4099, vocab=30011, dim=770,
             dtype="f32", scale=27.75, pad=0.15, offset=37, accumulate=False),
        # A long batch on a wide untied table: every row of the gradient is
        # written, the unused ones with zeros.
        dict(name="table_grad_65536x4096", op="embed_grad", tokens=65536, vocab=131072, dim=4096,
             dtype="bf16", scale=1.0, pad=0.02, offset=0, accumulate=False),
        # One decoding step: 8 rows of GPT-2-small's width.
        dict(name="norm_8x768", op="norm", tokens=8, dim=768, dtype="bf16", pad_cols=0, offset=0),
        # A long batch at the width of a Llama-3-8B layer.
        dict(name="norm_16384x4096", op="norm", tokens=16384, dim=4096, dtype="bf16", pad_cols=0,
             offset=0),
        # GPT-2-small, 8 sequences of 1024 tokens; the weight's gradient goes
        # to its place in the root unit's flat gradient.
        dict(name="norm_grad_8192x768", op="norm_grad", tokens=8192, dim=768, dtype="bf16",
             pad_cols=0, offset=64),
        # Odd width and rows of a wider fp32 buffer.
        dict(name="norm_grad_f32_5003x1501", op="norm_grad", tokens=5003, dim=1501, dtype="f32",
             pad_cols=3, offset=3),
        # Validation of a few sequences' last tokens against 32 stored logits.
        dict(name="distill_16x50257", op="distill", tokens=16, vocab=50257, top=32, dtype="bf16",
             temperature=1.0, masked=0.0, ragged=0.0, pad_cols=0),
        # Training on 4 sequences of 1024 tokens with GPT-2's odd vocabulary:
        # rows of logits start at every alignment; prompt tokens are masked.
        dict(name="distill_grad_4096x50257", op="distill_grad", tokens=4096, vocab=50257, top=64,
             dtype="bf16", temperature=2.0, masked=0.125, ragged=0.2, pad_cols=0),
        # fp32 logits of a small odd vocabulary, few teacher entries.
        dict(name="distill_grad_f32_1021x32003", op="distill_grad", tokens=1021, vocab=32003,
             top=17, dtype="f32", temperature=1.5, masked=0.0, ragged=0.5, pad_cols=5),
        # The largest: 8192 tokens of a 131072-token vocabulary.
        dict(name="distill_grad_8192x131072", op="distill_grad", tokens=8192, vocab=131072,
             top=128, dtype="bf16", temperature=1.0, masked=0.0, ragged=0.0, pad_cols=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad",
                     "distill", "distill_grad", "distill_grad"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("embed"):
        c["tokens"] = _log_int(rng, 1, 65536)
        c["vocab"] = _log_int(rng, 1000, 131072)
        # mostly whole vectors, as models have them; sometimes any width
        dim = _log_int(rng, 64, 4096)
        c["dim"] = dim if rng.random() < 0.3 else (dim + 7) // 8 * 8
        c["scale"] = rng.choice([1.0, round(math.sqrt(c["dim"]), 3)])
        c["pad"] = rng.choice([0.0, round(rng.uniform(0.0, 0.5), 3)])
        c["offset"] = rng.choice([0, 0, rng.randrange(1, 100)])
        c["accumulate"] = op == "embed_grad" and rng.random() < 0.5
    elif op.startswith("norm"):
        dim = _log_int(rng, 64, 8192)
        c["dim"] = dim if rng.random() < 0.3 else (dim + 7) // 8 * 8
        c["tokens"] = _log_int(rng, 1, min(65536, 2 ** 26 // c["dim"]))
        c["pad_cols"] = rng.choice([0, 0, 8, rng.randrange(1, 20)])
        c["offset"] = rng.choice([0, 0, rng.randrange(1, 100)])
    else:
        c["vocab"] = _log_int(rng, 1000, 131072)
        c["tokens"] = _log_int(rng, 1, min(8192, 2 ** 29 // c["vocab"]))
        c["top"] = _log_int(rng, 1, 256)
        c["temperature"] = round(rng.uniform(0.5, 4.0), 3)
        c["masked"] = rng.choice([0.0, round(rng.uniform(0.0, 0.9), 3)])
        c["ragged"] = rng.choice([0.0, round(rng.uniform(0.0, 1.0), 3)])
        c["pad_cols"] = rng.choice([0, 0, 8, rng.randrange(1, 20)])
    return c


# -------------------------------------------------------------- inputs ------

def _token_probs(vocab):
    """Word frequencies fall about as 1 / rank."""
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return p / p.sum()


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _rows(n, cols, pad_cols, dtype):
    """(n, cols) rows of an (n, cols + pad_cols) buffer, zeroed."""
    return torch.zeros((n, cols + pad_cols), device="cuda", dtype=dtype)[:, :cols]


def _flat(shape, offset, dtype):
    """A tensor at element `offset` of a flat buffer, zeroed."""
    n = math.prod(shape)
    return torch.zeros(offset + n, device="cuda", dtype=dtype)[offset:].view(shape)


def _scratch(s, nbytes):
    s["scratch"] = torch.empty(nbytes, device="cuda", dtype=torch.uint8)
    s["scratch_bytes"] = nbytes


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, dt, T = case["op"], _DTYPES[case["dtype"]], case["tokens"]
    s = dict(case)
    if op.startswith("embed"):
        V, d = case["vocab"], case["dim"]
        # inverse of the distribution function, summed on the host in one order
        cdf = torch.from_numpy(np.cumsum(_token_probs(V))).to("cuda")
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = torch.searchsorted(cdf, u).clamp_(max=V - 1)
        order = torch.randperm(V, generator=g, device="cuda")
        ids = order[ids]
        if case["pad"]:
            out = torch.rand(T, generator=g, device="cuda") < case["pad"]
            ids = torch.where(out, torch.full_like(ids, -1), ids)
        s["ids"] = ids.to(torch.int32)
        if op == "embed":
            s["weight"] = _flat((V, d), case["offset"], dt)
            s["weight"].copy_(_randn(g, (V, d), dt, 0.02))
            s["out"] = torch.zeros((T, d), device="cuda", dtype=dt)
        else:
            s["grad_out"] = _randn(g, (T, d), dt, 1e-2)
            s["grad_weight"] = _flat((V, d), case["offset"], dt)
            if case["accumulate"]:
                s["grad_weight"].copy_(_randn(g, (V, d), dt, 1e-2))
            _scratch(s, (64 << 20) + T * (64 + d))
    elif op.startswith("norm"):
        d = case["dim"]
        x = _rows(T, d, case["pad_cols"], dt)
        level = torch.randn((T, 1), generator=g, device="cuda").mul_(0.5)
        size = torch.rand((T, 1), generator=g, device="cuda").mul_(2.0).add_(0.5)
        x.copy_(torch.randn((T, d), generator=g, device="cuda").mul_(size).add_(level))
        s["x"] = x
        s["weight"] = _flat((d,), case["offset"], dt)
        s["weight"].copy_(torch.randn(d, generator=g, device="cuda").mul_(0.1).add_(1.0))
        s["bias"] = _randn(g, (d,), dt, 0.1)
        if op == "norm":
            s["out"] = _rows(T, d, case["pad_cols"], dt)
            s["mean"] = torch.zeros(T, device="cuda")
            s["rstd"] = torch.zeros(T, device="cuda")
        else:
            s["grad_out"] = _rows(T, d, case["pad_cols"], dt)
            s["grad_out"].copy_(torch.randn((T, d), generator=g, device="cuda").mul_(1e-2))
            xf = x.double()
            mean = xf.mean(1, keepdim=True)
            s["mean"] = mean[:, 0].float()
            s["rstd"] = torch.rsqrt((xf - mean).square().mean(1) + EPS).float()
            s["grad_x"] = _rows(T, d, case["pad_cols"], dt)
            flat = _flat((2 * d,), case["offset"], dt)
            s["grad_weight"], s["grad_bias"] = flat[:d], flat[d:]
            _scratch(s, (64 << 20) + 8192 * d)
    else:
        V, K, tau = case["vocab"], case["top"], case["temperature"]
        z = _rows(T, V, case["pad_cols"], dt)
        # the teacher's best tokens: distinct ones, spread over the vocabulary
        start = torch.randint(0, V, (T, 1), generator=g, device="cuda")
        step = 7919 if V % 7919 else 7907
        ids = (start + step * torch.arange(K, device="cuda")) % V
        # logits falling off with the rank; the student knows some of it
        top = torch.rand((T, K), generator=g, device="cuda").add_(0.02).log_().mul_(2.0)
        top = top.sort(1, descending=True).values + 12.0
        step_rows = max(1, (1 << 28) // V)
        for a in range(0, T, step_rows):
            b = min(T, a + step_rows)
            part = torch.randn((b - a, V), generator=g, device="cuda").mul_(2.0)
            near = top[a:b] + torch.randn((b - a, K), generator=g, device="cuda").mul_(2.0)
            part.scatter_(1, ids[a:b], near)
            z[a:b].copy_(part)
        if case["ragged"]:
            # a stored row keeps as many entries as its teacher was sure of;
            # some rows keep none
            keep = (torch.rand((T, 1), generator=g, device="cuda") * (K + 1)).floor()
            short = torch.rand((T, 1), generator=g, device="cuda") < case["ragged"]
            gone = short & (torch.arange(K, device="cuda") >= keep)
            ids = torch.where(gone, torch.full_like(ids, -1), ids)
        s["logits"], s["ids"], s["teacher"] = z, ids.to(torch.int32), top.to(dt)
        w = torch.full((T,), 1.0 / T, device="cuda")
        if case["masked"]:
            w[torch.rand(T, generator=g, device="cuda") < case["masked"]] = 0.0
        s["weights"] = w
        s["loss"] = torch.zeros(T, device="cuda")
        if op == "distill_grad":
            s["grad_logits"] = _rows(T, V, case["pad_cols"], dt)
    return s


# ----------------------------------------------------------- plain forms ----

def _plain_embed(s):
    W, ids = s["weight"], s["ids"].long()
    inside = (ids >= 0) & (ids < W.shape[0])
    y = W[torch.where(inside, ids, 0)].float() * s["scale"]
    return torch.where(inside[:, None], y, 0.0).to(W.dtype)


def _plain_embed_grad(s):
    G, ids = s["grad_weight"], s["ids"].long()
    inside = (ids >= 0) & (ids < G.shape[0])
    dy = torch.where(inside[:, None], s["grad_out"].float() * s["scale"], 0.0)
    total = torch.zeros(G.shape, device=G.device)
    total.index_add_(0, torch.where(inside, ids, 0), dy)
    if s["accumulate"]:
        total += G
    G.copy_(total)
    return G


def _plain_norm(s):
    x = s["x"].float()
    mean = x.sum(1, keepdim=True) / x.shape[1]
    rstd = 1.0 / torch.sqrt((x - mean).square().sum(1, keepdim=True) / x.shape[1] + EPS)
    y = (x - mean) * rstd * s["weight"].float() + s["bias"].float()
    return {"out": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(s):
    x, dy, d = s["x"].float(), s["grad_out"].float(), s["dim"]
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.sum(1, keepdim=True) / d - xh * ((g * xh).sum(1, keepdim=True) / d))
    dt = s["x"].dtype
    return {"grad_x": dx.to(dt), "grad_weight": (dy * xh).sum(0).to(dt),
            "grad_bias": dy.sum(0).to(dt)}


def _plain_distill(s, with_grad):
    z, ids, tau, w = s["logits"], s["ids"].long(), s["temperature"], s["weights"]
    V = z.shape[1]
    inside = (ids >= 0) & (ids < V)
    at = torch.where(inside, ids, 0)
    x = z.float() / tau
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    log_q = torch.gather(x, 1, at) - top - torch.log(total)
    t = torch.where(inside, s["teacher"].float() / tau, float("-inf"))
    best = t.amax(1, keepdim=True)
    some = best > float("-inf")
    t = t - torch.where(some, best, 0.0)
    te = torch.exp(t)
    ts = torch.where(some, te.sum(1, keepdim=True), 1.0)
    p = te / ts
    terms = torch.where(p > 0, p * (t - torch.log(ts) - log_q), 0.0)
    live = some[:, 0] & (w != 0)
    loss = torch.where(live, w * tau * tau * terms.sum(1), 0.0)
    if not with_grad:
        return {"loss": loss}
    q = e / total
    q.scatter_add_(1, at, -p)
    grad = torch.where(live[:, None], q * (tau * w[:, None]), 0.0)
    return {"loss": loss, "grad_logits": grad.to(z.dtype)}


def run(s):
    op = s["op"]
    if own:
        import fsdp_sharded_mixed_flatten_gb300 as zf
        if op == "embed":
            zf.zero_embedding(s["ids"], s["weight"], s["out"], s["scale"])
            return s["out"]
        if op == "embed_grad":
            zf.zero_embedding_grad(s["ids"], s["grad_out"], s["grad_weight"], s["scale"],
                                   s["accumulate"], s["scratch"], s["scratch_bytes"])
            return s["grad_weight"]
        if op == "norm":
            zf.zero_layer_norm(s["x"], s["weight"], s["bias"], EPS, s["out"], s["mean"],
                               s["rstd"])
            return {"out": s["out"], "mean": s["mean"], "rstd": s["rstd"]}
        if op == "norm_grad":
            zf.zero_layer_norm_grad(s["grad_out"], s["x"], s["weight"], s["mean"], s["rstd"],
                                    s["grad_x"], s["grad_weight"], s["grad_bias"], s["scratch"],
                                    s["scratch_bytes"])
            return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"],
                    "grad_bias": s["grad_bias"]}
        if op == "distill":
            zf.zero_distill_loss(s["logits"], s["ids"], s["teacher"], s["weights"],
                                 s["temperature"], s["loss"])
            return {"loss": s["loss"]}
        zf.zero_distill_loss_grad(s["logits"], s["ids"], s["teacher"], s["weights"],
                                  s["temperature"], s["loss"], s["grad_logits"])
        return {"loss": s["loss"], "grad_logits": s["grad_logits"]}
    if op == "embed":
        return _plain_embed(s)
    if op == "embed_grad":
        return _plain_embed_grad(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    return _plain_distill(s, op == "distill_grad")


# ---------------------------------------------------------------- work ------

def work(case):
    op, T, b = case["op"], case["tokens"], _BYTES[case["dtype"]]
    if op.startswith("embed"):
        V, d = case["vocab"], case["dim"]
        live = T * (1.0 - case["pad"])
        # distinct tokens expected among the live ones
        used = float(-np.expm1(live * np.log1p(-_token_probs(V))).sum())
        if op == "embed":
            return {"bytes": 4 * T + used * d * b + T * d * b, "flops": T * d}
        table = 2 * used * d * b if case["accumulate"] else V * d * b
        return {"bytes": 4 * T + live * d * b + table, "flops": 2 * live * d}
    if op == "norm":
        return {"bytes": 2 * T * case["dim"] * b + 2 * case["dim"] * b + 8 * T,
                "flops": 8 * T * case["dim"]}
    if op == "norm_grad":
        return {"bytes": 3 * T * case["dim"] * b + 3 * case["dim"] * b + 8 * T,
                "flops": 15 * T * case["dim"]}
    V, K = case["vocab"], case["top"]
    # rows with a weight and, where rows are cut short, an entry left
    live = T * (1.0 - case["masked"]) * (1.0 - case["ragged"] / (K + 1))
    moved = live * V * b + T * K * (4 + b) + 8 * T
    if op == "distill":
        return {"bytes": moved, "flops": 4 * live * V}
    return {"bytes": moved + T * V * b, "flops": 7 * live * V}


# --------------------------------------------------------------- exact ------

def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "embed":
        y = torch.zeros((case["tokens"], case["dim"]), dtype=f64, device="cuda")
        known = ((s["ids"] >= 0) & (s["ids"] < case["vocab"])).nonzero()[:, 0]
        y[known] = s["weight"].index_select(0, s["ids"][known]).to(f64) * case["scale"]
        return y
    if op == "embed_grad":
        # the sum over the tokens of a row, as a difference of running sums of
        # the tokens in the order of their rows would lose digits: one row
        # after another by groups of equal count
        ids = s["ids"].cpu().numpy()
        order = np.argsort(ids, kind="stable")
        order = order[(ids[order] >= 0) & (ids[order] < case["vocab"])]
        rows, first, count = np.unique(ids[order], return_index=True, return_counts=True)
        g = s["grad_weight"].to(f64) if case["accumulate"] else \
            torch.zeros(s["grad_weight"].shape, dtype=f64, device="cuda")
        for n in np.unique(count):
            which = np.nonzero(count == n)[0]
            for a in range(0, len(which), max(1, 65536 // int(n))):
                part = which[a:a + max(1, 65536 // int(n))]
                tok = order[first[part][:, None] + np.arange(n)]
                dy = s["grad_out"][torch.from_numpy(tok).cuda()].to(f64)
                g[torch.from_numpy(rows[part].astype(np.int64)).cuda()] += \
                    dy.sum(1) * case["scale"]
        return g
    if op == "norm":
        x = s["x"].to(f64)
        mean = torch.mean(x, 1)
        var = torch.mean(x * x, 1) - mean * mean
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["bias"].to(f64), (x - mean[:, None]) * rstd[:, None],
                          s["weight"].to(f64))
        return {"out": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        # dx as the Jacobian of (x - mean) * rstd applied to dy * w; the
        # statistics are inputs
        x, r = s["x"].to(f64), s["rstd"].to(f64)
        c = x - s["mean"].to(f64)[:, None]
        dy = s["grad_out"].to(f64)
        g = dy * s["weight"].to(f64)
        along = torch.einsum("td,td->t", g, c) * r ** 3 / case["dim"]
        dx = g * r[:, None] - (g.mean(1) * r)[:, None] - c * along[:, None]
        return {"grad_x": dx, "grad_weight": torch.einsum("td,td,t->d", dy, c, r),
                "grad_bias": torch.einsum("td->d", dy)}
    tau, V = case["temperature"], case["vocab"]
    loss = torch.zeros(case["tokens"], dtype=f64, device="cuda")
    grad = torch.zeros((case["tokens"], V), dtype=f64, device="cuda") \
        if op == "distill_grad" else None
    step = max(1, (1 << 26) // V)
    for a in range(0, case["tokens"], step):
        rows = slice(a, min(case["tokens"], a + step))
        logq = torch.log_softmax(s["logits"][rows].to(f64) / tau, 1)
        ids, w = s["ids"][rows].long(), s["weights"][rows].to(f64)
        dense = torch.full(logq.shape, float("-inf"), dtype=f64, device="cuda")
        r, k = ((ids >= 0) & (ids < V)).nonzero(as_tuple=True)
        dense[r, ids[r, k]] = s["teacher"][rows].to(f64)[r, k] / tau
        p = torch.nan_to_num(torch.softmax(dense, 1), nan=0.0)
        live = (p.sum(1) > 0) & (w != 0)
        kl = (torch.xlogy(p, p) - torch.where(p > 0, p * logq, 0.0)).sum(1)
        loss[rows] = torch.where(live, w * tau ** 2 * kl, 0.0)
        if grad is not None:
            d = (torch.exp(logq) - p) * (tau * w)[:, None]
            grad[rows] = torch.where(live[:, None], d, 0.0)
    return {"loss": loss} if grad is None else {"loss": loss, "grad_logits": grad}
