"""What the operators around the optimizer steps are measured on: the global
gradient norm and clipping, the embedding lookup and its gradient, and the
softmax cross entropy of the output layer with its gradient.

``run`` computes a case either in plain torch operations (``own`` false) or
through this package's entry points (``own`` true), on what ``prepare`` made.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6  # added to the norm that clipping divides by

# Matrix shapes of one layer of the benchmark's sets.
GPT2_LAYER = [(768, 2304), (768, 768), (768, 3072), (3072, 768)]
DENSE8B_LAYER = [(4096, 4096), (4096, 1024), (4096, 1024), (4096, 4096), (4096, 14336), (4096, 14336), (14336, 4096)]


def listed():
    return [
        # The gradients of a probe model: a few small matrices, a vector and a
        # scalar, where the call's own latency is what a user waits for.
        {"name": "norm-few-small", "op": "norm", "set": "random", "n": 6, "elems": 140000, "shape_seed": 3, "type": "mixed"},
        # Every gradient of a GPT-2-small step: the 48 matrices in bf16, the
        # embedding and the gain vectors in fp32.
        {"name": "norm-gpt2-all", "op": "norm", "set": "gpt2+", "type": "mixed"},
        # The hidden matrices of the benchmark's 8B-shaped set (224 tensors).
        {"name": "norm-dense8b", "op": "norm", "set": "dense8b", "type": "bf16"},
        # Clipping ragged tensors of a small model.
        {"name": "clip-ragged", "op": "clip", "set": "random", "n": 37, "elems": 3000000, "shape_seed": 8, "type": "mixed"},
        # Clipping the 48 matrices of GPT-2 small into the buffers a step reads.
        {"name": "clip-gpt2", "op": "clip", "set": "gpt2", "type": "bf16"},
        # One token per sequence of a small batch, fp32 master table.
        {"name": "embed-tokens-17", "op": "embed", "tokens": 17, "rows": 50257, "width": 768, "table": "f32", "out": "bf16", "ids": 64},
        # A training batch of long sequences on a wide table.
        {"name": "embed-batch-64k", "op": "embed", "tokens": 65536, "rows": 151936, "width": 2048, "table": "bf16", "out": "bf16", "ids": 64},
        # The table's gradient for one micro-batch, a small vocabulary.
        {"name": "embed-grad-8k", "op": "embed_grad", "tokens": 8192, "rows": 50257, "width": 768, "grad": "bf16", "out": "f32", "ids": 64},
        # The table's gradient for a large batch and vocabulary.
        {"name": "embed-grad-64k", "op": "embed_grad", "tokens": 65536, "rows": 151936, "width": 2048, "grad": "bf16", "out": "bf16", "ids": 32},
        # Scoring a ragged set of tokens: the loss alone.
        {"name": "xent-score-1000", "op": "xent", "tokens": 1000, "rows": 50257, "width": 768, "grad": False, "reduction": "sum"},
        # A training micro-batch of a small model: loss and both gradients.
        {"name": "xent-train-8k", "op": "xent", "tokens": 8192, "rows": 50257, "width": 768, "grad": True, "reduction": "mean"},
        # A training micro-batch on a wide model and a large vocabulary.
        {"name": "xent-train-wide", "op": "xent", "tokens": 8192, "rows": 151936, "width": 2048, "grad": True, "reduction": "mean"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "clip", "embed", "embed_grad", "xent", "xent"])
    if op in ("norm", "clip"):
        n = _log_int(rng, 1, 300 if op == "norm" else 60)
        return {"op": op, "set": "random", "n": n, "elems": max(n, _log_int(rng, 1000, 400000000)),
                "shape_seed": rng.randrange(1 << 30), "type": rng.choice(["bf16", "f32", "mixed"])}
    if op == "embed":
        return {"op": op, "tokens": _log_int(rng, 1, 65536), "rows": _log_int(rng, 1000, 151936),
                "width": _log_int(rng, 64, 4096), "table": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "ids": rng.choice([32, 64])}
    if op == "embed_grad":
        return {"op": op, "tokens": _log_int(rng, 1, 65536), "rows": _log_int(rng, 1000, 151936),
                "width": _log_int(rng, 64, 2048), "grad": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "ids": rng.choice([32, 64])}
    # half of the widths are whole multiples of 64, as models choose them
    width = _log_int(rng, 64, 2048)
    if rng.random() < 0.5:
        width = max(64, width // 64 * 64)
    return {"op": "xent", "tokens": _log_int(rng, 1, 8192), "rows": _log_int(rng, 1000, 151936), "width": width,
            "grad": rng.random() < 0.7, "reduction": rng.choice(["mean", "sum"])}


def _tensors(case):
    """(shape, type) of every gradient of a norm or clip case."""
    if case["set"] == "gpt2":
        return [(s, "bf16") for s in GPT2_LAYER * 12]
    if case["set"] == "gpt2+":
        return ([(s, "bf16") for s in GPT2_LAYER * 12] + [((50257, 768), "f32"), ((1024, 768), "f32")]
                + [((768,), "f32")] * 50)
    if case["set"] == "dense8b":
        return [(s, "bf16") for s in DENSE8B_LAYER * 32]
    # n tensors whose sizes spread over a factor of about a hundred, a third
    # of them vectors, summing to about elems
    rng = random.Random(case["shape_seed"])
    weight = [math.exp(rng.uniform(0.0, 4.6)) for _ in range(case["n"])]
    total = sum(weight)
    out = []
    for w in weight:
        e = max(1, int(case["elems"] * w / total))
        kind = rng.choice(["bf16", "f32"]) if case["type"] == "mixed" else case["type"]
        if rng.random() < 0.33:
            out.append(((e,), kind))
        else:
            cols = max(1, int(math.sqrt(e) * math.exp(rng.uniform(-0.7, 0.7))))
            out.append(((max(1, e // cols), cols), kind))
    return out


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0.0, scale, generator=g)


def _token_ids(g, tokens, rows, bits):
    """Token ids with frequency falling as one over the rank, one in forty of them padding."""
    u = torch.rand(tokens, generator=g, device=DEV, dtype=torch.float64)
    ids = (torch.exp(u * math.log(rows + 1.0)) - 1.0).long().clamp_(0, rows - 1)
    pad = torch.rand(tokens, generator=g, device=DEV) < 0.025
    return torch.where(pad, torch.full_like(ids, -100), ids).to(torch.int32 if bits == 32 else torch.int64)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm", "clip"):
        grads = [_randn(g, shape, TYPES[kind], 1e-3) for shape, kind in _tensors(case)]
        state = {"op": op, "grads": grads}
        if op == "clip":
            # half of the norm that these gradients have on average
            state["max_norm"] = 0.5e-3 * math.sqrt(sum(t.numel() for t in grads))
            state["outputs"] = [torch.empty_like(t) for t in grads]
        return state
    n, v, d = case["tokens"], case["rows"], case["width"]
    if op == "embed":
        return {"op": op, "table": _randn(g, (v, d), TYPES[case["table"]], 0.02), "scale": math.sqrt(d),
                "ids": _token_ids(g, n, v, case["ids"]), "out": TYPES[case["out"]]}
    if op == "embed_grad":
        return {"op": op, "ids": _token_ids(g, n, v, case["ids"]), "scale": math.sqrt(d), "rows": v,
                "dout": _randn(g, (n, d), TYPES[case["grad"]], 1e-3), "out": TYPES[case["out"]]}
    # normalised activations; weights that spread the logits by about three
    return {"op": op, "x": _randn(g, (n, d), torch.bfloat16, 1.0), "w": _randn(g, (v, d), torch.bfloat16, 3.0 / math.sqrt(d)),
            "targets": _token_ids(g, n, v, 64), "reduction": case["reduction"], "grad": case["grad"]}


def _norms(grads):
    norms = torch.stack([t.float().square().sum() for t in grads]).sqrt()
    return norms.square().sum().sqrt(), norms


def _plain(s):
    op = s["op"]
    if op == "norm":
        total, norms = _norms(s["grads"])
        return {"total": total, "norms": norms}
    if op == "clip":
        total, _ = _norms(s["grads"])
        coef = (s["max_norm"] / (total + EPS)).clamp(max=1.0)
        return {"total": total, "coef": coef, "grads": [o.copy_(t.float() * coef) for t, o in zip(s["grads"], s["outputs"])]}
    if op == "embed":
        ids = s["ids"].long()
        ok = (ids >= 0) & (ids < s["table"].shape[0])
        rows = s["table"][torch.where(ok, ids, 0)].float() * s["scale"]
        return torch.where(ok[:, None], rows, 0.0).to(s["out"])
    if op == "embed_grad":
        ids = s["ids"].long()
        ok = (ids >= 0) & (ids < s["rows"])
        grad = torch.where(ok[:, None], s["dout"].float() * s["scale"], 0.0)
        table = torch.zeros(s["rows"], grad.shape[1], device=grad.device)
        return table.index_add_(0, torch.where(ok, ids, 0), grad).to(s["out"])
    x, w = s["x"].float(), s["w"].float()
    t = s["targets"]
    ok = (t >= 0) & (t < w.shape[0])
    at = torch.where(ok, t, 0)
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    token_loss = torch.where(ok, lse - logits.gather(1, at[:, None])[:, 0], 0.0)
    count = ok.sum().clamp(min=1).float() if s["reduction"] == "mean" else torch.ones((), device=x.device)
    loss = token_loss.sum() / count
    if not s["grad"]:
        return {"loss": loss, "token_loss": token_loss}
    p = (logits - lse[:, None]).exp_()
    p.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    p *= (ok.float() / count)[:, None]
    return {"loss": loss, "token_loss": token_loss, "dx": (p @ w).bfloat16(), "dw": (p.t() @ x).bfloat16()}


def _own(s):
    import matrix_orthogonalizing_optimizer_momentum_amd as mm
    op = s["op"]
    if op == "norm":
        total, _, norms = mm.grad_norm(s["grads"])
        return {"total": total, "norms": norms}
    if op == "clip":
        total, coef = mm.clip_grads(s["grads"], s["max_norm"], outputs=s["outputs"])
        return {"total": total, "coef": coef, "grads": s["outputs"]}
    if op == "embed":
        return mm.embedding(s["table"], s["ids"], scale=s["scale"], out_dtype=s["out"])
    if op == "embed_grad":
        return mm.embedding_grad(s["ids"], s["dout"], s["rows"], scale=s["scale"], out_dtype=s["out"])
    loss, token_loss, dx, dw = mm.cross_entropy(s["x"], s["w"], s["targets"], reduction=s["reduction"], grad=s["grad"])
    return {"loss": loss, "token_loss": token_loss, "dx": dx, "dw": dw} if s["grad"] else {"loss": loss, "token_loss": token_loss}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        tensors = _tensors(case)
        elems = [math.prod(shape) for shape, _ in tensors]
        read = sum(e * SIZE[kind] for e, (_, kind) in zip(elems, tensors))
        if op == "norm":
            return {"bytes": read + 4 * (1 + len(elems)), "flops": 2 * sum(elems)}
        return {"bytes": 2 * read + 8, "flops": 3 * sum(elems)}
    n, v, d = case["tokens"], case["rows"], case["width"]
    if op == "embed":
        return {"bytes": n * (case["ids"] // 8) + min(n, v) * d * SIZE[case["table"]] + n * d * SIZE[case["out"]], "flops": n * d}
    if op == "embed_grad":
        return {"bytes": n * (case["ids"] // 8) + n * d * SIZE[case["grad"]] + v * d * SIZE[case["out"]], "flops": 2 * n * d}
    small = n * 12 + 4
    if not case["grad"]:
        return {"bytes": 2 * (n + v) * d + small, "flops": 2 * n * v * d}
    return {"bytes": 4 * (n + v) * d + small, "flops": 6 * n * v * d}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("norm", "clip"):
        sq = [torch.linalg.vector_norm(t, dtype=torch.float64) ** 2 for t in s["grads"]]
        total = torch.stack(sq).sum() ** 0.5
        if op == "norm":
            return {"total": total, "norms": torch.stack(sq) ** 0.5}
        coef = torch.minimum(torch.ones_like(total), s["max_norm"] / (total + EPS))
        return {"total": total, "coef": coef, "grads": [coef * t.double() for t in s["grads"]]}
    if op == "embed":
        ids = s["ids"].long()
        out = torch.zeros(len(ids), s["table"].shape[1], device=DEV, dtype=torch.float64)
        at = torch.nonzero(ids >= 0)[:, 0]
        out[at] = s["table"][ids[at]].double() * s["scale"]
        return out
    if op == "embed_grad":
        ids = s["ids"].long()
        at = torch.nonzero(ids >= 0)[:, 0]
        out = torch.zeros(s["rows"], s["dout"].shape[1], device=DEV, dtype=torch.float64)
        out.index_put_((ids[at],), s["dout"][at].double(), accumulate=True)
        return out * s["scale"]
    # by blocks of tokens, so that a block's logits fit in 64 bits
    w, t = s["w"].double(), s["targets"]
    counted = int((t >= 0).sum())
    per = 1.0 / max(1, counted) if s["reduction"] == "mean" else 1.0
    token_loss = torch.zeros(len(t), device=DEV, dtype=torch.float64)
    dx, dw = torch.zeros(len(t), w.shape[1], device=DEV, dtype=torch.float64), torch.zeros_like(w)
    for b in range(0, len(t), 1024):
        rows = torch.nonzero(t[b:b + 1024] >= 0)[:, 0] + b
        if not len(rows):
            continue
        x = s["x"][rows].double()
        logp = torch.log_softmax(torch.mm(x, w.t().contiguous()), 1)
        at = (torch.arange(len(rows), device=DEV), t[rows])
        token_loss[rows] = -logp[at]
        if s["grad"]:
            p = logp.exp()
            p[at] -= 1.0
            dx[rows] = torch.mm(p, w) * per
            dw += torch.mm(p.t().contiguous(), x) * per
    loss = token_loss.sum() * per
    return {"loss": loss, "token_loss": token_loss, "dx": dx, "dw": dw} if s["grad"] else {"loss": loss, "token_loss": token_loss}
