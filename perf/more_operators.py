"""What the operators between the embedding and the output layer are measured on:
the root-mean-square norm with the residual's addition, its gradient, activations
kept in 8 bits, and the gradient of a weight from activations kept so.

``run`` computes a case either in plain torch operations (``own`` false) or
through this package's entry points (``own`` true), on what ``prepare`` made.

Activations in 8 bits are e4m3 values in blocks of 32 along a row, each block with
the power of two that is the least with no value of the block above 448 of it
(and not below 2^-117).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, None: 0}
EPS = 1e-6
BLOCK = 32


def listed():
    return [
        # One token of a small model: the call's own latency.
        {"name": "norm-token", "op": "norm", "tokens": 1, "width": 768, "x": "bf16", "res": "bf16", "y": "bf16", "pack": None},
        # A training micro-batch of a small model, residual stream in fp32, the
        # normalised rows kept in 8 bits for the backward pass.
        {"name": "norm-train-8k", "op": "norm", "tokens": 8192, "width": 768, "x": "bf16", "res": "f32", "y": "bf16", "pack": "normalized"},
        # A large micro-batch of a wide model in bf16, kept in 8 bits too.
        {"name": "norm-train-wide", "op": "norm", "tokens": 16384, "width": 4096, "x": "bf16", "res": "bf16", "y": "bf16", "pack": "normalized"},
        # The gradient for an odd number of tokens and channels, all in fp32, from
        # the norm's own input.
        {"name": "norm-grad-ragged", "op": "norm_grad", "tokens": 777, "width": 1999, "dy": "f32", "stream": "f32", "kept": "input", "dres": False},
        # The gradient for the small model's micro-batch, from what was kept in 8 bits.
        {"name": "norm-grad-8k", "op": "norm_grad", "tokens": 8192, "width": 768, "dy": "bf16", "stream": "f32", "kept": "packed", "dres": True},
        # The same for the wide model.
        {"name": "norm-grad-wide", "op": "norm_grad", "tokens": 16384, "width": 4096, "dy": "bf16", "stream": "bf16", "kept": "packed", "dres": True},
        # An odd activation of a probe model, stored and read back.
        {"name": "pack-odd", "op": "pack", "tokens": 1021, "width": 331, "x": "f32"},
        # The inner activation of a wide feed-forward layer, stored and read back.
        {"name": "pack-wide", "op": "pack", "tokens": 8192, "width": 14336, "x": "bf16"},
        # A weight's gradient for a few tokens.
        {"name": "weight-few", "op": "weight", "tokens": 33, "rows": 768, "width": 768, "out": "bf16", "gain": True},
        # Odd sizes everywhere.
        {"name": "weight-odd", "op": "weight", "tokens": 3001, "rows": 1003, "width": 517, "out": "f32", "gain": False},
        # The joined query, key and value matrix of a small model's micro-batch.
        {"name": "weight-gpt2", "op": "weight", "tokens": 8192, "rows": 2304, "width": 768, "out": "f32", "gain": True},
        # The first matrix of a feed-forward layer of the benchmark's 8B-shaped set.
        {"name": "weight-8b", "op": "weight", "tokens": 8192, "rows": 14336, "width": 4096, "out": "bf16", "gain": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    # half of the widths are whole multiples of 64, as models choose them
    w = _log_int(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "pack", "weight"])
    kind = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op == "weight":
        case = {"op": op, "tokens": _log_int(rng, 1, 8192), "rows": _width(rng, 32, 14336), "width": _width(rng, 32, 14336),
                "out": kind(), "gain": rng.random() < 0.5}
        most = 8192 * 14336 * 4096
        case["tokens"] = max(1, min(case["tokens"], most // (case["rows"] * case["width"])))
        return case
    width = _width(rng, 32, 16384)
    tokens = _log_int(rng, 1, min(32768, 16384 * 4096 // (2 * width)))
    if op == "norm":
        pack = rng.choice([None, "normalized", "output"])
        return {"op": op, "tokens": tokens, "width": width, "x": kind(), "res": rng.choice([None, "bf16", "f32"]),
                "y": kind() if pack != "output" else None, "pack": pack}
    if op == "norm_grad":
        return {"op": op, "tokens": tokens, "width": width, "dy": kind(), "stream": kind(),
                "kept": rng.choice(["input", "packed"]), "dres": rng.random() < 0.7}
    return {"op": op, "tokens": tokens, "width": width, "x": kind()}


def _randn(g, shape, dtype, scale):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0.0, scale, generator=g)


def _stream_rows(g, n, d, dtype):
    """Rows of a residual stream: a few channels much larger than the others."""
    channel = 0.5 * torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
    channel[torch.rand(d, generator=g, device=DEV) < 0.005] *= 30.0
    return (_randn(g, (n, d), torch.float32, 1.0) * channel).to(dtype)


def _blocks(v):
    """Rows cut into blocks of 32, the last one filled with zeros."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))


def _quantise(v):
    """(e4m3 values, exponents of the blocks) of rows in fp32."""
    b = _blocks(v)
    m, ex = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 0.875, ex - 9, ex - 8).clamp_(min=-117)
    q = torch.ldexp(b, -e).flatten(-2)[..., :v.shape[-1]]
    return q.to(torch.float8_e4m3fn), e[..., 0]


def _values(q, e):
    """What 8-bit rows stand for, in fp32."""
    return torch.ldexp(_blocks(q.float()), e[..., None]).flatten(-2)[..., :q.shape[-1]]


def _store(q, e):
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _load(packed):
    q, scales = packed
    return _values(q, scales.view(torch.uint8).int() - 127)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, n, d = case["op"], case["tokens"], case["width"]
    gain = 1.0 + _randn(g, (d,), torch.float32, 0.2)
    if op == "norm":
        return {"op": op, "x": _randn(g, (n, d), TYPES[case["x"]], 0.3), "gain": gain, "y": TYPES.get(case["y"]), "pack": case["pack"],
                "res": None if case["res"] is None else _stream_rows(g, n, d, TYPES[case["res"]])}
    if op == "pack":
        # the inner activation of a feed-forward layer: a gate's product
        a, b = _randn(g, (n, d), torch.float32, 1.0), _randn(g, (n, d), torch.float32, 1.0)
        return {"op": op, "x": (a * torch.sigmoid(a) * b).to(TYPES[case["x"]])}
    if op == "norm_grad":
        h = _stream_rows(g, n, d, TYPES[case["stream"]])
        rstd = torch.rsqrt(h.double().square().mean(-1) + EPS).float()
        kept = h if case["kept"] == "input" else _store(*_quantise(h.float() * rstd[:, None]))
        return {"op": op, "dy": _randn(g, (n, d), TYPES[case["dy"]], 1e-3), "kept": kept, "rstd": rstd, "gain": gain,
                "dres": _randn(g, (n, d), h.dtype, 1e-3) if case["dres"] else None, "out": h.dtype}
    x = _stream_rows(g, n, d, torch.float32)
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True))
    return {"op": op, "dz": _randn(g, (n, case["rows"]), torch.bfloat16, 1e-3), "x": _store(*_quantise(x)),
            "gain": gain if case["gain"] else None, "out": TYPES[case["out"]]}


def _plain(s):
    op = s["op"]
    if op == "norm":
        x, res = s["x"], s["res"]
        h = x if res is None else (x.float() + res.float()).to(res.dtype)
        v = h.float()
        rstd = torch.rsqrt(v.square().mean(-1) + EPS)
        xn = v * rstd[:, None]
        y = xn * s["gain"]
        out = {"rstd": rstd}
        if res is not None:
            out["h"] = h
        if s["y"] is not None:
            out["y"] = y.to(s["y"])
        if s["pack"] is not None:
            out["packed"] = _values(*_quantise(xn if s["pack"] == "normalized" else y)).bfloat16()
        return out
    if op == "pack":
        return _values(*_quantise(s["x"].float())).bfloat16()
    if op == "norm_grad":
        rstd = s["rstd"][:, None]
        xn = _load(s["kept"]) if isinstance(s["kept"], tuple) else s["kept"].float() * rstd
        dy = s["dy"].float()
        gy = dy * s["gain"]
        dx = (gy - xn * (gy * xn).mean(-1, keepdim=True)) * rstd
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(s["out"]), "dgain": (dy * xn).sum(0)}
    dw = s["dz"].float().t() @ _load(s["x"])
    return (dw if s["gain"] is None else dw * s["gain"]).to(s["out"])


def _own(s):
    import matrix_orthogonalizing_optimizer_momentum_amd as mm
    op = s["op"]
    if op == "norm":
        r = mm.rms_norm(s["x"], s["gain"], residual=s["res"], eps=EPS, output=s["y"] is not None, out_dtype=s["y"], pack=s["pack"])
        out = {"rstd": r.rstd}
        if s["res"] is not None:
            out["h"] = r.h
        if s["y"] is not None:
            out["y"] = r.y
        if s["pack"] is not None:
            out["packed"] = mm.mx_unpack(r.packed)
        return out
    if op == "pack":
        return mm.mx_unpack(mm.mx_pack(s["x"]))
    if op == "norm_grad":
        dx, dgain = mm.rms_norm_grad(s["dy"], s["kept"], s["rstd"], s["gain"], dres=s["dres"], out_dtype=s["out"])
        return {"dx": dx, "dgain": dgain}
    return mm.weight_grad(s["dz"], s["x"], gain=s["gain"], out_dtype=s["out"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, n, d = case["op"], case["tokens"], case["width"]
    eight = n * d + n * -(-d // BLOCK)  # a matrix in 8 bits with its scales
    if op == "norm":
        moved = SIZE[case["x"]] + 2 * SIZE[case["res"]] + SIZE[case["y"]]
        # what is kept in 8 bits is written, read back and written as values
        return {"bytes": n * d * moved + 4 * n + 4 * d + (2 * eight + 2 * n * d if case["pack"] else 0), "flops": 5 * n * d}
    if op == "pack":
        return {"bytes": n * d * (SIZE[case["x"]] + 2) + 2 * eight, "flops": 3 * n * d}
    if op == "norm_grad":
        s = SIZE[case["stream"]]
        kept = eight if case["kept"] == "packed" else n * d * s
        return {"bytes": n * d * (SIZE[case["dy"]] + (2 if case["dres"] else 1) * s) + kept + 4 * n + 8 * d, "flops": 9 * n * d}
    return {"bytes": 2 * n * case["rows"] + eight + case["rows"] * d * SIZE[case["out"]] + (4 * d if case["gain"] else 0),
            "flops": 2 * n * case["rows"] * d}


def _rounded(v):
    """Rows in 64 bits rounded to e4m3 by blocks of 32: what the 8-bit rows stand for."""
    n, d = v.shape
    out = torch.zeros(n, -(-d // BLOCK) * BLOCK, device=v.device, dtype=torch.float64)
    out[:, :d] = v
    out = out.view(n, -1, BLOCK)
    top = out.abs().amax(2, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -117))))
    scale = torch.where(top > 448.0 * scale, 2 * scale, torch.where((top <= 224.0 * scale) & (scale > 2.0 ** -117), scale / 2, scale))
    unit = torch.exp2(torch.floor(torch.log2((out.abs() / scale).clamp(min=2.0 ** -6))) - 3.0) * scale
    return (torch.round(out / unit) * unit).view(n, -1)[:, :d]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "pack":
        return _rounded(s["x"].double())
    if op == "norm":
        h = s["x"].double()
        out = {}
        if s["res"] is not None:
            h = h + s["res"].double()
            out["h"] = h
            h = h.to(s["res"].dtype).double()
        out["rstd"] = (torch.linalg.vector_norm(h, dim=1) ** 2 / h.shape[1] + EPS) ** -0.5
        h = h * out["rstd"][:, None]
        y = h * s["gain"].double()
        if s["y"] is not None:
            out["y"] = y
        if s["pack"] is not None:
            out["packed"] = _rounded(h if s["pack"] == "normalized" else y)
        return out
    kept = s["kept"] if op == "norm_grad" else s["x"]
    if isinstance(kept, tuple):
        xn = kept[0].to(torch.float64) * kept[1].to(torch.float64).repeat_interleave(BLOCK, 1)[:, :kept[0].shape[1]]
    else:
        xn = kept.double() * s["rstd"].double()[:, None]
    if op == "norm_grad":
        dy = s["dy"].double()
        dgain = torch.linalg.vecdot(dy, xn, dim=0)
        dy = dy * s["gain"].double()
        dx = s["rstd"].double()[:, None] * (dy - xn * (torch.linalg.vecdot(dy, xn) / xn.shape[1])[:, None])
        return {"dx": dx if s["dres"] is None else dx + s["dres"].double(), "dgain": dgain}
    dw = torch.mm(s["dz"].double().t().contiguous(), xn)
    return dw if s["gain"] is None else dw * s["gain"].double()
