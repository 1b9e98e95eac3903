"""The operators of a sampled low-rank fit, as measured: row lookups of a table and their gradient,
the norm over many gradients with clipping, and the entries of a CP model at given coordinates with
the gradient of every factor.

`run` computes each in a plain form (elementary torch operations in 32 bits) or, where `own` is true,
through the framework's entry points."""
import functools
import operator

import numpy as np
import torch

own = False

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2, "int32": 4, "int64": 8}
MASKED = 0.02  # share of the tokens or samples that are padding (index -1)


# ----------------------------------------------------------------- cases

def _table(kind, name=None, *, tokens, rows, width, type, index="int64", skew=1.0, out="", scale=1.0):
    """kind: lookup or lookup_grad; skew: tokens are drawn as rows * u^skew, so a few rows are met often."""
    case = {"kind": kind, "tokens": tokens, "rows": rows, "width": width, "type": type, "index": index,
            "skew": skew, "scale": scale}
    if kind == "lookup_grad":
        case["out"] = out or type
    return {"name": name, **case} if name else case


def _grads(name=None, *, tensors, numel, type, clips=True, packed=False):
    """packed: the gradients are views of one buffer without gaps, at any offset; the raw ones are kept
    (to retry a step, to log them), the clipped ones go to a buffer of their own."""
    case = {"kind": "clip", "tensors": tensors, "numel": numel, "type": type, "clips": clips, "packed": packed}
    return {"name": name, **case} if name else case


def _model(kind, name=None, *, order, size, rank, samples, type="float32", index="int32", skew=1.0):
    """kind: entries or entries_grad of an order-way tensor, every mode of `size` indices (the last: one more)."""
    case = {"kind": kind, "order": order, "size": size, "rank": rank, "samples": samples, "type": type,
            "index": index, "skew": skew}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one token's row, as asked for at every step of a generation: latency alone
        _table("lookup", "lookup one", tokens=1, rows=65536, width=2000, type="bfloat16"),
        # a training batch's tokens from a large table, a few of them frequent
        _table("lookup", "lookup batch", tokens=16384, rows=131072, width=1024, type="bfloat16", skew=3.0, scale=32.0),
        # a long batch over a table whose rows start at any 4-byte offset
        _table("lookup", "lookup long odd", tokens=200003, rows=100003, width=1001, type="float32", index="int32"),
        # the rows of one small factor matrix that a minibatch touched
        _table("lookup_grad", "lookup grad few", tokens=48, rows=512, width=256, type="float32", index="int32"),
        # the same batch's gradient: most of the table gets zeros
        _table("lookup_grad", "lookup grad batch", tokens=16384, rows=131072, width=1024, type="bfloat16",
               skew=3.0, out="float32", scale=32.0),
        # many tokens over a small table: each row sums many, the first ones thousands
        _table("lookup_grad", "lookup grad long", tokens=524288, rows=32768, width=512, type="bfloat16", skew=3.0),
        # the factor gradients of a 512^3 model of rank 2000
        _grads("clip factors", tensors=3, numel=3 * 512 * 2000, type="float32"),
        # the gradients of a network: many matrices, as many short vectors
        _grads("clip many", tensors=194, numel=96_000_000, type="bfloat16"),
        # few large gradients in 32 bits, far more than the caches hold
        _grads("clip large", tensors=24, numel=512_000_000, type="float32"),
        # a million observed entries of a six-way tensor
        _model("entries", "entries 6-way", order=6, size=20, rank=128, samples=1_000_003),
        # a small minibatch
        _model("entries_grad", "entries grad small", order=3, size=256, rank=64, samples=4096),
        # a large minibatch of a three-way tensor
        _model("entries_grad", "entries grad 3-way", order=3, size=512, rank=256, samples=262144),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    kind = rng.choice(["lookup", "lookup_grad", "clip", "entries", "entries_grad"])
    type = rng.choice(["float32", "bfloat16", "float16"])
    index = rng.choice(["int32", "int64"])
    skew = rng.choice([1.0, 1.0, 2.0, 3.0])
    if kind in ("lookup", "lookup_grad"):
        width = log(8, 4096)
        rows = min(log(512, 262144), (1 << 27) // width)
        tokens = min(log(1, 524288), (1 << 27) // width)
        out = rng.choice(["float32", type])
        return _table(kind, tokens=tokens, rows=rows, width=width, type=type, index=index, skew=skew, out=out,
                      scale=rng.choice([1.0, 0.125, 32.0]))
    if kind == "clip":
        tensors = log(1, 400)
        return _grads(tensors=tensors, numel=max(tensors, log(1000, 400_000_000)), type=type,
                      clips=rng.random() < 0.7, packed=rng.random() < 0.3)
    order = rng.randint(2, 6)
    rank = log(8, 2000)
    most = 1_000_003 * 128 * 6 // (order * rank) if kind == "entries" else 262144 * 256 * 3 // (order * rank)
    return _model(kind, order=order, size=log(20, 2000), rank=rank, samples=min(log(100, 1_000_003), most),
                  type=type, index=index, skew=skew)


# ----------------------------------------------------------------- inputs

def _indices(gen, count, rows, case, valid=None):
    """`count` indices below `rows`, -1 where not valid."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    idx = (rows * u ** case["skew"]).long().clamp_(max=rows - 1)
    if valid is not None:
        idx = torch.where(valid, idx, -1)
    return idx.to(getattr(torch, case["index"]))


def _normal(gen, shape, case, std=1.0):
    x = torch.randn(shape, generator=gen, device="cuda")
    return x.mul_(std).to(TYPES[case["type"]])


def _valid(gen, count):
    return torch.rand(count, generator=gen, device="cuda") >= (MASKED if count > 1 else 0.0)


def _sizes(case):
    """The tensors' sizes, by the case alone: matrices and, after each, a short vector."""
    count, numel = case["tensors"], case["numel"]
    if count == 3:
        return [numel // 3, numel // 3, numel - 2 * (numel // 3)]
    most = max(1, numel // (16 * count))
    sizes = [0 if k % 2 == 0 else 1 + (k * 7919) % min(4096, most) for k in range(count)]
    matrices = [k for k in range(count) if k % 2 == 0]
    left = numel - sum(sizes)
    weights = [1 + (k * 31) % 7 for k in matrices]
    for k, w in zip(matrices, weights):
        sizes[k] = left * w // sum(weights)
    sizes[0] += numel - sum(sizes)
    return sizes


def _views(flat, sizes, packed):
    """Consecutive parts of one buffer, each at a multiple of 128 elements unless packed."""
    views, at = [], 0
    for n in sizes:
        views.append(flat[at:at + n])
        at += n if packed else -(-n // 128) * 128
    return views


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    state = {"case": case}
    if kind in ("lookup", "lookup_grad"):
        n = case["tokens"]
        state["idx"] = _indices(gen, n, case["rows"], case, _valid(gen, n))
        if kind == "lookup":
            state["table"] = _normal(gen, (case["rows"], case["width"]), case, 0.02)
        else:
            state["grad"] = _normal(gen, (n, case["width"]), case, 1e-2)
    elif kind == "clip":
        sizes = _sizes(case)
        room = sum(sizes) if case["packed"] else sum(-(-n // 128) * 128 for n in sizes)
        if case["packed"]:
            state["tensors"] = _views(_normal(gen, (room,), case, 1e-2), sizes, True)
        else:
            state["tensors"] = [_normal(gen, (n,), case, 1e-2) for n in sizes]
        state["flat"] = torch.zeros(room, device="cuda", dtype=TYPES[case["type"]])
        state["outs"] = _views(state["flat"], sizes, case["packed"])
        # the norm is about 0.01 sqrt(numel): a tenth of it is kept, or all
        state["max_norm"] = (1e-3 if case["clips"] else 1.0) * case["numel"] ** 0.5
    else:
        sizes = _dims(case)
        state["factors"] = [_normal(gen, (n, case["rank"]), case, 1.0) for n in sizes]
        valid = _valid(gen, case["samples"])
        state["dims"] = torch.tensor(sizes, device="cuda")
        state["coords"] = torch.stack([_indices(gen, case["samples"], n, case, valid) for n in sizes], 1)
        if kind == "entries_grad":
            state["g"] = torch.randn(case["samples"], generator=gen, device="cuda") / case["samples"]
    return state


def _dims(case):
    return [case["size"]] * (case["order"] - 1) + [case["size"] + 1]


# ----------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import dense_tensor_decomposition_gb300 as mk
    case = state["case"]
    kind = case["kind"]
    if kind == "lookup":
        return mk.embedding(state["table"], state["idx"], scale=case["scale"])
    if kind == "lookup_grad":
        return mk.embedding_grad(state["idx"], state["grad"], case["rows"], scale=case["scale"],
                                 dtype=TYPES[case["out"]])
    if kind == "clip":
        norm = mk.clip_grad_norm(state["tensors"], state["max_norm"], outs=state["outs"])
        return {"norm": norm, "clipped": state["flat"]}
    if kind == "entries":
        return mk.cp_entries(state["factors"], state["coords"])
    return mk.cp_entries_grad(state["factors"], state["coords"], state["g"])


def _run_plain(state):
    case = state["case"]
    kind = case["kind"]
    if kind == "lookup":
        idx, table = state["idx"].long(), state["table"]
        inside = (idx >= 0) & (idx < case["rows"])
        rows = table[idx.clamp(0, case["rows"] - 1)].float() * case["scale"]
        return torch.where(inside[:, None], rows, 0.0).to(table.dtype)
    if kind == "lookup_grad":
        idx = state["idx"].long()
        inside = (idx >= 0) & (idx < case["rows"])
        g = torch.where(inside[:, None], state["grad"].float() * case["scale"], 0.0)
        out = torch.zeros(case["rows"], case["width"], device=g.device)
        return out.index_add_(0, idx.clamp(0, case["rows"] - 1), g).to(TYPES[case["out"]])
    if kind == "clip":
        norm = torch.stack([t.float().square().sum() for t in state["tensors"]]).sum().sqrt()
        coef = (state["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        [o.copy_(t.float() * coef) for t, o in zip(state["tensors"], state["outs"])]
        return {"norm": norm, "clipped": state["flat"]}
    coords = state["coords"].long()
    inside = ((coords >= 0) & (coords < state["dims"])).all(1)
    coords = torch.where(inside[:, None], coords, 0)
    rows = [f[coords[:, n]].float() for n, f in enumerate(state["factors"])]
    if kind == "entries":
        return torch.where(inside, functools.reduce(operator.mul, rows).sum(1), 0.0)
    g = torch.where(inside, state["g"], 0.0)[:, None]
    others = [functools.reduce(operator.mul, rows[:n] + rows[n + 1:], g) for n in range(case["order"])]
    return [torch.zeros(f.shape, device=g.device).index_add_(0, coords[:, n], others[n])
            for n, f in enumerate(state["factors"])]


# ----------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definitions: gradients by differentiating the forward formula in 64 bits."""
    state = prepare(case, seed)
    kind = case["kind"]
    if kind in ("lookup", "lookup_grad"):
        idx, rows = state["idx"], case["rows"]
        kept = torch.nonzero((idx > -1) & (idx < rows)).flatten()
        if kind == "lookup":
            out = torch.zeros(case["tokens"], case["width"], device="cuda", dtype=torch.float64)
            out[kept] = state["table"].index_select(0, idx[kept]).double() * case["scale"]
            return out
        table = torch.zeros(rows, case["width"], device="cuda", dtype=torch.float64, requires_grad=True)
        for part in kept.split(65536):
            (table[idx[part].long()] * case["scale"]).backward(state["grad"][part].double())
        return table.grad if table.grad is not None else torch.zeros_like(table)
    if kind == "clip":
        norm = sum(float(part.double().pow(2).sum()) for t in state["tensors"] for part in t.split(1 << 25)) ** 0.5
        coef = min(1.0, state["max_norm"] / (norm + 1e-6))
        flat = torch.zeros(state["flat"].shape, device="cuda", dtype=torch.float64)
        sizes = _sizes(case)
        for t, o in zip(state["tensors"], _views(flat, sizes, case["packed"])):
            o.copy_(t).mul_(coef)
        return {"norm": torch.tensor(norm, dtype=torch.float64), "clipped": flat}
    factors = [f.double().requires_grad_(kind == "entries_grad") for f in state["factors"]]
    x = torch.zeros(case["samples"], device="cuda", dtype=torch.float64)
    kept = torch.nonzero(((state["coords"] > -1) & (state["coords"] < state["dims"])).all(1)).flatten()
    for part in kept.split(max(1, (1 << 24) // case["rank"])):
        at = state["coords"][part].long()
        values = torch.stack([f[at[:, n]] for n, f in enumerate(factors)]).prod(0).sum(1)
        if kind == "entries":
            x[part] = values
        else:
            values.backward(state["g"][part].double())
    if kind == "entries":
        return x
    return [f.grad if f.grad is not None else torch.zeros_like(f) for f in factors]


# ----------------------------------------------------------------- what a pass cannot do without

def _distinct(count, rows, skew):
    """How many of `rows` rows are met by `count` draws of rows * u^skew, on average."""
    edges = (np.arange(rows + 1) / rows) ** (1.0 / skew)
    return float(-np.expm1(count * np.log1p(-np.minimum(np.diff(edges), 1 - 1e-12))).sum())


def work(case):
    kind, e = case["kind"], SIZE[case["type"]]
    if kind in ("lookup", "lookup_grad"):
        n, d = case["tokens"], case["width"]
        flops, indices = n * d, n * SIZE[case["index"]]
        if kind == "lookup":
            return {"bytes": indices + (n + _distinct(n, case["rows"], case["skew"])) * d * e, "flops": flops}
        return {"bytes": indices + n * d * e + case["rows"] * d * SIZE[case["out"]], "flops": flops}
    if kind == "clip":
        return {"bytes": 2 * case["numel"] * e + 4, "flops": 3 * case["numel"]}
    s, d, r = case["samples"], case["order"], case["rank"]
    read = s * d * SIZE[case["index"]] + sum(_distinct(s, n, case["skew"]) for n in _dims(case)) * r * e
    if kind == "entries":
        return {"bytes": read + 4 * s, "flops": s * r * d}
    return {"bytes": read + 4 * s + 4 * r * sum(_dims(case)), "flops": s * r * (4 * d - 5)}
