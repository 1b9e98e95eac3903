"""Operators around orthogonal matrices, as measured: rotations of rows by their position with the
gradient, matrices orthogonalised by Newton-Schulz products, and the training step that applies such
an update to its weights.

`run` computes each in a plain form (elementary torch operations in 32 bits, angles in 64) or, where
`own` is true, through the framework's entry points."""
import math

import torch

own = False

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2, "int32": 4, "int64": 8}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # of the quintic, every step
STEPS = 5
EPS = 1e-7
MOMENTUM, LR, DECAY = 0.95, 0.02, 0.1


# ----------------------------------------------------------------- cases

def _rotary(kind, name=None, *, batch, length, heads, kv_heads, width, dims, type, interleaved=False,
            layout="bthd", positions="range", index="int64", base=10000.0, factor=1.0, scale=1.0):
    """kind: rotary or rotary_grad. heads of one tensor and kv_heads of a second one (0: there is none), rows of
    `width` of which the first `dims` are rotated. layout: the order in memory of batch, length (t), heads, width.
    positions: range (the same for every sequence), ragged (one behind the last of each sequence's past) or random."""
    case = {"kind": kind, "batch": batch, "length": length, "heads": heads, "kv_heads": kv_heads, "width": width,
            "dims": dims, "type": type, "interleaved": interleaved, "layout": layout, "positions": positions,
            "index": index, "base": base, "factor": factor, "scale": scale}
    return {"name": name, **case} if name else case


def _matrices(kind, name=None, *, count, rows, cols, type, batched=False, varied=False, weights="float32",
              momenta="float32", nesterov=True):
    """kind: orthogonalize or step. batched: one tensor of `count` matrices instead of a list of them; varied: every
    second matrix is turned, and each a little smaller than the one before."""
    case = {"kind": kind, "count": count, "rows": rows, "cols": cols, "type": type, "batched": batched,
            "varied": varied}
    if kind == "step":
        case.update(weights=weights, momenta=momenta, nesterov=nesterov)
    return {"name": name, **case} if name else case


def listed():
    return [
        # one token of each of eight sequences, far into long contexts: latency alone
        _rotary("rotary", "rotary tokens", batch=8, length=1, heads=32, kv_heads=8, width=128, dims=128,
                type="bfloat16", positions="ragged", base=500000.0, factor=8.0),
        # the queries and keys of a long batch
        _rotary("rotary", "rotary batch", batch=4, length=4096, heads=32, kv_heads=8, width=128, dims=128,
                type="bfloat16"),
        # rows of a factor matrix turned by the time they were observed at, neighbouring columns a pair
        _rotary("rotary", "rotary rows", batch=1, length=200003, heads=1, kv_heads=0, width=256, dims=256,
                type="float32", interleaved=True, positions="random", index="int32"),
        # the gradient of an odd batch whose heads lie outside the tokens and are rotated in part
        _rotary("rotary_grad", "rotary grad part", batch=3, length=1001, heads=20, kv_heads=4, width=96, dims=64,
                type="float16", layout="bhtd", scale=1.2),
        # the gradient of the long batch, in 32 bits
        _rotary("rotary_grad", "rotary grad batch", batch=2, length=8192, heads=16, kv_heads=16, width=128, dims=128,
                type="float32", interleaved=True),
        # the update of one small factor matrix
        _matrices("orthogonalize", "orthogonalize small", count=1, rows=256, cols=64, type="float32"),
        # the factors of a 512^3 model of rank 2000
        _matrices("orthogonalize", "orthogonalize factors", count=3, rows=512, cols=2000, type="float32"),
        # the matrices of many small blocks in one tensor, of an odd size
        _matrices("orthogonalize", "orthogonalize blocks", count=64, rows=501, cols=333, type="bfloat16", batched=True),
        # a network's matrices of different sizes, 16-bit gradients
        _matrices("orthogonalize", "orthogonalize network", count=12, rows=1024, cols=4096, type="bfloat16",
                  varied=True),
        # a training step of the six factors of a 20^6 model of rank 128
        _matrices("step", "step factors", count=6, rows=20, cols=128, type="float32"),
        # a network's training step: 16-bit gradients and weights
        _matrices("step", "step network", count=8, rows=2048, cols=1360, type="bfloat16", varied=True,
                  weights="bfloat16"),
        # the training step of two large square matrices, weights in 32 bits
        _matrices("step", "step large", count=2, rows=4096, cols=4096, type="bfloat16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    kind = rng.choice(["rotary", "rotary_grad", "orthogonalize", "step"])
    types = ["float32", "bfloat16", "float16"]
    type = rng.choice(types)
    if kind in ("rotary", "rotary_grad"):
        dims = 2 * log(8, 128)
        width = dims if rng.random() < 0.6 else dims + log(1, 128)
        heads, kv_heads = rng.choice([(1, 0), (1, 1), (8, 2), (20, 4), (32, 8), (16, 16)])
        most = (4 * 4096 * 40 * 128) // ((heads + kv_heads) * width)
        batch = log(1, 64)
        length = max(1, min(log(1, 32768), most // batch))
        return _rotary(kind, batch=batch, length=length, heads=heads, kv_heads=kv_heads, width=width, dims=dims,
                       type=type, interleaved=rng.random() < 0.5, layout=rng.choice(["bthd", "bthd", "bhtd"]),
                       positions=rng.choice(["range", "ragged", "random"]), index=rng.choice(["int32", "int64"]),
                       base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 1.0, 4.0, 8.0]),
                       scale=rng.choice([1.0, 1.0, 1.2]))
    rows, cols = log(8, 4096), log(8, 4096)
    batched = rng.random() < 0.3
    least, most = min(rows, cols), max(rows, cols)
    cost = least * least * (3 * most + least)
    count = max(1, min(log(1, 64 if batched else 32), 2 * 4 * 4096 ** 3 // cost))
    return _matrices(kind, count=count, rows=rows, cols=cols, type=type, batched=batched,
                     varied=not batched and rng.random() < 0.5, weights=rng.choice(["float32", type]),
                     momenta=rng.choice(["float32", type]), nesterov=rng.random() < 0.7)


# ----------------------------------------------------------------- inputs

def _frequencies(case):
    """Radians a position: base^(-2i / dims), those of long waves divided by `factor` (waves that turn less than once
    in 8192 positions; between 1 and 4 turns, in part)."""
    half = case["dims"] // 2
    freqs = []
    for i in range(half):
        f = case["base"] ** (-i / half)
        turns = 8192 * f / (2 * math.pi)
        share = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        freqs.append(f * (share + (1.0 - share) / case["factor"]))
    return torch.tensor(freqs, dtype=torch.float64)


def _shapes(case):
    shapes = []
    for k in range(case["count"]):
        r, c = case["rows"], case["cols"]
        if case["varied"]:
            r, c = max(1, r - r * k // (5 * case["count"])), max(1, c - c * k // (6 * case["count"]))
            r, c = (c, r) if k % 2 else (r, c)
        shapes.append((r, c))
    return shapes


def _gradient(gen, lead, shape, type):
    """A few strong directions over noise a tenth as large, as gradients of a batch are."""
    r, c = shape
    rank = max(1, min(r, c) // 16)
    u = torch.randn(*lead, r, rank, generator=gen, device="cuda")
    v = torch.randn(*lead, rank, c, generator=gen, device="cuda")
    noise = torch.randn(*lead, r, c, generator=gen, device="cuda")
    return (u @ v / rank ** 0.5 + 0.1 * noise).mul_(1e-3).to(type)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    state = {"case": case}
    if kind in ("rotary", "rotary_grad"):
        b, t = case["batch"], case["length"]
        state["freqs"] = _frequencies(case)
        index = getattr(torch, case["index"])
        if case["positions"] == "range":
            at = torch.arange(t, device="cuda")
        elif case["positions"] == "ragged":
            at = torch.randint(0, 131072, (b, 1), generator=gen, device="cuda") + torch.arange(t, device="cuda")
        else:
            at = torch.randint(0, 1 << 20, (b, t), generator=gen, device="cuda")
        state["positions"] = at.to(index)
        state["tensors"] = []
        for heads in (case["heads"], case["kv_heads"]):
            if heads == 0:
                continue
            if case["layout"] == "bthd":
                x = torch.randn(b, t, heads, case["width"], generator=gen, device="cuda")
                state["tensors"].append(x.to(TYPES[case["type"]]))
            else:
                x = torch.randn(b, heads, t, case["width"], generator=gen, device="cuda")
                state["tensors"].append(x.to(TYPES[case["type"]]).transpose(1, 2))
        return state
    shapes, type = _shapes(case), TYPES[case["type"]]
    if case["batched"]:
        shapes, lead = shapes[:1], (case["count"],)
    else:
        lead = ()
    state["grads"] = [_gradient(gen, lead, s, type) for s in shapes]
    if kind == "step":
        state["momenta"] = [_gradient(gen, lead, s, TYPES[case["momenta"]]).mul_(5.0) for s in shapes]
        state["weights"] = [torch.randn(*lead, *s, generator=gen, device="cuda").mul_(0.02).to(TYPES[case["weights"]])
                            for s in shapes]
        # the raw ones are kept, to take the step back
        state["weights_out"] = [torch.zeros_like(w) for w in state["weights"]]
        state["momenta_out"] = [torch.zeros_like(m) for m in state["momenta"]]
    return state


# ----------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import dense_tensor_decomposition_gb300 as mk
    case = state["case"]
    kind = case["kind"]
    if kind in ("rotary", "rotary_grad"):
        call = mk.rotary if kind == "rotary" else mk.rotary_grad
        return call(state["tensors"], state["positions"], state["freqs"], interleaved=case["interleaved"],
                    scale=case["scale"])
    if kind == "orthogonalize":
        return mk.orthogonalize(state["grads"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    mk.orthogonal_step(state["weights"], state["grads"], state["momenta"], LR, momentum=MOMENTUM,
                       nesterov=case["nesterov"], weight_decay=DECAY, steps=STEPS, coefficients=COEFFICIENTS, eps=EPS,
                       outs=state["weights_out"], momenta_outs=state["momenta_out"])
    return {"weights": state["weights_out"], "momenta": state["momenta_out"]}


def _newton_schulz(g):
    a, b, c = COEFFICIENTS
    x = g / (g.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    turned = x.shape[-2] > x.shape[-1]
    x = x.mT if turned else x
    for _ in range(STEPS):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.mT if turned else x


def _run_plain(state):
    case = state["case"]
    kind = case["kind"]
    if kind in ("rotary", "rotary_grad"):
        angles = state["positions"].double()[..., None] * state["freqs"].cuda()
        sign = 1.0 if kind == "rotary" else -1.0
        cos = (angles.cos() * case["scale"]).float()[..., None, :]
        sin = (angles.sin() * (sign * case["scale"])).float()[..., None, :]
        half, outs = case["dims"] // 2, []
        for x in state["tensors"]:
            part = x[..., :case["dims"]].float()
            if case["interleaved"]:
                u, v = part[..., 0::2], part[..., 1::2]
                turned = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
            else:
                u, v = part[..., :half], part[..., half:]
                turned = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
            outs.append(torch.cat((turned.to(x.dtype), x[..., case["dims"]:]), -1))
        return outs
    if kind == "orthogonalize":
        return [_newton_schulz(g.float()).to(g.dtype) for g in state["grads"]]
    for k, (w, g, m) in enumerate(zip(state["weights"], state["grads"], state["momenta"])):
        kept = MOMENTUM * m.float() + g.float()
        update = g.float() + MOMENTUM * kept if case["nesterov"] else kept
        scale = max(1.0, w.shape[-2] / w.shape[-1]) ** 0.5
        state["weights_out"][k].copy_((1.0 - LR * DECAY) * w.float() - LR * scale * _newton_schulz(update))
        state["momenta_out"][k].copy_(kept)
    return {"weights": state["weights_out"], "momenta": state["momenta_out"]}


# ----------------------------------------------------------------- in 64 bits

def _orthogonal_exact(g):
    """The quintic in the Gram matrix of the shorter side, for the matrix on its long side."""
    x = g.double()
    tall = x.size(-2) >= x.size(-1)
    if not tall:
        x = x.transpose(-1, -2)
    norm = torch.linalg.vector_norm(x.flatten(-2), dim=-1)[..., None, None]
    x = x.div(norm + EPS)
    eye = torch.eye(x.size(-1), dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        gram = torch.matmul(x.transpose(-1, -2), x)
        inner = eye * COEFFICIENTS[0] + torch.matmul(eye * COEFFICIENTS[1] + COEFFICIENTS[2] * gram, gram)
        x = torch.matmul(x, inner)
    return x if tall else x.transpose(-1, -2)


def exact(case, seed):
    """From the definitions: pairs as complex numbers, and the quintic as a function of the Gram matrix."""
    kind = case["kind"]
    if kind in ("orthogonalize", "step") and work(case)["flops"] > 8e12:
        return None
    state = prepare(case, seed)
    if kind in ("rotary", "rotary_grad"):
        turn = torch.outer(state["positions"].flatten().double(), state["freqs"].cuda())
        turn = torch.polar(torch.full_like(turn, case["scale"]), turn if kind == "rotary" else turn.neg())
        turn = turn.view(*state["positions"].shape, 1, -1)
        outs = []
        for x in state["tensors"]:
            out = x.double().contiguous()
            part = out[..., :case["dims"]]
            if case["interleaved"]:
                z = torch.view_as_complex(part.reshape(*part.shape[:-1], -1, 2).contiguous()) * turn
                part.copy_(torch.view_as_real(z).flatten(-2))
            else:
                z = torch.complex(*part.chunk(2, -1)) * turn
                part.copy_(torch.cat((z.real, z.imag), -1))
            outs.append(out)
        return outs
    if kind == "orthogonalize":
        return [_orthogonal_exact(g) for g in state["grads"]]
    weights, momenta = [], []
    for w, g, m in zip(state["weights"], state["grads"], state["momenta"]):
        momenta.append(m.double().mul(MOMENTUM).add(g))
        update = momenta[-1].mul(MOMENTUM).add(g) if case["nesterov"] else momenta[-1]
        ratio = w.size(-2) / w.size(-1)
        step = LR * (math.sqrt(ratio) if ratio > 1 else 1.0)
        weights.append(w.double().mul(1 - LR * DECAY).sub(_orthogonal_exact(update), alpha=step))
    return {"weights": weights, "momenta": momenta}


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    kind, e = case["kind"], SIZE[case["type"]]
    if kind in ("rotary", "rotary_grad"):
        tokens, rows = case["batch"] * case["length"], case["heads"] + case["kv_heads"]
        own_positions = case["length"] if case["positions"] == "range" else tokens
        return {"bytes": 2 * tokens * rows * case["width"] * e + own_positions * SIZE[case["index"]],
                "flops": 3 * tokens * rows * case["dims"]}
    numel = flops = 0
    for r, c in _shapes(case):
        least, most = min(r, c), max(r, c)
        numel += r * c
        # of the symmetric products one half each, and the product with the matrix
        flops += STEPS * least * least * (3 * most + least)
    moved = 2 * e
    if kind == "step":
        moved = e + 2 * SIZE[case["weights"]] + 2 * SIZE[case["momenta"]]
    return {"bytes": moved * numel, "flops": flops}
