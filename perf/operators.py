"""Cases of the language-model operators around the library's matrix-vector products.

Four operators on the two dense tables of a language model, the one its tokens index and the one
that its answers come from:

* ``q4_run``    y = A·x + c with A held as 4-bit codes and one scale (and, optionally, a zero
                point) per group of a row's columns: the product of a decoding step;
* ``quantize``  the conversion of a dense matrix into those codes, with the values that the codes
                stand for (what training with rounded weights, or a look at the loss, needs);
* ``embed``     the rows of a table, dense or 4-bit, that a list of tokens names, times a scale;
* ``grad``      the gradient of that lookup, summed by token: overwriting a dense gradient, or
                adding to one that a run of micro-batches accumulates.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once)
or, where ``own`` is true, by the library's calls. ``exact`` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def ceil_div(a, b):
    return -(-a // b)


# --- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a small model's layer: nothing but latency
        {"name": "q4 1024x1024, one vector", "op": "q4_run", "rows": 1024, "cols": 1024,
         "group": 32, "n": 1, "x": "bf16", "y": "bf16", "scale": "bf16", "zeros": False,
         "residual": False},
        # the output projection of a large layer for one token, added to the residual stream
        {"name": "q4 8192x28672, residual", "op": "q4_run", "rows": 8192, "cols": 28672,
         "group": 128, "n": 1, "x": "bf16", "y": "bf16", "scale": "f16", "zeros": False,
         "residual": True},
        # logits over a large vocabulary in 32 bits, the type of the library's other products
        {"name": "q4 131072x4096, f32 logits", "op": "q4_run", "rows": 131072, "cols": 4096,
         "group": 128, "n": 1, "x": "f32", "y": "f32", "scale": "f32", "zeros": False,
         "residual": False},
        # a batch of requests decoding together, weights with zero points
        {"name": "q4 16384x5120, 16 vectors", "op": "q4_run", "rows": 16384, "cols": 5120,
         "group": 64, "n": 16, "x": "f16", "y": "f16", "scale": "f16", "zeros": True,
         "residual": False},
        # odd sizes: a last group, a last byte and a last row block that are not full
        {"name": "q4 5003x4099, 3 vectors", "op": "q4_run", "rows": 5003, "cols": 4099,
         "group": 32, "n": 3, "x": "bf16", "y": "f32", "scale": "bf16", "zeros": True,
         "residual": True},
        # a small 32-bit matrix converted with 16-bit scales
        {"name": "quantize 1536x1000 f32", "op": "quantize", "rows": 1536, "cols": 1000,
         "group": 32, "w": "f32", "scale": "f16", "zeros": False},
        # one large layer of a model converted, with zero points
        {"name": "quantize 28672x8192 bf16", "op": "quantize", "rows": 28672, "cols": 8192,
         "group": 128, "w": "bf16", "scale": "bf16", "zeros": True},
        # the token that a decoding step starts from
        {"name": "embed 1 token of 131072x4096", "op": "embed", "vocab": 131072, "dim": 4096,
         "tokens": 1, "table": "bf16", "out": "bf16", "index": 64, "pad": 0.0},
        # a batch of ragged prompts or training sequences, padded, from a 32-bit table
        {"name": "embed 32768 of 65536x4096 f32", "op": "embed", "vocab": 65536, "dim": 4096,
         "tokens": 32768, "table": "f32", "out": "bf16", "index": 64, "pad": 0.05},
        # a prompt looked up in a 4-bit table that also serves as the output projection
        {"name": "embed 4096 of 131072x5120 q4", "op": "embed", "vocab": 131072, "dim": 5120,
         "tokens": 4096, "table": "q4", "group": 64, "scale": "bf16", "out": "bf16",
         "index": 32, "pad": 0.0},
        # one micro-batch of a small model added to a 32-bit gradient
        {"name": "grad 2048 of 32768x1000", "op": "grad", "vocab": 32768, "dim": 1000,
         "tokens": 2048, "g": "f32", "out": "f32", "index": 64, "pad": 0.05, "add": True},
        # a large training batch, the whole dense gradient written
        {"name": "grad 32768 of 131072x4096", "op": "grad", "vocab": 131072, "dim": 4096,
         "tokens": 32768, "g": "bf16", "out": "bf16", "index": 64, "pad": 0.02, "add": False},
    ]


def _spread(rng, low, high):
    """A whole number between the two, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _draw_once(rng):
    op = rng.choice(["q4_run", "q4_run", "quantize", "embed", "grad"])
    t = lambda: rng.choice(["f32", "f16", "bf16"])  # noqa: E731
    if op in ("q4_run", "quantize"):
        rows, cols = _spread(rng, 64, 131072), _spread(rng, 64, 32768)
        if rng.random() < 0.6:  # most layers are whole multiples of a group
            cols = max(64, cols // 64 * 64)
        c = {"op": op, "rows": rows, "cols": cols, "group": rng.choice([32, 64, 128]),
             "scale": t(), "zeros": rng.random() < 0.5}
        if op == "quantize":
            c["w"] = t()
            return c
        x = t()
        c.update(n=rng.choice([1, 1, 2, 4, rng.randint(3, 16)]), x=x,
                 y=rng.choice([x, "f32"]), residual=rng.random() < 0.5)
        return c
    c = {"op": op, "vocab": _spread(rng, 256, 131072), "dim": _spread(rng, 64, 8192),
         "tokens": _spread(rng, 1, 32768), "index": rng.choice([32, 64]),
         "pad": rng.choice([0.0, 0.05])}
    if rng.random() < 0.6:
        c["dim"] = max(64, c["dim"] // 64 * 64)
    if op == "embed":
        c["table"] = rng.choice(["f32", "f16", "bf16", "q4"])
        if c["table"] == "q4":
            c.update(group=rng.choice([32, 64, 128]), scale=t())
        c["out"] = t() if c["table"] in ("f32", "q4") else c["table"]
        return c
    g = t()
    c.update(g=g, out=rng.choice([g, "f32"]), add=rng.random() < 0.5)
    return c


def _cost(c):
    """Rough bytes that the plain form of a case moves: what bounds a drawn case."""
    if c["op"] in ("q4_run", "quantize"):
        return c["rows"] * c["cols"] * 4
    return (c["vocab"] + 2 * c["tokens"]) * c["dim"] * 4


def draw(rng):
    """One more case of the listed ones' ranges, no larger than the largest of its operator."""
    while True:
        c = _draw_once(rng)
        if _cost(c) <= max(_cost(k) for k in listed() if k["op"] == c["op"]):
            return c


# --- inputs ------------------------------------------------------------------------------------
def _probabilities(vocab):
    """How often each token comes: by its rank, as words do in text."""
    return 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)


def _tokens(case, seed):
    """Token numbers with the frequencies of text, a share of them padding (-1)."""
    rng = np.random.default_rng(seed)
    reach = np.cumsum(_probabilities(case["vocab"]))
    rank = np.searchsorted(reach, rng.random(case["tokens"]) * reach[-1], side="right")
    t = rng.permutation(case["vocab"])[np.minimum(rank, case["vocab"] - 1)]
    if case["pad"]:
        t[rng.random(case["tokens"]) < case["pad"]] = -1
    return torch.from_numpy(t.astype(np.int64 if case["index"] == 64 else np.int32)).cuda()


def _codes(rows, cols, group, scale, zeros, gen):
    """4-bit codes of normal weights (two to a byte, the earlier column in the low half), a scale
    for each group and, if asked for, its zero point."""
    groups = ceil_div(cols, group)

    def half():
        q = torch.randn(rows, ceil_div(cols, 2), device="cuda", generator=gen)
        return q.mul_(2.6).add_(8.0).round_().clamp_(0, 15).to(torch.uint8)

    codes = half()
    codes |= half() << 4
    scales = torch.rand(rows, groups, device="cuda", generator=gen).add_(0.5).mul_(0.008)
    z = (torch.randint(6, 11, (rows, groups), device="cuda", generator=gen).to(torch.uint8)
         if zeros else None)
    return codes, scales.to(TYPES[scale]), z


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, size=1.0):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(size)

    s = {"case": case}
    if op == "q4_run":
        rows, cols, n = case["rows"], case["cols"], case["n"]
        s["codes"], s["scales"], s["zeros"] = _codes(rows, cols, case["group"], case["scale"],
                                                     case["zeros"], gen)
        s["x"] = normal(n, cols).to(TYPES[case["x"]])
        s["c"] = normal(n, rows).to(TYPES[case["y"]]) if case["residual"] else None
        s["y"] = torch.empty(n, rows, dtype=TYPES[case["y"]], device="cuda")
    elif op == "quantize":
        rows, cols, w = case["rows"], case["cols"], TYPES[case["w"]]
        groups = ceil_div(cols, case["group"])
        s["w"] = normal(rows, cols, size=0.02).to(w)
        s["codes"] = torch.empty(rows, ceil_div(cols, 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(rows, groups, dtype=TYPES[case["scale"]], device="cuda")
        s["zeros"] = (torch.empty(rows, groups, dtype=torch.uint8, device="cuda")
                      if case["zeros"] else None)
        s["back"] = torch.empty_like(s["w"])
    elif op == "embed":
        s["tokens"] = _tokens(case, seed)
        if case["table"] == "q4":
            s["codes"], s["scales"], _ = _codes(case["vocab"], case["dim"], case["group"],
                                                case["scale"], False, gen)
        else:
            s["table"] = normal(case["vocab"], case["dim"]).to(TYPES[case["table"]])
        s["out"] = torch.empty(case["tokens"], case["dim"], dtype=TYPES[case["out"]],
                               device="cuda")
    else:
        s["tokens"] = _tokens(case, seed)
        s["g"] = normal(case["tokens"], case["dim"]).to(TYPES[case["g"]])
        # a gradient that is added to keeps its sums from pass to pass; one that is written does not
        s["dtable"] = (normal(case["vocab"], case["dim"]).to(TYPES[case["out"]]) if case["add"]
                       else torch.empty(case["vocab"], case["dim"], dtype=TYPES[case["out"]],
                                        device="cuda"))
    return s


def _factor(case):
    """The scale of a lookup: the square root of the width, as where a table also answers."""
    return math.sqrt(case["dim"])


# --- one pass ----------------------------------------------------------------------------------
def _unpack(codes, cols):
    return torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)[:, :cols]


def _spread_groups(v, group, cols):
    return v.float().repeat_interleave(group, 1)[:, :cols]


def _values(codes, scales, zeros, group, cols):
    q = _unpack(codes, cols).float()
    q -= 8.0 if zeros is None else _spread_groups(zeros, group, cols)
    return q.mul_(_spread_groups(scales, group, cols))


def _plain_quantize(w, group, scale_type, with_zeros):
    rows, cols = w.shape
    groups = ceil_div(cols, group)
    full = torch.zeros(rows, groups * group, device=w.device)
    full[:, :cols] = w
    f = full.view(rows, groups, group)
    if with_zeros:
        low, high = f.amin(2).clamp_(max=0), f.amax(2).clamp_(min=0)
        scales = ((high - low) / 15.0).to(scale_type)
        step = scales.float()
        safe = torch.where(step > 0, step, torch.ones_like(step))
        zeros = (-low / safe).round_().clamp_(0, 15)
        zeros = torch.where(step > 0, zeros, torch.zeros_like(zeros))
    else:
        scales = (f.abs().amax(2) / 7.0).to(scale_type)
        step = scales.float()
        safe = torch.where(step > 0, step, torch.ones_like(step))
        zeros = torch.full_like(step, 8.0)
    q = (f / safe[..., None]).round_().add_(zeros[..., None]).clamp_(0, 15)
    back = ((q - zeros[..., None]) * step[..., None]).view(rows, -1)[:, :cols]
    return scales, zeros.to(torch.uint8) if with_zeros else None, back.to(w.dtype)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "q4_run":
        a = _values(s["codes"], s["scales"], s["zeros"], case["group"], case["cols"])
        y = s["x"].float() @ a.t()
        if s["c"] is not None:
            y += s["c"].float()
        return y.to(s["y"].dtype)
    if op == "quantize":
        scales, zeros, back = _plain_quantize(s["w"], case["group"], s["scales"].dtype,
                                              case["zeros"])
        return {"scales": scales, "zeros": zeros, "back": back}
    t = s["tokens"].long()
    kept = t >= 0
    if op == "embed":
        at = t.clamp(min=0)
        if case["table"] == "q4":
            v = _values(s["codes"][at], s["scales"][at], None, case["group"], case["dim"])
        else:
            v = s["table"][at].float()
        return (v * _factor(case) * kept[:, None]).to(s["out"].dtype)
    sums = torch.zeros(case["vocab"], case["dim"], device="cuda")
    sums.index_add_(0, t[kept], s["g"][kept].float())
    sums *= _factor(case)
    if case["add"]:
        sums += s["dtable"].float()
    return s["dtable"].copy_(sums)


def _own(s):
    import spmv_sparse_storage_gb300 as sp
    case, op = s["case"], s["case"]["op"]
    if op == "q4_run":
        sp.spmv_q4_run(s["codes"], s["scales"], case["group"], s["x"], s["y"], c=s["c"],
                       zeros=s["zeros"])
        return s["y"]
    if op == "quantize":
        sp.spmv_q4_quantize(s["w"], s["codes"], s["scales"], case["group"], zeros=s["zeros"],
                            back=s["back"])
        return {"scales": s["scales"], "zeros": s["zeros"], "back": s["back"]}
    if op == "embed":
        if case["table"] == "q4":
            sp.spmv_embed_q4(s["codes"], s["scales"], case["group"], s["tokens"], s["out"],
                             scale=_factor(case))
        else:
            sp.spmv_embed(s["table"], s["tokens"], s["out"], scale=_factor(case))
        return s["out"]
    sp.spmv_embed_grad(s["g"], s["tokens"], s["dtable"], scale=_factor(case),
                       accumulate=case["add"])
    return s["dtable"]


def run(state):
    return _own(state) if own else _plain(state)


# --- what a pass cannot do without ---------------------------------------------------------------
def _distinct(case):
    """Expected number of distinct tokens, padding apart."""
    p = _probabilities(case["vocab"])
    t = case["tokens"] * (1.0 - case["pad"])
    return float(-np.expm1(t * np.log1p(-p / p.sum())).sum()) if case["vocab"] > 1 else 1.0


def work(case):
    op = case["op"]
    if op in ("q4_run", "quantize"):
        rows, cols = case["rows"], case["cols"]
        per_group = SIZE[case["scale"]] + (1 if case["zeros"] else 0)
        held = rows * (ceil_div(cols, 2) + ceil_div(cols, case["group"]) * per_group)
        if op == "quantize":
            return {"bytes": held + 2 * rows * cols * SIZE[case["w"]], "flops": 6 * rows * cols}
        n = case["n"]
        ends = n * (cols * SIZE[case["x"]] + rows * SIZE[case["y"]] * (1 + case["residual"]))
        return {"bytes": held + ends, "flops": 2 * rows * cols * n}
    tokens, dim, used = case["tokens"], case["dim"], _distinct(case)
    ids = tokens * case["index"] // 8
    if op == "embed":
        row = (ceil_div(dim, 2) + ceil_div(dim, case["group"]) * SIZE[case["scale"]]
               if case["table"] == "q4" else dim * SIZE[case["table"]])
        return {"bytes": ids + used * row + tokens * dim * SIZE[case["out"]],
                "flops": tokens * dim}
    kept = tokens * (1.0 - case["pad"])
    written = 2 * used if case["add"] else case["vocab"]
    return {"bytes": ids + kept * dim * SIZE[case["g"]] + written * dim * SIZE[case["out"]],
            "flops": kept * dim}


# --- the definition in 64 bits -------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "q4_run":
        rows, cols, group = case["rows"], case["cols"], case["group"]
        x = s["x"].double()
        y = torch.empty(case["n"], rows, dtype=torch.float64, device="cuda")
        column = torch.arange(cols, device="cuda")
        for r in range(0, rows, 8192):  # a block of rows at a time, in 64 bits
            b = s["codes"][r:r + 8192][:, column // 2]
            q = torch.where(column % 2 == 0, b % 16, b // 16).double()
            z = (s["zeros"][r:r + 8192][:, column // group].double() if case["zeros"]
                 else torch.tensor(8.0, dtype=torch.float64, device="cuda"))
            y[:, r:r + 8192] = torch.matmul(
                x, ((q - z) * s["scales"][r:r + 8192][:, column // group].double()).t())
        return y if s["c"] is None else y + s["c"].double()
    if op == "quantize":  # the steps round: what they give is the same in more bits
        w, group = s["w"].double(), case["group"]
        rows, cols = w.shape
        scales, zeros, back = [], [], torch.empty_like(w)
        for c in range(0, cols, group):
            part = w[:, c:c + group]
            if case["zeros"]:
                low = torch.minimum(part.min(1).values, torch.zeros(rows, device="cuda").double())
                high = torch.maximum(part.max(1).values, torch.zeros(rows, device="cuda").double())
                raw = (high - low) / 15
            else:
                raw = part.abs().max(1).values / 7
            held = raw.to(s["scales"].dtype).double()  # a scale is held in its own type
            z = torch.round(-low / held).clamp(0, 15) if case["zeros"] else torch.full_like(raw, 8)
            q = (torch.round(part / held[:, None]) + z[:, None]).clamp(0, 15)
            back[:, c:c + group] = (q - z[:, None]) * held[:, None]
            scales.append(raw)
            zeros.append(z)
        return {"scales": torch.stack(scales, 1), "zeros": None, "back": back}
    t = s["tokens"].cpu().numpy().astype(np.int64)
    kept = np.flatnonzero(t >= 0)
    factor = math.sqrt(case["dim"])
    if op == "embed":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        at, rows = torch.from_numpy(kept).cuda(), torch.from_numpy(t[kept]).cuda()
        if case["table"] == "q4":
            column = torch.arange(case["dim"], device="cuda")
            b = s["codes"][rows][:, column // 2]
            q = torch.where(column % 2 == 0, b % 16, b // 16).double() - 8
            out[at] = q * s["scales"][rows][:, column // case["group"]].double() * factor
        else:
            out[at] = s["table"][rows].double() * factor
        return out
    # gradients: the tokens in order, then differences of the running sums of their rows
    order = kept[np.argsort(t[kept], kind="stable")]
    names, first = np.unique(t[order], return_index=True)
    last = np.append(first[1:], len(order))
    sums = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    if len(order):
        ordered = torch.from_numpy(order).cuda()
        names, first, last = (torch.from_numpy(v).cuda() for v in (names, first, last))
        for c in range(0, case["dim"], 512):  # a block of columns at a time
            running = torch.zeros(len(order) + 1, min(512, case["dim"] - c), dtype=torch.float64,
                                  device="cuda")
            torch.cumsum(s["g"][:, c:c + 512][ordered].double(), 0, out=running[1:])
            sums[names, c:c + 512] = (running[last] - running[first]) * factor
    return sums + s["dtable"].double() if case["add"] else sums
