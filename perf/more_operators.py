"""The layers whose weight gradients the framework reduces -- an embedding, with
its gradient by sorted tokens, and experts' matrix products over ragged runs of
rows -- as measured calls: their inputs, their plain form in torch and the
framework's own calls.

  lookup   out[i] = scale * table[ids[i] - first], a row of zeros for an id of
           another shard of the table
  sort     the positions i in the order of their rows, equal rows in the order of
           i, without ids of another shard; starts[r] = where row r's begin
  rowgrad  the lookup's gradient, which sorts first: row r's is scale * the sum of
           dy[i] over its i; written over every row, or added to an FP32 array
  forward  y = x W_e^T for the rows x of starts[e] .. starts[e + 1]; W_e is
           [out, in].  Rows behind the last expert's stay as they were
  xgrad    dx = dy W_e
  wgrad    dW_e = dy^T x over the expert's rows; zeros, or what was there, for an
           expert without any
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------- cases
def rows_case(kind, n, rows, width, **more):
    case = {"kind": kind, "n": n, "rows": rows, "width": width, "ids": 64, "table": 16, "dy": 16, "out": 16, "add": False,
            "shards": 1, "pad": 0}
    case.update(more)
    return case


def experts_case(kind, rows, experts, inner, outer, **more):
    case = {"kind": kind, "rows": rows, "experts": experts, "in": inner, "out": outer, "skew": 0.7, "spare": 0, "sizes": 1,
            "type": 16, "add": False, "pad": 0}
    case.update(more)
    return case


def listed():
    return [
        # a token for each of 8 sequences of the draft model, whose table is the step's BF16 copy: latency
        {"name": "lookup tokens", **rows_case("lookup", 8, 16_384, 1024)},
        # a microbatch of a model of width 2048 and 32000 tokens
        {"name": "lookup batch", **rows_case("lookup", 65_536, 32_000, 2048)},
        # a router's choices by expert, on their way to the products below
        {"name": "sort choices", **rows_case("sort", 4_096, 64, 1, ids=32, even=True)},
        # a long microbatch's tokens by row of one of two shards of the table
        {"name": "sort batch", **rows_case("sort", 262_144, 16_000, 1, shards=2)},
        # a small odd table trained in FP32: latency
        {"name": "rowgrad few", **rows_case("rowgrad", 37, 1_001, 333, dy=32, out=32)},
        # the draft model's embedding gradient into its slot of a bucket
        {"name": "rowgrad draft", **rows_case("rowgrad", 8_192, 16_384, 1024)},
        # a large microbatch's, added to the FP32 gradient of a window; the commonest token is every fifteenth
        {"name": "rowgrad window", **rows_case("rowgrad", 65_536, 32_000, 2048, out=32, add=True)},
        # 32 sequences' single tokens with two choices each, of 64 experts: most experts have one row or none
        {"name": "forward tokens", **experts_case("forward", 64, 64, 1024, 4096)},
        # a training microbatch's first product in the experts
        {"name": "forward batch", **experts_case("forward", 32_768, 16, 2048, 8192)},
        # the draft model's second product backwards, on the way to its input
        {"name": "xgrad draft", **experts_case("xgrad", 16_384, 8, 4096, 1024, sizes=2)},
        # its weight gradient into a bucket's slot
        {"name": "wgrad draft", **experts_case("wgrad", 16_384, 8, 4096, 1024, sizes=2)},
        # a large microbatch's weight gradient added to the FP32 gradient of a window
        {"name": "wgrad window", **experts_case("wgrad", 32_768, 16, 2048, 8192, type=32, add=True, sizes=3)},
    ]


def between(rng, lo, hi):
    """Spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def size(rng, lo, hi):
    """A width: mostly a multiple of 8 or 64, else any."""
    n, step = between(rng, lo, hi), rng.choice((64, 64, 64, 8, 8, 1))
    return max(lo, n // step * step)


def draw(rng):
    kind = rng.choice(("lookup", "sort", "rowgrad", "rowgrad", "forward", "forward", "xgrad", "wgrad", "wgrad"))
    if kind == "sort":
        return rows_case("sort", between(rng, 1, 262_144), between(rng, 1, 64_000), 1, ids=rng.choice((32, 64)),
                         shards=rng.choice((1, 1, 2, 4)), even=rng.random() < 0.3)
    if kind in ("lookup", "rowgrad"):
        width, rows = size(rng, 32, 4096), between(rng, 100, 64_000)
        rows = min(rows, 65_536_000 // width)
        case = rows_case(kind, min(between(rng, 1, 65_536), 134_217_728 // width), rows, width, ids=rng.choice((32, 64, 64)),
                         shards=rng.choice((1, 1, 1, 2)), pad=rng.choice((0, 0, 0, 64, 3)))
        for part in ("table", "dy", "out"):
            case[part] = rng.choice((16, 16, 16, 32))
        case["add"] = kind == "rowgrad" and case["out"] == 32 and rng.random() < 0.5
        return case
    inner, outer = size(rng, 32, 8192), size(rng, 32, 8192)
    experts = min(between(rng, 1, 64), max(1, 268_435_456 // (inner * outer)))
    rows = min(between(rng, 1, 32_768), 549_755_813_888 // (inner * outer), 268_435_456 // max(inner, outer))
    out = rng.choice((16, 16, 32))
    return experts_case(kind, max(1, rows), experts, inner, outer, skew=rng.choice((0.0, 0.7, 1.5)), type=out,
                        spare=rng.choice((0, 0, 5, 100)), sizes=rng.randrange(1 << 20), pad=rng.choice((0, 0, 0, 64, 3)),
                        add=kind == "wgrad" and out == 32 and rng.random() < 0.5)


def sizes_of(case):
    """Rows of every expert: a router's choices with some experts commoner than others."""
    r = np.random.default_rng(case["sizes"])
    share = np.exp(r.normal(0.0, 1.0, size=case["experts"]) * case["skew"])
    return [int(n) for n in r.multinomial(case["rows"], share / share.sum())]


def different(case):
    """How many rows of the table the ids name, about: the k-th commonest of all is log(1 + 1/k) / log(1 + rows) of them."""
    every = case["rows"] * case["shards"]
    if case.get("even"):
        return case["rows"] * -math.expm1(case["n"] * math.log1p(-1.0 / every)) if every > 1 else 1.0
    k = np.arange(1, every + 1)
    p = np.log1p(1.0 / k) / math.log1p(every)
    return float(-np.expm1(case["n"] * np.log1p(-np.minimum(p, 1 - 1e-12))).sum()) / case["shards"]


def work(case):
    kind = case["kind"]
    if kind in ("lookup", "sort", "rowgrad"):
        n, width, index = case["n"], case["width"], case["ids"] // 8
        mine = n / case["shards"]
        if kind == "sort":
            return {"bytes": n * index + mine * 4 + case["rows"] * 4, "flops": n}
        if kind == "lookup":
            return {"bytes": n * index + different(case) * width * case["table"] // 8 + n * width * case["out"] // 8,
                    "flops": mine * width}
        out = 2 * different(case) if case["add"] else case["rows"]
        return {"bytes": n * index + mine * width * case["dy"] // 8 + out * width * case["out"] // 8, "flops": mine * width}
    rows, inner, outer, size_out = case["rows"], case["in"], case["out"], case["type"] // 8
    hit = sum(n > 0 for n in sizes_of(case))
    flops = 2 * rows * inner * outer
    if kind == "wgrad":
        written = 2 * hit if case["add"] else case["experts"]
        return {"bytes": 2 * rows * (inner + outer) + written * inner * outer * size_out, "flops": flops}
    read, written = (inner, outer) if kind == "forward" else (outer, inner)
    return {"bytes": 2 * rows * read + 2 * hit * inner * outer + rows * written * size_out, "flops": flops}


# ------------------------------------------------------------------ inputs
def float_of(bits):
    return F32 if bits == 32 else BF16


def normal(gen, scale, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=F32).mul_(scale).to(dtype)


def rows_of(gen, scale, dtype, n, width, pad):
    """n rows of normal values that lie `width + pad` elements apart."""
    return normal(gen, scale, dtype, n, width + pad)[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    return prepare_rows(case, gen) if case["kind"] in ("lookup", "sort", "rowgrad") else prepare_experts(case, gen)


def prepare_rows(case, gen):
    n, rows, width, kind = case["n"], case["rows"], case["width"], case["kind"]
    every = rows * case["shards"]
    u = torch.rand(n, generator=gen, device=DEVICE, dtype=F64)
    k = u * every if case.get("even") else torch.expm1(u * math.log1p(every))
    k = k.floor().clamp_(0, every - 1).to(torch.int64)
    name = torch.randperm(every, generator=gen, device=DEVICE)      # which token is how common
    s = {"kind": kind, "ids": name[k].to(torch.int32 if case["ids"] == 32 else torch.int64),
         "first": (case["shards"] - 1) * rows, "rows": rows, "scale": math.sqrt(width), "add": case["add"]}
    if kind == "lookup":
        s["table"] = normal(gen, 0.02, float_of(case["table"]), rows, width)
        s["out"] = torch.zeros(n, width + case["pad"], dtype=float_of(case["out"]), device=DEVICE)[:, :width]
        return s
    if kind == "rowgrad":
        s["dy"] = rows_of(gen, 1e-3, float_of(case["dy"]), n, width, case["pad"])
        s["out"] = normal(gen, 1e-2, float_of(case["out"]), rows, width)
    s["order"] = torch.zeros(n, dtype=torch.int32, device=DEVICE)
    s["at"] = torch.arange(n, device=DEVICE)
    s["every_row"] = torch.arange(rows + 1, device=DEVICE)
    if own:
        from gradient_reduction_optimizer_amd.layers import RowOrder
        s["by_row"] = RowOrder(n, rows, width, device=DEVICE)
    return s


def prepare_experts(case, gen):
    inner, outer, kind, pad = case["in"], case["out"], case["kind"], case["pad"]
    sizes = sizes_of(case)
    rows = case["rows"] + case["spare"]
    dtype = float_of(case["type"])
    s = {"kind": kind, "sizes": sizes, "add": case["add"], "used": case["rows"],
         "starts": torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEVICE)}
    if kind != "xgrad":
        s["x"] = rows_of(gen, 1.0, BF16, rows, inner, pad)
    if kind != "forward":
        s["dy"] = rows_of(gen, 1e-3, BF16, rows, outer, pad)
    if kind == "wgrad":
        s["out"] = normal(gen, 1e-2, dtype, case["experts"], outer, inner)
    else:
        s["w"] = normal(gen, 0.02, BF16, case["experts"], outer, inner)
        width = outer if kind == "forward" else inner
        s["out"] = torch.zeros(rows, width + pad, dtype=dtype, device=DEVICE)[:, :width]
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return {"lookup": run_lookup, "sort": run_sort, "rowgrad": run_rowgrad, "forward": run_forward, "xgrad": run_xgrad,
            "wgrad": run_wgrad}[s["kind"]](s)


def run_lookup(s):
    if own:
        from gradient_reduction_optimizer_amd import layers as L
        return L.lookup(s["table"], s["ids"], s["scale"], first_row=s["first"], out=s["out"])
    local = s["ids"].to(torch.int64) - s["first"]
    mine = (local >= 0) & (local < s["rows"])
    got = s["table"][torch.where(mine, local, 0)].float() * s["scale"]
    return s["out"].copy_(torch.where(mine[:, None], got, 0.0))


def by_row(s):
    """The ids' rows (the table's length for another shard's), in order, and where each row begins."""
    local = s["ids"].to(torch.int64) - s["first"]
    key = torch.where((local >= 0) & (local < s["rows"]), local, s["rows"])
    key, order = torch.sort(key, stable=True)
    return key, order, torch.searchsorted(key, s["every_row"])


def run_sort(s):
    if own:
        order, starts = s["by_row"].sort(s["ids"], first_row=s["first"])
        return {"order": order, "starts": starts}
    _, order, starts = by_row(s)
    order = torch.where(s["at"] < starts[-1], order, s["order"])
    return {"order": order.to(torch.int32), "starts": starts.to(torch.int32)}


def run_rowgrad(s):
    if own:
        s["by_row"].sort(s["ids"], first_row=s["first"])
        return s["by_row"].lookup_grad(s["dy"], s["scale"], out=s["out"], accumulate=s["add"])
    key, order, _ = by_row(s)
    total = torch.zeros(s["rows"] + 1, s["dy"].shape[1], dtype=F32, device=DEVICE)
    total = total.index_add_(0, key, s["dy"][order].float())[:-1] * s["scale"]
    return s["out"].copy_(total + s["out"] if s["add"] else total)


def products(s, rows, weights):
    """Every expert's rows times its matrix, in 32 bits."""
    parts = rows[:s["used"]].float().split(s["sizes"])
    s["out"][:s["used"]].copy_(torch.cat([p @ w for p, w in zip(parts, weights)]))
    return s["out"]


def run_forward(s):
    if own:
        from gradient_reduction_optimizer_amd import layers as L
        return L.experts_forward(s["x"], s["w"], s["starts"], out=s["out"])
    return products(s, s["x"], s["w"].float().transpose(1, 2))


def run_xgrad(s):
    if own:
        from gradient_reduction_optimizer_amd import layers as L
        return L.experts_input_grad(s["dy"], s["w"], s["starts"], out=s["out"])
    return products(s, s["dy"], s["w"].float())


def run_wgrad(s):
    if own:
        from gradient_reduction_optimizer_amd import layers as L
        return L.experts_weight_grad(s["dy"], s["x"], s["starts"], out=s["out"], accumulate=s["add"])
    pairs = zip(*(s[k][:s["used"]].float().split(s["sizes"]) for k in ("dy", "x")))
    total = torch.stack([dy.t() @ x for dy, x in pairs])
    return s["out"].copy_(total + s["out"] if s["add"] else total)


# --------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "sort":
        ids = s["ids"].cpu().numpy().astype(np.int64)
        at = np.flatnonzero((ids >= s["first"]) & (ids < s["first"] + case["rows"]))
        order = np.zeros(case["n"], np.int32)
        order[:at.size] = at[np.lexsort((at, ids[at]))]
        count = np.bincount(ids[at] - s["first"], minlength=case["rows"])
        return {"order": order, "starts": np.concatenate([[0], np.cumsum(count)]).astype(np.int32)}
    if kind in ("lookup", "rowgrad"):
        last = s["first"] + case["rows"]
        at = torch.nonzero((s["ids"] >= s["first"]) & (s["ids"] < last))[:, 0]
        row = s["ids"][at].to(torch.int64) - s["first"]
        if kind == "lookup":
            out = torch.zeros(case["n"], case["width"], dtype=F64, device=DEVICE)
            out[at] = s["table"].to(F64)[row] * math.sqrt(case["width"])
            return out
        out = s["out"].to(F64) if case["add"] else torch.zeros(case["rows"], case["width"], dtype=F64, device=DEVICE)
        return out.index_put_((row,), s["dy"][at].to(F64) * math.sqrt(case["width"]), accumulate=True)
    out = s["out"].to(F64) if kind != "wgrad" or case["add"] else torch.zeros_like(s["out"], dtype=F64)
    lo = 0
    for e, n in enumerate(sizes_of(case)):
        hi = lo + n
        if n and kind == "forward":
            out[lo:hi] = torch.mm(s["x"][lo:hi].to(F64), s["w"][e].to(F64).t())
        elif n and kind == "xgrad":
            out[lo:hi] = torch.mm(s["dy"][lo:hi].to(F64), s["w"][e].to(F64))
        elif n:
            out[e] += torch.mm(s["dy"][lo:hi].to(F64).t(), s["x"][lo:hi].to(F64))
        lo = hi
    return out
