"""The feed-forward of a mixture of experts and its 8-bit products, measured:
the router with the order of its rows, products grouped by expert, the
combination of a token's rows, the quantisation of rows to 8-bit integers, and
the product of such rows with 8-bit weights.

``run`` computes each in elementary torch operations in fp32, rounded once
(``own`` false), or through the library's entry points (``own`` true).
``exact`` has the same operators from their definitions in fp64, written
apart from the plain forms."""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the rows of a decode step before an 8-bit projection: all latency
        {"name": "quantise_8x4096", "op": "quantise", "rows": 8, "cols": 4096, "dtype": "bf16"},
        # a batch of prompts, an odd number of rows
        {"name": "quantise_16383x5120", "op": "quantise", "rows": 16383, "cols": 5120, "dtype": "f16"},
        # an 8-bit projection of a decode batch: the weights' bytes
        {"name": "i8_16x8192x8192", "op": "i8", "m": 16, "n": 8192, "k": 8192, "epilogue": "none", "residual": True,
         "out": "bf16"},
        # the same of a long prompt, with the bias and activation of a feed-forward
        {"name": "i8_8192x8192x8192", "op": "i8", "m": 8192, "n": 8192, "k": 8192, "epilogue": "bias_gelu",
         "residual": False, "out": "bf16"},
        # a prompt of an odd length, an odd number of columns
        {"name": "i8_1001x2055x4096", "op": "i8", "m": 1001, "n": 2055, "k": 4096, "epilogue": "bias_silu",
         "residual": True, "out": "f16"},
        # the router of a decode step
        {"name": "route_32_8of128", "op": "route", "tokens": 32, "experts": 128, "per": 8, "score": "softmax",
         "renormalise": True, "dtype": "f32"},
        # the router of a batch of prompts
        {"name": "route_16384_8of256", "op": "route", "tokens": 16384, "experts": 256, "per": 8, "score": "sigmoid",
         "renormalise": True, "dtype": "bf16"},
        # the gated first product of a decode step: few rows for each of many experts
        {"name": "grouped_32_4of64", "op": "grouped", "tokens": 32, "per": 4, "experts": 64, "n": 1024, "k": 2048,
         "first": True, "gated": True, "epilogue": "silu", "away": 0.0, "dtype": "bf16"},
        # the same of a batch of prompts with few large experts, the largest call
        {"name": "grouped_8192_2of8", "op": "grouped", "tokens": 8192, "per": 2, "experts": 8, "n": 4096, "k": 4096,
         "first": True, "gated": True, "epilogue": "silu", "away": 0.0, "dtype": "bf16"},
        # the second product in 8 bits, a quarter of the experts on other devices, rows in an odd number
        {"name": "grouped_4095_4of32_i8", "op": "grouped", "tokens": 4095, "per": 4, "experts": 32, "n": 4096,
         "k": 2048, "first": False, "gated": False, "epilogue": "none", "away": 0.25, "dtype": "i8"},
        # a decode step's rows brought together
        {"name": "combine_32x4", "op": "combine", "tokens": 32, "per": 4, "n": 2048, "away": 0.0, "residual": True,
         "dtype": "bf16"},
        # a batch of prompts, some experts on other devices
        {"name": "combine_8191x8", "op": "combine", "tokens": 8191, "per": 8, "n": 4096, "away": 0.25,
         "residual": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "i8", "i8", "route", "grouped", "grouped", "combine"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "quantise":
        cols = _log(rng, 16, 16384)
        if rng.random() < 0.7:
            cols = (cols + 15) // 16 * 16
        return {"op": op, "rows": _log(rng, 1, max(1, min(16384, 83886080 // cols))), "cols": cols, "dtype": dtype}
    if op == "i8":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 1, 8192), "k": _log(rng, 1, 512) * 16,
                "epilogue": rng.choice(["none", "relu", "silu", "bias", "bias_relu", "bias_gelu", "bias_silu"]),
                "residual": rng.random() < 0.4, "out": dtype}
    if op == "route":
        experts = rng.choice([4, 8, 16, 60, 64, 128, 160, 256, 384])
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "per": rng.randint(1, min(experts, 8)),
                "score": rng.choice(["softmax", "sigmoid"]), "renormalise": rng.random() < 0.6,
                "dtype": rng.choice(["f32", "f32", "f16", "bf16"])}
    per = rng.randint(1, 8)
    if op == "combine":
        return {"op": op, "tokens": _log(rng, 1, 8192), "per": per, "n": _log(rng, 64, 4096),
                "away": rng.choice([0.0, 0.25]), "residual": rng.random() < 0.6, "dtype": dtype}
    gated = rng.random() < 0.5
    return {"op": op, "tokens": _log(rng, 1, 16384 // per), "per": per, "experts": rng.choice([8, 16, 32, 60, 64]),
            "n": _log(rng, 64, 2048), "k": _log(rng, 4, 128) * 16, "first": rng.random() < 0.5, "gated": gated,
            "epilogue": "silu" if gated else rng.choice(["none", "relu", "bias", "bias_silu"]),
            "away": rng.choice([0.0, 0.0, 0.25]), "dtype": rng.choice(["f16", "bf16", "i8"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _counts(case):
    """Rows of each expert, uneven and the same for every seed, and the rows
    of none (experts of other devices)."""
    total, experts = case["tokens"] * case["per"], case["experts"]
    away = int(total * case["away"])
    # no expert has two of one token's rows
    share = [1.0 + 0.8 * math.cos(2.399963 * e) for e in range(experts)]
    most, counts = case["tokens"], []
    for e in range(experts):
        left = total - away - sum(counts)
        counts.append(min(most, left, max(0, round(left * share[e] / sum(share[e:])))))
    return counts, total - sum(counts)


def _ids(case, seed):
    """Experts of each token [tokens, per]: any order of those counts, -1 for
    an expert of another device."""
    counts, away = _counts(case)
    flat = torch.repeat_interleave(torch.arange(-1, case["experts"]), torch.tensor([away] + counts))
    g = torch.Generator().manual_seed(seed)
    return flat[torch.randperm(len(flat), generator=g)].view(case["tokens"], case["per"]).int().cuda()


def _rows_i8(x):
    """8-bit codes and fp32 scales of the rows of fp32 values."""
    s = (x.abs().amax(-1) / 127).clamp(min=2.0 ** -100)
    return (x / s[..., None]).round().clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def randn(*shape, std=1.0, dtype="f32"):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_DT[dtype])

    st = {"op": op, "case": case}
    if op == "quantise":
        rows, cols = case["rows"], case["cols"]
        # activations: some channels much larger than the others
        st["x"] = (randn(rows, cols) * (1 + 4 * randn(cols).square())).to(_DT[case["dtype"]])
        st["y"] = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
        st["scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    elif op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["a_scale"] = _rows_i8(randn(m, k))
        st["b"], st["b_scale"] = _rows_i8(randn(n, k, std=1 / math.sqrt(k)))
        st["bias"] = randn(n, dtype=case["out"]) if case["epilogue"].startswith("bias") else None
        st["residual"] = randn(m, n, dtype=case["out"]) if case["residual"] else None
        st["c"] = torch.empty(m, n, dtype=_DT[case["out"]], device="cuda")
    elif op == "route":
        t, e, p = case["tokens"], case["experts"], case["per"]
        st["logits"] = (randn(t, e) + randn(e)).to(_DT[case["dtype"]])  # some experts preferred
        st["ids"] = torch.empty(t, p, dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty(t, p, dtype=torch.float32, device="cuda")
        st["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
        st["order"] = torch.empty(t * p, dtype=torch.int32, device="cuda")
    elif op == "grouped":
        t, p, e, n, k = (case[x] for x in ("tokens", "per", "experts", "n", "k"))
        st["offsets"], st["order"] = _group(_ids(case, seed), e)
        st["most"] = max(_counts(case)[0])
        rows, out = n * (2 if case["gated"] else 1), "bf16" if case["dtype"] == "i8" else case["dtype"]
        x, w = randn(t if case["first"] else t * p, k), randn(e, rows, k, std=1 / math.sqrt(k))
        st["x_scale"] = st["w_scale"] = None
        if case["dtype"] == "i8":
            st["x"], st["x_scale"] = _rows_i8(x)
            st["w"], st["w_scale"] = _rows_i8(w)
        else:
            st["x"], st["w"] = x.to(_DT[out]), w.to(_DT[out])
        st["bias"] = randn(e, rows, dtype=out) if case["epilogue"].startswith("bias") else None
        st["c"] = torch.zeros(t * p, n, dtype=_DT[out], device="cuda")
    else:
        t, p, n, dtype = case["tokens"], case["per"], case["n"], case["dtype"]
        st["z"] = randn(t * p, n, dtype=dtype)
        st["weights"] = torch.softmax(randn(t, p), 1)
        away = torch.rand(t, p, generator=g, device="cuda") < case["away"]
        st["ids"] = torch.where(away, -1, torch.arange(p, device="cuda")).int()
        st["residual"] = randn(t, n, dtype=dtype) if case["residual"] else None
        st["y"] = torch.empty(t, n, dtype=_DT[dtype], device="cuda")
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _act(z, epilogue):
    if epilogue.endswith("relu"):
        return z.clamp(min=0)
    if epilogue.endswith("silu"):
        return z / (1 + torch.exp(-z))
    if epilogue.endswith("gelu"):
        return z / (1 + torch.exp(-1.5957691216 * (z + 0.044715 * z * z * z)))
    return z


def _quantise(st):
    x = st["x"].float()
    # the quotients in 64 bits, rounded to 32: next to a border between two
    # codes every bit of them counts
    s = (x.abs().amax(1).double() / 127).float().clamp(min=2.0 ** -100)
    return {"y": (x.double() / s.double()[:, None]).float().round().to(torch.int8), "scale": s}


def _i8(st):
    z = (st["a"].float() @ st["b"].float().t()) * st["a_scale"][:, None] * st["b_scale"][None]
    if st["bias"] is not None:
        z = z + st["bias"].float()
    z = _act(z, st["case"]["epilogue"])
    if st["residual"] is not None:
        z = z + st["residual"].float()
    return {"c": z.to(st["c"].dtype)}


def _group(ids, experts):
    """Where each expert's entries begin in the stable order of the entries by
    expert, and that order, -1 behind its end."""
    flat = ids.reshape(-1)
    key, order = torch.where((flat >= 0) & (flat < experts), flat, experts).sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device="cuda", dtype=torch.int32))
    return offsets.int(), torch.where(key < experts, order, -1).int()


def _route(st):
    case, logits = st["case"], st["logits"].float()
    top, ids = logits.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :case["per"]], ids[:, :case["per"]]
    if case["score"] == "sigmoid":
        w = 1 / (1 + torch.exp(-top))
    else:
        w = torch.exp(top - top[:, :1])
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    elif case["score"] == "softmax":
        w = w / torch.exp(logits - top[:, :1]).sum(1, keepdim=True)
    ids = ids.int()
    offsets, order = _group(ids, case["experts"])
    return {"ids": ids, "weights": w * 2.5, "offsets": offsets, "order": order}


def _grouped(st):
    """Every expert's rows beside each other, filled up to the most that one
    has, in one batched product."""
    case, off = st["case"], st["offsets"].long()
    at = off[:-1, None] + torch.arange(st["most"], device="cuda")[None]
    there = at < off[1:, None]
    at = at.clamp(max=st["order"].shape[0] - 1)
    entry = st["order"].long()[at].clamp(min=0)
    rows = entry // case["per"] if case["first"] else at
    x, w = st["x"].float()[rows], st["w"].float()
    if st["x_scale"] is not None:
        x, w = x * st["x_scale"][rows][..., None], w * st["w_scale"][..., None]
    z = torch.bmm(x, w.transpose(1, 2))
    if st["bias"] is not None:
        z = z + st["bias"].float()[:, None]
    if case["gated"]:
        z = _act(z[..., :case["n"]], case["epilogue"]) * z[..., case["n"]:]
    else:
        z = _act(z, case["epilogue"])
    c = torch.zeros_like(st["c"])
    c[(at if case["first"] else entry)[there]] = z[there].to(c.dtype)
    return {"c": c}


def _combine(st):
    t, p = st["ids"].shape
    z = st["z"].float().view(t, p, -1).masked_fill((st["ids"] < 0)[..., None], 0.0)
    y = (z * st["weights"][..., None]).sum(1)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.to(st["z"].dtype)}


def run(state):
    st, op, case = state, state["op"], state["case"]
    if not own:
        return {"quantise": _quantise, "i8": _i8, "route": _route, "grouped": _grouped, "combine": _combine}[op](st)
    from epilogue_gemm_amd import binding
    if op == "quantise":
        binding.quantise_i8(st["x"], st["y"], st["scale"])
        return {"y": st["y"], "scale": st["scale"]}
    if op == "i8":
        binding.i8_gemm(st["a"], st["a_scale"], st["b"], st["b_scale"], st["c"], bias=st["bias"],
                        residual=st["residual"], epilogue=case["epilogue"])
        return {"c": st["c"]}
    if op == "route":
        binding.route(st["logits"], st["ids"], st["weights"], score=case["score"], renormalise=case["renormalise"],
                      scale=2.5, offsets=st["offsets"], order=st["order"])
        return {n: st[n] for n in ("ids", "weights", "offsets", "order")}
    if op == "grouped":
        binding.grouped_gemm(st["x"], st["w"], st["c"], st["offsets"], st["order"], per=case["per"],
                             gather=case["first"], scatter=not case["first"], gated=case["gated"], bias=st["bias"],
                             epilogue=case["epilogue"], x_scale=st["x_scale"], w_scale=st["w_scale"])
        return {"c": st["c"]}
    binding.combine(st["z"], st["weights"], st["ids"], st["y"], experts=case["per"], residual=st["residual"])
    return {"y": st["y"]}


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 3 * n}
    if op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k + 4) + 2 * m * n * (2 if case["residual"] else 1), "flops": 2 * m * n * k}
    if op == "route":
        t, e, p = case["tokens"], case["experts"], case["per"]
        return {"bytes": t * e * (4 if case["dtype"] == "f32" else 2) + 12 * t * p + 4 * e + 4, "flops": 3 * t * e}
    if op == "combine":
        here = case["tokens"] * case["per"] * (1 - case["away"])
        rows = here + case["tokens"] * (2 if case["residual"] else 1)
        return {"bytes": int(2 * rows * case["n"] + 8 * case["tokens"] * case["per"]), "flops": int(2 * here * case["n"])}
    counts, _ = _counts(case)
    total, used = sum(counts), sum(c > 0 for c in counts)
    size = 1 if case["dtype"] == "i8" else 2
    cols = case["n"] * (2 if case["gated"] else 1)
    read = min(total, case["tokens"]) if case["first"] else total
    return {"bytes": size * case["k"] * (read + used * cols) + 2 * total * case["n"] + 4 * total,
            "flops": 2 * total * cols * case["k"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _activation(z, name):
    name = name.split("_")[-1]
    if name == "relu":
        return torch.maximum(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.sigmoid(1.5957691216 * (z + 0.044715 * z ** 3))
    return z


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        most = st["x"].double().abs().max(1).values
        return {"y": None, "scale": torch.clamp(most / 127, min=2.0 ** -100)}
    if op == "i8":
        c = torch.mm(st["a"].double(), st["b"].double().t().contiguous())
        c = c * torch.outer(st["a_scale"].double(), st["b_scale"].double())
        if st["bias"] is not None:
            c += st["bias"].double()[None]
        c = _activation(c, case["epilogue"])
        return {"c": c + st["residual"].double() if case["residual"] else c}
    if op == "route":
        logits, p = st["logits"].double(), case["per"]
        # (entries that are equal: the lower index before the higher one)
        rank = torch.argsort(-logits, dim=1, stable=True)[:, :p]
        prob = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
        w = prob.gather(1, rank)
        if case["renormalise"]:
            w = w / w.sum(1)[:, None]
        return {"ids": None, "weights": 2.5 * w, "offsets": None, "order": None}
    if op == "combine":
        t, p = case["tokens"], case["per"]
        y = st["residual"].double() if case["residual"] else torch.zeros(t, case["n"], dtype=torch.float64, device="cuda")
        for j in range(p):
            w = torch.where(st["ids"][:, j] >= 0, st["weights"][:, j].double(), 0.0)
            y = y + w[:, None] * st["z"][j::p].double()
        return {"y": y}
    c = torch.zeros(st["c"].shape, dtype=torch.float64, device="cuda")
    off, n = st["offsets"].tolist(), case["n"]
    for e in range(case["experts"]):
        if off[e + 1] == off[e]:
            continue
        entries = st["order"][off[e]:off[e + 1]].long()
        place = torch.arange(off[e], off[e + 1], device="cuda")
        rows = torch.div(entries, case["per"], rounding_mode="floor") if case["first"] else place
        z = torch.mm(st["x"][rows].double(), st["w"][e].double().t().contiguous())
        if case["dtype"] == "i8":
            z = z * torch.outer(st["x_scale"][rows].double(), st["w_scale"][e].double())
        if st["bias"] is not None:
            z += st["bias"][e].double()[None]
        if case["gated"]:
            z = _activation(z[:, :n].clone(), case["epilogue"]) * z[:, n:]
        else:
            z = _activation(z, case["epilogue"])
        c[place if case["first"] else entries] = z
    return {"c": c}
