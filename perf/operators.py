"""The operators of a decode step, measured: RMS norm with the residual's
addition, low-rank adapters of many requests, the paged key-value cache's
append and the attention of one new token over that cache.

``run`` computes each in elementary torch operations in fp32, rounded once
(``own`` false), or through the library's entry points (``own`` true).
``exact`` has the same operators from their definitions in fp64, written
apart from the plain forms."""
import math
import random

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user, a short conversation: the smallest call, all latency
        {"name": "decode_1x1000", "op": "decode", "batch": 1, "max_len": 1000, "ragged": False, "hq": 32, "hkv": 8,
         "d": 128, "page": 16, "dtype": "bf16", "cache": "bf16"},
        # a serving batch of mixed lengths, one row of it idle (length 0)
        {"name": "decode_32x8192_ragged", "op": "decode", "batch": 32, "max_len": 8192, "ragged": True, "hq": 32,
         "hkv": 8, "d": 128, "page": 16, "dtype": "bf16", "cache": "bf16"},
        # long documents over an 8-bit cache, eight query heads to a key head
        {"name": "decode_8x65536_fp8", "op": "decode", "batch": 8, "max_len": 65536, "ragged": True, "hq": 64,
         "hkv": 8, "d": 128, "page": 64, "dtype": "bf16", "cache": "fp8"},
        # a large batch with a key head to every query head, D = 64, pages of 48 tokens
        {"name": "decode_128x2047_mha64", "op": "decode", "batch": 128, "max_len": 2047, "ragged": True, "hq": 16,
         "hkv": 16, "d": 64, "page": 48, "dtype": "f16", "cache": "f16"},
        # the append of a decode step: one token a sequence
        {"name": "append_64x1", "op": "append", "batch": 64, "max_len": 2048, "new": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "dtype": "bf16", "cache": "bf16"},
        # the prompts of eight requests of mixed lengths, quantised on the way in
        {"name": "append_8x4096_fp8", "op": "append", "batch": 8, "max_len": 8192, "new": 4096, "hq": 64, "hkv": 8,
         "d": 128, "page": 64, "dtype": "f16", "cache": "fp8"},
        # the norm of a decode step
        {"name": "rmsnorm_4x4096", "op": "rmsnorm", "rows": 4, "cols": 4096, "residual": True, "dtype": "bf16",
         "out": "bf16"},
        # the norm of a long prompt batch
        {"name": "rmsnorm_16384x8192", "op": "rmsnorm", "rows": 16384, "cols": 8192, "residual": True,
         "dtype": "bf16", "out": "bf16"},
        # the last layer's norm (nothing to add) with an 8-bit output, an odd number of rows
        {"name": "rmsnorm_8191x5120_fp8", "op": "rmsnorm", "rows": 8191, "cols": 5120, "residual": False,
         "dtype": "f16", "out": "fp8"},
        # a decode step of 16 requests with 8 adapters in any order
        {"name": "lora_16_r16", "op": "lora", "rows": 16, "n": 4096, "k": 4096, "rank": 16, "adapters": 8,
         "run": 1, "dtype": "bf16"},
        # prompts: long runs of rows with the same adapter
        {"name": "lora_4096_r64", "op": "lora", "rows": 4096, "n": 4096, "k": 4096, "rank": 64, "adapters": 6,
         "run": 700, "dtype": "bf16"},
        # short prompts and decode rows mixed, a narrow projection, an odd number of rows
        {"name": "lora_257_r32", "op": "lora", "rows": 257, "n": 1000, "k": 8192, "rank": 32, "adapters": 12,
         "run": 9, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "append", "rmsnorm", "lora"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rmsnorm":
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = (cols + 7) // 8 * 8
        rows = _log(rng, 1, max(1, min(16384, 134217728 // cols)))
        return {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.7, "dtype": dtype,
                "out": rng.choice([dtype, dtype, "fp8"])}
    if op == "lora":
        return {"op": op, "rows": _log(rng, 1, 4096), "n": _log(rng, 64, 4096), "k": _log(rng, 8, 512) * 8,
                "rank": rng.choice([8, 16, 24, 32, 64]), "adapters": rng.randint(1, 16), "run": _log(rng, 1, 1024),
                "dtype": dtype}
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    case = {"op": op, "hq": hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16]), "hkv": hkv, "d": d,
            "page": rng.choice([16, 16, 32, 48, 64, 128]), "dtype": dtype, "cache": rng.choice([dtype, dtype, "fp8"])}
    if op == "decode":
        case["batch"] = _log(rng, 1, 128)
        case["max_len"] = _log(rng, 1, min(65536, 131072 // case["batch"]))
        case["ragged"] = rng.random() < 0.6
    else:
        case["batch"] = _log(rng, 1, 64)
        case["new"] = 1 if rng.random() < 0.4 else _log(rng, 2, 16384 // case["batch"])
        case["max_len"] = case["new"] + _log(rng, 1, 4096)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(n, most):
    """n lengths up to `most`, the same for every seed: the first is `most`,
    the others spread evenly over (0, most]."""
    return [most if i == 0 else max(1, math.ceil(most * ((i * 0.6180339887) % 1.0))) for i in range(n)]


def _lens(case):
    """Tokens in the cache of each sequence, the new ones included."""
    n = case["batch"]
    if case["op"] == "decode":
        lens = _spread(n, case["max_len"]) if case["ragged"] else [case["max_len"]] * n
        if case["ragged"] and n >= 16:
            lens[n // 2] = 0  # an idle row of the batch
        return lens
    return [max(a, b) for a, b in zip(_spread(n, case["max_len"]), _new(case))]


def _new(case):
    """New tokens of each sequence of an append."""
    return _spread(case["batch"], case["new"])


def _used(case):
    """The adapters that occur, and the adapter of each row (-1: none)."""
    ids = [(m // case["run"] * 19 + 1) % (case["adapters"] + 1) - 1 for m in range(case["rows"])]
    return sorted(set(ids) - {-1}), ids


def _paged(case, seed, g):
    """The cache, its page table and lengths: pages in any order, the table
    filled with -1 behind each sequence's last page."""
    rng, page = random.Random(seed), case["page"]
    lens = _lens(case)
    width = max(1, -(-max(lens) // page))
    counts = [-(-n // page) for n in lens]
    order = list(range(sum(counts) + 3))
    rng.shuffle(order)
    table, at = [], 0
    for c in counts:
        table.append(order[at:at + c] + [-1] * (width - c))
        at += c
    shape = (len(order), case["hkv"], page, case["d"])
    st = {}
    for n in ("k", "v"):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if case["cache"] == "fp8" else _DT[case["dtype"]])
        if case["cache"] == "fp8":
            st[n + "_cache"], st[n + "_scale"] = _quantise_rows(x)
        else:
            st[n + "_cache"], st[n + "_scale"] = x, None
    st["pages"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if own:
        from epilogue_gemm_amd import binding
        st["cache"] = binding.PagedCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    dt = _DT[case["dtype"]]

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    if op == "rmsnorm":
        rows, cols = case["rows"], case["cols"]
        st = {"x": randn(rows, cols), "residual": randn(rows, cols, std=2.0) if case["residual"] else None,
              "weight": (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt), "eps": 1e-6,
              "h": torch.empty(rows, cols, dtype=dt, device="cuda") if case["residual"] else None}
        fp8 = case["out"] == "fp8"
        st["y"] = torch.empty(rows, cols, dtype=torch.float8_e4m3fn if fp8 else dt, device="cuda")
        st["y_scale"] = torch.empty(rows, dtype=torch.float32, device="cuda") if fp8 else None
    elif op == "lora":
        m, n, k, r, count = (case[x] for x in ("rows", "n", "k", "rank", "adapters"))
        st = {"x": randn(m, k), "a": randn(count, r, k, std=1 / math.sqrt(k)), "b": randn(count, n, r, std=1 / math.sqrt(r)),
              "scale": 0.25 + torch.rand(count, generator=g, device="cuda"),
              "ids": torch.tensor(_used(case)[1], dtype=torch.int32, device="cuda"), "residual": randn(m, n),
              "c": torch.empty(m, n, dtype=dt, device="cuda"), "workspace": None}
        if own:
            from epilogue_gemm_amd import binding
            st["workspace"] = torch.empty(binding.lora_workspace_size(m, n, k, r, count), dtype=torch.uint8, device="cuda")
    else:
        st = _paged(case, seed, g)
        b, hq, hkv, d = (case[x] for x in ("batch", "hq", "hkv", "d"))
        # queries, keys and values stand side by side in the rows of one
        # projection, as the heads' products leave them
        tokens = b if op == "decode" else sum(_new(case))
        pad = 0 if op == "decode" or case["new"] == 1 else 5  # rows behind the last sequence
        rows = randn(tokens + pad, (hq + 2 * hkv) * d)
        if op == "decode":
            rows[:, :hq * d] *= 2  # attention that prefers some keys
            st["q"] = rows[:, :hq * d].view(tokens, hq, d)
            st["o"] = torch.empty(b, hq, d, dtype=dt, device="cuda")
            st["workspace"] = None
            if own:
                need = st["cache"].workspace_size(hq, st["pages"])
                st["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        else:
            st["new_k"] = rows[:, hq * d:(hq + hkv) * d].view(tokens + pad, hkv, d)
            st["new_v"] = rows[:, (hq + hkv) * d:].view(tokens + pad, hkv, d)
            st["tokens"], st["starts"] = tokens, None
            if case["new"] > 1:
                at = [0]
                for n in _new(case):
                    at.append(at[-1] + n)
                st["starts"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    st["op"] = op
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _quantise_rows(x):
    """E4M3 codes and fp32 scales of the last axis' rows: the scale is the
    smallest power of two, 2^-100 at least, with max|x| <= 448 scale."""
    frac, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(frac > 0.875, e - 8, e - 9).clamp(min=-100)
    scale = torch.ldexp(torch.ones_like(frac), e)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _rmsnorm(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + st["eps"]) * st["weight"].float()
    out = {}
    if st["residual"] is not None:
        out["h"] = h.to(st["x"].dtype)
    if st["y_scale"] is None:
        out["y"] = y.to(st["x"].dtype)
    else:
        out["y_scale"] = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
        out["y"] = (y / out["y_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return out


def _lora(st):
    count, r, k = st["a"].shape
    n = st["b"].shape[1]
    u = st["x"].float() @ st["a"].float().view(count * r, k).t()
    pick = st["ids"][:, None] == torch.arange(count, device="cuda")[None]
    u = u.view(-1, count, r) * torch.where(pick, st["scale"][None], 0.0)[..., None]
    delta = u.view(-1, count * r) @ st["b"].float().transpose(1, 2).reshape(count * r, n)
    return {"c": (st["residual"].float() + delta).to(st["x"].dtype)}


def _append(st):
    page = st["k_cache"].shape[2]
    t = torch.arange(st["tokens"], device="cuda")
    if st["starts"] is None:
        seq, pos = t, st["lens"] - 1
    else:
        seq = torch.searchsorted(st["starts"], t, right=True) - 1
        pos = st["lens"][seq] - (st["starts"][seq + 1] - t)
    where = st["pages"][seq, pos // page].long()
    out = {}
    for n in ("k", "v"):
        rows, cache, scale = st["new_" + n][:st["tokens"]], st[n + "_cache"], st[n + "_scale"]
        if scale is not None:
            rows, s = _quantise_rows(rows.float())
            scale[where, :, pos % page] = s
            cache.view(torch.uint8)[where, :, pos % page] = rows.view(torch.uint8)
            out[n + "_scale"] = scale
        else:
            cache[where, :, pos % page] = rows
        out[n + "_cache"] = cache
    return out


def _decode(st):
    b, hq, d = st["q"].shape
    _, hkv, page, _ = st["k_cache"].shape
    width = st["pages"].shape[1]
    at = st["pages"].clamp(min=0).long()

    def gather(n):
        x = st[n + "_cache"]
        x = x.view(torch.uint8)[at].view(x.dtype) if st[n + "_scale"] is not None else x[at]
        x = x.float()
        if st[n + "_scale"] is not None:
            x = x * st[n + "_scale"][at][..., None]
        return x.transpose(1, 2).reshape(b, hkv, width * page, d)

    s = (st["q"].float() / math.sqrt(d)).view(b, hkv, hq // hkv, d) @ gather("k").transpose(-1, -2)
    there = torch.arange(width * page, device="cuda")[None] < st["lens"][:, None]
    there &= (st["pages"] >= 0).repeat_interleave(page, 1)
    s = s.masked_fill(~there[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - m)
    o = (p @ gather("v")) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"o": o.view(b, hq, d).to(st["q"].dtype)}


def run(state):
    st, op = state, state["op"]
    if not own:
        return {"rmsnorm": _rmsnorm, "lora": _lora, "append": _append, "decode": _decode}[op](st)
    from epilogue_gemm_amd import binding
    if op == "rmsnorm":
        binding.rmsnorm(st["x"], st["weight"], st["y"], residual=st["residual"], residual_out=st["h"],
                        y_scale=st["y_scale"], eps=st["eps"])
        return {n: st[n] for n in ("h", "y", "y_scale") if st[n] is not None}
    if op == "lora":
        binding.lora(st["x"], st["a"], st["b"], st["ids"], st["c"], scale=st["scale"], residual=st["residual"],
                     workspace=st["workspace"])
        return {"c": st["c"]}
    if op == "append":
        st["cache"].append(st["new_k"], st["new_v"], st["pages"], st["lens"], starts=st["starts"])
        return {n: st[n] for n in ("k_cache", "k_scale", "v_cache", "v_scale") if st[n] is not None}
    st["cache"].attend(st["q"], st["o"], st["pages"], st["lens"], workspace=st["workspace"])
    return {"o": st["o"]}


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rmsnorm":
        n = case["rows"] * case["cols"]
        bytes_ = 2 * n + 2 * case["cols"] + (4 * n if case["residual"] else 0)
        bytes_ += n + 4 * case["rows"] if case["out"] == "fp8" else 2 * n
        return {"bytes": bytes_, "flops": 6 * n}
    if op == "lora":
        m, n, k, r = (case[x] for x in ("rows", "n", "k", "rank"))
        used, ids = _used(case)
        with_adapter = sum(i >= 0 for i in ids)
        return {"bytes": 2 * with_adapter * k + 4 * m * n + 2 * len(used) * r * (k + n) + 4 * m,
                "flops": 2 * with_adapter * r * (k + n)}
    row = case["hkv"] * case["d"]
    one = (row + 4 * case["hkv"]) if case["cache"] == "fp8" else 2 * row  # a token's keys (or values) in the cache
    if op == "append":
        tokens = sum(_new(case))
        return {"bytes": 2 * tokens * (2 * row + one) + 4 * tokens, "flops": tokens * row}
    tokens = sum(_lens(case))
    return {"bytes": 2 * tokens * one + 4 * case["batch"] * case["hq"] * case["d"] + 4 * (tokens // case["page"]),
            "flops": 4 * case["hq"] * case["d"] * tokens}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(x):
    """fp64 values rounded to the nearest E4M3 value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rmsnorm":
        h = st["x"].double() + (st["residual"].double() if case["residual"] else 0.0)
        y = h / (h.pow(2).sum(1) / case["cols"] + st["eps"]).sqrt()[:, None] * st["weight"].double()
        if case["out"] != "fp8":
            return {"h": h, "y": y} if case["residual"] else {"y": y}
        s = torch.clamp(y.abs().max(1).values / 448, min=2.0 ** -100)
        # the quotients before their rounding to 8 bits: where one lies on
        # a border between two codes, 32 bits may take either
        out = {"y": y / s[:, None], "y_scale": s}
        return {"h": h, **out} if case["residual"] else out
    if op == "lora":
        c = st["residual"].double()
        for i in _used(case)[0]:
            rows = (st["ids"] == i).nonzero()[:, 0]
            u = torch.mm(st["x"][rows].double(), st["a"][i].double().t().contiguous())
            c[rows] += float(st["scale"][i]) * torch.mm(u, st["b"][i].double().t().contiguous())
        return {"c": c}
    table, lens, page = st["pages"].tolist(), _lens(case), case["page"]
    caches = {}
    for n in ("k", "v"):
        caches[n + "_cache"] = st[n + "_cache"].double()
        if case["cache"] == "fp8":
            caches[n + "_scale"] = st[n + "_scale"].double()
    if op == "append":
        at = 0
        for i, n in enumerate(_new(case)):
            pos = torch.arange(lens[i] - n, lens[i], device="cuda")
            to = st["pages"][i].long()[pos // page], pos % page
            for name in ("k", "v"):
                x = st["new_" + name][at:at + n].double()
                if case["cache"] == "fp8":
                    most = x.abs().max(2).values
                    s = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(min=-100))
                    caches[name + "_scale"][to[0], :, to[1]] = s
                    x = _e4m3(x / s[..., None])
                caches[name + "_cache"][to[0], :, to[1]] = x
            at += n
        return caches
    o = torch.zeros(case["batch"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
    group = case["hq"] // case["hkv"]
    for i, n in enumerate(lens):
        if n == 0:
            continue
        rows = torch.tensor(table[i][:-(-n // page)], device="cuda")
        k, v = caches["k_cache"][rows], caches["v_cache"][rows]
        if case["cache"] == "fp8":
            k, v = k * caches["k_scale"][rows][..., None], v * caches["v_scale"][rows][..., None]
        for h in range(case["hkv"]):
            kh, vh = (x[:, h].reshape(-1, case["d"])[:n] for x in (k, v))
            q = st["q"][i, h * group:(h + 1) * group].double()
            w = torch.softmax(torch.mm(q, kh.t().contiguous()) * case["d"] ** -0.5, dim=1)
            o[i, h * group:(h + 1) * group] = torch.mm(w, vh)
    return {"o": o}
