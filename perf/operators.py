"""Four operators of decoders whose linear maps are stored in 4 bits or split
among experts, as cases that can be timed and compared.

q4       y = W x with W in 4 bits: w = scale (code - zero), a scale and a zero
         for every `group` columns of a row
rows     expert numbers of every token -> the tokens ordered by expert
grouped  y_r = W_e(r) x_src(r) for rows ordered by expert, W in bf16, fp32 or 4 bits
combine  each token's weighted sum of its experts' rows

run() computes them in elementary torch operations in 32 bits, rounded once
at the end, or, with `own`, by the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token through a square map at decode: the smallest call
        {"name": "q4 one token", "op": "q4", "d": 4096, "d_out": 4096, "tokens": 1, "group": 128, "dtype": "bf16"},
        # a few sequences decoding together through a vocabulary-sized map
        {"name": "q4 vocabulary", "op": "q4", "d": 4096, "d_out": 50400, "tokens": 5, "group": 64, "dtype": "bf16"},
        # fp32 activations, the finest groups, an odd batch
        {"name": "q4 fp32 batch", "op": "q4", "d": 5120, "d_out": 13824, "tokens": 13, "group": 32, "dtype": "fp32"},
        # a prompt of odd length through an MLP's input map
        {"name": "q4 prompt", "op": "q4", "d": 4096, "d_out": 16384, "tokens": 2047, "group": 128, "dtype": "bf16"},
        # one token's eight experts at decode, most experts without a row
        {"name": "grouped one token", "op": "grouped", "d": 2048, "d_out": 2816, "tokens": 1, "top": 8, "experts": 64, "weights": "bf16", "group": 0},
        # a decoding batch over many experts in 4 bits, one or two rows each
        {"name": "grouped q4 batch", "op": "grouped", "d": 4096, "d_out": 1536, "tokens": 24, "top": 8, "experts": 128, "weights": "q4", "group": 128},
        # fp32 maps of odd sizes with a few ragged experts
        {"name": "grouped fp32 ragged", "op": "grouped", "d": 1000, "d_out": 1208, "tokens": 333, "top": 3, "experts": 8, "weights": "fp32", "group": 0},
        # a prompt's rows over the experts' input maps
        {"name": "grouped prompt", "op": "grouped", "d": 2048, "d_out": 4096, "tokens": 4096, "top": 4, "experts": 32, "weights": "bf16", "group": 0},
        # the router's choice for one token, where latency is all
        {"name": "rows one token", "op": "rows", "tokens": 1, "top": 8, "experts": 64, "dropped": 0.0},
        # a long prompt over many experts, some choices dropped
        {"name": "rows prompt", "op": "rows", "tokens": 16384, "top": 8, "experts": 256, "dropped": 0.03},
        # the end of an expert layer at decode
        {"name": "combine decode", "op": "combine", "tokens": 3, "top": 8, "d": 4096, "dtype": "bf16", "base": True, "dropped": 0.0},
        # the same over a prompt, added to the residual stream, some choices dropped
        {"name": "combine prompt", "op": "combine", "tokens": 8191, "top": 4, "d": 4096, "dtype": "bf16", "base": True, "dropped": 0.02},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4", "q4", "grouped", "grouped", "rows", "combine"])
    if op == "q4":
        d, d_out = 32 * _log(rng, 4, 512), 8 * _log(rng, 16, 6300)
        while d * d_out > 4096 * 50400:
            d_out = 8 * _log(rng, 16, 6300)
        most = max(1, min(2047, 4096 * 16384 * 2047 // (d * d_out)))
        tokens = _log(rng, 1, most)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if dtype == "fp32":
            tokens = max(1, tokens // 4)
        return {"op": op, "d": d, "d_out": d_out, "tokens": tokens, "group": rng.choice([32, 64, 128]), "dtype": dtype}
    if op == "grouped":
        weights = rng.choice(["bf16", "q4", "fp32"])
        unit = 32 if weights == "q4" else 8
        d, d_out = unit * _log(rng, 256 // unit, 4096 // unit), 8 * _log(rng, 16, 512)
        experts = _log(rng, 2, 128)
        top = rng.randint(1, min(8, experts))
        most = 2048 * 4096 * 16384 // (d * d_out * top)
        tokens = _log(rng, 1, max(1, min(4096 if weights != "fp32" else 512, most)))
        return {"op": op, "d": d, "d_out": d_out, "tokens": tokens, "top": top, "experts": experts, "weights": weights, "group": rng.choice([32, 64, 128]) if weights == "q4" else 0}
    tokens = _log(rng, 1, 16384 if op == "rows" else 8191)
    if op == "rows":
        experts = _log(rng, 2, 256)
        return {"op": op, "tokens": tokens, "top": rng.randint(1, min(8, experts)), "experts": experts, "dropped": rng.choice([0.0, 0.05, 0.5])}
    return {"op": op, "tokens": tokens, "top": rng.randint(1, 8), "d": 8 * _log(rng, 32, 512), "dtype": rng.choice(["bf16", "fp32"]), "base": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.1])}


# ---- inputs ----


def _choices(g, tokens, top, experts):
    """Each token's `top` different experts, some experts much more wanted than others."""
    dev = g.device
    liked = 1.5 * torch.randn(experts, generator=g, device=dev)
    score = torch.randn(tokens, experts, generator=g, device=dev) + liked
    return torch.topk(score, top, dim=1).indices.to(torch.int32)


def _activations(g, tokens, d, dtype):
    """Activations as a normalised stream has them: near unit size, a few channels much larger."""
    channel = torch.where(torch.rand(d, generator=g, device=g.device) < 0.01, 12.0, 1.0)
    return (torch.randn(tokens, d, generator=g, device=g.device) * channel).to(dtype)


def _q4_weights(g, shape, d, group, dtype):
    """Codes [*shape][d/2] (even column in the low nibble), scales and zeros [*shape][ceil(d/group)]."""
    n = (d + group - 1) // group
    codes = torch.randint(0, 256, (*shape, d // 2), generator=g, device=g.device, dtype=torch.uint8)
    scales = ((0.5 + torch.rand(*shape, n, generator=g, device=g.device)) / (5.0 * math.sqrt(d))).to(dtype)
    zeros = torch.randint(4, 12, (*shape, n), generator=g, device=g.device, dtype=torch.uint8)
    return codes, scales, zeros


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "q4":
        dtype = DTYPES[case["dtype"]]
        s["x"] = _activations(g, case["tokens"], case["d"], dtype)
        s["w"] = _q4_weights(g, (case["d_out"],), case["d"], case["group"], dtype)
    elif op == "grouped":
        e, d, d_out = case["experts"], case["d"], case["d_out"]
        dtype = torch.float32 if case["weights"] == "fp32" else torch.bfloat16
        s["x"] = _activations(g, case["tokens"], d, dtype)
        if case["weights"] == "q4":
            s["w"] = _q4_weights(g, (e, d_out), d, case["group"], dtype)
        else:
            s["w"] = torch.empty(e, d_out, d, device=dev, dtype=dtype).normal_(0.0, d**-0.5, generator=g)
        s["offsets"], s["rows"], _ = _rows(_choices(g, case["tokens"], case["top"], e), e)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    elif op == "rows":
        ids = _choices(g, case["tokens"], case["top"], case["experts"])
        s["ids"] = torch.where(torch.rand(ids.shape, generator=g, device=dev) < case["dropped"], -1, ids).contiguous()
    else:
        n, d = case["tokens"] * case["top"], case["d"]
        dtype = DTYPES[case["dtype"]]
        s["y"] = torch.randn(n, d, generator=g, device=dev).to(dtype)
        pos = torch.randperm(n, generator=g, device=dev).to(torch.int32).view(case["tokens"], case["top"])
        s["pos"] = torch.where(torch.rand(pos.shape, generator=g, device=dev) < case["dropped"], -1, pos).contiguous()
        s["weights"] = torch.softmax(torch.randn(pos.shape, generator=g, device=dev), dim=1)
        s["base"] = torch.randn(case["tokens"], d, generator=g, device=dev).to(dtype) if case["base"] else None
    if own and isinstance(s.get("w"), tuple):  # the handle a program keeps beside such weights: their addresses and sizes
        from rank_gated_memory_amd import gsi

        s["map"] = gsi.Q4(*s["w"], group=s["group"])
    return s


# ---- the plain forms ----


def _dense(codes, scales, zeros, group):
    """W in fp32: scale (code - zero)."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    d = q.shape[-1]
    z = zeros.float().repeat_interleave(group, dim=-1)[..., :d]
    return (q - z) * scales.float().repeat_interleave(group, dim=-1)[..., :d]


def _rows(ids, experts):
    """offsets [experts + 1], the token of every grouped row, the grouped row of every choice."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    ordered, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=ids.device))
    kept = ordered < experts
    rows = torch.where(kept, order // ids.shape[1], -1)
    pos = torch.empty_like(order)
    pos[order] = torch.where(kept, torch.arange(order.numel(), device=ids.device), -1)
    return offsets.int(), rows.int(), pos.view(ids.shape).int()


def _grouped(s):
    offsets, rows = s["offsets"], s["rows"].long()
    n = rows.numel()
    r = torch.arange(n, device=rows.device)
    e = torch.searchsorted(offsets[1:].long(), r, right=True)
    x = s["x"].float()[rows]
    few = n <= s["experts"]  # few rows: each with its own expert's map; many: the experts' rows padded to the longest
    pick = (lambda w: w[e]) if few else (lambda w: w)
    w = _dense(*(pick(t) for t in s["w"]), s["group"]) if s["weights"] == "q4" else pick(s["w"]).float()
    if few:
        return torch.bmm(w, x[:, :, None])[:, :, 0].to(s["x"].dtype)
    slot = r - offsets.long()[e]
    padded = x.new_zeros(s["experts"], s["most"], s["d"])
    padded[e, slot] = x
    return torch.bmm(padded, w.transpose(1, 2))[e, slot].to(s["x"].dtype)


def _combine(s):
    y, pos = s["y"], s["pos"].long()
    taken = (y.float()[pos.clamp(min=0)] * s["weights"][:, :, None]).masked_fill((pos < 0)[:, :, None], 0.0)
    out = taken.sum(1)
    return (out if s["base"] is None else out + s["base"].float()).to(y.dtype)


def run(state):
    s = state
    op = s["op"]
    if own:
        from rank_gated_memory_amd import gsi

        if op == "q4":
            return gsi.gsi_q4_linear(s["map"], s["x"])
        if op == "grouped":
            return gsi.gsi_grouped_linear(s.get("map", s["w"]), s["x"], s["offsets"], s["rows"])
        if op == "rows":
            return gsi.gsi_group_rows(s["ids"], s["experts"])
        return gsi.gsi_group_combine(s["y"], s["pos"], s["weights"], base=s["base"])
    if op == "q4":
        return (s["x"].float() @ _dense(*s["w"], s["group"]).t()).to(s["x"].dtype)
    if op == "grouped":
        return _grouped(s)
    if op == "rows":
        return _rows(s["ids"], s["experts"])
    return _combine(s)


# ---- what a pass cannot do without ----


def _map_bytes(weights, d, d_out, group):
    if weights == "q4" or group:
        scale = 4 if weights == "fp32" else 2
        return d_out * (d / 2 + (d + group - 1) // group * (scale + 1))
    return d_out * d * (4 if weights == "fp32" else 2)


def work(case):
    op = case["op"]
    if op == "q4":
        es = 4 if case["dtype"] == "fp32" else 2
        t, d, o = case["tokens"], case["d"], case["d_out"]
        return {"bytes": _map_bytes(case["dtype"], d, o, case["group"]) + t * (d + o) * es, "flops": 2.0 * t * d * o}
    if op == "grouped":
        es = 4 if case["weights"] == "fp32" else 2
        t, d, o, n = case["tokens"], case["d"], case["d_out"], case["tokens"] * case["top"]
        # the experts that at least one row needs: at least `top`, about what this many even choices reach
        e = case["experts"]
        active = max(case["top"], e * (1.0 - (1.0 - case["top"] / e) ** t) * 0.8)
        return {"bytes": active * _map_bytes(case["weights"], d, o, case["group"]) + (t * d + n * o) * es + 4 * n, "flops": 2.0 * n * d * o}
    n = case["tokens"] * case["top"]
    if op == "rows":
        return {"bytes": 4.0 * (3 * n + case["experts"] + 1), "flops": 0.0}
    es = 4 if case["dtype"] == "fp32" else 2
    kept = n * (1.0 - case["dropped"])
    moved = (kept + case["tokens"] * (2 if case["base"] else 1)) * case["d"] * es
    return {"bytes": moved + 8.0 * n, "flops": 2.0 * kept * case["d"]}


# ---- the definitions in 64 bits ----


def _map64(w, group, i=None):
    """One map in 64 bits from its nibbles, column by column of a group."""
    if not isinstance(w, tuple):
        return w[i].double()
    codes, scales, zeros = (t if i is None else t[i] for t in w)
    nibble = torch.arange(16, dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    byte = codes.long()
    out[:, 0::2], out[:, 1::2] = nibble[byte % 16], nibble[byte // 16]
    for k in range(scales.shape[1]):
        part = out[:, k * group:(k + 1) * group]
        part.sub_(zeros[:, k:k + 1].double()).mul_(scales[:, k:k + 1].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "q4":
        return torch.matmul(s["x"].double(), _map64(s["w"], case["group"]).t())
    if op == "grouped":
        at, x, rows = s["offsets"].tolist(), s["x"].double(), s["rows"].long()
        out = torch.empty(rows.numel(), case["d_out"], dtype=torch.float64, device=x.device)
        for e in range(case["experts"]):
            if at[e + 1] > at[e]:
                out[at[e]:at[e + 1]] = torch.matmul(x[rows[at[e]:at[e + 1]]], _map64(s["w"], case["group"], e).t())
        return out
    if op == "rows":
        ids = s["ids"].cpu().numpy()
        tokens, top = ids.shape
        lists = [np.flatnonzero(ids.reshape(-1) == e) for e in range(case["experts"])]
        offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])]).astype(np.int32)
        order = np.concatenate(lists)
        rows, pos = np.full(tokens * top, -1, np.int32), np.full(tokens * top, -1, np.int32)
        rows[:len(order)] = order // top
        pos[order] = np.arange(len(order), dtype=np.int32)
        return offsets, rows, pos.reshape(tokens, top)
    y, out = s["y"], torch.zeros(case["tokens"], case["d"], dtype=torch.float64, device=s["y"].device)
    if s["base"] is not None:
        out += s["base"].double()
    for j in range(case["top"]):
        at = s["pos"][:, j].long()
        kept = torch.nonzero(at >= 0)[:, 0]
        out[kept] += s["weights"][kept, j, None].double() * y[at[kept]].double()
    return out
