"""The cases on which the token dispatch, the combine and the low-rank adapters are timed and compared.

Five operators, as a user of the package calls them:

  dispatch       rows[r] = (gates[s] *) x[s // topk] for the slot s = row_slot[r], with the row maps themselves
  dispatch_grad  its gradient: dx, and where the gates were applied dgates and the router logits' gradient
  combine        out[t] = sum_j (gates[t, j] *) rows[slot_row[t, j]]
  combine_grad   its gradient: drows, dgates and the router logits' gradient
  lora           out[t] = base[t] + scale_a * B_a (A_a x[t]) for the adapter a = ids[t] of row t's request

`run` computes them in plain torch operations in 32 bits, or with `own` set through nf3_moe_gb300.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    # 256 experts / H=6144 / top-8 and 128 experts / H=2048 / top-8 are the two layers of the benchmark, 8 experts /
    # H=256 / top-2 the one of the smoke test.
    return [
        # one decode step of 8 requests: 64 rows, latency counts
        _rows("dispatch_decode", "dispatch", 8, 6144, 256, 8, "bf16"),
        # a prompt batch: every token row goes to eight experts
        _rows("dispatch_prefill", "dispatch", 4096, 6144, 256, 8, "bf16"),
        # a training step with rows padded to GEMM tiles and a capacity limit, gates applied before the experts
        _rows("dispatch_grad_padded", "dispatch_grad", 2051, 2048, 128, 8, "f16", align=128, factor=1.25, weighted=True),
        # a small fp32 model with an odd width
        _rows("dispatch_grad_odd", "dispatch_grad", 333, 1001, 16, 2, "f32"),
        # one token's answer put together
        _rows("combine_token", "combine", 1, 2048, 128, 8, "bf16", weighted=True),
        # a prompt batch's answers
        _rows("combine_prefill", "combine", 4096, 6144, 256, 8, "f16", weighted=True),
        # the smoke test's layer trained on a ragged batch, some slots dropped
        _rows("combine_grad_small", "combine_grad", 37, 256, 8, 2, "bf16", factor=1.0, weighted=True),
        # a training step of the large layer: row gradients, gate gradients, router logits' gradients
        _rows("combine_grad_train", "combine_grad", 4096, 6144, 256, 8, "bf16", weighted=True),
        # one request's token beside a projection
        _lora("lora_token", 1, 1, 2048, 2048, 16, 16, "bf16"),
        # a decode step: every row another request, ranks 1 to 64
        _lora("lora_decode", 64, 64, 6144, 6144, 64, 64, "bf16"),
        # a mixed step on one column range of a fused projection: prompt chunks and single tokens, odd sizes
        _lora("lora_mixed", 1111, 70, 6144, 2056, 32, 48, "f16", gap=1032),
        # a prompt batch of a few requests
        _lora("lora_prefill", 8192, 12, 6144, 6144, 8, 64, "bf16"),
    ]


def _rows(name, op, tokens, width, experts, topk, dtype, align=1, factor=0.0, weighted=False):
    return {"name": name, "op": op, "tokens": tokens, "width": width, "experts": experts, "topk": topk, "dtype": dtype,
            "align": align, "factor": factor, "weighted": weighted}


def _lora(name, tokens, requests, k, n, slots, max_rank, dtype, gap=0, base=True):
    return {"name": name, "op": "lora", "tokens": tokens, "requests": requests, "k": k, "n": n, "slots": slots,
            "max_rank": max_rank, "dtype": dtype, "gap": gap, "base": base}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "lora", "lora", "lora"])
    if op != "lora":
        width = _log(rng, 64, 6144)
        width = width if rng.random() < 0.4 else -(-width // 8) * 8  # odd widths too
        experts = _log(rng, 2, 512)
        topk = rng.randint(1, min(8, experts))
        most = 4096 * 8 * 6144 // (topk * width)
        case = _rows("", op, _log(rng, 1, min(8192, most)), width, experts, topk, rng.choice(["bf16", "f16", "f32"]),
                     rng.choice([1, 1, 16, 128]), rng.choice([0.0, 0.0, 1.0, 1.25]), rng.random() < (0.4 if "dispatch" in op else 0.8))
        largest = _rows("", op, 4096, 6144, 256, 8, "bf16", weighted=True)
    else:
        k, n = (8 * _log(rng, 8, 1024) for _ in range(2))
        tokens = _log(rng, 1, 8192)
        rank, slots = rng.choice([4, 8, 13, 16, 32, 48, 64, 100, 128]), _log(rng, 1, 256)
        case = _lora("", tokens, rng.choice([tokens, _log(rng, 1, tokens)]), k, n, slots, rank, rng.choice(["bf16", "f16"]),
                     rng.choice([0, 0, 64, 1000]), rng.random() < 0.8)
        largest = _lora("", 8192, 12, 6144, 6144, 8, 64, "bf16")
        # the plain form multiplies by every adapter
        while case["slots"] > 1 and tokens * case["slots"] * rank * (k + n) > 8192 * 512 * 12288:
            case["slots"] //= 2
    while work(case)["bytes"] > work(largest)["bytes"] or work(case)["flops"] > work(largest)["flops"]:
        case["tokens"] = max(1, case["tokens"] * 2 // 3)
        case["requests"] = min(case.get("requests", 1), case["tokens"])
    if op != "lora":
        case.pop("requests", None)
    case.pop("name")
    return case


# ------------------------------------------------------------------ sizes
def _capacity(case):
    """Rows that one expert may get; 0: no limit."""
    return math.ceil(case["factor"] * case["tokens"] * case["topk"] / case["experts"]) if case["factor"] else 0


def _most_rows(case):
    """Rows of the sorted buffer: every slot, with each expert that has any padded to the alignment."""
    slots, align, cap = case["tokens"] * case["topk"], case["align"], _capacity(case)
    most = slots + min(case["experts"], slots) * (align - 1)
    return min(most, case["experts"] * -(-cap // align) * align) if cap else most


def work(case):
    t = case["tokens"]
    if case["op"] == "lora":
        k, n, r = case["k"], case["n"], (case["max_rank"] + 1) / 2  # ranks are spread over 1 to max_rank
        used = min(case["slots"], case["requests"])
        return {"bytes": 2 * (t * k + t * n * (2 if case["base"] else 1) + used * r * (k + n)) + 4 * t,
                "flops": 2 * t * r * (k + n) + t * n}
    size, slots, rows = (2 if case["dtype"] != "f32" else 4), t * case["topk"], _most_rows(case)
    one, many, w = t * case["width"] * size, min(rows, slots) * case["width"] * size, case["weighted"]
    every = rows * case["width"] * size
    logits = 4 * t * case["experts"] + 12 * slots if w else 0
    if case["op"] == "dispatch":  # x, the permutation and offsets in; every row and the maps out
        return {"bytes": one + every + 4 * (2 * slots + rows), "flops": many // size if w else 1}
    if case["op"] == "dispatch_grad":  # row gradients (and x) in; dx (and dgates, dlogits) out
        return {"bytes": many + one * (2 if w else 1) + 4 * slots + logits, "flops": (4 if w else 1) * many // size}
    if case["op"] == "combine":
        return {"bytes": many + one + 4 * slots * (2 if w else 1), "flops": (2 if w else 1) * many // size}
    return {"bytes": one + every + (many if w else 0) + 4 * slots + logits, "flops": (3 if w else 1) * many // size}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _routes(case, gen):
    """ids, gates, perm, offsets as the package's routing gives them, of skewed router logits."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    popular = 0.5 * torch.randn((1, e), generator=gen, device="cuda")
    logits = torch.randn((t, e), generator=gen, device="cuda") + popular
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = ids[:, :k].to(torch.int32).contiguous()
    z = torch.exp(top[:, :k] - top[:, :1])
    gates = (z / z.sum(dim=1, keepdim=True)).contiguous()
    flat = ids.reshape(-1).long()
    perm = torch.sort(flat, stable=True)[1].to(torch.int32)
    counts = torch.zeros(e, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return ids, gates, perm, offsets


def _maps(case, perm, offsets):
    """row_slot [rows], slot_row [tokens, topk] and row_offsets [experts + 1] in plain operations: each expert's slots in
    ascending order, the first `capacity` of them with a row, each expert's rows padded to the alignment."""
    rows, cap, align = _most_rows(case), _capacity(case), case["align"]
    off = offsets.long()
    counts = off[1:] - off[:-1]
    kept = counts.clamp(max=cap) if cap else counts
    padded = (kept + align - 1) // align * align
    row_off = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    p = torch.arange(perm.numel(), device=perm.device)
    e = torch.searchsorted(off, p, right=True) - 1
    rank = p - off[e]
    there = rank < kept[e]
    row = row_off[e] + rank
    slot_row = torch.empty_like(perm)
    slot_row[perm.long()] = torch.where(there, row, torch.full_like(row, -1)).to(torch.int32)
    row_slot = torch.full((rows + 1,), -1, dtype=torch.int32, device=perm.device)
    row_slot[torch.where(there, row, torch.full_like(row, rows))] = perm  # the dropped ones go to one place past the end
    return row_slot[:rows].contiguous(), slot_row.reshape(case["tokens"], case["topk"]), row_off.to(torch.int32)


def _randn(gen, shape, dtype, std=1.0):
    return (std * torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)).to(DTYPES[dtype])


def _inputs(case, seed):
    gen, t, dt = _gen(seed), case["tokens"], case["dtype"]
    s = {"case": dict(case)}
    if case["op"] == "lora":
        k, n, slots, most = case["k"], case["n"], case["slots"], case["max_rank"]
        # rows of one request lie side by side and share its adapter; about one request in ten has none
        cuts = torch.sort(torch.randint(0, t, (case["requests"] - 1,), generator=gen, device="cuda"))[0]
        request = torch.searchsorted(cuts, torch.arange(t, device="cuda"), right=True)
        if case["requests"] >= t:
            request = torch.arange(t, device="cuda")
        adapter = torch.randint(0, slots, (case["requests"],), generator=gen, device="cuda")
        without = torch.rand(case["requests"], generator=gen, device="cuda") < (0.1 if t > 1 else 0.0)
        s["ids"] = torch.where(without, torch.full_like(adapter, -1), adapter)[request].to(torch.int32)
        s["ranks"] = [1 + (seed * 31 + 17 * i * i + 5 * i) % most for i in range(slots)]
        s["ranks"][0] = most
        s["scales"] = [0.25 * (1 + (seed + 3 * i) % 8) for i in range(slots)]
        s["scale"] = torch.tensor(s["scales"], dtype=torch.float32, device="cuda")
        live = torch.arange(most, device="cuda")[None, :] < torch.tensor(s["ranks"], device="cuda")[:, None]
        zero = torch.zeros((), dtype=DTYPES[dt], device="cuda")
        s["a"] = torch.where(live[:, :, None], _randn(gen, (slots, most, k), dt, k ** -0.5), zero)
        s["b"] = torch.where(live[:, None, :], _randn(gen, (slots, n, most), dt, most ** -0.5), zero)
        s["x"] = _randn(gen, (t, k), dt)
        # the shared projection's result: a range of columns of a wider one where `gap` is given
        s["base"] = _randn(gen, (t, n + case["gap"]), dt)[:, case["gap"]:] if case["base"] else None
        return s
    s["ids"], s["gates"], s["perm"], s["offsets"] = _routes(case, gen)
    s["row_slot"], s["slot_row"], s["row_offsets"] = _maps(case, s["perm"], s["offsets"])
    rows, width = s["row_slot"].numel(), case["width"]
    if case["op"] in ("dispatch", "dispatch_grad"):
        s["x"] = _randn(gen, (t, width), dt)
    if case["op"] in ("dispatch_grad", "combine", "combine_grad"):
        s["rows"] = _randn(gen, (rows, width), dt)  # pad rows hold whatever the experts made of them
    if case["op"] == "combine_grad":
        s["dout"] = _randn(gen, (t, width), dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import nf3_moe_gb300 as hm
    t, dt = case["tokens"], DTYPES[case["dtype"]]
    if case["op"] == "lora":
        act = hm.ACT_F16 if case["dtype"] == "f16" else hm.ACT_BF16
        s["adapters"] = hm.LoraAdapters(case["k"], case["n"], case["slots"], case["max_rank"], max_tokens=t, act_dtype=act)
        for i, (r, scale) in enumerate(zip(s["ranks"], s["scales"])):
            s["adapters"].load(i, s["a"][i, :r].contiguous(), s["b"][i, :, :r].contiguous(), scale)
        s["out"] = torch.empty((t, case["n"]), dtype=dt, device="cuda")
        return s
    row = {"bf16": hm.ROW_BF16, "f16": hm.ROW_F16, "f32": hm.ROW_F32}[case["dtype"]]
    s["desc"] = hm.DispatchDesc(case["width"], case["experts"], case["topk"], row, case["align"], _capacity(case))
    rows = hm.hmoe_dispatch_rows(s["desc"], t)
    s["ws"] = torch.empty(hm.hmoe_dispatch_workspace_size(s["desc"], t), dtype=torch.uint8, device="cuda")
    hm.hmoe_workspace_init(s["ws"])
    ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    wide = lambda n: torch.empty((n, case["width"]), dtype=dt, device="cuda")  # noqa: E731
    s["made"] = {"dispatch": lambda: (wide(rows), ints(rows), ints(t, case["topk"]), ints(case["experts"] + 1)),
                 "dispatch_grad": lambda: (wide(t),), "combine": lambda: (wide(t),), "combine_grad": lambda: (wide(rows),)}[case["op"]]()
    if "grad" in case["op"] and case["weighted"]:
        s["dgates"] = torch.empty_like(s["gates"])
        s["dlogits"] = torch.empty((t, case["experts"]), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import nf3_moe_gb300 as hm
    case = s["case"]
    op, w = case["op"], case.get("weighted")
    if op == "lora":
        return {"out": s["adapters"](s["x"], s["ids"], base=s["base"], out=s["out"])}
    gates = s["gates"] if w else None
    if op == "dispatch":
        rows, row_slot, slot_row, row_offsets = s["made"]
        hm.hmoe_dispatch(s["desc"], s["x"], s["perm"], s["offsets"], rows, row_slot, slot_row, row_offsets, s["ws"], gates=gates)
        return {"rows": rows, "row_slot": row_slot, "slot_row": slot_row, "row_offsets": row_offsets}
    if op == "combine":
        hm.hmoe_combine(s["desc"], s["rows"], s["slot_row"], s["made"][0], s["ws"], gates=gates)
        return {"out": s["made"][0]}
    more = {"gates": gates, "ids": s["ids"], "dgates": s["dgates"], "dlogits": s["dlogits"]} if w else {}
    got = {"dgates": s["dgates"], "dlogits": s["dlogits"]} if w else {}
    if op == "dispatch_grad":
        hm.hmoe_dispatch_backward(s["desc"], s["rows"], s["slot_row"], s["made"][0], s["ws"], x=s["x"] if w else None, **more)
        return {"dx": s["made"][0], **got}
    hm.hmoe_combine_backward(s["desc"], s["dout"], s["row_slot"], s["slot_row"], s["made"][0], s["ws"],
                             rows=s["rows"] if w else None, **more)
    return {"drows": s["made"][0], **got}


def _spread(case, row_slot, gates, v):
    """A row for each entry of row_slot, of v's row of that slot's token times the slot's gate; zeros where there is none."""
    slot = row_slot.long().clamp(min=0)
    r = v.float()[slot // case["topk"]]
    if case["weighted"]:
        r = r * gates.reshape(-1)[slot][:, None]
    return torch.where((row_slot >= 0)[:, None], r, torch.zeros((), device=r.device)).to(v.dtype)


def _picked(slot_row, rows):
    """rows[slot_row] as [tokens, topk, width] in 32 bits, zeros where a slot has no row."""
    r = rows.float()[slot_row.long().clamp(min=0)]
    return torch.where((slot_row >= 0)[:, :, None], r, torch.zeros((), device=r.device))


def _gate_grads(case, ids, gates, picked, v):
    dg = (picked * v.float()[:, None, :]).sum(dim=2)
    dl = gates * (dg - (gates * dg).sum(dim=1, keepdim=True))
    return dg, torch.zeros((case["tokens"], case["experts"]), device=dg.device).scatter(1, ids.long(), dl)


def _run_plain(s):
    case = s["case"]
    op, w = case["op"], case.get("weighted")
    if op == "lora":
        slots, most, k = s["a"].shape
        t, n = case["tokens"], case["n"]
        u = (s["x"].float() @ s["a"].float().reshape(slots * most, k).T).reshape(t, slots, most)
        mine = s["ids"][:, None] == torch.arange(slots, device="cuda")[None, :]
        u = torch.where(mine[:, :, None], u * s["scale"][None, :, None], torch.zeros((), device="cuda"))
        delta = u.reshape(t, slots * most) @ s["b"].float().permute(0, 2, 1).reshape(slots * most, n)
        return {"out": (delta if s["base"] is None else s["base"].float() + delta).to(s["x"].dtype)}
    if op == "dispatch":
        row_slot, slot_row, row_offsets = _maps(case, s["perm"], s["offsets"])
        return {"rows": _spread(case, row_slot, s["gates"], s["x"]), "row_slot": row_slot, "slot_row": slot_row, "row_offsets": row_offsets}
    if op == "combine_grad":
        got = {"drows": _spread(case, s["row_slot"], s["gates"], s["dout"])}
        if w:
            got["dgates"], got["dlogits"] = _gate_grads(case, s["ids"], s["gates"], _picked(s["slot_row"], s["rows"]), s["dout"])
        return got
    picked = _picked(s["slot_row"], s["rows"])
    total = ((s["gates"][:, :, None] * picked) if w else picked).sum(dim=1).to(s["rows"].dtype)
    if op == "combine":
        return {"out": total}
    got = {"dx": total}
    if w:
        got["dgates"], got["dlogits"] = _gate_grads(case, s["ids"], s["gates"], picked, s["x"])
    return got


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    op, t = case["op"], case["tokens"]
    if op == "lora":
        out = s["base"].double() if s["base"] is not None else torch.zeros((t, case["n"]), dtype=torch.float64, device="cuda")
        for i in sorted(set(s["ids"].tolist()) - {-1}):
            mine, r = (s["ids"] == i).nonzero()[:, 0], s["ranks"][i]
            out[mine] += s["scales"][i] * ((s["x"][mine].double() @ s["a"][i, :r].double().T) @ s["b"][i, :, :r].double().T)
        return {"out": out}
    k, w, cap, align = case["topk"], case["weighted"], _capacity(case), case["align"]
    # each expert's rows, straight from the chosen ids
    flat, start, row_of = s["ids"].reshape(-1).cpu(), 0, [-1] * (t * k)
    for e in range(case["experts"]):
        mine = (flat == e).nonzero()[:, 0].tolist()
        mine = mine[:cap] if cap else mine
        for i, slot in enumerate(mine):
            row_of[slot] = start + i
        start += -(-len(mine) // align) * align
    row = torch.tensor(row_of, device="cuda").reshape(t, k)
    gates = s["gates"].double() if w else torch.ones((t, k), dtype=torch.float64, device="cuda")
    there = row >= 0
    if op in ("dispatch", "combine_grad"):
        v = (s["x"] if op == "dispatch" else s["dout"]).double()
        rows = torch.zeros((s["row_slot"].numel(), case["width"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = there[:, j].nonzero()[:, 0]
            rows[row[at, j]] = gates[at, j][:, None] * v[at]
        if op == "dispatch":
            return {"rows": rows, "row_slot": None, "slot_row": None, "row_offsets": None}
        got = {"drows": rows}
    else:
        total = torch.zeros((t, case["width"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = there[:, j].nonzero()[:, 0]
            total[at] += gates[at, j][:, None] * s["rows"][row[at, j]].double()
        if op == "combine":
            return {"out": total}
        got = {"dx": total}
    if w:
        v = (s["dout"] if op == "combine_grad" else s["x"]).double()
        dg = torch.zeros((t, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = there[:, j].nonzero()[:, 0]
            dg[at, j] = torch.linalg.vecdot(v[at], s["rows"][row[at, j]].double())
        dl = torch.zeros((t, case["experts"]), dtype=torch.float64, device="cuda")
        for j in range(k):  # the softmax over the chosen logits: d gate_i / d logit_j = gate_i (delta_ij - gate_j)
            for i in range(k):
                dl[torch.arange(t, device="cuda"), s["ids"][:, j].long()] += dg[:, i] * gates[:, i] * (float(i == j) - gates[:, j])
        got["dgates"], got["dlogits"] = dg, dl
    return got
