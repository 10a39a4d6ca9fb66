"""The cases on which the whole layer for a few tokens and the 4-bit integer linear are timed and compared.

Two operators, as a user of the package calls them, the 4-bit work of a decode step:

  moe    the whole mixture-of-experts layer from the hidden states of 1 to 8 tokens: the router's logits, its top-k
         and gates, and out[t] = sum_j gates[t, j] * W2_e (silu(W1_e x_t) * W3_e x_t) with e = ids[t, j], over
         experts held as NVFP4 or MXFP4 (the kept tier) and NF3
  int4   y[t] = W x[t] (+ bias) with W[n, k] = (q[n, k] - z[n, k / group]) * s[n, k / group], q and z of 4 bits

`run` computes them in plain torch operations in 32 bits, or with `own` set through nf3_moe_gb300.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# magnitudes of E2M1 and the 3-bit NormalFloat levels (bf16 values)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NF3 = (-1.0, -0.53515625, -0.2470703125, 0.0, 0.18359375, 0.3828125, 0.62109375, 1.0)


def listed():
    # 256 experts / H=6144 / I=2048 / top-8 and 128 experts / H=2048 / I=768 / top-8 are the two layers of the
    # benchmark, 8 experts / H=256 / I=128 / top-2 the one of the smoke test.
    return [
        # the smoke test's layer, two tokens: nothing but latency
        _moe("moe_tiny", 2, 256, 128, 8, 2, "nvfp4", 4, "bf16"),
        # one request's token through the uniform layer
        _moe("moe_uniform_token", 1, 2048, 768, 128, 8, "nvfp4", 0, "bf16"),
        # eight requests' tokens through the uniform layer, fp16 activations
        _moe("moe_uniform_batch", 8, 2048, 768, 128, 8, "nvfp4", 0, "f16"),
        # one token through the large hybrid layer
        _moe("moe_hybrid_token", 1, 6144, 2048, 256, 8, "nvfp4", 192, "bf16"),
        # a decode step of eight requests through it, the benchmark's headline batch
        _moe("moe_hybrid_batch", 8, 6144, 2048, 256, 8, "nvfp4", 192, "bf16"),
        # its MXFP4 form with a router bias, a token and three drafted ones, fp16 activations
        _moe("moe_mxfp4_draft", 4, 6144, 2048, 256, 8, "mxfp4", 192, "f16", bias=True),
        # one token through a small projection
        _int4("int4_token_small", 1, 2048, 2048, 128, "bf16"),
        # one token through a square projection of the large layer's width
        _int4("int4_token", 1, 6144, 6144, 128, "bf16", zeros=True),
        # a token and four drafted ones, finer groups, fp16
        _int4("int4_draft", 5, 4096, 6144, 64, "f16", zeros=True, bias=True),
        # odd sizes
        _int4("int4_odd", 3, 1001, 1056, 32, "bf16", zeros=True, bias=True),
        # a decode step of sixteen requests through a fused projection, its input a column range of a wider tensor
        _int4("int4_batch", 16, 12288, 6144, 128, "bf16", gap=2048),
        # eight requests' logits
        _int4("int4_head", 8, 32768, 6144, 128, "bf16", zeros=True),
    ]


def _moe(name, tokens, h, i, experts, topk, kept, nf3, dtype, bias=False):
    """nf3: experts in the NF3 tier (0: no bit map)."""
    return {"name": name, "op": "moe", "tokens": tokens, "h": h, "i": i, "experts": experts, "topk": topk, "kept": kept,
            "nf3": nf3, "dtype": dtype, "bias": bias}


def _int4(name, tokens, n, k, group, dtype, zeros=False, bias=False, gap=0):
    return {"name": name, "op": "int4", "tokens": tokens, "n": n, "k": k, "group": group, "dtype": dtype, "zeros": zeros,
            "bias": bias, "gap": gap}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        experts = _log(rng, 2, 256)
        case = _moe("", rng.randint(1, 8), 128 * _log(rng, 1, 48), 64 * _log(rng, 1, 32), experts,
                    rng.randint(1, min(8, experts)), rng.choice(["nvfp4", "nvfp4", "mxfp4"]),
                    rng.choice([0, experts // 2, experts - experts // 4, experts]), rng.choice(["bf16", "f16"]), rng.random() < 0.4)
        largest = _moe("", 8, 6144, 2048, 256, 8, "nvfp4", 192, "bf16")
    else:
        group = rng.choice([32, 64, 128])
        case = _int4("", _log(rng, 1, 32), _log(rng, 16, 32768), group * _log(rng, 1, 8192 // group), group,
                     rng.choice(["bf16", "f16"]), rng.random() < 0.6, rng.random() < 0.4, rng.choice([0, 0, 8, 1024]))
        largest = _int4("", 16, 32768, 6144, 128, "bf16", zeros=True)
    while work(case)["bytes"] > work(largest)["bytes"] or work(case)["flops"] > work(largest)["flops"]:
        case["tokens"] -= 1
        if case["tokens"] == 0:
            case["tokens"], case["n" if case["op"] == "int4" else "i"] = 1, case["n"] // 2 if case["op"] == "int4" else 64
    case.pop("name")
    return case


def work(case):
    t = case["tokens"]
    if case["op"] == "int4":
        n, k = case["n"], case["k"]
        groups = n * (k // case["group"])
        return {"bytes": n * k // 2 + 2 * groups + (groups // 2 if case["zeros"] else 0) + 2 * t * (n + k) + (2 * n if case["bias"] else 0),
                "flops": 2 * t * n * k}
    h, i, e, k = case["h"], case["i"], case["experts"], case["topk"]
    touched = e * (1 - (1 - k / e) ** t)  # experts that some token chose, were the choices even
    share = case["nf3"] / e
    per = (1 - share) * (9 / 16 if case["kept"] == "nvfp4" else 17 / 32) + share * 13 / 32
    return {"bytes": int(touched * 3 * h * i * per) + 2 * e * h + 4 * t * h + 8 * t * k + (4 * e if case["bias"] else 0),
            "flops": 2 * t * (3 * k * h * i + e * h)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(gen, shape, std=1.0):
    return std * torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _nibbles(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8).contiguous()


def _quantise(w, fmt):
    """codes, scales and the global scale of weights [rows, K] in the checkpoint's layout of that format."""
    rows, k = w.shape
    if fmt == "nf3":
        scale = w.view(rows, k // 64, 64).abs().amax(dim=2).to(torch.bfloat16)
        mid = torch.tensor([(a + b) / 2 for a, b in zip(NF3, NF3[1:])], device=w.device)
        code = torch.bucketize(w.view(rows, k // 64, 64) / scale.float()[:, :, None], mid, out_int32=True)
        word = (code.view(rows, k // 8, 8) << (3 * torch.arange(8, device=w.device, dtype=torch.int32))).sum(dim=2, dtype=torch.int32)
        return torch.stack([word & 255, (word >> 8) & 255, word >> 16], dim=2).to(torch.uint8).view(rows, 3 * k // 8), scale, 1.0
    size = 16 if fmt == "nvfp4" else 32
    g = w.view(rows, k // size, size)
    amax = g.abs().amax(dim=2)
    if fmt == "nvfp4":
        one = 0.08 / (6 * 448)  # a global scale near the largest weight's over 6 * 448, the same for every matrix
        e4m3 = (amax / (6 * one)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale, by = e4m3.view(torch.uint8), e4m3.float() * one
    else:
        e = torch.floor(torch.log2(amax)) - 2
        one, scale, by = 1.0, (e + 127).to(torch.uint8), torch.exp2(e)
    mid = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=w.device)
    v = g / by[:, :, None]
    code = torch.bucketize(v.abs(), mid, out_int32=True) | ((v < 0).to(torch.int32) << 3)
    return _nibbles(code.view(rows, k)), scale.contiguous(), one


def _tier(gen, fmt, count, h, i):
    """One tier's experts: codes and scales of W13 [count, 2 i, h] and W2 [count, h, i], and the global scales."""
    made = []
    for rows, k in ((2 * i, h), (h, i)):
        each = [_quantise(_randn(gen, (rows, k), 0.02), fmt) for _ in range(count)]
        made.append((torch.stack([c for c, _, _ in each]), torch.stack([s for _, s, _ in each]), each[0][2]))
    return made


def _inputs(case, seed):
    gen, t, dt = _gen(seed), case["tokens"], DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"] == "int4":
        n, k, groups = case["n"], case["k"], case["k"] // case["group"]
        s["x"] = _randn(gen, (t, k + case["gap"])).to(dt)[:, case["gap"]:]
        # weights about a random zero point, or about 8, with scales of a matrix of std 0.02
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s["scales"] = (0.005 * (0.5 + torch.rand((n, groups), generator=gen, device="cuda"))).to(dt)
        s["zeros"] = torch.randint(4, 12, (n, groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["bias"] = _randn(gen, (n,), 0.1).to(dt) if case["bias"] else None
        return s
    h, i, e, nf3 = case["h"], case["i"], case["experts"], case["nf3"]
    s["x"] = _randn(gen, (t, h)).to(dt)
    s["router"] = _randn(gen, (e, h), h ** -0.5).to(dt)
    s["bias"] = _randn(gen, (e,), 0.1) if case["bias"] else None
    # every tier's experts spread over the ids
    order = torch.randperm(e, generator=gen, device="cuda").tolist()
    s["bits"] = [3 if order[x] < nf3 else 4 for x in range(e)]
    place, seen = [], {3: 0, 4: 0}
    for b in s["bits"]:
        place.append(seen[b])
        seen[b] += 1
    s["place"] = place
    s["tiers"] = {f: _tier(gen, f, c, h, i) for f, c in ((case["kept"], e - nf3), ("nf3", nf3)) if c}
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    t, dev = case["tokens"], "cuda"
    if case["op"] == "moe":
        s["where"] = torch.tensor(s["place"], device=dev)
        s["is_nf3"] = torch.tensor([b == 3 for b in s["bits"]], device=dev)
    if not own:
        return s
    import nf3_moe_gb300 as hm
    act = hm.ACT_F16 if case["dtype"] == "f16" else hm.ACT_BF16
    if case["op"] == "int4":
        s["linear"] = hm.LinearInt4(case["n"], case["k"], case["group"], s["codes"], s["scales"], s["zeros"], max_tokens=t, act_dtype=act)
        s["out"] = torch.empty((t, case["n"]), dtype=DTYPES[case["dtype"]], device=dev)
        return s
    kept = hm.FMT_NVFP4 if case["kept"] == "nvfp4" else hm.FMT_MXFP4
    experts = []
    for b, p in zip(s["bits"], s["place"]):
        (c13, s13, g13), (c2, s2, g2) = s["tiers"]["nf3" if b == 3 else case["kept"]]
        experts.append((c13[p], s13[p], g13, c2[p], s2[p], g2))
    s["layer"] = hm.HybridMoELayer(case["h"], case["i"], case["experts"], case["topk"], s["bits"] if case["nf3"] else None, experts,
                                   kept_format=kept, max_tokens=t, act_dtype=act)
    s["out"] = torch.empty((t, case["h"]), dtype=DTYPES[case["dtype"]], device=dev)
    s["ids"] = torch.empty((t, case["topk"]), dtype=torch.int32, device=dev)
    s["gates"] = torch.empty((t, case["topk"]), dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    if s["case"]["op"] == "int4":
        return {"out": s["linear"](s["x"], bias=s["bias"], out=s["out"])}
    out, ids, gates = s["layer"].decode(s["x"], s["router"], bias=s["bias"], out=s["out"], ids=s["ids"], gates=s["gates"])
    return {"out": out, "ids": ids, "gates": gates}


def _both_nibbles(codes):
    c = torch.stack([codes & 15, codes >> 4], dim=-1)
    return c.reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def _weights(fmt, codes, scales, one):
    """[..., rows, K] in 32 bits from a tier's codes and scales of any leading shape."""
    dev = codes.device
    if fmt == "nf3":
        b = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 3, 3).to(torch.int32)
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        code = (word[..., None] >> (3 * torch.arange(8, device=dev, dtype=torch.int32))) & 7
        value = torch.tensor(NF3, device=dev).index_select(0, code.reshape(-1))
        return (value.view(*scales.shape, 64) * scales.float()[..., None]).flatten(-2)
    level = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=dev)
    value = level.index_select(0, _both_nibbles(codes).reshape(-1).to(torch.int32))
    scale = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(scales.float() - 127)
    return (value.view(*scales.shape, -1) * (scale * one)[..., None]).flatten(-2)


def _expert_product(s, which, chosen, v):
    """v[s] [width] times the matrix `which` of the expert chosen[s], [S, rows]."""
    result = None
    at, mine = s["where"][chosen], s["is_nf3"][chosen]
    for fmt, tier in s["tiers"].items():
        codes, scales, one = tier[which]
        p = torch.where(mine == (fmt == "nf3"), at, torch.zeros_like(at))
        y = torch.matmul(_weights(fmt, codes[p], scales[p], one), v[:, :, None])[:, :, 0]
        y = torch.where((mine == (fmt == "nf3"))[:, None], y, torch.zeros((), device=y.device))
        result = y if result is None else result + y
    return result


def _route(s, x):
    """ids and gates of the router's logits in 64 bits: neighbours in rank lie closer than 32 bits tell apart."""
    logits = x.double() @ s["router"].double().T
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :s["case"]["topk"]], ids[:, :s["case"]["topk"]]
    z = torch.exp(top - top[:, :1])
    return ids, z / z.sum(dim=1, keepdim=True)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "int4":
        n, k = case["n"], case["k"]
        q = _both_nibbles(s["codes"]).float().view(n, k // case["group"], case["group"])
        z = 8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None]
        y = s["x"].float() @ ((q - z) * s["scales"].float()[:, :, None]).view(n, k).T
        return {"out": (y if s["bias"] is None else y + s["bias"].float()).to(s["x"].dtype)}
    t, k, i = case["tokens"], case["topk"], case["i"]
    ids, gates = _route(s, s["x"])
    chosen = ids.reshape(-1)
    x = s["x"].float().repeat_interleave(k, dim=0)
    gu = _expert_product(s, 0, chosen, x)
    a = gu[:, :i]
    h = a / (1 + torch.exp(-a)) * gu[:, i:]
    y = _expert_product(s, 1, chosen, h).view(t, k, case["h"])
    out = (gates.float()[:, :, None] * y).sum(dim=1)
    return {"out": out.to(s["x"].dtype), "ids": ids.to(torch.int32), "gates": gates.float()}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    t, x = case["tokens"], s["x"].double()
    if case["op"] == "int4":
        n, k, g = case["n"], case["k"], case["group"]
        out = torch.zeros((t, n), dtype=torch.float64, device="cuda")
        for lo in range(0, n, 4096):  # a range of rows at a time
            c = s["codes"][lo:lo + 4096]
            w = torch.empty((c.shape[0], k), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (c % 16).double(), (c // 16).double()
            zero = s["zeros"][lo:lo + 4096].double() if case["zeros"] else torch.full((c.shape[0], k // g), 8.0, dtype=torch.float64, device="cuda")
            w = (w - zero.repeat_interleave(g, dim=1)) * s["scales"][lo:lo + 4096].double().repeat_interleave(g, dim=1)
            out[:, lo:lo + 4096] = torch.einsum("tk,nk->tn", x, w)
        return {"out": out if s["bias"] is None else out + s["bias"].double()[None, :]}
    k, i = case["topk"], case["i"]
    logits = torch.einsum("th,eh->te", x, s["router"].double()).cpu()
    logits = logits if s["bias"] is None else logits + s["bias"].double().cpu()[None, :]
    out = torch.zeros((t, case["h"]), dtype=torch.float64, device="cuda")
    gates = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    picks = {}
    for row in range(t):
        l = logits[row].tolist()
        best = sorted(range(len(l)), key=lambda e: (-l[e], e))[:k]
        total = sum(math.exp(l[e] - l[best[0]]) for e in best)
        for j, e in enumerate(best):
            g = math.exp(l[e] - l[best[0]]) / total
            gates[row, j] = g
            picks.setdefault(e, []).append((row, g))

    def matrix(e, which):
        fmt = "nf3" if s["bits"][e] == 3 else case["kept"]
        codes, scales, one = s["tiers"][fmt][which]
        c, sc = codes[s["place"][e]], scales[s["place"][e]]
        rows = c.shape[0]
        if fmt == "nf3":  # code j of a row: bits 3j to 3j + 2 of its bytes, the lowest first
            bits = torch.stack([(c >> b) & 1 for b in range(8)], dim=2).view(rows, -1, 3).long()
            value = torch.tensor(NF3, dtype=torch.float64, device="cuda")[bits[..., 0] + 2 * bits[..., 1] + 4 * bits[..., 2]]
            return value * sc.double().repeat_interleave(64, dim=1)
        w = torch.empty((rows, 2 * c.shape[1]), dtype=torch.float64, device="cuda")
        for half, nib in ((0, c % 16), (1, c // 16)):
            m = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[(nib % 8).long()]
            w[:, half::2] = torch.where(nib >= 8, -m, m)
        if fmt == "nvfp4":
            return w * sc.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1) * one
        return torch.ldexp(w, (sc.int() - 127).repeat_interleave(32, dim=1))

    for e, rows in picks.items():
        at = torch.tensor([r for r, _ in rows], device="cuda")
        g = torch.tensor([v for _, v in rows], dtype=torch.float64, device="cuda")
        gu = x[at] @ matrix(e, 0).T
        act = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
        out.index_add_(0, at, g[:, None] * (act @ matrix(e, 1).T))
    return {"out": out, "ids": None, "gates": gates}
