"""Measured cases of the serving operators: a whole mixture-of-experts layer for
a few tokens, the product of 8-bit integers with a scale for each token and
channel, and the quantiser that makes its operands.

Formulas:

* moe:      l = x r^T (x BF16 [T, D], r [E, D]); scores s = softmax(l) over the
            experts, or the logistic function of l; the k experts of a token
            with the largest l (logistic with a bias b: the largest s + b), ties
            to the lowest index; weights s of the chosen, divided by their sum
            where renormalised. With W = codes times one power of two per
            128 x 128 block: g = x Wg^T, u = x Wu^T, h = act(g) u of each chosen
            expert, y = c + sum over them of weight h Wd^T, rounded once
* int8:     D = c + sa[m] sb[n] sum over k of a[m, k] b[n, k], a and b int8
* quantise: amax of a row, scale = amax / 127, code = the integer nearest to
            127 x / amax, ties to even
"""
import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # generation at batch one: each chosen expert is read once, for one token
        {"name": "moe one token", "op": "moe", "t": 1, "d": 7168, "f": 2048, "e": 32, "k": 8, "score": "softmax",
         "router": "fp32", "bias": False, "renormalize": True, "activation": "silu", "residual": False, "padded": False},
        # a small model's layer for three requests: latency counts; widths that fill no tile, an odd number of experts
        {"name": "moe small odd", "op": "moe", "t": 3, "d": 1152, "f": 384, "e": 7, "k": 2, "score": "softmax",
         "router": "bf16", "bias": False, "renormalize": False, "activation": "gelu_tanh", "residual": True, "padded": False},
        # a decode batch: most experts hit, by one to three tokens each
        {"name": "moe decode batch", "op": "moe", "t": 16, "d": 7168, "f": 2048, "e": 64, "k": 8, "score": "sigmoid",
         "router": "fp32", "bias": True, "renormalize": True, "activation": "silu", "residual": True, "padded": False},
        # the largest batch, padded for a captured graph, many tokens an expert
        {"name": "moe many tokens", "op": "moe", "t": 64, "d": 7168, "f": 2048, "e": 16, "k": 4, "score": "softmax",
         "router": "bf16", "bias": False, "renormalize": True, "activation": "silu", "residual": True, "padded": True},
        # one token through a projection
        {"name": "int8 one token", "op": "int8", "m": 1, "n": 7168, "k": 2048, "out": "bf16", "c": False},
        # a decode batch through a projection
        {"name": "int8 decode", "op": "int8", "m": 64, "n": 4096, "k": 7168, "out": "bf16", "c": True},
        # a short prompt, sizes that fill no tile
        {"name": "int8 odd sizes", "op": "int8", "m": 333, "n": 1001, "k": 1552, "out": "fp16", "c": False},
        # a prompt
        {"name": "int8 prefill", "op": "int8", "m": 4096, "n": 4096, "k": 7168, "out": "bf16", "c": True},
        # a prompt through a wide projection of short rows: much output for its work
        {"name": "int8 wide", "op": "int8", "m": 4096, "n": 24576, "k": 1536, "out": "bf16", "c": False},
        # one token's row as the product's operand
        {"name": "quantise one token", "op": "quantise", "m": 1, "n": 7168, "type": "bf16"},
        # a short batch of odd width in single precision
        {"name": "quantise odd width", "op": "quantise", "m": 197, "n": 1001, "type": "fp32"},
        # the rows of a long prompt
        {"name": "quantise prompt", "op": "quantise", "m": 16384, "n": 7168, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["moe", "moe", "moe", "int8", "int8", "int8", "quantise", "quantise"])
    if op == "moe":
        e = _log(rng, 2, 64)
        score = rng.choice(["softmax", "softmax", "sigmoid"])
        return {"op": op, "t": _log(rng, 1, 64), "d": 128 * _log(rng, 1, 56), "f": 128 * _log(rng, 1, 16), "e": e,
                "k": min(e, _log(rng, 1, 8)), "score": score, "router": rng.choice(["bf16", "fp32"]),
                "bias": score == "sigmoid" and rng.random() < 0.6, "renormalize": rng.random() < 0.7,
                "activation": rng.choice(["silu", "silu", "gelu_tanh"]), "residual": rng.random() < 0.6,
                "padded": rng.random() < 0.3}
    if op == "int8":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 8, 16384), "k": 16 * _log(rng, 1, 512),
                "out": rng.choice(["bf16", "bf16", "fp16"]), "c": rng.random() < 0.4}
    return {"op": op, "m": _log(rng, 1, 16384), "n": _log(rng, 8, 8192), "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}


def _up(x, to):
    return (x + to - 1) // to * to


def _live(case):
    """Tokens of a padded batch: a fixed part of its rows."""
    return max(1, case["t"] * 5 // 8) if case["padded"] else case["t"]


# ------------------------------------------------------------------ inputs


def _blocks8(w):
    """FP32 [rows, cols] -> (E4M3 codes, packed scale words int32 [ceil(cols / 512), align(rows, 4)]): one scale
    2^e per 128 x 128 block, e the smallest integer with 448 * 2^e >= the block's largest magnitude."""
    rows, cols = w.shape
    p = torch.nn.functional.pad(w, (0, 0, 0, _up(rows, 128) - rows)).view(-1, 128, cols // 128, 128)
    frac, e = torch.frexp(p.abs().amax((1, 3)))
    e = (e - 9 + (frac > 0.875)).clamp(-127, 127).to(torch.int32)  # 448 = 0.875 * 2^9
    q = (p * torch.exp2(-e.float())[:, None, :, None]).to(FP8).view(-1, cols)[:rows]
    b = (e + 127).to(torch.uint8).repeat_interleave(128, 0)[:rows]
    b = torch.nn.functional.pad(b, (0, _up(cols // 128, 4) - cols // 128, 0, _up(rows, 4) - rows))
    return q, b.unflatten(1, (-1, 4)).transpose(0, 1).contiguous().view(torch.int32).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "moe":
        t, d, f, e = case["t"], case["d"], case["f"], case["e"]
        up, up_sf, down, down_sf = [], [], [], []
        for _ in range(e):
            q, sf = _blocks8(normal(2 * f, d) * d ** -0.5)
            up.append(q)
            up_sf.append(sf)
            q, sf = _blocks8(normal(d, f) * f ** -0.5)
            down.append(q)
            down_sf.append(sf)
        # (stacked as bytes: not every version of torch stacks 8-bit floating types)
        stack = lambda v: torch.stack([q.view(torch.uint8) for q in v]).view(FP8)  # noqa: E731
        s["up"], s["up_sf"] = stack(up), torch.stack(up_sf)
        s["down"], s["down_sf"] = stack(down), torch.stack(down_sf)
        # normed activations with a few loud channels
        s["x"] = (normal(t, d) * torch.exp2(0.5 * normal(1, d))).to(torch.bfloat16)
        s["r"] = (normal(e, d) * d ** -0.5).to(TYPES[case["router"]])
        s["b"] = 0.1 * normal(e) if case["bias"] else None
        s["c"] = normal(t, d).to(torch.bfloat16) if case["residual"] else None
        s["n"] = s["y"] = None
        if case["padded"]:  # a captured graph's batch: the count is on the device, rows past it stay as they are
            s["n"] = torch.tensor([_live(case)], dtype=torch.int32, device="cuda")
            s["y"] = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "int8":
        m, n, k = case["m"], case["n"], case["k"]
        codes = lambda rows: (normal(rows, k) * 32).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
        s["a"], s["w"] = codes(m), codes(n)
        s["sa"] = torch.exp2(normal(m)) / 32
        s["sb"] = torch.exp2(0.25 * normal(n)) / 32 * k ** -0.5
        s["res"] = normal(m, n).to(TYPES[case["out"]]) if case["c"] else None
    else:
        s["x"] = (normal(case["m"], case["n"]) * torch.exp2(normal(1, case["n"]))).to(TYPES[case["type"]])
    return s


# ------------------------------------------------------------------ plain forms


def _values(q, words):
    """E4M3 codes [rows, cols] with packed scale words -> FP32."""
    rows, cols = q.shape
    e = words.unsqueeze(-1).view(torch.uint8).transpose(0, 1).flatten(1)[:rows, :cols // 128]
    return (q.float().unflatten(1, (-1, 128)) * torch.exp2(e.float() - 127).unsqueeze(-1)).flatten(1)


def _route(s, live):
    """The chosen experts [live, k] and their weights; in 64 bits, so that near scores keep their order."""
    l = s["x"][:live].double() @ s["r"].double().t()
    score = 1 / (1 + torch.exp(-l)) if s["score"] == "sigmoid" else torch.exp(l - l.amax(1, keepdim=True))
    if s["score"] == "softmax":
        score = score / score.sum(1, keepdim=True)
    by = l if s["b"] is None else score + s["b"].double()
    chosen = torch.sort(by, dim=1, descending=True, stable=True)[1][:, :s["k"]]
    w = score.gather(1, chosen)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return chosen, w.float()


def _plain(s):
    if s["op"] == "moe":
        live, f = _live(s), s["f"]
        chosen, w = _route(s, live)
        x = s["x"][:live].float()
        y = s["c"][:live].float() if s["c"] is not None else torch.zeros_like(x)
        for e in sorted(set(chosen.flatten().tolist())):
            t, j = torch.nonzero(chosen == e, as_tuple=True)
            gu = x[t] @ _values(s["up"][e], s["up_sf"][e]).t()
            g, u = gu[:, :f], gu[:, f:]
            if s["activation"] == "silu":
                h = g / (1 + torch.exp(-g)) * u
            else:
                h = 0.5 * g * (1 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))) * u
            y[t] += w[t, j].unsqueeze(1) * (h @ _values(s["down"][e], s["down_sf"][e]).t())
        more = s["t"] - live
        pad = lambda v, value: torch.nn.functional.pad(v, (0, 0, 0, more), value=value)  # noqa: E731
        return {"y": pad(y.to(torch.bfloat16), 0.0), "experts": pad(chosen.to(torch.int32), -1), "weights": pad(w, 0.0)}
    if s["op"] == "int8":
        d = (s["a"].float() @ s["w"].float().t()) * s["sa"].unsqueeze(1) * s["sb"]
        return {"d": (d if s["res"] is None else d + s["res"].float()).to(TYPES[s["out"]])}
    x = s["x"].float()
    amax = x.abs().amax(1)
    q = torch.round(127 * x.double() / torch.where(amax > 0, amax, 1).double().unsqueeze(1))
    return {"q": q.to(torch.int8), "scales": amax / 127}


def run(s):
    if not own:
        return _plain(s)
    import moe_grouped_gemm_fp8_gb300 as dg
    if s["op"] == "moe":
        r = dg.fp8_moe_few_tokens(s["x"], s["r"], s["up"], s["up_sf"], s["down"], s["down_sf"], s["k"],
                                  router_bias=s["b"], score=s["score"], renormalize=s["renormalize"],
                                  activation=s["activation"], c=s["c"], num_tokens=s["n"], d=s["y"])
        return {"y": r.y, "experts": r.experts, "weights": r.weights}
    if s["op"] == "int8":
        return {"d": dg.int8_gemm_nt(s["a"], s["sa"], s["w"], s["sb"], c=s["res"], out_dtype=TYPES[s["out"]])}
    q, scales = dg.quantize_int8(s["x"])
    return {"q": q, "scales": scales}


# ------------------------------------------------------------------ 64 bits


def _real64(q, words):
    b = words.contiguous().view(torch.uint8).reshape(words.shape[0], words.shape[1], 4).double().permute(1, 0, 2)
    scale = 2.0 ** (b.reshape(words.shape[1], -1)[:q.shape[0], :q.shape[1] // 128] - 127)
    return q.double() * scale.repeat_interleave(128, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        t, d, f, e, k = (case[n] for n in ("t", "d", "f", "e", "k"))
        y = torch.zeros(t, d, dtype=torch.float64, device="cuda")
        experts = torch.full((t, k), -1, dtype=torch.int64)
        weights = torch.zeros(t, k, dtype=torch.float64)
        x, logits = s["x"].double(), torch.einsum("td,ed->te", s["x"].double(), s["r"].double())
        probability = (torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)).tolist()
        rank = logits.tolist()
        bias = s["b"].double().tolist() if case["bias"] else None
        for i in range(_live(case)):
            key = rank[i] if bias is None else [p + b for p, b in zip(probability[i], bias)]
            best = sorted(range(e), key=lambda j: (-key[j], j))[:k]
            total = sum(probability[i][j] for j in best) if case["renormalize"] else 1.0
            for j, expert in enumerate(best):
                experts[i, j] = expert
                weights[i, j] = probability[i][expert] / total
            if case["residual"]:
                y[i] = s["c"][i].double()
        share = torch.zeros(t, e, dtype=torch.float64)
        for i in range(_live(case)):
            share[i, experts[i]] = weights[i]
        share = share.cuda()
        for j in range(e):
            rows = torch.nonzero(share[:, j] != 0).squeeze(1)
            if len(rows):
                w = _real64(s["up"][j], s["up_sf"][j])
                g, u = x[rows] @ w[:f].t(), x[rows] @ w[f:].t()
                if case["activation"] == "silu":
                    h = g * torch.sigmoid(g) * u
                else:  # (1 + tanh(z)) / 2 is the logistic function of 2 z
                    h = g * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)) * u
                y[rows] += share[rows, j].unsqueeze(1) * (h @ _real64(s["down"][j], s["down_sf"][j]).t())
        return {"y": y, "experts": experts.to(torch.int32).cuda(), "weights": weights.cuda()}
    if case["op"] == "int8":
        d = torch.einsum("mk,nk->mn", s["a"].double(), s["w"].double())
        d = s["sa"].double()[:, None] * d * s["sb"].double()[None, :]
        return {"d": d if s["res"] is None else d + s["res"].double()}
    x = s["x"].double()
    top = torch.linalg.vector_norm(x, ord=float("inf"), dim=1)
    q = x * 127 / torch.where(top == 0, 1.0, top)[:, None]
    low = torch.floor(q)
    up = (q - low > 0.5) | ((q - low == 0.5) & (low % 2 != 0))
    return {"q": (low + up).to(torch.int8), "scales": top / 127}


# ------------------------------------------------------------------ work


def work(case):
    """Bytes: each input read once (of the experts those that a token chose, as many as are hit on average),
    each output written once; operations: two a multiply-add of the products."""
    if case["op"] == "moe":
        t, d, f, e, k = _live(case), case["d"], case["f"], case["e"], case["k"]
        hit = e * (1 - (1 - k / e) ** t)
        b = hit * 3 * f * d * (1 + 1 / 128) + e * d * (4 if case["router"] == "fp32" else 2)
        return {"bytes": b + t * d * (6 if case["residual"] else 4) + 8 * t * k,
                "flops": 6.0 * t * k * f * d + 2.0 * t * e * d}
    if case["op"] == "int8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k + 4) + m * n * (4 if case["c"] else 2), "flops": 2.0 * m * n * k}
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    return {"bytes": case["m"] * case["n"] * (size + 1) + 4 * case["m"], "flops": 3.0 * case["m"] * case["n"]}
