"""Measured cases of the gated feed-forward operators: the gated product with
its activation, its backward pass from an 8-bit checkpoint, the checkpoint's
own two directions, and layer norm.

Formulas (x E4M3 codes times one power-of-two scale per 1 x 128 group, w E4M3
codes times one per 128 x 128 block; Q(.) the library's quantisation: scale
2^e with e the smallest integer such that 448 * 2^e >= amax of the group of
128, codes rounded to nearest even):

* gated:          g = x w[:F]^T, u = x w[F:]^T, h = act(g) * u, given as BF16
                  or as Q(h) over 1 x 128 groups; the checkpoint is Q([g | u])
* gated backward: from the checkpoint's g, u and dh:
                  dg = dh * u * act'(g), du = dh * act(g), h = act(g) * u,
                  given as Q([dg | du]) over rows, Q([dg | du]) over columns
                  (groups of 128 rows) and Q(h) over columns: the operands of
                  the input's and the weights' gradient products
* save:           Q(x) over 1 x 128 groups of a BF16 activation
* use:            the saved rows, requantised over groups of 128 rows a column
* layer norm:     y = (x - mean) rstd w + b, or Q(y); backward: with
                  xh = (x - mean) rstd and t = w dy,
                  dx = rstd (t - mean(t) - xh mean(t xh)),
                  dw = sum over rows of dy xh, db = sum over rows of dy

Codes are returned as float8_e4m3fn tensors and scales as float8_e8m0fnu
tensors (the packed scale words seen byte by byte).
"""
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token through one expert-sized layer: generation at batch one, latency counts
        {"name": "gated one token", "op": "gated", "form": "dense", "m": 1, "k": 7168, "f": 2048, "groups": 1,
         "out": "bf16", "checkpoint": False, "activation": "silu"},
        # a short prompt through a narrow layer whose width fills no tile
        {"name": "gated odd sizes", "op": "gated", "form": "dense", "m": 333, "k": 1536, "f": 1000, "groups": 1,
         "out": "bf16", "checkpoint": False, "activation": "gelu_tanh"},
        # a decode batch routed to 16 experts of capacity 256, counts only known on the device
        {"name": "gated masked experts", "op": "gated", "form": "masked", "m": 256, "k": 7168, "f": 2048,
         "groups": 16, "out": "fp8", "checkpoint": False, "activation": "silu"},
        # a training step's forward pass over 4096 tokens, with the checkpoint for its backward pass
        {"name": "gated training", "op": "gated", "form": "dense", "m": 4096, "k": 7168, "f": 2048, "groups": 1,
         "out": "fp8", "checkpoint": True, "activation": "silu"},
        # a prefill batch over 8 experts, 256 to 8192 tokens each
        {"name": "gated experts", "op": "gated", "form": "contiguous", "m": 8192, "k": 7168, "f": 2048, "groups": 8,
         "out": "fp8", "checkpoint": False, "activation": "silu"},
        # the backward pass of a short batch whose rows fill no block of 128
        {"name": "gated backward odd rows", "op": "gated backward", "form": "dense", "m": 77, "f": 384, "groups": 1,
         "activation": "gelu_tanh"},
        # the backward pass of the experts' training step
        {"name": "gated backward experts", "op": "gated backward", "form": "contiguous", "m": 8192, "f": 2048,
         "groups": 8, "activation": "silu"},
        # saving the activations of 4096 tokens in 8 bits
        {"name": "checkpoint save", "op": "save", "m": 4096, "k": 7168},
        # the saved activations as an operand of the weights' gradient, over a ragged number of tokens
        {"name": "checkpoint use", "op": "use", "form": "contiguous", "m": 4097, "k": 7168, "groups": 8},
        # a short batch of odd width in single precision
        {"name": "layer norm odd width", "op": "layer norm", "m": 197, "n": 1001, "type": "fp32", "out": "same",
         "bias": True},
        # the norm before the feed-forward block, its result as the product's 8-bit operand
        {"name": "layer norm to 8 bits", "op": "layer norm", "m": 16384, "n": 7168, "type": "bf16", "out": "fp8",
         "bias": True},
        # its backward pass with the weight's and the bias's gradients
        {"name": "layer norm backward", "op": "layer norm backward", "m": 16384, "n": 7168, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated", "gated backward", "gated backward", "save", "use", "layer norm",
                     "layer norm", "layer norm backward"])
    act = rng.choice(["silu", "silu", "gelu_tanh"])
    if op == "gated":
        form = rng.choice(["dense", "dense", "contiguous", "masked"])
        out = rng.choice(["bf16", "fp8"])
        checkpoint = form != "masked" and rng.random() < 0.4
        f = 128 * _log(rng, 1, 16) if out == "fp8" or checkpoint else 8 * _log(rng, 1, 256)
        return {"op": op, "form": form, "m": _log(rng, 1, 256 if form == "masked" else 4096),
                "k": 128 * _log(rng, 1, 56), "f": f, "groups": 1 if form == "dense" else _log(rng, 2, 8),
                "out": out, "checkpoint": checkpoint, "activation": act}
    if op == "gated backward":
        form = rng.choice(["dense", "contiguous"])
        return {"op": op, "form": form, "m": _log(rng, 1, 8192), "f": 128 * _log(rng, 1, 16),
                "groups": 1 if form == "dense" else _log(rng, 2, 8), "activation": act}
    if op == "save":
        return {"op": op, "m": _log(rng, 1, 16384), "k": 128 * _log(rng, 1, 56)}
    if op == "use":
        form = rng.choice(["dense", "contiguous"])
        return {"op": op, "form": form, "m": _log(rng, 1, 8192), "k": 128 * _log(rng, 1, 56),
                "groups": 1 if form == "dense" else _log(rng, 2, 8)}
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    m = _log(rng, 1, 16384)
    if op == "layer norm backward":
        return {"op": op, "m": m, "n": _log(rng, 16, 8192), "type": kind}
    out = rng.choice(["same", "same", "fp8"])
    return {"op": op, "m": m, "n": 128 * _log(rng, 1, 64) if out == "fp8" else _log(rng, 8, 8192), "type": kind,
            "out": out, "bias": rng.random() < 0.7}


def _up(x, to):
    return (x + to - 1) // to * to


def _counts(case):
    """Tokens of each expert: a fixed spread over the case's range (some experts may get none)."""
    r = random.Random(1000 * case["m"] + case["groups"])
    return [r.randint(case["m"] // 32, case["m"]) for _ in range(case["groups"])]


# ------------------------------------------------------------------ inputs


def _exponent(amax):
    """The smallest integer e in [-127, 127] with 448 * 2^e >= amax (448 = 0.875 * 2^9); 0 where amax is 0."""
    frac, e = torch.frexp(amax)
    e = (e - 9 + (frac > 0.875)).clamp(-127, 127)
    return torch.where(amax > 0, e, 0).to(torch.int32)


def _words(e):
    """Exponents [.., rows, blocks] -> packed scale words int32 [.., ceil(blocks / 4), align(rows, 4)]."""
    rows, blocks = e.shape[-2:]
    b = (e + 127).to(torch.uint8)
    b = torch.nn.functional.pad(b, (0, _up(blocks, 4) - blocks, 0, _up(rows, 4) - rows))
    b = b.unflatten(-1, (-1, 4)).transpose(-3, -2).contiguous()
    return b.view(torch.int32).squeeze(-1)


def _rows8(x):
    """Q over 1 x 128 groups: FP32 [.., rows, cols] -> (codes, packed scale words)."""
    x = x.unflatten(-1, (-1, 128))
    e = _exponent(x.abs().amax(-1))
    return torch.ldexp(x, -e.unsqueeze(-1)).to(FP8).flatten(-2), _words(e)


def _cols8(x):
    """Q over groups of 128 rows of each column: FP32 [rows, cols], rows a multiple of 128."""
    x = x.unflatten(0, (-1, 128))
    e = _exponent(x.abs().amax(1))
    return torch.ldexp(x, -e.unsqueeze(1)).to(FP8).flatten(0, 1), _words(e.t().contiguous())


def _blocks8(w):
    """Q over 128 x 128 blocks: FP32 [.., rows, cols] -> (codes, packed scale words, one a row)."""
    rows = w.shape[-2]
    p = torch.nn.functional.pad(w, (0, 0, 0, _up(rows, 128) - rows)).unflatten(-2, (-1, 128)).unflatten(-1, (-1, 128))
    e = _exponent(p.abs().amax((-1, -3)))
    q = torch.ldexp(p, -e[..., :, None, :, None]).to(FP8).flatten(-2).flatten(-3, -2)[..., :rows, :]
    return q.contiguous(), _words(e.repeat_interleave(128, -2)[..., :rows, :].contiguous())


def _layout(case, seed):
    """Rows of the contiguous layout: (row count, m_indices, [(expert, first row, tokens)])."""
    counts = _counts(case)
    at = seed % len(counts)
    counts = counts[at:] + counts[:at]
    index, spans = [], []
    for g, c in enumerate(counts):
        spans.append((g, sum(len(i) for i in index), c))
        index.append([g] * c + [-1] * (_up(c, 128) - c))
    index = [i for part in index for i in part] or [-1] * 128
    return len(index), torch.tensor(index, dtype=torch.int32, device="cuda"), spans


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = dict(case)
    op = case["op"]
    if op == "gated":
        g, m, k, f = case["groups"], case["m"], case["k"], case["f"]
        w = normal(g, 2 * f, k) if case["form"] != "dense" else normal(2 * f, k)
        s["w"], s["w_sf"] = _blocks8(w * k ** -0.5)
        rows = (g, m) if case["form"] == "masked" else (m,)
        if case["form"] == "contiguous":
            n, s["m_indices"], s["spans"] = _layout(case, seed)
            rows = (n,)
        if case["form"] == "masked":
            counts = _counts(case)
            at = seed % g
            s["masked_m"] = torch.tensor(counts[at:] + counts[:at], dtype=torch.int32, device="cuda")
        x = normal(*rows, k)
        s["x"], s["x_sf"] = _rows8(x)
        if case["form"] == "contiguous":  # rows of padding hold whatever was there before
            s["x"].view(torch.uint8)[s["m_indices"] < 0] = 0x7F
        lead = rows[:-1]
        n = rows[-1]
        # the buffers a serving program keeps; rows that are not an expert's tokens stay as they are
        if case["form"] != "dense":
            words = lambda c: torch.zeros(*lead, _up(c, 512) // 512, _up(n, 4), dtype=torch.int32, device="cuda")  # noqa: E731
            codes = lambda c: torch.zeros(*rows, c, dtype=torch.uint8, device="cuda").view(FP8)  # noqa: E731
            s["d"] = (codes(f), words(f)) if case["out"] == "fp8" else \
                torch.zeros(*rows, f, dtype=torch.bfloat16, device="cuda")
            s["kept"] = (codes(2 * f), words(2 * f)) if case["checkpoint"] else False
    elif op == "gated backward":
        m, f = case["m"], case["f"]
        s["m_indices"] = None
        if case["form"] == "contiguous":
            m, s["m_indices"], _ = _layout(case, seed)
        s["kept"], s["kept_sf"] = _rows8(normal(m, 2 * f))
        s["dh"] = (normal(m, f) * 2.0 ** -8 * torch.exp2(normal(m, 1))).to(torch.bfloat16)
        if s["m_indices"] is not None:  # rows of padding hold whatever was there before
            s["dh"][s["m_indices"] < 0] = float("nan")
    elif op in ("save", "use"):
        m = case["m"]
        if op == "use":
            s["m_indices"] = None
            if case["form"] == "contiguous":
                m, s["m_indices"], _ = _layout(case, seed)
        x = normal(m, case["k"]) * torch.exp2(normal(1, case["k"]))
        if op == "save":
            s["x"] = x.to(torch.bfloat16)
        else:
            s["q"], s["sf"] = _rows8(x)
            if s["m_indices"] is not None:
                s["q"].view(torch.uint8)[s["m_indices"] < 0] = 0x7F
    else:
        m, n = case["m"], case["n"]
        kind = TYPES[case["type"]]
        # a residual stream: a mean of its own in each row and a few loud channels
        s["x"] = (normal(m, n) * torch.exp2(normal(1, n)) + normal(m, 1)).to(kind)
        s["weight"] = 1 + 0.1 * normal(n)
        s["shift"] = 0.1 * normal(n) if case.get("bias", True) else None
        if op == "layer norm backward":
            s["dy"] = normal(m, n).to(kind)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x.var(1, unbiased=False) + 1e-5).rsqrt()
    return s


# ------------------------------------------------------------------ plain forms


def _scales(words, rows, blocks):
    """Packed scale words -> FP32 scales [.., rows, blocks]."""
    e = words.unsqueeze(-1).view(torch.uint8).transpose(-3, -2).flatten(-2)[..., :rows, :blocks]
    return torch.exp2(e.float() - 127)


def _values(q, words):
    """Codes with packed scale words, groups of 128 along the last axis -> FP32."""
    s = _scales(words, q.shape[-2], q.shape[-1] // 128)
    return (q.float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


def _act(g, activation):
    """act(g) and act'(g)."""
    if activation == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    t = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
    dt = (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * g * g)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * dt


def _scale_values(words):
    return words.view(torch.float8_e8m0fnu)


def _gated_values(s):
    """h and [g | u] in FP32, zero in rows that belong to no token."""
    x, w = _values(s["x"], s["x_sf"]), _values(s["w"], s["w_sf"])
    f = s["f"]
    if s["form"] == "dense":
        gu = x @ w.t()
    elif s["form"] == "masked":
        gu = x @ w.transpose(1, 2)
        live = torch.arange(s["m"], device="cuda") < s["masked_m"][:, None]
        gu = torch.where(live.unsqueeze(-1), gu, 0)
    else:
        gu = torch.zeros(x.shape[0], 2 * f, device="cuda")
        for g, row, count in s["spans"]:  # one product an expert
            torch.mm(x[row:row + count], w[g].t(), out=gu[row:row + count])
    g, u = gu[..., :f], gu[..., f:]
    return _act(g, s["activation"])[0] * u, gu


def _untouched(s, out):
    """Rows that belong to no token keep what their buffers held (zeros)."""
    if s["form"] == "dense":
        return out
    live = s["m_indices"] >= 0 if s["form"] == "contiguous" else \
        torch.arange(s["m"], device="cuda") < s["masked_m"][:, None]
    q, words = out
    live = torch.nn.functional.pad(live, (0, words.shape[-1] - live.shape[-1]))
    return q, torch.where(live.unsqueeze(-2), words, 0)


def _plain(s):
    op = s["op"]
    if op == "gated":
        h, gu = _gated_values(s)
        out = {"h": h.to(torch.bfloat16)}
        if s["out"] == "fp8":
            q, words = _untouched(s, _rows8(h))
            out = {"h": q, "h scales": _scale_values(words)}
        if s["checkpoint"]:
            q, words = _untouched(s, _rows8(gu))
            out |= {"kept": q, "kept scales": _scale_values(words)}
        return out
    if op == "gated backward":
        f = s["f"]
        gu = _values(s["kept"], s["kept_sf"])
        g, u, dh = gu[:, :f], gu[:, f:], s["dh"].float()
        a, da = _act(g, s["activation"])
        both = torch.cat([dh * u * da, dh * a, a * u], 1)
        if s["m_indices"] is not None:
            both = torch.where((s["m_indices"] >= 0).unsqueeze(1), both, 0)
        q, words = _rows8(both[:, :2 * f])
        both = torch.nn.functional.pad(both, (0, 0, 0, _up(len(both), 128) - len(both)))
        qc, wc = _cols8(both[:, :2 * f])
        hc, hwc = _cols8(both[:, 2 * f:])
        return {"rows": q, "rows scales": _scale_values(words), "columns": qc, "columns scales": _scale_values(wc),
                "h": hc, "h scales": _scale_values(hwc)}
    if op == "save":
        q, words = _rows8(s["x"].float())
        return {"q": q, "scales": _scale_values(words)}
    if op == "use":
        x = _values(s["q"], s["sf"])
        if s["m_indices"] is not None:
            x = torch.where((s["m_indices"] >= 0).unsqueeze(1), x, 0)
        q, words = _cols8(torch.nn.functional.pad(x, (0, 0, 0, _up(len(x), 128) - len(x))))
        return {"q": q, "scales": _scale_values(words)}
    x, w = s["x"].float(), s["weight"]
    if op == "layer norm":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5)
        y = d * rstd * w
        y = y if s["shift"] is None else y + s["shift"]
        out = {"mean": mean.squeeze(1), "rstd": rstd.squeeze(1)}
        if s["out"] == "same":
            return out | {"y": y.to(s["x"].dtype)}
        q, words = _rows8(y)
        return out | {"y": q, "y scales": _scale_values(words)}
    dy = s["dy"].float()
    xh = (x - s["mean"].unsqueeze(1)) * s["rstd"].unsqueeze(1)
    t = dy * w
    dx = (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True)) * s["rstd"].unsqueeze(1)
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def run(s):
    if not own:
        return _plain(s)
    import moe_grouped_gemm_fp8_gb300 as dg
    op = s["op"]
    if op == "gated":
        kw = {"activation": s["activation"], "out_format": s["out"]}
        if s["form"] == "dense":
            r = dg.fp8_gated_gemm_nt(s["x"], s["x_sf"], s["w"], s["w_sf"], checkpoint=s["checkpoint"], **kw)
        elif s["form"] == "masked":
            r = dg.m_grouped_fp8_gated_gemm_nt_masked(s["x"], s["x_sf"], s["w"], s["w_sf"], s["masked_m"], d=s["d"], **kw)
        else:
            r = dg.m_grouped_fp8_gated_gemm_nt_contiguous(s["x"], s["x_sf"], s["w"], s["w_sf"], s["m_indices"], d=s["d"],
                                                          checkpoint=s["kept"], **kw)
        out = {"h": r.h}
        if r.h_sf is not None:
            out["h scales"] = _scale_values(r.h_sf)
        if r.checkpoint is not None:
            out |= {"kept": r.checkpoint, "kept scales": _scale_values(r.checkpoint_sf)}
        return out
    if op == "gated backward":
        r = dg.fp8_gated_backward(s["dh"], s["kept"], s["kept_sf"], m_indices=s["m_indices"], activation=s["activation"])
        return {"rows": r.q, "rows scales": _scale_values(r.sf), "columns": r.q_cols,
                "columns scales": _scale_values(r.sf_cols), "h": r.h_cols, "h scales": _scale_values(r.h_sf_cols)}
    if op == "save":
        q, sf = dg.quantize_fp8(s["x"], 1)
        return {"q": q, "scales": _scale_values(sf)}
    if op == "use":
        q, sf = dg.requantize_fp8_cols(s["q"], s["sf"], m_indices=s["m_indices"])
        return {"q": q, "scales": _scale_values(sf)}
    if op == "layer norm":
        r = dg.layer_norm(s["x"], s["weight"], s["shift"], eps=1e-5, out_format=s["out"])
        out = {"mean": r.mean, "rstd": r.rstd, "y": r.y}
        return out if r.sf is None else out | {"y scales": _scale_values(r.sf)}
    dx, dw, db = dg.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    return {"dx": dx, "dw": dw, "db": db}


# ------------------------------------------------------------------ 64 bits


def _scale64(amax):
    """2^e of the quantisation rule, from the binary logarithm, put right where that was rounded."""
    e = torch.ceil(torch.log2(amax / 448))
    e = torch.where(448 * torch.exp2(e - 1) >= amax, e - 1, e)
    e = torch.where(448 * torch.exp2(e) < amax, e + 1, e)
    return torch.exp2(torch.where(amax > 0, e, 0.0).clamp(-127, 127))


def _round64(x):
    """To the nearest E4M3 value, ties to even: steps of 2^-3 of the value's power of two, of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _bytes64(s, live=None):
    """Scales [.., rows, blocks] in the order of the packed words, 2^-127 (a zero byte) where a word has no block."""
    rows, blocks = s.shape[-2:]
    if live is not None:
        s = torch.where(live.unsqueeze(-1), s, 2.0 ** -127)
    s = torch.nn.functional.pad(s, (0, -blocks % 4, 0, -rows % 4), value=2.0 ** -127)
    s = s.reshape(*s.shape[:-1], -1, 4).transpose(-3, -2)
    return s.reshape(*s.shape[:-2], -1)


def _q64(x, axis, live=None, rounded=False):
    """Codes and scales of x, groups of 128 along the axis (-1 or 0). Where x is a computed number its codes are
    left as x / scale, as a result given in BF16 is left unrounded too: the rounding to eight bits is part of what
    separates a result from its exact value. Where the rounding is all there is to compute, they are rounded."""
    t = x if axis == -1 else x.t()
    g = t.reshape(*t.shape[:-1], -1, 128)
    s = _scale64(g.abs().amax(-1))
    q = g / s.unsqueeze(-1)
    q = (_round64(q) if rounded else q).reshape(t.shape)
    return (q if axis == -1 else q.t()).contiguous(), _bytes64(s, live).contiguous()


def _real64(q, words):
    rows, blocks = q.shape[-2], q.shape[-1] // 128
    b = words.contiguous().view(torch.uint8).reshape(*words.shape, 4).double()
    s = torch.exp2(b.transpose(-3, -2).reshape(*words.shape[:-2], words.shape[-1], -1)[..., :rows, :blocks] - 127)
    return q.double() * s.repeat_interleave(128, -1)


def _act64(g, activation):
    if activation == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    c = (2 / torch.pi) ** 0.5
    z = 2 * c * (g + 0.044715 * g ** 3)  # (1 + tanh(z / 2)) / 2 is the logistic function of z
    p = torch.sigmoid(z)
    return g * p, p + g * p * torch.sigmoid(-z) * 2 * c * (1 + 3 * 0.044715 * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        f = case["f"]
        live = None
        if case["form"] == "contiguous":
            live = s["m_indices"] >= 0
            x = torch.where(live.unsqueeze(1), _real64(s["x"], s["x_sf"]), 0)
            gu = torch.zeros(len(x), 2 * f, dtype=torch.float64, device="cuda")
            for g in range(case["groups"]):
                rows = torch.nonzero(s["m_indices"] == g).squeeze(1)
                gu[rows] = x[rows] @ _real64(s["w"][g], s["w_sf"][g]).t()
        else:
            gu = _real64(s["x"], s["x_sf"]) @ _real64(s["w"], s["w_sf"]).transpose(-1, -2)
            if case["form"] == "masked":
                live = torch.arange(case["m"], device="cuda").expand(case["groups"], -1) < s["masked_m"].unsqueeze(1)
                gu = torch.where(live.unsqueeze(-1), gu, 0)
        h = _act64(gu[..., :f], case["activation"])[0] * gu[..., f:]
        out = {"h": h}
        if case["out"] == "fp8":
            out["h"], out["h scales"] = _q64(h, -1, live)
        if case["checkpoint"]:
            out["kept"], out["kept scales"] = _q64(gu, -1, live)
        return out
    if op == "gated backward":
        f = case["f"]
        kept, dh = _real64(s["kept"], s["kept_sf"]), s["dh"].double()
        if s["m_indices"] is not None:
            dead = (s["m_indices"] < 0).unsqueeze(1)
            kept, dh = kept.masked_fill(dead, 0), dh.masked_fill(dead, 0)
        a, da = _act64(kept[:, :f], case["activation"])
        grad = torch.cat((da * kept[:, f:] * dh, a * dh), 1)
        h = a * kept[:, f:]
        out = {}
        out["rows"], out["rows scales"] = _q64(grad, -1)
        more = (0, 0, 0, -len(h) % 128)
        out["columns"], out["columns scales"] = _q64(torch.nn.functional.pad(grad, more), 0)
        out["h"], out["h scales"] = _q64(torch.nn.functional.pad(h, more), 0)
        return out
    if op == "save":
        q, b = _q64(s["x"].double(), -1, rounded=True)
        return {"q": q, "scales": b}
    if op == "use":
        x = _real64(s["q"], s["sf"])
        if s["m_indices"] is not None:
            x = x.masked_fill((s["m_indices"] < 0).unsqueeze(1), 0)
        q, b = _q64(torch.nn.functional.pad(x, (0, 0, 0, -len(x) % 128)), 0, rounded=True)
        return {"q": q, "scales": b}
    x, w = s["x"].double(), s["weight"].double()
    if op == "layer norm":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * w
        if s["shift"] is not None:
            y = y + s["shift"].double()
        out = {"mean": mean, "rstd": rstd, "y": y}
        if case["out"] == "fp8":
            out["y"], out["y scales"] = _q64(y, -1)
        return out
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    xh = (x - s["mean"].double()[:, None]) * rstd
    t = w * dy
    dx = rstd * (t - (t.sum(1, keepdim=True) + xh * (xh * t).sum(1, keepdim=True)) / case["n"])
    return {"dx": dx, "dw": torch.einsum("rc,rc->c", dy, xh), "db": dy.sum(0)}


# ------------------------------------------------------------------ work


def work(case):
    """Bytes: each input read once, each output written once; operations: two a multiply-add of the products,
    and about 20 an element of the activation's and the norm's arithmetic."""
    op = case["op"]
    sf = lambda rows, cols: rows * cols / 128  # noqa: E731
    if op in ("gated", "gated backward", "use"):
        live = case["m"] if case.get("form", "dense") == "dense" else sum(_counts(case))
        rows = sum(_up(c, 128) for c in _counts(case)) if case.get("form") == "contiguous" else live
    if op == "gated":
        k, f = case["k"], case["f"]
        used = sum(c > 0 for c in _counts(case)) if case["form"] != "dense" else 1
        b = used * (2 * f * k + 4 * 2 * f * k / 512) + live * k + sf(live, k)
        b += live * f * (2 if case["out"] == "bf16" else 1 + 1 / 128)
        b += 2 * (live * f + sf(live, f)) if case["checkpoint"] else 0
        return {"bytes": b, "flops": 2.0 * live * k * 2 * f + 20.0 * live * f}
    if op == "gated backward":
        f = case["f"]
        b = live * f * 2 + 2 * live * f + sf(live, 2 * f)
        return {"bytes": b + rows * f * (2 + 2 + 1) * (1 + 1 / 128) + (4 * rows if case["form"] != "dense" else 0),
                "flops": 20.0 * live * f}
    if op == "save":
        n = case["m"] * case["k"]
        return {"bytes": n * (2 + 1 + 1 / 128), "flops": 3.0 * n}
    if op == "use":
        return {"bytes": live * case["k"] * (1 + 1 / 128) + rows * case["k"] * (1 + 1 / 128)
                + (4 * rows if case["form"] != "dense" else 0), "flops": 3.0 * live * case["k"]}
    n, size = case["m"] * case["n"], {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    if op == "layer norm":
        wrote = n * size if case["out"] == "same" else n * (1 + 1 / 128)
        return {"bytes": n * size + wrote + 8 * case["m"] + 8 * case["n"], "flops": 8.0 * n}
    return {"bytes": 3 * n * size + 8 * case["m"] + 12 * case["n"], "flops": 14.0 * n}
