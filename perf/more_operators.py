"""The operators of a chunk's mixture of experts, measured by themselves.

They are the other half of a layer over a chunk of new tokens (a prompt, a part
of one, a single next token, a few drafted tokens of several requests):

  norm      add the terms of the block before to the residual, normalise (root
            mean square), give the rows as bf16 or in 8 bits
  quantize  rows, or weights once, to 8 bits
  route     the k experts of each row with their gates, and the rows of each
            expert side by side
  up        each expert's gate and up products over its rows, with SwiGLU
  down      each expert's down product, times the rows' gates

8 bits means e4m3 codes with a power-of-two scale for every 32 consecutive
values of a row.  Shapes are those of the model that the decode step is quoted
on (hidden 2048, 128 experts of 768, 8 for each row), of its mid and tiny
forms, and odd ones around them.
"""
import math
import types

import torch

own = False

EPS = 1e-6
GROUP = 32
# hidden, experts, experts of a row, ffn
MOE = {"full": (2048, 128, 8, 768), "mid": (2048, 64, 8, 768), "tiny": (256, 8, 2, 512), "odd": (1056, 37, 3, 352),
       "dense": (1024, 1, 1, 1408)}


def listed():
    return [
        # eight requests' drafted tokens behind the attention's projection, on their way to 8-bit experts: latency counts
        dict(name="norm_drafts_e4m3", op="norm", rows=37, n=2048, x="fp32", terms=1, out="e4m3"),
        # a prompt's rows behind the experts: the sum of eight terms, the residual, the next layer's input
        dict(name="norm_prompt", op="norm", rows=8143, n=2048, x="fp32", terms=8, out="bf16"),
        # the attention's rows of a prompt, on their way to an 8-bit projection
        dict(name="quantize_rows", op="quantize", rows=2049, n=4096, x="bf16"),
        # a layer's gate and up weights, once
        dict(name="quantize_weights", op="quantize", rows=128 * 1536, n=2048, x="bf16"),
        # one request's next token: latency counts
        dict(name="route_token", op="route", moe="full", rows=1),
        # a prompt
        dict(name="route_prompt", op="route", moe="full", rows=8143),
        # one request's next token: eight experts with one row each
        dict(name="up_token", op="up", moe="full", kind="bf16", rows=1),
        # a prompt of a few thousand tokens: each expert has a tile or two of rows
        dict(name="up_prompt", op="up", moe="full", kind="bf16", rows=2049),
        # a long prompt through 8-bit experts
        dict(name="up_long_e4m3", op="up", moe="full", kind="e4m3", rows=8143),
        # eight requests' drafted tokens through 8-bit experts: nearly every expert has a row or two
        dict(name="down_drafts_e4m3", op="down", moe="full", kind="e4m3", rows=37),
        # the same prompt, and the long one
        dict(name="down_prompt", op="down", moe="full", kind="bf16", rows=2049),
        dict(name="down_long", op="down", moe="full", kind="bf16", rows=8143),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "route", "up", "up", "down", "down"))
    if op == "norm":
        out = rng.choice(("bf16", "e4m3"))
        n = _log(rng, 2, 256) * 32 if out == "e4m3" else _log(rng, 8, 1024) * 8
        return dict(op=op, rows=_log(rng, 1, 8192 * 2048 // max(n, 2048)), n=n, x=rng.choice(("fp32", "fp32", "bf16")),
                    terms=rng.choice((0, 1, 1, 2, 8)), out=out)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 20000), n=_log(rng, 1, 200) * 32, x=rng.choice(("bf16", "fp32")))
    rows = _log(rng, 1, 8192)
    if op == "route":
        return dict(op=op, moe=rng.choice(("full", "mid", "tiny", "odd")), rows=rows)
    return dict(op=op, moe=rng.choice(("full", "full", "mid", "tiny", "odd", "dense")), kind=rng.choice(("bf16", "e4m3")), rows=rows)


# ---- what the cases share ----

def _stored(kind, n):
    """Bytes of n values."""
    return {"fp32": 4, "bf16": 2, "e4m3": 1 + 1 / GROUP}[kind] * n


def work(case):
    op, t = case["op"], case["rows"]
    if op == "norm":
        n = t * case["n"]
        return {"bytes": _stored(case["x"], n) * (2 if case["terms"] else 1) + 2 * n * case["terms"] + _stored(case["out"], n),
                "flops": n * (case["terms"] + 4)}
    if op == "quantize":
        n = t * case["n"]
        return {"bytes": _stored(case["x"], n) + _stored("e4m3", n), "flops": 2 * n}
    h, e, k, f = MOE[case["moe"]]
    if op == "route":
        return {"bytes": t * (4 * e + 12 * k), "flops": t * e * k}
    active = e * (1 - (1 - k / e) ** t) if e > k else e       # experts that have a row
    size, pairs = lambda n: _stored(case["kind"], n), t * k   # noqa: E731
    if op == "up":
        return {"bytes": size(active * 2 * f * h + t * h + pairs * f) + 4 * pairs, "flops": 4 * pairs * f * h}
    return {"bytes": size(active * f * h + pairs * f) + 8 * pairs + 2 * pairs * h, "flops": 2 * pairs * f * h}


def _quantised(x):
    """Rows of the last axis in 8 bits: e4m3 codes, and for every 32 values the exponent + 127 of the smallest power of
    two that brings their largest magnitude within 448."""
    g = x.unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(g.abs().amax(-1))
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(m == 0, torch.full_like(k, -127), k).clamp(-127, 127)
    return torch.ldexp(g, -k.unsqueeze(-1)).flatten(-2).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _values(codes, scales):
    """What 8-bit rows stand for, in 32 bits."""
    return torch.ldexp(codes.float().unflatten(-1, (-1, GROUP)), scales.int().unsqueeze(-1) - 127).flatten(-2)


def _normal(shape, gen, scale=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0, scale, generator=gen)


def _routed(logits, k):
    """ids and gates [rows, k], first [experts + 1], order [rows * k]."""
    top, ids = logits.sort(dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = (top - top[:, :1]).exp()
    flat = ids.flatten()
    first = torch.zeros(logits.shape[1] + 1, dtype=torch.int64, device=logits.device)
    first[1:] = torch.bincount(flat, minlength=logits.shape[1]).cumsum(0)
    return ids.int(), w / w.sum(-1, keepdim=True), first.int(), flat.sort(stable=True)[1].int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = types.SimpleNamespace(case=case)
    op, t, kinds = case["op"], case["rows"], {"fp32": torch.float32, "bf16": torch.bfloat16}
    new = lambda shape, kind: torch.empty(shape, dtype=kind, device="cuda")   # noqa: E731
    if op in ("norm", "quantize"):
        n = case["n"]
        if op == "quantize":
            # rows of different sizes, as activations and weights have them
            s.x = (_normal((t, n), gen) * _normal((t, 1), gen).exp()).to(kinds[case["x"]])
            s.codes, s.scales = (new((t, n), torch.float8_e4m3fn), new((t, n // GROUP), torch.uint8)) if own else (None, None)
            return s
        s.x = _normal((t, n), gen, 2.0).to(kinds[case["x"]])
        s.add = _normal((t, case["terms"], n), gen, 0.5, torch.bfloat16) if case["terms"] else None
        s.gamma = (1 + _normal((n,), gen, 0.02)).bfloat16()
        if own:
            s.total = torch.empty_like(s.x) if case["terms"] else None
            s.out = new((t, n), torch.bfloat16 if case["out"] == "bf16" else torch.float8_e4m3fn)
            s.scales = new((t, n // GROUP), torch.uint8) if case["out"] == "e4m3" else None
        return s
    h, e, k, f = MOE[case["moe"]]
    # the router's logits of a layer that has its favourites
    s.logits = _normal((t, e), gen, 0.9) + _normal((1, e), gen, 0.3)
    if op == "route":
        if own:
            s.ids, s.gates = new((t, k), torch.int32), new((t, k), torch.float32)
            s.first, s.order = new((e + 1,), torch.int32), new((t * k,), torch.int32)
        return s
    s.ids, s.gates, s.first, s.order = _routed(s.logits, k)
    bf16 = case["kind"] == "bf16"
    if op == "up":
        x, shape, width = _normal((t, h), gen), (e, 2 * f, h), f
    else:
        a = _normal((t * k, f), gen, 0.9)
        # bf16: an expert's rows of w are its ffn units; 8 bits: its hidden units, so that the products run along a row
        x, shape, width = a / (1 + torch.exp(-a)) * _normal((t * k, f), gen, 0.9), (e, f, h) if bf16 else (e, h, f), h
    w = _normal(shape, gen, 0.02, torch.bfloat16)
    if bf16:
        s.x, s.xs, s.w, s.ws = x.bfloat16(), None, w, None
    else:
        (s.x, s.xs), (s.w, s.ws) = _quantised(x), _quantised(w.float())
    if own:
        from persistent_moe_decode_02_gb300 import mk
        s.experts = mk.Experts(types.SimpleNamespace(hidden=h, n_experts=e, top_k=k, expert_ffn=f), case["kind"])
        s.out = new((t * k, width), torch.bfloat16 if bf16 or op == "down" else torch.float8_e4m3fn)
        s.scales = new((t * k, width // GROUP), torch.uint8) if op == "up" and not bf16 else None
    else:
        s.most = int((s.first[1:] - s.first[:-1]).max())      # rows of the busiest expert
    return s


# ---- one pass ----

def _eights(codes, scales):
    return {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}


def _plain_norm(s):
    total = s.x.float()
    if s.add is not None:
        total = total + s.add.float().sum(1)
    y = total * torch.rsqrt(total.square().mean(-1, keepdim=True) + EPS) * s.gamma.float()
    out = {"out": y.bfloat16()} if s.case["out"] == "bf16" else _eights(*_quantised(y))
    return out if s.add is None else {"total": total.to(s.x.dtype), **out}


def _plain_products(s, rows, transposed):
    """Each expert's product over its rows [pairs, n], in the order of its rows."""
    first = s.first.long()
    pairs = rows.shape[0]
    expert = torch.searchsorted(first[1:].contiguous(), torch.arange(pairs, device="cuda"), right=True)
    some = pairs <= s.w.shape[0]                              # few rows: the weights of each row's expert
    w, ws = (s.w[expert], None if s.ws is None else s.ws[expert]) if some else (s.w, s.ws)
    w = w.float() if ws is None else _values(w, ws)
    w = w if transposed else w.transpose(1, 2)
    if some:
        return torch.bmm(rows.unsqueeze(1), w).squeeze(1)
    place = torch.arange(pairs, device="cuda") - first[expert]
    each = torch.zeros(s.w.shape[0], s.most, rows.shape[1], device="cuda")
    each[expert, place] = rows
    return torch.bmm(each, w)[expert, place]


def _plain_up(s):
    k = s.ids.shape[1]
    x = s.x.float() if s.xs is None else _values(s.x, s.xs)
    y = _plain_products(s, x[s.order.long() // k], False)
    gate, up = y[:, 0::2], y[:, 1::2]                         # a unit's gate and up rows lie side by side
    h = gate / (1 + torch.exp(-gate)) * up
    return h.bfloat16() if s.xs is None else _eights(*_quantised(h))


def _plain_down(s):
    x = s.x.float() if s.xs is None else _values(s.x, s.xs)
    y = _plain_products(s, x, s.xs is None)
    order = s.order.long()
    out = torch.empty_like(y)
    out[order] = y * s.gates.flatten()[order].unsqueeze(1)
    return out.bfloat16()


def run(s):
    op = s.case["op"]
    if own:
        from persistent_moe_decode_02_gb300 import mk
        if op == "norm":
            mk.norm(s.x, s.gamma, EPS, s.out, add=s.add, total=s.total, scales=s.scales)
            out = {"out": s.out} if s.scales is None else _eights(s.out, s.scales)
            return out if s.add is None else {"total": s.total, **out}
        if op == "quantize":
            mk.quantize(s.x, s.codes, s.scales)
            return _eights(s.codes, s.scales)
        if op == "route":
            mk.route(s.logits, s.ids, s.gates, s.first, s.order)
            return {"ids": s.ids, "gates": s.gates, "first": s.first, "order": s.order}
        if op == "up":
            s.experts.up(s.x, s.w, s.first, s.order, s.out, x_scales=s.xs, w_scales=s.ws, h_scales=s.scales)
            return s.out if s.scales is None else _eights(s.out, s.scales)
        s.experts.down(s.x, s.w, s.first, s.order, s.gates, s.out, h_scales=s.xs, w_scales=s.ws)
        return s.out
    if op == "norm":
        return _plain_norm(s)
    if op == "quantize":
        return _eights(*_quantised(s.x.float()))
    if op == "route":
        ids, gates, first, order = _routed(s.logits, MOE[s.case["moe"]][2])
        return {"ids": ids, "gates": gates, "first": first, "order": order}
    return _plain_up(s) if op == "up" else _plain_down(s)


# ---- the definitions in 64 bits ----

def _exact_eights(v):
    top = v.view(v.shape[0], -1, GROUP).abs().amax(-1)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448) - 1e-12).clamp(min=-127))
    return {"codes": v / scale.repeat_interleave(GROUP, 1), "scales": scale}


def _wide(x, scales):
    if scales is None:
        return x.double()
    return x.double() * torch.exp2(scales.double() - 127).repeat_interleave(GROUP, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_eights(s.x.double())
    if op == "norm":
        t = s.x.double()
        for j in range(case["terms"]):
            t = t + s.add[:, j].double()
        y = t / torch.sqrt((t * t).mean(1, keepdim=True) + EPS) * s.gamma.double()
        out = {"out": y} if case["out"] == "bf16" else _exact_eights(y)
        return {"total": t, **out} if case["terms"] else out
    if op == "route":
        k = MOE[case["moe"]][2]
        top = s.logits.double().topk(k, dim=1).values
        return {"ids": None, "gates": torch.softmax(top, 1), "first": None, "order": None}
    first, order, k = s.first.tolist(), s.order.long(), s.ids.shape[1]
    out = torch.zeros(order.numel(), MOE[case["moe"]][3] if op == "up" else MOE[case["moe"]][0], dtype=torch.float64, device="cuda")
    for e in range(len(first) - 1):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        w = _wide(s.w[e], None if s.ws is None else s.ws[e])
        rows = order[a:b] // k if op == "up" else torch.arange(a, b, device="cuda")
        x = _wide(s.x[rows], None if s.xs is None else s.xs[rows])
        if op == "up":
            y = (x @ w.T).view(b - a, -1, 2)
            out[a:b] = y[:, :, 0] * torch.sigmoid(y[:, :, 0]) * y[:, :, 1]
        else:
            y = x @ (w if s.xs is None else w.T)
            out[order[a:b]] = y * s.gates.double().view(-1)[order[a:b], None]
    return _exact_eights(out) if op == "up" and s.xs is not None else out
