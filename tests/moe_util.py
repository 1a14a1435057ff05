"""64-bit CPU forms of the mixture-of-experts operators, written from their
definitions in include/mk.h, with how far a kernel's results may be off, and the
inputs that their tests share."""
from types import SimpleNamespace

import torch

GROUP = 32
BF16 = torch.finfo(torch.bfloat16).eps / 2     # a rounding to bf16, relative
F32 = torch.finfo(torch.float32).eps / 2
E4M3_STEP, E4M3_MIN = 2.0 ** -4, 2.0 ** -10    # a rounding to e4m3: relative, and absolute below its normal numbers


def dims(hidden, experts, k, ffn):
    return SimpleNamespace(hidden=hidden, n_experts=experts, top_k=k, expert_ffn=ffn)


def normal(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def scale_of(top):
    """k of groups with these largest magnitudes."""
    m, e = torch.frexp(top.float())
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(top == 0, torch.full_like(k, -127), k).clamp(-127, 127)
    return torch.where(torch.isinf(top), torch.full_like(k, 127), k)


def quantise(x):
    """Codes (float8_e4m3fn) and scales (uint8) of float32 or bf16 rows, exactly as mk.h says."""
    g = x.double().unflatten(-1, (-1, GROUP))
    top = torch.nan_to_num(g.abs(), nan=0.0, posinf=float("inf")).amax(-1)
    k = scale_of(top)
    v = torch.ldexp(g, -k.unsqueeze(-1).double())
    v = torch.where(torch.isnan(v), v, v.clamp(-448, 448)).float().to(torch.float8_e4m3fn)
    return v.flatten(-2), (k + 127).to(torch.uint8)


def values(codes, scales):
    """What 8-bit rows (CPU) stand for, in 64 bits."""
    return torch.ldexp(codes.double().unflatten(-1, (-1, GROUP)), scales.double().unsqueeze(-1) - 127).flatten(-2)


def check_eights(codes, scales, ref, slack):
    """8-bit results against 64-bit ones that the unrounded results were within `slack` of: a scale is that of a
    largest magnitude within slack, and a code half a step of it off, and the slack."""
    top, s = (x.unflatten(-1, (-1, GROUP)).amax(-1) for x in (ref.abs(), slack))
    k = scales.int() - 127
    # (a float32 in between has the scale of one of the two ends, or theirs if they agree)
    lo, hi = scale_of((top - s).clamp(min=0) * (1 - F32)), scale_of((top + s) * (1 + F32))
    assert ((k >= lo) & (k <= hi)).all(), ((k < lo) | (k > hi)).nonzero()[:5].tolist()
    unit = torch.ldexp(torch.ones((), dtype=torch.float64), k.double()).repeat_interleave(GROUP, -1)
    err = (values(codes, scales) - ref).abs()
    bad = err > E4M3_STEP * ref.abs() + E4M3_MIN * unit + (1 + E4M3_STEP) * slack
    assert not bad.any(), (int(bad.sum()), float(err.max()), bad.nonzero()[:5].tolist())


def check_eights_strictly(codes, scales, ref, slack):
    """check_eights for finite results: a NaN is none (a comparison with one is false, so it passes there)."""
    v = values(codes, scales)
    assert torch.isfinite(ref).all() and torch.isfinite(v).all(), (~torch.isfinite(v)).nonzero()[:5].tolist()
    check_eights(codes, scales, ref, slack)


def norm(x, add, gamma, eps):
    """(t, out, slack of t, slack of out) in 64 bits.  Each of the j sums in fp32 is off by half a step of what has
    been summed.  The square sum's error is that of t and of its own sums: a thread adds 64 squares one after another,
    then come 5 and 8 more (77 roundings, half of them under the root), the root, the quotient and two products."""
    x = x.double()
    terms = 0 if add is None else add.shape[1]
    t = x if add is None else x + add.double().sum(1)
    size = x.abs() if add is None else x.abs() + add.double().abs().sum(1)
    dt = terms * F32 * size
    rms = torch.sqrt(t.square().mean(-1, keepdim=True) + eps)
    g = torch.ones(x.shape[-1]).double() if gamma is None else gamma.double()
    out = t / rms * g
    rel = 48 * F32 + dt.norm(dim=-1, keepdim=True) / t.norm(dim=-1, keepdim=True).clamp(min=1e-300)
    return t, out, dt, dt / rms * g.abs() + rel * out.abs()


def route(logits, k):
    """ids, gates (64 bits), first, order as Python does them."""
    rows, experts = logits.shape
    ids = torch.full((rows, k), -1, dtype=torch.int32)
    gates = torch.zeros(rows, k, dtype=torch.float64)
    for r in range(rows):
        row = logits[r].tolist()
        some = sorted((e for e in range(experts) if row[e] == row[e] and row[e] != float("-inf")), key=lambda e: (-row[e], e))[:k]
        ids[r, :len(some)] = torch.tensor(some, dtype=torch.int32)
        if some:
            w = torch.exp(logits[r, some].double() - logits[r, some[0]].double())
            gates[r, :len(some)] = w / w.sum()
            if any(v != v for v in row):
                gates[r, :len(some)] = float("nan")
    first, order = lists(ids, experts)
    return ids, gates, first, order


def lists(ids, experts):
    flat = ids.flatten().tolist()
    order = sorted(range(len(flat)), key=lambda p: (flat[p] if flat[p] >= 0 else experts, p))
    first = [sum(1 for x in flat if 0 <= x < e) for e in range(experts + 1)]
    return torch.tensor(first, dtype=torch.int32), torch.tensor(order, dtype=torch.int32)


def products(rows, w, first):
    """Each expert's product of its rows [pairs, K] with w [experts, K, N], and the sum of the magnitudes; live pairs
    alone."""
    y = torch.zeros(rows.shape[0], w.shape[2], dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(first[e]), int(first[e + 1])
        if b > a:
            y[a:b] = rows[a:b] @ w[e]
            mag[a:b] = rows[a:b].abs() @ w[e].abs()
    return y, mag


def sum_slack(mag, k):
    """An instruction adds 16 products (8 bits: 32) to an fp32 sum; taken to be off by a step of fp32 twice over for
    each one, relative to the magnitudes."""
    return (k / 16 + 1) * 2.0 ** -22 * mag


def up(x, w, first, order, k):
    """h and its slack in 64 bits; x [rows, H], w [experts, 2 F, H] in 64 bits."""
    y, mag = products(x[order.long() // k], w.transpose(1, 2), first)
    d = sum_slack(mag, x.shape[1])
    g, u, dg, du = y[:, 0::2], y[:, 1::2], d[:, 0::2], d[:, 1::2]
    s = g * torch.sigmoid(g)
    # |silu'| < 1.1; the fast exponential is off by 2^-21 (1 + |g|) at most, the fast quotient by 2^-22
    return s * u, 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + (s * u).abs() * 2.0 ** -20 * (1 + g.abs())


def down(h, w, first, order, gates):
    """y [pairs, H] and its slack; h [pairs, F] (sorted), w [experts, F, H] in 64 bits; gates [pairs] or None."""
    y, mag = products(h, w, first)
    d = sum_slack(mag, h.shape[1]) + F32 * y.abs()
    live = int(first[-1])
    out, slack = torch.zeros_like(y), torch.zeros_like(y)
    at = order[:live].long()
    g = torch.ones(h.shape[0]).double() if gates is None else gates.double().flatten()
    out[at], slack[at] = y[:live] * g[at].unsqueeze(1), d[:live] * g[at].abs().unsqueeze(1)
    return out, slack


def within(got, ref, slack, step=BF16):
    """Results rounded once."""
    err = (got.double() - ref).abs()
    bad = ~(err <= step * ref.abs() + (1 + step) * slack + 1e-38)
    assert not bad.any(), (int(bad.sum()), float(err.max()), bad.nonzero()[:5].tolist())
