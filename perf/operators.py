"""The operators beside the decode megakernel that are measured by themselves.

They are the pieces of a step over a chunk of new tokens of each request (a
prompt, a part of one, a request's single next token, or a few drafted tokens
to be checked):

  append   rotate the chunk's queries and keys, write its keys and values into
           the paged cache (bf16, or 8 bits with a power-of-two scale for each
           token, head and K or V)
  attend   causal attention of the chunk's rows over the paged cache, grouped
           heads, requests of different lengths
  read     cached rows back out of the pages, as bf16
  probs    logits to probabilities at a temperature
  verify   drafted tokens checked against the target's probabilities

Shapes are those of the model that the decode step is quoted on (32 query and
4 key/value heads of 128, vocabulary 151936, pages of 16 tokens), of its mid
and tiny forms, and odd ones around them.
"""
import math
import types

import torch

own = False

PAGE = 16
THETA = 1e4
HEADS = {"full": (32, 4, 128), "tiny": (4, 2, 64), "wide": (12, 2, 128), "one": (5, 5, 64)}
VOCABS = (4096, 32000, 151936)


def listed():
    return [
        # one request's next token at 8K cached tokens: the decode step's own attention, latency counts
        dict(name="attend_token_8k", op="attend", heads="full", kv="bf16", cached="8191", new="1"),
        # eight requests check four drafted tokens each over an 8-bit cache of ragged lengths
        dict(name="attend_drafts_b8_e4m3", op="attend", heads="full", kv="e4m3",
             cached="8200,39997,1023,16384,512,27001,12345,4095", new="5,5,5,5,4,5,3,5"),
        # three whole prompts of different lengths, nothing cached yet
        dict(name="attend_prompts", op="attend", heads="full", kv="bf16", cached="0,0,0", new="2049,517,1000"),
        # the next 2048 tokens of a long prompt whose first 30000 are cached
        dict(name="attend_long_chunk", op="attend", heads="full", kv="bf16", cached="30000", new="2048"),
        # eight requests' drafted tokens enter the bf16 cache: latency counts
        dict(name="append_drafts_b8", op="append", heads="full", kv="bf16", rows="bf16",
             cached="8200,39997,1023,16384,512,27001,12345,4095", new="5,5,5,5,4,5,3,5"),
        # a prompt's part enters an 8-bit cache behind 1000 cached tokens, and a shorter one beside it
        dict(name="append_prompt_e4m3", op="append", heads="full", kv="e4m3", rows="fp32",
             cached="1000,0", new="6143,2001"),
        # a short request leaves the bf16 pool
        dict(name="read_short", op="read", heads="full", kv="bf16", cached="333", new="0"),
        # requests come back from 8 bits
        dict(name="read_e4m3", op="read", heads="full", kv="e4m3", cached="30011,9000,16384", new="0,0,0"),
        # one request's five checked positions
        dict(name="probs_5", op="probs", rows=5, vocab=151936, temperature=0.7),
        # 32 requests with five positions each
        dict(name="probs_160", op="probs", rows=160, vocab=151936, temperature=1.0),
        # one request with four drafted tokens: latency counts
        dict(name="verify_b1", op="verify", batch=1, drafts=4, vocab=151936, point=False),
        # 32 requests with up to five drafted tokens
        dict(name="verify_b32", op="verify", batch=32, drafts=5, vocab=151936, point=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(v):
    return ",".join(str(x) for x in v)


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "read", "probs", "verify"))
    if op == "probs":
        return dict(op=op, rows=_log(rng, 1, 160), vocab=rng.choice(VOCABS + (_log(rng, 1000, 151936),)),
                    temperature=round(rng.uniform(0.3, 1.5), 3))
    if op == "verify":
        return dict(op=op, batch=_log(rng, 1, 32), drafts=rng.randint(1, 7),
                    vocab=rng.choice(VOCABS[1:] + (_log(rng, 1000, 151936),)), point=rng.random() < 0.25)
    heads, kv = rng.choice(("full", "full", "tiny", "wide", "one")), rng.choice(("bf16", "e4m3"))
    batch = rng.randint(1, 6)
    if op == "read":
        cached = [_log(rng, 1, 16384) for _ in range(batch)]
        return dict(op=op, heads=heads, kv=kv, cached=_lens(cached), new=_lens([0] * batch))
    if rng.random() < 0.5:   # single tokens and drafts
        cached = [_log(rng, 1, 32768) for _ in range(batch)]
        new = [rng.randint(1, 8) for _ in range(batch)]
    else:                    # prompts and their parts
        batch = min(batch, 3)
        cached = [rng.choice((0, _log(rng, 1, 8192))) for _ in range(batch)]
        new = [_log(rng, 9, 2500) for _ in range(batch)]
    case = dict(op=op, heads=heads, kv=kv, cached=_lens(cached), new=_lens(new))
    return dict(case, rows=rng.choice(("bf16", "fp32"))) if op == "append" else case


# ---- what the cases share ----

def _sizes(case):
    nq, nkv, d = HEADS[case["heads"]]
    return nq, nkv, d, [int(x) for x in case["cached"].split(",")], [int(x) for x in case["new"].split(",")]


def work(case):
    op = case["op"]
    if op == "probs":
        n = case["rows"] * case["vocab"]
        return {"bytes": 8 * n, "flops": 5 * n}
    if op == "verify":
        # the row that the answer is drawn from: the target's, and the draft's where one was rejected
        n = case["batch"] * case["vocab"]
        return {"bytes": 4 * n * (1 if case["point"] else 2), "flops": 4 * n}
    nq, nkv, d, cached, new = _sizes(case)
    el = 2 * d if case["kv"] == "bf16" else d + 1          # one cached vector
    total = sum(cached) + sum(new)
    if op == "read":
        return {"bytes": total * nkv * 2 * (el + 2 * d), "flops": total * nkv * 2 * d}
    rows = sum(new)
    if op == "append":
        act = 2 if case["rows"] == "bf16" else 4
        return {"bytes": rows * ((nq + 2 * nkv) * d * act + nq * d * 2 + 2 * nkv * el), "flops": rows * (nq + nkv) * d * 3}
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    return {"bytes": total * nkv * 2 * el + rows * nq * d * 4, "flops": 4 * pairs * nq * d}


def _quantised(x):
    """Rows of the last axis as 8-bit floating point (e4m3) and a power-of-two scale: codes' bytes and the scales'
    exponents + 127.  The scale is the smallest power of two that brings the row's largest magnitude within 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(m == 0, torch.full_like(k, -127), k).clamp(-127, 127)
    codes = torch.ldexp(x.double(), -k.unsqueeze(-1)).float().to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (k + 127).to(torch.uint8)


def _pool(case, pages, nkv, d, gen):
    """A pool as the cache of other requests left it: [pages, nkv, 2, d, 16], K and V ~ N(0, 1); in 8 bits with one
    more row, the scales' exponents of the page's tokens."""
    if case["kv"] == "bf16":
        return torch.empty(pages, nkv, 2, d, PAGE, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    codes, exps = _quantised(torch.empty(pages, nkv, 2, PAGE, d, device="cuda").normal_(generator=gen))
    return torch.cat([codes.transpose(-1, -2), exps.unsqueeze(-2)], -2).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = types.SimpleNamespace(case=case)
    if case["op"] == "probs":
        s.logits = torch.empty(case["rows"], case["vocab"], device="cuda").normal_(0, 3, generator=gen)
        if own:
            s.out = torch.empty_like(s.logits)
        return s
    if case["op"] == "verify":
        b, k, v = case["batch"], case["drafts"], case["vocab"]
        base = torch.empty(b, k + 1, v, device="cuda").normal_(0, 3, generator=gen)
        near = base[:, :k] + torch.empty(b, k, v, device="cuda").normal_(0, 0.7, generator=gen)
        s.p = torch.softmax(base, -1)
        s.q = torch.softmax(near, -1)
        s.drafts = torch.multinomial(s.q.view(b * k, v), 1, generator=gen).view(b, k).int()
        s.count = torch.randint(0 if b > 1 else k, k + 1, (b,), device="cuda", generator=gen).int()
        if case["point"]:   # drafts by lookup, with no distribution of their own
            s.q = None
        s.u = torch.rand(b, k, device="cuda", generator=gen)
        s.r = torch.rand(b, device="cuda", generator=gen)
        if own:
            s.tokens = torch.empty(b, k + 1, dtype=torch.int32, device="cuda")
            s.accepted = torch.empty(b, dtype=torch.int32, device="cuda")
        return s
    nq, nkv, d, cached, new = _sizes(case)
    s.nq, s.nkv, s.d = nq, nkv, d
    per = [-(-(c + n) // PAGE) for c, n in zip(cached, new)]
    pages, width = sum(per) + 3, max(per)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
    table, at = [], 0
    for n in per:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    s.table = torch.tensor(table, device="cuda")
    s.pool = _pool(case, pages, nkv, d, gen)
    if own:
        from persistent_moe_decode_02_gb300 import mk
        s.chunk = mk.Chunk(types.SimpleNamespace(n_q_heads=nq, n_kv_heads=nkv, head_dim=d, page_size=PAGE, rope_theta=THETA),
                           case["kv"], pages, cached, new, [p for row in table for p in row], width)
    else:
        # each new row's request, position and place among its request's rows; each cached row's page and slot
        s.cached, s.new = torch.tensor(cached, device="cuda"), torch.tensor(new, device="cuda")
        s.req = torch.repeat_interleave(torch.arange(len(new), device="cuda"), s.new)
        s.place = torch.arange(sum(new), device="cuda") - (s.new.cumsum(0) - s.new)[s.req]
        s.pos = s.cached[s.req] + s.place
        s.most, s.longest = max(new), max(c + n for c, n in zip(cached, new))
    rows = sum(new)
    if case["op"] == "attend":
        s.q = torch.empty(rows, nq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if own:
            s.out = torch.empty_like(s.q)
    elif case["op"] == "append":
        s.qkv = torch.empty(rows, nkv, nq // nkv + 2, d, device="cuda",
                            dtype=torch.bfloat16 if case["rows"] == "bf16" else torch.float32).normal_(generator=gen)
        if own:
            s.q = torch.empty(rows, nq, d, dtype=torch.bfloat16, device="cuda")
    elif own:
        s.out = torch.empty(sum(cached) + rows, nkv, 2, d, dtype=torch.bfloat16, device="cuda")
    return s


# ---- one pass ----

def _pool_parts(s):
    """The pool as the numbers that it holds: in 8 bits the codes' and the scales' values, each as its own type has it."""
    if s.case["kv"] == "bf16":
        return {"pool": s.pool}
    return {"codes": s.pool[..., :s.d, :].view(torch.float8_e4m3fn), "scales": s.pool[..., s.d, :].view(torch.float8_e8m0fnu)}


def _unpacked(s, page, slot):
    """K and V [..., nkv, 2, d] at these pages and slots, in 32 bits."""
    x = s.pool[page, :, :, :, slot]
    if s.case["kv"] == "bf16":
        return x.float()
    return torch.ldexp(x[..., :s.d].contiguous().view(torch.float8_e4m3fn).float(), x[..., s.d:].int() - 127)


def _plain_attend(s):
    nq, nkv, d = s.nq, s.nkv, s.d
    keys = torch.arange(s.longest, device="cuda")
    total = (s.cached + s.new).unsqueeze(1)
    page = torch.where(keys < total, s.table[:, keys // PAGE], 0)
    kv = _unpacked(s, page, (keys % PAGE).expand_as(page))                       # [batch, keys, nkv, 2, d]
    k, v = kv[..., 0, :].permute(0, 2, 3, 1), kv[..., 1, :].transpose(1, 2)
    q = torch.zeros(len(s.new), s.most, nq, d, device="cuda")
    q[s.req, s.place] = s.q.float()
    q = q.view(len(s.new), s.most, nkv, nq // nkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    at = (s.cached.unsqueeze(1) + torch.arange(s.most, device="cuda")).repeat(1, nq // nkv)
    seen = keys <= at.unsqueeze(-1)                                              # [batch, heads of a group x rows, keys]
    x = (q @ k).div_(math.sqrt(d)).masked_fill_(~seen.unsqueeze(1), -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = (x @ v) / x.sum(-1, keepdim=True)
    o = o.view(len(s.new), nkv, nq // nkv, s.most, d).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return o[s.req, s.place].to(torch.bfloat16)


def _rotated(x, pos, theta):
    """Rotary embedding of rows [rows, ..., d] at their positions, angles in 64 bits."""
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = (pos.double().unsqueeze(1) * freq).view(-1, *[1] * (x.dim() - 2), half)
    c, s = angle.cos().to(x.dtype), angle.sin().to(x.dtype)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_append(s):
    x = s.qkv.float()
    q = _rotated(x[:, :, :-2], s.pos, THETA).flatten(1, 2).to(torch.bfloat16)
    kv = torch.stack([_rotated(x[:, :, -2], s.pos, THETA), x[:, :, -1]], 2)      # [rows, nkv, 2, d]
    page, slot = s.table[s.req, s.pos // PAGE], s.pos % PAGE
    if s.case["kv"] == "bf16":
        s.pool[page, :, :, :, slot] = kv.to(torch.bfloat16)
    else:
        codes, exps = _quantised(kv)
        s.pool[page, :, :, :, slot] = torch.cat([codes, exps.unsqueeze(-1)], -1)
    return q


def _plain_read(s):
    total = s.cached + s.new
    req = torch.repeat_interleave(torch.arange(len(total), device="cuda"), total)
    at = torch.arange(req.numel(), device="cuda") - (total.cumsum(0) - total)[req]
    return _unpacked(s, s.table[req, at // PAGE], at % PAGE).to(torch.bfloat16)


def _plain_verify(s):
    b, k, v = s.case["batch"], s.case["drafts"], s.case["vocab"]
    each, step = torch.arange(b, device="cuda"), torch.arange(k, device="cuda")
    drafts = s.drafts.long()
    p = s.p[:, :k].gather(2, drafts.unsqueeze(2)).squeeze(2).double()
    q = s.q.gather(2, drafts.unsqueeze(2)).squeeze(2).double() if s.q is not None else torch.ones_like(p)
    taken = (s.u.double() * q < p) & (step < s.count.unsqueeze(1))
    n = taken.int().cumprod(1).sum(1)
    row, stop = s.p[each, n], n.clamp(max=k - 1)
    if s.q is not None:
        less = s.q[each, stop]
    else:
        less = torch.zeros_like(row).scatter_(1, drafts[each, stop].unsqueeze(1), 1.0)
    left = torch.where((n < s.count).unsqueeze(1), (row - less).clamp(min=0), row)
    mass = torch.ldexp(left.clamp(max=1).double(), torch.tensor(40, device="cuda")).round().long()
    whole = torch.ldexp(row.clamp(max=1).double(), torch.tensor(40, device="cuda")).round().long()
    mass = torch.where(mass.sum(1, keepdim=True) > 0, mass, whole)
    upto = mass.cumsum(1)
    total, u = upto[:, -1:], (s.r.double() * 2 ** 24).long().unsqueeze(1)
    at = (total >> 24) * u + (((total & (2 ** 24 - 1)) * u) >> 24)
    token = torch.where(total.squeeze(1) > 0, (upto <= at).sum(1), -1)
    spot = torch.arange(k + 1, device="cuda")
    out = torch.where(spot < n.unsqueeze(1), torch.nn.functional.pad(drafts, (0, 1)), -1)
    return {"tokens": torch.where(spot == n.unsqueeze(1), token.unsqueeze(1), out).int(), "accepted": n.int()}


def _plain_probs(s):
    x = (s.logits - s.logits.amax(-1, keepdim=True)) / s.case["temperature"]
    x = x.exp()
    return x / x.sum(-1, keepdim=True)


def run(s):
    op = s.case["op"]
    if own:
        from persistent_moe_decode_02_gb300 import mk
        if op == "attend":
            s.chunk.attend(s.q, s.pool, s.out)
            return s.out
        if op == "append":
            s.chunk.append(s.qkv, s.pool, s.q)
            return {"q": s.q, **_pool_parts(s)}
        if op == "read":
            s.chunk.read(s.pool, s.out)
            return s.out
        if op == "probs":
            mk.probs(s.logits, s.case["temperature"], s.out)
            return s.out
        mk.verify(s.p, s.q, s.drafts, s.u, s.r, s.tokens, s.accepted, s.count)
        return {"tokens": s.tokens, "accepted": s.accepted}
    if op == "attend":
        return _plain_attend(s)
    if op == "append":
        return {"q": _plain_append(s), **_pool_parts(s)}
    if op == "read":
        return _plain_read(s)
    return _plain_probs(s) if op == "probs" else _plain_verify(s)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None    # whole numbers
    s = prepare(case, seed)
    if op == "probs":
        w = torch.exp((s.logits.double() - s.logits.double().amax(1, keepdim=True)) / case["temperature"])
        return w / w.sum(1, keepdim=True)
    nq, nkv, d, cached, new = _sizes(case)
    g, rows, first = nq // nkv, [], 0
    if op == "append":
        pos = torch.cat([torch.arange(c, c + n, device="cuda") for c, n in zip(cached, new)]).double()
        x = s.qkv.double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           pos[:, None] * THETA ** (-2.0 * torch.arange(d // 2, device="cuda").double() / d))
        z = torch.complex(x[:, :, :g + 1, :d // 2].contiguous(), x[:, :, :g + 1, d // 2:].contiguous()) * turn[:, None, None]
        z = torch.cat([z.real, z.imag], -1)
        kv = torch.stack([z[:, :, g], x[:, :, g + 1]], 2)
        page = torch.cat([s.table[b, torch.arange(c, c + n, device="cuda") // PAGE] for b, (c, n) in enumerate(zip(cached, new))])
        slot = pos.long() % PAGE
        q = z[:, :, :g].reshape(-1, nq, d)
        if case["kv"] == "bf16":
            pool = s.pool.double()
            pool[page, :, :, :, slot] = kv
            return {"q": q, "pool": pool}
        top = kv.abs().amax(-1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(top / 448) - 1e-12))
        codes = s.pool[..., :d, :].view(torch.float8_e4m3fn).double()
        scales = torch.exp2(s.pool[..., d, :].double() - 127)
        codes[page, :, :, :, slot] = kv / scale
        scales[page, :, :, slot] = scale.squeeze(-1)
        return {"q": q, "codes": codes, "scales": scales}
    for b, (c, n) in enumerate(zip(cached, new)):
        x = s.pool[s.table[b, :-(-(c + n) // PAGE)].long()].double()             # [pages, nkv, 2, d, 16]
        if case["kv"] == "e4m3":
            codes = s.pool[s.table[b, :-(-(c + n) // PAGE)].long()]
            x = codes[..., :d, :].contiguous().view(torch.float8_e4m3fn).double() * torch.exp2(codes[..., d:, :].double() - 127)
        kv = x.permute(0, 4, 1, 2, 3).reshape(-1, nkv, 2, d)[:c + n]
        if op == "read":
            rows.append(kv)
            continue
        out = torch.empty(n, nq, d, dtype=torch.float64, device="cuda")
        for h in range(nq):
            for i in range(0, n, 1024):
                m = min(n, i + 1024)
                w = s.q[first + i:first + m, h].double() @ kv[:c + m, h // g, 0].T / math.sqrt(d)
                hidden = torch.arange(c + m, device="cuda")[None] > torch.arange(c + i, c + m, device="cuda")[:, None]
                w = torch.softmax(w.masked_fill(hidden, -math.inf), 1)
                out[i:m, h] = w @ kv[:c + m, h // g, 1]
        rows.append(out)
        first += n
    return torch.cat(rows)
