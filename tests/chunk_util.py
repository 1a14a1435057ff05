"""64-bit CPU forms of the chunk operators, written from their definitions in
include/mk.h, and the inputs that their tests share."""
import math
from types import SimpleNamespace

import numpy as np
import torch

PAGE = 16
BF16 = torch.finfo(torch.bfloat16).eps / 2     # a rounding to bf16, relative
E4M3_STEP, E4M3_MIN = 2.0 ** -4, 2.0 ** -10    # a rounding to e4m3: relative, and absolute below its normal numbers


def dims(nq, nkv, d, theta=1e4):
    return SimpleNamespace(n_q_heads=nq, n_kv_heads=nkv, head_dim=d, page_size=PAGE, rope_theta=theta)


class Batch:
    """Lengths and a shuffled page table in a pool with pages to spare."""

    def __init__(self, cached, new, seed=0, spare=3, wider=0):
        self.cached, self.new = list(cached), list(new)
        self.total = [c + n for c, n in zip(cached, new)]
        per = [-(-t // PAGE) for t in self.total]
        self.num_pages, self.width = sum(per) + spare, max(max(per), 1) + wider
        order = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed + 77)).tolist()
        self.table, at = [], 0
        for n in per:
            self.table.append(order[at:at + n] + [-1] * (self.width - n))
            at += n
        self.flat = [p for row in self.table for p in row]
        self.rows = sum(new)

    def slots(self, b, begin, end):
        pos = torch.arange(begin, end)
        return torch.tensor(self.table[b], dtype=torch.int64)[pos // PAGE], pos % PAGE

    def new_slots(self):
        s = [self.slots(b, c, t) for b, (c, t) in enumerate(zip(self.cached, self.total)) if t > c]
        return torch.cat([x[0] for x in s]), torch.cat([x[1] for x in s])

    def positions(self):
        return torch.cat([torch.arange(c, t) for c, t in zip(self.cached, self.total)])


def normal(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def quantise(x):
    """Codes (uint8) and k of the last axis, as mk.h says."""
    m, e = torch.frexp(x.float().abs().amax(-1))
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(m == 0, torch.full_like(k, -127), k).clamp(-127, 127)
    code = torch.ldexp(x.double(), -k.unsqueeze(-1).double()).float().to(torch.float8_e4m3fn)
    return code.view(torch.uint8), k


def make_pool(kv, pages, nkv, d, seed):
    if kv == "bf16":
        return normal((pages, nkv, 2, d, PAGE), seed).bfloat16()
    code, k = quantise(normal((pages, nkv, 2, PAGE, d), seed))
    return torch.cat([code.transpose(-1, -2), (k + 127).to(torch.uint8).unsqueeze(-2)], -2).contiguous()


def values(pool, kv):
    """What a pool (CPU) stands for, in 64 bits."""
    if kv == "bf16":
        return pool.double()
    code = pool[..., :-1, :].contiguous().view(torch.float8_e4m3fn).double()
    return torch.ldexp(code, pool[..., -1:, :].double() - 127)


def rows_of(pool, kv, batch, b):
    """K and V [total, nkv, 2, d] of request b in 64 bits."""
    page, slot = batch.slots(b, 0, batch.total[b])
    return values(pool[page.unique()], kv)[torch.searchsorted(page.unique(), page), :, :, :, slot]


def attend(q, pool, kv, batch, nkv):
    """(result, sum of p |v|) in 64 bits."""
    out, mag, first = [], [], 0
    nq, d = q.shape[1:]
    for b, (c, n) in enumerate(zip(batch.cached, batch.new)):
        if not n:
            continue
        x = rows_of(pool, kv, batch, b)
        k = x[:, :, 0].repeat_interleave(nq // nkv, 1).transpose(0, 1)
        v = x[:, :, 1].repeat_interleave(nq // nkv, 1).transpose(0, 1)
        qq = q[first:first + n].double().transpose(0, 1)
        s = qq @ k.transpose(1, 2) / math.sqrt(d)
        s.masked_fill_(torch.arange(c + n) > torch.arange(c, c + n).unsqueeze(1), -math.inf)
        p = torch.softmax(s, -1)
        out.append((p @ v).transpose(0, 1))
        mag.append((p @ v.abs()).transpose(0, 1))
        first += n
    return torch.cat(out), torch.cat(mag)


def attend_bound(ref, mag):
    """The result is rounded to bf16 once, and each weight before it meets its value: half a step of bf16 of
    the result, and of the sum of the weights' magnitudes.  fp32 scores and sums add less than 2^-13 of that
    sum (scores of a few units, off by 128 products' roundings at most)."""
    return BF16 * ref.abs() + (BF16 + 2.0 ** -13) * mag + 1e-30


def rotate(x, pos, theta):
    if theta == 0:
        return x.double()
    half = x.shape[-1] // 2
    a = (pos.double().unsqueeze(1) * theta ** (-torch.arange(half).double() / half)).view(-1, *[1] * (x.dim() - 2), half)
    lo, hi = x.double()[..., :half], x.double()[..., half:]
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def mass(w):
    w = np.asarray(w, dtype=np.float32).astype(np.float64)
    w = np.where(w > 0, np.minimum(w, 1.0), 0.0)      # a NaN compares false
    return np.rint(w * 2.0 ** 40).astype(object)


def verify(target, draft, drafts, u, r, count=None):
    """tokens, accepted from Python integers."""
    t = target.numpy()
    b, k1, vocab = t.shape
    k = k1 - 1
    tokens, accepted = np.full((b, k1), -1, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        n = k if count is None else min(max(int(count[i]), 0), k)
        a = 0
        while a < n:
            x = int(drafts[i, a])
            if not 0 <= x < vocab:
                break
            q = 1.0 if draft is None else float(draft[i, a, x])
            if not float(u[i, a]) * q < float(t[i, a, x]):
                break
            tokens[i, a] = x
            a += 1
        accepted[i] = a
        row = t[i, a]
        m = mass(row)
        if a < n:
            less = np.zeros(vocab, np.float32)
            if draft is not None:
                less = draft[i, a].numpy()
            elif 0 <= int(drafts[i, a]) < vocab:
                less[int(drafts[i, a])] = 1
            left = mass(row - less)
            if left.sum() > 0:
                m = left
        total = int(m.sum())
        if total:
            rv = float(r[i])
            step = min(int(math.floor(rv * 2 ** 24)), 2 ** 24 - 1) if rv > 0 else 0
            tokens[i, a] = int(np.argmax(np.cumsum(m) > total * step // 2 ** 24))
    return tokens, accepted
