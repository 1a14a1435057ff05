"""More of the mixture-of-experts operators on a GPU against 64-bit CPU forms:
gates where SiLU saturates, 8-bit results without a NaN."""
import math

import pytest
import torch

from tests import moe_util as mu
from tests import test_moe_ops as T

pytestmark = pytest.mark.gpu
BF16, F32, U8, E4M3 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mk(built):
    from persistent_moe_decode_02_gb300 import mk
    return mk


# ---- gates of any size ----

def saturating(kind, rows, ffn):
    """One expert whose products are single numbers (a row of x is 1, 0, 0, ...), so h is silu(g) u of known g and u:
    gates from -104 to 104, ups around 1 and, for every other group of 32, around 2^90."""
    c = T.Case(kind, (64, 1, 1, ffn), torch.zeros(rows, 1, dtype=torch.int32), 3)
    x, w = torch.zeros(rows, 64), torch.zeros(1, 2 * ffn, 64)
    x[:, 0] = 1
    w[0, 0::2, 0] = torch.linspace(-104, 104, ffn)
    u = mu.normal((ffn,), 4)
    u.view(-1, 32)[1::2] *= 2.0 ** 90
    w[0, 1::2, 0] = u
    if kind == "bf16":
        c.x, c.gu = (x.bfloat16(), None), (w.bfloat16(), None)
        c.vx, c.vgu = c.x[0].double(), c.gu[0].double()
    else:
        c.x, c.gu = mu.quantise(x), mu.quantise(w)
        c.vx, c.vgu = mu.values(*c.x), mu.values(*c.gu)
    return c


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_gates_of_any_size(mk, kind, rows):
    ffn = 4160
    c = saturating(kind, rows, ffn)
    g, u = c.vgu[0, 0::2, 0], c.vgu[0, 1::2, 0]
    ref = (g * torch.sigmoid(g) * u).expand(rows, -1)
    # fp32: the exponential's root is off by 4 F32 (2 units in the last place) and by its argument's |g| / 2 times 1.5 F32
    # (a rounded constant, a product), the exponential by twice that (8 and 1.5 |g|), the sum by 1, its reciprocal by 2,
    # four products by 4: 15 and 1.5 |g|; below the normal numbers by 2^-149
    slack = (15 + 1.5 * g.abs()) * 1.01 * mu.F32 * ref.abs() + 2.0 ** -149
    (x, xs), (w, ws) = T.cuda(c.x), T.cuda(c.gu)
    h = torch.empty(rows, ffn, dtype=BF16 if kind == "bf16" else E4M3, device="cuda")
    s = torch.empty(rows, ffn // 32, dtype=U8, device="cuda") if kind == "e4m3" else None
    m = c.experts_of(mk)
    m.up(x, w, c.first.cuda(), c.order.cuda(), h, x_scales=xs, w_scales=ws, h_scales=s)
    assert m.sync() == mk.MK_OK
    assert not h.float().isnan().any()
    if kind == "bf16":
        # (bf16 itself is off by 2^-134 below its normal numbers)
        err = (h.cpu().double() - ref).abs()
        bad = ~(err <= mu.BF16 * ref.abs() + 1.01 * slack + 2.0 ** -134)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), g[bad[0]][:5].tolist())
    else:
        mu.check_eights_strictly(h.cpu(), s.cpu(), ref, slack)


@pytest.mark.parametrize("rows", [2600])
def test_gates_of_any_size_in_two_sms(mk, rows):
    ffn = 4160
    c = saturating("bf16", rows, ffn)
    g, u = c.vgu[0, 0::2, 0], c.vgu[0, 1::2, 0]
    ref = g * torch.sigmoid(g) * u
    slack = (15 + 1.5 * g.abs()) * 1.01 * mu.F32 * ref.abs() + 2.0 ** -149
    h = torch.empty(rows, ffn, dtype=BF16, device="cuda")
    m = c.experts_of(mk)
    m.up(c.x[0].cuda(), c.gu[0].cuda(), c.first.cuda(), c.order.cuda(), h)
    assert m.sync() == mk.MK_OK and torch.equal(h, h[:1].expand(rows, -1))
    err = (h[0].cpu().double() - ref).abs()
    bad = ~(err <= mu.BF16 * ref.abs() + 1.01 * slack + 2.0 ** -134)
    assert not bad.any(), (int(bad.sum()), g[bad][:5].tolist())


# ---- 8-bit results hold no NaN ----

@pytest.fixture
def strict(monkeypatch):
    """The tests of 8-bit results with the check that a NaN does not pass."""
    monkeypatch.setattr(mu, "check_eights", _strictly(mu.check_eights))


def _strictly(check):
    def both(codes, scales, ref, slack):
        v = mu.values(codes, scales)
        assert torch.isfinite(v).all(), (~torch.isfinite(v)).nonzero()[:5].tolist()
        check(codes, scales, ref, slack)
    return both


@pytest.mark.parametrize("case", [c for c in T.NORM if c[5] is E4M3], ids=str)
def test_norm_to_8_bits(mk, strict, case):
    T.test_norm(mk, *case)


@pytest.mark.parametrize("name,rows", T.ROWS)
def test_up_in_8_bits(mk, strict, name, rows):
    T.check_up(mk, T.Case("e4m3", T.DIMS[name], T.routed(T.DIMS[name], rows), rows))


@pytest.mark.parametrize("rows", [1, 3, 37, 150])
def test_up_in_8_bits_full_size(mk, strict, rows):
    D = (2048, 12, 8, 768)
    T.check_up(mk, T.Case("e4m3", D, T.routed(D, rows), rows))


@pytest.mark.parametrize("name,rows", [("odd", 77), ("odd", 600), ("odd", 601), ("tail", 300)])
def test_up_in_8_bits_between_alignments(mk, strict, name, rows):
    # a scale that is none (255) lies right behind the last one, and right before the first
    T.test_products_between_alignments(mk, name, rows, "e4m3")


@pytest.mark.parametrize("before,behind", [(1, 2), (3, 1), (2, 3), (0, 1)])
@pytest.mark.parametrize("hidden", [32, 96, 160, 1056])
@pytest.mark.parametrize("rows", [1, 5, 130])
def test_scales_beside_others_that_are_none(mk, strict, before, behind, hidden, rows):
    # bytes of 255 (a NaN as a scale) on both sides of every buffer of scales, in the words that its ends share
    c = T.Case("e4m3", (hidden, 3, 1, 96), T.routed((hidden, 3, 1, 96), rows), 61)

    def among(t):
        whole = torch.full((4 + before + t.numel() + behind + 4,), 255, dtype=U8, device="cuda")
        part = whole[4 + before:4 + before + t.numel()].view(t.shape)
        part.copy_(t.cuda())
        return part

    (x, w, hh, d), (xs, ws, hs, ds) = ([p[i].cuda() if i == 0 else among(p[i]) for p in (c.x, c.gu, c.h, c.dn)] for i in (0, 1))
    m = c.experts_of(mk)
    first, order, gates = c.first.cuda(), c.order.cuda(), c.gates.cuda()
    h, s = torch.empty(c.pairs, c.ffn, dtype=E4M3, device="cuda"), among(torch.zeros(c.pairs, c.ffn // 32, dtype=U8))
    y = torch.empty(c.rows, 1, c.hidden, dtype=BF16, device="cuda")
    m.up(x, w, first, order, h, x_scales=xs, w_scales=ws, h_scales=s)
    m.down(hh, d, first, order, gates, y, h_scales=hs, w_scales=ds)
    assert m.sync() == mk.MK_OK
    mu.check_eights(h.cpu(), s.cpu(), *mu.up(c.vx, c.vgu, c.first, c.order, 1))
    mu.within(y.cpu().flatten(0, 1), *mu.down(c.vh, c.vdn, c.first, c.order, c.gates))


# ---- lists of tiles ----

def tiles_a_block(D, first, up, sms, group):
    """The largest number of tiles that a block gets of the products with tiles of 32 rows and up to 192 columns: the
    rule of set_width (the width with the fewest rounds times columns and 32 beside them, the widest of equal ones)."""
    hidden, experts, _, ffn = D
    n = 2 * ffn if up else hidden
    rows = (first[1:] - first[:-1]).tolist()
    row_tiles = sum((r + 31) // 32 for r in rows)
    cost = {w: -(-row_tiles * -(-n // w) // sms) * (w + 32) for w in range(group, 193, group)}
    width = max(w for w in cost if cost[w] == min(cost.values()))
    return -(-row_tiles * -(-n // width) // sms)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("up", [True, False])
def test_lists_of_several_parts(mk, strict, kind, up):
    # a block's list is planned 32 tiles at a time, in two places in turn: more than 96 tiles use each place twice, so the
    # planning warp waits for its readers
    D = (32, 256, 8, 5120) if up else (10240, 256, 8, 32)
    c = T.Case(kind, D, T.routed(D, 512), 71)
    assert 32 < c.pairs <= 16 * c.experts           # tiles of 32 rows
    group = {(True, "bf16"): 16, (True, "e4m3"): 64, (False, "bf16"): 64, (False, "e4m3"): 16}[up, kind]
    assert tiles_a_block(D, c.first, up, torch.cuda.get_device_properties(0).multi_processor_count, group) > 96
    (T.check_up if up else T.check_down)(mk, c)


@pytest.mark.parametrize("up", [True, False])
def test_lists_of_several_parts_in_two_sms(mk, up):
    D = (64, 2, 1, 16384) if up else (32768, 2, 1, 64)
    rows = 16000
    c = T.Case("bf16", D, torch.randint(0, 2, (rows, 1), generator=torch.Generator().manual_seed(2)).int(), 72)
    n, sms = 32768, torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(-(-int(r) // 256) for r in c.first[1:] - c.first[:-1]) * (n // 256) > 96 * (sms // 2)
    m = c.experts_of(mk)
    some = torch.arange(3, rows, 397)               # pairs, in the sorted order
    one = torch.stack([torch.zeros(()), (some < c.first[1]).sum(), torch.tensor(len(some))]).int()
    if up:
        w_h, h = T.cuda_empty((rows, c.ffn), BF16)
        m.up(c.x[0].cuda(), c.gu[0].cuda(), c.first.cuda(), c.order.cuda(), h)
        got, (ref, slack) = h[some.cuda()], mu.up(c.vx[c.order[some].long()], c.vgu, one, torch.arange(len(some)), 1)
    else:
        w_h, y = T.cuda_empty((rows, 1, c.hidden), BF16)
        m.down(c.h[0].cuda(), c.dn[0].cuda(), c.first.cuda(), c.order.cuda(), c.gates.cuda(), y)
        at = c.order[some].long()
        got = y[at.cuda(), 0]
        ref, slack = mu.down(c.vh[some], c.vdn, one, torch.arange(len(some)), c.gates[at])
    assert m.sync() == mk.MK_OK and T.behind(w_h)
    mu.within(got.cpu(), ref, slack)
