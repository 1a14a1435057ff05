"""The mixture-of-experts operators over chunks (mk_norm, mk_quantize, mk_route,
mk_experts_*) on a GPU against 64-bit CPU forms, at the sizes and masks where
they can go wrong, and run together as a model uses them."""
import math

import pytest
import torch

import synth
from synth.device import DeviceModel, kv_pages_needed
from tests import moe_util as mu

pytestmark = pytest.mark.gpu

BF16, F32, U8, E4M3 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mk(built):
    from persistent_moe_decode_02_gb300 import mk
    return mk


def cuda_empty(shape, dtype):
    """A result's buffer with a row more, which has to stay as it is; (whole, the result's part)."""
    whole = torch.full((shape[0] + 1, *shape[1:]), 7.0, device="cuda").to(dtype)
    return whole, whole[:-1]


def behind(whole):
    return (whole[-1].float().cpu() == 7).all()


# ---- norm ----

NORM = [  # rows, n, x, add, terms, out
    (1, 2048, F32, BF16, 8, BF16), (37, 2048, F32, BF16, 1, E4M3), (5, 2048, BF16, None, 0, BF16), (300, 2048, F32, F32, 3, F32),
    (3, 8, F32, BF16, 1, BF16), (9, 32, BF16, BF16, 2, E4M3), (17, 264, F32, BF16, 5, BF16), (4, 4104, BF16, F32, 1, F32),
    (2, 16384, F32, BF16, 8, E4M3), (3, 8224, F32, None, 0, E4M3), (1000, 96, BF16, BF16, 9, E4M3), (33, 1056, F32, BF16, 3, E4M3),
    (6, 6144, BF16, BF16, 4, BF16), (2, 5000, F32, F32, 2, BF16),
]


@pytest.mark.parametrize("rows,n,xt,at,terms,ot", NORM)
def test_norm(mk, rows, n, xt, at, terms, ot):
    wide = mu.normal((rows, n + 16), n, 2.0).to(xt)            # rows lie apart
    wide[0, :n] *= 1e-3
    x = wide[:, :n]
    add = mu.normal((rows, terms, n), n + 1, 0.5).to(at) if terms else None
    gamma = (1 + mu.normal((n,), n + 2, 0.1)).bfloat16()
    eps = 1e-6
    t, ref, dt, slack = mu.norm(x, add, gamma, eps)
    w_total, total = cuda_empty((rows, n), xt)
    w_out, out = cuda_empty((rows, n), ot)
    w_s, s = cuda_empty((rows, n // 32), U8)
    mk.norm(wide.cuda()[:, :n], gamma.cuda(), eps, out, add=None if add is None else add.cuda(), total=total,
            scales=s if ot is E4M3 else None)
    mu.within(total.cpu(), t, dt, mu.BF16 if xt is BF16 else mu.F32)
    if ot is E4M3:
        mu.check_eights(out.cpu(), s.cpu(), ref, slack)
        assert behind(w_s)
    else:
        mu.within(out.cpu(), ref, slack, mu.BF16 if ot is BF16 else mu.F32)
    assert behind(w_total) and behind(w_out)


def test_norm_in_place_and_sum_alone(mk):
    x, add = mu.normal((70, 512), 1), mu.normal((70, 512), 2).bfloat16()
    g = x.cuda()
    out = torch.empty(70, 512, device="cuda")
    mk.norm(g, None, 0.0, out, add=add.cuda(), total=g)
    t, ref, dt, slack = mu.norm(x, add.unsqueeze(1), None, 0.0)
    mu.within(g.cpu(), t, dt, mu.F32)
    mu.within(out.cpu(), ref, slack, mu.F32)
    mk.norm(g, None, 0.0, None, add=add.cuda(), total=g)       # the sum alone, onto itself
    assert torch.equal(g.cpu(), x + add.float() + add.float())


def test_norm_special_rows(mk):
    # a row of zeros is zeros; a NaN or an infinity stays in its row
    x = mu.normal((5, 64), 3)
    x[1], x[2, 5], x[3, 7] = 0, math.nan, math.inf
    out, s = torch.empty(5, 64, dtype=E4M3, device="cuda"), torch.empty(5, 2, dtype=U8, device="cuda")
    mk.norm(x.cuda(), None, 1e-6, out, scales=s)
    o = out.cpu().float()
    assert (o[1] == 0).all() and (s.cpu()[1] == 0).all() and o[2].isnan().all()
    plain = torch.empty(5, 64, device="cuda")
    mk.norm(x.cuda(), None, 1e-6, plain)
    p = plain.cpu()
    assert (p[1] == 0).all() and p[2].isnan().all() and p[3, 7].isnan() and (p[3, :7] == 0).all()
    _, ref, _, slack = mu.norm(x[[0, 4]], None, None, 1e-6)
    mu.within(p[[0, 4]], ref, slack, mu.F32)


# ---- quantize ----

@pytest.mark.parametrize("rows,n", [(1, 32), (3, 96), (37, 2048), (513, 4096), (1000, 64), (2, 20000)])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_quantize(mk, rows, n, xt):
    wide = (mu.normal((rows, n + 8), rows + n) * torch.exp(4 * mu.normal((rows, n + 8), n))).to(xt)
    x = wide[:, :n]
    x[0, :32] = 0
    if rows > 2:
        x[1, :32] = torch.tensor([448 * 2.0 ** -6] * 16 + [-447 * 2.0 ** -6] * 16)   # the largest code, and next to it
        x[2, :32] = torch.linspace(449, 460, 32)                                      # just above it
    codes, scales = mu.quantise(x)
    w_c, c = cuda_empty((rows, n), E4M3)
    w_s, s = cuda_empty((rows, n // 32), U8)
    mk.quantize(wide.cuda()[:, :n], c, s)
    assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu().view(U8), codes.view(U8))
    assert behind(w_c) and behind(w_s)


def test_quantize_extremes(mk):
    x = mu.normal((8, 32), 4)
    x[0, 3], x[1, 4], x[2] = math.nan, math.inf, 1e-44
    x[3] *= 2.0 ** 126
    x[4] *= 2.0 ** -126
    x[5, 1:] = 0
    x[6] = math.nan
    x[7] *= 1e-30
    x[7, 0] = 3e38
    c, s = torch.empty(8, 32, dtype=E4M3, device="cuda"), torch.empty(8, 1, dtype=U8, device="cuda")
    mk.quantize(x.cuda(), c, s)
    codes, scales = mu.quantise(x)
    assert torch.equal(s.cpu(), scales), (s.cpu().flatten(), scales.flatten())
    got, want = c.cpu().float(), codes.float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


# ---- route ----

def check_route(mk, logits, k, wide=None):
    rows, experts = logits.shape
    ids, gates, first, order = mu.route(logits, k)
    g_ids, g_gates = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")
    w_first, g_first = cuda_empty((experts + 1,), torch.int32)
    w_order, g_order = cuda_empty((rows * k,), torch.int32)
    mk.route((logits if wide is None else wide).cuda()[:, :experts], g_ids, g_gates, g_first, g_order)
    assert torch.equal(g_ids.cpu(), ids)
    assert torch.equal(g_first.cpu(), first)
    assert torch.equal(g_order.cpu(), order)
    assert behind(w_first) and behind(w_order)
    # the difference of two logits is off by half a step, the exponential by 2, its sum by 3, the quotient by 1
    live = ids >= 0
    finite = torch.where(torch.isfinite(logits), logits, torch.zeros(()))
    spread = (finite.amax(1) - finite.amin(1)).clamp(min=0).double().unsqueeze(1)
    got = g_gates.cpu().double()
    assert torch.equal(got.isnan(), gates.isnan())
    assert (got[~live] == 0).all()
    err = (got - gates).abs().nan_to_num(0)
    assert (err <= (16 + 4 * spread) * mu.F32 * gates.nan_to_num(0) + 1e-37).all(), float(err.max())


@pytest.mark.parametrize("rows,experts,k", [(1, 128, 8), (37, 128, 8), (513, 128, 8), (1, 1, 1), (300, 1, 1), (700, 5, 3),
                                            (64, 8, 8), (2000, 33, 4), (100, 64, 8), (129, 256, 8), (1500, 200, 1), (4097, 37, 3),
                                            (8192, 16, 8), (8193, 16, 8), (20011, 9, 2)])
def test_route(mk, rows, experts, k):
    wide = mu.normal((rows, experts + 3), rows + experts, 0.9)
    check_route(mk, wide[:, :experts].contiguous(), k, wide)


def test_route_ties_and_masks(mk):
    x = torch.randint(-2, 3, (900, 64), generator=torch.Generator().manual_seed(5)).float()   # equal logits everywhere
    x[0] = 0
    x[1, ::2] = -0.0                                          # equal to 0
    x[1, 1::2] = 0.0
    check_route(mk, x, 8)
    m = mu.normal((600, 40), 6)
    m[torch.rand(600, 40, generator=torch.Generator().manual_seed(7)) < 0.9] = -math.inf       # rows with fewer than k
    m[3] = -math.inf                                          # none at all
    m[4] = torch.finfo(F32).min                               # masked by the type's lowest value: chosen, alike
    m[5, :39] = torch.finfo(F32).min
    m[6, 2], m[7, 3], m[8] = math.nan, math.inf, math.nan
    check_route(mk, m, 6)
    check_route(mk, m[3:4].contiguous(), 6)
    check_route(mk, torch.full((3, 9), -math.inf), 2)
    x = mu.normal((9000, 12), 8)                              # more than the sort holds at a time
    x[torch.rand(9000, 12, generator=torch.Generator().manual_seed(9)) < 0.8] = -math.inf
    check_route(mk, x, 5)


def test_route_one_expert_for_all(mk):
    x = torch.zeros(3000, 128)
    x[:, 77], x[:, 5] = 9, 8
    check_route(mk, x, 2)


def test_route_nothing(mk):
    e = lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device="cuda")   # noqa: E731
    first = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    mk.route(e(0, 5, t=F32), e(0, 2), e(0, 2, t=F32), first, e(0))
    assert (first.cpu() == 0).all()


# ---- the experts' products ----

DIMS = {"full": (2048, 128, 8, 768), "tiny": (256, 8, 2, 512), "odd": (1056, 37, 3, 352), "small": (32, 3, 2, 32),
        "dense": (1024, 1, 1, 1408), "many": (64, 256, 8, 96), "tail": (288, 4, 1, 160)}
ROWS = [("tiny", 1), ("tiny", 5), ("tiny", 300), ("odd", 1), ("odd", 77), ("odd", 1000), ("small", 1), ("small", 700),
        ("dense", 1), ("dense", 127), ("dense", 129), ("dense", 1000), ("many", 40), ("many", 2000), ("tail", 131), ("tail", 600)]


class Case:
    """Rows, lists and weights of one layer on the CPU; kind bf16 or e4m3.  64-bit values beside them."""

    def __init__(self, kind, D, ids, seed=0):
        self.kind, self.D = kind, D
        self.hidden, self.experts, self.k, self.ffn = D
        self.ids, self.rows = ids, ids.shape[0]
        self.first, self.order = mu.lists(ids, self.experts)
        self.pairs = self.rows * self.k
        x, h = mu.normal((self.rows, self.hidden), seed + 1), mu.normal((self.pairs, self.ffn), seed + 2, 0.5)
        gu = mu.normal((self.experts, 2 * self.ffn, self.hidden), seed + 3, 1.5 / math.sqrt(self.hidden))
        dn = mu.normal((self.experts, self.ffn, self.hidden), seed + 4, 0.05)
        self.gates = torch.softmax(mu.normal((self.rows, self.k), seed + 5), 1)
        if kind == "bf16":
            self.x, self.h, self.gu, self.dn = ((t.bfloat16(), None) for t in (x, h, gu, dn))
            self.vx, self.vh, self.vgu, self.vdn = (t[0].double() for t in (self.x, self.h, self.gu, self.dn))
        else:
            self.x, self.h, self.gu, self.dn = (mu.quantise(t) for t in (x, h, gu, dn.transpose(1, 2).contiguous()))
            self.vx, self.vh, self.vgu = (mu.values(*t) for t in (self.x, self.h, self.gu))
            self.vdn = mu.values(*self.dn).transpose(1, 2)

    def experts_of(self, mk):
        return mk.Experts(mu.dims(*self.D), self.kind)


def cuda(pair):
    return tuple(None if t is None else t.cuda() for t in pair)


def routed(D, rows, seed=11, bias=0.5):
    _, experts, k, _ = D
    logits = mu.normal((rows, experts), seed) + bias * mu.normal((1, experts), seed + 1)
    return logits.topk(k, 1).indices.int()


def check_up(mk, c, m=None):
    m = m or c.experts_of(mk)
    (x, xs), (w, ws) = cuda(c.x), cuda(c.gu)
    w_h, h = cuda_empty((c.pairs, c.ffn), BF16 if c.kind == "bf16" else E4M3)
    w_s, s = cuda_empty((c.pairs, c.ffn // 32), U8) if c.kind == "e4m3" else (None, None)
    m.up(x, w, c.first.cuda(), c.order.cuda(), h, x_scales=xs, w_scales=ws, h_scales=s)
    assert m.sync() == mk.MK_OK
    ref, slack = mu.up(c.vx, c.vgu, c.first, c.order, c.k)
    live = int(c.first[-1])
    if c.kind == "bf16":
        mu.within(h.cpu()[:live], ref[:live], slack[:live])
    else:
        mu.check_eights(h.cpu()[:live], s.cpu()[:live], ref[:live], slack[:live])
        assert behind(w_s) and (s.cpu()[live:] == 7).all()
    assert behind(w_h) and (h.cpu()[live:].float() == 7).all()     # rows of no expert are left as they were


def check_down(mk, c, gates=True, m=None):
    m = m or c.experts_of(mk)
    (h, hs), (w, ws) = cuda(c.h), cuda(c.dn)
    w_y, y = cuda_empty((c.rows, c.k, c.hidden), BF16)
    m.down(h, w, c.first.cuda(), c.order.cuda(), c.gates.cuda() if gates else None, y, h_scales=hs, w_scales=ws)
    assert m.sync() == mk.MK_OK
    ref, slack = mu.down(c.vh, c.vdn, c.first, c.order, c.gates if gates else None)
    mu.within(y.cpu().flatten(0, 1), ref, slack)
    assert behind(w_y)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("name,rows", ROWS)
def test_products(mk, name, rows, kind):
    c = Case(kind, DIMS[name], routed(DIMS[name], rows), rows)
    check_up(mk, c)
    check_down(mk, c, gates=rows % 2 == 1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 3, 37, 150])
def test_products_full_size(mk, kind, rows):
    # few enough experts for a 64-bit product on the CPU, all of the full model's widths
    D = (2048, 12, 8, 768)
    c = Case(kind, D, routed(D, rows), rows)
    check_up(mk, c)
    check_down(mk, c)


@pytest.mark.parametrize("kind,D", [("bf16", (8, 1, 1, 8)), ("bf16", (16, 2, 2, 8)), ("bf16", (8, 256, 8, 16)), ("e4m3", (32, 1, 1, 32)),
                                    ("bf16", (32768, 2, 1, 32)), ("e4m3", (32768, 2, 1, 32)), ("bf16", (32, 2, 1, 32768)),
                                    ("e4m3", (32, 2, 1, 32768))])
@pytest.mark.parametrize("rows", [1, 9, 300])
def test_products_of_the_smallest_and_widest(mk, kind, D, rows):
    c = Case(kind, D, routed(D, rows), rows + 40)
    check_up(mk, c)
    check_down(mk, c)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_products_of_many_tiles(mk, kind):
    # more than 64 tiles a block: the list of tiles is planned piece by piece, the rings turn over many times
    c = Case(kind, (32, 256, 8, 2560), routed((32, 256, 8, 2560), 512), 21)
    check_up(mk, c)
    c = Case(kind, (5120, 256, 8, 32), routed((5120, 256, 8, 32), 512), 22)
    check_down(mk, c)


TWO = [(2200, [1, 1, 1, 1]), (2311, [5, 0, 1, 3]), (2500, [0, 0, 1, 0]), (2250, [70, 1, 0, 30])]


@pytest.mark.parametrize("rows,weights", TWO)
@pytest.mark.parametrize("lost", [False, True])
def test_products_of_two_sms(mk, rows, weights, lost):
    # enough rows an expert and columns for tiles of two SMs: even, uneven, all with one expert, pairs without one
    g = torch.Generator().manual_seed(rows)
    ids = torch.multinomial(torch.tensor(weights).float(), rows * 2, replacement=True, generator=g).int().view(rows, 2)
    if lost:
        ids[torch.rand(rows, 2, generator=g) < 0.02] = -1
    check_up(mk, Case("bf16", (72, 4, 2, 2040), ids, 31))
    check_down(mk, Case("bf16", (4088, 4, 2, 72), ids, 32), gates=not lost)


def test_products_of_two_sms_special(mk):
    # a NaN stays with its rows; lists that hold anything read and write nothing outside
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(0, 4, (2300, 2), generator=g).int()
    c = Case("bf16", (64, 4, 2, 2048), ids, 33)
    c.x[0][7] = math.nan
    m = c.experts_of(mk)
    x, w, first, order = c.x[0].cuda(), c.gu[0].cuda(), c.first.cuda(), c.order.cuda()
    w_h, h = cuda_empty((c.pairs, c.ffn), BF16)
    m.up(x, w, first, order, h)
    bad = h.float().isnan().any(1).cpu()
    assert m.sync() == mk.MK_OK and int(bad.sum()) == 2 and bad[(c.order == 14).nonzero()] and bad[(c.order == 15).nonzero()]
    again = h.clone()
    m.up(x, w, first, order, h)
    assert m.sync() == mk.MK_OK and torch.equal(again.view(torch.int16), h.view(torch.int16))   # the same bits
    d = Case("bf16", (4096, 4, 2, 64), ids, 34)
    md, hh, dn = d.experts_of(mk), d.h[0].cuda(), d.dn[0].cuda()
    big = 2 ** 31 - 1
    for first, order in ([[0, 9000, -5, 100, 40], c.order], [[-big, big, big, 0, 300], c.order], [c.first, torch.full((4600,), big)],
                         [c.first, torch.arange(4600) * 7 - 100], [[4000, 4100, 4050, 4600, 4580], c.order]):
        first, order = torch.as_tensor(first).int().cuda(), order.int().cuda()
        w_h, h = cuda_empty((c.pairs, c.ffn), BF16)
        m.up(x, w, first, order, h)
        w_y, y = cuda_empty((d.rows, 2, d.hidden), BF16)
        md.down(hh, dn, first, order, d.gates.cuda(), y)
        assert m.sync() == mk.MK_OK and md.sync() == mk.MK_OK and behind(w_h) and behind(w_y)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("counts", [[0, 128, 0, 0], [127, 0, 1, 129], [0, 0, 0, 513], [256, 255, 257, 1], [16, 17, 15, 4]])
def test_products_tile_borders(mk, kind, counts):
    D = DIMS["tail"]
    ids = torch.cat([torch.full((n,), e) for e, n in enumerate(counts)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(3))].int().unsqueeze(1)
    c = Case(kind, D, ids, 5)
    check_up(mk, c)
    check_down(mk, c)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_products_of_pairs_without_expert(mk, kind):
    D = DIMS["odd"]
    ids = routed(D, 200)
    ids[torch.rand(200, 3, generator=torch.Generator().manual_seed(4)) < 0.4] = -1
    c = Case(kind, D, ids, 6)
    check_up(mk, c)
    check_down(mk, c)
    none = Case(kind, D, torch.full((50, 3), -1, dtype=torch.int32), 7)
    check_up(mk, none)
    check_down(mk, none)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_products_keep_a_nan_to_its_rows(mk, kind):
    # a row's NaN reaches its own pairs alone; weights of an expert without rows reach nobody
    D = DIMS["tail"]
    ids = torch.tensor([0, 1, 3, 1, 0, 3, 3, 1] * 20).int().unsqueeze(1)
    c = Case(kind, D, ids, 8)
    nan = lambda t, at: t.__setitem__(at, torch.full_like(t[at].float(), math.nan).to(t.dtype))   # noqa: E731
    for w in (c.gu[0], c.dn[0]):
        nan(w, 2)
    nan(c.x[0], 7)
    at = (c.order == 7).nonzero().item()
    nan(c.h[0], at)
    m = c.experts_of(mk)
    (x, xs), (w, ws), (h, hs), (d, ds) = cuda(c.x), cuda(c.gu), cuda(c.h), cuda(c.dn)
    first, order = c.first.cuda(), c.order.cuda()
    out = torch.empty(c.pairs, c.ffn, dtype=BF16 if kind == "bf16" else E4M3, device="cuda")
    s = None if kind == "bf16" else torch.empty(c.pairs, c.ffn // 32, dtype=U8, device="cuda")
    m.up(x, w, first, order, out, x_scales=xs, w_scales=ws, h_scales=s)
    y = torch.empty(c.rows, 1, c.hidden, dtype=BF16, device="cuda")
    m.down(h, d, first, order, None, y, h_scales=hs, w_scales=ds)
    assert m.sync() == mk.MK_OK
    bad = out.float().isnan().any(1).cpu()
    assert bad[at] and int(bad.sum()) == 1
    bad = y.float().isnan().any(2).flatten().cpu()
    assert bad[7] and int(bad.sum()) == 1


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_products_of_lists_that_hold_anything(mk, kind):
    # entries out of range or out of order read and write nothing outside the buffers
    D = DIMS["tail"]
    c = Case(kind, D, routed(D, 300), 9)
    m = c.experts_of(mk)
    (x, xs), (w, ws), (h, hs), (d, ds) = cuda(c.x), cuda(c.gu), cuda(c.h), cuda(c.dn)
    big = 2 ** 31 - 1
    for first, order in ([[0, 900, -5, 100, 40], c.order], [[-big, big, big, 0, 300], c.order],
                         [c.first, torch.full((300,), big)], [c.first, torch.full((300,), -1)],
                         [[250, 260, 255, 300, 280], torch.arange(300) * 7 - 100]):
        first = torch.as_tensor(first).int().cuda()
        order = order.int().cuda()
        w_h, out = cuda_empty((c.pairs, c.ffn), BF16 if kind == "bf16" else E4M3)
        s = None if kind == "bf16" else torch.empty(c.pairs, c.ffn // 32, dtype=U8, device="cuda")
        m.up(x, w, first, order, out, x_scales=xs, w_scales=ws, h_scales=s)
        w_y, y = cuda_empty((c.rows, 1, c.hidden), BF16)
        m.down(h, d, first, order, c.gates.cuda(), y, h_scales=hs, w_scales=ds)
        assert m.sync() == mk.MK_OK
        assert behind(w_h) and behind(w_y)


# ---- together ----

class Layer:
    """A layer's expert half as a model runs it: norm, router product, route, up, down, and the sum in the next norm."""

    def __init__(self, mk, kind, D, rows, seed=1):
        self.mk, self.kind, self.D, self.rows = mk, kind, D, rows
        h, e, k, f = D
        self.x, self.attn = mu.normal((rows, h), seed, 2.0), mu.normal((rows, h), seed + 1).bfloat16()
        self.g1, self.g2 = ((1 + mu.normal((h,), seed + i, 0.1)).bfloat16() for i in (2, 3))
        self.router = mu.normal((h, e), seed + 4, 2.0 / math.sqrt(h))
        gu, dn = mu.normal((e, 2 * f, h), seed + 5, 1.5 / math.sqrt(h)), mu.normal((e, f, h), seed + 6, 1.0 / math.sqrt(f))
        if kind == "bf16":
            self.gu, self.dn = (gu.bfloat16(), None), (dn.bfloat16(), None)
            self.vgu, self.vdn = self.gu[0].double(), self.dn[0].double()
        else:
            self.gu, self.dn = mu.quantise(gu), mu.quantise(dn.transpose(1, 2).contiguous())
            self.vgu, self.vdn = mu.values(*self.gu), mu.values(*self.dn).transpose(1, 2)
        c = lambda *s, t=F32: torch.empty(*s, dtype=t, device="cuda")   # noqa: E731
        rt = BF16 if kind == "bf16" else E4M3
        sc = (lambda *s: None) if kind == "bf16" else lambda *s: c(*s, t=U8)   # noqa: E731
        self.total, self.n, self.n_s, self.nf = c(rows, h), c(rows, h, t=rt), sc(rows, h // 32), c(rows, h)
        self.ids, self.gates, self.first, self.order = (c(rows, k, t=torch.int32), c(rows, k), c(e + 1, t=torch.int32),
                                                        c(rows * k, t=torch.int32))
        self.h, self.h_s, self.y = c(rows * k, f, t=rt), sc(rows * k, f // 32), c(rows, k, h, t=BF16)
        self.sum, self.out = c(rows, h), c(rows, h, t=BF16)
        self.w = {n: t.cuda() for n, t in (("x", self.x), ("attn", self.attn), ("g1", self.g1), ("g2", self.g2), ("router", self.router))}
        self.wgu, self.wdn = cuda(self.gu), cuda(self.dn)
        self.experts = mk.Experts(mu.dims(*D), kind)

    def run(self):
        mk, w, m = self.mk, self.w, self.experts
        mk.norm(w["x"], w["g1"], 1e-6, self.n, add=w["attn"], total=self.total, scales=self.n_s)
        mk.norm(self.total, w["g1"], 1e-6, self.nf)
        torch.mm(self.nf, w["router"], out=self.logits) if hasattr(self, "logits") else setattr(self, "logits", self.nf @ w["router"])
        mk.route(self.logits, self.ids, self.gates, self.first, self.order)
        m.up(self.n, self.wgu[0], self.first, self.order, self.h, x_scales=self.n_s, w_scales=self.wgu[1], h_scales=self.h_s)
        m.down(self.h, self.wdn[0], self.first, self.order, self.gates, self.y, h_scales=self.h_s, w_scales=self.wdn[1])
        mk.norm(self.total, w["g2"], 1e-6, self.out, add=self.y, total=self.sum)

    def check(self):
        """Against 64 bits from the kernel's own choice of experts, which must be the best of its logits."""
        assert self.experts.sync() == self.mk.MK_OK
        h, e, k, f = self.D
        ids = self.ids.cpu()
        assert torch.equal(ids, mu.route(self.logits.cpu(), k)[0])
        t = self.x.double() + self.attn.double()
        n = t / torch.sqrt(t.square().mean(1, keepdim=True) + 1e-6) * self.g1.double()
        want = torch.gather(n @ self.router.double(), 1, ids.long())
        gates = torch.softmax(want, 1)
        first, order = mu.lists(ids, e)
        # the rows that the products read are rounded
        step = mu.BF16 if self.kind == "bf16" else mu.E4M3_STEP
        hh, _ = mu.up(n, self.vgu, first, order, k)
        y, _ = mu.down(hh, self.vdn, first, order, gates)
        total = t + y.view(self.rows, k, h).sum(1)
        out = total / torch.sqrt(total.square().mean(1, keepdim=True) + 1e-6) * self.g2.double()
        # rounding n, h and y moves each by up to a step, independently: well within 3 steps of y's norm
        err = (self.sum.cpu().double() - total).norm() / y.view(self.rows, k, h).sum(1).norm()
        assert err < 3 * step, float(err)
        err = (self.out.cpu().double() - out).norm() / out.norm()
        assert err < 3 * step, float(err)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("name,rows", [("tiny", 1), ("tiny", 200), ("odd", 37), ("wide", 600)])
def test_layer(mk, kind, name, rows):
    layer = Layer(mk, kind, {**DIMS, "wide": (4096, 2, 2, 2048)}[name], rows)
    layer.run()
    layer.check()
    first = layer.out.clone()
    for _ in range(5):                              # without a wait in between, the same bits
        layer.run()
    assert layer.experts.sync() == mk.MK_OK and torch.equal(layer.out, first)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_layer_in_a_graph(mk, kind):
    layer = Layer(mk, kind, DIMS["tiny"], 40)
    layer.run()
    torch.cuda.synchronize()
    want = layer.out.clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        layer.run()
    for _ in range(3):
        layer.out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.out, want)
    # other rows in the same buffers: the lists are made anew on the device
    layer.x = mu.normal(layer.x.shape, 99, 2.0)
    layer.w["x"].copy_(layer.x)
    graph.replay()
    layer.check()


def test_layers_on_two_streams(mk):
    a, b = Layer(mk, "bf16", DIMS["odd"], 300), Layer(mk, "e4m3", DIMS["tiny"], 500, seed=50)
    b_shared = Layer(mk, "bf16", DIMS["odd"], 120, seed=90)
    b_shared.experts = a.experts                     # one object, two streams
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, layer in zip(streams, (a, b, b_shared)):
            with torch.cuda.stream(s):
                layer.run()
    torch.cuda.synchronize()
    for layer in (a, b, b_shared):
        layer.check()


def test_layer_beside_a_capture_from_a_new_process(mk):
    # a process's first calls, inside a capture
    import subprocess
    import sys

    code = """
import torch
from persistent_moe_decode_02_gb300 import mk
from tests import test_moe_ops as T
layer = T.Layer(mk, "bf16", T.DIMS["tiny"], 300)
layer.logits = torch.empty(300, 8, device="cuda")
torch.mm(layer.w["x"], layer.w["router"])        # (the library's own first call)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    layer.run()
g.replay()
layer.check()
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_nothing_to_do(mk):
    m = mk.Experts(mu.dims(64, 4, 2, 32), "bf16")
    e = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")   # noqa: E731
    first, order = torch.zeros(5, dtype=torch.int32, device="cuda"), e(0, t=torch.int32)
    m.up(e(0, 64), e(4, 64, 64), first, order, e(0, 32))
    m.down(e(0, 32), e(4, 32, 64), first, order, None, e(0, 2, 64))
    mk.norm(e(0, 64), None, 1e-6, e(0, 64))
    mk.quantize(e(0, 64), e(0, 64, t=E4M3), e(0, 2, t=U8))
    assert m.sync() == mk.MK_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("name,rows", [("odd", 77), ("odd", 600), ("tail", 300)])
def test_products_between_alignments(mk, name, rows, kind):
    # rows and weights 16 bytes past a larger alignment, scales at any byte, and no scale behind the last one
    c = Case(kind, DIMS[name], routed(DIMS[name], rows), 41)
    m = c.experts_of(mk)

    def shifted(t, by):
        if t is None:
            return None
        whole = torch.full((t.numel() + by + 8,), 255 if t.dtype is U8 else 0, device="cuda").to(t.dtype)
        part = whole[by:-8].view(t.shape)
        part.copy_(t.cuda())
        return part

    el = 1 if kind == "e4m3" else 2
    (x, xs), (w, ws), (h, hs), (d, ds) = ((shifted(a, 16 // el), shifted(b, 3)) for a, b in (c.x, c.gu, c.h, c.dn))
    out, s = shifted(torch.zeros(c.pairs, c.ffn).to(BF16 if kind == "bf16" else E4M3), 16 // el), shifted(
        None if kind == "bf16" else torch.zeros(c.pairs, c.ffn // 32, dtype=U8), 5)
    y = shifted(torch.zeros(c.rows, c.k, c.hidden, dtype=BF16), 8)
    first, order, gates = shifted(c.first, 1), shifted(c.order, 1), shifted(c.gates, 1)
    m.up(x, w, first, order, out, x_scales=xs, w_scales=ws, h_scales=s)
    m.down(h, d, first, order, gates, y, h_scales=hs, w_scales=ds)
    assert m.sync() == mk.MK_OK
    ref, slack = mu.up(c.vx, c.vgu, c.first, c.order, c.k)
    if kind == "bf16":
        mu.within(out.cpu(), ref, slack)
    else:
        mu.check_eights(out.cpu(), s.cpu(), ref, slack)
    ref, slack = mu.down(c.vh, c.vdn, c.first, c.order, c.gates)
    mu.within(y.cpu().flatten(0, 1), ref, slack)


def test_rows_beyond_4_gb(mk):
    # the last rows of buffers of more than 4 GB: rows to 8 bits, norm, up and down
    x = torch.zeros(70000, 32768, dtype=BF16, device="cuda")
    some = mu.normal((3, 32768), 1).bfloat16()
    x[-3:] = some.cuda()
    codes, scales = torch.empty(70000, 32768, dtype=E4M3, device="cuda"), torch.empty(70000, 1024, dtype=U8, device="cuda")
    mk.quantize(x, codes, scales)
    want = mu.quantise(some)
    assert torch.equal(codes[-3:].cpu().view(U8), want[0].view(U8)) and torch.equal(scales[-3:].cpu(), want[1])
    del codes, scales
    y = x.view(280000, 8192)
    out = torch.empty_like(y)
    mk.norm(y, None, 1e-6, out)
    _, ref, _, slack = mu.norm(some.view(12, 8192), None, None, 1e-6)
    mu.within(out[-12:].cpu(), ref, slack)
    del x, y, out
    D = (64, 2, 1, 4096)
    rows = 600000
    ids = (torch.arange(rows) % 2).int().unsqueeze(1)
    order = torch.cat([torch.arange(0, rows, 2), torch.arange(1, rows, 2)]).int()
    first = torch.tensor([0, rows // 2, rows], dtype=torch.int32)
    xx, gu = mu.normal((rows, 64), 2).bfloat16(), mu.normal((2, 8192, 64), 3, 0.1).bfloat16()
    m = mk.Experts(mu.dims(*D), "bf16")
    h = torch.empty(rows, 4096, dtype=BF16, device="cuda")
    m.up(xx.cuda(), gu.cuda(), first.cuda(), order.cuda(), h)
    assert m.sync() == mk.MK_OK
    last = order[-5:].long()
    ref, slack = mu.up(xx[last].double(), gu.double(), torch.tensor([0, 0, 5]), torch.arange(5), 1)
    mu.within(h[-5:].cpu(), ref, slack)
    del h
    D = (4096, 2, 1, 64)
    hh, dn = mu.normal((rows, 64), 4).bfloat16(), mu.normal((2, 64, 4096), 5, 0.1).bfloat16()
    m = mk.Experts(mu.dims(*D), "bf16")
    y = torch.empty(rows, 4096, dtype=BF16, device="cuda")
    m.down(hh.cuda(), dn.cuda(), first.cuda(), order.cuda(), None, y)
    assert m.sync() == mk.MK_OK
    ref, slack = mu.down(hh[-5:].double(), dn.double(), torch.tensor([0, 0, 5]), torch.arange(5), None)
    mu.within(y[last.cuda()].cpu(), ref, slack)
    assert int(ids[last[-1]]) == 1


def test_refused_tensors(mk):
    c = lambda *s, t=F32: torch.empty(*s, dtype=t, device="cuda")   # noqa: E731
    x = c(4, 64)
    with pytest.raises(ValueError):
        mk.norm(x.cpu(), None, 1e-6, c(4, 64))
    with pytest.raises(ValueError):
        mk.norm(x.half(), None, 1e-6, c(4, 64))
    with pytest.raises(ValueError):
        mk.norm(x, None, 1e-6, c(4, 64, t=E4M3))                   # 8 bits without scales
    with pytest.raises(ValueError):
        mk.norm(x, None, 1e-6, c(4, 64), scales=c(4, 2, t=U8))
    with pytest.raises(ValueError):
        mk.norm(x, c(64), 1e-6, c(4, 64))                           # gamma is bf16
    with pytest.raises(ValueError):
        mk.norm(x, None, 1e-6, c(4, 64), add=c(4, 32))
    with pytest.raises(ValueError):
        mk.norm(x, None, 1e-6, c(4, 64), total=c(4, 64, t=BF16))
    with pytest.raises(ValueError):
        mk.norm(c(64, 4).t(), None, 1e-6, c(4, 64))                 # columns apart
    with pytest.raises(mk.MkError):
        mk.norm(x, None, 1e-6, x)                                   # onto its input
    with pytest.raises(mk.MkError):
        mk.norm(c(4, 68)[:, 1:65], None, 1e-6, c(4, 64))            # not 16-byte aligned
    with pytest.raises(ValueError):
        mk.quantize(x, c(4, 64, t=U8), c(4, 2, t=U8))
    with pytest.raises(mk.MkError):
        mk.quantize(c(4, 40), c(4, 40, t=E4M3), c(4, 1, t=U8))
    i = lambda *s: c(*s, t=torch.int32)   # noqa: E731
    with pytest.raises(ValueError):
        mk.route(c(4, 8, t=BF16), i(4, 2), c(4, 2), i(9), i(8))
    with pytest.raises(ValueError):
        mk.route(c(4, 8), i(4, 2), c(4, 2), i(8), i(8))
    with pytest.raises(mk.MkError):
        mk.route(c(4, 8), i(4, 9), c(4, 9), i(9), i(36))
    m, m8 = mk.Experts(mu.dims(64, 4, 2, 32), "bf16"), mk.Experts(mu.dims(64, 4, 2, 32), "e4m3")
    b = lambda *s: c(*s, t=BF16)   # noqa: E731
    with pytest.raises(ValueError):
        m.up(b(3, 64), b(4, 64, 64), i(5), i(7), b(6, 32))          # pairs that are no rows
    with pytest.raises(ValueError):
        m.up(b(3, 64), b(4, 64, 32), i(5), i(6), b(6, 32))
    with pytest.raises(ValueError):
        m.up(b(3, 64), b(4, 64, 64), i(5), i(6), b(6, 32), x_scales=c(3, 2, t=U8))
    with pytest.raises(ValueError):
        m8.up(c(3, 64, t=E4M3), c(4, 64, 64, t=E4M3), i(5), i(6), c(6, 32, t=E4M3))
    with pytest.raises(ValueError):
        m.down(b(6, 32), b(4, 64, 32), i(5), i(6), c(3, 2), b(3, 2, 64))   # bf16 weights lie [experts, ffn, hidden]
    h = b(6, 64)
    with pytest.raises(mk.MkError):
        m.down(h.view(-1)[:192].view(6, 32), b(4, 32, 64), i(5), i(6), None, h.view(3, 2, 64))   # y on its input


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_prompt_through_the_operators(mk, kind):
    # a two-layer model's prompt by the chunk operators (dense products by torch) against the decode step's prefill
    # rows: the same choice of experts from the same logits, and the hidden states of every layer
    D, seed, n = synth.TINY, 5, 8
    w = DeviceModel(D, seed).weights()
    pages, width, table = kv_pages_needed(D, [16], 2) + 2, 3, [2, 0, 1]
    pools = lambda: [torch.zeros(pages, D.n_kv_heads, 2, D.head_dim, 16, dtype=BF16, device="cuda") for _ in range(D.n_layers)]   # noqa: E731
    tok = torch.tensor([(37 * i + 11) % D.vocab for i in range(n)], dtype=torch.int32, device="cuda")
    plan = mk.Plan(D, w, pools(), [0], table, width, max_batch=8)
    plan.update_rows(list(range(n)), table * n, width, [0] * n)
    nxt = torch.empty(n, dtype=torch.int32, device="cuda")
    assert plan.step(tok, nxt) == mk.MK_OK
    c = lambda *s, t=F32: torch.empty(*s, dtype=t, device="cuda")   # noqa: E731
    hid, ids, gates, logits = (plan.read_debug(what, c(n, D.n_layers, m, t=t)) for what, m, t in (
        (mk.MK_DBG_HIDDEN, D.hidden, F32), (mk.MK_DBG_EXPERT_IDS, D.top_k, torch.int32), (mk.MK_DBG_GATES, D.top_k, F32),
        (mk.MK_DBG_ROUTER_LOGITS, D.n_experts, F32)))
    assert plan.sync() == mk.MK_OK
    chunk = mk.Chunk(D, "bf16", pages, [0], [n], table, width)
    m, mine, kv = mk.Experts(D, kind), pools(), None
    e8 = kind == "e4m3"
    x = w["embed"][tok.long()].float()
    for l in range(D.n_layers):
        nf, q = c(n, D.hidden), c(n, D.n_q_heads, D.head_dim, t=BF16)
        mk.norm(x, w["attn_norm"][l], D.rms_eps, nf)
        chunk.append(nf @ w["wqkv"][l].float().T, mine[l], q)
        chunk.attend(q, mine[l], q)
        o = q.float().flatten(1) @ w["wo"][l].float().T
        x2, rows, s = c(n, D.hidden), c(n, D.hidden, t=E4M3 if e8 else BF16), c(n, D.hidden // 32, t=U8) if e8 else None
        mk.norm(x, w["ffn_norm"][l], D.rms_eps, rows, add=o, total=x2, scales=s)
        g_ids, g, first, order = c(n, D.top_k, t=torch.int32), c(n, D.top_k), c(D.n_experts + 1, t=torch.int32), c(n * D.top_k, t=torch.int32)
        mk.route(logits[:, l], g_ids, g, first, order)             # the decode step's logits, which lie apart
        assert torch.equal(g_ids, ids[:, l])
        assert ((g - gates[:, l]).abs() < 1e-6).all()              # either a softmax in fp32
        gu, dn = w["w_gate_up"][l], w["w_down"][l]
        gu, gus, dn, dns = gu.view(D.n_experts, 2 * D.expert_ffn, D.hidden), None, dn.view(D.n_experts, D.expert_ffn, D.hidden), None
        h, hs = c(n * D.top_k, D.expert_ffn, t=E4M3 if e8 else BF16), c(n * D.top_k, D.expert_ffn // 32, t=U8) if e8 else None
        if e8:
            def eight(t):
                codes, scales = c(*t.shape, t=E4M3), c(*t.shape[:-1], t.shape[-1] // 32, t=U8)
                k = t.shape[-1]
                mk.quantize(t.reshape(-1, k), codes.view(-1, k), scales.view(-1, k // 32))
                return codes, scales
            (gu, gus), (dn, dns) = eight(gu), eight(dn.transpose(1, 2).contiguous())
        y = c(n, D.top_k, D.hidden, t=BF16)
        m.up(rows, gu, first, order, h, x_scales=s, w_scales=gus, h_scales=hs)
        m.down(h, dn, first, order, g, y, h_scales=hs, w_scales=dns)
        mk.norm(x2, None, 0.0, None, add=y, total=x2)
        assert m.sync() == mk.MK_OK and chunk.sync() == mk.MK_OK
        # bf16: the framework's own bound for hidden states; 8 bits: the experts' share of them is rounded to 4 bits
        # three times (rows, weights, h), each to within 2^-4, and the layer before comes in
        off = (x2 - hid[:, l]).norm() / hid[:, l].norm()
        share = (x2 - x).norm() / hid[:, l].norm()
        assert off < (1e-2 if not e8 else 1e-2 + 3 * 2 ** -4 * share * (l + 1)), (l, float(off), float(share))
        x = x2
    plan.close()
