"""More of the mixture-of-experts operators on a GPU against 64-bit CPU forms:
gates where SiLU saturates."""
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
        mu.check_eights(h.cpu(), s.cpu(), ref, slack)


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
