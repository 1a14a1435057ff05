"""The mixture-of-experts operators on the host (no GPU): what mk_norm,
mk_quantize, mk_route and mk_experts_* refuse."""
import ctypes

import pytest
import torch

from tests import moe_util as mu


@pytest.fixture(scope="module")
def mk(built):
    from persistent_moe_decode_02_gb300 import mk
    return mk


vp = ctypes.c_void_p
MB = 1 << 20


def at(i, off=0):
    return vp(i * 64 * MB + off)   # aligned, apart, never read: every call below is refused before a CUDA call


def test_refused_norms(mk):
    L, bad, uns = mk.lib(), mk.MK_ERR_INVALID, mk.MK_ERR_UNSUPPORTED

    def norm(rows=2, n=64, x=at(1), xt=1, stride=64, add=at(2), at_=0, terms=1, gamma=at(3), eps=1e-6, total=at(4), out=at(5),
             ot=0, s=None):
        return L.mk_norm(rows, n, x, xt, stride, add, at_, terms, gamma, eps, total, out, ot, s, None)

    assert norm(rows=-1) == norm(n=0) == norm(n=60, stride=64) == norm(xt=2) == norm(xt=-1) == norm(at_=2) == norm(terms=-1) == bad
    assert norm(ot=3) == norm(ot=2, n=40, stride=40, s=at(6)) == norm(stride=63) == norm(stride=66) == bad
    assert norm(eps=-1.0) == norm(eps=float("nan")) == norm(eps=float("inf")) == bad
    assert norm(total=None, out=None) == norm(x=None) == norm(add=None) == norm(ot=2) == bad
    assert norm(x=at(1, 8)) == norm(add=at(2, 2)) == norm(gamma=at(3, 4)) == norm(total=at(4, 4)) == norm(out=at(5, 8)) == bad
    assert norm(n=16392, stride=16392) == norm(terms=70000) == uns
    # results on other buffers
    assert norm(out=at(1)) == norm(out=at(2, 16)) == norm(out=at(4, 256)) == norm(out=at(3)) == bad
    assert norm(total=at(2)) == norm(total=at(1, 16)) == norm(total=at(1), stride=68) == bad
    assert norm(ot=2, s=at(5, 64)) == norm(ot=2, s=at(1, 4)) == bad
    assert norm(rows=0) == norm(rows=0, x=None, add=None, total=None) == mk.MK_OK


def test_refused_quantisations(mk):
    L, bad = mk.lib(), mk.MK_ERR_INVALID
    q = lambda rows=2, n=64, x=at(1), xt=0, stride=64, c=at(2), s=at(3): L.mk_quantize(rows, n, x, xt, stride, c, s, None)   # noqa: E731
    assert q(rows=-1) == q(n=0) == q(n=48) == q(xt=2) == q(stride=32) == q(stride=68) == bad
    assert q(x=None) == q(c=None) == q(s=None) == q(x=at(1, 2)) == q(c=at(2, 8)) == bad
    assert q(c=at(1, 128)) == q(s=at(1)) == q(s=at(2, 127)) == bad
    assert q(rows=0, x=None, c=None, s=None) == mk.MK_OK


def test_refused_routes(mk):
    L, bad, uns = mk.lib(), mk.MK_ERR_INVALID, mk.MK_ERR_UNSUPPORTED

    def route(rows=2, e=16, k=4, x=at(1), stride=16, ids=at(2), gates=at(3), first=at(4), order=at(5)):
        return L.mk_route(rows, e, k, x, stride, ids, gates, first, order, None)

    assert route(rows=-1) == route(e=0) == route(k=0) == route(k=17) == route(stride=15) == bad
    assert route(x=None) == route(ids=None) == route(gates=None) == route(first=None) == route(order=None) == route(x=at(1, 2)) == bad
    assert route(rows=0, first=None) == bad
    assert route(e=257, stride=257) == route(k=9) == route(rows=1 << 28) == uns
    assert route(order=at(2, 16)) == route(first=at(5)) == route(gates=at(1, 64)) == bad


def test_refused_experts(mk):
    bad, uns = mk.MK_ERR_INVALID, mk.MK_ERR_UNSUPPORTED

    def refused(code, *d, kind="bf16"):
        with pytest.raises(mk.MkError) as e:
            mk.Experts(mu.dims(*d), kind)
        assert e.value.code == code, e.value

    refused(bad, 0, 8, 2, 64)
    refused(bad, 64, 0, 2, 64)
    refused(bad, 64, 8, 0, 64)
    refused(bad, 64, 8, 9, 64)
    refused(bad, 64, 8, 2, -8)
    refused(uns, 64, 257, 2, 64)
    refused(uns, 64, 16, 9, 64)
    refused(uns, 60, 8, 2, 64)
    refused(uns, 64, 8, 2, 48, kind="e4m3")
    refused(uns, 32776, 8, 2, 64)
    with pytest.raises(ValueError):
        mk.Experts(mu.dims(64, 8, 2, 64), "fp8")
    L = mk.lib()
    one = at(1)
    assert L.mk_experts_create(None, 0, ctypes.byref(vp())) == bad
    d = mk.MkModelDims(hidden=64, n_experts=8, top_k=2, expert_ffn=64)
    assert L.mk_experts_create(ctypes.byref(d), 0, None) == L.mk_experts_create(ctypes.byref(d), 1, ctypes.byref(vp())) == bad
    assert L.mk_experts_up(None, 1, one, None, one, None, one, one, one, None, None) == bad
    assert L.mk_experts_down(None, 1, one, None, one, None, one, one, one, one, None) == bad
    assert L.mk_experts_sync(None, None) == bad
    L.mk_experts_destroy(None)


def test_refused_tensors(mk):
    # (no device here: every call is refused by its own checks, or for the device)
    cpu = torch.zeros(2, 64)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        mk.norm(cpu, None, 1e-6, cpu)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        mk.quantize(cpu, cpu, cpu)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        mk.route(cpu, cpu, cpu, cpu, cpu)


def test_the_quantised_form():
    # the tests' own rule: nothing above 448, the next smaller scale would overflow, codes off by half a step
    x = mu.normal((50, 64), 1) * torch.exp(3 * mu.normal((50, 64), 2))
    codes, scales = mu.quantise(x)
    top = x.double().unflatten(-1, (-1, 32)).abs().amax(-1)
    unit = torch.exp2(scales.double() - 127)
    assert (top <= 448 * unit).all() and (top > 448 * unit / 2).all()
    err = (mu.values(codes, scales) - x.double()).abs()
    assert (err <= mu.E4M3_STEP * x.double().abs() + mu.E4M3_MIN * unit.repeat_interleave(32, -1)).all()


def test_the_check_of_8_bit_results():
    # one code that is off, or none, is seen, wherever it lies in its group
    ref = mu.normal((3, 64), 5).double()
    codes, scales = mu.quantise(ref.float())
    slack = torch.zeros_like(ref)
    mu.check_eights_strictly(codes, scales, ref.float().double(), slack)
    for at in ((0, 0), (1, 31), (2, 63)):
        bad = codes.clone().view(torch.uint8)
        bad[at] = 0x7f                                                     # NaN
        with pytest.raises(AssertionError):
            mu.check_eights_strictly(bad.view(torch.float8_e4m3fn), scales, ref, slack)
        bad = codes.clone().view(torch.uint8)
        bad[at] ^= 0x80                                                    # the other sign
        with pytest.raises(AssertionError):
            mu.check_eights_strictly(bad.view(torch.float8_e4m3fn), scales, ref, slack)
        for s in (1, 255):                                                 # the next scale; a scale that is none
            wrong = scales.clone()
            wrong[at[0], at[1] // 32] = 255 if s == 255 else wrong[at[0], at[1] // 32] + 1
            with pytest.raises(AssertionError):
                mu.check_eights_strictly(codes, wrong, ref, slack)
