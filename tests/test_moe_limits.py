"""The experts' products when a wait inside them runs out: they give up, say so,
and touch nothing that is not theirs (GPU); what the test hook refuses (host)."""
import pytest
import torch

from tests import moe_util as mu
from tests import test_moe_ops as T

BF16, U8, E4M3 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn
LIMIT_US = 20000


@pytest.fixture(scope="module")
def mk(built):
    from persistent_moe_decode_02_gb300 import mk
    return mk


def test_the_hook_is_refused_without_an_object(mk):
    assert mk.lib().mk_experts_set_debug(None, 0, 0) == mk.MK_ERR_INVALID


@pytest.mark.gpu
def test_refused_limits(mk):
    m = mk.Experts(mu.dims(64, 4, 2, 32), "bf16")
    for bad in ((-1, 0), (2000001, 0), (0, -1), (0, 4)):
        assert mk.lib().mk_experts_set_debug(m.h, *bad) == mk.MK_ERR_INVALID
    with pytest.raises(mk.MkError):
        mk.Experts(mu.dims(64, 4, 2, 32), "bf16", timeout_us=-5)
    assert mk.lib().mk_experts_set_debug(m.h, 2000000, 0) == mk.MK_OK


class Run:
    """Up and down of one layer in guarded buffers."""

    def __init__(self, mk, kind, D, ids, **limits):
        self.mk, self.kind = mk, kind
        self.c = c = T.Case(kind, D, ids, 17)
        self.m = mk.Experts(mu.dims(*D), kind, **limits)
        (self.x, self.xs), (self.w, self.ws), (self.hh, self.hs), (self.d, self.ds) = map(T.cuda, (c.x, c.gu, c.h, c.dn))
        self.first, self.order, self.gates = c.first.cuda(), c.order.cuda(), c.gates.cuda()
        e8 = kind == "e4m3"
        self.w_h, self.h = T.cuda_empty((c.pairs, c.ffn), E4M3 if e8 else BF16)
        self.w_s, self.s = T.cuda_empty((c.pairs, c.ffn // 32), U8) if e8 else (None, None)
        self.w_y, self.y = T.cuda_empty((c.rows, c.k, c.hidden), BF16)

    def up(self):
        self.m.up(self.x, self.w, self.first, self.order, self.h, x_scales=self.xs, w_scales=self.ws, h_scales=self.s)
        return self.m.sync()

    def down(self):
        self.m.down(self.hh, self.d, self.first, self.order, self.gates, self.y, h_scales=self.hs, w_scales=self.ds)
        return self.m.sync()

    def guarded(self):
        return T.behind(self.w_h) and T.behind(self.w_y) and (self.w_s is None or T.behind(self.w_s))

    def check(self):
        T.check_up(self.mk, self.c, self.m)
        T.check_down(self.mk, self.c, m=self.m)


# an instance each: up to 32 pairs, up to 16 an expert, more; a block has a step or many, a tile or several
SHAPES = [((2048, 8, 2, 768), 9), ((1056, 37, 3, 352), 100), ((512, 4, 1, 1024), 400), ((64, 256, 8, 1280), 512)]


def lost_some(ids):
    ids = ids.clone()
    ids[::3, 0] = -1                                # pairs without an expert, whose rows down zeroes itself
    return ids


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,rows", SHAPES)
def test_no_list_comes(mk, kind, D, rows):
    # nothing is known of the tiles: nothing is read by them, nothing is written
    r = Run(mk, kind, D, lost_some(T.routed(D, rows)), timeout_us=LIMIT_US, debug_drop=1)
    assert r.up() == mk.MK_ERR_DEP_TIMEOUT and r.down() == mk.MK_ERR_DEP_TIMEOUT
    assert (r.w_h.float() == 7).all() and (r.w_y == 7).all()
    Run(mk, kind, D, r.c.ids).check()               # the device is fine


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,rows", [s for s in SHAPES if s[0][0] > 64])
def test_copies_stop(mk, kind, D, rows):
    # up has 4 steps of K at least, so every block with a tile gives up
    r = Run(mk, kind, D, lost_some(T.routed(D, rows)), timeout_us=LIMIT_US, debug_drop=2)
    assert r.up() == mk.MK_ERR_DEP_TIMEOUT and r.down() == mk.MK_ERR_DEP_TIMEOUT
    assert r.guarded()
    Run(mk, kind, D, r.c.ids).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [(32, 256, 8, 2560), (2560, 256, 8, 32)])
def test_accumulators_are_not_released(mk, kind, D):
    r = Run(mk, kind, D, T.routed(D, 512), timeout_us=LIMIT_US, debug_drop=3)
    assert (r.up() if D[0] == 32 else r.down()) == mk.MK_ERR_DEP_TIMEOUT   # (many tiles a block)
    assert r.guarded()
    Run(mk, kind, D, r.c.ids).check()


TWO = [("up", (256, 4, 2, 2048)), ("down", (4096, 4, 2, 256))]


@pytest.mark.gpu
@pytest.mark.parametrize("op,D", TWO)
@pytest.mark.parametrize("drop", [1, 2, 3])
def test_two_sms_give_up(mk, op, D, drop):
    # drop 2: the odd block's copies stop, the even one waits for them
    rows = 4600 if drop == 3 else 2600
    ids = torch.randint(0, 4, (rows, 2), generator=torch.Generator().manual_seed(3)).int()
    r = Run(mk, "bf16", D, lost_some(ids) if drop == 1 else ids, timeout_us=LIMIT_US, debug_drop=drop)
    assert (r.up() if op == "up" else r.down()) == mk.MK_ERR_DEP_TIMEOUT
    assert r.guarded()
    if drop == 1:
        assert (r.w_h == 7).all() and (r.w_y == 7).all()
    fine = Run(mk, "bf16", D, r.c.ids)
    (T.check_up if op == "up" else T.check_down)(mk, fine.c, m=fine.m)


@pytest.mark.gpu
def test_a_short_limit_that_nothing_runs_into(mk):
    # the limit is of a wait, not of a call
    Run(mk, "bf16", (2048, 8, 2, 768), T.routed((2048, 8, 2, 768), 500), timeout_us=LIMIT_US).check()


@pytest.mark.gpu
def test_giving_up_takes_one_limit(mk):
    # the even block's stages never fill up (the odd one's copies stop): what is in flight is waited for once (2 s), not
    # for each of five or six stages
    import time
    r = Run(mk, "bf16", (256, 4, 2, 2048), torch.randint(0, 4, (2600, 2), generator=torch.Generator().manual_seed(3)).int(),
            timeout_us=LIMIT_US, debug_drop=2)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    assert r.up() == mk.MK_ERR_DEP_TIMEOUT
    assert time.monotonic() - t0 < 3.9


@pytest.mark.gpu
def test_every_stream_hears_of_it_once(mk):
    # a wait that runs out on one stream is not lost to it because another one asked first, and is told once
    D, rows = (64, 4, 2, 64), 20
    r = Run(mk, "bf16", D, T.routed(D, rows))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    assert r.m.sync(a) == r.m.sync(b) == r.m.sync() == mk.MK_OK
    limits = mk.lib().mk_experts_set_debug

    def product(stream):
        r.m.up(r.x, r.w, r.first, r.order, r.h, stream=stream)

    torch.cuda.synchronize()
    assert limits(r.m.h, LIMIT_US, 1) == mk.MK_OK
    product(b)
    assert limits(r.m.h, 0, 0) == mk.MK_OK
    torch.cuda.synchronize()
    assert r.m.sync(a) == mk.MK_ERR_DEP_TIMEOUT and r.m.sync(a) == mk.MK_OK
    assert r.m.sync(b) == mk.MK_ERR_DEP_TIMEOUT and r.m.sync(b) == mk.MK_OK
    assert r.m.sync() == mk.MK_ERR_DEP_TIMEOUT and r.m.sync() == mk.MK_OK
    product(a)                                      # a good one
    assert r.m.sync(a) == r.m.sync(b) == mk.MK_OK
    assert limits(r.m.h, LIMIT_US, 1) == mk.MK_OK
    product(a)                                      # and again a bad one
    torch.cuda.synchronize()
    assert r.m.sync(b) == mk.MK_ERR_DEP_TIMEOUT and r.m.sync(a) == mk.MK_ERR_DEP_TIMEOUT
    assert r.m.sync(a) == r.m.sync(b) == mk.MK_OK


@pytest.mark.gpu
def test_an_object_dies_beside_a_capture(mk):
    # the garbage collector may take an object at any time, while the thread captures a graph too
    r = Run(mk, "bf16", (64, 4, 2, 64), T.routed((64, 4, 2, 64), 20))
    other = mk.Experts(mu.dims(64, 4, 2, 32), "e4m3")
    r.up()
    want = r.h.clone()
    r.h.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        other.close()
        r.m.up(r.x, r.w, r.first, r.order, r.h)
    g.replay()
    assert r.m.sync() == mk.MK_OK and torch.equal(r.h, want)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["plan", "chunk"])
def test_plans_and_chunks_die_beside_a_capture(mk, what):
    import synth
    from synth.device import DeviceModel
    D = synth.TINY
    pools = [torch.zeros(4, D.n_kv_heads, 2, D.head_dim, 16, dtype=BF16, device="cuda") for _ in range(D.n_layers)]
    if what == "plan":
        gone = mk.Plan(D, DeviceModel(D, 1).weights(), pools, [0], [0, 1, 2], 3)
        nxt = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert gone.step(nxt, nxt) == mk.MK_OK and gone.sync() == mk.MK_OK
    else:
        gone = mk.Chunk(D, "bf16", 4, [0], [3], [0, 1, 2], 3)
        gone.update([0], [5], [0, 1, 2], 3)         # (an upload, whose buffer is released too)
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gone.close()
        x += 1
    g.replay()
    assert (x.cpu() == 1).all()
