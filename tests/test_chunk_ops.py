"""The operators over chunks (mk_chunk_*, mk_probs, mk_verify) on a GPU against
64-bit CPU forms, at the sizes and masks where they can go wrong, and run
together as a server uses them."""
import ctypes
import dataclasses
import math

import pytest
import torch

import synth
from synth.device import DeviceModel, PagedKV, kv_pages_needed
from tests import chunk_util as cu

pytestmark = pytest.mark.gpu

HEADS = {"g8": (32, 4, 128), "g2d64": (4, 2, 64), "g6": (12, 2, 128), "g1d64": (5, 5, 64), "g3": (3, 1, 128),
         "g7d64": (14, 2, 64)}
LENS = {
    "one_token_alone": ([0], [1]),
    "one_token": ([333], [1]),
    "page_ends": ([15, 16, 17, 31], [1, 1, 16, 17]),
    "tile_ends": ([127, 128, 0], [1, 129, 128]),
    "drafts": ([700, 0, 41, 1023, 1024, 5], [5, 3, 1, 4, 5, 8]),
    "prompts": ([0, 0, 0], [300, 77, 129]),
    "behind_cache": ([500, 1100], [210, 33]),
    "an_empty_request": ([40, 0, 10], [0, 0, 6]),
    "long_one_token": ([9001], [1]),
}


@pytest.fixture(scope="module")
def mk(built):
    from persistent_moe_decode_02_gb300 import mk
    return mk


def make(mk, heads, kv, lens, seed=1, theta=1e4):
    nq, nkv, d = HEADS[heads]
    batch = cu.Batch(*LENS[lens] if isinstance(lens, str) else lens, seed=seed)
    D = cu.dims(nq, nkv, d, theta)
    return D, batch, mk.Chunk(D, kv, batch.num_pages, batch.cached, batch.new, batch.flat, batch.width)


def behind(batch):
    """Slots of the requests' last pages behind their last tokens."""
    s = [batch.slots(b, t, -(-t // cu.PAGE) * cu.PAGE) for b, t in enumerate(batch.total) if t % cu.PAGE]
    return (torch.cat([x[0] for x in s]), torch.cat([x[1] for x in s])) if s else None


def check_attend(mk, heads, kv, lens, seed=1, scale=1.0):
    D, batch, chunk = make(mk, heads, kv, lens, seed)
    pool = cu.make_pool(kv, batch.num_pages, D.n_kv_heads, D.head_dim, seed + 2)
    q = cu.normal((batch.rows, D.n_q_heads, D.head_dim), seed + 3, scale).bfloat16()
    ref, mag = cu.attend(q, pool, kv, batch, D.n_kv_heads)
    gone = behind(batch)
    if gone is not None:   # what lies behind a request's end is no number at all
        if kv == "bf16":
            pool[gone[0], :, :, :, gone[1]] = math.nan
        else:
            pool[gone[0], :, :, :, gone[1]] = 255   # e4m3 NaN, E8M0 NaN
    out = torch.full((batch.rows + 1, D.n_q_heads, D.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    chunk.attend(q.cuda(), pool.cuda(), out[:-1])
    assert chunk.sync() == mk.MK_OK
    got = out.cpu()
    assert (got[-1] == 7).all()    # the row behind the last one is left
    err = (got[:-1].double() - ref).abs()
    bad = err > cu.attend_bound(ref, mag)
    assert not bad.any(), (int(bad.sum()), float(err.max()), bad.nonzero()[:5].tolist())
    chunk.close()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("heads", ["g8", "g2d64"])
def test_attend_lengths(mk, heads, kv, lens):
    check_attend(mk, heads, kv, lens)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", ["g6", "g1d64", "g3", "g7d64"])
def test_attend_groups(mk, heads, kv):
    for lens in ("drafts", "behind_cache"):
        check_attend(mk, heads, kv, lens, seed=5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_peaked_scores(mk, kv):
    # scores of tens of units: the running maximum moves often
    check_attend(mk, "g8", kv, ([300, 40], [40, 300]), seed=9, scale=6.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,most", [("g8", 16), ("g2d64", 70), ("g8", 300)])
def test_attend_many_requests(mk, heads, kv, most):
    # more blocks of rows than CTAs: each works through several tasks, of one query tile and of two
    g = torch.Generator().manual_seed(most)
    cached = torch.randint(0, 700, (70,), generator=g).tolist()
    new = torch.randint(0, most + 1, (70,), generator=g).tolist()
    check_attend(mk, heads, kv, (cached, new), seed=most)
    check_attend(mk, heads, kv, (cached + [30000], new + [1]), seed=most + 1)   # and one that is split


def test_attend_shared_prefix_pages(mk):
    # two requests read the same cached pages and add rows in pages of their own
    D = cu.dims(8, 2, 128)
    batch = cu.Batch([64, 64], [3, 20], seed=3)
    batch.table[1][:4] = batch.table[0][:4]
    batch.flat = [p for row in batch.table for p in row]
    chunk = mk.Chunk(D, "bf16", batch.num_pages, batch.cached, batch.new, batch.flat, batch.width)
    pool = cu.make_pool("bf16", batch.num_pages, 2, 128, 5)
    q = cu.normal((23, 8, 128), 6).bfloat16()
    ref, mag = cu.attend(q, pool, "bf16", batch, 2)
    out = torch.empty(23, 8, 128, dtype=torch.bfloat16, device="cuda")
    chunk.attend(q.cuda(), pool.cuda(), out)
    assert chunk.sync() == mk.MK_OK
    assert ((out.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()


@pytest.mark.parametrize("rows_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,lens", [("g8", "drafts"), ("g8", "behind_cache"), ("g2d64", "page_ends"),
                                        ("g6", "prompts"), ("g1d64", "an_empty_request"), ("g7d64", "one_token_alone")])
def test_append(mk, heads, lens, kv, rows_type):
    D, batch, chunk = make(mk, heads, kv, lens, seed=2)
    nq, nkv, d = D.n_q_heads, D.n_kv_heads, D.head_dim
    pool = cu.make_pool(kv, batch.num_pages, nkv, d, 4)
    wide = cu.normal((batch.rows, nkv * (nq // nkv + 2) * d + 64), 5).to(rows_type)   # rows lie apart
    wide[0, (nq // nkv) * d:(nq // nkv + 1) * d] = 0                                  # a key of zeros
    x = wide[:, :-64].view(batch.rows, nkv, nq // nkv + 2, d)
    pos = batch.positions()
    turned = cu.rotate(x[:, :, :-1], pos, D.rope_theta)
    size = (x[:, :, :-1].double()[..., :d // 2].abs() + x[:, :, :-1].double()[..., d // 2:].abs()).repeat(1, 1, 1, 2)
    ref_q, ref_k, ref_v = turned[:, :, :-1].flatten(1, 2), turned[:, :, -1], x[:, :, -1]
    # cos and sin rounded to fp32, two products and a sum: under 4 roundings of the pair's size
    slack = 4 * 2.0 ** -24 * size
    gpool, gq = pool.cuda(), torch.empty(batch.rows, nq, d, dtype=torch.bfloat16, device="cuda")
    chunk.append(wide.cuda()[:, :-64], gpool, gq)
    assert chunk.sync() == mk.MK_OK
    assert ((gq.cpu().double() - ref_q).abs() <= cu.BF16 * ref_q.abs() + slack[:, :, :-1].flatten(1, 2) * 1.01).all()
    got, (page, slot) = gpool.cpu(), batch.new_slots()
    new = got[page, :, :, :, slot]
    kept, was = got.clone(), pool.clone()
    kept[page, :, :, :, slot] = 0
    was[page, :, :, :, slot] = 0
    assert torch.equal(kept.view(torch.uint8), was.view(torch.uint8))   # nothing but the new slots is written
    if kv == "bf16":
        assert torch.equal(new[:, :, 1], ref_v.bfloat16())
        assert ((new[:, :, 0].double() - ref_k).abs() <= cu.BF16 * ref_k.abs() + slack[:, :, -1] * 1.01).all()
        return
    code, k = cu.quantise(ref_v.float())
    assert torch.equal(new[:, :, 1, :-1], code) and torch.equal(new[:, :, 1, -1].int() - 127, k)
    k = new[:, :, 0, -1].double() - 127
    val = torch.ldexp(new[:, :, 0, :-1].contiguous().view(torch.float8_e4m3fn).double(), k.unsqueeze(-1))
    unit = torch.exp2(k).unsqueeze(-1)
    assert ((val - ref_k).abs() <= torch.maximum(cu.E4M3_STEP * ref_k.abs(), cu.E4M3_MIN * unit) + 2 * slack[:, :, -1]).all()
    top = ref_k.abs().amax(-1)
    # the smallest scale that holds the vector, up to the rotation's own roundings
    assert (top <= 448 * torch.exp2(k) * (1 + 2.0 ** -20)).all()
    assert ((top >= 224 * torch.exp2(k) * (1 - 2.0 ** -20)) | (k == -127)).all()


def test_append_far_position_and_no_rotation(mk):
    # a position near 2^18: angles keep their fraction; theta 0 leaves the rows
    far = 262143
    for theta in (1e4, 0.0):
        D = cu.dims(2, 1, 64, theta)
        width = far // cu.PAGE + 2
        table = [0] * width
        table[far // cu.PAGE:] = [1, 2]
        chunk = mk.Chunk(D, "bf16", 3, [far], [3], table, width)
        x = cu.normal((3, 1, 4, 64), 8)
        pool, q = torch.zeros(3, 1, 2, 64, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        chunk.append(x.cuda(), pool, q)
        assert chunk.sync() == mk.MK_OK
        ref = cu.rotate(x[:, :, :2], torch.arange(far, far + 3), theta).flatten(1, 2)
        assert ((q.cpu().double() - ref).abs() <= cu.BF16 * ref.abs() + 2.0 ** -20).all()


def test_append_infinities_and_nan_in_8_bits(mk):
    D = cu.dims(0, 1, 64, 0.0)
    chunk = mk.Chunk(D, "e4m3", 1, [0], [4], [0], 1)
    x = cu.normal((4, 1, 2, 64), 3)
    x[0, 0, 0, 5], x[1, 0, 1, 6], x[2, 0, 0, 7] = math.inf, math.nan, 3e38
    x[3] = 1e-44
    pool = torch.zeros(1, 1, 2, 65, 16, dtype=torch.uint8, device="cuda")
    chunk.append(x.cuda(), pool)
    out = torch.empty(4, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    chunk.read(pool, out)
    assert chunk.sync() == mk.MK_OK
    got = out.cpu()
    assert got[0, 0, 0, 5] == math.inf
    assert got[1, 0, 1, 6].isnan() and got[1].isnan().sum() == 1      # the vector's others are numbers
    fine = torch.ones(64, dtype=torch.bool)
    fine[6] = False
    assert ((got[1, 0, 1].double() - x[1, 0, 1].double()).abs() <= 2.0 ** -4 * x[1, 0, 1].abs() + 2.0 ** -9)[fine].all()
    assert abs(float(got[2, 0, 0, 7]) / 3e38 - 1) <= 2.0 ** -4 + cu.BF16
    assert (got[3].abs() <= 2e-44).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,lens", [("g8", "drafts"), ("g2d64", "an_empty_request"), ("g3", "tile_ends")])
def test_read(mk, heads, lens, kv):
    D, batch, chunk = make(mk, heads, kv, lens)
    pool = cu.make_pool(kv, batch.num_pages, D.n_kv_heads, D.head_dim, 4)
    ref = torch.cat([cu.rows_of(pool, kv, batch, b) for b in range(len(batch.new)) if batch.total[b]])
    out = torch.full((ref.shape[0] + 1, *ref.shape[1:]), 7.0, dtype=torch.bfloat16, device="cuda")
    chunk.read(pool.cuda(), out[:-1])
    assert chunk.sync() == mk.MK_OK
    assert torch.equal(out[:-1].cpu(), ref.bfloat16()) and (out[-1] == 7).all()


def test_rows_move_between_pools(mk):
    # out of an 8-bit pool and into a bf16 one at other pages, values unchanged
    D = cu.dims(0, 2, 128, 0.0)
    batch, other = cu.Batch([100, 31], [0, 0], seed=1), cu.Batch([0, 0], [100, 31], seed=2)
    pool = cu.make_pool("e4m3", batch.num_pages, 2, 128, 4)
    src = mk.Chunk(D, "e4m3", batch.num_pages, batch.cached, batch.new, batch.flat, batch.width)
    dst = mk.Chunk(D, "bf16", other.num_pages, other.cached, other.new, other.flat, other.width)
    rows = torch.empty(131, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    to = torch.zeros(other.num_pages, 2, 2, 128, 16, dtype=torch.bfloat16, device="cuda")
    src.read(pool.cuda(), rows)
    dst.append(rows, to)
    assert dst.sync() == mk.MK_OK
    for b in range(2):
        assert torch.equal(cu.rows_of(to.cpu(), "bf16", other, b), cu.rows_of(pool, "e4m3", batch, b).bfloat16().double())


# ---- probabilities and verification ----

def probs_bound(ref):
    """The exponent's argument is rounded three times (2^-22 of it), the sum about 130 times (2^-17), and the
    result twice."""
    x = torch.log2(ref / ref.amax(-1, keepdim=True)).abs().nan_to_num(0, posinf=0)
    return ref * (2.0 ** -16 + 2.0 ** -22 * x) + 2.0 ** -126


@pytest.mark.parametrize("vocab", [1, 3, 4, 127, 2048, 2051, 32000, 151936, 393216])
@pytest.mark.parametrize("temperature", [0.7, 1.0, 0.05, 40.0])
def test_probs(mk, vocab, temperature):
    rows = 3
    x = cu.normal((rows, vocab + 5), vocab, 3.0)[:, :vocab]
    ref = torch.softmax(x.double() / torch.tensor(temperature, dtype=torch.float32).double(), -1)
    gx = torch.empty(rows, vocab + 5, device="cuda")[:, :vocab]
    gx.copy_(x)
    out = torch.full((rows + 1, vocab), 7.0, device="cuda")
    mk.probs(gx, temperature, out[:-1])
    got = out.cpu()
    assert ((got[:-1].double() - ref).abs() <= probs_bound(ref)).all()
    assert (got[-1] == 7).all()


@pytest.mark.parametrize("vocab", [5, 3001, 151936])
def test_probs_masks_and_ends(mk, vocab):
    low = torch.finfo(torch.float32).min
    x = cu.normal((8, vocab), 1)
    x[0, 1:] = -math.inf                  # one left
    x[1] = -math.inf                      # nothing left
    x[2] = low                            # every logit the lowest number
    x[3, ::2] = low                       # some
    x[4, vocab - 1] = math.nan
    x[5, 0] = math.inf
    x[6, vocab // 2:] = -math.inf
    x[7, 0], x[7, 1] = torch.finfo(torch.float32).max, low
    for t in (1.0, 0.0):
        out = torch.empty(8, vocab, device="cuda")
        mk.probs(x.cuda(), t, out)
        got = out.cpu()
        assert got[4].isnan().all() and got[5].isnan().all() and (got[1] == 0).all()
        fine = [0, 2, 3, 6, 7]
        if t:
            ref = torch.softmax(x[fine].double(), -1)
            assert ((got[fine].double() - ref).abs() <= probs_bound(ref)).all()
        else:
            ref = torch.zeros(len(fine), vocab)
            for i, r in enumerate(fine):   # the lowest index of equal ones
                ref[i, int((x[r] == x[r].max()).nonzero()[0])] = 1
            assert torch.equal(got[fine], ref)


def test_probs_in_place_and_tiny_temperature(mk):
    x = cu.normal((4, 4099), 5).cuda()
    ref = torch.empty_like(x)
    mk.probs(x, 0.9, ref)
    mk.probs(x, 0.9, x)
    assert torch.equal(x, ref)
    y, out = cu.normal((2, 100), 6).cuda(), torch.empty(2, 100, device="cuda")
    mk.probs(y, 3e-39, out)               # as good as greedy, and no NaN
    assert torch.equal(out.argmax(1), y.argmax(1)) and float(out.sum()) == 2


def draws(b, k, vocab, seed, near=0.7):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(b, k + 1, vocab, generator=g) * 2
    d = t[:, :k] + near * torch.randn(b, k, vocab, generator=g)
    t, d = torch.softmax(t, -1), torch.softmax(d, -1)
    x = torch.multinomial(d.reshape(-1, vocab), 1, generator=g).view(b, k).int() if k else torch.zeros(b, 0, dtype=torch.int32)
    return t, d, x, torch.rand(b, k, generator=g), torch.rand(b, generator=g)


def check_verify(mk, t, d, x, u, r, count=None):
    b, k1, _ = t.shape
    tokens = torch.full((b + 1, k1), 77, dtype=torch.int32, device="cuda")
    accepted = torch.full((b + 1,), 77, dtype=torch.int32, device="cuda")
    mk.verify(t.cuda(), None if d is None else d.cuda(), x.cuda(), u.cuda(), r.cuda(), tokens[:-1], accepted[:-1],
              None if count is None else count.cuda())
    ref_t, ref_a = cu.verify(t, d, x, u, r, count)
    assert torch.equal(accepted[:-1].cpu(), torch.from_numpy(ref_a))
    assert torch.equal(tokens[:-1].cpu(), torch.from_numpy(ref_t))
    assert (tokens[-1] == 77).all() and int(accepted[-1]) == 77


@pytest.mark.parametrize("b,k,vocab", [(1, 0, 11), (1, 1, 1), (3, 4, 5), (7, 3, 2047), (4, 5, 2049), (5, 7, 32000),
                                       (2, 2, 151936), (1, 1, 393215), (2, 40, 513)])
@pytest.mark.parametrize("point", [False, True])
def test_verify(mk, b, k, vocab, point):
    for seed in range(4):
        t, d, x, u, r = draws(b, k, vocab, 100 * seed + vocab)
        count = torch.randint(-1, k + 2, (b,), generator=torch.Generator().manual_seed(seed)).int() if seed % 2 else None
        check_verify(mk, t, None if point or not k else d, x, u, r, count)


def test_verify_ends(mk):
    vocab = 4097
    t, d, x, u, r = draws(9, 2, vocab, 5)
    r[0], r[1], r[2] = 0.0, 1.0, math.nan
    x[3, 0], x[4, 1] = -1, vocab            # drafts that are no tokens
    u[5, 0] = math.nan
    u[0, 0] = u[1, 0] = 2.0                 # refused
    t[6, 0, 5] = math.nan
    t[7] = 0                                # nothing to draw
    d[8] = t[8, :2]                         # no difference, yet refused
    u[8] = 2.0
    check_verify(mk, t, d, x, u, r)
    t[7] = math.nan
    check_verify(mk, t, None, x, u, r)


def test_verify_follows_the_target(mk):
    # whatever the drafts, the first token's law is the target's: the counts of 60000
    # draws over 6 tokens, each within 5 standard deviations
    n, vocab = 60000, 6
    g = torch.Generator().manual_seed(3)
    p, q = torch.softmax(torch.randn(vocab, generator=g), 0), torch.softmax(torch.randn(vocab, generator=g), 0)
    x = torch.multinomial(q, n, replacement=True, generator=g).view(n, 1).int()
    tokens = torch.empty(n, 2, dtype=torch.int32, device="cuda")
    accepted = torch.empty(n, dtype=torch.int32, device="cuda")
    mk.verify(p.expand(n, 2, vocab).contiguous().cuda(), q.expand(n, 1, vocab).contiguous().cuda(), x.cuda(),
              torch.rand(n, 1, generator=g).cuda(), torch.rand(n, generator=g).cuda(), tokens, accepted)
    got = torch.bincount(tokens[:, 0].cpu().long(), minlength=vocab).double()
    assert ((got - n * p.double()).abs() <= 5 * (n * p.double() * (1 - p.double())).sqrt()).all()


# ---- how they are called ----

def test_streams_graphs_and_updates(mk):
    # captured with its inputs, replayed after they changed; a second chunk runs on another stream at the same time
    D, batch, chunk = make(mk, "g8", "bf16", "drafts", seed=4)
    D2, batch2, chunk2 = make(mk, "g8", "bf16", "behind_cache", seed=6)
    work = []
    for b, c in ((batch, chunk), (batch2, chunk2)):
        work.append(dict(b=b, c=c, pool=cu.make_pool("bf16", b.num_pages, 4, 128, 9).cuda(),
                         qkv=torch.empty(b.rows, 4, 10, 128, dtype=torch.bfloat16, device="cuda"),
                         q=torch.empty(b.rows, 32, 128, dtype=torch.bfloat16, device="cuda"),
                         out=torch.empty(b.rows, 32, 128, dtype=torch.bfloat16, device="cuda"),
                         stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph()))
    for w in work:
        w["qkv"].copy_(cu.normal(w["qkv"].shape, 3).bfloat16())
    torch.cuda.synchronize()
    for w in work:
        with torch.cuda.graph(w["graph"], stream=w["stream"]):
            w["c"].append(w["qkv"], w["pool"], w["q"])
            w["c"].attend(w["q"], w["pool"], w["out"])
            with pytest.raises(mk.MkError):
                w["c"].update(w["b"].cached, w["b"].new, w["b"].flat, w["b"].width, stream=w["stream"])
    for turn in range(3):
        for w in work:
            w["qkv"].copy_(cu.normal(w["qkv"].shape, 10 + turn).bfloat16())
        torch.cuda.synchronize()
        for w in work:
            with torch.cuda.stream(w["stream"]):
                w["graph"].replay()
        torch.cuda.synchronize()
        for w in work:
            ref, mag = cu.attend(w["q"].cpu(), w["pool"].cpu(), "bf16", w["b"], 4)
            assert ((w["out"].cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()
    # another batch for the same chunk, larger and smaller, on a side stream
    side = torch.cuda.Stream()
    for lens in ("prompts", "one_token", "behind_cache"):
        b = cu.Batch(*LENS[lens], seed=8)
        pool = cu.make_pool("bf16", max(b.num_pages, batch.num_pages), 4, 128, 2)
        c = mk.Chunk(D, "bf16", pool.shape[0], batch.cached, batch.new, batch.flat, batch.width)
        c.update(b.cached, b.new, b.flat, b.width, stream=side)
        q, out = cu.normal((b.rows, 32, 128), 1).bfloat16(), torch.empty(b.rows, 32, 128, dtype=torch.bfloat16, device="cuda")
        gq, gp = q.cuda(), pool.cuda()
        side.wait_stream(torch.cuda.current_stream())
        c.attend(gq, gp, out, stream=side)
        assert c.sync(side) == mk.MK_OK
        ref, mag = cu.attend(q, pool, "bf16", b, 4)
        assert ((out.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()


def test_graph_of_an_earlier_batch_does_nothing(mk):
    # a captured call whose chunk was updated since: reported, and nothing is written
    D, batch, chunk = make(mk, "g8", "bf16", "behind_cache", seed=4)
    pool = cu.make_pool("bf16", batch.num_pages, 4, 128, 9).cuda()
    was = pool.clone()
    qkv = cu.normal((batch.rows, 4, 10, 128), 3).bfloat16().cuda()
    q = torch.full((batch.rows, 32, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out, back = q.clone(), torch.full((sum(batch.total), 4, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk.append(qkv, pool, q)
        chunk.attend(q, pool, out)
        chunk.read(pool, back)
    for cached, new in (([3], [1]), ([0] * 40, [70] * 40)):
        b = cu.Batch(cached, new, spare=0)
        table = [p % batch.num_pages if p >= 0 else -1 for p in b.flat] if len(cached) == 1 else None
        if table is None:   # far more pages than the pool has: only the tables grow
            big = mk.Chunk(D, "bf16", b.num_pages, [1], [1], [0], 1)
            big.update(b.cached, b.new, b.flat, b.width)
            big.close()
            continue
        chunk.update(cached, new, table, b.width)
        graph.replay()
        assert chunk.sync() == mk.MK_ERR_INVALID
        assert torch.equal(pool, was) and (q == 5).all() and (out == 5).all() and (back == 5).all()
    chunk.update(batch.cached, batch.new, batch.flat, batch.width)
    assert chunk.sync() == mk.MK_OK
    chunk.append(qkv, pool, q)
    chunk.attend(q, pool, out)
    assert chunk.sync() == mk.MK_OK
    ref, mag = cu.attend(q.cpu(), pool.cpu(), "bf16", batch, 4)
    assert ((out.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()


def test_attend_onto_its_queries(mk):
    for lens in ("prompts", "long_one_token"):
        D, batch, chunk = make(mk, "g8", "bf16", lens)
        pool = cu.make_pool("bf16", batch.num_pages, 4, 128, 3).cuda()
        q = cu.normal((batch.rows, 32, 128), 3).bfloat16().cuda()
        out = torch.empty_like(q)
        chunk.attend(q, pool, out)
        chunk.attend(q, pool, q)
        assert chunk.sync() == mk.MK_OK and torch.equal(q, out)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_beyond_4_gb(mk, kv):
    # pages at both ends of a pool of more than 2^32 bytes
    D = cu.dims(8, 8, 128)
    d = 128 + (kv == "e4m3")
    pages = (1 << 32) // (8 * 2 * d * 16 * (1 if kv == "e4m3" else 2)) + 50
    pool = torch.zeros(pages, 8, 2, d, 16, dtype=torch.uint8 if kv == "e4m3" else torch.bfloat16, device="cuda")
    batch = cu.Batch([70], [5], seed=1, spare=0)
    far = [pages - 1 - 2 * p if p % 2 else p for p in batch.flat]
    chunk = mk.Chunk(D, kv, pages, [0], [75], far, batch.width)
    x = cu.normal((75, 8, 3, 128), 4).bfloat16().cuda()
    q = torch.empty(75, 8, 128, dtype=torch.bfloat16, device="cuda")
    chunk.append(x, pool, q)
    out, back = torch.empty_like(q), torch.empty(75, 8, 2, 128, dtype=torch.bfloat16, device="cuda")
    chunk.attend(q, pool, out)
    chunk.read(pool, back)
    assert chunk.sync() == mk.MK_OK
    near = torch.zeros(batch.num_pages, 8, 2, d, 16, dtype=pool.dtype)
    for mine, there in zip(batch.flat, far):
        near[mine] = pool[there].cpu()
    whole = cu.Batch([0], [75], spare=0)
    whole.table, whole.num_pages = batch.table, batch.num_pages
    ref, mag = cu.attend(q.cpu(), near, kv, whole, 8)
    assert ((out.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()
    assert torch.equal(back.cpu(), cu.rows_of(near, kv, whole, 0).bfloat16())
    assert (back.cpu()[:, :, 1].double() - x.cpu()[:, :, 2].double()).abs().max() <= 2.0 ** -4 * 6


def test_same_bits_every_time(mk):
    D, batch, chunk = make(mk, "g8", "e4m3", ([4000, 9000, 100], [5, 1, 200]))
    pool = cu.make_pool("e4m3", batch.num_pages, 4, 128, 3).cuda()
    q = cu.normal((batch.rows, 32, 128), 3).bfloat16().cuda()
    outs = [torch.empty_like(q) for _ in range(4)]
    for o in outs:
        chunk.attend(q, pool, o)
    assert chunk.sync() == mk.MK_OK
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_refused_tensors(mk):
    D, batch, chunk = make(mk, "g8", "bf16", "one_token")
    pool = torch.zeros(batch.num_pages, 4, 2, 128, 16, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 32, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (q.cpu(), q.float(), q[:, :31], q.new_zeros(1, 128, 32).transpose(1, 2)):
        with pytest.raises(ValueError):
            chunk.attend(bad, pool, q)
    with pytest.raises(ValueError):
        chunk.attend(q, pool[:-1], q)
    with pytest.raises(ValueError):
        chunk.append(torch.zeros(1, 4, 10, 128, device="cuda").double(), pool, q)
    with pytest.raises(ValueError):
        chunk.append(torch.zeros(1, 4, 10, 128, device="cuda"), pool)
    with pytest.raises(mk.MkError) as e:   # rows 10 bytes apart from 16-byte steps
        D1, b1, c1 = make(mk, "g8", "bf16", ([0], [2]))
        wide = torch.zeros(2, 5125, device="cuda")[:, :5120]
        c1.append(wide, torch.zeros(b1.num_pages, 4, 2, 128, 16, dtype=torch.bfloat16, device="cuda"), q.new_zeros(2, 32, 128))
    assert e.value.code == mk.MK_ERR_INVALID
    x = torch.zeros(4, 100, device="cuda")
    with pytest.raises(mk.MkError):        # the output starts inside the input
        mk.probs(x[:2], 1.0, x[1:3])


# ---- a run of them, as a server uses them ----

def test_prompt_layer_by_pieces_equals_whole(mk):
    # one layer's cache filled and attended in one chunk, and in pieces of several sizes: the same values
    D = cu.dims(32, 4, 128)
    n = 150
    x = cu.normal((n, 4, 10, 128), 4).bfloat16().cuda()
    results = []
    for cuts in ([n], [1, 15, 17, 64, 53], [128, 22]):
        batch = cu.Batch([0], [n], seed=1)
        pool = torch.zeros(batch.num_pages, 4, 2, 128, 16, dtype=torch.bfloat16, device="cuda")
        out, at = torch.empty(n, 32, 128, dtype=torch.bfloat16, device="cuda"), 0
        for c in cuts:
            chunk = mk.Chunk(D, "bf16", batch.num_pages, [at], [c], batch.flat, batch.width)
            q = torch.empty(c, 32, 128, dtype=torch.bfloat16, device="cuda")
            chunk.append(x[at:at + c], pool, q)
            chunk.attend(q, pool, out[at:at + c])
            assert chunk.sync() == mk.MK_OK
            at += c
        results.append((pool.cpu(), out.cpu()))
    for pool, out in results[1:]:
        assert torch.equal(pool, results[0][0])
        # weights rounded against another running maximum: one rounding of the weights and one of the result each
        assert ((out.double() - results[0][1].double()).abs() <= 4 * cu.BF16 * 1.5).all()


def tiny_model():
    return dataclasses.replace(synth.TINY, n_layers=1), 3


def test_appended_prompt_feeds_the_decode_step(mk):
    # a one-layer model's prompt enters its cache through mk_chunk_append; the
    # decode step continues from it as from its own prefill rows
    D, seed = tiny_model()
    model = DeviceModel(D, seed)
    w = model.weights()
    prompt = [(37 * i + 11) % D.vocab for i in range(8)]
    pages, width = kv_pages_needed(D, [16], 2) + 2, 3
    table = [2, 0, 1]

    def pools():
        return [torch.zeros(pages, D.n_kv_heads, 2, D.head_dim, 16, dtype=torch.bfloat16, device="cuda")]

    a, b = pools(), pools()
    tok = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    first = mk.Plan(D, w, a, [0], table, width, max_batch=8)
    first.update_rows(list(range(8)), table * 8, width, [0] * 8)
    nxt = torch.empty(8, dtype=torch.int32, device="cuda")
    assert first.step(tok, nxt) == mk.MK_OK and first.sync() == mk.MK_OK
    # the same rows by hand: embedding, norm and projection in fp32, then the append
    x = w["embed"][tok.long()].float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + D.rms_eps) * w["attn_norm"][0].float()
    qkv = (x @ w["wqkv"][0].float().T).view(8, D.n_kv_heads, D.group + 2, D.head_dim)
    chunk = mk.Chunk(D, "bf16", pages, [0], [8], table, width)
    q = torch.empty(8, D.n_q_heads, D.head_dim, dtype=torch.bfloat16, device="cuda")
    chunk.append(qkv, b[0], q)
    assert chunk.sync() == mk.MK_OK
    ka, kb = (p[0][table[0], :, :, :, :8].float() for p in (a, b))
    # both round fp32 sums of other orders to bf16: at most a step apart
    assert ((ka - kb).abs() <= 2.01 * cu.BF16 * ka.abs() + 1e-4).all()
    logits = []
    for pool in (a, b):
        plan = mk.Plan(D, w, pool, [8], table, width)
        lg, n1 = torch.empty(1, D.vocab, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        assert plan.step(nxt[7:8].contiguous(), n1, lg) == mk.MK_OK and plan.sync() == mk.MK_OK
        logits.append(lg.double())
        plan.close()
    first.close()
    assert float((logits[0] - logits[1]).norm() / logits[0].norm()) <= 1e-2


def test_drafted_tokens_through_plan_probs_and_verify(mk):
    # speculative greedy decoding: the target checks drafts as chunk rows, and what it
    # accepts is its own greedy continuation, whatever is drafted
    D, seed = dataclasses.replace(synth.TINY), 3
    model = DeviceModel(D, seed)
    w, k, steps = model.weights(), 3, 12
    width, pages = 4, 8
    table = [5, 1, 6, 0]

    def pools():
        return [torch.zeros(pages, D.n_kv_heads, 2, D.head_dim, 16, dtype=torch.bfloat16, device="cuda")
                for _ in range(D.n_layers)]

    plan = mk.Plan(D, w, pools(), [0], table, width)
    tok = torch.tensor([7], dtype=torch.int32, device="cuda")
    plain = [7]
    for _ in range(steps):
        nxt = torch.empty(1, dtype=torch.int32, device="cuda")
        assert plan.step(tok, nxt) == mk.MK_OK and plan.sync() == mk.MK_OK
        plain.append(int(nxt))
        tok = nxt
    plan.close()
    plan = mk.Plan(D, w, pools(), [0], table, width, max_batch=8)
    got, turn = [7], 0
    while len(got) <= steps:
        right = plain[len(got):len(got) + k]
        drafts = [x if (turn + i) % 3 else (x + 1) % D.vocab for i, x in enumerate(right)] + [0] * (k - len(right))
        turn += 1
        at = len(got) - 1
        plan.update_rows(list(range(at, at + k + 1)), table * (k + 1), width, [0] * (k + 1))
        rows = torch.tensor([got[-1]] + drafts, dtype=torch.int32, device="cuda")
        logits = torch.empty(k + 1, D.vocab, device="cuda")
        nxt = torch.empty(k + 1, dtype=torch.int32, device="cuda")
        assert plan.step(rows, nxt, logits) == mk.MK_OK
        target = torch.empty(k + 1, D.vocab, device="cuda")
        mk.probs(logits, 0.0, target)
        tokens, accepted = torch.empty(1, k + 1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        mk.verify(target.view(1, k + 1, -1), None, rows[1:].view(1, k), torch.rand(1, k, device="cuda"),
                  torch.rand(1, device="cuda"), tokens, accepted)
        assert plan.sync() == mk.MK_OK
        n = int(accepted)
        new = tokens[0, :n + 1].tolist()
        assert (tokens[0, n + 1:] == -1).all() and new[:n] == drafts[:n]
        got += new
    plan.close()
    assert got[:steps + 1] == plain


def test_beside_decode_steps_on_another_stream(mk):
    # a chunk's calls on one stream while decode steps run on another: the results of either alone
    D, seed = synth.TINY, 3
    w, width, pages, steps = DeviceModel(D, seed).weights(), 3, 6, 12
    tokens = []
    C, batch, chunk = make(mk, "g8", "e4m3", ([4000, 9000, 100], [5, 1, 200]))
    pool = cu.make_pool("e4m3", batch.num_pages, 4, 128, 3).cuda()
    q = cu.normal((batch.rows, 32, 128), 3).bfloat16().cuda()
    alone = torch.empty_like(q)
    chunk.attend(q, pool, alone)
    assert chunk.sync() == mk.MK_OK
    for beside in (False, True):
        pools = [torch.zeros(pages, D.n_kv_heads, 2, D.head_dim, 16, dtype=torch.bfloat16, device="cuda")
                 for _ in range(D.n_layers)]
        plan = mk.Plan(D, w, pools, [0], [4, 1, 2], width)
        out = torch.zeros(steps + 1, 1, dtype=torch.int32, device="cuda")
        out[0] = 7
        outs = [torch.empty_like(q) for _ in range(steps)]
        torch.cuda.synchronize()
        one, two = torch.cuda.Stream(), torch.cuda.Stream()
        for i in range(steps):
            assert plan.step(out[i], out[i + 1], stream=one) == mk.MK_OK
            if beside:
                chunk.attend(q, pool, outs[i], stream=two)
        assert plan.sync(one) == mk.MK_OK and chunk.sync(two) == mk.MK_OK
        tokens.append(out.tolist())
        assert not beside or all(torch.equal(alone, o) for o in outs)
        plan.close()
    assert tokens[0] == tokens[1]


def test_nothing_new(mk):
    # no rows: the calls do nothing, and what is cached can be read
    D, batch, chunk = make(mk, "g8", "bf16", ([20, 0], [0, 0]))
    pool = cu.make_pool("bf16", batch.num_pages, 4, 128, 3)
    none = torch.empty(0, 32, 128, dtype=torch.bfloat16, device="cuda")
    chunk.append(torch.empty(0, 4, 10, 128, device="cuda"), pool.cuda(), none)
    chunk.attend(none, pool.cuda(), none)
    out = torch.empty(20, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    chunk.read(pool.cuda(), out)
    assert chunk.sync() == mk.MK_OK
    assert torch.equal(out.cpu(), cu.rows_of(pool, "bf16", batch, 0).bfloat16())
    mk.probs(torch.empty(0, 50, device="cuda"), 1.0, torch.empty(0, 50, device="cuda"))


# ---- graphs of an earlier batch, once more ----

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_graph_of_an_earlier_batch_over_other_tables(mk, kv):
    # the captured chunk itself gets batches whose tables, angles and split rows lie where the captured calls' join
    # records were (a page table of 512 entries puts those at byte 10272 of the chunk's memory)
    D, width, pages = cu.dims(32, 4, 128), 512, 600
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
    table = lambda n, first=0: order[first:first + n] + [-1] * (width - n)
    chunk = mk.Chunk(D, kv, pages, [8191], [1], table(512), width)
    assert chunk.info()["joined_rows"] == 32
    pool = cu.make_pool(kv, pages, 4, 128, 3)
    gpool = pool.cuda()
    full = lambda *shape: torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda")
    qkv, q, out, back = cu.normal((1, 4, 10, 128), 4).bfloat16().cuda(), full(1, 32, 128), full(1, 32, 128), full(8192, 4, 2, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk.append(qkv, gpool, q)
        chunk.attend(q, gpool, out)
        chunk.read(gpool, back)
    for cached, new in (([0], [300]), ([7], [1]), ([100, 3000], [2, 40]), ([0, 0, 0], [1100, 1, 90])):
        tables, at = [], 0
        for c, n in zip(cached, new):
            tables += table(-(-(c + n) // cu.PAGE), at)
            at += -(-(c + n) // cu.PAGE)
        chunk.update(cached, new, tables, width)
        graph.replay()
        assert chunk.sync() == mk.MK_ERR_INVALID
        assert torch.equal(gpool.cpu().view(torch.uint8), pool.view(torch.uint8))
        assert (q == 5).all() and (out == 5).all() and (back == 5).all()
        # and the new batch is served
        chunk.update(cached, new, tables, width)
        b = cu.Batch(cached, new)
        b.table = [tables[i * width:(i + 1) * width] for i in range(len(new))]
        q2 = cu.normal((b.rows, 32, 128), 6).bfloat16()
        out2 = torch.empty(b.rows, 32, 128, dtype=torch.bfloat16, device="cuda")
        chunk.attend(q2.cuda(), gpool, out2)
        assert chunk.sync() == mk.MK_OK
        ref, mag = cu.attend(q2, pool, kv, b, 4)
        assert ((out2.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()


# ---- calls that follow one another without a wait ----

def stored(kv, x):
    """What a pool gives back for rows x, as bf16."""
    if kv == "bf16":
        return x.bfloat16()
    code, k = cu.quantise(x.float())
    return torch.ldexp(code.view(torch.float8_e4m3fn).double(), k.double().unsqueeze(-1)).bfloat16()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", ["drafts", "behind_cache"])
def test_chain_on_one_stream_reads_what_was_just_written(mk, kv, lens, captured):
    # read, append and attend over the same slots and buffers turn after turn, nothing waited for; no rotation, so
    # that queries and cached rows are known to the last bit
    D, batch, chunk = make(mk, "g8", kv, lens, seed=4, theta=0.0)
    turns, stream = 6, torch.cuda.Stream()
    pool = cu.make_pool(kv, batch.num_pages, 4, 128, 9)
    x = [cu.normal((batch.rows, 4, 10, 128), 50 + i).bfloat16() for i in range(turns)]
    gpool, gx = pool.cuda(), [t.cuda() for t in x]
    page, slot = (t.cuda() for t in batch.new_slots())
    qkv, q = torch.empty_like(gx[0]), torch.empty(batch.rows, 32, 128, dtype=torch.bfloat16, device="cuda")
    out, back = torch.empty_like(q), torch.empty(sum(batch.total), 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    again = torch.empty_like(back)

    def calls():
        chunk.read(gpool, back)
        chunk.append(qkv, gpool, q)
        chunk.attend(q, gpool, out)
        chunk.read(gpool, again)

    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(stream):
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                calls()
        for i in range(turns):
            qkv.copy_(gx[i])
            if i % 2:      # what a call that wrote nothing would leave
                q.fill_(math.nan)
                gpool[page, :, :, :, slot] = 3
            graph.replay() if captured else calls()
            got.append([t.clone() for t in (q, out, back, again)])
    assert chunk.sync(stream) == mk.MK_OK
    page, slot = page.cpu(), slot.cpu()
    rows = torch.cat([torch.arange(sum(batch.total[:b]) + c, sum(batch.total[:b]) + t)
                      for b, (c, t) in enumerate(zip(batch.cached, batch.total))])
    for i in range(turns):
        gq, gout, gback, gagain = (t.cpu() for t in got[i])
        assert torch.equal(gq, x[i][:, :, :8].flatten(1, 2))
        assert torch.equal(gagain[rows], stored(kv, x[i][:, :, 8:]))
        if i and not i % 2:
            assert torch.equal(gback, got[i - 1][3].cpu())
        code = x[i][:, :, 8:]
        if kv == "bf16":
            pool[page, :, :, :, slot] = code
        else:
            c, k = cu.quantise(code.float())
            pool[page, :, :, :, slot] = torch.cat([c, (k + 127).to(torch.uint8).unsqueeze(-1)], -1)
        ref, mag = cu.attend(gq, pool, kv, batch, 4)
        assert ((gout.double() - ref).abs() <= cu.attend_bound(ref, mag)).all()
        assert torch.equal(gagain, torch.cat([cu.rows_of(pool, kv, batch, b) for b in range(len(batch.new))]).bfloat16())


@pytest.mark.parametrize("rows,vocab", [(4, 32000), (48, 2051)])
def test_probabilities_in_place_then_verified_without_a_wait(mk, rows, vocab):
    # logits become probabilities in their own buffer, which the verification reads; the next logits come into the same
    k, turns = 3, 5
    b = rows // (k + 1)
    logits = [cu.normal((rows, vocab), 7 + i, 2.0).cuda() for i in range(turns)]
    near = [cu.normal((b * k, vocab), 70 + i, 2.0).cuda() for i in range(turns)]
    g = torch.Generator().manual_seed(1)
    x = torch.randint(0, vocab, (b, k), generator=g).int().cuda()
    u, r = torch.rand(b, k, generator=g).cuda() * 2, torch.rand(b, generator=g).cuda()
    t, d = torch.empty(rows, vocab, device="cuda"), torch.empty(b * k, vocab, device="cuda")
    tokens, accepted = torch.empty(b, k + 1, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(turns):
        t.copy_(logits[i])
        d.copy_(near[i])
        mk.probs(t, 0.8, t)
        mk.probs(d, 0.8, d)
        mk.verify(t.view(b, k + 1, vocab), d.view(b, k, vocab), x, u, r, tokens, accepted)
        got.append([y.clone() for y in (t, d, tokens, accepted)])
    for i in range(turns):
        gt, gd, gtok, gacc = (y.cpu() for y in got[i])
        for y, l in ((gt, logits[i]), (gd, near[i])):
            ref = torch.softmax(l.cpu().double() / torch.tensor(0.8, dtype=torch.float32).double(), -1)
            assert ((y.double() - ref).abs() <= probs_bound(ref)).all()
        ref_t, ref_a = cu.verify(gt.view(b, k + 1, vocab), gd.view(b, k, vocab), x.cpu(), u.cpu(), r.cpu())
        assert torch.equal(gacc, torch.from_numpy(ref_a)) and torch.equal(gtok, torch.from_numpy(ref_t))


# ---- values at the ends of the 8-bit pool's range ----

def test_attend_reads_8_bit_vectors_of_the_smallest_scale(mk):
    # keys and values of 2^-121: their scale is 2^-127, which no normal bf16 number holds; queries of 2^121 bring
    # the scores back to a few units
    n, D = 5, cu.dims(8, 2, 128, 0.0)
    batch = cu.Batch([0], [n], seed=2)
    chunk = mk.Chunk(D, "e4m3", batch.num_pages, batch.cached, batch.new, batch.flat, batch.width)
    x = cu.normal((n, 2, 6, 128), 1)
    x[:, :, :4] *= 2.0 ** 121
    x[:, :, 4:] *= 2.0 ** -121
    pool = torch.zeros(batch.num_pages, 2, 2, 129, 16, dtype=torch.uint8, device="cuda")
    q = torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    chunk.append(x.cuda(), pool, q)
    chunk.attend(q, pool, out)
    assert chunk.sync() == mk.MK_OK
    page, slot = batch.new_slots()
    assert (pool.cpu()[page, :, :, -1, slot] == 0).all()
    ref, mag = cu.attend(q.cpu(), pool.cpu(), "e4m3", batch, 2)
    # attend_bound without its absolute part, and what a product or a sum may lose below fp32's normal numbers: one
    # 2^-126 for each of the row's keys (which is why there are few)
    bound = cu.BF16 * ref.abs() + (cu.BF16 + 2.0 ** -13) * mag + n * 2.0 ** -126
    assert ((out.cpu().double() - ref).abs() <= bound).all()
    assert (ref.abs() > bound).double().mean() > 0.8   # zeros would not do
    back = torch.empty(n, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    chunk.read(pool, back)
    assert torch.equal(back.cpu(), cu.rows_of(pool.cpu(), "e4m3", batch, 0).bfloat16())


# ---- updates ----

def test_updates_do_not_wait_for_the_stream(mk):
    # batches of 1000 requests (tables of more than 64 KB) behind work of a tenth of a second: the first two updates
    # return before it ends, the third takes the first one's memory, and every call sees its own batch
    D, n = cu.dims(8, 1, 64, 0.0), 1000
    batches = [cu.Batch([40 + 16 * i] * n, [1 + i] * n, seed=i) for i in range(3)]
    pages = max(b.num_pages for b in batches)
    pool = cu.make_pool("bf16", pages, 1, 64, 3)
    gpool, width = pool.cuda(), max(b.width for b in batches)
    flat = [[p for row in b.table for p in row + [-1] * (width - b.width)] for b in batches]
    first = max(batches, key=lambda b: b.rows)
    chunk = mk.Chunk(D, "bf16", pages, first.cached, first.new, flat[2], width)
    for _ in range(2):      # both buffers and the device's memory have their size
        chunk.update(first.cached, first.new, flat[2], width)
    q = [cu.normal((b.rows, 8, 64), 5 + i).bfloat16() for i, b in enumerate(batches)]
    gq, out = [t.cuda() for t in q], [torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in q]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    asleep = torch.cuda.Event()
    asleep.record()
    for i, b in enumerate(batches):
        chunk.update(b.cached, b.new, flat[i], width)
        assert i == 2 or not asleep.query()
        chunk.attend(gq[i], gpool, out[i])
    assert chunk.sync() == mk.MK_OK
    for i, b in enumerate(batches):
        ref, mag = cu.attend(q[i], pool, "bf16", b, 1)
        assert ((out[i].cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()


# ---- many rows: clusters of 1 to 8 blocks, every number of passes, the rows fetched ahead ----

@pytest.mark.parametrize("vocab", [8, 9, 10, 11, 12, 13, 16, 17])
def test_probs_many_rows_of_a_few(mk, vocab):
    # more rows than run at once: each block fetches a later row's segment ahead, or nothing of one too short
    rows = 700
    for stride in (vocab, vocab + 3):
        x = cu.normal((rows, stride), vocab, 3.0)
        ref = torch.softmax(x[:, :vocab].double(), -1)
        out = torch.full((rows + 1, vocab), 7.0, device="cuda")
        mk.probs(x.cuda()[:, :vocab], 1.0, out[:-1])
        got = out.cpu()
        assert ((got[:-1].double() - ref).abs() <= probs_bound(ref)).all() and (got[-1] == 7).all()


@pytest.mark.parametrize("rows,vocab,stride", [
    (9, 16385, 16385), (10, 2049, 2050), (10, 8193, 8193), (10, 16385, 16390), (40, 32769, 32769), (320, 9001, 9003),
    (160, 32000, 32000), (40, 151935, 151935), (40, 151936, 151936), (10, 151936, 151939), (10, 230000, 230001),
    (9, 393216, 393216), (10, 393213, 393213), (10, 393214, 393217), (10, 393216, 393216), (12, 393212, 393215)])
def test_probs_many_rows(mk, rows, vocab, stride):
    for temperature in (0.7, 0.0):
        x = cu.normal((rows, stride), vocab % 1000 + rows, 3.0)
        x[rows // 2, vocab - 1] = 50.0     # (its last element leads one row)
        out = torch.full((rows + 1, vocab), 7.0, device="cuda")
        mk.probs(x.cuda()[:, :vocab], temperature, out[:-1])
        got = out.cpu()
        assert (got[-1] == 7).all()
        if temperature:
            ref = torch.softmax(x[:, :vocab].double() / torch.tensor(temperature, dtype=torch.float32).double(), -1)
            assert ((got[:-1].double() - ref).abs() <= probs_bound(ref)).all()
        else:
            ref = torch.zeros(rows, vocab).scatter_(1, x[:, :vocab].argmax(1, keepdim=True), 1.0)
            assert torch.equal(got[:-1], ref)


@pytest.mark.parametrize("b,k,vocab", [(9, 2, 151936), (10, 1, 151935), (33, 2, 50257), (40, 3, 9001), (12, 2, 32000),
                                       (10, 1, 230001), (10, 0, 393216), (11, 1, 393215), (160, 1, 2052)])
def test_verify_many_requests(mk, b, k, vocab):
    t, d, x, u, r = draws(b, k, vocab, vocab + b)
    check_verify(mk, t, d if k else None, x, u, r)
    if k:
        u[::2] = 2.0                       # every other request's first draft is refused: a row of differences
        check_verify(mk, t, d, x, u, r)
        check_verify(mk, t, None, x, u, r)


@pytest.mark.parametrize("b", [3, 12])
def test_verify_rows_that_are_not_16_byte_aligned(mk, b):
    # a vocabulary of whole 16-byte pieces in buffers that start 4 bytes into one
    t, d, x, u, r = draws(b, 2, 4096, 31)
    u[0, 0] = 2.0

    def shifted(y):
        flat = torch.empty(y.numel() + 1, device="cuda")[1:]
        flat.copy_(y.flatten())
        return flat.view(y.shape)

    tokens, accepted = torch.empty(b, 3, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
    ref_t, ref_a = cu.verify(t, d, x, u, r)
    for gt, gd in ((shifted(t), d.cuda()), (t.cuda(), shifted(d)), (shifted(t), shifted(d))):
        assert (gt.data_ptr() | gd.data_ptr()) % 16 == 4
        mk.verify(gt, gd, x.cuda(), u.cuda(), r.cuda(), tokens, accepted)
        assert torch.equal(tokens.cpu(), torch.from_numpy(ref_t)) and torch.equal(accepted.cpu(), torch.from_numpy(ref_a))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_into_rows_between_sectors(mk, kv):
    # an output that is 16- but not 32-byte aligned, whole and split rows
    for lens in ("prompts", "long_one_token"):
        D, batch, chunk = make(mk, "g2d64", kv, lens, seed=7)
        pool = cu.make_pool(kv, batch.num_pages, 2, 64, 3).cuda()
        q = cu.normal((batch.rows, 4, 64), 3).bfloat16().cuda()
        out = torch.empty_like(q)
        flat = torch.full((q.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        odd = flat[8:-8].view(q.shape)
        assert odd.data_ptr() % 32 == 16
        chunk.attend(q, pool, out)
        chunk.attend(q, pool, odd)
        assert chunk.sync() == mk.MK_OK
        assert torch.equal(odd, out) and (flat[:8] == 7).all() and (flat[-8:] == 7).all()


def test_attend_over_a_large_8_bit_pool(mk):
    # 139 GB of pages (as many as a bf16 pool of 256 GB has), the batch's at its end: the same bits as in a small pool
    D = cu.dims(16, 8, 128)
    pages = (1 << 31) // (8 * 2 * 32) + 96
    if torch.cuda.mem_get_info()[0] < 170 << 30:
        pytest.skip("needs 170 GB of free memory")
    batch = cu.Batch([0], [75], seed=1, spare=0)
    x = cu.normal((75, 8, 4, 128), 4).bfloat16().cuda()
    results = []
    for size, table in ((batch.num_pages, batch.flat), (pages, [pages - 1 - p for p in batch.flat])):
        pool = torch.empty(size, 8, 2, 129, 16, dtype=torch.uint8, device="cuda")
        for p in table:
            pool[p].zero_()
        chunk = mk.Chunk(D, "e4m3", size, [0], [75], table, batch.width)
        q = torch.empty(75, 16, 128, dtype=torch.bfloat16, device="cuda")
        out, back = torch.empty_like(q), torch.empty(75, 8, 2, 128, dtype=torch.bfloat16, device="cuda")
        chunk.append(x, pool, q)
        chunk.attend(q, pool, out)
        chunk.read(pool, back)
        assert chunk.sync() == mk.MK_OK
        results.append((out, back))
        del pool
        torch.cuda.empty_cache()
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert results[0][0].float().abs().max() > 0.1
    # a bf16 pool of as many pages is refused before anything is launched
    chunk = mk.Chunk(D, "bf16", pages, [0], [75], batch.flat, batch.width)
    q = results[0][0]
    at = [ctypes.c_void_p(t.data_ptr()) for t in (q, x, torch.empty_like(q))]
    assert mk.lib().mk_chunk_attend(chunk.h, *at, None) == mk.MK_ERR_UNSUPPORTED


# ---- buffers that overlap ----

def test_refused_overlaps(mk):
    D, batch, chunk = make(mk, "g2d64", "bf16", ([30], [4]))
    pages, n = batch.num_pages, 4
    whole = torch.zeros(pages * 2 * 2 * 64 * 16 + 8192, dtype=torch.bfloat16, device="cuda")
    was = whole.clone()
    pool = whole[:-8192].view(pages, 2, 2, 64, 16)
    edge = lambda size, shape: whole[-8192 - 8:][:size].view(shape)        # its first 16 bytes are the pool's last
    rows, q = torch.zeros(n, 2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 4, 64, dtype=torch.bfloat16, device="cuda")
    both = torch.zeros(n * 512 + n * 256, dtype=torch.bfloat16, device="cuda")
    bad = [lambda: chunk.append(edge(n * 512, (n, 2, 4, 64)), pool, q), lambda: chunk.append(rows, pool, edge(n * 256, (n, 4, 64))),
           lambda: chunk.append(both[:n * 512].view(n, 2, 4, 64), pool, both[n * 512 - 8:][:n * 256].view(n, 4, 64)),
           lambda: chunk.attend(q, pool, edge(n * 256, (n, 4, 64))),
           lambda: chunk.attend(both[:n * 256].view(n, 4, 64), pool, both[8:][:n * 256].view(n, 4, 64)),
           lambda: chunk.read(pool, whole[8:][:34 * 256].view(34, 2, 2, 64))]
    for call in bad:
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.code == mk.MK_ERR_INVALID
    assert torch.equal(whole, was)
    # side by side is apart
    chunk.append(both[:n * 512].view(n, 2, 4, 64), pool, both[n * 512:].view(n, 4, 64))
    chunk.attend(whole[-8192:][:n * 256].view(n, 4, 64), pool, whole[-8192 + n * 256:][:n * 256].view(n, 4, 64))
    assert chunk.sync() == mk.MK_OK


def test_verify_one_request_in_its_drafts_place(mk):
    t, d, x, u, r = draws(1, 4, 5000, 3)
    for u0 in (0.0, 2.0):
        u[0, 2] = u0
        ref_t, ref_a = cu.verify(t, d, x, u, r)
        tokens, accepted = torch.full((1, 5), 9, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        tokens[0, :4] = x[0].cuda()
        mk.verify(t.cuda(), d.cuda(), tokens[:, :4], u.cuda(), r.cuda(), tokens, accepted)
        assert torch.equal(tokens.cpu(), torch.from_numpy(ref_t)) and torch.equal(accepted.cpu(), torch.from_numpy(ref_a))


# ---- captures, and sizes at their limits ----

FIRST_CALLS = """
import sys, torch
sys.path.insert(0, {root!r})
from tests import chunk_util as cu
from persistent_moe_decode_02_gb300 import mk
D, batch = cu.dims(8, 2, 128), cu.Batch([5000], [3], seed=1)
chunk = mk.Chunk(D, "bf16", batch.num_pages, batch.cached, batch.new, batch.flat, batch.width)
pool = cu.make_pool("bf16", batch.num_pages, 2, 128, 3).cuda()
qkv = cu.normal((3, 2, 6, 128), 4).bfloat16().cuda()
new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
logits = cu.normal((3, 40000), 5).cuda()
x, u, r = new(1, 2, t=torch.int32), torch.full((1, 2), 2.0, device="cuda"), torch.full((1,), 0.5, device="cuda")

def calls():
    q, out, back = new(3, 8, 128), new(3, 8, 128), new(5003, 2, 2, 128)
    p, tokens, accepted = torch.zeros_like(logits), new(1, 3, t=torch.int32), new(1, t=torch.int32)
    chunk.append(qkv, pool, q)
    chunk.attend(q, pool, out)
    chunk.read(pool, back)
    mk.probs(logits, 0.9, p)
    mk.verify(p.view(1, 3, -1), None, x, u, r, tokens, accepted)
    return q, out, back, p, tokens, accepted

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
assert chunk.sync() == mk.MK_OK
want = calls()
assert chunk.sync() == mk.MK_OK
assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[1].abs().max() > 0 and int(want[4][0, 0]) > 0
print("the same")
"""


def test_first_calls_of_a_process_inside_a_capture(mk):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "the same" in run.stdout, run.stderr[-2000:]


def test_capture_over_two_streams(mk):
    # a captured fork: two chunks' calls on streams of their own, joined, and a call after the join
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    work = []
    for lens, seed in (("drafts", 4), ("behind_cache", 6)):
        D, b, c = make(mk, "g8", "bf16", lens, seed=seed, theta=0.0)
        work.append(dict(b=b, c=c, pool=cu.make_pool("bf16", b.num_pages, 4, 128, 9).cuda(),
                         qkv=torch.zeros(b.rows, 4, 10, 128, dtype=torch.bfloat16, device="cuda"),
                         q=torch.empty(b.rows, 32, 128, dtype=torch.bfloat16, device="cuda"),
                         out=torch.empty(b.rows, 32, 128, dtype=torch.bfloat16, device="cuda")))
    back = torch.empty(sum(work[1]["b"].total), 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        two.wait_stream(one)
        for w, s in zip(work, (one, two)):
            w["c"].append(w["qkv"], w["pool"], w["q"], stream=s)
            w["c"].attend(w["q"], w["pool"], w["out"], stream=s)
        one.wait_stream(two)
        work[1]["c"].read(work[1]["pool"], back, stream=one)
    for turn in range(3):
        x = [cu.normal(w["qkv"].shape, 20 + turn + i).bfloat16() for i, w in enumerate(work)]
        with torch.cuda.stream(one):
            for w, t in zip(work, x):
                w["qkv"].copy_(t)
            graph.replay()
        assert all(w["c"].sync(one) == mk.MK_OK for w in work)
        for w, t in zip(work, x):
            assert torch.equal(w["q"].cpu(), t[:, :, :8].flatten(1, 2))
            ref, mag = cu.attend(w["q"].cpu(), w["pool"].cpu(), "bf16", w["b"], 4)
            assert ((w["out"].cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()
        b = work[1]["b"]
        assert torch.equal(back.cpu(), torch.cat([cu.rows_of(work[1]["pool"].cpu(), "bf16", b, i) for i in range(2)]).bfloat16())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_the_largest_batch(mk, kv):
    # 65535 requests of one new token behind 0 to 3 cached ones; one more is refused
    n, D = 65535, cu.dims(2, 1, 64, 0.0)
    cached = torch.arange(n) % 4
    table = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    chunk = mk.Chunk(D, kv, n, cached.numpy(), torch.ones(n, dtype=torch.int64).numpy(), table.numpy(), 1)
    pool = cu.make_pool(kv, n, 1, 64, 5)
    x = cu.normal((n, 1, 4, 64), 6).bfloat16()
    gpool, q = pool.cuda(), torch.empty(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, back = torch.empty_like(q), torch.empty(int(cached.sum()) + n, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    chunk.append(x.cuda(), gpool, q)
    chunk.attend(q, gpool, out)
    chunk.read(gpool, back)
    assert chunk.sync() == mk.MK_OK
    assert torch.equal(q.cpu(), x[:, 0, :2])
    rows = cu.values(gpool.cpu(), kv)[table][:, 0].permute(0, 3, 1, 2)[:, :4]         # [n, 4 slots, 2, 64]
    assert torch.equal(rows[torch.arange(n), cached].bfloat16(), stored(kv, x[:, 0, 2:]))
    seen = torch.arange(4) <= cached.unsqueeze(1)
    assert torch.equal(back.cpu(), rows[seen].unsqueeze(1).bfloat16())
    s = torch.einsum("nhd,ntd->nht", q.cpu().double(), rows[:, :, 0]) / 8
    p = torch.softmax(s.masked_fill(~seen.unsqueeze(1), -math.inf), -1)
    ref, mag = torch.einsum("nht,ntd->nhd", p, rows[:, :, 1]), torch.einsum("nht,ntd->nhd", p, rows[:, :, 1].abs())
    assert ((out.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()
    with pytest.raises(mk.MkError) as e:
        mk.Chunk(D, kv, n + 1, [0] * (n + 1), [1] * (n + 1), list(range(n + 1)), 1)
    assert e.value.code == mk.MK_ERR_UNSUPPORTED


def test_rows_beyond_4_gb(mk):
    # a request of 4.4 million tokens: rows, queries and what is read back pass 2^32 bytes
    n, D = 4_400_003, cu.dims(8, 1, 64)
    pages = -(-n // 16)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2))
    qkv = torch.empty(n, 1, 10, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    q = torch.empty(n, 8, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(pages, 1, 2, 64, 16, dtype=torch.bfloat16, device="cuda")
    chunk = mk.Chunk(D, "bf16", pages, [0], [n], table.numpy(), pages)
    chunk.append(qkv, pool, q)
    assert chunk.sync() == mk.MK_OK
    last = torch.cat([torch.arange(0, 3), torch.arange(n - 50, n)])
    x = qkv[last.cuda()].cpu()
    turned = cu.rotate(x[:, :, :9], last, D.rope_theta)
    slack = 4 * 2.0 ** -24 * (x[:, :, :9].double()[..., :32].abs() + x[:, :, :9].double()[..., 32:].abs()).repeat(1, 1, 1, 2)
    bound = cu.BF16 * turned.abs() + 1.01 * slack
    assert ((q[last.cuda()].cpu().double() - turned[:, 0, :8]).abs() <= bound[:, 0, :8]).all()
    got = pool[table[last // 16].cuda()].cpu()[torch.arange(len(last)), 0, :, :, last % 16]
    assert torch.equal(got[:, 1], x[:, 0, 9]) and ((got[:, 0].double() - turned[:, 0, 8]).abs() <= bound[:, 0, 8]).all()
    chunk.close()
    del qkv
    copies = 4                             # the same pages four times over: 17.6 million tokens of 256 bytes
    reader = mk.Chunk(D, "bf16", pages, [pages * 16] * copies, [0] * copies, table.repeat(copies).numpy(), pages)
    back = torch.empty(pages * 16 * copies, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    reader.read(pool, back)
    assert reader.sync() == mk.MK_OK
    want = pool[table.cuda()].squeeze(1).permute(0, 3, 1, 2).reshape(-1, 2, 64)
    for i in range(copies):
        assert torch.equal(back[i * pages * 16:(i + 1) * pages * 16, 0], want)


def test_update_beside_a_capture(mk):
    # one chunk's calls are captured on a stream while another's batch changes, and grows, on a second one
    D, batch, chunk = make(mk, "g8", "bf16", "drafts", seed=4)
    b2 = cu.Batch(*LENS["prompts"], seed=5)
    other = mk.Chunk(D, "bf16", b2.num_pages, [0], [1], [0], 1)
    pool, pool2 = (cu.make_pool("bf16", b.num_pages, 4, 128, 9) for b in (batch, b2))
    q, q2 = (cu.normal((b.rows, 32, 128), 3).bfloat16() for b in (batch, b2))
    on = [(x.cuda(), y.cuda(), torch.zeros_like(x, device="cuda")) for x, y in ((q, pool), (q2, pool2))]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chunk.attend(*on[0])
        other.update(b2.cached, b2.new, b2.flat, b2.width, stream=side)
        other.attend(*on[1], stream=side)
    graph.replay()
    assert chunk.sync() == mk.MK_OK and other.sync(side) == mk.MK_OK
    for x, y, b, (_, _, out) in ((q, pool, batch, on[0]), (q2, pool2, b2, on[1])):
        ref, mag = cu.attend(x, y, "bf16", b, 4)
        assert ((out.cpu().double() - ref).abs() <= cu.attend_bound(ref, mag)).all()
