"""The chunk operators on the host (no GPU): what mk_chunk_create, mk_probs and
mk_verify refuse, and the attention task lists."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from tests import chunk_util as cu


@pytest.fixture(scope="module")
def mk(built):
    from persistent_moe_decode_02_gb300 import mk
    return mk


def refused(mk, code, D=None, kv="bf16", pages=8, cached=(20,), new=(4,), table=(0, 1), width=2):
    with pytest.raises(mk.MkError) as e:
        mk.Chunk(D or cu.dims(8, 2, 64), kv, pages, list(cached), list(new), list(table), width)
    assert e.value.code == code, e.value


def test_refused_batches(mk):
    bad, cap, uns = mk.MK_ERR_INVALID, mk.MK_ERR_CAPACITY, mk.MK_ERR_UNSUPPORTED
    refused(mk, bad, cu.dims(6, 4, 64))                       # heads that are no groups
    refused(mk, bad, cu.dims(8, 0, 64))
    refused(mk, uns, cu.dims(8, 2, 96))
    refused(mk, uns, cu.dims(18, 2, 64))                      # 9 query heads a group
    refused(mk, uns, SimpleNamespace(n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=32, rope_theta=1e4))
    refused(mk, bad, cu.dims(8, 2, 64, theta=-1.0))
    refused(mk, bad, cu.dims(8, 2, 64, theta=float("nan")))
    refused(mk, bad, cu.dims(8, 2, 64, theta=float("inf")))
    refused(mk, bad, pages=0)
    refused(mk, bad, cached=(-1,))
    refused(mk, bad, new=(-1,))
    refused(mk, bad, table=(0, 8))                            # a page outside the pool
    refused(mk, bad, table=(0, -1))
    refused(mk, cap, new=(13,))                               # 33 tokens on 2 pages
    refused(mk, uns, cached=(2 ** 31 - 1,), new=(2 ** 31 - 1,), table=(0, 1))
    refused(mk, bad, cached=(), new=(), table=(), width=2)    # no request
    refused(mk, bad, cached=(0, 0), new=(1, 1), table=(3, 3), width=1)          # two requests write one page
    refused(mk, bad, cached=(16, 0), new=(1, 1), table=(3, 4, 3, -1))           # one writes what another reads
    refused(mk, bad, cached=(0,), new=(20,), table=(5, 5))                      # the same page twice
    refused(mk, bad, cached=(16,), new=(4,), table=(5, 5))
    with pytest.raises(ValueError):
        mk.Chunk(cu.dims(8, 2, 64), "fp8", 8, [0], [1], [0], 1)
    with pytest.raises(ValueError):
        mk.Chunk(cu.dims(8, 2, 64), "bf16", 8, [0, 1], [1], [0], 1)
    for cached, new, table in (([2 ** 32 + 5], [1], [0]), ([0], [1.5], [0]), ([0], [1], [2 ** 31]), ([[0]], [[1]], [0])):
        with pytest.raises(ValueError):
            mk.Chunk(cu.dims(8, 2, 64), "bf16", 8, cached, new, table, 1)


def test_refused_null_and_numbers(mk):
    L, vp = mk.lib(), ctypes.c_void_p
    one = vp(1 << 20)     # aligned, never read: every call below is refused before a CUDA call
    assert L.mk_chunk_create(None, 0, 1, 1, None, None, None, 1, ctypes.byref(vp())) == mk.MK_ERR_INVALID
    assert L.mk_chunk_update(None, 1, None, None, None, 1, None) == mk.MK_ERR_INVALID
    assert L.mk_chunk_append(None, one, 0, 8, one, one, None) == mk.MK_ERR_INVALID
    assert L.mk_chunk_attend(None, one, one, one, None) == mk.MK_ERR_INVALID
    assert L.mk_chunk_read(None, one, one, None) == mk.MK_ERR_INVALID
    assert L.mk_chunk_sync(None, None) == mk.MK_ERR_INVALID
    assert L.mk_chunk_info(None, None, 0) == mk.MK_ERR_INVALID
    L.mk_chunk_destroy(None)
    probs = lambda rows=1, v=8, stride=8, t=1.0, a=one, b=vp(1 << 21): L.mk_probs(a, rows, v, stride, t, b, None)
    assert probs(rows=-1) == probs(v=0) == probs(stride=7) == mk.MK_ERR_INVALID
    assert probs(t=-1.0) == probs(t=float("nan")) == probs(t=float("inf")) == probs(t=1e-39) == mk.MK_ERR_INVALID
    assert probs(a=None) == probs(b=None) == probs(a=vp(2)) == mk.MK_ERR_INVALID
    assert probs(b=vp((1 << 20) + 4)) == mk.MK_ERR_INVALID                     # overlap
    assert probs(rows=2, stride=9, b=one) == mk.MK_ERR_INVALID                  # in place, rows apart
    assert probs(v=393217, stride=393217) == mk.MK_ERR_UNSUPPORTED
    assert probs(rows=0) == mk.MK_OK
    verify = lambda b=1, k=2, v=8, t=one, d=one, x=one, n=None, u=one, r=one, o=one, c=one: L.mk_verify(
        b, k, v, t, d, x, n, u, r, o, c, None)
    assert verify(b=-1) == verify(k=-1) == verify(v=0) == mk.MK_ERR_INVALID
    assert verify(t=None) == verify(r=None) == verify(o=None) == verify(c=None) == mk.MK_ERR_INVALID
    assert verify(x=None) == verify(u=None) == verify(d=vp(2)) == verify(n=vp(2)) == mk.MK_ERR_INVALID
    assert verify(v=393217) == mk.MK_ERR_UNSUPPORTED
    assert verify(b=0) == mk.MK_OK


CASES = [((32, 4, 128), [8191], [1]), ((32, 4, 128), [0, 0, 0], [2049, 517, 1000]), ((32, 4, 128), [30000], [2048]),
         ((4, 2, 64), [5, 0, 77, 1000], [0, 1, 300, 64]), ((14, 2, 64), [100] * 50, [3] * 50), ((5, 5, 64), [0], [1]),
         ((12, 2, 128), list(range(0, 4000, 61)), [17] * 66)]


@pytest.mark.parametrize("heads,cached,new", CASES)
@pytest.mark.parametrize("ctas", [1, 7, 152])
def test_tasks_cover_every_row_and_key_once(mk, heads, cached, new, ctas):
    D = cu.dims(*heads)
    tasks = mk.inspect_chunk(D, cached, new, ctas).tolist()
    per_block = 2 * (128 // (heads[0] // heads[1]))
    G = heads[0] // heads[1]
    blocks, split = {}, []
    for req, g, tok0, n, tile0, tiles, part, cta in tasks:
        assert tiles > 0 and 0 <= cta < ctas and 0 <= g < heads[1]
        blocks.setdefault((req, g, tok0), []).append((tile0, tiles, n, part))
        if part >= 0:
            split.append((part, n * G))
    want = {(b, g, t): min(per_block, n - t) for b, n in enumerate(new) for t in range(0, n, per_block)
            for g in range(heads[1])}
    assert set(blocks) == set(want)
    for (b, g, t), parts in blocks.items():
        parts.sort()
        n, end = want[b, g, t], -(-(cached[b] + t + want[b, g, t]) // 64)
        assert all(p[2] == n for p in parts)
        at = 0
        for tile0, tiles, _, _ in parts:      # its key tiles, each in one task, up to its last row's position
            assert tile0 == at
            at += tiles
        assert at == end
        assert [p[3] >= 0 for p in parts] == [len(parts) > 1] * len(parts)
        if len(parts) > 1:                    # split rows lie one part after another
            assert [p[3] for p in parts] == [parts[0][3] + i * n * G for i in range(len(parts))]
    split.sort()
    at = 0
    for part, rows in split:                  # and no two parts share a row
        assert part == at
        at += rows
    ctas_seen = [t[7] for t in tasks]
    assert ctas_seen == sorted(ctas_seen)


def test_tasks_are_even(mk):
    # a long chunk and a single token leave no CTA with much more than its share (a task counts 8 tiles beside its own)
    for cached, new in (([30000], [2048]), ([8191], [1]), ([262143], [1]), ([8200, 39997, 1023], [5, 5, 4])):
        tasks = mk.inspect_chunk(cu.dims(32, 4, 128), cached, new, 152)
        load = torch.zeros(152, dtype=torch.int64).index_add_(0, tasks[:, 7], tasks[:, 5] + 8)
        assert int(load.max()) <= float(load.double().mean()) * 1.05 + 3


def test_inspect_refuses(mk):
    for code, cached, new in ((mk.MK_ERR_INVALID, [-1], [1]), (mk.MK_ERR_INVALID, [], [])):
        with pytest.raises(mk.MkError) as e:
            mk.inspect_chunk(cu.dims(8, 2, 64), cached, new, 4)
        assert e.value.code == code
    with pytest.raises(mk.MkError):
        mk.inspect_chunk(cu.dims(8, 2, 64), [1], [1], 0)
    with pytest.raises(ValueError):
        mk.inspect_chunk(cu.dims(8, 2, 64), [1, 2], [1], 4)


def test_the_64_bit_forms_themselves():
    # attention over shuffled pages is attention over the plain order, and the quantiser keeps its promise
    batch = cu.Batch([20, 3], [2, 1], seed=1)
    pool = cu.make_pool("bf16", batch.num_pages, 2, 64, 3)
    q = cu.normal((3, 4, 64), 4).bfloat16()
    ref, _ = cu.attend(q, pool, "bf16", batch, 2)
    rows = torch.stack([pool[batch.table[0][s // 16], :, :, :, s % 16] for s in range(22)]).double()
    w = torch.softmax(rows[:21, 1, 0] @ q[0, 3].double() / 8, 0) @ rows[:21, 1, 1]
    assert torch.allclose(ref[0, 3], w, atol=1e-12)
    x = cu.normal((100, 64), 5, 30.0)
    code, k = cu.quantise(x)
    back = torch.ldexp(code.view(torch.float8_e4m3fn).double(), k.unsqueeze(-1).double())
    err = torch.maximum(cu.E4M3_STEP * x.double().abs(), cu.E4M3_MIN * torch.exp2(k.double()).unsqueeze(-1))
    assert ((back - x.double()).abs() <= err).all()
    assert (x.abs().amax(-1) <= 448 * torch.exp2(k.float())).all() and (x.abs().amax(-1) > 224 * torch.exp2(k.float())).all()


def test_rows_are_split_by_what_the_device_has(tmp_path):
    # the host rule of mk_probs and mk_verify by itself: 16 blocks a row only where few rows leave each block an SM and
    # the device offers clusters of 16, and every row fits the largest instance
    import os
    import subprocess
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "persistent_moe_decode_02_gb300", "csrc")
    src = tmp_path / "rows.cpp"
    src.write_text('''#include <cstdio>
#include <initializer_list>
#include "rows.h"
int main() {
  for (int sms : {152, 80, 16, 8})
    for (int most : {16, 8})
      for (long long rows : {1, 5, 9, 10, 160})
        for (int vocab : {1, 2048, 2049, 16385, 151936, 393213, 393216})
          std::printf("%d %d %lld %d %d %d %d\\n", sms, most, rows, vocab, mk::cluster_of(vocab, rows, sms, most),
                      mk::passes_of(vocab, mk::cluster_of(vocab, rows, sms, most)), mk::blocks_at_once(sms));
}
''')
    exe = tmp_path / "rows"
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    table = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        sms, most, rows, vocab, c, passes, ahead = map(int, line.split())
        table[sms, most, rows, vocab] = c
        assert c in (1, 2, 4, 8, 16) and passes <= 24
        assert c <= (most if rows * 16 <= sms else 8)
        assert ahead % 16 == 0 and 0 < ahead <= 2 * sms
    assert len(table) == 4 * 2 * 5 * 7
    assert [table[152, 16, r, 151936] for r in (1, 9, 10, 160)] == [16, 16, 8, 8]
    assert table[152, 8, 1, 151936] == 8 and table[152, 8, 1, 393216] == 8
    assert table[80, 16, 5, 151936] == 16 and table[80, 16, 9, 151936] == 8   # 144 blocks on 80 SMs are not few
    assert table[8, 16, 1, 151936] == 8
    assert table[152, 16, 1, 2048] == 1 and table[152, 16, 1, 2049] == 2 and table[152, 16, 160, 16385] == 4


def test_verify_refuses_outputs_over_other_buffers(mk):
    # addresses that nothing reads: every call is refused before a CUDA call
    L, vp = mk.lib(), ctypes.c_void_p
    at = {n: (i + 1) << 20 for i, n in enumerate(("t", "d", "x", "n", "u", "r", "o", "c"))}

    def verify(b=2, k=2, v=8, **over):
        a = {**at, **over}
        return L.mk_verify(b, k, v, *(vp(a[n]) for n in ("t", "d", "x", "n", "u", "r", "o", "c")), None)

    b, k, v = 2, 2, 8
    size = {"t": b * (k + 1) * v * 4, "d": b * k * v * 4, "x": b * k * 4, "n": b * 4, "u": b * k * 4, "r": b * 4}
    for name, n in size.items():
        for out, m in (("o", b * (k + 1) * 4), ("c", b * 4)):
            for place in (at[name], at[name] + n - 4, at[name] - m + 4):     # whole, its last word, its first
                assert verify(**{out: place}) == mk.MK_ERR_INVALID, (name, out)
    assert verify(c=at["o"]) == verify(c=at["o"] + b * (k + 1) * 4 - 4) == mk.MK_ERR_INVALID
    assert verify(b=1, o=at["x"] + 4) == mk.MK_ERR_INVALID
