// Host side of the chunk operators: the checks of a batch, the attention task
// list and the C ABI of mk_chunk_* (include/mk.h).
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <functional>
#include <new>
#include <stdexcept>
#include <vector>

#include "chunk.h"
#include "mk.h"

namespace mk {
void set_last_error(const char* msg);
}

using mk::AppendPage;
using mk::AttnTask;
using mk::ChunkReq;
using mk::JoinTask;

namespace {

int fail(int code, const char* msg) {
  mk::set_last_error(msg);
  return code;
}

int fail_cuda(const char* what, cudaError_t e) {
  cudaGetLastError();   // reported here: not to the caller's next question
  mk::allowed = {};
  char buf[224];
  snprintf(buf, sizeof(buf), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  return fail(MK_ERR_CUDA, buf);
}

// No C++ exception leaves a C entry: a failed host allocation is reported.
template <class F>
int guarded(F&& f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(MK_ERR_CAPACITY, "out of host memory");
  } catch (const std::length_error&) {
    return fail(MK_ERR_CAPACITY, "out of host memory");
  }
}

struct Shape {
  int nq, nkv, d, G;
  double theta;
};

int check_shape(const mk_model_dims* m, Shape& s) {
  if (!m) return fail(MK_ERR_INVALID, "mk_chunk: dims is NULL");
  s.nq = m->n_q_heads; s.nkv = m->n_kv_heads; s.d = m->head_dim; s.theta = m->rope_theta;
  if (s.nq < 0 || s.nkv < 1 || s.nq % s.nkv) return fail(MK_ERR_INVALID, "mk_chunk: head counts");
  if (!(s.theta >= 0.) || s.theta > 3e38) return fail(MK_ERR_INVALID, "mk_chunk: rope_theta must be finite and not negative");
  s.G = s.nq / s.nkv;
  if (m->page_size != mk::PAGE) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: page_size must be 16");
  if (s.d != 64 && s.d != 128) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: head_dim must be 64 or 128");
  if (s.G > 8 || s.nkv > 65535) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: at most 8 query heads per KV head");
  return MK_OK;
}

// What one batch needs on the device, built on the host.
struct Built {
  std::vector<ChunkReq> reqs;
  std::vector<int> pt;
  std::vector<AppendPage> appends;
  std::vector<AttnTask> tasks;
  std::vector<JoinTask> joins;
  std::vector<int> cta_start;
  long long rows = 0, tokens = 0, pages = 0, split_rows = 0, nsplit = 0, joined_rows = 0;
  int max_new = 0;               // rows of one request
};

// Row counts and prefix sums; no pages yet.
int set_lens(const Shape& s, int batch, const int* seq_lens, const int* new_lens, Built& b) {
  if (batch < 1 || !seq_lens || !new_lens) return fail(MK_ERR_INVALID, "mk_chunk: batch or lengths");
  if (batch > 65535) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: at most 65535 requests");
  b.reqs.resize(batch);
  for (int i = 0; i < batch; ++i) {
    if (seq_lens[i] < 0 || new_lens[i] < 0) return fail(MK_ERR_INVALID, "mk_chunk: a negative length");
    const long long total = (long long)seq_lens[i] + new_lens[i];
    // positions and the ends of the tiles around them stay 32-bit
    if (total > INT_MAX - 1024) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: a request of over 2^31 - 1025 tokens");
    ChunkReq& r = b.reqs[i];
    r = {};
    r.seq = seq_lens[i]; r.nnew = new_lens[i]; r.row0 = (int)b.rows; r.tok0 = b.tokens;
    b.rows += new_lens[i];
    b.tokens += total;
    if (b.rows > INT_MAX - 1024) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: over 2^31 - 1025 new rows");
    r.page0 = (int)b.pages;
    b.pages += (total + mk::PAGE - 1) / mk::PAGE;
    if (b.pages > INT_MAX - 1024) return fail(MK_ERR_UNSUPPORTED, "mk_chunk: over 2^31 - 1025 pages");
    b.max_new = std::max(b.max_new, new_lens[i]);
  }
  return MK_OK;
}

int set_pages(int num_pages, const int* page_table, int max_pages, Built& b) {
  if (!page_table || max_pages < 1) return fail(MK_ERR_INVALID, "mk_chunk: page table");
  const int batch = (int)b.reqs.size();
  std::vector<char> written((size_t)num_pages, 0);
  for (int i = 0; i < batch; ++i) {
    ChunkReq& r = b.reqs[i];
    r.pt = (long long)i * max_pages;
    const int np = (r.seq + r.nnew + mk::PAGE - 1) / mk::PAGE;
    if (np > max_pages) return fail(MK_ERR_CAPACITY, "mk_chunk: a request's tokens need more pages than its table row holds");
    for (int j = 0; j < np; ++j) {
      const int pg = page_table[r.pt + j];
      if (pg < 0 || pg >= num_pages) return fail(MK_ERR_INVALID, "mk_chunk: a page outside the pool");
      if (r.nnew && j >= r.seq / mk::PAGE) {
        if (written[pg]) return fail(MK_ERR_INVALID, "mk_chunk: two requests' new tokens, or two pages of one, in one page");
        written[pg] = 1;
        const int p0 = std::max(j * mk::PAGE, r.seq), p1 = std::min(j * mk::PAGE + mk::PAGE, r.seq + r.nnew);
        b.appends.push_back({pg, r.row0 + p0 - r.seq, p1 - p0, p0 - j * mk::PAGE});
      }
    }
  }
  for (const ChunkReq& r : b.reqs) {
    const int np = (r.seq + r.nnew + mk::PAGE - 1) / mk::PAGE;
    const int keep = r.nnew ? r.seq / mk::PAGE : np;   // pages that receive none of its new tokens
    for (int j = 0; j < keep; ++j)
      if (written[page_table[r.pt + j]])
        return fail(MK_ERR_INVALID, "mk_chunk: a page that receives new tokens belongs to another place too");
  }
  b.pt.assign(page_table, page_table + (size_t)batch * max_pages);
  return MK_OK;
}

// Attention tasks.  A block is the rows of up to two query tiles of one
// request and KV head (a tile: the G heads of Q_TILE / G tokens); its keys run
// to its last row's position, in tiles of KV_TILE.  A CTA works through a list
// of tasks.  Two schedules are weighed against each other, in units of a tile
// (about 0.75 us): whole blocks, the longest first, each to the CTA with the
// least work; and the blocks' tiles in one row, cut into runs that are as even
// as whole tiles allow, where a block that a cut goes through is joined
// afterwards.  A task costs SETUP beside its tiles (its queries, its first
// latencies and its epilogue), a join JOIN.  (SETUP 2, 4, 6, 8, 10: 161, 129,
// 120, 117 and 122 us for requests of 1500, 900 and 333 new rows behind 0, 5000
// and 8192 cached ones; batches of one kind hardly move.)
struct Block {
  int req, kvh, tok0, ntok, tiles;
};
constexpr int SETUP = 8, JOIN = 5;

// Gives every CTA tiles up to `limit` (its tasks' SETUP included) in the row's
// order; emits (block, first tile, tiles, CTA).  False if the CTAs do not do.
template <class F>
bool deal(const std::vector<Block>& blocks, int ctas, long long limit, F&& emit) {
  int c = 0;
  long long room = limit;
  for (size_t i = 0; i < blocks.size(); ++i) {
    int at = 0;
    while (at < blocks[i].tiles) {
      if (room <= SETUP) {
        if (++c == ctas) return false;
        room = limit;
      }
      const int n = (int)std::min<long long>(blocks[i].tiles - at, room - SETUP);
      emit(i, at, n, c);
      room -= SETUP + n;
      at += n;
    }
  }
  return true;
}

void set_tasks(const Shape& s, int ctas, Built& b) {
  b.tasks.clear();
  b.joins.clear();
  b.cta_start.assign(1, 0);
  b.split_rows = b.nsplit = b.joined_rows = 0;
  if (!s.G) return;
  const int per_tile = mk::Q_TILE / s.G, per_block = 2 * per_tile;
  std::vector<Block> blocks;
  long long work = 0, longest = 0;
  for (int i = 0; i < (int)b.reqs.size(); ++i) {
    const ChunkReq& r = b.reqs[i];
    for (int t = 0; t < r.nnew; t += per_block) {
      const int n = std::min(per_block, r.nnew - t), tiles = (r.seq + t + n + mk::KV_TILE - 1) / mk::KV_TILE;
      longest = std::max<long long>(longest, tiles);
      work += (long long)(tiles + SETUP) * s.nkv;
      for (int g = 0; g < s.nkv; ++g) blocks.push_back({i, g, t, n, tiles});
    }
  }
  if (blocks.empty()) return;
  // whole blocks
  std::vector<int> order(blocks.size()), owner(blocks.size());
  for (size_t i = 0; i < order.size(); ++i) order[i] = (int)i;
  std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return blocks[x].tiles > blocks[y].tiles; });
  std::vector<std::pair<long long, int>> heap;   // (load, CTA), the least first
  long long whole = 0;
  for (int i : order) {
    std::pair<long long, int> at = {0, (int)heap.size()};
    if ((int)heap.size() >= ctas) {
      std::pop_heap(heap.begin(), heap.end(), std::greater<>());
      at = heap.back();
      heap.pop_back();
    }
    at.first += blocks[i].tiles + SETUP;
    owner[i] = at.second;
    whole = std::max(whole, at.first);
    heap.push_back(at);
    std::push_heap(heap.begin(), heap.end(), std::greater<>());
  }
  // even runs: the smallest limit for which the CTAs do
  long long lo = std::max<long long>(SETUP + 1, work / ctas), hi = whole;
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (deal(blocks, ctas, mid, [](size_t, int, int, int) {})) hi = mid;
    else lo = mid + 1;
  }
  const bool runs = hi + JOIN < whole;
  auto add = [&](size_t i, int tile0, int n, int cta, int part) {
    const Block& k = blocks[i];
    const ChunkReq& r = b.reqs[k.req];
    b.tasks.push_back({k.req, k.kvh, k.tok0, k.ntok, tile0, n, part, cta, r.row0 + k.tok0, r.seq + k.tok0, r.seq + r.nnew,
                       0, r.pt, 0});
  };
  if (runs) {
    std::vector<int> parts(blocks.size(), 0), first(blocks.size(), -1);
    deal(blocks, ctas, hi, [&](size_t i, int, int, int) { ++parts[i]; });
    for (size_t i = 0; i < blocks.size(); ++i)
      if (parts[i] > 1) {
        const Block& k = blocks[i];
        const long long rows = (long long)k.ntok * s.G;
        first[i] = (int)b.split_rows;
        b.joins.push_back({k.req, k.kvh, k.tok0, k.ntok, first[i], parts[i], b.reqs[k.req].row0 + k.tok0, 0});
        b.joined_rows += rows;
        b.split_rows += rows * parts[i];
        b.nsplit += parts[i];
      }
    deal(blocks, ctas, hi, [&](size_t i, int at, int n, int c) {
      add(i, at, n, c, first[i]);
      if (first[i] >= 0) first[i] += blocks[i].ntok * s.G;
    });
  } else {
    for (int i : order) add(i, 0, blocks[i].tiles, owner[i], -1);
    std::stable_sort(b.tasks.begin(), b.tasks.end(), [](const AttnTask& x, const AttnTask& y) { return x.cta < y.cta; });
  }
  b.cta_start.assign(b.tasks.back().cta + 2, 0);
  for (const AttnTask& t : b.tasks) ++b.cta_start[t.cta + 1];
  for (size_t i = 1; i < b.cta_start.size(); ++i) b.cta_start[i] += b.cta_start[i - 1];
  for (size_t c = 0; c + 1 < b.cta_start.size(); ++c) {
    int two = 0;
    for (int i = b.cta_start[c]; i < b.cta_start[c + 1]; ++i) two |= b.tasks[i].ntok > per_tile;
    for (int i = b.cta_start[c]; i < b.cta_start[c + 1]; ++i) b.tasks[i].two = two;
  }
}

}  // namespace

// Page-locked memory that an upload leaves from.  Two take turns: an update
// waits for the upload two before it, never for the work in front of its own
// (from pageable memory a copy of more than 64 KB waited for all of it).
struct Stage {
  char* mem = nullptr;
  size_t cap = 0;
  cudaEvent_t sent = nullptr;    // behind the last upload
};

struct mk_chunk {
  Shape s;
  int type = 0, num_pages = 0, device = 0, ctas = 0;
  Built b;
  // requests, page table, tasks, joins, CTAs' first tasks; the rotation's
  // angles; split rows: sums, then (maximum, sum) pairs
  char* mem = nullptr;
  size_t mem_cap = 0;
  int* status = nullptr;         // [0] first recorded error, [1] generation of the tables
  int gen = 0;
  Stage stage[2];
  int turn = 0;                  // the one used last
  bool lost = false;             // an upload failed: the tables hold no batch
  std::vector<void*> retired;    // outgrown memory: graphs of earlier batches may name it, so it stays
  mk::ChunkView view = {};
};

namespace {

// Allocations of this thread while it captures some other stream: without it
// they would fail, and end that capture.
struct BesideCaptures {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  BesideCaptures() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~BesideCaptures() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

cudaError_t grow(mk_chunk* c, size_t need) {
  if (need <= c->mem_cap) return cudaSuccess;
  void* q = nullptr;
  c->retired.reserve(c->retired.size() + 1);
  need = std::max(need, c->mem_cap + c->mem_cap / 2);
  const cudaError_t e = cudaMalloc(&q, need);
  if (e != cudaSuccess) return e;
  if (c->mem) c->retired.push_back(c->mem);
  c->mem = (char*)q;
  c->mem_cap = need;
  return cudaSuccess;
}

// The next stage with room for `need` bytes.
cudaError_t next_stage(mk_chunk* c, size_t need, Stage** out) {
  Stage& s = *(*out = &c->stage[c->turn ^ 1]);
  cudaError_t e = s.sent ? cudaEventSynchronize(s.sent) : cudaEventCreateWithFlags(&s.sent, cudaEventDisableTiming);
  if (e == cudaSuccess && need > s.cap) {
    if (s.mem) cudaFreeHost(s.mem);
    s.mem = nullptr;
    s.cap = 0;
    e = cudaMallocHost((void**)&s.mem, need + need / 2);
    if (e == cudaSuccess) s.cap = need + need / 2;
  }
  if (e == cudaSuccess) c->turn ^= 1;
  return e;
}

int build(const mk_chunk* c, int batch, const int* seq_lens, const int* new_lens, const int* page_table, int max_pages,
          Built& b) {
  int rc = set_lens(c->s, batch, seq_lens, new_lens, b);
  if (rc == MK_OK) rc = set_pages(c->num_pages, page_table, max_pages, b);
  return rc;
}

// `once`: the caller waits for the stream, so any memory will do (a stage costs
// 0.1 ms to make and 0.2 to give back, more than a chunk of one batch).
int commit(mk_chunk* c, Built&& nb, cudaStream_t st, bool once) {
  const size_t d = c->s.d;
  const size_t n_req = up16(nb.reqs.size() * sizeof(ChunkReq)), n_pt = up16(nb.pt.size() * sizeof(int)),
               n_task = up16(nb.tasks.size() * sizeof(AttnTask)), n_join = up16(nb.joins.size() * sizeof(JoinTask)),
               n_cta = up16(nb.cta_start.size() * sizeof(int)), n_app = nb.appends.size() * sizeof(AppendPage),
               n_all = n_req + n_pt + n_task + n_join + n_app + n_cta;
  const size_t n_rope = c->s.theta > 0. ? up16((size_t)nb.rows * (d / 2) * sizeof(float2)) : 0;
  const size_t off_rope = (n_all + 255) / 256 * 256, off_part = (off_rope + n_rope + 255) / 256 * 256;
  cudaError_t e = grow(c, off_part + (size_t)nb.split_rows * (d + 2) * sizeof(float));
  if (e != cudaSuccess) return fail_cuda("mk_chunk: device memory", e);
  std::vector<char> plain(once ? n_all + 2 * sizeof(int) : 0);
  Stage* stage = nullptr;
  if (!once) {
    e = next_stage(c, n_all + 2 * sizeof(int), &stage);
    if (e != cudaSuccess) return fail_cuda("mk_chunk: page-locked memory", e);
  }
  char* host = once ? plain.data() : stage->mem;
  memcpy(host, nb.reqs.data(), nb.reqs.size() * sizeof(ChunkReq));
  memcpy(host + n_req, nb.pt.data(), nb.pt.size() * sizeof(int));
  if (!nb.tasks.empty()) memcpy(host + n_req + n_pt, nb.tasks.data(), nb.tasks.size() * sizeof(AttnTask));
  if (!nb.joins.empty())
    memcpy(host + n_req + n_pt + n_task, nb.joins.data(), nb.joins.size() * sizeof(JoinTask));
  if (n_app) memcpy(host + n_all - n_cta - n_app, nb.appends.data(), n_app);
  memcpy(host + n_all - n_cta, nb.cta_start.data(), nb.cta_start.size() * sizeof(int));
  const int head[2] = {0, ++c->gen};
  memcpy(host + n_all, head, sizeof(head));
  e = cudaMemcpyAsync(c->mem, host, n_all, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(c->status, host + n_all, sizeof(head), cudaMemcpyHostToDevice, st);
  const cudaError_t sent = once ? cudaStreamSynchronize(st) : cudaEventRecord(stage->sent, st);   // after a failed copy too
  if (e == cudaSuccess) e = sent;
  c->b = std::move(nb);
  mk::ChunkView& v = c->view;
  char* base = c->mem;
  v.nq = c->s.nq; v.nkv = c->s.nkv; v.d = c->s.d; v.G = c->s.G;
  v.batch = (int)c->b.reqs.size(); v.rows = (int)c->b.rows; v.num_pages = c->num_pages;
  v.reqs = (const ChunkReq*)base;
  v.pt = (const int*)(base + n_req);
  v.tasks = (const AttnTask*)(base + n_req + n_pt);
  v.joins = (const JoinTask*)(base + n_req + n_pt + n_task);
  v.cta_start = (const int*)(base + n_all - n_cta);
  v.appends = (const AppendPage*)(base + n_all - n_cta - n_app);
  v.nappends = (int)c->b.appends.size(); v.npages = (int)c->b.pages;
  v.ctas = (int)c->b.cta_start.size() - 1; v.njoins = (int)c->b.joins.size();
  v.max_parts = v.max_join_rows = 0;
  for (const JoinTask& j : c->b.joins) {
    v.max_parts = std::max(v.max_parts, j.nparts);
    v.max_join_rows = std::max(v.max_join_rows, j.ntok * v.G);
  }
  v.rope = c->s.theta > 0. ? (const float2*)(base + off_rope) : nullptr;
  v.part_o = (float*)(base + off_part);
  v.part_ml = (float2*)(v.part_o + (size_t)c->b.split_rows * d);
  v.status = c->status;
  v.gen = c->gen;
  if (e == cudaSuccess && v.rope && v.rows)
    e = mk::launch_chunk_rope(v, c->s.theta, (float2*)(base + off_rope), c->b.max_new, st);
  c->lost = e != cudaSuccess;
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_chunk: upload", e);
}

// The chunk's memory lives on one device.
int check_device(const mk_chunk* c) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda("mk_chunk: current device", e);
  if (c->lost) return fail(MK_ERR_INVALID, "mk_chunk: the last update failed; update again");
  return dev == c->device ? MK_OK : fail(MK_ERR_INVALID, "mk_chunk: the chunk belongs to another device than the current one");
}

size_t pool_bytes(const mk_chunk* c) {
  return (size_t)c->num_pages * c->s.nkv * 2 * mk::PAGE * (c->type == MK_KV_E4M3 ? c->s.d + 1 : c->s.d * 2);
}
size_t query_bytes(const mk_chunk* c) { return (size_t)c->b.rows * c->s.nq * c->s.d * 2; }

bool aligned16(const void* p) { return p && (uintptr_t)p % 16 == 0; }

}  // namespace

extern "C" {

void mk_chunk_destroy(mk_chunk* c) {
  if (!c) return;
  for (Stage& s : c->stage) {
    if (s.sent) {
      cudaEventSynchronize(s.sent);
      cudaEventDestroy(s.sent);
    }
    if (s.mem) cudaFreeHost(s.mem);
  }
  cudaFree(c->mem);
  cudaFree(c->status);
  for (void* p : c->retired) cudaFree(p);
  delete c;
}

int mk_chunk_create(const mk_model_dims* dims, int kv_type, int num_pages, int batch, const int* seq_lens,
                    const int* new_lens, const int* page_table, int max_pages_per_seq, mk_chunk** out) {
  if (!out) return fail(MK_ERR_INVALID, "mk_chunk_create: out is NULL");
  *out = nullptr;
  Shape s;
  const int rs = check_shape(dims, s);
  if (rs != MK_OK) return rs;
  if (kv_type != MK_KV_BF16 && kv_type != MK_KV_E4M3) return fail(MK_ERR_INVALID, "mk_chunk_create: kv_type");
  if (num_pages < 1) return fail(MK_ERR_INVALID, "mk_chunk_create: num_pages");
  mk_chunk* c = nullptr;
  const int rc = guarded([&] {
    c = new mk_chunk();
    c->s = s; c->type = kv_type; c->num_pages = num_pages;
    Built b;
    int r = build(c, batch, seq_lens, new_lens, page_table, max_pages_per_seq, b);
    if (r != MK_OK) return r;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->ctas, cudaDevAttrMultiProcessorCount, c->device);
    if (e == cudaSuccess) e = cudaMalloc((void**)&c->status, 4 * sizeof(int));
    if (e != cudaSuccess) return fail_cuda("mk_chunk_create", e);
    set_tasks(s, c->ctas, b);
    r = commit(c, std::move(b), 0, true);
    if (r != MK_OK) return r;
    e = cudaStreamSynchronize(0);
    return e == cudaSuccess ? MK_OK : fail_cuda("mk_chunk_create", e);
  });
  if (rc != MK_OK) {
    mk_chunk_destroy(c);
    return rc;
  }
  *out = c;
  return MK_OK;
}

int mk_chunk_update(mk_chunk* c, int batch, const int* seq_lens, const int* new_lens, const int* page_table,
                    int max_pages_per_seq, mk_stream stream) {
  if (!c) return fail(MK_ERR_INVALID, "mk_chunk_update: chunk is NULL");
  return guarded([&] {
    Built b;
    int rc = build(c, batch, seq_lens, new_lens, page_table, max_pages_per_seq, b);
    if (rc != MK_OK) return rc;
    const bool lost = c->lost;
    c->lost = false;
    rc = check_device(c);
    if (rc != MK_OK) {
      c->lost = lost;
      return rc;
    }
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &cap);
    c->lost = lost;
    if (e != cudaSuccess) return fail_cuda("mk_chunk_update", e);
    if (cap != cudaStreamCaptureStatusNone) return fail(MK_ERR_INVALID, "mk_chunk_update: the stream is being captured");
    set_tasks(c->s, c->ctas, b);
    BesideCaptures relaxed;
    return commit(c, std::move(b), (cudaStream_t)stream, false);
  });
}

int mk_chunk_append(mk_chunk* c, const void* qkv, int rows_type, long long row_stride, void* kv_pool, void* q,
                    mk_stream stream) {
  if (!c) return fail(MK_ERR_INVALID, "mk_chunk_append: chunk is NULL");
  if (rows_type != MK_ROWS_BF16 && rows_type != MK_ROWS_F32) return fail(MK_ERR_INVALID, "mk_chunk_append: rows_type");
  const long long el = rows_type == MK_ROWS_F32 ? 4 : 2, width = (long long)c->s.nkv * (c->s.G + 2) * c->s.d;
  if (row_stride < width || row_stride > (LLONG_MAX >> 36) || row_stride * el % 16)
    return fail(MK_ERR_INVALID, "mk_chunk_append: row_stride");
  if (c->b.rows == 0) return check_device(c);
  if (!aligned16(kv_pool) || !aligned16(qkv) || (c->s.nq ? !aligned16(q) : q != nullptr))
    return fail(MK_ERR_INVALID, "mk_chunk_append: a buffer is NULL or not 16-byte aligned");
  const size_t nx = (size_t)((c->b.rows - 1) * row_stride + width) * el, nq = q ? query_bytes(c) : 0;
  if (mk::meet(qkv, nx, kv_pool, pool_bytes(c)) || mk::meet(q, nq, qkv, nx) || mk::meet(q, nq, kv_pool, pool_bytes(c)))
    return fail(MK_ERR_INVALID, "mk_chunk_append: two of the buffers overlap");
  const int rc = check_device(c);
  if (rc != MK_OK) return rc;
  const cudaError_t e = mk::launch_append(c->view, c->type == MK_KV_E4M3, rows_type == MK_ROWS_F32, qkv, row_stride,
                                          kv_pool, q, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_chunk_append", e);
}

int mk_chunk_attend(mk_chunk* c, const void* q, const void* kv_pool, void* out, mk_stream stream) {
  if (!c) return fail(MK_ERR_INVALID, "mk_chunk_attend: chunk is NULL");
  if (!c->s.nq) return fail(MK_ERR_INVALID, "mk_chunk_attend: a chunk without query heads");
  if (c->b.rows == 0) return check_device(c);
  // a bf16 pool's 128-byte rows are counted in 32 bits
  if (c->type == MK_KV_BF16 && (long long)c->num_pages * c->s.nkv * 2 * (c->s.d / 4) > INT_MAX - 64)
    return fail(MK_ERR_UNSUPPORTED, "mk_chunk_attend: a bf16 pool of 256 GB or more");
  if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(out))
    return fail(MK_ERR_INVALID, "mk_chunk_attend: a buffer is NULL or not 16-byte aligned");
  if ((out != q && mk::meet(out, query_bytes(c), q, query_bytes(c))) || mk::meet(out, query_bytes(c), kv_pool, pool_bytes(c)))
    return fail(MK_ERR_INVALID, "mk_chunk_attend: out overlaps the pool, or q in another place than its own");
  const int rc = check_device(c);
  if (rc != MK_OK) return rc;
  const cudaError_t e = mk::launch_attend(c->view, c->type == MK_KV_E4M3, q, kv_pool, out, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_chunk_attend", e);
}

int mk_chunk_read(mk_chunk* c, const void* kv_pool, void* out, mk_stream stream) {
  if (!c) return fail(MK_ERR_INVALID, "mk_chunk_read: chunk is NULL");
  if (c->b.tokens == 0) return check_device(c);
  if (!aligned16(kv_pool) || !aligned16(out))
    return fail(MK_ERR_INVALID, "mk_chunk_read: a buffer is NULL or not 16-byte aligned");
  if (mk::meet(out, (size_t)c->b.tokens * c->s.nkv * 2 * c->s.d * 2, kv_pool, pool_bytes(c)))
    return fail(MK_ERR_INVALID, "mk_chunk_read: out overlaps the pool");
  const int rc = check_device(c);
  if (rc != MK_OK) return rc;
  const cudaError_t e = mk::launch_read(c->view, c->type == MK_KV_E4M3, kv_pool, out, (cudaStream_t)stream);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_chunk_read", e);
}

int mk_chunk_sync(mk_chunk* c, mk_stream stream) {
  if (!c) return fail(MK_ERR_INVALID, "mk_chunk_sync: chunk is NULL");
  const int rc = check_device(c);
  if (rc != MK_OK) return rc;
  int st = 0;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&st, c->status, sizeof(int), cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  return e == cudaSuccess ? st : fail_cuda("mk_chunk_sync", e);
}

int mk_chunk_info(const mk_chunk* c, int* out, int n) {
  if (!c || (!out && n > 0)) return fail(MK_ERR_INVALID, "mk_chunk_info");
  const int v[7] = {(int)c->b.reqs.size(), (int)c->b.rows, (int)std::min<long long>(c->b.tokens, INT_MAX),
                    (int)c->b.tasks.size(), (int)c->b.nsplit, (int)c->b.joined_rows, c->ctas};
  for (int i = 0; i < std::min(n, 7); ++i) out[i] = v[i];
  return MK_OK;
}

int mk_chunk_inspect(const mk_model_dims* dims, int batch, const int* seq_lens, const int* new_lens, int num_ctas,
                     int* tasks, int max_tasks) {
  Shape s;
  int rc = check_shape(dims, s);
  if (rc != MK_OK) return rc;
  if (num_ctas < 1 || max_tasks < 0 || (max_tasks && !tasks)) return fail(MK_ERR_INVALID, "mk_chunk_inspect");
  return guarded([&] {
    Built b;
    int r = set_lens(s, batch, seq_lens, new_lens, b);
    if (r != MK_OK) return r;
    set_tasks(s, num_ctas, b);
    const int n = std::min<int>(max_tasks, (int)b.tasks.size());
    for (int i = 0; i < n; ++i) memcpy(tasks + 8 * i, &b.tasks[i], 8 * sizeof(int));   // the record's first words
    return (int)b.tasks.size();
  });
}

}  // extern "C"
