// Attention of a chunk's rows over the paged cache.
//
// out = sum_s p_s v_s / sum_s p_s, p_s = 2^((q . k_s - m) log2(e) / sqrt(d)),
// over the positions s up to the row's own, in one pass over the cache with the
// running maximum m and sum of each row in fp32.
//
// A block works through its list of tasks; a task is up to two query tiles of
// one request (128 rows each: 128 / G tokens with the G heads that share a KV
// head, so a key tile is fetched once for all of them) against a run of key
// tiles (64 keys, 4 pages).  Products run on the tensor cores: S = Q K^T into
// tensor memory, softmax in registers (one thread a row), P back to tensor
// memory as bf16 (half a step of bf16 off; the decode step, which waits for
// memory anyway, multiplies queries and weights as pairs of bf16 instead: here
// a pair would double the products of P V), O += P V.  Each query tile has two
// S buffers, so the next tile's scores are there when a softmax ends, whatever
// its latency.  (Tiles of 128 keys with one S buffer, whose products take a
// fifth less of the pipe's time, took 997 us for the chunk below: a softmax then
// waits for the scores and the scores for it.)
//
// What bounds it.  Two query tiles take about 1440 cycles a key tile, of which
// the products need 1280 (Q K^T with 64 keys reads Q from shared memory for
// half the work, 48 cycles an instruction instead of 32): 2048 rows of 32 heads
// over 30000 cached tokens take 627 us in short bursts, 1.66 PFLOP/s, 0.88 of a
// large library product, and 675 to 680 call after call, when the clock falls
// (1.53 PFLOP/s).  At head_dim 64 the products are half and the time is not:
// the softmax's own chain takes 1450 cycles for the same scores (1024 rows over
// 30000: 293 us, 318 at 128).  One query tile (single tokens, drafts) is bound
// by device memory: one token over 262144 takes 85 us, 6.3 TB/s, 0.94 of a
// copy's rate.  What a task adds (its queries, its epilogue: 4 to 5 us) weighs
// on short prompts: 4095 rows from nothing take 99 us, 0.73 of the products'
// floor.
//
// How the pages meet the matrix instructions.  A page's K or V block is
// [d][16 slots] bf16, 32 bytes a dimension: with a 32-byte swizzle that is
// exactly a K-major B operand of 16 keys for P V, and an MN-major one for
// Q K^T.  Copies of 32-byte rows would be slow, so a block is copied as rows
// of 128 bytes with the 128-byte swizzle.  That one moves address bits 4-6 by
// bits 7-9; the 32-byte swizzle only moves bit 4 by bit 7.  The difference
// exchanges dimensions: row r of the operand holds dimension r ^ ((r >> 3) & 3).
// Q's columns are stored in the same order, and O's are read in it.
//
// 8-bit blocks (codes, then the slots' scales) are copied as they are and
// turned into that layout by warps of their own: a code times a power of two is
// a bf16 number, so nothing is rounded (outside bf16's normal range).  A tile
// then passes one step more before its products, and no pipe is full: of few
// rows the issue slots are half taken, shared memory's data pipe 0.6 (warps and
// matrix instructions together), the ALUs 0.36, XU 0.08.  37 rows over 109594
// tokens take 43.3 us (the same over bf16 pages, twice the bytes, 42.6), 1024
// rows over 30000 cached ones 428 us.  The 15 warps' 128 registers a thread
// spill 60 bytes at head_dim 128 and 52 at 64; the 11 warps of bf16 have 168
// and spill none at 128, 4 at 64.
// (K's codes fed to 8-bit products as they lie, with Q in two parts and the
// scales on the scores, left V alone to convert, and took 75 and 546 us with
// 57 and 580 at the time: the softmax then had the scales' work.)
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <math.h>

#include "chunk.h"
#include "mk.h"
#include "ptx.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr unsigned FULL = 0xffffffffu;
constexpr int TILE_PAGES = KV_TILE / PAGE;
constexpr unsigned long long WAIT_NS = 2000000000ull;   // limit of every wait
constexpr float RESCALE = 8.f;     // a row's sums are rescaled when its maximum grew by a factor of 2^8

// Warps: 0-3 softmax of query tile 0, 4-7 of tile 1 (without one: conversion),
// 8 copies, 9 and 10 matrix instructions of each query tile (two, so that one's
// products run while the other waits), 11-14 conversion of 8-bit tiles.  A block
// whose tasks all have one query tile converts K in warps 11-14 and V in 4-7,
// a page each; another one K in 11 and 12, V in 13 and 14, two pages each.
constexpr int W_COPY = 8, W_MMA = 9, W_CONV = 11;

template <int D, bool E4M3>
struct Cfg {
  static constexpr int THREADS = (E4M3 ? 15 : 11) * 32;
  static constexpr int Q_BYTES = Q_TILE * D * 2;
  static constexpr int PAGE_BYTES = D * PAGE * 2;             // a page's K or V as bf16
  static constexpr int STAGE = TILE_PAGES * PAGE_BYTES;       // a key tile's K or V
  static constexpr int RAW_PAGE = (D + 1) * PAGE;             // a page's 8-bit block
  static constexpr int RAW = TILE_PAGES * 2 * RAW_PAGE;       // a tile's K and V, page by page as in the pool
  // shared memory: two query tiles, K's and V's rings of bf16 tiles, a ring
  // of 8-bit tiles; D = 64 has twice the stages in the same bytes
  static constexpr int NST = (E4M3 ? 3 : 5) * (128 / D);
  static constexpr int NRAW = E4M3 ? 4 * (128 / D) : 0;
  static constexpr int OFF_KV = 2 * Q_BYTES, OFF_RAW = OFF_KV + 2 * NST * STAGE, OFF_CTL = OFF_RAW + NRAW * RAW;
  // V is 0 for K's ring, 1 for V's
  __device__ static constexpr int kv(int v, int i) { return OFF_KV + (v * NST + i) * STAGE; }
  __device__ static constexpr int raw(int i, int page, int v) { return OFF_RAW + i * RAW + (page * 2 + v) * RAW_PAGE; }
  static constexpr int SMEM = OFF_CTL + 1024 + 1024;          // control words, and room to align the base
  // tensor memory columns: two S buffers (and P over them) of each query tile, O of each
  static constexpr int T_S = 0, T_O = 4 * KV_TILE, T_COLS = 512;
  static_assert(T_O + 2 * D <= T_COLS, "tensor memory");
  static_assert(SMEM <= 232448, "shared memory");
};

struct Ctl {
  uint64_t full[2][10], empty[2][10], raw_full[8], raw_empty[8];
  uint64_t q_ready[2], s_full[2][2], p_ready[2][2], o_done[2], o_full[2], drain;
  uint32_t tmem;
  int fail;
};
static_assert(sizeof(Ctl) <= 1024, "control words");

struct Args {
  ChunkView c;
  const __nv_bfloat16* q;
  const uint8_t* pool;       // 8-bit pool
  __nv_bfloat16* out;
  bool wide_out;             // out is 32-byte aligned
  int oob;                   // a row of the tensor map past its end: reads zeros
};

// A wait that gives up after WAIT_NS, or once another of the block did.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try(bar, parity)) {
    if (*(volatile int*)&ctl->fail) return false;
    if (now_ns() - t0 > WAIT_NS) {
      *(volatile int*)&ctl->fail = 1;
      atomicCAS(status, 0, MK_ERR_DEP_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same for one thread, and for a warp, whose lanes agree on the outcome.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  return mbar_try(bar, parity) || wait_slow(bar, parity, ctl, status);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  const bool ok = mbar_try(bar, parity) || wait_slow(bar, parity, ctl, status);
  return __all_sync(FULL, ok);
}
// Two of them at once.
__device__ __forceinline__ bool wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, Ctl* ctl, int* status) {
  const bool ra = mbar_try(a, pa), rb = mbar_try(b, pb);
  const bool ok = (ra || wait_slow(a, pa, ctl, status)) && (rb || wait_slow(b, pb, ctl, status));
  return __all_sync(FULL, ok);
}

// Softmax of one query tile over a task's key tiles; a thread has a row.  g
// counts the query tile's key tiles over the tasks before, v_last is the page of
// V that the request ends within (in the stage that v_full tells of), if any.
// False when a wait gave up.
struct RowSums {
  float m, l;                    // maximum and sum of the softmax
};
template <int D, bool E4M3>
__device__ __forceinline__ bool softmax_rows(const Args& a, const AttnTask& t, int qt, int g, uint32_t tmem, uint8_t* v_last,
                                             uint64_t* v_full, uint32_t v_phase, RowSums& sums, Ctl* ctl) {
  using C = Cfg<D, E4M3>;
  int* status = a.c.status;
  const int warp = threadIdx.x / 32 % 4, lane = threadIdx.x % 32, row = warp * 32 + lane;
  const int G = a.c.G, per = Q_TILE / G;
  const int ntok = min(per, t.ntok - qt * per), rows = ntok * G;
  const bool live = warp * 32 < rows;            // a warp without rows only keeps the pace
  const int first_pos = t.pos + qt * per, pos = first_pos + min(row / G, ntok - 1);   // the tile's lowest, the row's own
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t ts = tmem + lanes + C::T_S + qt * 2 * KV_TILE, to = tmem + lanes + C::T_O + qt * D;
  const float sc = 1.4426950408889634f * rsqrtf((float)D);   // log2(e) / sqrt(d)
  float m = -INFINITY;
  f32x2 l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
  for (int j = 0; j < t.ntile; ++j) {
    const int at = g + j, buf = at & 1;
    if (!wait(&ctl->s_full[qt][buf], at >> 1 & 1, ctl, status)) return false;
    tc_after();
    if (live) {
      const int key0 = (t.tile0 + j) * KV_TILE;
      uint32_t s[KV_TILE];
#pragma unroll
      for (int c = 0; c < KV_TILE; c += 32) tmem_ld32(ts + buf * KV_TILE + c, s + c);
      tmem_wait_ld();
      if (key0 + KV_TILE - 1 > first_pos) {      // keys behind a row's position
        const int seen = pos - key0 + 1;
#pragma unroll
        for (int c = 0; c < KV_TILE; ++c)
          if (c >= seen) s[c] = 0xff800000u;
      }
      float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < KV_TILE; c += 2) mx[c / 2 % 4] = max3(mx[c / 2 % 4], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
      const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
      // The old maximum serves while it is not far below: the weights stay
      // within 2^RESCALE, and O keeps its scale.
      if (j == 0) {
        m = top;
      } else if (__any_sync(FULL, (top - m) * sc > RESCALE)) {
        const float f = top > m ? exp2_approx((m - top) * sc) : 1.f;
        l2[0] = mul2(l2[0], pair(f, f));
        l2[1] = mul2(l2[1], pair(f, f));
        m = top;
        if (!wait(&ctl->o_done[qt], (at - 1) & 1, ctl, status)) return false;   // the tile before is in O
        tc_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(to + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(to + c, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : -m * sc;   // a row that sees none of these keys: all weights 0
      const f32x2 sc2 = pair(sc, sc), base2 = pair(base, base);
#pragma unroll
      for (int c = 0; c < KV_TILE; c += 2) {
        float p0, p1;
        split(fma2(pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, base2), p0, p1);
        p0 = exp2_approx(p0);
        p1 = exp2_approx(p1);
        l2[c / 2 % 2] = add2(l2[c / 2 % 2], pair(p0, p1));
        s[c / 2] = pack_bf16(p0, p1);            // weights meet V as bf16, their sum stays fp32
      }
      tmem_st32(ts + buf * KV_TILE, s);
      tmem_wait_st();
    }
    if (!E4M3 && j == t.ntile - 1 && v_last) {
      // Slots behind the request's end hold anything, and 0 times a NaN is
      // one: in V they become 0 (both query tiles' threads write the same).
      if (!wait(v_full, v_phase, ctl, status)) return false;
      if (row < D) {
        const int keep = t.total % PAGE;         // slots of the last page that are the request's
        uint32_t* chunk = reinterpret_cast<uint32_t*>(v_last + row * 32);
        const int flip = (row >> 2 & 1) * 4;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const uint32_t mask = keep >= 2 * w + 2 ? ~0u : keep == 2 * w + 1 ? 0xffffu : 0u;
          if (mask != ~0u) chunk[w ^ flip] &= mask;
        }
      }
      fence_async();
    }
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->p_ready[qt][buf]);
  }
  float la, lb, lc, ld;
  split(l2[0], la, lb);
  split(l2[1], lc, ld);
  sums = {m, (la + lb) + (lc + ld)};
  return true;
}

// 32 bytes of a thread: a whole sector in one store where the address allows
// it (16-byte stores of 32 rows took 3.1 us a tile, these 1.9).
__device__ __forceinline__ void store32(void* p, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// O to its place: rows of the output, or split rows with their sums.
template <int D, bool E4M3>
__device__ __forceinline__ void store_rows(const Args& a, const AttnTask& t, int qt, uint32_t tmem, RowSums sums) {
  using C = Cfg<D, E4M3>;
  const int warp = threadIdx.x / 32 % 4, row = warp * 32 + threadIdx.x % 32;
  const int G = a.c.G, per = Q_TILE / G, rows = min(per, t.ntok - qt * per) * G;
  if (warp * 32 >= rows) return;
  const uint32_t to = tmem + ((uint32_t)(warp * 32) << 16) + C::T_O + qt * D;
  const int in_block = qt * per * G + row;       // row of the task's block
  const size_t at = ((size_t)(t.row + qt * per + row / G) * a.c.nq + (size_t)t.kvh * G + row % G) * D;
  const float inv = 1.f / sums.l;
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld32(to + c, o);
    tmem_wait_ld();
    if (row < rows) {
      uint32_t v[32];                            // 8 columns at a time: dimensions exchanged by (column >> 3) & 3
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = o[(i & ~7) + ((i & 7) ^ (i >> 3))];
      if (t.part < 0) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
        store32(a.out + at + c, w, a.wide_out);
        store32(a.out + at + c + 16, w + 8, a.wide_out);
      } else {
        float* po = a.c.part_o + ((size_t)t.part + in_block) * D + c;
#pragma unroll
        for (int i = 0; i < 32; i += 8) store32(po + i, v + i, true);
      }
    }
  }
  if (t.part >= 0 && row < rows)
    a.c.part_ml[(size_t)t.part + in_block] = make_float2(sums.m * (1.4426950408889634f * rsqrtf((float)D)), sums.l);
}

// A query tile into shared memory: two column halves of 128-byte rows with the
// 128-byte swizzle, dimensions in the cache's order; rows past the last are 0.
template <int D>
__device__ __forceinline__ void load_q(const Args& a, const AttnTask& t, int qt, uint8_t* dst) {
  const int G = a.c.G, per = Q_TILE / G, rows = min(per, t.ntok - qt * per) * G, tid = threadIdx.x % 128;
  const __nv_bfloat16* src = a.q + ((size_t)(t.row + qt * per) * a.c.nq + (size_t)t.kvh * G) * D;
  constexpr int N = D / 8;                       // 16-byte pieces of a row, and of a thread: all in flight at once
  const int g = tid % N, by_g = (65536 + G - 1) / G;   // row / G = row * by_g >> 16 for rows of a tile
  uint4 piece[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = tid / N + i * (128 / N);
    piece[i] = make_uint4(0, 0, 0, 0);
    const int token = row * by_g >> 16;
    if (row < rows) piece[i] = reinterpret_cast<const uint4*>(src + ((size_t)token * a.c.nq + (row - token * G)) * D)[g];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = tid / N + i * (128 / N);
    uint4 v = piece[i];
    if (g & 1) {                                 // neighbours exchanged
      v.x = v.x << 16 | v.x >> 16; v.y = v.y << 16 | v.y >> 16;
      v.z = v.z << 16 | v.z >> 16; v.w = v.w << 16 | v.w >> 16;
    }
    if (g & 2) v = make_uint4(v.y, v.x, v.w, v.z);   // pairs exchanged
    *reinterpret_cast<uint4*>(dst + (g / 8) * (Q_TILE * 128) + row * 128 + ((g % 8) ^ (row & 7)) * 16) = v;
  }
}

// The same queries on their way to L2 while the task before is worked on.
template <int D>
__device__ __forceinline__ void prefetch_q(const Args& a, const AttnTask& t, int qt) {
  const int G = a.c.G, per = Q_TILE / G, rows = min(per, t.ntok - qt * per) * G, row = threadIdx.x % 128;
  if (row >= rows) return;
  const __nv_bfloat16* src = a.q + ((size_t)(t.row + qt * per + row / G) * a.c.nq + (size_t)t.kvh * G + row % G) * D;
#pragma unroll
  for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
}

// One page's 8-bit block as bf16 in the operands' layout, by a warp: rows
// (dimensions) me, me + 32, ...; `live` slots, the others 0.
template <int D>
__device__ __forceinline__ void convert_page(const uint8_t* raw, uint8_t* dst, int live, int me) {
  // 2^(e - 127): e is a bf16 number's exponent too, and 2^-127 the subnormal
  // 0x40 (its maximum is a fiftieth of the time of few rows; asking first
  // whether a page has such a slot was no less)
  uint32_t scale[8];
  uint4 code[D / 32];                            // every row's read before the first write: they may not alias
  {
    const uint4 e4 = *reinterpret_cast<const uint4*>(raw + D * PAGE);
    const uint32_t ew[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) scale[i] = __vmaxu2(__byte_perm(ew[i / 2], 0, i % 2 ? 0x4342 : 0x4140) << 7, 0x00400040u);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) code[i] = *reinterpret_cast<const uint4*>(raw + (me + i * 32) * PAGE);
  }
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    const int d = me + k * 32;
    const uint32_t cw[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(e4m3x2_to_bf16x2(cw[i / 2] >> (i % 2 * 16)), scale[i]);
    if (live < PAGE) {                           // the request's last page
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = live >= 2 * i + 2 ? o[i] : live == 2 * i + 1 ? o[i] & 0xffffu : 0u;
    }
    const int row = d ^ (d >> 3 & 3), flip = row >> 2 & 1;
    *reinterpret_cast<uint4*>(dst + row * 32 + flip * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + row * 32 + (flip ^ 1) * 16) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// The K (v = 0) or V tiles of a block's tasks to bf16, pages [p0, p1) of each:
// every converting warp passes every tile in turn, so a barrier is never two
// phases away from what the warp waits for.
template <int D>
__device__ __forceinline__ void convert_tiles(const Args& a, int t0, int t1, uint8_t* smem, int v, int p0, int p1, Ctl* ctl) {
  using C = Cfg<D, true>;
  const int lane = threadIdx.x % 32;
  int ri = 0, si = 0, r_ph = 0, s_ph = 0;
  for (int i = t0; i < t1; ++i) {
    const int tile0 = __ldg(&a.c.tasks[i].tile0), ntile = __ldg(&a.c.tasks[i].ntile), total = __ldg(&a.c.tasks[i].total);
    for (int j = 0; j < ntile; ++j) {
      // (a fresh barrier has no phase behind it, and says that one of parity 1 is over)
      if (!wait_both(&ctl->raw_full[ri], r_ph, &ctl->empty[v][si], s_ph ^ 1, ctl, a.c.status)) return;
      const int left = total - (tile0 + j) * KV_TILE;   // the request's keys from the tile on
      for (int p = p0; p < p1; ++p)
        convert_page<D>(smem + C::raw(ri, p, v), smem + C::kv(v, si) + p * C::PAGE_BYTES,
                        min(PAGE, max(0, left - p * PAGE)), lane);
      fence_async();
      __syncwarp();
      if (lane < 2) mbar_arrive(lane ? &ctl->raw_empty[ri] : &ctl->full[v][si]);
      if (++ri == C::NRAW) { ri = 0; r_ph ^= 1; }
      if (++si == C::NST) { si = 0; s_ph ^= 1; }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::THREADS, 1)
    k_attend(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map) {
  using C = Cfg<D, E4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int per = Q_TILE / a.c.G;
  const int t0 = __ldg(a.c.cta_start + blockIdx.x), t1 = __ldg(a.c.cta_start + blockIdx.x + 1);
  int* status = a.c.status;
  if (stale(a.c)) return;
  // the first task, and the copying warp's first pages, arrive during the setup
  AttnTask t = a.c.tasks[t0];
  const bool two = t.two;
  constexpr int GROUP = 32 / TILE_PAGES;         // tiles whose page numbers a warp's lanes hold
  auto pages = [&](const AttnTask& t, int j) {
    const int page = (t.tile0 + j) * TILE_PAGES + lane;
    return page < (t.total + PAGE - 1) / PAGE ? __ldg(a.c.pt + t.pt + page) : -1;
  };
  int ids = -1, more = -1;
  if (warp == W_COPY) {
    ids = pages(t, 0);
    more = pages(t, GROUP);
  }
  if (tid == 0) {
    for (int v = 0; v < 2; ++v) {
      for (int i = 0; i < C::NST; ++i) {
        mbar_init(&ctl->full[v][i], !E4M3 ? 1 : two ? 2 : 4);   // the copies' issue, or the converting warps
        mbar_init(&ctl->empty[v][i], 2);                        // both query tiles' products
      }
    }
    for (int i = 0; i < C::NRAW; ++i) {
      mbar_init(&ctl->raw_full[i], 1);
      mbar_init(&ctl->raw_empty[i], two ? 4 : 8);   // the converting warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_ready[i], 4);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&ctl->s_full[i][k], 1);
        mbar_init(&ctl->p_ready[i][k], 4);
      }
      mbar_init(&ctl->o_done[i], 1);
      mbar_init(&ctl->o_full[i], 1);
    }
    mbar_init(&ctl->drain, 2);
    ctl->fail = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) tmem_alloc<C::T_COLS>(&ctl->tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl->tmem;
  bool ok = true;
  // So far only the chunk's own tables were read, which no kernel writes.
  await_stream();
  allow_next();

  if (warp < 8 && (warp < 4 || two)) {           // ---- softmax of a query tile
    const int qt = warp / 4;
    uint8_t* const q_smem = smem + qt * C::Q_BYTES;
    auto has = [&](const AttnTask& t) { return qt == 0 || t.ntok > per; };
    auto queries = [&](const AttnTask& t) {      // the tile's queries; the last task's scores are done
      load_q<D>(a, t, qt, q_smem);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_ready[qt]);
    };
    int g = 0, all = 0;                          // key tiles so far: of this query tile, of the block
    uint32_t tasks = 0;                          // of this query tile
    if (has(t)) queries(t);
    for (int i = t0; i < t1; ++i) {
      const AttnTask next = a.c.tasks[min(i + 1, t1 - 1)];
      all += t.ntile;
      if (i + 1 < t1 && has(next)) prefetch_q<D>(a, next, qt);
      if (has(t)) {
        const int left = t.total - (t.tile0 + t.ntile - 1) * KV_TILE, last = (all - 1) % C::NST;
        uint8_t* v_last = left < KV_TILE && t.total % PAGE ? smem + C::kv(1, last) + left / PAGE * C::PAGE_BYTES : nullptr;
        RowSums sums;
        if (!softmax_rows<D, E4M3>(a, t, qt, g, tmem, v_last, &ctl->full[1][last], (all - 1) / C::NST & 1, sums, ctl)) break;
        if (i + 1 < t1 && has(next)) queries(next);
        if (!wait(&ctl->o_full[qt], tasks & 1, ctl, status)) break;
        tc_after();
        store_rows<D, E4M3>(a, t, qt, tmem, sums);
        g += t.ntile;
        ++tasks;
      } else if (i + 1 < t1 && has(next)) {
        queries(next);
      }
      t = next;
    }
  } else if (warp == W_COPY) {                   // ---- copies
    // issued by one lane: by four, a page each, they took twice the time
    constexpr int N = E4M3 ? C::NRAW : C::NST;
    int at[2] = {0, 0};                          // tiles issued of K and V (8 bits: of both)
    auto full = [&](int v, int i) { return E4M3 ? &ctl->raw_full[i] : &ctl->full[v][i]; };
    auto copy = [&](const AttnTask& t, int v, int j, int ids) {
      const int u = at[v], s = u % N;
      if (u >= N && !wait(E4M3 ? &ctl->raw_empty[s] : &ctl->empty[v][s], (u / N & 1) ^ 1, ctl, status)) return false;
      int id[TILE_PAGES];
#pragma unroll
      for (int p = 0; p < TILE_PAGES; ++p) id[p] = __shfl_sync(FULL, ids, (j * TILE_PAGES + p) % 32);
      if (elect_one()) {
        if constexpr (E4M3) {                    // a page's K and V blocks lie side by side
          uint32_t pages = 0;
#pragma unroll
          for (int p = 0; p < TILE_PAGES; ++p) pages += id[p] >= 0;
          mbar_arrive_tx(full(v, s), pages * 2 * C::RAW_PAGE);
#pragma unroll
          for (int p = 0; p < TILE_PAGES; ++p)
            if (id[p] >= 0)
              bulk_copy(smem + C::raw(s, p, 0), a.pool + ((size_t)id[p] * a.c.nkv + t.kvh) * 2 * C::RAW_PAGE, 2 * C::RAW_PAGE,
                        full(v, s));
        } else {                                 // a page past the end: zeros
          mbar_arrive_tx(full(v, s), C::STAGE);
#pragma unroll
          for (int p = 0; p < TILE_PAGES; ++p)
            tma_2d(smem + C::kv(v, s) + p * C::PAGE_BYTES, &map, 0,
                   id[p] >= 0 ? (int)(((size_t)id[p] * a.c.nkv + t.kvh) * 2 + v) * (D / 4) : a.oob, full(v, s));
        }
      }
      __syncwarp();
      ++at[v];
      return true;
    };
    for (int i = t0; i < t1 && ok; ++i) {        // page numbers: those of 8 tiles, and of the next 8
      if (i > t0) {
        t = a.c.tasks[i];
        ids = pages(t, 0);
        more = pages(t, GROUP);
      }
      if (!E4M3) ok = copy(t, 0, 0, ids);        // in the order of use: K goes one tile ahead
      for (int j = 0; j < t.ntile && ok; ++j) {
        if (j > 0 && j % GROUP == 0) {
          ids = more;
          more = pages(t, j + GROUP);
        }
        if (E4M3) ok = copy(t, 0, j, ids);
        else ok = (j + 1 == t.ntile || copy(t, 0, j + 1, (j + 1) % GROUP ? ids : more)) && copy(t, 1, j, ids);
      }
    }
    if (!ok)                                     // given up: what is in flight still lands before the block ends
      for (int v = 0; v < 2; ++v)
        for (int u = max(0, at[v] - N); u < at[v]; ++u) {
          const unsigned long long since = now_ns();
          while (!mbar_try(full(v, u % N), u / N & 1) && now_ns() - since < WAIT_NS) {}
        }
  } else if (warp == W_MMA || warp == W_MMA + 1) {   // ---- matrix instructions: one thread a query tile
    const int qt = warp - W_MMA;
    if (elect_one()) {
      constexpr uint32_t I_QK = umma_idesc(Q_TILE, KV_TILE, true), I_PV = umma_idesc(Q_TILE, D, false);
      const uint64_t q_desc = umma_desc(smem_u32(smem + qt * C::Q_BYTES), 16, 1024, 2);
      const uint64_t k_desc = umma_desc(smem_u32(smem + C::kv(0, 0)), C::PAGE_BYTES, 256, 6);
      const uint64_t v_desc = umma_desc(smem_u32(smem + C::kv(1, 0)), 16, 256, 6);
      const uint32_t ts = tmem + C::T_S + qt * 2 * KV_TILE, to = tmem + C::T_O + qt * D;
      int ki = 0, vi = 0, g = 0;                 // ring places, key tiles of this query tile
      uint32_t k_ph = 0, v_ph = 0, tasks = 0;
      auto next_k = [&] { if (++ki == C::NST) { ki = 0; k_ph ^= 1; } };
      auto next_v = [&] { if (++vi == C::NST) { vi = 0; v_ph ^= 1; } };
      auto scores = [&](int buf) {               // S = Q K^T, 16 dimensions at a time
        const uint64_t kd = k_desc + (uint32_t)(ki * C::STAGE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ss(ts + buf * KV_TILE, q_desc + (((k / 4) * (Q_TILE * 128) + (k % 4) * 32) >> 4), kd + (k * 512 >> 4), I_QK, k > 0);
        umma_commit(&ctl->s_full[qt][buf]);
        umma_commit(&ctl->empty[0][ki]);
        next_k();
      };
      for (int i = t0; i < t1 && ok; ++i) {
        const int ntile = __ldg(&a.c.tasks[i].ntile), ntok = __ldg(&a.c.tasks[i].ntok);
        if (qt == 1 && ntok <= per) {            // no rows: every tile is done at once
          for (int j = 0; j < ntile; ++j) {
            if (!(ok = wait_one(&ctl->full[0][ki], k_ph, ctl, status))) break;
            mbar_arrive(&ctl->empty[0][ki]);
            next_k();
            if (!(ok = wait_one(&ctl->full[1][vi], v_ph, ctl, status))) break;
            mbar_arrive(&ctl->empty[1][vi]);
            next_v();
          }
          continue;
        }
        ok = wait_one(&ctl->q_ready[qt], tasks & 1, ctl, status) && wait_one(&ctl->full[0][ki], k_ph, ctl, status);
        if (!ok) break;
        ++tasks;
        tc_after();
        scores(g & 1);
        // Scores go one tile ahead, into the buffer that the products of the
        // tile before have left.
        for (int j = 0; j < ntile; ++j, ++g) {
          const bool more = j + 1 < ntile;
          if (more) {
            if (!(ok = wait_one(&ctl->full[0][ki], k_ph, ctl, status))) break;
            scores((g + 1) & 1);
          }
          if (!(ok = wait_one(&ctl->full[1][vi], v_ph, ctl, status))) break;
          if (!(ok = wait_one(&ctl->p_ready[qt][g & 1], g >> 1 & 1, ctl, status))) break;
          tc_after();
          const uint64_t vd = v_desc + (uint32_t)(vi * C::STAGE >> 4);
#pragma unroll
          for (int k = 0; k < TILE_PAGES; ++k)   // O += P V, a page's 16 keys at a time
            umma_ts(to, ts + (g & 1) * KV_TILE + k * 8, vd + (k * C::PAGE_BYTES >> 4), I_PV, j > 0 || k > 0);
          umma_commit(&ctl->empty[1][vi]);
          umma_commit(&ctl->o_done[qt]);
          if (!more) umma_commit(&ctl->o_full[qt]);
          next_v();
        }
      }
      // Products and their arrivals are done before the block's memory is
      // given back, after a wait that gave up too.
      umma_commit(&ctl->drain);
      const unsigned long long since = now_ns();
      while (!mbar_try(&ctl->drain, 0) && now_ns() - since < WAIT_NS) {}
    }
    __syncwarp();
  } else if constexpr (E4M3) {                   // ---- 8-bit tiles to bf16
    if (!two) convert_tiles<D>(a, t0, t1, smem, warp < 8, warp < 8 ? warp - 4 : warp - W_CONV,
                               (warp < 8 ? warp - 4 : warp - W_CONV) + 1, ctl);
    else convert_tiles<D>(a, t0, t1, smem, (warp - W_CONV) / 2, (warp - W_CONV) % 2 * 2, (warp - W_CONV) % 2 * 2 + 2, ctl);
  }

  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == W_MMA) tmem_free<C::T_COLS>(tmem);
}

// Joins the parts of rows whose keys were split; W warps share a row (4 where
// a row has many parts: 38 of them took 4.9 us with one).  The order of the
// sums is fixed, so the same call gives the same bits.
template <int D, int W>
__global__ void __launch_bounds__(128) k_join(ChunkView c, __nv_bfloat16* out) {
  constexpr int E = D / 32;
  __shared__ float part[W][D + 1];
  const JoinTask t = c.joins[blockIdx.x];        // within the chunk's memory; nothing of it is used before the next line
  if (stale(c)) return;
  allow_next();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rows = t.ntok * c.G, row = W == 4 ? blockIdx.y : blockIdx.y * 4 + warp, w = W == 4 ? warp : 0;
  if (row >= rows) return;                       // the whole block where warps share a row
  await_stream();
  const float2* ml = c.part_ml + (size_t)t.part0 + row;
  const float* po = c.part_o + ((size_t)t.part0 + row) * D + lane * E;
  float m = -INFINITY;
  for (int p = lane; p < t.nparts; p += 32) m = fmaxf(m, ml[(size_t)p * rows].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
  float acc[E] = {}, l = 0.f;
#pragma unroll 8
  for (int p = w; p < t.nparts; p += W) {
    const float2 s = ml[(size_t)p * rows];
    const float f = exp2f(s.x - m);              // 0 for a part whose keys this row does not see
    l += s.y * f;
    float v[E];
    if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(po + (size_t)p * rows * D);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(po + (size_t)p * rows * D);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * v[e];
  }
  if constexpr (W == 4) {
#pragma unroll
    for (int e = 0; e < E; ++e) part[w][lane * E + e] = acc[e];
    if (lane == 0) part[w][D] = l;
    __syncthreads();
    if (w) return;
    l = (part[0][D] + part[1][D]) + (part[2][D] + part[3][D]);
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = (part[0][lane * E + e] + part[1][lane * E + e]) + (part[2][lane * E + e] + part[3][lane * E + e]);
  }
  const float inv = 1.f / l;
  uint32_t* o = reinterpret_cast<uint32_t*>(
      out + ((size_t)(t.row + row / c.G) * c.nq + (size_t)t.kvh * c.G + row % c.G) * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) o[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
}

// The pool's K and V blocks as rows of 128 bytes, one block a box.
cudaError_t pool_map(const ChunkView& c, const void* pool, CUtensorMap* map, int* oob) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return cudaErrorNotSupported;
  const long long rows = (long long)c.num_pages * c.nkv * 2 * (c.d / 4);
  const cuuint64_t dim[2] = {64, (cuuint64_t)rows}, stride[1] = {128};
  const cuuint32_t box[2] = {64, (cuuint32_t)(c.d / 4)}, step[2] = {1, 1};
  *oob = (int)rows;
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dim, stride, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int D, bool E4M3>
cudaError_t launch(const ChunkView& c, const void* q, const void* pool, void* out, cudaStream_t st) {
  using C = Cfg<D, E4M3>;
  Args a = {c, (const __nv_bfloat16*)q, (const uint8_t*)pool, (__nv_bfloat16*)out, (uintptr_t)out % 32 == 0, 0};
  CUtensorMap map = {};
  cudaError_t e = E4M3 ? cudaSuccess : pool_map(c, pool, &map, &a.oob);
  if (e == cudaSuccess) e = allow((const void*)k_attend<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(k_attend<D, E4M3>, c.ctas, C::THREADS, C::SMEM, 1, st, a, map);
  if (e != cudaSuccess || !c.njoins) return e;
  const bool many = c.max_parts > 8;
  return launch_kernel(many ? k_join<D, 4> : k_join<D, 1>, dim3(c.njoins, many ? c.max_join_rows : (c.max_join_rows + 3) / 4),
                       128, 0, 1, st, c, (__nv_bfloat16*)out);
}

}  // namespace

cudaError_t launch_attend(const ChunkView& c, bool e4m3, const void* q, const void* pool, void* out, cudaStream_t st) {
  if (c.d == 64) return e4m3 ? launch<64, true>(c, q, pool, out, st) : launch<64, false>(c, q, pool, out, st);
  return e4m3 ? launch<128, true>(c, q, pool, out, st) : launch<128, false>(c, q, pool, out, st);
}

}  // namespace mk
