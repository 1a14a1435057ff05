// Attention of a chunk's rows over the paged cache.
//
// out = sum_s p_s v_s / sum_s p_s, p_s = 2^((q . k_s - m) log2(e) / sqrt(d)),
// over the positions s up to the row's own, in one pass over the cache with the
// running maximum m and sum of each row in fp32.
//
// One block works on one task: up to two query tiles (128 rows each: 128 / G
// tokens with the G heads that share a KV head, so a key tile is fetched once
// for all of them) of one request, against a run of key tiles (128 keys, 8
// pages).  Products run on the tensor cores: S = Q K^T into tensor memory,
// softmax in registers (one thread a row), P back to tensor memory as bf16, O
// += P V.  With two tiles one's products run while the other's softmax does.
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
// turned into that layout by four warps of their own: a code is a bf16 number
// after a shift, up to a factor 2^120 that its scale's multiplication takes
// along, so nothing is rounded.
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

// Warps: 0-3 softmax of query tile 0, 4-7 of tile 1, 8 copies, 9 matrix
// instructions, 10-13 conversion of 8-bit blocks.
constexpr int W_COPY = 8, W_MMA = 9, W_CONV = 10;

template <int D, bool E4M3>
struct Cfg {
  static constexpr int THREADS = (E4M3 ? 14 : 10) * 32;
  static constexpr int Q_BYTES = Q_TILE * D * 2;
  static constexpr int PAGE_BYTES = D * PAGE * 2;             // a page's K or V as bf16
  static constexpr int STAGE = TILE_PAGES * PAGE_BYTES;       // a key tile's K or V
  static constexpr int RAW_PAGE = (D + 1) * PAGE;             // a page's 8-bit block
  static constexpr int RAW = TILE_PAGES * RAW_PAGE;
  // shared memory: two query tiles, the ring of bf16 tiles, the ring of 8-bit
  // tiles; D = 64 has twice the stages in the same bytes
  static constexpr int NST = (E4M3 ? 3 : 5) * (128 / D);
  static constexpr int NRAW = E4M3 ? 4 * (128 / D) : 0;
  static constexpr int OFF_KV = 2 * Q_BYTES, OFF_RAW = OFF_KV + NST * STAGE, OFF_CTL = OFF_RAW + NRAW * RAW;
  static constexpr int SMEM = OFF_CTL + 1024 + 1024;          // control words, and room to align the base
  // tensor memory columns: S (and P over it) of each tile, O of each tile
  static constexpr int T_S = 0, T_O = 2 * KV_TILE, T_COLS = 512;
  static_assert(T_O + 2 * D <= T_COLS, "tensor memory");
  static_assert(SMEM <= 232448, "shared memory");
};

struct Ctl {
  uint64_t full[16], empty[16], raw_full[8], raw_empty[8];
  uint64_t q_ready, s_full[2], p_ready[2], o_full[2], drain;
  uint32_t tmem;
  int fail;
};
static_assert(sizeof(Ctl) <= 1024, "control words");

struct Args {
  ChunkView c;
  const __nv_bfloat16* q;
  const uint8_t* pool;       // 8-bit pool
  __nv_bfloat16* out;
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
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  const bool ok = mbar_try(bar, parity) || wait_slow(bar, parity, ctl, status);
  return __all_sync(FULL, ok);
}

// Place in a ring of n stages.
struct Ring {
  int n, i = 0;
  uint32_t ph = 0;
  __device__ explicit Ring(int n_) : n(n_) {}
  __device__ void next() {
    if (++i == n) {
      i = 0;
      ph ^= 1;
    }
  }
};

// Softmax of one query tile and its epilogue; a thread has a row.  False when
// a wait gave up.
template <int D, bool E4M3>
__device__ __forceinline__ bool softmax_rows(const Args& a, const AttnTask& t, const ChunkReq& r, int qt, uint32_t tmem,
                                             Ctl* ctl, int* status) {
  using C = Cfg<D, E4M3>;
  const int warp = threadIdx.x / 32 % 4, lane = threadIdx.x % 32, row = warp * 32 + lane;
  const int G = a.c.G, per = Q_TILE / G;
  const int ntok = min(per, t.ntok - qt * per), rows = ntok * G;
  const bool live = warp * 32 < rows;            // a warp without rows only keeps the pace
  const int tok = t.tok0 + qt * per + min(row / G, ntok - 1), pos = r.seq + tok;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t ts = tmem + lanes + C::T_S + qt * KV_TILE, to = tmem + lanes + C::T_O + qt * D;
  const float sc = 1.4426950408889634f * rsqrtf((float)D);   // log2(e) / sqrt(d)
  const int first_pos = r.seq + t.tok0 + qt * per;           // the tile's lowest position
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < t.ntile; ++j) {
    if (!wait(&ctl->s_full[qt], j & 1, ctl, status)) return false;
    tc_after();
    if (live) {
      const int key0 = (t.tile0 + j) * KV_TILE;
      uint32_t s[KV_TILE];
#pragma unroll
      for (int c = 0; c < KV_TILE; c += 32) tmem_ld32(ts + c, s + c);
      tmem_wait_ld();
      if (key0 + KV_TILE - 1 > first_pos) {      // keys behind a row's position
        const int seen = pos - key0 + 1;
#pragma unroll
        for (int c = 0; c < KV_TILE; ++c)
          if (c >= seen) s[c] = 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < KV_TILE; ++c) mx[c % 4] = fmaxf(mx[c % 4], __uint_as_float(s[c]));
      const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      // The old maximum serves while it is not far below: the weights stay
      // within 2^RESCALE, and O keeps its scale.
      if (j == 0) {
        m = top;
      } else if (__any_sync(FULL, (top - m) * sc > RESCALE)) {
        const float f = top > m ? exp2_approx((m - top) * sc) : 1.f;
        l *= f;
        m = top;
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
      float sum[4] = {};
#pragma unroll
      for (int c = 0; c < KV_TILE; c += 2) {
        const float p0 = exp2_approx(fmaf(__uint_as_float(s[c]), sc, base));
        const float p1 = exp2_approx(fmaf(__uint_as_float(s[c + 1]), sc, base));
        sum[c / 2 % 4] += p0 + p1;
        s[c / 2] = pack_bf16(p0, p1);            // weights meet V as bf16, their sum stays fp32
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st32(ts, s);
      tmem_st32(ts + 32, s + 32);
      tmem_wait_st();
    }
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->p_ready[qt]);
  }
  if (!wait(&ctl->o_full[qt], 0, ctl, status)) return false;
  tc_after();
  if (!live) return true;
  const int in_block = qt * per * G + row;       // row of the task's block
  const size_t at = ((size_t)(r.row0 + tok) * a.c.nq + (size_t)t.kvh * G + row % G) * D;
  const float inv = 1.f / l;
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld32(to + c, o);
    tmem_wait_ld();
    if (row < rows) {
#pragma unroll
      for (int g = 0; g < 32; g += 8) {          // 8 columns: dimensions exchanged by (column >> 3) & 3
        const int x = g >> 3 & 3;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(o[g + (i ^ x)]);
        if (t.part < 0) {
          *reinterpret_cast<uint4*>(a.out + at + c + g) =
              make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                         pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
        } else {
          float4* po = reinterpret_cast<float4*>(a.c.part_o + ((size_t)t.part + in_block) * D + c + g);
          po[0] = make_float4(v[0], v[1], v[2], v[3]);
          po[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
  if (t.part >= 0 && row < rows) a.c.part_ml[(size_t)t.part + in_block] = make_float2(m * sc, l);
  return true;
}

// A query tile into shared memory: two column halves of 128-byte rows with the
// 128-byte swizzle, dimensions in the cache's order; rows past the last are 0.
template <int D>
__device__ __forceinline__ void load_q(const Args& a, const AttnTask& t, const ChunkReq& r, int qt, uint8_t* dst) {
  const int G = a.c.G, per = Q_TILE / G, rows = min(per, t.ntok - qt * per) * G, tid = threadIdx.x % 128;
  const __nv_bfloat16* src = a.q + ((size_t)(r.row0 + t.tok0 + qt * per) * a.c.nq + (size_t)t.kvh * G) * D;
#pragma unroll 4
  for (int x = tid; x < Q_TILE * (D / 8); x += 128) {
    const int row = x / (D / 8), g = x % (D / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows) v = __ldg(reinterpret_cast<const uint4*>(src + ((size_t)(row / G) * a.c.nq + row % G) * D) + g);
    if (g & 1) {                                 // neighbours exchanged
      v.x = v.x << 16 | v.x >> 16; v.y = v.y << 16 | v.y >> 16;
      v.z = v.z << 16 | v.z >> 16; v.w = v.w << 16 | v.w >> 16;
    }
    if (g & 2) v = make_uint4(v.y, v.x, v.w, v.z);   // pairs exchanged
    *reinterpret_cast<uint4*>(dst + (g / 8) * (Q_TILE * 128) + row * 128 + ((g % 8) ^ (row & 7)) * 16) = v;
  }
}

// One page's 8-bit block as bf16 in the operands' layout, by 16 threads: rows
// (dimensions) me, me + 16, ...; `live` slots, the others 0.
template <int D>
__device__ __forceinline__ void convert_page(const uint8_t* raw, uint8_t* dst, int live, int me) {
  uint32_t mul[8], far[8];
  bool any_far = false;
  if (live > 0) {
    const uint4 e4 = *reinterpret_cast<const uint4*>(raw + D * PAGE);
    const uint32_t ew[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t a[2], b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = 2 * i + h;
        const int e = ew[slot / 4] >> (slot % 4 * 8) & 0xff;
        // scale 2^(e - 127) times 2^120, as a bf16 number's exponent; above
        // 2^127 the rest comes as a second factor
        const int lo = min(e, 134);
        a[h] = slot < live ? (uint32_t)(lo + 120) << 7 : 0u;
        b[h] = (uint32_t)(e - lo + 127) << 7;
        any_far |= e > 134 && slot < live;
      }
      mul[i] = a[0] | a[1] << 16;
      far[i] = b[0] | b[1] << 16;
    }
  }
#pragma unroll 2
  for (int d = me; d < D; d += 16) {
    uint32_t o[8] = {};
    if (live > 0) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(raw + d * PAGE);
      const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // two codes into the high bytes of 16-bit halves; sign stays, the
        // other 7 bits go to bf16's lowest exponent and highest mantissa bits
        const uint32_t x = __byte_perm(cw[i / 2], 0, i % 2 ? 0x3424 : 0x1404);
        o[i] = mul_bf16x2((x & 0x80008000u) | (x >> 4 & 0x07f007f0u), mul[i]);
      }
      if (any_far)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], far[i]);
    }
    const int row = d ^ (d >> 3 & 3), flip = row >> 2 & 1;
    *reinterpret_cast<uint4*>(dst + row * 32 + flip * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + row * 32 + (flip ^ 1) * 16) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::THREADS, 1)
    k_attend(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map) {
  using C = Cfg<D, E4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const AttnTask t = a.c.tasks[blockIdx.x];
  const ChunkReq r = a.c.reqs[t.req];
  const int nqt = t.ntok > Q_TILE / a.c.G ? 2 : 1;
  int* status = a.c.status;
  if (tid == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&ctl->full[i], E4M3 ? 4 : 1);    // converting warps, or the copy's issue
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < C::NRAW; ++i) {
      mbar_init(&ctl->raw_full[i], 1);
      mbar_init(&ctl->raw_empty[i], 4);
    }
    mbar_init(&ctl->q_ready, 4 * nqt);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_ready[i], 4);
      mbar_init(&ctl->o_full[i], 1);
    }
    mbar_init(&ctl->drain, 1);
    ctl->fail = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) tmem_alloc<C::T_COLS>(&ctl->tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl->tmem;
  const int total = r.seq + r.nnew, npages = (total + PAGE - 1) / PAGE;
  // K and V tiles pass through the ring in the order of their use: K 0, then
  // K j + 1 and V j for every j
  const int uses = 2 * t.ntile;
  auto tile_of = [&](int u, bool& v) -> int {
    v = u > 0 && (u % 2 == 0 || u == uses - 1);
    return u == 0 ? 0 : u == uses - 1 ? t.ntile - 1 : v ? u / 2 - 1 : (u + 1) / 2;
  };
  bool ok = true;

  if (warp < 4 * nqt) {                          // ---- softmax
    load_q<D>(a, t, r, warp / 4, smem + (warp / 4) * C::Q_BYTES);
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->q_ready);
    ok = softmax_rows<D, E4M3>(a, t, r, warp / 4, tmem, ctl, status);
  } else if (warp == W_COPY) {                   // ---- copies: a lane has a page
    const int n = E4M3 ? C::NRAW : C::NST;
    uint64_t* full = E4M3 ? ctl->raw_full : ctl->full;
    uint64_t* empty = E4M3 ? ctl->raw_empty : ctl->empty;
    Ring ring(n);
    int issued = 0;
    for (int u = 0; u < uses && ok; ++u, ring.next()) {
      if (u >= n && !(ok = wait(&empty[ring.i], ring.ph ^ 1, ctl, status))) break;
      bool v;
      const int page = (t.tile0 + tile_of(u, v)) * TILE_PAGES + lane;
      const bool there = lane < TILE_PAGES && page < npages;
      const int id = there ? __ldg(a.c.pt + r.pt + page) : 0;
      const size_t block = ((size_t)id * a.c.nkv + t.kvh) * 2 + v;
      if (E4M3) {
        const uint32_t bytes = __popc(__ballot_sync(FULL, there)) * C::RAW_PAGE;
        if (lane == 0) mbar_arrive_tx(&full[ring.i], bytes);
        __syncwarp();
        if (there)
          bulk_copy(smem + C::OFF_RAW + ring.i * C::RAW + lane * C::RAW_PAGE, a.pool + block * C::RAW_PAGE, C::RAW_PAGE,
                    &full[ring.i]);
      } else {
        if (lane == 0) mbar_arrive_tx(&full[ring.i], C::STAGE);
        __syncwarp();
        if (lane < TILE_PAGES)                   // a page past the end: zeros
          tma_2d(smem + C::OFF_KV + ring.i * C::STAGE + lane * C::PAGE_BYTES, &map, 0,
                 there ? (int)(block * (D / 4)) : a.oob, &full[ring.i]);
      }
      ++issued;
    }
    if (!ok)                                     // given up: what is in flight still lands before the block ends
      for (int u = max(0, issued - n); u < issued; ++u) {
        const unsigned long long t0 = now_ns();
        while (!mbar_try(&full[u % n], (u / n) & 1) && now_ns() - t0 < WAIT_NS) {}
      }
  } else if (warp == W_MMA) {                    // ---- matrix instructions
    constexpr uint32_t I_QK = umma_idesc(Q_TILE, KV_TILE, true), I_PV = umma_idesc(Q_TILE, D, false);
    const uint32_t sq = smem_u32(smem), skv = smem_u32(smem + C::OFF_KV);
    Ring ring(C::NST);
    auto scores = [&](int stage, int qt) {       // S = Q K^T, 16 dimensions at a time
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        umma_ss(tmem + C::T_S + qt * KV_TILE,
                umma_desc(sq + qt * C::Q_BYTES + (k / 4) * (Q_TILE * 128) + (k % 4) * 32, 16, 1024, 2),
                umma_desc(skv + stage * C::STAGE + k * 512, C::PAGE_BYTES, 256, 6), I_QK, k > 0);
      umma_commit(&ctl->s_full[qt]);
    };
    ok = wait(&ctl->q_ready, 0, ctl, status) && wait(&ctl->full[0], 0, ctl, status);
    if (ok) {
      tc_after();
      if (lane == 0) {
        for (int qt = 0; qt < nqt; ++qt) scores(0, qt);
        umma_commit(&ctl->empty[0]);
      }
      ring.next();
    }
    for (int j = 0; j < t.ntile && ok; ++j) {
      const bool more = j + 1 < t.ntile;
      int ks = 0;
      if (more) {
        ks = ring.i;
        if (!(ok = wait(&ctl->full[ring.i], ring.ph, ctl, status))) break;
        ring.next();
      }
      const int vs = ring.i;
      if (!(ok = wait(&ctl->full[ring.i], ring.ph, ctl, status))) break;
      ring.next();
      const int key0 = (t.tile0 + j) * KV_TILE;
      if (!E4M3 && total - key0 < KV_TILE && total % PAGE) {
        // slots behind the request's end hold anything, and 0 times a NaN is
        // one: they become 0 (conversion does it for 8-bit blocks)
        uint8_t* page = smem + C::OFF_KV + vs * C::STAGE + (total - key0) / PAGE * C::PAGE_BYTES;
        for (int row = lane; row < D; row += 32)
          for (int s = total % PAGE; s < PAGE; ++s)
            *reinterpret_cast<uint16_t*>(page + row * 32 + ((s >> 3) ^ (row >> 2 & 1)) * 16 + (s & 7) * 2) = 0;
        fence_async();
        __syncwarp();
      }
      for (int qt = 0; qt < nqt; ++qt) {
        if (!(ok = wait(&ctl->p_ready[qt], j & 1, ctl, status))) break;
        tc_after();
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < TILE_PAGES; ++k)   // O += P V, a page's 16 keys at a time
            umma_ts(tmem + C::T_O + qt * D, tmem + C::T_S + qt * KV_TILE + k * 8,
                    umma_desc(skv + vs * C::STAGE + k * C::PAGE_BYTES, 16, 256, 6), I_PV, j > 0 || k > 0);
          if (more) scores(ks, qt);
          else umma_commit(&ctl->o_full[qt]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0 && more) {                   // (nobody waits for the last stages)
        umma_commit(&ctl->empty[vs]);
        umma_commit(&ctl->empty[ks]);
      }
      __syncwarp();
    }
  } else if (E4M3 && warp >= W_CONV) {           // ---- 8-bit blocks to bf16
    Ring ring(C::NST), raw(C::NRAW);
    const int me = tid - W_CONV * 32;
    for (int u = 0; u < uses; ++u, ring.next(), raw.next()) {
      if (!(ok = wait(&ctl->raw_full[raw.i], raw.ph, ctl, status))) break;
      if (u >= C::NST && !(ok = wait(&ctl->empty[ring.i], ring.ph ^ 1, ctl, status))) break;
      bool v;
      const int key = (t.tile0 + tile_of(u, v)) * KV_TILE + me / 16 * PAGE;
      convert_page<D>(smem + C::OFF_RAW + raw.i * C::RAW + me / 16 * C::RAW_PAGE,
                      smem + C::OFF_KV + ring.i * C::STAGE + me / 16 * C::PAGE_BYTES, min(PAGE, max(0, total - key)), me % 16);
      fence_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->full[ring.i]);
        mbar_arrive(&ctl->raw_empty[raw.i]);
      }
    }
  }

  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == W_MMA) {
    if (ctl->fail && lane == 0) {                // products in flight end before their memory is given back
      umma_commit(&ctl->drain);
      const unsigned long long t0 = now_ns();
      while (!mbar_try(&ctl->drain, 0) && now_ns() - t0 < WAIT_NS) {}
    }
    __syncwarp();
    tmem_free<C::T_COLS>(tmem);
  }
}

// Joins the parts of rows whose keys were split: a warp has a row.  The order
// of the sum is the parts', so the same call gives the same bits.
template <int D>
__global__ void __launch_bounds__(128) k_join(ChunkView c, __nv_bfloat16* out) {
  constexpr int E = D / 32;
  const JoinTask t = c.joins[blockIdx.x];
  const int rows = t.ntok * c.G, row = blockIdx.y * 4 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (row >= rows) return;
  float m = -INFINITY;
  for (int p = lane; p < t.nparts; p += 32) m = fmaxf(m, c.part_ml[(size_t)t.part0 + (size_t)p * rows + row].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
  float acc[E] = {}, l = 0.f;
#pragma unroll 4
  for (int p = 0; p < t.nparts; ++p) {
    const size_t at = (size_t)t.part0 + (size_t)p * rows + row;
    const float2 ml = c.part_ml[at];
    const float w = exp2f(ml.x - m);             // 0 for a part whose keys this row does not see
    l += ml.y * w;
    float v[E];
    if (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(c.part_o + at * D + lane * 4);
      v[0] = x.x; v[1] = x.y; v[E - 2] = x.z; v[E - 1] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(c.part_o + at * D + lane * 2);
      v[0] = x.x; v[1] = x.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * v[e];
  }
  const float inv = 1.f / l;
  const ChunkReq r = c.reqs[t.req];
  uint32_t* o = reinterpret_cast<uint32_t*>(
      out + ((size_t)(r.row0 + t.tok0 + row / c.G) * c.nq + (size_t)t.kvh * c.G + row % c.G) * D + lane * E);
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
  Args a = {c, (const __nv_bfloat16*)q, (const uint8_t*)pool, (__nv_bfloat16*)out, 0};
  CUtensorMap map = {};
  cudaError_t e = E4M3 ? cudaSuccess : pool_map(c, pool, &map, &a.oob);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_attend<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  k_attend<D, E4M3><<<c.ntasks, C::THREADS, C::SMEM, st>>>(a, map);
  if (c.njoins) k_join<D><<<dim3(c.njoins, (2 * Q_TILE + 3) / 4), 128, 0, st>>>(c, (__nv_bfloat16*)out);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(const ChunkView& c, bool e4m3, const void* q, const void* pool, void* out, cudaStream_t st) {
  if (c.d == 64) return e4m3 ? launch<64, true>(c, q, pool, out, st) : launch<64, false>(c, q, pool, out, st);
  return e4m3 ? launch<128, true>(c, q, pool, out, st) : launch<128, false>(c, q, pool, out, st);
}

}  // namespace mk
