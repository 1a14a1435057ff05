// The experts' products over a chunk's rows (mk_experts_* in include/mk.h): gate
// and up with SwiGLU, and down with the gates, for each expert over the rows
// that were routed to it.
//
// C[rows of e, n] = A[rows of e, :] . W_e, on the tensor cores: tiles of 128 rows
// of one expert by NT columns, K in steps of 128 bytes.  A tile's rows are
// gathered by their token numbers on the way to shared memory (up: 16-byte
// copies of four warps), or lie side by side (down: boxes of a tensor map); its
// weights are one box of a tensor map.  A block works through the tiles t, t +
// blocks, ... of all experts; neighbours in that order share an expert's weights,
// which so come from device memory once.  One accumulator in tensor memory is
// read (SwiGLU or gates, rounding, stores) while the next one is summed.
//
// What bounds them (2048 hidden, 128 experts of 768, 8 a row).  Up to a few
// hundred rows the weights' bytes: 37 rows of up 96 us, 6.6 TB/s of what comes
// from device memory (0.81 of its cycles), 300 rows of down 64 us.  One row is a
// chain of latencies (lists, first weights, one tile of 96 columns a block of
// 128) and takes 12.8 us for 50 MB, down 7.5 us for 25 MB.  Of thousands of rows
// in bf16 a step of 128 bytes of K takes 48 KB and 416 ns, 118 GB/s an SM, which
// is what L2 gives it; the tiles of two SMs take over (experts_two.cu).  In 8 bits
// it takes 40 KB (192 columns) and some 400 ns, where the products need 246 at
// twice bf16's measured rate: 8143 rows take up 198 us (2.1 PFLOP/s) and down 118.
// Neither the scales, nor the gather, nor the results bound up by themselves: each
// left out gives about a twelfth, all three a fifth.  Down is bound by its
// results (88 us without).  (Times in short bursts; call after call for tenths of
// a second the clock falls, and up of 8143 rows takes 223 us.)
//
// 8 bits: codes and scales are what the block-scaled matrix instructions take.
// The scales pass through shared memory to tensor memory; up's epilogue has a
// thread for each row, so its groups of 32 results and their scale stay within a
// thread.
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "experts.cuh"

struct mk_experts {
  int hidden, experts, k, ffn;
  bool e4m3;
  int device;
  int* status;                   // waits that ran out, counted
  unsigned long long limit;      // of every device wait, ns
  int drop;
  // What each stream's mk_experts_sync has reported (none: 0).  The count itself is
  // never cleared: another stream has yet to hear of it.
  std::mutex lock;
  std::vector<std::pair<cudaStream_t, int>> told;
};

namespace mk {
namespace {

// Warps: 0 boxes of tensor maps, 1 matrix instructions, 2 tensor memory, 3 the
// list of tiles, 4-7 results, then four for gathered rows (up) and four for scales
// (8 bits).
//
// AM: rows of a tile in shared memory.  The instructions take 128; what lies
// behind a tile's rows (an older stage, weights) is multiplied too, into rows
// that nobody reads.  NT: columns of a tile at most, G: what their number is a
// multiple of.
template <bool E4M3, bool UP, int AM, int NT>
struct Cfg {
  static constexpr bool MN = !E4M3 && !UP;                    // weights lie along the columns
  static constexpr int NGW = UP ? 4 : 0, NSW = E4M3 ? 4 : 0;   // warps that gather rows, scales
  static constexpr int THREADS = (8 + NGW + NSW) * 32;
  static constexpr int G = MN || (E4M3 && UP) ? 64 : 16;      // a swizzled row of columns; 32 results that share a scale
  static constexpr int KE = E4M3 ? 128 : 64;                  // elements of a stage
  static constexpr int A_BYTES = AM * 128, B_BYTES = NT * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int BOX = AM < 64 ? 16 : 64;               // rows of a box of rows that lie side by side
  static constexpr int SF_B = (NT + 127) / 128, SF = E4M3 ? 512 * (1 + SF_B) : 0;
  // Results leave by rows of RB bytes that are put together in shared memory:
  // whole lines instead of a sector of each of 32 rows.
  static constexpr int RB = !E4M3 ? 128 : UP ? 96 : 64, PITCH = RB + 16, OUT = AM * PITCH;
  static constexpr int STEP = UP ? 64 : RB / 2;               // columns at a time
  static constexpr int FIT = (SMEM_MOST - CTL - 1024 - OUT) / (STAGE + SF), NST = FIT < MAX_STAGES ? FIT : MAX_STAGES;
  static constexpr int OFF_SF = NST * STAGE, OFF_OUT = OFF_SF + NST * SF, OFF_CTL = OFF_OUT + OUT, SMEM = OFF_CTL + CTL + 1024;
  static constexpr int T_SF = 2 * NT, T_COLS = 512;           // tensor memory: two accumulators, each stage's scales
  static constexpr int ARRIVALS = 1 + NGW * 32 + NSW;   // the boxes' issue, rows by thread, scales by warp
  static_assert(T_SF + (E4M3 ? NST * 16 : 0) <= T_COLS, "tensor memory");
  static_assert(SMEM <= SMEM_MOST, "shared memory");
  static_assert(NT % 64 == 0 && AM % 32 == 0 && STAGE >= 128 * 128, "a tile");
};

// What tiles of this width cost: their rounds over the blocks, times the columns
// of one and what it takes beside them.  (At most 2^18 + 256 tiles of rows and
// 2^12 of columns: 32 bits.)
__host__ __device__ __forceinline__ unsigned cost_of(unsigned row_tiles, unsigned n, unsigned width, unsigned blocks, unsigned extra) {
  const unsigned rounds = (row_tiles * ((n + width - 1) / width) + blocks - 1) / blocks;
  return (rounds < 1u << 22 ? rounds : 1u << 22) * (width + extra);
}

// The width of all tiles: rounds of tiles that the blocks take, times what one
// takes.
template <int NT, int G>
__device__ __forceinline__ void set_width(const Args& a, Ctl* ctl) {
  const int lane = threadIdx.x % 32, width = G * (lane + 1);
  const unsigned cost = width <= NT ? cost_of(ctl->tile0[a.experts], a.n, width, gridDim.x, a.extra) : 0xffffffffu;
  const unsigned best = __reduce_min_sync(FULL, cost);
  const int who = __reduce_max_sync(FULL, cost == best ? lane : 0);
  if (lane == who) {
    ctl->width = width;
    ctl->columns = (a.n + width - 1) / width;
  }
}

// A block's tiles are t, t + blocks, ...: neighbours share an expert's weights
// in L2.  One warp plans 32 at a time (a search and divisions, which took the
// issuing thread 500 cycles a tile) and the others read them.  (Sharing the last
// tiles out by columns cost more than it gave: a tile takes its steps of K
// however narrow it is.)
template <int AM, int G>
__device__ __forceinline__ void plan_tiles(const Args& a, Ctl* ctl) {
  const int lane = threadIdx.x % 32, columns = ctl->columns, width = ctl->width, tiles = ctl->tile0[a.experts] * columns;
  for (int c = 0;; ++c) {
    if (!wait(&ctl->list_free[c & 1], (c >> 1 & 1) ^ 1, ctl, a.status)) return;
    const int t = (c * 32 + lane) * (int)gridDim.x + (int)blockIdx.x;
    int4 v = make_int4(0, 0, 0, 0);
    if (t < tiles) {
      const int g = t / columns; // an expert's tiles are side by side, those of its columns in turn
      int lo = 0, hi = a.experts - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (ctl->tile0[mid] <= g) lo = mid;
        else hi = mid - 1;
      }
      const int mt = ctl->tile0[lo + 1] - ctl->tile0[lo], in = t - ctl->tile0[lo] * columns;
      const int n = in / mt, row0 = ctl->row0[lo] + (in - n * mt) * AM;
      v = make_int4(lo | min(AM, ctl->row0[lo + 1] - row0) << 16, row0, n * width, min(width, (a.n - n * width + G - 1) / G * G));
    }
    ctl->list[c & 1][lane] = v;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->list_full[c & 1]);
    if (!__all_sync(FULL, t < tiles)) return;    // an entry without rows is behind the last one
  }
}
// Columns of a row as results, 16 bytes at a time: up's (gate and up columns in
// turn; 8 bits: and the scale of 32 of them), or down's times the gate.
__device__ __forceinline__ void put16(uint8_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
// up: 64 columns, 32 results.
template <bool E4M3>
__device__ __forceinline__ void put_up(uint32_t acc, uint8_t* to, uint8_t* scale) {
  float v[32];
  uint32_t r[32];
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    tmem_ld32(acc + c, r);
    tmem_wait_ld();
    landed<32>(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[c / 2 + i] = swiglu(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
  }
  if constexpr (E4M3) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
    const int k = scale_exp(m);
    const Factors s = factors(k);
#pragma unroll
    for (int i = 0; i < 32; i += 16)
      *reinterpret_cast<uint4*>(to + i) =
          make_uint4(codes4(v[i], v[i + 1], v[i + 2], v[i + 3], s.f, s.g), codes4(v[i + 4], v[i + 5], v[i + 6], v[i + 7], s.f, s.g),
                     codes4(v[i + 8], v[i + 9], v[i + 10], v[i + 11], s.f, s.g),
                     codes4(v[i + 12], v[i + 13], v[i + 14], v[i + 15], s.f, s.g));
    if (scale) *scale = (uint8_t)(k + 127);
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 8) put16(to + 2 * i, v + i);
  }
}
// down: N columns that are on their way to registers.
template <int N>
__device__ __forceinline__ void load_down(uint32_t acc, uint32_t* r) {
#pragma unroll
  for (int c = 0; c < N; c += 32) tmem_ld32(acc + c, r + c);
}
template <int N>
__device__ __forceinline__ void put_down(const uint32_t* r, uint8_t* to, float gate) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[i + j]) * gate;
    put16(to + 2 * i, v);
  }
}

template <bool E4M3, bool UP, int AM, int NT>
__global__ void __launch_bounds__(Cfg<E4M3, UP, AM, NT>::THREADS, 1)
    k_experts(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_d) {
  using C = Cfg<E4M3, UP, AM, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int* status = a.status;
  if (tid == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&ctl->full[i], C::ARRIVALS);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->list_full[i], 1);
      mbar_init(&ctl->list_free[i], 6 + C::NGW + C::NSW);   // the reading warps
    }
    mbar_init(&ctl->drain, 1);
    ctl->fail = 0;
    ctl->limit = a.limit;
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<C::T_COLS>(&ctl->tmem);
  tc_before();
  __syncthreads();
  tc_after();
  await_stream();
  allow_next();
  const uint32_t tmem = ctl->tmem;
  const int kbs = (a.k + C::KE - 1) / C::KE;
  Reader list;
  Tile tile;

  if (warp == 0) {                               // ---- boxes: weights, rows that lie side by side; by one thread
    if (elect_one()) {
      const int stop = a.drop == DROP_COPIES ? 3 : 0x7fffffff;
      int s = 0, sent = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && list.next<false>(ctl, status, tile)) {
        const int boxes = UP ? 0 : (tile.rows + C::BOX - 1) / C::BOX;
        const uint32_t bytes = (boxes * C::BOX + tile.width) * 128;
        const int steps = min(kbs, stop - sent);
        for (int kb = 0; kb < steps; ++kb) {
          uint64_t *full = &ctl->full[s], *empty = &ctl->empty[s];
          if (!(ok = wait_one(empty, ph ^ 1, ctl, status))) break;
          uint8_t *dst = smem + s * C::STAGE, *w = dst + C::A_BYTES;
          mbar_arrive_tx(full, bytes);
          if constexpr (C::MN) {
            for (int n = 0; n < tile.width; n += 64) tma_3d(w + n * 128, &map_c, tile.n0 + n, kb * C::KE, tile.e, full);
          } else if (tile.width == a.box) {
            tma_3d(w, &map_b, kb * C::KE, tile.n0, tile.e, full);
          } else {
            int n = 0;
            for (; n + 64 <= tile.width; n += 64) tma_3d(w + n * 128, &map_c, kb * C::KE, tile.n0 + n, tile.e, full);
            if constexpr (C::G < 64)
              for (; n < tile.width; n += 16) tma_3d(w + n * 128, &map_d, kb * C::KE, tile.n0 + n, tile.e, full);
          }
          for (int i = 0; i < boxes; ++i) tma_2d(dst + i * C::BOX * 128, &map_a, kb * C::KE, tile.row0 + i * C::BOX, full);
          ++sent;
          if (++s == C::NST) { s = 0; ph ^= 1; }
        }
        ok = ok && steps == kbs;
      }
      if (!ok) {                                 // given up: what is in flight still lands before the block ends
        const unsigned long long since = now_ns();
        for (int u = max(0, sent - C::NST); u < sent; ++u)
          while (!mbar_try(&ctl->full[u % C::NST], u / C::NST & 1) && now_ns() - since < WAIT_NS) {}
      }
    }
    __syncwarp();
  } else if (warp == 1) {                        // ---- matrix instructions, by one thread
    if (elect_one()) {
      const uint64_t a_desc = umma_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t b_desc = umma_desc(smem_u32(smem + C::A_BYTES), C::MN ? 8192 : 16, 1024, 2);
      const uint64_t s_desc = umma_desc(smem_u32(smem + C::OFF_SF), 16, 128, 0);
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (; ok && list.next<false>(ctl, status, tile); ++i) {
        const uint32_t acc = tmem + (i & 1) * NT;
        const uint32_t columns = (uint32_t)(tile.width >> 3) << 17;
        if (!(ok = wait_one(&ctl->acc_empty[i & 1], (i >> 1 & 1) ^ 1, ctl, status))) break;
        tc_after();
        for (int kb = 0; kb < kbs; ++kb) {
          if (!(ok = wait_one(&ctl->full[s], ph, ctl, status))) break;
          if (UP) fence_async();                 // the threads' copies, before the matrix instructions read them
          tc_after();
          const uint64_t ad = a_desc + (uint32_t)(s * C::STAGE >> 4), bd = b_desc + (uint32_t)(s * C::STAGE >> 4);
          if constexpr (E4M3) {
            const uint64_t sd = s_desc + (uint32_t)(s * C::SF >> 4);
            const uint32_t sf = tmem + C::T_SF + s * 16;
#pragma unroll
            for (int j = 0; j < 1 + C::SF_B; ++j) tmem_scales(sf + 4 * j, sd + (512 * j >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_mx8(acc, ad + 2 * k, bd + 2 * k, umma_idesc_mx8(128, 0, k) | columns, sf, sf + 4, kb > 0 || k > 0);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_ss(acc, ad + 2 * k, bd + (C::MN ? 2048 * k >> 4 : 2 * k), umma_idesc(128, 0, C::MN) | columns, kb > 0 || k > 0);
          }
          umma_commit(&ctl->empty[s]);
          if (kb == kbs - 1) umma_commit(&ctl->acc_full[i & 1]);
          if (++s == C::NST) { s = 0; ph ^= 1; }
        }
      }
      // Products and their arrivals are done before the block's memory is given
      // back, after a wait that gave up too.
      umma_commit(&ctl->drain);
      const unsigned long long since = now_ns();
      while (!mbar_try(&ctl->drain, 0) && now_ns() - since < WAIT_NS) {}
    }
    __syncwarp();
  } else if (warp == 3) {                        // ---- the list of tiles
    set_tables<AM>(a, ctl);
    __syncwarp();
    set_width<NT, C::G>(a, ctl);
    __syncwarp();
    if (a.drop != DROP_LIST) plan_tiles<AM, C::G>(a, ctl);
  } else if (warp >= 4 && warp < 8) {            // ---- results: one thread a row
    const int row = (warp - 4) * 32 + lane;
    constexpr int EL = E4M3 && UP ? 1 : 2, LANES = C::RB > 64 ? 8 : 4;   // bytes of a result; lanes that write a row's piece
    const size_t pitch = (size_t)(UP ? a.n / 2 : a.n) * EL;
    uint8_t* const mine = smem + C::OFF_OUT + row * C::PITCH;
    // The row's place in the output, -1 for none, and its gate: those of the next
    // tile are read while this one is worked on (two dependent loads).
    auto place_of = [&](const Tile& t) {
      if (row >= t.rows) return -1;
      const int at = t.row0 + row;
      return UP ? at : a.order[at];
    };
    auto gate_of = [&](int& at) {
      if (UP) return 1.f;
      if ((unsigned)at >= (unsigned)a.pairs) at = -1;
      return at >= 0 && a.gates ? a.gates[at] : 1.f;
    };
    bool more = list.next<true>(ctl, status, tile);
    int next_at = more ? place_of(tile) : -1;
    float next_gate = gate_of(next_at);
    for (int i = 0; more; ++i) {
      const int rows = min(32, tile.rows - (warp - 4) * 32);   // of this warp
      const int n0 = tile.n0, width = min(tile.width, a.n - tile.n0), at = next_at;
      const float gate = next_gate;
      if ((more = list.next<true>(ctl, status, tile))) next_at = place_of(tile);
      if (!wait(&ctl->acc_full[i & 1], i >> 1 & 1, ctl, status)) break;
      tc_after();
      const uint32_t acc = tmem + (i & 1) * NT + ((uint32_t)((warp - 4) * 32) << 16);
      constexpr int EACH = 32 / LANES;           // rows that the warp writes at a time
      int place[LANES];
#pragma unroll
      for (int j = 0; j < LANES; ++j) place[j] = __shfl_sync(FULL, at, j * EACH + lane / LANES);
      const int piece = lane % LANES * 16;
      uint8_t* out = a.out + (size_t)(UP ? n0 / 2 : n0) * EL + piece;
      const uint8_t* from = smem + C::OFF_OUT + ((warp - 4) * 32 + lane / LANES) * C::PITCH + piece;
      uint32_t r[UP ? 1 : C::STEP];
      if (!UP && rows > 0) load_down<C::STEP>(acc, r);
      int fill = 0;                              // bytes of the rows' pieces
#pragma unroll 1
      for (int c = 0; c < width; c += C::STEP) {
        const bool last = c + C::STEP >= width;
        if (UP && rows > 0)
          put_up<E4M3>(acc + c, mine + fill, E4M3 && at >= 0 ? a.out_scales + (size_t)at * (a.n / 2 / GROUP) + (n0 + c) / 64 : nullptr);
        if constexpr (!UP) {
          tmem_wait_ld();
          landed<C::STEP>(r);
        }
        if (last) {                              // all of it read: the accumulator may be summed into again
          tc_before();
          __syncwarp();
          if (lane == 0 && a.drop != DROP_ACC) mbar_arrive(&ctl->acc_empty[i & 1]);
        }
        if (!UP && rows > 0) {
          put_down<C::STEP>(r, mine, gate);
          if (!last) load_down<C::STEP>(acc + c + C::STEP, r);
        }
        if (c == 0) next_gate = gate_of(next_at);
        fill += (UP ? min(C::STEP, width - c) / 2 : min(C::STEP, width - c)) * EL;
        if (fill < C::RB && !last) continue;
        __syncwarp();
        if (rows > 0) {
          uint4 v[LANES];
#pragma unroll
          for (int j = 0; j < LANES; ++j) v[j] = *reinterpret_cast<const uint4*>(from + j * EACH * C::PITCH);
#pragma unroll
          for (int j = 0; j < LANES; ++j)
            if (place[j] >= 0 && piece < fill) *reinterpret_cast<uint4*>(out + (size_t)place[j] * pitch) = v[j];
        }
        __syncwarp();
        out += fill;
        fill = 0;
      }
    }
    if (!UP && list.known) {                     // pairs without an expert
      for (int x = ctl->row0[a.experts] + blockIdx.x; x < a.pairs; x += gridDim.x) {
        const int p = a.order[x];
        if (p >= 0 && p < a.pairs)
          for (int n = row * 8; n < a.n; n += 1024)
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (size_t)p * a.n + n) = make_uint4(0, 0, 0, 0);
      }
    }
  } else if (UP && warp >= 8 && warp < 8 + C::NGW) {   // ---- gathered rows
    constexpr int RW = AM / (UP ? C::NGW : 1), NI = RW / 4;   // the warp's rows of a stage, its copies of 4 rows
    const int w = warp - 8, piece = lane % 8;
    const size_t pitch = (size_t)a.k * (E4M3 ? 1 : 2);
    // rows 4 i + lane / 8 of the warp's: a row's 8 pieces by neighbours, swizzled as the tensor maps do
    uint32_t to[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = w * RW + 4 * i + lane / 8;
      to[i] = smem_u32(smem) + row * 128 + (piece ^ (row & 7)) * 16;
    }
    int from[(RW + 31) / 32];                    // the lane's rows of x, of the tile to come
    auto rows_of = [&](const Tile& t) {
#pragma unroll
      for (int j = 0; j < (RW + 31) / 32; ++j) {
        const int r = j * 32 + lane;
        from[j] = r < RW && w * RW + r < t.rows ? token_of(a, t.row0 + w * RW + r) : a.rows;
      }
    };
    int s = 0;
    uint32_t ph = 0;
    bool ok = true, more = list.next<true>(ctl, status, tile);
    if (more) rows_of(tile);
    while (ok && more) {
      const int mine = min(RW, max(0, tile.rows - w * RW));
      const uint8_t* src[NI];
      uint32_t some = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = __shfl_sync(FULL, from[i / 8], 4 * i % 32 + lane / 8);
        some |= (uint32_t)(r < a.rows) << i;
        src[i] = a.x + (r < a.rows ? r * pitch : 0) + piece * 16;
      }
      if ((more = list.next<true>(ctl, status, tile))) rows_of(tile);
      for (int kb = 0; kb < kbs; ++kb) {
        if (!(ok = wait(&ctl->empty[s], ph ^ 1, ctl, status))) break;
        const bool in = kb * 128 + piece * 16 < (int)pitch;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (4 * i < mine)
            copy16(to[i & 1] + s * C::STAGE + (i >> 1) * 1024, src[i] + (in ? kb * 128 : 0), in && (some >> i & 1));
        mbar_arrive_copies(&ctl->full[s]);
        if (++s == C::NST) { s = 0; ph ^= 1; }
      }
    }
    copies_done();                               // nothing lands after the block's end
  } else if (E4M3 && warp >= 8 + C::NGW) {       // ---- scales: a warp has a quarter of every stage's rows
    // (Every warp passes every stage: a phase is told from its neighbours by its
    // parity alone, so nobody may be two of them away from the one it waits for.)
    constexpr int RW = AM / 4, SF_B = C::SF_B;
    const int w = warp - 8 - C::NGW, groups = a.k / GROUP, r = w * RW + lane, c = w * 32 + lane;
    // row r's scales of a stage are the word at r % 32, r / 32 of its 128 rows
    uint8_t *const sf_a = smem + C::OFF_SF + r % 32 * 16 + r / 32 * 4, *const sf_b = smem + C::OFF_SF + 512 + lane * 16 + w * 4;
    struct Four {                                // the lane's rows' scales of four stages
      uint4 a, b[SF_B ? SF_B : 1];
    };
    const uint8_t *pa = nullptr, *pb = nullptr;  // the lane's rows of the tile that is being fetched
    int kb = kbs;
    auto fetch = [&](Four& f) {                  // the next four stages, of the next tile where need be
      if (kb >= kbs) {
        if (!list.next<true>(ctl, status, tile)) return false;
        const int limit = UP ? a.rows : a.pairs;
        const int from = lane >= RW || r >= tile.rows ? limit : UP ? token_of(a, tile.row0 + r) : tile.row0 + r;
        pa = from < limit ? a.a_scales + (size_t)from * groups : nullptr;
        pb = a.b_scales + ((size_t)tile.e * a.n + tile.n0 + c) * groups;
        kb = 0;
      }
      const uint4 none = make_uint4(0, 0, 0, 0);
      f.a = pa ? scales16(pa, groups, kb, a.a_wide) : none;
#pragma unroll
      for (int j = 0; j < SF_B; ++j) {
        const int n = j * 128 + c;
        f.b[j] = n < tile.width && tile.n0 + n < a.n ? scales16(pb + (size_t)(j * 128) * groups, groups, kb, a.b_wide) : none;
      }
      kb += 4;
      return true;
    };
    Four now, next, after;                       // two are on their way while one is stored
    bool has = fetch(now), has_next = has && fetch(next), ok = true;
    int s = 0, at = 0;
    uint32_t ph = 0;
    while (has && ok) {
      const bool has_after = has_next && fetch(after);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at + i >= kbs || !ok || !(ok = wait(&ctl->empty[s], ph ^ 1, ctl, status))) break;
        if (lane < RW) *reinterpret_cast<uint32_t*>(sf_a + s * C::SF) = word(now.a, i);
#pragma unroll
        for (int j = 0; j < SF_B; ++j)
          if (NT % 128 == 0 || j * 128 + w * 32 < NT) *reinterpret_cast<uint32_t*>(sf_b + s * C::SF + j * 512) = word(now.b[j], i);
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[s]);
        if (++s == C::NST) { s = 0; ph ^= 1; }
      }
      at = at + 4 < kbs ? at + 4 : 0;
      now = next;
      next = after;
      has = has_next;
      has_next = has_after;
    }
  }

  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 2) tmem_free<C::T_COLS>(tmem);
}

template <bool E4M3, bool UP, int AM, int NT>
cudaError_t launch(Args a, const void* rows, const void* w, int sms, cudaStream_t st) {
  using C = Cfg<E4M3, UP, AM, NT>;
  a.extra = AM;                  // the rows' bytes (none: down of 37 rows in 8 bits 136 us instead of 31; three times: the same)
  a.a_wide = scales_wide(a.a_scales, a.k / GROUP);
  a.b_wide = scales_wide(a.b_scales, a.k / GROUP);
  const unsigned some = a.pairs < a.experts ? a.pairs : a.experts;   // experts with rows, if all the pairs' differ
  const long long most = ((long long)a.pairs / AM + some) * ((a.n + C::G - 1) / C::G);
  const unsigned blocks = (unsigned)(most < sms ? most : sms);
  // The width that the blocks will choose if so: one box a stage then.
  a.box = NT;
  for (int w = NT; w > 0 && a.pairs <= a.experts; w -= C::G)
    if (cost_of(some, a.n, w, blocks, a.extra) < cost_of(some, a.n, a.box, blocks, a.extra)) a.box = w;
  const cuuint64_t dim_a[2] = {(cuuint64_t)a.k, (cuuint64_t)a.pairs};
  const cuuint32_t box_a[2] = {C::KE, C::BOX};
  const cuuint64_t dim_b[3] = {(cuuint64_t)(C::MN ? a.n : a.k), (cuuint64_t)(C::MN ? a.k : a.n), (cuuint64_t)a.experts};
  const cuuint32_t box_b[3] = {C::KE, (cuuint32_t)a.box, 1}, box_c[3] = {C::KE, 64, 1}, box_d[3] = {C::KE, 16, 1};
  CUtensorMap map_a = {}, map_b = {}, map_c, map_d = {};
  cudaError_t e = UP ? cudaSuccess : tensor_map(&map_a, E4M3, rows, 2, dim_a, box_a);
  if (e == cudaSuccess && !C::MN) e = tensor_map(&map_b, E4M3, w, 3, dim_b, box_b);
  if (e == cudaSuccess) e = tensor_map(&map_c, E4M3, w, 3, dim_b, box_c);
  if (e == cudaSuccess && C::G < 64) e = tensor_map(&map_d, E4M3, w, 3, dim_b, box_d);
  if (e == cudaSuccess) e = allow((const void*)k_experts<E4M3, UP, AM, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_kernel(k_experts<E4M3, UP, AM, NT>, blocks, C::THREADS, C::SMEM, 1, st, a,
                       map_a, map_b, map_c, map_d);
}

template <bool E4M3, bool UP>
cudaError_t launch(const Args& a, const void* rows, const void* w, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  // bf16 with 128 rows an expert: tiles of two SMs (8143 rows of the full model, in
  // short bursts: up 284 us, 311 with one; down 155 and 175; 2500 rows: 144 and 150,
  // 82 and 85; 1200, 75 an expert: 135 and 130), where they are enough for four rounds of
  // the SMs and little of their 256 columns is lost (hidden 1056: 28.6 us with
  // one, 32.6).
  const long long cols = (a.n + 255) / 256;
  if (!E4M3 && a.pairs >= 128 * a.experts && (a.pairs / 256 + a.experts / 2) * cols >= 2 * sms && 10 * a.n >= 9 * 256 * cols)
    return launch_two(UP, a, rows, w, sms, st);
  // Few rows an expert: tiles of 32 rows leave the shared memory to the weights
  // on their way; a token or a few take narrow tiles anyway and more steps of
  // them (one token of up 13.1 us, 13.5 of the wider), others fewer rounds (64
  // rows of 37 experts of 352 in 8 bits 10.5 us, 14.2 of the narrower).
  if (a.pairs <= 32) return launch<E4M3, UP, 32, 128>(a, rows, w, sms, st);
  if (a.pairs <= 16 * a.experts) return launch<E4M3, UP, 32, 192>(a, rows, w, sms, st);
  return launch<E4M3, UP, 128, E4M3 ? 192 : 256>(a, rows, w, sms, st);
}

int check_device(const mk_experts* m) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda("mk_experts: current device", e);
  return dev == m->device ? MK_OK : fail(MK_ERR_INVALID, "mk_experts: the object belongs to another device than the current one");
}

}  // namespace
}  // namespace mk

extern "C" {

int mk_experts_create(const mk_model_dims* dims, int rows_type, mk_experts** out) {
  using namespace mk;
  if (!out) return fail(MK_ERR_INVALID, "mk_experts_create: out is NULL");
  *out = nullptr;
  if (!dims) return fail(MK_ERR_INVALID, "mk_experts_create: dims is NULL");
  if (rows_type != MK_ROWS_BF16 && rows_type != MK_ROWS_E4M3) return fail(MK_ERR_INVALID, "mk_experts_create: rows_type");
  const bool e4m3 = rows_type == MK_ROWS_E4M3;
  const int h = dims->hidden, f = dims->expert_ffn, of = e4m3 ? GROUP : 8;
  if (h < 1 || f < 1 || dims->n_experts < 1 || dims->top_k < 1 || dims->top_k > dims->n_experts)
    return fail(MK_ERR_INVALID, "mk_experts_create: hidden, expert_ffn, n_experts or top_k");
  if (h % of || f % of)
    return fail(MK_ERR_UNSUPPORTED, "mk_experts_create: hidden and expert_ffn must be multiples of 8 (8 bits: of 32)");
  if (dims->n_experts > MAX_EXPERTS || dims->top_k > 8 || h > 32768 || f > 32768)
    return fail(MK_ERR_UNSUPPORTED, "mk_experts_create: at most 256 experts, 8 of them a row, hidden and expert_ffn at most 32768");
  mk_experts* m = new (std::nothrow) mk_experts();
  if (!m) return fail(MK_ERR_CAPACITY, "out of host memory");
  m->hidden = h; m->ffn = f; m->experts = dims->n_experts; m->k = dims->top_k; m->e4m3 = e4m3; m->limit = WAIT_NS;
  cudaError_t e = cudaGetDevice(&m->device);
  if (e == cudaSuccess) e = cudaMalloc((void**)&m->status, sizeof(int));
  if (e == cudaSuccess) {
    e = cudaMemset(m->status, 0, sizeof(int));
    if (e == cudaSuccess) e = cudaStreamSynchronize(0);
    if (e != cudaSuccess) cudaFree(m->status);
  }
  if (e != cudaSuccess) {
    delete m;
    return fail_cuda("mk_experts_create", e);
  }
  *out = m;
  return MK_OK;
}

int mk_experts_set_debug(mk_experts* m, int timeout_us, int drop) {
  using namespace mk;
  if (!m) return fail(MK_ERR_INVALID, "mk_experts_set_debug: experts is NULL");
  if (timeout_us < 0 || timeout_us > 2000000 || drop < 0 || drop > DROP_ACC)
    return fail(MK_ERR_INVALID, "mk_experts_set_debug: timeout_us (at most 2000000) or drop");
  m->limit = timeout_us ? timeout_us * 1000ull : WAIT_NS;
  m->drop = drop;
  return MK_OK;
}

int mk_experts_up(mk_experts* m, int rows, const void* x, const uint8_t* x_scales, const void* w, const uint8_t* w_scales,
                  const int* first, const int* order, void* h, uint8_t* h_scales, mk_stream stream) {
  using namespace mk;
  if (!m) return fail(MK_ERR_INVALID, "mk_experts_up: experts is NULL");
  if (rows < 0) return fail(MK_ERR_INVALID, "mk_experts_up: rows");
  if (rows > (1 << 25) / m->k) return fail(MK_ERR_UNSUPPORTED, "mk_experts_up: more than 2^25 pairs");
  if (rows == 0) return check_device(m);
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(h, 16) || !aligned(first, 4) || !aligned(order, 4) ||
      (m->e4m3 && (!x_scales || !w_scales || !h_scales)))
    return fail(MK_ERR_INVALID, "mk_experts_up: a buffer is NULL or not aligned (rows and weights 16 bytes)");
  const size_t el = m->e4m3 ? 1 : 2, t = rows, p = t * m->k, wide = m->hidden, f = m->ffn, e = m->experts;
  const bool s8 = m->e4m3;
  const Span s[8] = {{h, p * f * el},
                     {s8 ? h_scales : nullptr, p * f / GROUP},
                     {x, t * wide * el},
                     {s8 ? x_scales : nullptr, t * wide / GROUP},
                     {w, e * 2 * f * wide * el},
                     {s8 ? w_scales : nullptr, e * 2 * f * wide / GROUP},
                     {first, 4 * (e + 1)},
                     {order, 4 * p}};
  if (clash(s, 2, 8)) return fail(MK_ERR_INVALID, "mk_experts_up: a result overlaps another buffer");
  const int rc = check_device(m);
  if (rc != MK_OK) return rc;
  Args a = {first, order, nullptr, (const uint8_t*)x, x_scales, w_scales, (uint8_t*)h, h_scales, m->status, (int)p, rows, m->k, m->experts,
            m->hidden, 2 * m->ffn};
  a.limit = m->limit;
  a.drop = m->drop;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t err = s8 ? launch<true, true>(a, x, w, st) : launch<false, true>(a, x, w, st);
  return err == cudaSuccess ? MK_OK : fail_cuda("mk_experts_up", err);
}

int mk_experts_down(mk_experts* m, int rows, const void* h, const uint8_t* h_scales, const void* w, const uint8_t* w_scales,
                    const int* first, const int* order, const float* gates, void* y, mk_stream stream) {
  using namespace mk;
  if (!m) return fail(MK_ERR_INVALID, "mk_experts_down: experts is NULL");
  if (rows < 0) return fail(MK_ERR_INVALID, "mk_experts_down: rows");
  if (rows > (1 << 25) / m->k) return fail(MK_ERR_UNSUPPORTED, "mk_experts_down: more than 2^25 pairs");
  if (rows == 0) return check_device(m);
  if (!aligned(h, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(first, 4) || !aligned(order, 4) ||
      (gates && !aligned(gates, 4)) || (m->e4m3 && (!h_scales || !w_scales)))
    return fail(MK_ERR_INVALID, "mk_experts_down: a buffer is NULL or not aligned (rows and weights 16 bytes)");
  const size_t el = m->e4m3 ? 1 : 2, p = (size_t)rows * m->k, wide = m->hidden, f = m->ffn, e = m->experts;
  const bool s8 = m->e4m3;
  const Span s[8] = {{y, p * wide * 2},
                     {h, p * f * el},
                     {s8 ? h_scales : nullptr, p * f / GROUP},
                     {w, e * f * wide * el},
                     {s8 ? w_scales : nullptr, e * f * wide / GROUP},
                     {first, 4 * (e + 1)},
                     {order, 4 * p},
                     {gates, 4 * p}};
  if (clash(s, 1, 8)) return fail(MK_ERR_INVALID, "mk_experts_down: y overlaps another buffer");
  const int rc = check_device(m);
  if (rc != MK_OK) return rc;
  Args a = {first, order, gates, nullptr, h_scales, w_scales, (uint8_t*)y, nullptr, m->status, (int)p, rows, m->k, m->experts,
            m->ffn, m->hidden};
  a.limit = m->limit;
  a.drop = m->drop;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t err = s8 ? launch<true, false>(a, h, w, st) : launch<false, false>(a, h, w, st);
  return err == cudaSuccess ? MK_OK : fail_cuda("mk_experts_down", err);
}

int mk_experts_sync(mk_experts* m, mk_stream stream) {
  using namespace mk;
  if (!m) return fail(MK_ERR_INVALID, "mk_experts_sync: experts is NULL");
  const int rc = check_device(m);
  if (rc != MK_OK) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  int n = 0;
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&n, m->status, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return fail_cuda("mk_experts_sync", e);
  if (n == 0) return MK_OK;
  try {
    std::lock_guard<std::mutex> hold(m->lock);
    for (auto& t : m->told)
      if (t.first == st) {
        const bool heard = t.second == n;
        t.second = n;
        return heard ? MK_OK : MK_ERR_DEP_TIMEOUT;
      }
    m->told.emplace_back(st, n);
  } catch (...) {
  }                              // (no memory for it: this stream hears of it again)
  return MK_ERR_DEP_TIMEOUT;
}

void mk_experts_destroy(mk_experts* m) {
  if (!m) return;
  mk::BesideCaptures relaxed;
  cudaFree(m->status);
  delete m;
}

}  // extern "C"
