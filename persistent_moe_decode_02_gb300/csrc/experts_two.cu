// The experts' products in bf16 with many rows an expert: tiles of two SMs.
//
// The roles are turned round here: the weights are A (256 rows of them, 128 in
// each block of a pair), the expert's rows are B, up to 256 of them, half in each
// block.  A tile of 128 rows by 256 columns in one SM takes 48 KB for each 128
// bytes of K, and its products wait for them (8143 rows of up: 416 ns a step,
// 118 GB/s an SM, as much as L2 gives it; the products need 270 at the rated
// clock, 328 at the rate that large library products reach); a pair's blocks take
// 32 KB each for the same products.  (A step of theirs takes some 335 ns on the
// average, though the mean tile has 212 of 256 tokens: why a narrower step is
// hardly shorter was not found.  Without the gather up is a tenth faster, without
// the results a sixteenth.)  And an expert's rows are cut into tiles
// of any multiple of 32 instead of 128: of 8143 tokens' 65144 pairs 3 in 100 rows
// are padding, not 13.
//
// What the pair costs: the even block issues for both, so the odd one's copies
// are told to it by a relay (its own barrier first, then the leader's), and
// results lie with a weight row a lane and a token a column, so they are turned
// in shared memory on their way out, by two groups of four warps.
//
// (In 8 bits, where the scales leave room for 224 rows a tile and each block has
// all their scales to fetch, the pair was no faster than one SM.)
#include "experts.cuh"

namespace mk {
namespace {

template <bool UP>
struct Two {
  static constexpr int NGW = UP ? 4 : 0;                      // warps that gather rows
  static constexpr int GROUPS = 2, W_LOAD = 4 + 4 * GROUPS;   // groups of four warps for results, then those
  static constexpr int THREADS = (W_LOAD + NGW) * 32;
  static constexpr int KE = 64, W = 256;                      // elements of a stage; tokens of a tile at most
  static constexpr int A_BYTES = 128 * 128, B_BYTES = W / 2 * 128, STAGE = A_BYTES + B_BYTES;
  // Results on their way out, a buffer for each group: tokens by units (up: 64 of
  // 64) or by columns (down: 32 of 128); down: places and gates of two tiles' tokens.
  static constexpr int TOKENS = UP ? 64 : 32, PITCH = UP ? 144 : 272, BUF = TOKENS * PITCH;
  static constexpr int EACH = BUF + (UP ? 0 : 2 * 256 * 8), OUT = GROUPS * EACH;
  static constexpr int FIT = (SMEM_MOST - CTL - 1024 - OUT) / STAGE, NST = FIT < MAX_STAGES ? FIT : MAX_STAGES;
  static constexpr int OFF_OUT = NST * STAGE, OFF_CTL = OFF_OUT + OUT, SMEM = OFF_CTL + CTL + 1024;
  static constexpr int T_COLS = 512;                          // tensor memory: two accumulators
  static constexpr int ARRIVALS = 1 + NGW * 32;               // of a block: the boxes' issue, rows by thread
  static_assert(2 * W <= T_COLS, "tensor memory");
  static_assert(SMEM <= SMEM_MOST, "shared memory");
};

// A group's four warps: together, and together with whether all are well.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool group_all(int group, bool ok) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.and.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(r)
               : "r"(1 + group), "r"((uint32_t)ok)
               : "memory");
  return r != 0;
}

// A pair's tiles: 32 at a time, the same list in both blocks.  An expert's rows
// are cut into tiles of about the same size.
template <int W>
__device__ __forceinline__ void plan_two(const Args& a, Ctl* ctl) {
  const int lane = threadIdx.x % 32, columns = (a.n + 255) / 256, tiles = ctl->tile0[a.experts] * columns;
  for (int c = 0;; ++c) {
    if (!wait(&ctl->list_free[c & 1], (c >> 1 & 1) ^ 1, ctl, a.status)) return;
    const int t = (c * 32 + lane) * (int)(gridDim.x / 2) + (int)(blockIdx.x / 2);
    int4 v = make_int4(0, 0, 0, 0);
    if (t < tiles) {
      const int g = t / columns;
      int lo = 0, hi = a.experts - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (ctl->tile0[mid] <= g) lo = mid;
        else hi = mid - 1;
      }
      const int mt = ctl->tile0[lo + 1] - ctl->tile0[lo], in = t - ctl->tile0[lo] * columns, n = in / mt, m = in - n * mt;
      const int end = ctl->row0[lo + 1], each = ((end - ctl->row0[lo] + mt - 1) / mt + 31) / 32 * 32;   // at most W
      const int row0 = ctl->row0[lo] + m * each, rows = min(each, end - row0);   // at least 1
      v = make_int4(lo | rows << 16, row0, n * 256, (rows + 31) / 32 * 32);
    }
    ctl->list[c & 1][lane] = v;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->list_full[c & 1]);
    if (!__all_sync(FULL, t < tiles)) return;
  }
}

template <bool UP>
__global__ void __launch_bounds__(Two<UP>::THREADS, 1)
    k_two(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h) {
  using C = Two<UP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = (int)cluster_rank();
  int* status = a.status;
  if (tid == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&ctl->full[i], C::ARRIVALS + (rank == 0));   // the leader's: the other block's relay too
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], 8 * C::GROUPS);   // (the leader's is used: both blocks' warps)
      mbar_init(&ctl->list_full[i], 1);
      mbar_init(&ctl->list_free[i], 2 + 4 * C::GROUPS + C::NGW);
    }
    mbar_init(&ctl->drain, 1);
    ctl->fail = 0;
    ctl->limit = a.limit;
    fence_barrier_init();
  }
  if (warp == 2) tmem2_alloc<C::T_COLS>(&ctl->tmem);
  tc_before();
  __syncthreads();
  cluster_barrier();                             // both blocks' barriers are there
  tc_after();
  await_stream();
  allow_next();
  const uint32_t tmem = ctl->tmem;
  const int kbs = (a.k + C::KE - 1) / C::KE;
  Reader list;
  Tile tile;

  if (warp == 0) {                               // ---- boxes: weights, rows that lie side by side; by one thread
    if (elect_one()) {
      const int stop = a.drop == DROP_COPIES && rank == 1 ? 3 : 0x7fffffff;
      int s = 0, sent = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && list.next<false>(ctl, status, tile)) {
        const int half = tile.width / 2, mine = UP ? 0 : min(half, max(0, tile.rows - rank * half)), boxes = (mine + 15) / 16;
        const int n0 = tile.n0 + rank * 128, r0 = tile.row0 + rank * half;
        const uint32_t bytes = C::A_BYTES + boxes * 2048;
        const int steps = min(kbs, stop - sent);
        for (int kb = 0; kb < steps; ++kb) {
          uint64_t *full = &ctl->full[s], *empty = &ctl->empty[s];
          if (!(ok = wait_one(empty, ph ^ 1, ctl, status))) break;
          uint8_t* dst = smem + s * C::STAGE;
          mbar_arrive_tx(full, bytes);
          if constexpr (!UP) {
            tma_3d(dst, &map_w, n0, kb * C::KE, tile.e, full);
            tma_3d(dst + 8192, &map_w, n0 + 64, kb * C::KE, tile.e, full);
          } else {
            tma_3d(dst, &map_w, kb * C::KE, n0, tile.e, full);
          }
          for (int i = 0; i < boxes; ++i) tma_2d(dst + C::A_BYTES + i * 2048, &map_h, kb * C::KE, r0 + i * 16, full);
          ++sent;
          if (++s == C::NST) { s = 0; ph ^= 1; }
        }
        ok = ok && steps == kbs;
      }
      const unsigned long long since = now_ns();
      for (int u = max(0, sent - C::NST); u < sent; ++u) {
        if (ok) {                                // the leader's last arrivals here, before the block ends
          wait_one(&ctl->empty[u % C::NST], u / C::NST & 1, ctl, status);
        } else {                                 // given up: what is in flight still lands
          while (!mbar_try(&ctl->full[u % C::NST], u / C::NST & 1) && now_ns() - since < WAIT_NS) {}
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      if (rank == 0) {                           // ---- matrix instructions of both blocks, by one thread
        const uint64_t a_desc = umma_desc(smem_u32(smem), !UP ? 8192 : 16, 1024, 2);
        const uint64_t b_desc = umma_desc(smem_u32(smem + C::A_BYTES), 16, 1024, 2);
        int i = 0;
        for (; ok && list.next<false>(ctl, status, tile); ++i) {
          const uint32_t acc = tmem + (i & 1) * C::W, columns = (uint32_t)(tile.width >> 3) << 17;
          if (!(ok = wait_one(&ctl->acc_empty[i & 1], (i >> 1 & 1) ^ 1, ctl, status))) break;
          tc_after();
          for (int kb = 0; kb < kbs; ++kb) {
            if (!(ok = wait_one(&ctl->full[s], ph, ctl, status))) break;
            if (UP) fence_async();               // the threads' copies, before the matrix instructions read them
            tc_after();
            const uint64_t ad = a_desc + (uint32_t)(s * C::STAGE >> 4), bd = b_desc + (uint32_t)(s * C::STAGE >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma2_ss(acc, ad + (UP ? 2 * k : 2048 * k >> 4), bd + 2 * k, umma_idesc(256, 0, false) | (UP ? 0u : 1u << 15) | columns,
                       kb > 0 || k > 0);
            umma2_commit(&ctl->empty[s]);
            if (kb == kbs - 1) umma2_commit(&ctl->acc_full[i & 1]);
            if (++s == C::NST) { s = 0; ph ^= 1; }
          }
        }
        umma2_commit(&ctl->drain);
      } else {                                   // ---- the relay: what has landed here is told to the leader
        while (ok && list.next<false>(ctl, status, tile))
          for (int kb = 0; kb < kbs; ++kb) {
            if (!(ok = wait_one(&ctl->full[s], ph, ctl, status))) break;
            fence_async();
            mbar_arrive_at(&ctl->full[s], 0);
            if (++s == C::NST) { s = 0; ph ^= 1; }
          }
      }
      // Products and their arrivals, here and there, are done before the blocks'
      // memory is given back, after a wait that gave up too.
      const unsigned long long since = now_ns();
      while (!mbar_try(&ctl->drain, 0) && now_ns() - since < 2 * WAIT_NS) {}
    }
    __syncwarp();
  } else if (warp == 3) {                        // ---- the list of tiles
    set_tables<C::W>(a, ctl);
    __syncwarp();
    if (a.drop != DROP_LIST) plan_two<C::W>(a, ctl);
  } else if (warp >= 4 && warp < C::W_LOAD) {    // ---- results: a weight row a lane, a token a column
    const int group = (warp - 4) / 4, q = warp % 4, et = tid % 128;
    constexpr int TURN = C::GROUPS * C::TOKENS;
    const int width = UP ? a.n / 2 : a.n;        // of a row of results
    uint8_t* const out = smem + C::OFF_OUT + group * C::EACH;
    int* const places = reinterpret_cast<int*>(out + C::BUF);              // down: [2][256], and the gates behind them
    float* const gates = reinterpret_cast<float*>(places) + 512;
    int next_at[2];                              // down: the places of two tokens of the tile to come
    float next_gate[2] = {1.f, 1.f};
    auto places_of = [&](const Tile& t) {
#pragma unroll
      for (int j = 0; j < 2; ++j) next_at[j] = et + 128 * j < t.rows ? a.order[t.row0 + et + 128 * j] : -1;
    };
    auto gates_of = [&] {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if ((unsigned)next_at[j] >= (unsigned)a.pairs) next_at[j] = -1;
        next_gate[j] = next_at[j] >= 0 && a.gates ? a.gates[next_at[j]] : 1.f;
      }
    };
    // (A group's warps go on or stop together: they meet at barriers.)
    bool more = group_all(group, list.next<true>(ctl, status, tile));
    if (!UP && more) {
      places_of(tile);
      gates_of();
    }
    for (int i = 0; more; ++i) {
      const int rows = tile.rows, row0 = tile.row0, wide = tile.width, c0 = tile.n0 + rank * 128;
      int* const place = places + (i & 1) * 256;
      float* const gate = gates + (i & 1) * 256;
      if constexpr (!UP) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          place[et + 128 * j] = next_at[j];
          gate[et + 128 * j] = next_gate[j];
        }
      }
      more = group_all(group, list.next<true>(ctl, status, tile));
      if (!UP && more) places_of(tile);
      if (!group_all(group, wait(&ctl->acc_full[i & 1], i >> 1 & 1, ctl, status))) break;
      tc_after();
      const uint32_t acc = tmem + (i & 1) * C::W + ((uint32_t)(q * 32) << 16);
      uint32_t r[32];
      auto release = [&] {                       // all of it read: the accumulator may be summed into again
        tc_before();
        __syncwarp();
        if (lane == 0 && a.drop != DROP_ACC) mbar_arrive_at(&ctl->acc_empty[i & 1], 0);
      };
      if (group * C::TOKENS >= wide) release();
      else if (!UP) tmem_ld32(acc + group * C::TOKENS, r);
      if (!UP) gates_of();
#pragma unroll 1
      for (int c = group * C::TOKENS; c < wide; c += TURN) {
        const bool last = c + TURN >= wide;
        if constexpr (UP) {
          const int unit = q * 16 + lane / 2, odd = lane & 1;
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            if (c + h >= wide) break;
            tmem_ld32(acc + c + h, r);
            tmem_wait_ld();
            landed<32>(r);
#pragma unroll
            for (int t = 0; t < 16; ++t) {       // an even lane has a unit's gate and takes tokens 0-15, the odd one its up, 16-31
              const float other = __uint_as_float(__shfl_xor_sync(FULL, odd ? r[t] : r[t + 16], 1));
              const float v = odd ? swiglu(other, __uint_as_float(r[t + 16])) : swiglu(__uint_as_float(r[t]), other);
              const int token = h + t + 16 * odd;
              *reinterpret_cast<__nv_bfloat16*>(out + token * C::PITCH + unit * 2) = __float2bfloat16_rn(v);
            }
          }
          if (last) release();
        } else {
          tmem_wait_ld();
          landed<32>(r);
          if (last) release();
          uint8_t* const o = out + (q * 32 + lane) * 2;
#pragma unroll
          for (int t = 0; t < 32; t += 4) {
            const float4 g = *reinterpret_cast<const float4*>(gate + c + t);
            const uint32_t lo = pack_bf16(__uint_as_float(r[t]) * g.x, __uint_as_float(r[t + 1]) * g.y);
            const uint32_t hi = pack_bf16(__uint_as_float(r[t + 2]) * g.z, __uint_as_float(r[t + 3]) * g.w);
            *reinterpret_cast<uint16_t*>(o + t * C::PITCH) = (uint16_t)lo;
            *reinterpret_cast<uint16_t*>(o + (t + 1) * C::PITCH) = (uint16_t)(lo >> 16);
            *reinterpret_cast<uint16_t*>(o + (t + 2) * C::PITCH) = (uint16_t)hi;
            *reinterpret_cast<uint16_t*>(o + (t + 3) * C::PITCH) = (uint16_t)(hi >> 16);
          }
          if (!last) tmem_ld32(acc + c + TURN, r);
        }
        group_sync(group);
        constexpr int PIECES = UP ? 8 : 16, AT_ONCE = 128 / PIECES;   // 16-byte pieces of a token; tokens at a time
        const int piece = et % PIECES, col = (UP ? c0 / 2 : c0) + piece * 8;
        uint4 v[4];
        int at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = et / PIECES + j * AT_ONCE;
          v[j] = *reinterpret_cast<const uint4*>(out + t * C::PITCH + piece * 16);
          at[j] = UP ? row0 + c + t : place[min(c + t, 255)];
          if (c + t >= rows || col >= width) at[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (at[j] >= 0) *reinterpret_cast<uint4*>(a.out + ((size_t)at[j] * width + col) * 2) = v[j];
        group_sync(group);
      }
    }
    if (!UP && list.known) {                     // pairs without an expert
      for (int x = ctl->row0[a.experts] + blockIdx.x; x < a.pairs; x += gridDim.x) {
        const int p = a.order[x];
        if (p >= 0 && p < a.pairs)
          for (int n = (tid - 128) * 8; n < a.n; n += 1024 * C::GROUPS)
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (size_t)p * a.n + n) = make_uint4(0, 0, 0, 0);
      }
    }
  } else if (UP && warp >= C::W_LOAD && warp < C::W_LOAD + C::NGW) {   // ---- gathered rows: this block's half of the tokens
    const int w = warp - C::W_LOAD, piece = lane % 8;
    const size_t pitch = (size_t)a.k * 2;
    uint32_t to[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = w * 32 + 4 * i + lane / 8;
      to[i] = smem_u32(smem) + C::A_BYTES + row * 128 + (piece ^ (row & 7)) * 16;
    }
    auto mine_of = [&](const Tile& t) { return min(32, max(0, min(t.width / 2, t.rows - rank * (t.width / 2)) - w * 32)); };
    auto row_of = [&](const Tile& t) { return lane < mine_of(t) ? token_of(a, t.row0 + rank * (t.width / 2) + w * 32 + lane) : a.rows; };
    int s = 0;
    uint32_t ph = 0;
    bool ok = true, more = list.next<true>(ctl, status, tile);
    int from = more ? row_of(tile) : a.rows;
    while (ok && more) {
      const int mine = mine_of(tile);
      const uint8_t* src[8];
      uint32_t some = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = __shfl_sync(FULL, from, 4 * i + lane / 8);
        some |= (uint32_t)(r < a.rows) << i;
        src[i] = a.x + (r < a.rows ? r * pitch : 0) + piece * 16;
      }
      if ((more = list.next<true>(ctl, status, tile))) from = row_of(tile);
      for (int kb = 0; kb < kbs; ++kb) {
        if (!(ok = wait(&ctl->empty[s], ph ^ 1, ctl, status))) break;
        const bool in = kb * 128 + piece * 16 < (int)pitch;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (4 * i < mine)
            copy16(to[i & 1] + s * C::STAGE + (i >> 1) * 1024, src[i] + (in ? kb * 128 : 0), in && (some >> i & 1));
        mbar_arrive_copies(&ctl->full[s]);
        if (++s == C::NST) { s = 0; ph ^= 1; }
      }
    }
    copies_done();                               // nothing lands after the block's end
  }

  __syncwarp();
  tc_before();
  __syncthreads();
  cluster_barrier();                             // nobody reads the other block's memory any more
  tc_after();
  if (warp == 2) tmem2_free<C::T_COLS>(tmem);
  cluster_barrier();
}

template <bool UP>
cudaError_t launch_two(const ExpertArgs& a, const void* rows, const void* w, int sms, cudaStream_t st) {
  using C = Two<UP>;
  const cuuint64_t dim_w[3] = {(cuuint64_t)(UP ? a.k : a.n), (cuuint64_t)(UP ? a.n : a.k), (cuuint64_t)a.experts};
  const cuuint32_t box_w[3] = {C::KE, UP ? 128u : 64u, 1};
  const cuuint64_t dim_h[2] = {(cuuint64_t)a.k, (cuuint64_t)a.pairs};
  const cuuint32_t box_h[2] = {C::KE, 16};
  CUtensorMap map_w, map_h = {};
  cudaError_t e = tensor_map(&map_w, false, w, 3, dim_w, box_w);
  if (e == cudaSuccess && !UP) e = tensor_map(&map_h, false, rows, 2, dim_h, box_h);
  if (e == cudaSuccess) e = allow((const void*)k_two<UP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_kernel(k_two<UP>, sms / 2 * 2, C::THREADS, C::SMEM, 2, st, a, map_w, map_h);
}

}  // namespace

cudaError_t launch_two(bool up, const ExpertArgs& a, const void* rows, const void* w, int sms, cudaStream_t st) {
  return up ? launch_two<true>(a, rows, w, sms, st) : launch_two<false>(a, rows, w, sms, st);
}

}  // namespace mk
