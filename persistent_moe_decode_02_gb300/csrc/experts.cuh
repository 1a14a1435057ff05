// What the kernels of the experts' products share (experts.cu, experts_two.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "eights.cuh"
#include "host.h"
#include "launch.cuh"
#include "mk.h"
#include "ptx.cuh"

namespace mk {

struct ExpertArgs {
  const int *first, *order;
  const float* gates;
  const uint8_t *x, *a_scales, *b_scales;   // x: rows to gather (up)
  uint8_t* out;
  uint8_t* out_scales;
  int* status;
  int pairs, rows, top_k, experts;
  int k, n;                      // elements of a row of A; columns of C
  int extra;                     // what a tile costs beside its columns, in columns
  int box;                       // columns of the large boxes
  int a_wide, b_wide;            // bytes that a row's scales may be read by
  int drop;                      // what stays away (mk_experts_set_debug)
  unsigned long long limit;      // of every wait, ns
};
enum { DROP_LIST = 1, DROP_COPIES = 2, DROP_ACC = 3 };

// Tiles of two SMs (experts_two.cu).
cudaError_t launch_two(bool up, const ExpertArgs& a, const void* rows, const void* w, int sms, cudaStream_t st);

namespace {

using namespace ptx;

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_EXPERTS = 256, MAX_STAGES = 12, SMEM_MOST = 232448;
constexpr unsigned long long WAIT_NS = 2000000000ull;   // limit of every wait, if none is set; and of what is in flight at the end

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], list_full[2], list_free[2], drain;
  unsigned long long limit;
  uint32_t tmem;
  int fail;
  int4 list[2][32];              // the block's next tiles, as they are planned
  int width, columns;            // columns of a tile, tiles of columns
  int row0[MAX_EXPERTS + 1];     // an expert's first row in the sorted order
  int tile0[MAX_EXPERTS + 1];    // and its first tile of rows
};
constexpr int CTL = 4096;
static_assert(sizeof(Ctl) <= CTL, "control words");

using Args = ExpertArgs;

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try(bar, parity)) {
    if (*(volatile int*)&ctl->fail) return false;
    if (now_ns() - t0 > ctl->limit) {
      *(volatile int*)&ctl->fail = 1;
      atomicAdd(status, 1);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  return mbar_try(bar, parity) || wait_slow(bar, parity, ctl, status);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* ctl, int* status) {
  return __all_sync(FULL, wait_one(bar, parity, ctl, status));
}

// Each expert's rows and tiles from `first`, by one warp; entries out of order or
// out of range are moved into it, so whatever they hold, the rows stay within
// the pairs and no row is counted twice.
template <int AM>
__device__ __forceinline__ void set_tables(const Args& a, Ctl* ctl) {
  constexpr int PER = MAX_EXPERTS / 32;
  const int lane = threadIdx.x % 32;
  int f[PER], top = 0;           // ends of the lane's experts, the largest so far
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    f[i] = e < a.experts ? min(max(a.first[e + 1], 0), a.pairs) : 0;
  }
  const int f0 = min(max(a.first[0], 0), a.pairs);
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = top = max(top, f[i]);
  int before = top;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, before, o);
    if (lane >= o) before = max(before, v);
  }
  before = __shfl_up_sync(FULL, before, 1);
  if (lane == 0) before = 0;
  before = max(before, f0);
  int tiles = 0, from = before;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    f[i] = max(f[i], before);
    tiles += (f[i] - from + AM - 1) / AM;
    from = f[i];
  }
  int at = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, at, o);
    if (lane >= o) at += v;
  }
  at -= tiles;
  from = before;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    if (e <= a.experts) {
      ctl->row0[e] = from;
      ctl->tile0[e] = at;
    }
    at += (f[i] - from + AM - 1) / AM;
    from = f[i];
  }
  if (lane == 31 && a.experts == MAX_EXPERTS) {
    ctl->row0[MAX_EXPERTS] = from;
    ctl->tile0[MAX_EXPERTS] = at;
  }
}

struct Tile {
  int e, row0, rows, n0, width;  // expert, first row in the sorted order, rows, first column, columns
};
// The next tile of the list, for a thread (or a warp: the same for all its
// lanes); one arrival frees 32 of them.
struct Reader {
  int i = 0;
  bool known = false;            // a part of the list has come, so the tables behind it are there
  template <bool WARP>
  __device__ __forceinline__ bool next(Ctl* ctl, int* status, Tile& t) {
    const int c = i / 32;
    uint64_t* full = &ctl->list_full[c & 1];
    if (i % 32 == 0 && !(WARP ? wait(full, c >> 1 & 1, ctl, status) : wait_one(full, c >> 1 & 1, ctl, status))) return false;
    known = true;
    const int4 v = ctl->list[c & 1][i % 32];
    if (v.x >> 16 == 0) return false;
    if (++i % 32 == 0) {
      if (WARP) __syncwarp();
      if (!WARP || threadIdx.x % 32 == 0) mbar_arrive(&ctl->list_free[c & 1]);
    }
    t = {v.x & 0xffff, v.y, v.x >> 16, v.z, v.w};
    return true;
  }
};

// A pair's row of x; one that is none reads zeros.
__device__ __forceinline__ int token_of(const Args& a, int at) {
  const int p = a.order[at];
  return p >= 0 && p < a.pairs ? p / a.top_k : a.rows;
}

// silu(gate) * up, with t = e^-|gate|: gate t / (1 + t) * up for a negative gate,
// gate / (1 + t) * up otherwise, so nothing overflows (e^-gate does from gate
// -88.7 on, where silu is 3e-37 still).  t = h * h, and h = 2^y, y = -|gate|
// log2(e) / 2, is a normal number down to gate -174.  Off by (15 + 1.5 |gate|) of
// 2^-24 at most: 8 and 1.5 |gate| of t (2 units in the last place of ex2; y's
// constant and rounding), 1 of the sum, 2 of the reciprocal of a number between 1
// and 2, 4 products; what follows rounds to bf16 (2^-8) or 8 bits (2^-4).   (expf
// and __fdividef: within 9, but up of 8143 rows in 8 bits 236 us instead of 226.)
// An infinite gate is as in gate / (1 + e^-gate), a NaN stays one.
__device__ __forceinline__ float swiglu(float gate, float up) {
  const float h = exp2_approx(-fabsf(gate) * 0.72134752044448170368f), p = gate < 0.f ? h : 1.f;
  return gate * p * (p * rcp_approx(fmaf(h, h, 1.f)) * up);
}

// Behind a wait for loads: their registers are used after it, not before.
template <int N>
__device__ __forceinline__ void landed(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A row's scales of four stages from kb on, a word each, 0 behind the row's end
// (what lies there may be no scale, and 0 times a NaN is one).  By pieces of
// `wide` bytes, or where rows begin at any byte by the aligned words that hold
// them (bytes one by one: up of 8192 rows of 1056, 33 scales a row, 46 us, 37 so).
// A word at the buffer's ends may hold up to 3 bytes of another one: masked, as
// a neighbouring row's are.  (Reading such words byte by byte: 41 us where none
// came up, 44 where some did.)
__device__ __forceinline__ uint4 scales16(const uint8_t* row, int groups, int kb, int wide) {
  const uint8_t* p = row + kb * 4;
  const int left = groups - kb * 4;
  if (wide == 16) return *reinterpret_cast<const uint4*>(p);
  uint32_t v[4] = {0, 0, 0, 0};
  if (wide == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (8 * i < left) {
        const uint2 w = reinterpret_cast<const uint2*>(p)[i];
        v[2 * i] = w.x;
        v[2 * i + 1] = w.y;
      }
  } else {
    const int off = (int)((uintptr_t)p & 3), n = off + min(16, left);   // words with a byte of the row
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - off);
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = 4 * i < n ? q[i] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int here = left - 4 * i;
      v[i] = __funnelshift_r(w[i], w[i + 1], off * 8) & (here >= 4 ? ~0u : here <= 0 ? 0u : (1u << 8 * here) - 1);
    }
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A matrix (or one for each expert) as boxes of 128-byte rows.
cudaError_t tensor_map(CUtensorMap* map, bool e4m3, const void* base, int dims, const cuuint64_t* dim, const cuuint32_t* box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t el = e4m3 ? 1 : 2, stride[2] = {dim[0] * el, dim[0] * dim[1] * el};
  const cuuint32_t step[3] = {1, 1, 1};
  return encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void*>(base), dim,
                stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

int scales_wide(const void* p, int groups) {
  for (int w = 16; w > 4; w /= 2)
    if (groups % w == 0 && (uintptr_t)p % w == 0) return w;
  return 1;
}

}  // namespace
}  // namespace mk
