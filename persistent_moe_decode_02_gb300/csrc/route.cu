// Routing of a chunk's rows to experts (mk_route in include/mk.h): each row's k
// largest router logits, their softmax, and the (row, choice) pairs sorted by
// expert.
//
// A warp takes a row: its logits as integers in the order of their values, k
// rounds of a warp's maximum and the lowest index that has it.  The sort counts:
// each warp of one cluster counts its run of pairs by expert, the counts are
// summed over warps, blocks and experts, and a second pass puts each pair at
// its place, so the order is the pairs' own within an expert and the same on
// every call.
#include <cooperative_groups.h>
#include <math.h>

#include "host.h"
#include "launch.cuh"
#include "mk.h"

namespace cg = cooperative_groups;

namespace mk {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_EXPERTS = 256, MAX_TOP = 8;
constexpr int NT = 1024, NW = NT / 32, BUCKETS = MAX_EXPERTS + 1;   // the last one: pairs without an expert

struct RouteArgs {
  const float* logits;
  long long stride;
  int rows, experts, k;
  int* ids;
  float* gates;
  int *first, *order;
};

// A logit as an integer in the order of the values, 0 for -infinity and NaN,
// which no row chooses.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);   // (-0 is 0)
  const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
  return x == -INFINITY || isnan(x) ? 0u : key;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// One row's choice by a warp; V logits a lane.
template <int V>
__device__ __forceinline__ void choose(const RouteArgs& a, int row) {
  const int lane = threadIdx.x % 32;
  const float* src = a.logits + row * a.stride;
  uint32_t key[V];
  bool none = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    const float x = e < a.experts ? src[e] : -INFINITY;
    none |= isnan(x);
    key[v] = key_of(x);
  }
  const bool spoilt = __any_sync(FULL, none);
  int id = -1;
  uint32_t mine = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
    int at = lane;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v * 32 + lane;
      }
    const uint32_t top = __reduce_max_sync(FULL, best);
    if (top == 0) break;                         // nothing is left to choose
    const int e = __reduce_min_sync(FULL, best == top ? at : 0x7fffffff);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == v * 32 + lane) key[v] = 0;
    if (lane == j) {
      id = e;
      mine = top;
    }
  }
  const float x = value_of(mine), m = __shfl_sync(FULL, x, 0);
  float w = id >= 0 ? expf(x - m) : 0.f;         // +infinity, the row's largest: NaN
  float sum = w;
#pragma unroll
  for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  if (lane < a.k) {
    a.ids[(size_t)row * a.k + lane] = id;
    a.gates[(size_t)row * a.k + lane] = id < 0 ? 0.f : spoilt ? NAN : w / sum;
  }
}
__device__ __forceinline__ void choose_rows(const RouteArgs& a, int warp, int warps) {
  for (int row = warp; row < a.rows; row += warps) {
    if (a.experts <= 32) choose<1>(a, row);
    else if (a.experts <= 64) choose<2>(a, row);
    else if (a.experts <= 128) choose<4>(a, row);
    else choose<8>(a, row);
  }
}

__global__ void __launch_bounds__(256) k_choose(const __grid_constant__ RouteArgs a) {
  allow_next();
  await_stream();
  choose_rows(a, (blockIdx.x * 256 + threadIdx.x) / 32, gridDim.x * 8);
}

// The sort, in one cluster; `all`: the choice too.
__global__ void __launch_bounds__(NT) k_sort(const __grid_constant__ RouteArgs a, bool all) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int hist[NW][BUCKETS], total[BUCKETS], start[BUCKETS + 1];
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nb = a.experts + 1;
  allow_next();
  for (int i = tid; i < NW * BUCKETS; i += NT) (&hist[0][0])[i] = 0;
  await_stream();
  if (all) {
    choose_rows(a, rank * NW + warp, blocks * NW);
    __threadfence();
    cluster.sync();
  } else {
    __syncthreads();
  }
  const long long pairs = (long long)a.rows * a.k;
  const long long chunks = (pairs + 31) / 32, per = (chunks + blocks * NW - 1) / (blocks * NW);
  const long long c0 = (rank * NW + warp) * per, c1 = min(chunks, c0 + per);
  auto bucket = [&](long long p) {
    const int id = p < pairs ? *(volatile const int*)(a.ids + p) : -1;
    return p >= pairs ? BUCKETS : id < 0 ? a.experts : id;
  };
  for (long long c = c0; c < c1; ++c) {
    const int b = bucket(c * 32 + lane);
    const unsigned same = __match_any_sync(FULL, b);
    if (b < BUCKETS && lane == __ffs(same) - 1) hist[warp][b] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  if (tid < nb) {                                // the warps before, within the block
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < NW; ++w) {
      const int n = hist[w][tid];
      hist[w][tid] = sum;
      sum += n;
    }
    total[tid] = sum;
  }
  cluster.sync();
  int before = 0, whole = 0;
  if (tid < nb)
    for (int r = 0; r < blocks; ++r) {           // the blocks before
      const int n = *cluster.map_shared_rank(&total[tid], r);
      before += r < rank ? n : 0;
      whole += n;
    }
  if (tid < nb) start[tid] = whole;
  __syncthreads();
  if (warp == 0) {                               // the experts before
    constexpr int PER = (BUCKETS + 31) / 32;
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = lane * PER + i;
      n[i] = b < nb ? start[b] : 0;
      sum += n[i];
    }
    int up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(FULL, up, o);
      if (lane >= o) up += v;
    }
    up -= sum;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = lane * PER + i;
      if (b < nb) {
        start[b] = up;
        if (rank == 0) a.first[b] = up;
      }
      up += n[i];
    }
  }
  __syncthreads();
  if (tid < nb) {
    before += start[tid];
#pragma unroll 8
    for (int w = 0; w < NW; ++w) hist[w][tid] += before;
  }
  __syncthreads();
  for (long long c = c0; c < c1; ++c) {
    const long long p = c * 32 + lane;
    const int b = bucket(p);
    const unsigned same = __match_any_sync(FULL, b);
    const int at = b < BUCKETS ? hist[warp][b] : 0;
    __syncwarp();
    if (b < BUCKETS) {
      a.order[at + __popc(same & ((1u << lane) - 1))] = (int)p;
      if (lane == __ffs(same) - 1) hist[warp][b] = at + __popc(same);
    }
    __syncwarp();
  }
  cluster.sync();                                // nobody leaves while its counts are read
}

}  // namespace
}  // namespace mk

extern "C" int mk_route(int rows, int n_experts, int top_k, const float* logits, long long row_stride, int* ids, float* gates,
                        int* first, int* order, mk_stream stream) {
  using namespace mk;
  if (rows < 0 || n_experts < 1 || top_k < 1 || top_k > n_experts) return fail(MK_ERR_INVALID, "mk_route: rows, n_experts or top_k");
  if (n_experts > MAX_EXPERTS || top_k > MAX_TOP) return fail(MK_ERR_UNSUPPORTED, "mk_route: at most 256 experts, 8 of them a row");
  if (rows > (1 << 27)) return fail(MK_ERR_UNSUPPORTED, "mk_route: rows above 2^27");
  if (row_stride < n_experts || row_stride > (1ll << 34)) return fail(MK_ERR_INVALID, "mk_route: row_stride");
  if (!aligned(first, 4) || (rows && (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(gates, 4) || !aligned(order, 4))))
    return fail(MK_ERR_INVALID, "mk_route: a buffer is NULL or not aligned to its type");
  const size_t pairs = (size_t)rows * top_k;
  const Span s[5] = {{ids, 4 * pairs},
                     {gates, 4 * pairs},
                     {first, 4 * (size_t)(n_experts + 1)},
                     {order, 4 * pairs},
                     {rows ? logits : nullptr, rows ? 4 * ((size_t)(rows - 1) * row_stride + n_experts) : 0}};
  if (clash(s, 4, 5)) return fail(MK_ERR_INVALID, "mk_route: two of the buffers overlap");
  const RouteArgs a = {logits, row_stride, rows, n_experts, top_k, ids, gates, first, order};
  const cudaStream_t st = (cudaStream_t)stream;
  int sms = 0;
  cudaError_t e = multiprocessors(&sms);
  const bool all = rows <= 512;
  if (e == cudaSuccess && !all) {
    const int most = (rows + 7) / 8;
    e = launch_kernel(k_choose, dim3(most < sms * 8 ? most : sms * 8), 256, 0, 1, st, a);
  }
  const int blocks = pairs <= 1024 ? 1 : pairs <= 4096 ? 4 : 8;
  if (e == cudaSuccess) e = launch_kernel(k_sort, dim3(blocks), NT, 0, blocks, st, a, all);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_route", e);
}
