// Routing of a chunk's rows to experts (mk_route in include/mk.h): each row's k
// largest router logits, their softmax, and the (row, choice) pairs sorted by
// expert.
//
// A warp takes a row: its logits as integers in the order of their values, k
// rounds of a warp's maximum and the lowest index that has it.  The sort is one
// cluster's: each block counts its rows' pairs by expert, the counts are summed
// over blocks and experts, and each pair goes to its place, so the order is the
// pairs' own within an expert and the same on every call.
//
// Neither moves much: 8143 rows of 128 logits are 5 MB.  They take 10.5 us, 4.9
// for the choice (450 instructions a row; the SMs issue 2.7 a cycle) and the rest
// for the sort, a chain of ten barriers over 16 SMs; one row takes 1.9 us, one
// block; 37 rows 4.7 us, 2049 rows 6.4.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "host.h"
#include "launch.cuh"
#include "mk.h"

namespace cg = cooperative_groups;

namespace mk {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_EXPERTS = 256, MAX_TOP = 8;
constexpr int NT = 1024, BUCKETS = MAX_EXPERTS + 1;   // the last one: pairs without an expert
constexpr int FEW_PAIRS = 128;

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
  return x > -INFINITY ? b ^ ((uint32_t)((int)b >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// One row's logits, V a lane, and a warp's choice among them: the lane's place
// among the choices (lane < k) has the expert that is returned, -1 for none.
template <int V>
struct Row {
  float x[V];
};
template <int V>
__device__ __forceinline__ Row<V> load_row(const RouteArgs& a, int row) {
  Row<V> r;
  const float* src = a.logits + row * a.stride;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + threadIdx.x % 32;
    r.x[v] = e < a.experts && row < a.rows ? src[e] : -INFINITY;
  }
  return r;
}
template <int V>
__device__ __forceinline__ int choose(const RouteArgs& a, int row, const Row<V>& r) {
  const int lane = threadIdx.x % 32;
  uint32_t key[V];
  bool none = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    none |= isnan(r.x[v]);
    key[v] = key_of(r.x[v]);
  }
  const bool spoilt = __any_sync(FULL, none);
  // The lane's own, the largest first and the lower index first among equal
  // ones: a round then looks at one a lane.
  int at[V];
#pragma unroll
  for (int v = 0; v < V; ++v) at[v] = v * 32 + lane;
#pragma unroll
  for (int n = V - 1; n > 0; --n)
#pragma unroll
    for (int v = 0; v < n; ++v)
      if (key[v + 1] > key[v]) {
        const uint32_t k0 = key[v];
        const int a0 = at[v];
        key[v] = key[v + 1];
        at[v] = at[v + 1];
        key[v + 1] = k0;
        at[v + 1] = a0;
      }
  int id = -1;
  uint32_t mine = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t top = __reduce_max_sync(FULL, key[0]);
    if (top == 0) break;                         // nothing is left to choose
    const unsigned who = __ballot_sync(FULL, key[0] == top);
    int winner = __ffs(who) - 1;
    if (who & (who - 1)) {                       // equal ones: the lowest index
      const int e = __reduce_min_sync(FULL, key[0] == top ? at[0] : 0x7fffffff);
      winner = e % 32;
    }
    const int e = __shfl_sync(FULL, at[0], winner);
    if (lane == winner) {
#pragma unroll
      for (int v = 0; v + 1 < V; ++v) {
        key[v] = key[v + 1];
        at[v] = at[v + 1];
      }
      key[V - 1] = 0;
    }
    if (lane == j) {
      id = e;
      mine = top;
    }
  }
  const float x = value_of(mine), m = __shfl_sync(FULL, x, 0);
  const float w = id >= 0 ? expf(x - m) : 0.f;   // +infinity, the row's largest: NaN
  float sum = w;
#pragma unroll
  for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  if (lane < a.k) {
    a.ids[(size_t)row * a.k + lane] = id;
    a.gates[(size_t)row * a.k + lane] = id < 0 ? 0.f : spoilt ? NAN : w / sum;
  }
  return id;
}
// f(V) for the logits of a lane.
template <class F>
__device__ __forceinline__ void with_width(int experts, F&& f) {
  if (experts <= 32) f(std::integral_constant<int, 1>());
  else if (experts <= 64) f(std::integral_constant<int, 2>());
  else if (experts <= 128) f(std::integral_constant<int, 4>());
  else f(std::integral_constant<int, 8>());
}

__global__ void __launch_bounds__(256) k_choose(const __grid_constant__ RouteArgs a) {
  allow_next();
  await_stream();
  const int row = (int)(((long long)blockIdx.x * 256 + threadIdx.x) / 32);
  if (row < a.rows)
    with_width(a.experts, [&](auto n) {
      constexpr int V = decltype(n)::value;
      choose<V>(a, row, load_row<V>(a, row));
    });
}

// Few rows in one block: a pair's place is the number of pairs before it, an
// expert's first the number of those of lower experts, counted one by one.
__global__ void __launch_bounds__(1024) k_few(const __grid_constant__ RouteArgs a) {
  __shared__ alignas(16) int keys[FEW_PAIRS];    // expert (the last one: none), pair
  allow_next();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, pairs = a.rows * a.k, padded = (pairs + 3) / 4 * 4;
  if ((int)threadIdx.x < padded - pairs) keys[pairs + threadIdx.x] = INT_MAX;
  await_stream();
  with_width(a.experts, [&](auto n) {
    constexpr int V = decltype(n)::value;
    const int warps = blockDim.x / 32;
    Row<V> r = load_row<V>(a, warp);
    for (int row = warp; row < a.rows; row += warps) {
      const Row<V> now = r;
      r = load_row<V>(a, row + warps);           // the next one is on its way
      const int id = choose<V>(a, row, now);
      if (lane < a.k) keys[row * a.k + lane] = (id < 0 ? a.experts : id) * FEW_PAIRS + row * a.k + lane;
    }
  });
  __syncthreads();
  for (int i = threadIdx.x; i < pairs + a.experts + 1; i += blockDim.x) {
    const int key = i < pairs ? keys[i] : (i - pairs) * FEW_PAIRS;
    int n = 0;
#pragma unroll 8
    for (int q = 0; q < padded; q += 4) {
      const int4 v = *reinterpret_cast<const int4*>(keys + q);
      n += (v.x < key) + (v.y < key) + (v.z < key) + (v.w < key);
    }
    if (i < pairs) a.order[n] = i;
    else a.first[i - pairs] = n;
  }
}

// Exclusive sums of n <= BUCKETS numbers, by one warp.
__device__ __forceinline__ void scan(const int* in, int* out, int n) {
  constexpr int PER = (BUCKETS + 31) / 32;
  const int lane = threadIdx.x % 32;
  int v[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = lane * PER + i < n ? in[lane * PER + i] : 0;
    sum += v[i];
  }
  int up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, up, o);
    if (lane >= o) up += x;
  }
  up -= sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (lane * PER + i < n) out[lane * PER + i] = up;
    up += v[i];
  }
}

// The sort, in one cluster, a run of rows for each block.  A row has an expert
// once, so an expert's pairs of 32 rows are a word with a bit for each row, and a
// pair's place among them is the number of bits before its own.  (Places without
// an expert: a word for each of the k.)  Blocks take BATCH rows at a time.
constexpr int BATCH = 512, GROUPS = BATCH / 32, MAX_BLOCKS = 16;
__global__ void __launch_bounds__(NT) k_sort(const __grid_constant__ RouteArgs a, int rows_per) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ uint32_t word[GROUPS][MAX_EXPERTS + MAX_TOP];
  __shared__ uint16_t pre[GROUPS][BUCKETS];      // pairs of the groups before
  __shared__ int sorted[MAX_BLOCKS * BUCKETS];   // every block's totals; then expert, pair of the batch
  __shared__ int count[BUCKETS], whole[BUCKETS], start[BUCKETS], local[BUCKETS], base[BUCKETS], none[GROUPS];
  static_assert(MAX_BLOCKS * BUCKETS >= BATCH * MAX_TOP, "a batch's pairs");
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid / 32, nb = a.experts + 1;
  const int row0 = min(a.rows, rank * rows_per), row1 = min(a.rows, row0 + rows_per);
  constexpr int MINE = BATCH * MAX_TOP / NT;
  int id[MINE];                                  // of pairs tid, tid + NT, ... of the batch
  const int inv = (65536 + a.k - 1) / a.k;       // p / k = p * inv >> 16 for p < 4096, k <= 8
  auto build = [&](int r0) {
    const int pairs = (min(row1, r0 + BATCH) - r0) * a.k;
    const int* ids = a.ids + (size_t)r0 * a.k;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int p = i * NT + tid;
      if (p < pairs) {
        const int x = ids[p], r = p * inv >> 16;
        id[i] = x < 0 ? a.experts + p - r * a.k : x;
        atomicOr(&word[r / 32][id[i]], 1u << r % 32);
        if (x < 0) atomicAdd(&none[r / 32], 1);
      }
    }
    __syncthreads();
    if (tid < nb) {
      int n[GROUPS], sum = 0;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) n[g] = tid == a.experts ? none[g] : (int)word[g][tid];
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        pre[g][tid] = (uint16_t)sum;
        sum += tid == a.experts ? n[g] : __popc(n[g]);
      }
      count[tid] = sum;
    }
  };
  auto clear = [&] {
    for (int i = tid; i < GROUPS * (MAX_EXPERTS + MAX_TOP); i += NT) (&word[0][0])[i] = 0;
    if (tid < GROUPS) none[tid] = 0;
    __syncthreads();
  };
  allow_next();
  clear();
  cluster.sync();                                // every block is there to be written to
  await_stream();
  int total = 0;
  if (row0 == row1 && tid < nb) count[tid] = 0;
  for (int r0 = row0; r0 < row1; r0 += BATCH) {
    if (r0 > row0) {
      __syncthreads();
      clear();
    }
    build(r0);
    if (tid < nb) total += count[tid];
  }
  if (tid < nb)
    for (int r = 0; r < blocks; ++r) *cluster.map_shared_rank(&sorted[rank * BUCKETS + tid], r) = total;
  cluster.sync();
  int before = 0;                                // the blocks before
  if (tid < nb) {
    int all = 0;
#pragma unroll 8
    for (int r = 0; r < blocks; ++r) {
      const int n = sorted[r * BUCKETS + tid];
      before += r < rank ? n : 0;
      all += n;
    }
    whole[tid] = all;
  }
  __syncthreads();
  if (warp == 0) scan(whole, start, nb);         // the experts before
  if (warp == 1) scan(count, local, nb);
  __syncthreads();
  if (tid < nb) {
    base[tid] = start[tid] + before;
    if (rank == 0) a.first[tid] = start[tid];
  }
  const bool once = row1 - row0 <= BATCH;        // the first pass's words are still there
  for (int r0 = row0; r0 < row1; r0 += BATCH) {
    if (!once) {
      __syncthreads();
      clear();
      build(r0);
      __syncthreads();
      if (warp == 0) scan(count, local, nb);
      __syncthreads();
    }
    const int pairs = (min(row1, r0 + BATCH) - r0) * a.k;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int p = i * NT + tid;
      if (p < pairs) {
        const int r = p * inv >> 16, g = r / 32, e = min(id[i], a.experts);
        const uint32_t less = (1u << r % 32) - 1;
        int at = local[e] + pre[g][e];
        if (id[i] < a.experts) {
          at += __popc(word[g][e] & less);
        } else {
          for (int j = 0; j < a.k; ++j) {
            const uint32_t w = word[g][a.experts + j];
            at += __popc(w & less) + (a.experts + j < id[i] ? w >> r % 32 & 1 : 0);
          }
        }
        sorted[at] = e << 16 | p;
      }
    }
    __syncthreads();
    for (int l = tid; l < pairs; l += NT) {      // an expert's pairs side by side
      const int v = sorted[l], e = v >> 16;
      a.order[base[e] + l - local[e]] = r0 * a.k + (v & 0xffff);
    }
    if (!once) {
      __syncthreads();
      if (tid < nb) base[tid] += count[tid];
    }
  }
}

// Whether the current device has room for a cluster of 16 (beyond what every
// device has to offer), asked for once by each host thread.
cudaError_t wide_cluster(bool* ok) {
  thread_local int device = -1;
  thread_local bool room = false;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != device) {
    e = cudaFuncSetAttribute(k_sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 16;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = 16;
    cfg.blockDim = NT;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_sort, &cfg) != cudaSuccess) {   // no room is an answer too
      cudaGetLastError();
      n = 0;
    }
    room = n > 0;
    device = dev;
  }
  *ok = room;
  return e;
}

// A block for every 128 rows, 16 of them at most.
cudaError_t launch_sort(const RouteArgs& a, cudaStream_t st) {
  int blocks = 1;
  while (blocks < 16 && a.rows > blocks * 128) blocks *= 2;
  if (blocks == 16) {
    bool ok = false;
    const cudaError_t e = wide_cluster(&ok);
    if (e != cudaSuccess) return e;
    if (!ok) blocks = 8;
  }
  const int rows_per = ((a.rows + blocks - 1) / blocks + 31) / 32 * 32;
  return launch_kernel(k_sort, blocks, NT, 0, blocks, st, a, rows_per);
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
  cudaError_t e;
  if (pairs <= FEW_PAIRS) {
    e = launch_kernel(k_few, 1, rows <= 8 ? 256 : 1024, 0, 1, st, a);
  } else {
    e = launch_kernel(k_choose, (rows + 7) / 8, 256, 0, 1, st, a);
    if (e == cudaSuccess) e = launch_sort(a, st);
  }
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_route", e);
}
