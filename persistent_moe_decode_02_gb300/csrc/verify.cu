// Probabilities from logits, and the verification of drafted tokens against
// them (mk_probs, mk_verify in include/mk.h).
//
// A row of the vocabulary is one cluster's work: each block holds its segment
// of the row in shared memory, so the row is read once whatever is done with
// it, and the blocks exchange their totals through distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mk.h"

namespace cg = cooperative_groups;

namespace mk {
void set_last_error(const char* msg);
namespace {

constexpr int NT = 512, NW = NT / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_VOCAB = 393216;            // a block's segment of it: 192 KB of shared memory
constexpr int STEP = NT * 4;                  // elements of one pass of a block: 4 consecutive ones a thread
constexpr int MAX_PASSES = MAX_VOCAB / MAX_CLUSTER / STEP;
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 4 elements of a row into shared memory without a stay in registers; those
// past the end are not read.  `wide`: both addresses are 16-byte aligned.
__device__ __forceinline__ void fetch4(float* dst, const float* src, int left, bool wide) {
  if (wide && left >= 4) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + e)), "l"(src + e) : "memory");
  }
}
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 4 elements of a row, 0 past its end.
__device__ __forceinline__ float4 load4(const float* p, int left, bool wide) {
  if (wide && left >= 4) return __ldg(reinterpret_cast<const float4*>(p));
  return make_float4(__ldg(p), left > 1 ? __ldg(p + 1) : 0.f, left > 2 ? __ldg(p + 2) : 0.f, left > 3 ? __ldg(p + 3) : 0.f);
}

// One block's segment of a row.
struct Segment {
  int begin, n;                               // first element, elements (0 for a block past the end)
};
__device__ __forceinline__ Segment segment(int vocab, int blocks, int rank) {
  const int per = ((vocab + blocks - 1) / blocks + 3) / 4 * 4;
  const int b = min(vocab, rank * per);
  return {b, min(per, vocab - b)};
}

// (maximum, its lowest index, unusable) of a set of logits.
struct Top {
  float m;
  int at;
  int bad;
};
__device__ __forceinline__ Top join(Top a, Top b) {
  const bool second = b.m > a.m || (b.m == a.m && b.at < a.at);
  return {second ? b.m : a.m, second ? b.at : a.at, a.bad | b.bad};
}

__global__ void __launch_bounds__(NT) k_probs(const float* logits, int vocab, long long row_stride, float scale,
                                              float* probs, int wide_in, int wide_out) {
  extern __shared__ float4 seg4[];
  float* x = reinterpret_cast<float*>(seg4);
  __shared__ Top wtop[NW];
  __shared__ float wsum[NW];
  __shared__ struct { Top top; float sum; } parts[MAX_CLUSTER];
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();                        // every block of the cluster runs before one writes into another
  const int blocks = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x;
  const size_t row = blockIdx.x / blocks;
  const Segment s = segment(vocab, blocks, rank);
  const float* src = logits + row * row_stride + s.begin;
  for (int i = tid * 4; i < s.n; i += STEP) fetch4(x + i, src + i, s.n - i, wide_in);
  fetch_wait();                               // a thread reads only what it fetched
  Top t = {-INFINITY, 0x7fffffff, 0};
  for (int i = tid * 4; i < s.n; i += STEP)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < s.n) {
        const float v = x[i + e];
        if (!(v < INFINITY)) t.bad = 1;       // NaN or +infinity
        if (v > t.m) { t.m = v; t.at = s.begin + i + e; }   // strictly: the lowest index stays
      }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    t = join(t, {__shfl_xor_sync(FULL, t.m, o), __shfl_xor_sync(FULL, t.at, o), __shfl_xor_sync(FULL, t.bad, o)});
  if (tid % 32 == 0) wtop[tid / 32] = t;
  __syncthreads();
  t = wtop[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) t = join(t, wtop[w]);
  float sum = 0.f;
  if (scale > 0.f && t.m > -INFINITY)
    for (int i = tid * 4; i < s.n; i += STEP)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < s.n) sum += exp2f((x[i + e] - t.m) * scale);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  if (tid % 32 == 0) wsum[tid / 32] = sum;
  __syncthreads();
  cl.barrier_wait();
  if (tid < blocks) {                         // this block's totals into every block's table
    float b = 0.f;
    for (int w = 0; w < NW; ++w) b += wsum[w];
    auto* p = cl.map_shared_rank(&parts[rank], tid);
    p->top = t;
    p->sum = b;
  }
  cl.sync();
  t = parts[0].top;
  for (int r = 1; r < blocks; ++r) t = join(t, parts[r].top);
  float total = 0.f;
  for (int r = 0; r < blocks; ++r)
    if (parts[r].sum > 0.f) total += parts[r].sum * exp2f((parts[r].top.m - t.m) * scale);
  const float inv = 1.f / total;
  float* dst = probs + row * vocab + s.begin;
  for (int i = tid * 4; i < s.n; i += STEP) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (scale > 0.f) v[e] = i + e < s.n && t.m > -INFINITY ? exp2f((x[i + e] - t.m) * scale) * inv : 0.f;
      else v[e] = s.begin + i + e == t.at && t.m > -INFINITY ? 1.f : 0.f;
      if (t.bad) v[e] = __int_as_float(0x7fffffff);
    }
    if (wide_out && i + 4 <= s.n) {
      *reinterpret_cast<float4*>(dst + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < s.n) dst[i + e] = v[e];
    }
  }
}

// A weight as a whole number of 2^-40: sums of those do not depend on their
// order, so any split of the row draws the same token.
__device__ __forceinline__ unsigned long long mass(float w) {
  return w > 0.f ? __float2ull_rn(fminf(w, 1.f) * 1099511627776.f) : 0ull;
}

struct VerifyArgs {
  int drafts, vocab, wide;
  const float *target, *draft;
  const int *tok, *count;
  const float *u, *r;
  int *out, *accepted;
};

__global__ void __launch_bounds__(NT) k_verify(VerifyArgs a) {
  extern __shared__ float4 seg4[];
  __shared__ unsigned long long sums[MAX_PASSES * NW], totals[MAX_CLUSTER];
  __shared__ int n_acc;
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();
  const int blocks = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int b = blockIdx.x / blocks, V = a.vocab;
  const int n = a.count ? min(max(a.count[b], 0), a.drafts) : a.drafts;
  const float* target = a.target + (size_t)b * (a.drafts + 1) * V;
  const float* draft = a.draft ? a.draft + (size_t)b * a.drafts * V : nullptr;
  const int* tok = a.tok + (size_t)b * a.drafts;
  if (warp == 0) {                            // every block of the cluster decides alike
    int first = n;
    for (int i0 = 0; i0 < n && first == n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n) {
        const int x = tok[i];
        ok = x >= 0 && x < V;
        if (ok) {
          const double q = draft ? draft[(size_t)i * V + x] : 1.0;   // products of 24-bit factors are exact in 53
          ok = (double)a.u[(size_t)b * a.drafts + i] * q < (double)target[(size_t)i * V + x];
        }
      }
      const unsigned no = __ballot_sync(FULL, !ok);
      if (no) first = i0 + __ffs(no) - 1;
    }
    if (lane == 0) n_acc = first;
  }
  __syncthreads();
  const int acc = n_acc;
  const bool refused = acc < n;
  const Segment s = segment(V, blocks, rank);
  float* w = reinterpret_cast<float*>(seg4);
  const float* trow = target + (size_t)acc * V + s.begin;
  const float* drow = refused && draft ? draft + (size_t)acc * V + s.begin : nullptr;
  const int gone = refused && !draft ? tok[acc] - s.begin : -1;   // a certain draft's place in this segment
  const int passes = (s.n + STEP - 1) / STEP;
  cl.barrier_wait();
  unsigned long long total = 0, before = 0;
  for (int whole = refused ? 0 : 1; whole < 2; ++whole) {
    const float* less = whole ? nullptr : drow;
#pragma unroll 4
    for (int i = tid * 4; i < s.n; i += STEP) {
      float4 t = load4(trow + i, s.n - i, a.wide);
      if (less) {
        const float4 d = load4(less + i, s.n - i, a.wide);
        t.x -= d.x; t.y -= d.y; t.z -= d.z; t.w -= d.w;
      }
      *reinterpret_cast<float4*>(w + i) = t;
    }
    if (!whole && gone >= 0 && gone < s.n && gone % STEP / 4 == tid) w[gone] -= 1.f;
    for (int p = 0; p < passes; ++p) {
      const int i = p * STEP + tid * 4;
      unsigned long long m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < s.n) m += mass(w[i + e]);
#pragma unroll
      for (int o = 16; o; o >>= 1) m += __shfl_xor_sync(FULL, m, o);
      if (lane == 0) sums[p * NW + warp] = m;
    }
    __syncthreads();
    if (warp == 0) {
      unsigned long long m = 0;
      for (int k = lane; k < passes * NW; k += 32) m += sums[k];
#pragma unroll
      for (int o = 16; o; o >>= 1) m += __shfl_xor_sync(FULL, m, o);
      if (lane < blocks) *cl.map_shared_rank(&totals[rank], lane) = m;
    }
    cl.sync();
    total = before = 0;
    for (int r = 0; r < blocks; ++r) {
      if (r < rank) before += totals[r];
      total += totals[r];
    }
    if (total > 0) {
      if (warp == 0) {
        const float rv = a.r[b];
        // floor(r 2^24), 0 for a NaN
        const unsigned long long U = rv > 0.f ? (unsigned long long)fminf(floorf(rv * 16777216.f), 16777215.f) : 0ull;
        unsigned long long at = __umul64hi(total, U << 40);       // floor(total U / 2^24)
        const unsigned long long mine = totals[rank];
        if (at >= before && at - before < mine) {                  // the token lies in this segment
          at -= before;
          int k = 0;
          for (;; k += 32) {                                       // its group of 128
            const unsigned long long v = k + lane < passes * NW ? sums[k + lane] : 0ull;
            unsigned long long up = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned long long o2 = __shfl_up_sync(FULL, up, o);
              if (lane >= o) up += o2;
            }
            const unsigned hit = __ballot_sync(FULL, up > at);
            if (hit) {
              const int l = __ffs(hit) - 1;
              at -= __shfl_sync(FULL, up - v, l);
              k += l;
              break;
            }
            at -= __shfl_sync(FULL, up, 31);
          }
          const int i = k / NW * STEP + k % NW * 128 + lane * 4;
          unsigned long long m[4], v = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            m[e] = i + e < s.n ? mass(w[i + e]) : 0ull;
            v += m[e];
          }
          unsigned long long up = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long o2 = __shfl_up_sync(FULL, up, o);
            if (lane >= o) up += o2;
          }
          const unsigned hit = __ballot_sync(FULL, up > at);
          if (lane == __ffs(hit) - 1) {
            at -= up - v;
            int e = 0;
            while (e < 3 && at >= m[e]) at -= m[e++];
            a.out[(size_t)b * (a.drafts + 1) + acc] = s.begin + i + e;
          }
        }
      }
      break;
    }
    cl.sync();                                // every block has read the totals: the next round writes them again
  }
  if (rank == 0) {
    for (int i = tid; i <= a.drafts; i += NT)
      if (i != acc) a.out[(size_t)b * (a.drafts + 1) + i] = i < acc ? tok[i] : -1;
      else if (total == 0) a.out[(size_t)b * (a.drafts + 1) + i] = -1;
    if (tid == 0) a.accepted[b] = acc;
  }
}

int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

int fail_cuda(const char* what, cudaError_t e) {
  char buf[224];
  snprintf(buf, sizeof(buf), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  return fail(MK_ERR_CUDA, buf);
}

// Blocks of a row's cluster: enough that a segment has a pass or more for each.
int cluster_of(int vocab) {
  int c = 1;
  while (c < MAX_CLUSTER && vocab > c * STEP) c *= 2;
  return c;
}

template <class... A>
cudaError_t launch_rows(void (*k)(A...), long long rows, int cluster, size_t smem, cudaStream_t st, A... args) {
  cudaError_t e = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cluster));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

size_t segment_bytes(int vocab, int cluster) {
  return (size_t)((vocab + cluster - 1) / cluster + 3) / 4 * 16;
}

bool aligned(const void* p, size_t n) { return p && (uintptr_t)p % n == 0; }

}  // namespace
}  // namespace mk

extern "C" {

int mk_probs(const float* logits, int rows, int vocab, long long row_stride, float temperature, float* probs,
             mk_stream stream) {
  using namespace mk;
  if (rows < 0 || vocab < 1) return fail(MK_ERR_INVALID, "mk_probs: rows or vocab");
  if (vocab > MAX_VOCAB) return fail(MK_ERR_UNSUPPORTED, "mk_probs: vocab above 393216");
  if (rows > (1 << 27)) return fail(MK_ERR_UNSUPPORTED, "mk_probs: rows above 2^27");
  if (row_stride < vocab || row_stride > (1ll << 34)) return fail(MK_ERR_INVALID, "mk_probs: row_stride");
  if (!(temperature >= 0.f) || !isfinite(temperature) || (temperature > 0.f && !isfinite(1.f / temperature)))
    return fail(MK_ERR_INVALID, "mk_probs: temperature must be 0 (greedy) or a finite value whose inverse is finite");
  if (!aligned(logits, 4) || !aligned(probs, 4)) return fail(MK_ERR_INVALID, "mk_probs: a buffer is NULL or not aligned to its type");
  {
    const char *l0 = (const char*)logits, *p0 = (const char*)probs;
    const char* l1 = l0 + 4 * ((size_t)(rows ? rows - 1 : 0) * row_stride + vocab);
    const char* p1 = p0 + 4 * (size_t)rows * vocab;
    if (rows && l0 < p1 && p0 < l1 && !(l0 == p0 && row_stride == vocab))
      return fail(MK_ERR_INVALID, "mk_probs: probs overlaps the logits in other places than their own");
  }
  if (rows == 0) return MK_OK;
  const int c = cluster_of(vocab);
  const float scale = temperature > 0.f ? fminf(1.4426950408889634f / temperature, 3.4e38f) : 0.f;   // log2(e) / T
  const int win = aligned(logits, 16) && row_stride % 4 == 0, wout = aligned(probs, 16) && vocab % 4 == 0;
  const cudaError_t e = launch_rows(k_probs, rows, c, segment_bytes(vocab, c), (cudaStream_t)stream, logits, vocab,
                                    row_stride, scale, probs, win, wout);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_probs", e);
}

int mk_verify(int batch, int max_draft, int vocab, const float* target, const float* draft, const int* drafts,
              const int* n_draft, const float* u, const float* r, int* tokens, int* accepted, mk_stream stream) {
  using namespace mk;
  if (batch < 0 || max_draft < 0 || vocab < 1) return fail(MK_ERR_INVALID, "mk_verify: batch, max_draft or vocab");
  if (vocab > MAX_VOCAB) return fail(MK_ERR_UNSUPPORTED, "mk_verify: vocab above 393216");
  if (batch > (1 << 20) || max_draft > (1 << 20)) return fail(MK_ERR_UNSUPPORTED, "mk_verify: batch or max_draft above 2^20");
  if (!aligned(target, 4) || !aligned(r, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) ||
      (max_draft && (!aligned(drafts, 4) || !aligned(u, 4))) || (draft && !aligned(draft, 4)) ||
      (n_draft && !aligned(n_draft, 4)))
    return fail(MK_ERR_INVALID, "mk_verify: a buffer is NULL or not aligned to its type");
  if (batch == 0) return MK_OK;
  const int c = cluster_of(vocab);
  VerifyArgs a = {max_draft, vocab, 0, target, draft, drafts, n_draft, u, r, tokens, accepted};
  a.wide = aligned(target, 16) && (!draft || aligned(draft, 16)) && vocab % 4 == 0;
  const size_t smem = segment_bytes(vocab, c);
  const cudaError_t e = launch_rows(k_verify, batch, c, smem, (cudaStream_t)stream, a);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_verify", e);
}

}  // extern "C"
