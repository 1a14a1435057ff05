// Probabilities from logits, and the verification of drafted tokens against
// them (mk_probs, mk_verify in include/mk.h).
//
// A row of the vocabulary is one cluster's work: each block holds its segment
// of the row in registers, so the row is read once whatever is done with
// it, and the blocks exchange their totals through distributed shared memory.
// 160 rows of 151936 take 40.0 us (4.9 TB/s, 0.73 of a copy's rate: clusters of
// 8 are 1280 blocks, 4.2 rounds of the 304 that run at once); one row 4.2 us.  A
// verification reads the row or two that its draw needs, not the others: 32 of
// them with up to five drafts take 12.3 us, one 5.8 us, a chain of five
// dependent reads and two exchanges.  At vocabularies that are no multiple of 4
// it reads element by element (32 requests whose first draft is refused: 12.6 us
// of 151935, 9.9 of 151936).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <type_traits>

#include "launch.cuh"
#include "mk.h"
#include "rows.h"

namespace cg = cooperative_groups;

namespace mk {
void set_last_error(const char* msg);
namespace {

constexpr int NT = ROW_THREADS, NW = NT / 32;
constexpr unsigned FULL = 0xffffffffu;

// 4 elements of a row, `none` past its end and in the `skip` places before its
// start.  `wide`: the address is 16-byte aligned.
__device__ __forceinline__ float4 load4(const float* p, int left, bool wide, float none, int skip = 0) {
  if (wide && left >= 4 && skip <= 0) return *reinterpret_cast<const float4*>(p);
  float4 v = make_float4(none, none, none, none);
  if (left > 0 && skip <= 0) v.x = p[0];
  if (left > 1 && skip <= 1) v.y = p[1];
  if (left > 2 && skip <= 2) v.z = p[2];
  if (left > 3) v.w = p[3];
  return v;
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

// The larger of two, a NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// softmax(logits * scale / log2(e)), scale 0: greedy.  A block holds PASSES x
// STEP elements of its row in registers: the row is read once, the exponential
// taken once (against the block's own maximum), and written once.
template <int PASSES>
__global__ void __launch_bounds__(NT) k_probs(const float* logits, int vocab, long long row_stride, float scale,
                                              float* probs, int shiftable, int at_once) {
  __shared__ float wmax[NW], wsum[NW];
  __shared__ int wat[NW];
  __shared__ struct { float m, sum; int at; } parts[FEW];
  await_stream();
  allow_next();
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();                        // every block of the cluster runs before one writes into another
  const int blocks = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x;
  const size_t row = blockIdx.x / blocks;
  // A row may start anywhere, and its 16-byte pieces where its address says: it
  // is taken to begin `shift` elements earlier, whose places stay empty.
  const float* first = logits + row * row_stride;
  const int shift = shiftable ? (int)((uintptr_t)first / 4 % 4) : 0;
  const Segment s = segment(vocab + shift, blocks, rank);
  const float* src = first - shift + s.begin;
  const bool wide_in = (uintptr_t)src % 16 == 0;
  const int skip = shift - s.begin;           // (positive in the first block of the row only)
  float4 x[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = p * STEP + tid * 4;
    x[p] = load4(src + i, s.n - i, wide_in, -INFINITY, skip - i);
  }
  // The segment that a block of the next round will read is on its way to L2
  // while this one computes and writes.
  const unsigned ahead = blockIdx.x + at_once;
  if (ahead < gridDim.x && tid == 0 && s.n >= 12) {   // (s.n - 8: whatever the rows' shifts, within the row)
    const uintptr_t at = ((uintptr_t)(logits + (ahead / blocks) * row_stride + s.begin) + 15) & ~(uintptr_t)15;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"((s.n - 8) / 4 * 16));
  }
  float m = -INFINITY;                        // a NaN or +infinity in the row makes this one
#pragma unroll
  for (int p = 0; p < PASSES; ++p) m = max_nan(m, max_nan(max_nan(x[p].x, x[p].y), max_nan(x[p].z, x[p].w)));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(FULL, m, o));
  if (tid % 32 == 0) wmax[tid / 32] = m;
  __syncthreads();
  m = wmax[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) m = max_nan(m, wmax[w]);
  float sum = 0.f;
  int at = 0x7fffffff;                        // greedy: the maximum's lowest index
  if (scale > 0.f) {
    const float base = m == -INFINITY ? 0.f : m;   // a segment of nothing but -infinity: zeros
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      x[p].x = exp2f((x[p].x - base) * scale);
      x[p].y = exp2f((x[p].y - base) * scale);
      x[p].z = exp2f((x[p].z - base) * scale);
      x[p].w = exp2f((x[p].w - base) * scale);
      sum += (x[p].x + x[p].y) + (x[p].z + x[p].w);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    if (tid % 32 == 0) wsum[tid / 32] = sum;
  } else {
#pragma unroll
    for (int p = PASSES - 1; p >= 0; --p) {
      const int i = s.begin - shift + p * STEP + tid * 4;
      at = x[p].x == m ? i : x[p].y == m ? i + 1 : x[p].z == m ? i + 2 : x[p].w == m ? i + 3 : at;
    }
    at = __reduce_min_sync(FULL, at);
    if (tid % 32 == 0) wat[tid / 32] = at;
  }
  cl.barrier_wait();
  __syncthreads();
  if (tid < blocks) {                         // this block's totals into every block's table
    sum = 0.f;
    at = 0x7fffffff;
    for (int w = 0; w < NW; ++w)
      if (scale > 0.f) sum += wsum[w];
      else at = min(at, wat[w]);
    auto* p = cl.map_shared_rank(&parts[rank], tid);
    p->m = m;
    p->sum = sum;
    p->at = at;
  }
  cl.sync();
  float top = parts[0].m;
  for (int r = 1; r < blocks; ++r) top = max_nan(top, parts[r].m);
  float* dst = probs + row * vocab - shift + s.begin;
  const bool wide_out = (uintptr_t)dst % 16 == 0;
  const int base_at = s.begin - shift;
  float f = 0.f;                              // from the block's own maximum and sum to the row's
  if (!(top < INFINITY)) {
    f = NAN;
  } else if (scale > 0.f && top > -INFINITY) {
    float total = 0.f;
    for (int r = 0; r < blocks; ++r) total += parts[r].sum * exp2f((parts[r].m - top) * scale);
    f = exp2f((m - top) * scale) / total;
  }
  int pick = 0x7fffffff;
  if (scale == 0.f && top > -INFINITY)
    for (int r = 0; r < blocks; ++r)
      if (parts[r].m == top) pick = min(pick, parts[r].at);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = p * STEP + tid * 4;
    float4 v;
    if (scale > 0.f && f == f) v = make_float4(x[p].x * f, x[p].y * f, x[p].z * f, x[p].w * f);
    else v = make_float4(f, f, f, f);
    if (f == f && pick >= base_at + i && pick < base_at + i + 4) {
      v.x = pick == base_at + i;
      v.y = pick == base_at + i + 1;
      v.z = pick == base_at + i + 2;
      v.w = pick == base_at + i + 3;
    }
    if (wide_out && i + 4 <= s.n && i >= skip) {
      *reinterpret_cast<float4*>(dst + i) = v;
    } else {
      if (i < s.n && i >= skip) dst[i] = v.x;
      if (i + 1 < s.n && i + 1 >= skip) dst[i + 1] = v.y;
      if (i + 2 < s.n && i + 2 >= skip) dst[i + 2] = v.z;
      if (i + 3 < s.n && i + 3 >= skip) dst[i + 3] = v.w;
    }
  }
}

// A weight as a whole number of 2^-40: sums of those do not depend on their
// order, so any split of the row draws the same token.  In two 20-bit parts, so
// that a group's sums fit 32 bits and a warp adds them in one instruction.  Both
// parts come by adding 2^23, whose mantissa then holds the whole number:
// rounded down the first time (scaling by 2^20 and the remainder are exact), to
// the nearest the second (conversions run at a quarter of the rate).
struct Mass {
  uint32_t hi, lo;
};
constexpr uint32_t BIAS = 0x4b000000u;            // the bits of 2^23
__device__ __forceinline__ Mass biased_mass(float w) {
  const float x = __saturatef(w) * 1048576.f;    // (0 for a NaN)
  const float h = __fadd_rz(x, 8388608.f);
  return {__float_as_uint(h), __float_as_uint(fmaf(x - (h - 8388608.f), 1048576.f, 8388608.f))};
}
__device__ __forceinline__ unsigned long long whole_mass(Mass m) { return ((unsigned long long)m.hi << 20) + m.lo; }
__device__ __forceinline__ unsigned long long mass(float w) {
  const Mass m = biased_mass(w);
  return whole_mass({m.hi - BIAS, m.lo - BIAS});
}
__device__ __forceinline__ Mass mass4(float4 w) {
  const Mass a = biased_mass(w.x), b = biased_mass(w.y), c = biased_mass(w.z), d = biased_mass(w.w);
  return {a.hi + b.hi + c.hi + d.hi - 4 * BIAS, a.lo + b.lo + c.lo + d.lo - 4 * BIAS};
}

struct VerifyArgs {
  int drafts, vocab, wide;
  const float *target, *draft;
  const int *tok, *count;
  const float *u, *r;
  int *out, *accepted;
};

template <int PASSES>
__global__ void __launch_bounds__(NT, PASSES <= 10 ? 2 : 1) k_verify(VerifyArgs a) {
  __shared__ unsigned long long sums[PASSES * NW], totals[FEW];
  __shared__ int n_acc, n_all;
  await_stream();
  allow_next();
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();
  const int blocks = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int b = blockIdx.x / blocks, V = a.vocab;
  const float* target = a.target + (size_t)b * (a.drafts + 1) * V;
  const float* draft = a.draft ? a.draft + (size_t)b * a.drafts * V : nullptr;
  const int* tok = a.tok + (size_t)b * a.drafts;
  if (warp == 0) {                            // every block of the cluster decides alike
    const int given = a.count ? a.count[b] : a.drafts, n = min(max(given, 0), a.drafts);
    int first = n;
    for (int i0 = 0; i0 < a.drafts; i0 += 32) {
      const int i = i0 + lane;                // (tokens and numbers of places past n are read, in their rows)
      const int x = i < a.drafts ? tok[i] : -1;
      const float u = i < a.drafts ? a.u[(size_t)b * a.drafts + i] : 0.f;
      bool ok = x >= 0 && x < V;
      if (ok) {
        const double q = draft ? draft[(size_t)i * V + x] : 1.0;   // products of 24-bit factors are exact in 53
        ok = (double)u * q < (double)target[(size_t)i * V + x];
      }
      const unsigned no = __ballot_sync(FULL, i < n && !ok);
      if (no) first = i0 + __ffs(no) - 1;
      if (no || i0 + 32 >= n) break;
    }
    if (lane == 0) {
      n_acc = first;
      n_all = n;
    }
  }
  __syncthreads();
  const int acc = n_acc, n = n_all;
  const bool refused = acc < n;
  const Segment s = segment(V, blocks, rank);
  const float* trow = target + (size_t)acc * V + s.begin;
  const float* drow = refused && draft ? draft + (size_t)acc * V + s.begin : nullptr;
  const int gone = refused && !draft ? tok[acc] - s.begin : -1;   // a certain draft's place in this segment
  cl.barrier_wait();
  unsigned long long total = 0, before = 0;
  for (int whole = refused ? 0 : 1; whole < 2; ++whole) {
    const float* less = whole ? nullptr : drow;
    auto spared = [&](float4 w, float4 d, int i) {   // weights at element i of the segment
      const int at = whole ? -1 : gone - i;
      return make_float4(w.x - d.x - (at == 0), w.y - d.y - (at == 1), w.z - d.z - (at == 2), w.w - d.w - (at == 3));
    };
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 w[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = p * STEP + tid * 4;
      w[p] = load4(trow + i, s.n - i, a.wide, 0.f);
    }
    if (less) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = p * STEP + tid * 4;
        w[p] = spared(w[p], load4(less + i, s.n - i, a.wide, 0.f), i);
      }
    } else {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) w[p] = spared(w[p], none, p * STEP + tid * 4);
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const Mass m = mass4(w[p]);
      const Mass g = {__reduce_add_sync(FULL, m.hi), __reduce_add_sync(FULL, m.lo)};
      if (lane == 0) sums[p * NW + warp] = whole_mass(g);
    }
    __syncthreads();
    if (warp == 0) {
      unsigned long long m = 0;
      for (int k = lane; k < PASSES * NW; k += 32) m += sums[k];
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
      const float rv = a.r[b];
      // floor(r 2^24), 0 for a NaN
      const unsigned long long U = rv > 0.f ? (unsigned long long)fminf(floorf(rv * 16777216.f), 16777215.f) : 0ull;
      unsigned long long at = __umul64hi(total, U << 40);         // floor(total U / 2^24)
      const unsigned long long mine = totals[rank];
      if (at >= before && at - before < mine) {                    // the token lies in this segment
        at -= before;
        int k = 0;
        for (;; k += 32) {                                         // its group of 128: every warp finds it
          const unsigned long long v = k + lane < PASSES * NW ? sums[k + lane] : 0ull;
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
        if (warp == k % NW) {                                      // and the one that holds it the token
          const int i = k / NW * STEP + tid * 4;
          const float4 g = spared(load4(trow + i, s.n - i, a.wide, 0.f), less ? load4(less + i, s.n - i, a.wide, 0.f) : none, i);
          const unsigned long long m[4] = {mass(g.x), mass(g.y), mass(g.z), mass(g.w)};
          const unsigned long long v = m[0] + m[1] + m[2] + m[3];
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

// What a thread of the host knows of the device that it launches on.
struct Known {
  int dev = -1, sms = 0;
  struct {
    const void* kernel;
    bool ok;
  } wide[16] = {};                            // whether 16 blocks of a kernel can run as one cluster
  int n = 0;
};
thread_local Known known;

int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

int fail_cuda(const char* what, cudaError_t e) {
  cudaGetLastError();   // reported here: not to the caller's next question
  allowed = {};
  known = {};
  char buf[224];
  snprintf(buf, sizeof(buf), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  return fail(MK_ERR_CUDA, buf);
}

// The instance whose registers hold a segment: f(passes) with one of a few.
template <class F>
cudaError_t with_passes(int vocab, int cluster, F&& f) {
  const int n = passes_of(vocab, cluster);
  if (n <= 2) return f(std::integral_constant<int, 2>());
  if (n <= 3) return f(std::integral_constant<int, 3>());
  if (n <= 4) return f(std::integral_constant<int, 4>());
  if (n <= 6) return f(std::integral_constant<int, 6>());
  if (n <= 8) return f(std::integral_constant<int, 8>());
  if (n <= 10) return f(std::integral_constant<int, 10>());
  if (n <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, MAX_PASSES>());
}

cudaError_t know_device() {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev == known.dev) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  known = {};
  known.dev = dev;
  known.sms = sms;
  return cudaSuccess;
}

// Allows a kernel clusters of 16 and asks whether the device has room for one.
cudaError_t wide_cluster(const void* kernel, bool* ok) {
  cudaError_t e = allow(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  for (const auto& w : known.wide)
    if (w.kernel == kernel) {
      *ok = w.ok;
      return cudaSuccess;
    }
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = FEW;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = FEW;
  cfg.blockDim = NT;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
  if (e != cudaSuccess) {                     // no room is an answer too
    cudaGetLastError();
    n = 0;
  }
  *ok = n > 0;
  known.wide[known.n++ % 16] = {kernel, *ok};
  return cudaSuccess;
}

// Launches rows of (at most) `vocab` elements: kernel(passes) is the instance,
// launch(instance, cluster) its call.
template <class K, class L>
cudaError_t launch_rows(int vocab, int limit, long long rows, K&& kernel, L&& launch) {
  cudaError_t e = know_device();
  if (e != cudaSuccess) return e;
  int c = cluster_of(limit, rows, known.sms, FEW);
  if (c > MANY) {
    bool ok = false;
    e = with_passes(vocab, c, [&](auto n) { return wide_cluster((const void*)kernel(n), &ok); });
    if (e != cudaSuccess) return e;
    if (!ok) c = cluster_of(limit, rows, known.sms, MANY);
  }
  return with_passes(vocab, c, [&](auto n) { return launch(kernel(n), c); });
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
  if (rows == 0) return MK_OK;
  if (!aligned(logits, 4) || !aligned(probs, 4)) return fail(MK_ERR_INVALID, "mk_probs: a buffer is NULL or not aligned to its type");
  {
    const char *l0 = (const char*)logits, *p0 = (const char*)probs;
    const char* l1 = l0 + 4 * ((size_t)(rows - 1) * row_stride + vocab);
    const char* p1 = p0 + 4 * (size_t)rows * vocab;
    if (l0 < p1 && p0 < l1 && !(l0 == p0 && row_stride == vocab))
      return fail(MK_ERR_INVALID, "mk_probs: probs overlaps the logits in other places than their own");
  }
  const float scale = temperature > 0.f ? fminf(1.4426950408889634f / temperature, 3.4e38f) : 0.f;   // log2(e) / T
  const int shiftable = vocab + 3 <= MAX_VOCAB;   // (at the limit itself there is no room for a shift)
  const cudaError_t e = launch_rows(
      vocab + 3 * shiftable, vocab, rows, [](auto n) { return k_probs<n.value>; },
      [&](auto k, int c) {
        return launch_kernel(k, dim3((unsigned)(rows * c)), NT, 0, c, (cudaStream_t)stream, logits, vocab, row_stride, scale,
                             probs, shiftable, blocks_at_once(known.sms));
      });
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_probs", e);
}

int mk_verify(int batch, int max_draft, int vocab, const float* target, const float* draft, const int* drafts,
              const int* n_draft, const float* u, const float* r, int* tokens, int* accepted, mk_stream stream) {
  using namespace mk;
  if (batch < 0 || max_draft < 0 || vocab < 1) return fail(MK_ERR_INVALID, "mk_verify: batch, max_draft or vocab");
  if (vocab > MAX_VOCAB) return fail(MK_ERR_UNSUPPORTED, "mk_verify: vocab above 393216");
  if (batch > (1 << 20) || max_draft > (1 << 20)) return fail(MK_ERR_UNSUPPORTED, "mk_verify: batch or max_draft above 2^20");
  if (batch == 0) return MK_OK;
  if (!aligned(target, 4) || !aligned(r, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) ||
      (max_draft && (!aligned(drafts, 4) || !aligned(u, 4))) || (draft && !aligned(draft, 4)) ||
      (n_draft && !aligned(n_draft, 4)))
    return fail(MK_ERR_INVALID, "mk_verify: a buffer is NULL or not aligned to its type");
  {
    const size_t b = 4 * (size_t)batch, k = max_draft, v = vocab;
    const struct {
      const void* at;
      size_t n;
    } in[] = {{target, b * (k + 1) * v}, {draft, draft ? b * k * v : 0}, {drafts, b * k}, {n_draft, n_draft ? b : 0},
              {u, b * k}, {r, b}};
    bool bad = meet(tokens, b * (k + 1), accepted, b);
    for (const auto& i : in)      // (one request's tokens may take its drafts' place: each draft stays where it is)
      bad |= i.n && (meet(accepted, b, i.at, i.n) ||
                     (meet(tokens, b * (k + 1), i.at, i.n) && !(i.at == drafts && tokens == drafts && batch == 1)));
    if (bad) return fail(MK_ERR_INVALID, "mk_verify: tokens or accepted overlap another buffer");
  }
  VerifyArgs a = {max_draft, vocab, 0, target, draft, drafts, n_draft, u, r, tokens, accepted};
  a.wide = aligned(target, 16) && (!draft || aligned(draft, 16)) && vocab % 4 == 0;
  const cudaError_t e = launch_rows(
      vocab, vocab, batch, [](auto n) { return k_verify<n.value>; },
      [&](auto k, int c) { return launch_kernel(k, dim3((unsigned)(batch * c)), NT, 0, c, (cudaStream_t)stream, a); });
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_verify", e);
}

}  // extern "C"
