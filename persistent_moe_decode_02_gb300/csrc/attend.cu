// Attention of a chunk's rows over the paged cache.
//
// out = sum_s p_s v_s / sum_s p_s, p_s = exp(q . k_s / sqrt(d) - m), over the
// positions s <= the row's own, with the running maximum m and sum kept in
// fp32 (one pass over the cache).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "chunk.h"

namespace mk {
namespace {

constexpr int NT = 128;

// One block per (new row, KV head): the G heads of the row over all pages.
template <int D, bool E4M3>
__global__ void __launch_bounds__(NT) k_attend(ChunkView c, const __nv_bfloat16* q, const void* pool, __nv_bfloat16* out) {
  __shared__ float qs[8][D], part[8][8][PAGE], p[8][PAGE], corr[8], sum_s[8], max_s[8];
  const int row = blockIdx.x, g = blockIdx.y, G = c.G, tid = threadIdx.x;
  int lo = 0, hi = c.batch - 1;                  // the request of this row: the last one that starts at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (c.reqs[mid].row0 <= row) lo = mid;
    else hi = mid - 1;
  }
  const ChunkReq r = c.reqs[lo];
  const int pos = r.seq + row - r.row0;
  const float scale = 1.4426950408889634f * rsqrtf((float)D);   // log2(e) / sqrt(d): exponentials in base 2
  for (int x = tid; x < G * D; x += NT)
    qs[x / D][x % D] = __bfloat162float(q[((size_t)row * c.nq + (size_t)g * G + x / D) * D + x % D]) * scale;
  if (tid < 8) {
    max_s[tid] = -INFINITY;
    sum_s[tid] = 0.f;
  }
  float acc[8] = {};
  __syncthreads();
  auto value = [&](size_t block, int i, int s) -> float {
    if (E4M3) {
      const uint8_t* b = reinterpret_cast<const uint8_t*>(pool) + block * (D + 1) * PAGE;
      const __half_raw h = __nv_cvt_fp8_to_halfraw(b[(size_t)i * PAGE + s], __NV_E4M3);
      return ldexpf(__half2float(__half(h)), (int)b[(size_t)D * PAGE + s] - 127);
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(pool)[(block * D + i) * PAGE + s]);
  };
  for (int j = 0; j <= pos / PAGE; ++j) {
    const size_t block = ((size_t)c.pt[r.pt + j] * c.nkv + g) * 2;
    const int n = min(PAGE, pos + 1 - j * PAGE);
    {
      const int s = tid % PAGE, w = tid / PAGE;
      float dot[8] = {};
      if (s < n)
        for (int i = w * (D / 8); i < (w + 1) * (D / 8); ++i) {
          const float k = value(block, i, s);
#pragma unroll
          for (int h = 0; h < 8; ++h)
            if (h < G) dot[h] += qs[h][i] * k;
        }
#pragma unroll
      for (int h = 0; h < 8; ++h) part[w][h][s] = dot[h];
    }
    __syncthreads();
    if (tid < G) {
      float x[PAGE], m = max_s[tid];
      for (int s = 0; s < n; ++s) {
        x[s] = 0.f;
        for (int w = 0; w < 8; ++w) x[s] += part[w][tid][s];
        m = fmaxf(m, x[s]);
      }
      const float f = exp2f(max_s[tid] - m);
      float sum = sum_s[tid] * f;
      for (int s = 0; s < PAGE; ++s) {
        p[tid][s] = s < n ? exp2f(x[s] - m) : 0.f;
        sum += p[tid][s];
      }
      corr[tid] = f;
      sum_s[tid] = sum;
      max_s[tid] = m;
    }
    __syncthreads();
    if (tid < D) {
      for (int h = 0; h < G; ++h) acc[h] *= corr[h];
      for (int s = 0; s < n; ++s) {
        const float v = value(block + 1, tid, s);
        for (int h = 0; h < G; ++h) acc[h] += p[h][s] * v;
      }
    }
  }
  __syncthreads();
  if (tid < D)
    for (int h = 0; h < G; ++h)
      out[((size_t)row * c.nq + (size_t)g * G + h) * D + tid] = __float2bfloat16_rn(acc[h] / sum_s[h]);
}

}  // namespace

cudaError_t launch_attend(const ChunkView& c, bool e4m3, const void* q, const void* pool, void* out, cudaStream_t st) {
  const dim3 grid(c.rows, c.nkv);
  const auto qi = (const __nv_bfloat16*)q;
  const auto o = (__nv_bfloat16*)out;
  if (c.d == 64) {
    if (e4m3) k_attend<64, true><<<grid, NT, 0, st>>>(c, qi, pool, o);
    else k_attend<64, false><<<grid, NT, 0, st>>>(c, qi, pool, o);
  } else {
    if (e4m3) k_attend<128, true><<<grid, NT, 0, st>>>(c, qi, pool, o);
    else k_attend<128, false><<<grid, NT, 0, st>>>(c, qi, pool, o);
  }
  return cudaGetLastError();
}

}  // namespace mk
