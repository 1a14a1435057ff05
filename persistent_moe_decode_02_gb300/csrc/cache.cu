// The paged cache's own operators: the rows of a chunk into its pages (rotary
// embedding, rounding or quantising, the pages' transposed layout) and back.
//
// Both move bytes and compute next to nothing, so device memory bounds the
// large calls and launch latency the small ones.  A block takes one page of
// one KV head: its 16 tokens x 2 vectors are transposed through shared memory,
// so global memory sees whole rows of a token on one side and the page's
// contiguous block on the other.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "chunk.h"

namespace mk {
namespace {

constexpr int NT = 128;          // threads of a block

// 8 consecutive elements as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// Two 8-element pieces of one head, half a head apart, rotated at row `row`.
template <int D>
__device__ __forceinline__ void rotate8(const float2* rope, int row, int i, float (&a)[8], float (&b)[8]) {
  if (!rope) return;
  const float4* cs = reinterpret_cast<const float4*>(rope + (size_t)row * (D / 2) + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 t = __ldg(cs + j);   // (cos, sin) of two dimensions
    const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
    a[2 * j] = a0 * t.x - b0 * t.y;
    b[2 * j] = b0 * t.x + a0 * t.y;
    a[2 * j + 1] = a1 * t.z - b1 * t.w;
    b[2 * j + 1] = b1 * t.z + a1 * t.w;
  }
}

// cos and sin of position * theta^(-2i/d), the angle and its functions in 64
// bits: in 32 an angle near 2^18 would be off by 2^-7.  Once for a chunk, read
// by every layer's append.
__global__ void k_chunk_rope(const ChunkReq* reqs, int half, int d, double theta, float2* tab) {
  const ChunkReq r = reqs[blockIdx.y];
  const long long n = (long long)r.nnew * half;
  for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (long long)gridDim.x * blockDim.x) {
    const int t = (int)(x / half), i = (int)(x % half);
    double s, c;
    sincos((double)(r.seq + t) * pow(theta, -2.0 * i / d), &s, &c);
    tab[(size_t)(r.row0 + t) * half + i] = make_float2((float)c, (float)s);
  }
}

// Smallest k with amax <= 448 * 2^k (448 = 0.875 * 2^9, the largest e4m3
// value), from the bits of amax: exact, no rounding of a logarithm.
__device__ __forceinline__ int scale_exp(float amax) {
  if (amax == 0.f) return -127;
  int e;
  const float m = frexpf(amax, &e);              // amax = m 2^e, m in [0.5, 1)
  if (!isfinite(amax)) return 127;
  const int k = m <= 0.875f ? e - 9 : e - 8;
  return k < -127 ? -127 : k;
}

// A value by 2^-k, exactly or correctly rounded (two factors: 2^127 alone is
// beyond a float's exponent when k is -127 and -k + 127 overflows).
__device__ __forceinline__ float times_pow2(float x, int k) { return ldexpf(x, k); }

// Append: grid (pages that receive rows, KV heads, requests).
template <int D, bool E4M3, class T>
__global__ void __launch_bounds__(NT) k_append(ChunkView c, const T* qkv, long long row_stride, void* pool,
                                               __nv_bfloat16* q) {
  constexpr int LD = D + 1;                      // odd pitch: columns of the transpose fall into different banks
  __shared__ float kv[2][PAGE][LD];
  __shared__ int exps[2][PAGE];
  const ChunkReq r = c.reqs[blockIdx.z];
  const int g = blockIdx.y, G = c.G, tid = threadIdx.x;
  const int j = r.seq / PAGE + blockIdx.x;       // page of the request
  const int p0 = max(j * PAGE, r.seq), p1 = min(j * PAGE + PAGE, r.seq + r.nnew);
  if (p0 >= p1) return;
  const int n = p1 - p0, slot0 = p0 - j * PAGE, row = r.row0 + p0 - r.seq;
  constexpr int C = D / 16;                      // 8-element pieces of half a head
  const T* src = qkv + (size_t)row * row_stride + (size_t)g * (G + 2) * D;
  // queries and keys: a thread takes the pieces at i and i + D / 2 of a head
  for (int x = tid; x < n * (G + 1) * C; x += NT) {
    const int i = x % C * 8, h = x / C % (G + 1), t = x / (C * (G + 1));
    const T* p = src + (size_t)t * row_stride + (size_t)h * D + i;
    float a[8], b[8];
    load8(p, a);
    load8(p + D / 2, b);
    rotate8<D>(c.rope, row + t, i, a, b);
    if (h < G) {
      __nv_bfloat16* o = q + ((size_t)(row + t) * c.nq + (size_t)g * G + h) * D + i;
      *reinterpret_cast<uint4*>(o) = pack8(a);
      *reinterpret_cast<uint4*>(o + D / 2) = pack8(b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        kv[0][t][i + e] = a[e];
        kv[0][t][i + D / 2 + e] = b[e];
      }
    }
  }
  for (int x = tid; x < n * (D / 8); x += NT) {
    const int i = x % (D / 8) * 8, t = x / (D / 8);
    float a[8];
    load8(src + (size_t)t * row_stride + (size_t)(G + 1) * D + i, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) kv[1][t][i + e] = a[e];
  }
  __syncthreads();
  const size_t block = ((size_t)c.pt[r.pt + j] * c.nkv + g) * 2;   // the page's K block, in blocks
  if (E4M3) {
    // 4 threads take one vector's largest magnitude
    const int w = tid / 4, t = w % PAGE, which = w / PAGE;
    float m = 0.f;
    if (t < n)
      for (int i = tid % 4; i < D; i += 4) {
        const float v = fabsf(kv[which][t][i]);
        m = fmaxf(m, v);                         // a NaN leaves the others' maximum
      }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (tid % 4 == 0) exps[which][t] = scale_exp(m);
    __syncthreads();
    uint8_t* out = reinterpret_cast<uint8_t*>(pool) + block * (D + 1) * PAGE;
    for (int x = tid; x < 2 * (D + 1); x += NT) {
      const int which2 = x / (D + 1), i = x % (D + 1);
      uint8_t* o = out + (size_t)x * PAGE + slot0;
      alignas(16) uint8_t b[PAGE];
#pragma unroll
      for (int t2 = 0; t2 < PAGE; ++t2) {
        if (t2 >= n) break;
        const int k = exps[which2][t2];
        b[t2] = i == D ? (uint8_t)(k + 127)
                       : (uint8_t)__nv_cvt_float_to_fp8(times_pow2(kv[which2][t2][i], -k), __NV_SATFINITE, __NV_E4M3);
      }
      if (n == PAGE) {
        *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(b);
      } else {
#pragma unroll
        for (int t2 = 0; t2 < PAGE; ++t2)
          if (t2 < n) o[t2] = b[t2];             // only the new tokens' slots
      }
    }
  } else {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(pool) + block * D * PAGE;
    for (int x = tid; x < 2 * D; x += NT) {
      const int which = x / D, i = x % D;
      __nv_bfloat16* o = out + (size_t)x * PAGE + slot0;
      if (n == PAGE) {
        uint32_t w[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = pack2(kv[which][2 * t][i], kv[which][2 * t + 1][i]);
        reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        for (int t = 0; t < n; ++t) o[t] = __float2bfloat16_rn(kv[which][t][i]);
      }
    }
  }
}

// Read: grid (pages, KV heads, requests).  Codes and scales give the value
// exactly in fp32; the rounding to bf16 changes it only outside bf16's normal
// range.
template <int D, bool E4M3>
__global__ void __launch_bounds__(NT) k_read(ChunkView c, const void* pool, __nv_bfloat16* out) {
  constexpr int LD = 2 * D + 8;                  // 16-byte rows for the way out
  __shared__ alignas(16) __nv_bfloat16 buf[PAGE][LD];
  const ChunkReq r = c.reqs[blockIdx.z];
  const int g = blockIdx.y, j = blockIdx.x, tid = threadIdx.x;
  const int n = min(PAGE, r.seq + r.nnew - j * PAGE);
  if (n <= 0) return;
  const size_t block = ((size_t)c.pt[r.pt + j] * c.nkv + g) * 2;
  for (int x = tid; x < 2 * D; x += NT) {
    if (E4M3) {
      const uint8_t* b = reinterpret_cast<const uint8_t*>(pool) + (block + x / D) * (D + 1) * PAGE;
      alignas(16) uint8_t code[PAGE], ex[PAGE];
      *reinterpret_cast<uint4*>(code) = __ldg(reinterpret_cast<const uint4*>(b + (size_t)(x % D) * PAGE));
      *reinterpret_cast<uint4*>(ex) = __ldg(reinterpret_cast<const uint4*>(b + (size_t)D * PAGE));
#pragma unroll
      for (int t = 0; t < PAGE; ++t) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(code[t], __NV_E4M3);
        buf[t][x] = __float2bfloat16_rn(times_pow2(__half2float(__half(h)), (int)ex[t] - 127));
      }
    } else {
      const uint4* b = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(pool) + block * D * PAGE +
                                                      (size_t)x * PAGE);
      alignas(16) __nv_bfloat16 v[PAGE];
      reinterpret_cast<uint4*>(v)[0] = __ldg(b);
      reinterpret_cast<uint4*>(v)[1] = __ldg(b + 1);
#pragma unroll
      for (int t = 0; t < PAGE; ++t) buf[t][x] = v[t];
    }
  }
  __syncthreads();
  const size_t row0 = (size_t)r.tok0 + (size_t)j * PAGE;
  for (int x = tid; x < n * (D / 4); x += NT) {
    const int i = x % (D / 4) * 8, t = x / (D / 4);
    *reinterpret_cast<uint4*>(out + ((row0 + t) * c.nkv + g) * 2 * D + i) = *reinterpret_cast<const uint4*>(&buf[t][i]);
  }
}

}  // namespace

cudaError_t launch_chunk_rope(const ChunkView& c, double theta, float2* tab, cudaStream_t st) {
  const int half = c.d / 2;
  const long long most = (long long)c.rows * half;
  const int blocks = (int)(most < 256 * 1024 ? (most + 255) / 256 : 1024);
  k_chunk_rope<<<dim3(blocks, c.batch), 256, 0, st>>>(c.reqs, half, c.d, theta, tab);
  return cudaGetLastError();
}

cudaError_t launch_append(const ChunkView& c, bool e4m3, bool f32, const void* qkv, long long row_stride, void* pool,
                          void* q, int max_new_pages, cudaStream_t st) {
  const dim3 grid(max_new_pages, c.nkv, c.batch);
  const auto bf = (const __nv_bfloat16*)qkv;
  const auto fl = (const float*)qkv;
  const auto o = (__nv_bfloat16*)q;
  if (c.d == 64) {
    if (e4m3) f32 ? k_append<64, true><<<grid, NT, 0, st>>>(c, fl, row_stride, pool, o)
                  : k_append<64, true><<<grid, NT, 0, st>>>(c, bf, row_stride, pool, o);
    else f32 ? k_append<64, false><<<grid, NT, 0, st>>>(c, fl, row_stride, pool, o)
             : k_append<64, false><<<grid, NT, 0, st>>>(c, bf, row_stride, pool, o);
  } else {
    if (e4m3) f32 ? k_append<128, true><<<grid, NT, 0, st>>>(c, fl, row_stride, pool, o)
                  : k_append<128, true><<<grid, NT, 0, st>>>(c, bf, row_stride, pool, o);
    else f32 ? k_append<128, false><<<grid, NT, 0, st>>>(c, fl, row_stride, pool, o)
             : k_append<128, false><<<grid, NT, 0, st>>>(c, bf, row_stride, pool, o);
  }
  return cudaGetLastError();
}

cudaError_t launch_read(const ChunkView& c, bool e4m3, const void* pool, void* out, int max_pages, cudaStream_t st) {
  const dim3 grid(max_pages, c.nkv, c.batch);
  const auto o = (__nv_bfloat16*)out;
  if (c.d == 64) {
    if (e4m3) k_read<64, true><<<grid, NT, 0, st>>>(c, pool, o);
    else k_read<64, false><<<grid, NT, 0, st>>>(c, pool, o);
  } else {
    if (e4m3) k_read<128, true><<<grid, NT, 0, st>>>(c, pool, o);
    else k_read<128, false><<<grid, NT, 0, st>>>(c, pool, o);
  }
  return cudaGetLastError();
}

}  // namespace mk
