// The paged cache's own operators: the rows of a chunk into its pages (rotary
// embedding, rounding or quantising, the pages' transposed layout) and back.
//
// Both move bytes and compute next to nothing, so device memory bounds the
// large calls and launch latency the small ones.  A block takes one page of
// one KV head: its 16 tokens x 2 vectors are transposed through shared memory,
// so global memory sees whole rows of a token on one side and the page's
// contiguous block on the other.  8000 rows of 32 query and 4 KV heads of 128
// enter bf16 pages in 27.5 us (6.0 TB/s, 0.89 of a copy's rate), 8144 fp32 rows
// 8-bit pages in 43.6 us (5.5 TB/s); 65000 tokens come back from bf16 pages in
// 42.0 us (6.3 TB/s), 55395 from 8 bits in 27.4 us (6.2 TB/s).  A few rows take
// 1.5 to 3.5 us, a launch and its chain of loads.  Grids hold the pages that
// are there: with the longest request's for each, a ragged batch (14700 tokens
// and three short ones) took 16.4 us to read, 11 so.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "chunk.h"
#include "eights.cuh"

namespace mk {
namespace {

constexpr int NT = 128;          // threads of a block

// 8 consecutive elements as they lie, and as fp32.
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  return *reinterpret_cast<const Raw8<T>*>(p);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// (cos, sin) of 8 dimensions of a row.
struct Turn {
  float4 cs[4];
};
// Two 8-element pieces of one head, half a head apart, rotated.
__device__ __forceinline__ void rotate8(const Turn& t, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 c = t.cs[j];
    const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
    a[2 * j] = a0 * c.x - b0 * c.y;
    b[2 * j] = b0 * c.x + a0 * c.y;
    a[2 * j + 1] = a1 * c.z - b1 * c.w;
    b[2 * j + 1] = b1 * c.z + a1 * c.w;
  }
}

// cos and sin of position * theta^(-2i/d), the angle and its functions in 64
// bits: in 32 an angle near 2^18 would be off by 2^-7.  Once for a chunk, read
// by every layer's append.  A thread turns one dimension pair through
// ROPE_RUN positions by the angle between neighbours, which costs 4 operations
// a position instead of about 100 (errors add up to less than 2^-48).
constexpr int ROPE_RUN = 16;
struct Freq {
  double of[64];                                 // theta^(-2i/d)
};
__global__ void k_chunk_rope(const ChunkReq* reqs, int half, const __grid_constant__ Freq freq, float2* tab) {
  await_stream();
  allow_next();
  const ChunkReq r = reqs[blockIdx.y];
  const long long n = (long long)((r.nnew + ROPE_RUN - 1) / ROPE_RUN) * half;
  for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (long long)gridDim.x * blockDim.x) {
    const int t0 = (int)(x / half) * ROPE_RUN, i = (int)(x % half);
    double s, c, ds, dc;
    sincos((double)(r.seq + t0) * freq.of[i], &s, &c);
    sincos(freq.of[i], &ds, &dc);
    for (int t = t0; t < min(t0 + ROPE_RUN, r.nnew); ++t) {
      tab[(size_t)(r.row0 + t) * half + i] = make_float2((float)c, (float)s);
      const double c1 = c * dc - s * ds;
      s = s * dc + c * ds;
      c = c1;
    }
  }
}

// Append: grid (pages that receive rows, KV heads).  A thread has one
// token and the same 8 dimensions of either half of a head: its angles are read
// once for all heads, whose loads do not wait for one another.
template <int D, bool E4M3, class T>
__global__ void __launch_bounds__(NT) k_append(ChunkView c, const T* qkv, long long row_stride, void* pool,
                                               __nv_bfloat16* q) {
  constexpr int LD = D + 1;                      // odd pitch: columns of the transpose fall into different banks
  constexpr int C = D / 16;                      // threads of a token and head
  constexpr int HS = NT / (PAGE * C);            // heads at a time
  constexpr int AHEAD = 8 / sizeof(T);           // and in flight for each thread: 128 bytes
  __shared__ float kv[2][PAGE][LD];
  __shared__ int exps[2][PAGE];
  const AppendPage at = c.appends[blockIdx.x];   // the chunk's tables: no kernel writes them
  if (stale(c)) return;
  allow_next();
  const int g = blockIdx.y, G = c.G, tid = threadIdx.x, n = at.n, slot0 = at.slot, row = at.row;
  const int i = tid % C * 8, t = tid / C % PAGE, hs = tid / (C * PAGE);
  const size_t block = ((size_t)at.page * c.nkv + g) * 2;   // the page's K block, in blocks
  await_stream();
  if (t < n) {
    const T* src = qkv + (size_t)(row + t) * row_stride + (size_t)g * (G + 2) * D + i;
    Turn turn;
    if (c.rope) {
      const float4* cs = reinterpret_cast<const float4*>(c.rope + (size_t)(row + t) * (D / 2) + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) turn.cs[e] = cs[e];
    }
    __nv_bfloat16* dst = q + ((size_t)(row + t) * c.nq + (size_t)g * G) * D + i;
    // A load does not pass a store that might meet it, so AHEAD heads' loads
    // come before their stores.
    for (int h0 = hs; h0 < G; h0 += AHEAD * HS) {
      Raw8<T> lo[AHEAD], hi[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (h0 + k * HS < G) {
          lo[k] = load8(src + (size_t)(h0 + k * HS) * D);
          hi[k] = load8(src + (size_t)(h0 + k * HS) * D + D / 2);
        }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (h0 + k * HS < G) {
          float a[8], b[8];
          unpack8(lo[k], a);
          unpack8(hi[k], b);
          if (c.rope) rotate8(turn, a, b);
          *reinterpret_cast<uint4*>(dst + (size_t)(h0 + k * HS) * D) = pack8(a);
          *reinterpret_cast<uint4*>(dst + (size_t)(h0 + k * HS) * D + D / 2) = pack8(b);
        }
    }
    if (hs == 0) {
      float a[8], b[8], v[8], w[8];
      unpack8(load8(src + (size_t)G * D), a);
      unpack8(load8(src + (size_t)G * D + D / 2), b);
      unpack8(load8(src + (size_t)(G + 1) * D), v);
      unpack8(load8(src + (size_t)(G + 1) * D + D / 2), w);
      if (c.rope) rotate8(turn, a, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        kv[0][t][i + e] = a[e];
        kv[0][t][i + D / 2 + e] = b[e];
        kv[1][t][i + e] = v[e];
        kv[1][t][i + D / 2 + e] = w[e];
      }
    }
  }
  __syncthreads();
  if constexpr (E4M3) {
    // 4 threads take one vector's largest magnitude
    const int w = tid / 4, tw = w % PAGE, which = w / PAGE;
    float m = 0.f;
    if (tw < n)
      for (int x = tid % 4; x < D; x += 4) m = fmaxf(m, fabsf(kv[which][tw][x]));   // a NaN leaves the others' maximum
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (tid % 4 == 0) exps[which][tw] = scale_exp(m);
    __syncthreads();
    uint8_t* out = reinterpret_cast<uint8_t*>(pool) + block * (D + 1) * PAGE;
    for (int x = tid; x < 2 * (D + 1); x += NT) {
      const int which2 = x / (D + 1), d = x % (D + 1);
      uint8_t* o = out + (size_t)x * PAGE + slot0;
      uint32_t b[4];
#pragma unroll
      for (int w4 = 0; w4 < 4; ++w4) {
        b[w4] = 0;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int t2 = w4 * 4 + e;
          const int k0 = exps[which2][t2], k1 = exps[which2][t2 + 1];
          uint32_t two;
          if (d == D) {
            two = (uint32_t)(k0 + 127) | (uint32_t)(k1 + 127) << 8;
          } else {
            // by 2^-k in two factors: 2^127 and beyond is no factor of its own
            const float v0 = kv[which2][t2][d] * pow2(-(k0 >> 1)) * pow2(-(k0 - (k0 >> 1)));
            const float v1 = kv[which2][t2 + 1][d] * pow2(-(k1 >> 1)) * pow2(-(k1 - (k1 >> 1)));
            two = __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
          }
          b[w4] |= two << (8 * e);
        }
      }
      if (n == PAGE) {
        *reinterpret_cast<uint4*>(o) = make_uint4(b[0], b[1], b[2], b[3]);
      } else {
#pragma unroll
        for (int t2 = 0; t2 < PAGE; ++t2)
          if (t2 < n) o[t2] = (uint8_t)(b[t2 / 4] >> (t2 % 4 * 8));   // only the new tokens' slots
      }
    }
  } else {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(pool) + block * D * PAGE;
    for (int x = tid; x < 2 * D; x += NT) {
      const int which = x / D, d = x % D;
      __nv_bfloat16* o = out + (size_t)x * PAGE + slot0;
      if (n == PAGE) {
        uint32_t w[8];
#pragma unroll
        for (int t2 = 0; t2 < 8; ++t2) w[t2] = pack2(kv[which][2 * t2][d], kv[which][2 * t2 + 1][d]);
        reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        for (int t2 = 0; t2 < n; ++t2) o[t2] = __float2bfloat16_rn(kv[which][t2][d]);
      }
    }
  }
}

// Read: grid (all requests' pages, KV heads).  A thread has two dimensions of the
// page's 16 tokens.  Codes and scales give the value exactly in fp32; the
// rounding to bf16 changes it only outside bf16's normal range.
template <int D, bool E4M3>
__global__ void __launch_bounds__(NT) k_read(ChunkView c, const void* pool, __nv_bfloat16* out) {
  constexpr int LD = D + 4;                      // words of a token's row: 16-byte rows for the way out
  __shared__ alignas(16) uint32_t buf[PAGE][LD];
  if (stale(c)) return;
  allow_next();
  int lo = 0, hi = c.batch - 1;                  // the request of this page: the last one that starts at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (__ldg(&c.reqs[mid].page0) <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const ChunkReq r = c.reqs[lo];
  const int g = blockIdx.y, j = blockIdx.x - r.page0, tid = threadIdx.x, n = min(PAGE, r.seq + r.nnew - j * PAGE);
  const size_t block = ((size_t)__ldg(c.pt + r.pt + j) * c.nkv + g) * 2;
  await_stream();
  for (int x = tid; x < D; x += NT) {            // dimensions 2x and 2x + 1 of K, then V
    if constexpr (E4M3) {
      const uint8_t* b = reinterpret_cast<const uint8_t*>(pool) + (block + x / (D / 2)) * (D + 1) * PAGE;
      const uint4* rows = reinterpret_cast<const uint4*>(b) + x % (D / 2) * 2;
      const uint4 lo4 = rows[0], hi4 = rows[1], ex4 = reinterpret_cast<const uint4*>(b)[D];
      const uint32_t lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w},
                     ex[4] = {ex4.x, ex4.y, ex4.z, ex4.w};
#pragma unroll
      for (int t = 0; t < PAGE; t += 2) {
        const int at = t % 4 * 8;
        const __half2 l = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(lo[t / 4] >> at), __NV_E4M3));
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(hi[t / 4] >> at), __NV_E4M3));
        const uint32_t e0 = ex[t / 4] >> at & 0xff, e1 = ex[t / 4] >> (at + 8) & 0xff;
        const float s0 = e0 ? __uint_as_float(e0 << 23) : __uint_as_float(0x400000u);   // 2^(e - 127)
        const float s1 = e1 ? __uint_as_float(e1 << 23) : __uint_as_float(0x400000u);
        buf[t][x] = pack2(__low2float(l) * s0, __low2float(h) * s0);
        buf[t + 1][x] = pack2(__high2float(l) * s1, __high2float(h) * s1);
      }
    } else {
      const uint4* rows = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(pool) + block * D * PAGE) +
                          (size_t)x * 4;
      const uint4 v[4] = {rows[0], rows[1], rows[2], rows[3]};
      const uint32_t lo[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
      const uint32_t hi[8] = {v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        buf[2 * t][x] = __byte_perm(lo[t], hi[t], 0x5410);
        buf[2 * t + 1][x] = __byte_perm(lo[t], hi[t], 0x7632);
      }
    }
  }
  __syncthreads();
  const size_t row0 = (size_t)r.tok0 + (size_t)j * PAGE;
  for (int x = tid; x < n * (D / 4); x += NT) {
    const int i = x % (D / 4), t = x / (D / 4);
    *reinterpret_cast<uint4*>(out + ((row0 + t) * c.nkv + g) * 2 * D + i * 8) = *reinterpret_cast<const uint4*>(&buf[t][i * 4]);
  }
}

}  // namespace

cudaError_t launch_chunk_rope(const ChunkView& c, double theta, float2* tab, int max_new, cudaStream_t st) {
  const int half = c.d / 2;
  const long long most = ((long long)max_new + ROPE_RUN - 1) / ROPE_RUN * half;
  const int blocks = (int)(most < 256 * 1024 ? (most + 255) / 256 : 1024);
  Freq freq = {};
  for (int i = 0; i < half; ++i) freq.of[i] = pow(theta, -2.0 * i / c.d);
  return launch_kernel(k_chunk_rope, dim3(blocks, c.batch), 256, 0, 1, st, c.reqs, half, freq, tab);
}

namespace {

template <int D, bool E4M3>
cudaError_t append(const ChunkView& c, bool f32, const void* qkv, long long row_stride, void* pool, void* q, dim3 grid,
                   cudaStream_t st) {
  const auto o = (__nv_bfloat16*)q;
  if (f32) return launch_kernel(k_append<D, E4M3, float>, grid, NT, 0, 1, st, c, (const float*)qkv, row_stride, pool, o);
  return launch_kernel(k_append<D, E4M3, __nv_bfloat16>, grid, NT, 0, 1, st, c, (const __nv_bfloat16*)qkv, row_stride,
                       pool, o);
}

}  // namespace

cudaError_t launch_append(const ChunkView& c, bool e4m3, bool f32, const void* qkv, long long row_stride, void* pool,
                          void* q, cudaStream_t st) {
  const dim3 grid(c.nappends, c.nkv);
  if (c.d == 64)
    return e4m3 ? append<64, true>(c, f32, qkv, row_stride, pool, q, grid, st)
                : append<64, false>(c, f32, qkv, row_stride, pool, q, grid, st);
  return e4m3 ? append<128, true>(c, f32, qkv, row_stride, pool, q, grid, st)
              : append<128, false>(c, f32, qkv, row_stride, pool, q, grid, st);
}

cudaError_t launch_read(const ChunkView& c, bool e4m3, const void* pool, void* out, cudaStream_t st) {
  const dim3 grid(c.npages, c.nkv);
  const auto k = c.d == 64 ? (e4m3 ? k_read<64, true> : k_read<64, false>) : (e4m3 ? k_read<128, true> : k_read<128, false>);
  return launch_kernel(k, grid, NT, 0, 1, st, c, pool, (__nv_bfloat16*)out);
}

}  // namespace mk
