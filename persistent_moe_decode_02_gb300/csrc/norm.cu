// Root-mean-square norm with the addition in front of it, and rows to 8 bits
// (mk_norm, mk_quantize in include/mk.h).
//
// t = x + sum_j add_j in fp32 (j in order), out = t / sqrt(mean(t^2) + eps) *
// gamma.  Both read each number once, hold it in registers and write each
// result once, so device memory bounds the large calls and launch latency the
// small ones.  8143 rows of 2048 with eight terms to bf16 take 64 us (6.8 TB/s, a
// copy's rate), with one term to 8 bits 32.6 us (5.6 TB/s: nearly half of it is
// written); 196608 rows of 2048 to 8 bits 186 us (6.6 TB/s).  One row takes 2.1
// us, 500 rows of 8192 9.4 us, two rounds of blocks of 1024 threads.
#include <cuda_bf16.h>

#include "eights.cuh"
#include "host.h"
#include "launch.cuh"
#include "mk.h"

namespace mk {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_N = 16384;

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
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// 8 elements of a group whose four threads are neighbours: codes, and the scale
// from the first of them.
__device__ __forceinline__ void store_eights(uint8_t* codes, uint8_t* scale, const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));   // a NaN leaves the others' maximum
  m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
  m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
  const int k = scale_exp(m);
  const Factors s = factors(k);
  if (codes) {
    *reinterpret_cast<uint2*>(codes) =
        make_uint2(codes4(v[0], v[1], v[2], v[3], s.f, s.g), codes4(v[4], v[5], v[6], v[7], s.f, s.g));
    if (threadIdx.x % 4 == 0) *scale = (uint8_t)(k + 127);
  }
}

enum { OUT_NONE = 3 };

struct NormArgs {
  const void* x;
  long long x_stride;            // elements
  const void* add;               // [rows, terms, n]
  const __nv_bfloat16* gamma;
  void *total, *out;
  uint8_t* scales;
  long long rows;
  int n, terms;
  float eps;
};

// A row is the work of blockDim.x threads (a multiple of 32; blockDim.y rows a
// block), 8 elements a thread and pass, AHEAD terms in flight at a time.  Few
// terms: 32 registers and all 2048 threads of an SM (8143 rows of 2048 with one
// term to 8 bits take 32.8 us so, 36.8 with 46 registers).  With fp32 terms and
// blocks of 1024 threads a register is spilled, which is no reason for fewer of
// them: 2000 rows of 8192 with one fp32 term 44.0 us, 52.3 with half the threads.
template <class X, class A, int OUT, int PASSES, int AHEAD, int MAX_NT>
__global__ void __launch_bounds__(MAX_NT, PASSES > 1 ? 1 : (AHEAD == 1 ? 2048 : sizeof(A) == 4 ? 1024 : 1280) / MAX_NT)
    k_norm(const __grid_constant__ NormArgs a) {
  __shared__ float part[MAX_NT / 32];
  allow_next();
  const int tx = threadIdx.x, w0 = threadIdx.y * (blockDim.x / 32), warp = w0 + tx / 32;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const long long r = live ? row : 0;
  float t[PASSES][8];
  await_stream();
  float ss = 0.f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = (p * blockDim.x + tx) * 8;
    if (live && i < a.n) {
      unpack8(load8((const X*)a.x + r * a.x_stride + i), t[p]);
      const A* add = (const A*)a.add + r * a.terms * a.n + i;
      for (int j0 = 0; j0 < a.terms; j0 += AHEAD) {
        Raw8<A> raw[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (j0 + j < a.terms) raw[j] = load8(add + (size_t)(j0 + j) * a.n);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (j0 + j < a.terms) {
            float v[8];
            unpack8(raw[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[p][e] += v[e];
          }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += t[p][e] * t[p][e];
      if (a.total) store8((X*)a.total + r * a.n + i, t[p]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[p][e] = 0.f;
    }
  }
  if constexpr (OUT != OUT_NONE) {
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
    if (tx % 32 == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) ss += part[w0 + w];
    const float inv = 1.f / sqrtf(ss / (float)a.n + a.eps);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = (p * blockDim.x + tx) * 8;
      const bool here = live && i < a.n;
      float g[8], v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = 1.f;
      if (here && a.gamma) unpack8(load8(a.gamma + i), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = t[p][e] * inv * g[e];
      if constexpr (OUT == MK_ROWS_E4M3) {
        store_eights(here ? (uint8_t*)a.out + r * a.n + i : nullptr, a.scales + (r * a.n + i) / GROUP, v);
      } else if constexpr (OUT == MK_ROWS_BF16) {
        if (here) store8((__nv_bfloat16*)a.out + r * a.n + i, v);
      } else if constexpr (OUT == MK_ROWS_F32) {
        if (here) store8((float*)a.out + r * a.n + i, v);
      }
    }
  }
}

// Rows to 8 bits: pieces of 8 elements, `per` of them a row.
template <class X>
__global__ void __launch_bounds__(256) k_quantize(const X* x, long long stride, int per, long long pieces, uint8_t* codes,
                                                  uint8_t* scales) {
  constexpr int AHEAD = 4;
  allow_next();
  await_stream();
  const long long step = (long long)gridDim.x * blockDim.x;
  const bool packed = stride == (long long)per * 8;
  for (long long i0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; i0 - threadIdx.x < pieces; i0 += AHEAD * step) {
    Raw8<X> raw[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const long long i = i0 + k * step;
      raw[k] = {};
      if (i < pieces) raw[k] = load8(packed ? x + i * 8 : x + i / per * stride + i % per * 8);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const long long i = i0 + k * step;
      float v[8];
      unpack8(raw[k], v);
      store_eights(i < pieces ? codes + i * 8 : nullptr, scales + i / 4, v);
    }
  }
}

template <class X, class A, int OUT>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  // several short rows in a block of 256 threads, or one long row in up to 1024
  const int want = (a.n / 8 + 31) / 32 * 32;
  const int tx = want < 1024 ? want : 1024, ty = tx < 256 ? 256 / tx : 1;
  const dim3 grid((unsigned)((a.rows + ty - 1) / ty)), block(tx, ty);
  const bool few = a.terms <= 1;
  auto k = want > 1024  ? k_norm<X, A, OUT, 2, 1, 1024>
           : want > 256 ? few ? k_norm<X, A, OUT, 1, 1, 1024> : k_norm<X, A, OUT, 1, 4, 1024>
           : few        ? k_norm<X, A, OUT, 1, 1, 256>
                        : k_norm<X, A, OUT, 1, 4, 256>;
  return launch_kernel(k, grid, block, 0, 1, st, a);
}
template <class X, class A>
cudaError_t launch_norm(const NormArgs& a, int out, cudaStream_t st) {
  switch (out) {
    case MK_ROWS_BF16: return launch_norm<X, A, MK_ROWS_BF16>(a, st);
    case MK_ROWS_F32: return launch_norm<X, A, MK_ROWS_F32>(a, st);
    case MK_ROWS_E4M3: return launch_norm<X, A, MK_ROWS_E4M3>(a, st);
  }
  return launch_norm<X, A, OUT_NONE>(a, st);
}

size_t el(int type) { return type == MK_ROWS_F32 ? 4 : type == MK_ROWS_BF16 ? 2 : 1; }

}  // namespace
}  // namespace mk

extern "C" {

int mk_norm(int rows, int n, const void* x, int x_type, long long x_stride, const void* add, int add_type, int terms,
            const void* gamma, float eps, void* total, void* out, int out_type, uint8_t* scales, mk_stream stream) {
  using namespace mk;
  if (rows < 0 || n < 1 || n % 8) return fail(MK_ERR_INVALID, "mk_norm: rows or n (a multiple of 8)");
  if (x_type != MK_ROWS_BF16 && x_type != MK_ROWS_F32) return fail(MK_ERR_INVALID, "mk_norm: x_type");
  if (terms < 0 || (terms && add_type != MK_ROWS_BF16 && add_type != MK_ROWS_F32))
    return fail(MK_ERR_INVALID, "mk_norm: terms or add_type");
  if (out && out_type != MK_ROWS_BF16 && out_type != MK_ROWS_F32 && out_type != MK_ROWS_E4M3)
    return fail(MK_ERR_INVALID, "mk_norm: out_type");
  const bool eights = out && out_type == MK_ROWS_E4M3;
  if (eights && n % GROUP) return fail(MK_ERR_INVALID, "mk_norm: 8-bit rows are a multiple of 32 long");
  if (n > MAX_N) return fail(MK_ERR_UNSUPPORTED, "mk_norm: n above 16384");
  if (terms > (1 << 16)) return fail(MK_ERR_UNSUPPORTED, "mk_norm: terms above 65536");
  if (x_stride < n || x_stride > (1ll << 34) || x_stride * (long long)el(x_type) % 16)
    return fail(MK_ERR_INVALID, "mk_norm: x_stride");
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(MK_ERR_INVALID, "mk_norm: eps");
  if (!out && !total) return fail(MK_ERR_INVALID, "mk_norm: neither total nor out");
  if (rows == 0) return MK_OK;
  if (!aligned(x, 16) || (terms && !aligned(add, 16)) || (gamma && !aligned(gamma, 16)) || (total && !aligned(total, 16)) ||
      (out && !aligned(out, 16)) || (eights && !scales))
    return fail(MK_ERR_INVALID, "mk_norm: a buffer is NULL or not 16-byte aligned");
  const size_t r = rows, w = n;
  const bool in_place = total == x && x_stride == n;
  const Span s[6] = {{out, r * w * el(out_type)},
                     {eights ? scales : nullptr, r * w / GROUP},
                     {total, r * w * el(x_type)},
                     {in_place ? nullptr : x, ((r - 1) * (size_t)x_stride + w) * el(x_type)},
                     {terms ? add : nullptr, r * terms * w * el(add_type)},
                     {gamma, 2 * w}};
  if (clash(s, 3, 6)) return fail(MK_ERR_INVALID, "mk_norm: a result overlaps another buffer (total may be x's own packed one)");
  const NormArgs a = {x, x_stride, add, (const __nv_bfloat16*)gamma, total, out, scales, rows, n, terms, eps};
  const int o = out ? out_type : OUT_NONE;
  const bool xf = x_type == MK_ROWS_F32, af = terms && add_type == MK_ROWS_F32;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = xf ? af ? launch_norm<float, float>(a, o, st) : launch_norm<float, __nv_bfloat16>(a, o, st)
                           : af ? launch_norm<__nv_bfloat16, float>(a, o, st) : launch_norm<__nv_bfloat16, __nv_bfloat16>(a, o, st);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_norm", e);
}

int mk_quantize(int rows, int n, const void* x, int x_type, long long x_stride, uint8_t* codes, uint8_t* scales,
                mk_stream stream) {
  using namespace mk;
  if (rows < 0 || n < 1 || n % GROUP) return fail(MK_ERR_INVALID, "mk_quantize: rows or n (a multiple of 32)");
  if (x_type != MK_ROWS_BF16 && x_type != MK_ROWS_F32) return fail(MK_ERR_INVALID, "mk_quantize: x_type");
  if (x_stride < n || x_stride > (1ll << 34) || x_stride * (long long)el(x_type) % 16)
    return fail(MK_ERR_INVALID, "mk_quantize: x_stride");
  if (rows == 0) return MK_OK;
  if (!aligned(x, 16) || !aligned(codes, 16) || !scales)
    return fail(MK_ERR_INVALID, "mk_quantize: a buffer is NULL or not 16-byte aligned");
  const size_t r = rows, w = n;
  const Span s[3] = {{codes, r * w}, {scales, r * w / GROUP}, {x, ((r - 1) * (size_t)x_stride + w) * el(x_type)}};
  if (clash(s, 2, 3)) return fail(MK_ERR_INVALID, "mk_quantize: two of the buffers overlap");
  int sms = 0;
  cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return fail_cuda("mk_quantize", e);
  const long long pieces = (long long)rows * (n / 8), most = (pieces + 1023) / 1024, full = (long long)sms * 32;   // about five rounds (one: 202 us, 186 so)
  const dim3 grid((unsigned)(most < full ? most : full));
  const cudaStream_t st = (cudaStream_t)stream;
  if (x_type == MK_ROWS_F32)
    e = launch_kernel(k_quantize<float>, grid, 256, 0, 1, st, (const float*)x, x_stride, n / 8, pieces, codes, scales);
  else
    e = launch_kernel(k_quantize<__nv_bfloat16>, grid, 256, 0, 1, st, (const __nv_bfloat16*)x, x_stride, n / 8, pieces, codes,
                      scales);
  return e == cudaSuccess ? MK_OK : fail_cuda("mk_quantize", e);
}

}  // extern "C"
