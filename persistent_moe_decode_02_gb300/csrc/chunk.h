// Records shared by the chunk operators' host side (chunk.cu) and their
// kernels (cache.cu, attend.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.cuh"

namespace mk {

constexpr int PAGE = 16;         // tokens of a page
constexpr int KV_TILE = 64;      // keys of an attention tile (4 pages)
constexpr int Q_TILE = 128;      // query rows (tokens x the group's heads) of an attention tile

// One request of a chunk.
struct alignas(16) ChunkReq {
  int seq, nnew;                 // cached tokens, new tokens
  int row0;                      // first packed row of its new tokens
  int page0;                     // first page of it, counted over all requests' pages
  long long tok0;                // first packed row of all its tokens (mk_chunk_read)
  long long pt;                  // first entry of its page-table row
};
static_assert(sizeof(ChunkReq) == 32, "request record is 32 bytes");

// One page that receives new rows (mk_chunk_append).
struct alignas(16) AppendPage {
  int page;                      // in the pool
  int row, n;                    // first packed row, rows
  int slot;                      // of the first row
};
static_assert(sizeof(AppendPage) == 16, "append record is 16 bytes");

// One attention task: new rows [tok0, tok0 + ntok) of a request, one KV head,
// key tiles [tile0, tile0 + ntile).  part >= 0: the task holds a part of the
// keys and writes its unnormalised rows at split row `part`.  The rest says
// again what the kernel would have to look up for it.
struct alignas(16) AttnTask {
  int req, kvh, tok0, ntok, tile0, ntile, part, cta;
  int row, pos;                  // packed row and position of the first row
  int total;                     // cached and new tokens of the request
  int two;                       // 1: some task of this CTA has two query tiles
  long long pt;                  // its page-table row
  long long pad2;
};
static_assert(sizeof(AttnTask) == 64, "attention task is 64 bytes");

// The join of a block of rows whose keys were split over `nparts` tasks, whose
// split rows start at part0 + i * (ntok * G).
struct alignas(16) JoinTask {
  int req, kvh, tok0, ntok, part0, nparts;
  int row;                       // packed row of the first row
  int pad;
};
static_assert(sizeof(JoinTask) == 32, "join task is 32 bytes");

// What the kernels of a chunk read.
struct ChunkView {
  int nq, nkv, d, G;
  int batch, rows, num_pages;
  const ChunkReq* reqs;
  const AppendPage* appends;     // every page that receives rows
  int nappends, npages;          // and their number; all requests' pages
  const int* pt;
  const float2* rope;            // [rows][d / 2] (cos, sin) of the new rows; NULL: no rotation
  const AttnTask* tasks;         // in the order of the CTAs
  const int* cta_start;          // [ctas + 1]
  const JoinTask* joins;
  int ctas, njoins;
  int max_parts, max_join_rows;  // of one join
  float* part_o;                 // [split rows][d] unnormalised sums
  float2* part_ml;               // [split rows] (maximum, sum) of the softmax
  int* status;                   // [0] first recorded error, 0 = none; [1] generation of the tables
  int gen;                       // the generation that this view was made for
};

cudaError_t launch_chunk_rope(const ChunkView& c, double theta, float2* tab, int max_new, cudaStream_t st);
cudaError_t launch_append(const ChunkView& c, bool e4m3, bool f32, const void* qkv, long long row_stride, void* pool,
                          void* q, cudaStream_t st);
cudaError_t launch_read(const ChunkView& c, bool e4m3, const void* pool, void* out, cudaStream_t st);
cudaError_t launch_attend(const ChunkView& c, bool e4m3, const void* q, const void* pool, void* out, cudaStream_t st);

// A graph may replay a call whose chunk was updated since: the view's counts
// then no longer fit the tables, and the kernel leaves everything as it is.
// Asked before anything that a table holds is used as an index: the bytes
// there may be another table's, or angles.
__device__ __forceinline__ bool stale(const ChunkView& c) {
  if (__ldg(c.status + 1) == c.gen) return false;   // (nothing writes it while a kernel runs)
  await_stream();                // a kernel does not end before the one before it
  if (blockIdx.x + blockIdx.y + blockIdx.z + threadIdx.x == 0) atomicCAS(c.status, 0, -1);   // MK_ERR_INVALID
  return true;
}

}  // namespace mk
