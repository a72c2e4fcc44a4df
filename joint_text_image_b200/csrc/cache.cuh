// cache.cuh -- what the operators over the paged key/value cache share: the
// device view of a hia_cache_chunk with its checks, and the host checks of a
// hia_cache and a hia_cache_chunk.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "sm100.cuh"

namespace hia {

constexpr int kStatusBadChunk = HIA_ERR_BAD_CHUNK;

// Device arrays of a chunk (hia_cache_chunk) and the sizes their values are
// checked against.
struct ChunkDev {
  const int32_t* rows;
  const int32_t* past;
  const int32_t* pages;
  int64_t page_stride;
  int32_t B, T, max_pages, n_pages, page_shift;
  int* status;
};

struct Seq {
  int row0, n, past;
};

__device__ __forceinline__ void flag_bad_chunk(int* status) { atomicCAS(status, 0, kStatusBadChunk); }

// Sequence b, or n = 0 (and the status set) if its rows or lengths do not fit.
__device__ __forceinline__ Seq chunk_seq(const ChunkDev& c, int b) {
  const int r0 = __ldg(c.rows + b), r1 = __ldg(c.rows + b + 1), p = __ldg(c.past + b);
  Seq s{r0, r1 - r0, p};
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= c.T && p >= 0 &&
                  int64_t(p) + (r1 - r0) <= (int64_t(c.max_pages) << c.page_shift);
  if (!ok) {
    flag_bad_chunk(c.status);
    s = Seq{0, 0, 0};
  }
  return s;
}

// Page of the cache positions [i << page_shift, ...) of sequence b, or n_pages
// (and the status set) for a number that is no page: the tensor maps read
// zeros there and the append writes nothing.
__device__ __forceinline__ int chunk_page(const ChunkDev& c, int b, int i) {
  const int p = __ldg(c.pages + int64_t(b) * c.page_stride + i);
  if (p >= 0 && p < c.n_pages) return p;
  flag_bad_chunk(c.status);
  return c.n_pages;
}

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks of a cache and a chunk that every entry point makes.
int cache_check(const hia_cache* cache, const hia_cache_chunk* chunk, int64_t T, int Hq);
// A packed [T, heads, D] tensor of elements of `size` bytes.
int rows_check(const hia_tensor& t, bool q_heads, int g, size_t size);
// Such a tensor whose rows and heads may not share memory.
int own_rows_check(const hia_tensor& t, int64_t T, int Hkv, int g);
ChunkDev chunk_dev(const hia_cache& cache, const hia_cache_chunk& chunk, int64_t T, int* status);

int* device_status_word();

}  // namespace hia
