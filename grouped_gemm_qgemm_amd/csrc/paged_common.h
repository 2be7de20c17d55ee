// Shared by the kernels that move rows of a paged cache: the sequence of a ragged row, and
// the cache row of a position.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace qg {

// Sets x / page_size for x < 2^31 as (umulhi(x, mul) + x) >> shift.
inline void divide_pages(CacheArgs& kv) {
  kv.div_shift = 0;
  while ((1ll << kv.div_shift) < kv.page_size) ++kv.div_shift;
  kv.div_mul = (uint32_t)((((1ull << 32) * ((1ull << kv.div_shift) - (uint64_t)kv.page_size)) / (uint64_t)kv.page_size) + 1);
}

// Row (page * page_size + slot) of a plane that holds position `pos` of sequence b.
__device__ __forceinline__ long long cache_row(const CacheArgs& kv, int b, uint32_t pos) {
  const uint32_t pg = (__umulhi(pos, kv.div_mul) + pos) >> kv.div_shift;
  return (long long)kv.page_table[(size_t)b * kv.max_pages + pg] * kv.page_size + (pos - pg * (uint32_t)kv.page_size);
}

// The sequence of ragged row r, the last b with offs[b] <= r (of sequences that share a
// start, the one that is not empty); -1 for rows from offs[batch] on. The calling wave
// searches together, 64 places at a time (r the same in every lane): one memory latency
// for up to 64 sequences, two for up to 4096.
__device__ __forceinline__ int owner_of(const uint32_t* __restrict__ offs, int batch, uint32_t r) {
  const int lane = threadIdx.x & 63;
  const uint32_t rows = offs[batch];
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = lane * step;
    const bool below = at < n && offs[lo + min(at, n - 1)] <= r;
    const int last = __popcll(__ballot(below)) - 1;   // (offs[0] = 0: lane 0 always is)
    lo += max(last, 0) * step;
    n = min(step, n - max(last, 0) * step);
  }
  return r < rows ? __builtin_amdgcn_readfirstlane(lo) : -1;
}

}  // namespace qg
