// Tables of a paged KV cache, built on the device from the sequences' lengths:
// the ragged row offsets, the page table's new entries (taken from a stack of
// free pages) and each new token's slot.
//
// With c_b tokens cached and n_b new ones, S slots per page:
//
//   offsets[b + 1] = n_0 + ... + n_b
//   held_b = ceil(c_b / S), need_b = ceil((c_b + n_b) / S)
//   page_table[b][held_b + i] = free[count - 1 - (first_b + i)]   i < need_b - held_b
//   slot of token j = page_table[b][(c_b + j) / S] * S + (c_b + j) % S
//
// where first_b counts the new pages of the sequences before b. Two prefix sums
// over the sequences, then independent writes. All of it moves a few bytes per
// token, so a call is bound by its latency: one launch, in which every workgroup
// repeats the prefix sums (2 x 4 bytes per sequence, from L2; totals in 64 bits,
// so that lengths which are too long are seen as such) and writes its share of the
// outputs. Nothing that one workgroup writes is read by another:
// entries added by this call are taken from the free stack again where a
// token's slot needs them.
//
// Measured: 4.3 us on the GPU for 32 sequences of one token (9 us a call from
// Python, which the binding bounds), 11.4 us for 2048 sequences with 0.52 million
// tokens (2.4 MB).
#include "device_common.h"
#include "launch.h"

namespace qg {

namespace {

constexpr int TT = 256;              // threads per workgroup
constexpr int TSEQ = kTablesMaxBatch;
constexpr int TLD = 8;               // sequences a thread loads at a time
constexpr int TTOK = 4;              // consecutive tokens per thread and pass: one search, one 16-byte store

// last b with first[b] <= x: among sequences that share a start, the one that is
// not empty
__device__ __forceinline__ int owner(const uint32_t* first, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ __launch_bounds__(TT) void tables_ragged_kernel(
    uint32_t* __restrict__ offsets, int32_t* __restrict__ slots, uint32_t* __restrict__ table,
    uint32_t* __restrict__ result, const uint32_t* __restrict__ cached, const uint32_t* __restrict__ fresh,
    const uint32_t* __restrict__ free_pages, const uint32_t* __restrict__ free_count, int batch, int max_pages,
    uint32_t free_len, long long slot_len, uint32_t page_size, uint32_t div_mul, uint32_t div_shift) {
  __shared__ uint32_t s_tok[TSEQ], s_pg[TSEQ];
  __shared__ unsigned long long w_tok[TT / 64], w_pg[TT / 64];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t count = free_count[0];
  // x / page_size, for positions that the page table has room for (below 2^31)
  auto page_of = [&](uint32_t x) { return (__umulhi(x, div_mul) + x) >> div_shift; };
  if (tid == 0) s_bad = 0;
  __syncthreads();

  const unsigned long long room = (unsigned long long)max_pages * page_size;   // below 2^31
  bool bad = false;
  for (int b0 = tid; b0 < batch; b0 += TLD * TT) {   // new tokens and pages of each sequence
    uint32_t n[TLD], c[TLD];
#pragma unroll
    for (int k = 0; k < TLD; ++k) {
      const int b = min(b0 + k * TT, batch - 1);
      n[k] = fresh[b];
      c[k] = cached[b];
    }
#pragma unroll
    for (int k = 0; k < TLD; ++k) {
      uint32_t more = 0;
      const unsigned long long len = (unsigned long long)c[k] + n[k];
      if (n[k] == 0) {
        // a sequence without new tokens is left alone, whatever its length
      } else if (len <= room) {
        more = page_of(c[k] + n[k] + page_size - 1) - page_of(c[k] + page_size - 1);
      } else {   // past what page_of takes
        bad = true;
        const unsigned long long m = (len + page_size - 1) / page_size - ((unsigned long long)c[k] + page_size - 1) / page_size;
        more = (uint32_t)min(m, 0xFFFFFFFFull);
      }
      if (b0 + k * TT < batch) {
        s_tok[b0 + k * TT] = n[k];
        s_pg[b0 + k * TT] = more;
      }
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  // their starts: each thread sums consecutive sequences
  const int per = (batch + TT - 1) / TT;
  unsigned long long tok = 0, pg = 0;
  for (int b = tid * per; b < min(batch, tid * per + per); ++b) {
    tok += s_tok[b];
    pg += s_pg[b];
  }
  unsigned long long it = tok, ip = pg;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const unsigned long long vt = __shfl_up(it, d), vp = __shfl_up(ip, d);
    if (lane >= d) { it += vt; ip += vp; }
  }
  if (lane == 63) { w_tok[wave] = it; w_pg[wave] = ip; }
  __syncthreads();
  unsigned long long bt = 0, bp = 0, tokens = 0, pages = 0;
#pragma unroll
  for (int w = 0; w < TT / 64; ++w) {
    if (w < wave) { bt += w_tok[w]; bp += w_pg[w]; }
    tokens += w_tok[w];
    pages += w_pg[w];
  }
  unsigned long long xt = bt + it - tok, xp = bp + ip - pg;
  for (int b = tid * per; b < min(batch, tid * per + per); ++b) {
    const uint32_t n = s_tok[b], more = s_pg[b];
    s_tok[b] = (uint32_t)xt;
    s_pg[b] = (uint32_t)xp;
    xt += n;
    xp += more;
  }
  __syncthreads();

  uint32_t status = 0;
  if (count > free_len || pages > count) status |= 1;
  if (s_bad) status |= 2;
  if (tokens > 0x7FFFFFFFull || (slots && tokens > (unsigned long long)slot_len)) status |= 4;
  if (blockIdx.x == 0 && tid == 0) {
    result[0] = status ? count : count - (uint32_t)pages;
    result[1] = status;
  }
  if (status) return;

  const uint32_t gid = blockIdx.x * TT + tid, threads = gridDim.x * TT;
  for (uint32_t b = gid; b <= (uint32_t)batch; b += threads) offsets[b] = b < (uint32_t)batch ? s_tok[b] : (uint32_t)tokens;
  for (uint32_t j = gid; j < (uint32_t)pages; j += threads) {
    const int b = owner(s_pg, batch, j);
    const uint32_t held = page_of(cached[b] + page_size - 1);
    table[(size_t)b * max_pages + held + (j - s_pg[b])] = free_pages[count - 1 - j];
  }
  if (!slots) return;
  const uint32_t all = (uint32_t)tokens;
  for (uint32_t t0 = gid * TTOK; t0 < all; t0 += threads * TTOK) {
    int b = owner(s_tok, batch, t0);
    int32_t v[TTOK];
    uint32_t c = cached[b], pos = c + (t0 - s_tok[b]), next = b + 1 < batch ? s_tok[b + 1] : all;
    uint32_t held = page_of(c + page_size - 1), seen = ~0u, page = 0;
#pragma unroll
    for (int k = 0; k < TTOK; ++k) {
      const uint32_t t = t0 + k;
      if (t < all) {
        if (t >= next) {   // on to the next sequence that has tokens
          do {
            ++b;
            next = b + 1 < batch ? s_tok[b + 1] : all;
          } while (t >= next);
          pos = c = cached[b];
          held = page_of(c + page_size - 1);
          seen = ~0u;
        }
        const uint32_t col = page_of(pos);
        if (col != seen) {
          seen = col;
          page = col < held ? table[(size_t)b * max_pages + col] : free_pages[count - 1 - (s_pg[b] + col - held)];
        }
        v[k] = (int32_t)(page * page_size + (pos - col * page_size));
        ++pos;
      }
    }
    if (t0 + TTOK <= all) {
      *reinterpret_cast<int4*>(slots + t0) = int4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int k = 0; k < TTOK; ++k)
        if (t0 + k < all) slots[t0 + k] = v[k];
    }
  }
}

hipError_t launch_tables_ragged(const TablesArgs& p, hipStream_t stream) {
  // x / page_size for x < 2^31 as (umulhi(x, mul) + x) >> shift
  uint32_t shift = 0;
  while ((1u << shift) < (uint32_t)p.page_size) ++shift;
  const uint32_t mul = (uint32_t)((((1ull << 32) * ((1ull << shift) - (uint64_t)p.page_size)) / (uint64_t)p.page_size) + 1);
  // a workgroup per 2048 tokens (two passes of its threads), at most two per CU (64 KB of LDS)
  const long long want = (p.slot_len + 2 * TTOK * TT - 1) / (2 * TTOK * TT);
  const int grid = (int)(want < 1 ? 1 : want > 2 * p.num_cus ? 2 * p.num_cus : want);
  tables_ragged_kernel<<<grid, TT, 0, stream>>>(p.offsets, p.slots, p.table, p.result, p.cached, p.fresh, p.free_pages,
                                                p.free_count, p.batch, p.max_pages, (uint32_t)p.free_len, p.slot_len,
                                                (uint32_t)p.page_size, mul, shift);
  return hipGetLastError();
}

}  // namespace qg
