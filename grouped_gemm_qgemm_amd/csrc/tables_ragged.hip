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
// repeats the prefix sums (2 x 4 bytes per sequence, from L2) and writes its
// share of the outputs. Nothing that one workgroup writes is read by another:
// entries added by this call are taken from the free stack again where a
// token's slot needs them.
#include "device_common.h"
#include "launch.h"

namespace qg {

namespace {

constexpr int TT = 1024;             // threads per workgroup
constexpr int TSEQ = kTablesMaxBatch;
constexpr int TPER = TSEQ / TT;      // consecutive sequences per thread, at most

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
    uint32_t free_len, long long slot_len, uint32_t page_size) {
  __shared__ uint32_t s_tok[TSEQ], s_pg[TSEQ];
  __shared__ unsigned long long w_tok[TT / 64], w_pg[TT / 64];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) s_bad = 0;
  __syncthreads();

  // sums in 64 bits, so that lengths which are too long are seen as such
  const int per = (batch + TT - 1) / TT;
  unsigned long long tok = 0, pg = 0;
  uint32_t n_own[TPER], p_own[TPER];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < TPER; ++k) {
    const int b = tid * per + k;
    n_own[k] = p_own[k] = 0;
    if (k < per && b < batch) {
      const unsigned long long c = cached[b], n = fresh[b];
      if (n != 0) {   // a sequence without new tokens is left alone, whatever its length
        const unsigned long long need = (c + n + page_size - 1) / page_size;
        bad |= need > (unsigned long long)max_pages;
        n_own[k] = (uint32_t)n;
        p_own[k] = (uint32_t)(need - (c + page_size - 1) / page_size);
        tok += n;
        pg += p_own[k];
      }
    }
  }
  if (bad) s_bad = 1;
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
#pragma unroll
  for (int k = 0; k < TPER; ++k) {
    const int b = tid * per + k;
    if (k < per && b < batch) {
      s_tok[b] = (uint32_t)xt;
      s_pg[b] = (uint32_t)xp;
      xt += n_own[k];
      xp += p_own[k];
    }
  }
  __syncthreads();

  const uint32_t count = free_count[0];
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
    const uint32_t held = (cached[b] + page_size - 1) / page_size;
    table[(size_t)b * max_pages + held + (j - s_pg[b])] = free_pages[count - 1 - j];
  }
  if (!slots) return;
  for (uint32_t t = gid; t < (uint32_t)tokens; t += threads) {
    const int b = owner(s_tok, batch, t);
    const uint32_t c = cached[b], pos = c + (t - s_tok[b]);
    const uint32_t held = (c + page_size - 1) / page_size;
    const uint32_t col = pos / page_size;
    const uint32_t page = col < held ? table[(size_t)b * max_pages + col] : free_pages[count - 1 - (s_pg[b] + col - held)];
    slots[t] = (int32_t)(page * page_size + pos % page_size);
  }
}

hipError_t launch_tables_ragged(const TablesArgs& p, hipStream_t stream) {
  // one workgroup per 4096 tokens (four passes of its threads), at most two per CU
  const long long want = (p.slot_len + 4 * TT - 1) / (4 * TT);
  const int grid = (int)(want < 1 ? 1 : want > 2 * p.num_cus ? 2 * p.num_cus : want);
  tables_ragged_kernel<<<grid, TT, 0, stream>>>(p.offsets, p.slots, p.table, p.result, p.cached, p.fresh, p.free_pages,
                                                p.free_count, p.batch, p.max_pages, (uint32_t)p.free_len, p.slot_len,
                                                (uint32_t)p.page_size);
  return hipGetLastError();
}

}  // namespace qg
