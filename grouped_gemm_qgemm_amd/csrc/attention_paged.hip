// Attention over the paged cache: which kernel a call takes, and the join of
// tiles whose positions were cut into parts.
//
// A part leaves, per row, its maximum M_s (base-2 exponent), its sum of weights
// L_s and its unnormalised output O_s, all fp32. The join is
//
//   out = sum_s 2^(M_s - M) O_s / sum_s 2^(M_s - M) L_s,   M = max_s M_s
//
// It is a second launch on the same stream rather than the task of the last
// part to finish: that needs counters which every call must find at zero, and
// ordering between the XCDs' caches within a kernel.
#include <algorithm>

#include "attention_common.h"

namespace qg {

namespace {

constexpr int JT = 256;
constexpr int kRowsMost = 512, kRowsStep = 32, kRowsUnits = 4, kRowsHeads = 4;
constexpr int kTileTarget = 512, kTileMinChunk = 256, kTileStep = 64;

constexpr int dp_of(int64_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

}  // namespace

// WPR waves share a row's parts (4 where rows are few, 1 else).
template <int DP, int WPR>
__global__ __launch_bounds__(JT) void attention_join_kernel(AttnArgs p, int parts, int rows_per_wg) {
  constexpr int VL = DP / 64;   // floats per lane
  __shared__ float part[WPR > 1 ? 4 : 1][DP + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x % p.hkv, at = blockIdx.x / p.hkv;
  if (at / parts >= *attn_record_count(p)) return;
  const AttnRecord t = *attn_record(p, at / parts);
  const int ns = t.parts;
  if (ns <= 1) return;   // written by the one that computed it
  const long long slot_floats = attn_slot_floats(p.bm, DP);
  const float* slots = p.workspace + attn_header_floats(p.target);
  auto part_at = [&](int s) {
    return slots + (long long)((s == 0 ? t.first : t.next + (s - 1) * t.step) + h * t.head_step) * slot_floats;
  };
  const int r0 = at % parts * rows_per_wg, r1 = min(t.r_count, r0 + rows_per_wg);
  for (int r = r0 + (WPR > 1 ? 0 : wave); r < r1; r += WPR > 1 ? 1 : 4) {
    const int ml = p.bm * DP + 2 * r;   // a row's maximum and sum in a slot
    float top = -INFINITY;
    for (int s = lane; s < ns; s += 64) top = fmaxf(top, part_at(s)[ml]);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float base = top == -INFINITY ? 0.f : top;
    float o[VL], sum = 0.f;
#pragma unroll
    for (int i = 0; i < VL; ++i) o[i] = 0.f;
    for (int s0 = 0; s0 < ns; s0 += 64) {
      float f = 0.f;
      if (s0 + lane < ns) {
        const float* x = part_at(s0 + lane) + ml;
        f = __builtin_amdgcn_exp2f(x[0] - base);
        sum = __builtin_fmaf(x[1], f, sum);
      }
      const int n = min(64, ns - s0);
      for (int s = WPR > 1 ? wave : 0; s < n; s += 8 * WPR) {   // eight parts' loads in flight
        float x[8][VL], fs[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int su = s + u * WPR;
          fs[u] = su < n ? __shfl(f, su) : 0.f;
          const float* at_u = part_at(s0 + min(su, n - 1)) + r * DP + lane * VL;
#pragma unroll
          for (int i = 0; i < VL; ++i) x[u][i] = at_u[i];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int i = 0; i < VL; ++i) o[i] = __builtin_fmaf(x[u][i], fs[u], o[i]);
      }
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);   // every wave has all parts' sums
    if constexpr (WPR > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VL; ++i) part[wave][lane * VL + i] = o[i];
      __syncthreads();
      if (wave != 0) continue;
#pragma unroll
      for (int i = 0; i < VL; ++i) o[i] = (part[0][lane * VL + i] + part[1][lane * VL + i]) + (part[2][lane * VL + i] + part[3][lane * VL + i]);
    }
    const float inv = 1.f / sum;
    const int row = t.r_first + r;
    uint16_t* to = p.out + ((size_t)(t.row0 + row / p.group) * p.hq + h * p.group + row % p.group) * p.d;
#pragma unroll
    for (int i = 0; i < VL; ++i)
      if (lane * VL + i < p.d) to[lane * VL + i] = (uint16_t)f2bf2_rn(o[i] * inv, 0.f);
  }
}

// cut: records, at most
static hipError_t launch_join(const AttnArgs& p, long long cut, hipStream_t stream) {
  const long long rows = std::min<long long>(p.bm, p.T * p.group);
  const bool few = cut * p.hkv * rows <= 8 * p.num_cus;
  const int per_wg = few ? 1 : 16;
  const long long parts = (rows + per_wg - 1) / per_wg;
  const dim3 grid((unsigned)(cut * parts * p.hkv));
#define QG_JOIN(DP)                                                                                 \
  do {                                                                                              \
    if (few) attention_join_kernel<DP, 4><<<grid, JT, 0, stream>>>(p, (int)parts, per_wg);          \
    else attention_join_kernel<DP, 1><<<grid, JT, 0, stream>>>(p, (int)parts, per_wg);              \
  } while (0)
  if (p.d <= 64) QG_JOIN(64);
  else if (p.d <= 128) QG_JOIN(128);
  else QG_JOIN(256);
#undef QG_JOIN
  return hipGetLastError();
}

int64_t attention_paged_workspace(int64_t T, int64_t batch, int64_t hq, int64_t hkv, int64_t d) {
  (void)T; (void)batch; (void)hq;
  // two slots per share and head
  const int64_t rt = std::max<int64_t>(kRowsMost, hkv), tt = std::max<int64_t>(kTileTarget, hkv);
  return std::max(attn_header_floats((int)rt) + 2 * kRowsHeads * rt * attn_slot_floats(32, dp_of(d)),
                  attn_header_floats((int)tt) + 2 * tt * attn_slot_floats(128, dp_of(d)));
}

hipError_t launch_attention_paged(const AttnArgs& args, hipStream_t stream) {
  AttnArgs p = args;
  // x / page_size for x < 2^31: (umulhi(x, mul) + x) >> shift
  int shift = 0;
  while ((1u << shift) < (uint32_t)p.page_size) ++shift;
  p.div_shift = shift;
  p.div_mul = (uint32_t)((((1ull << 32) * ((1ull << shift) - (uint64_t)p.page_size)) / (uint64_t)p.page_size) + 1);
  const long long rows = p.T * p.group;
  const bool few = rows <= 32LL * p.batch;
  const int mt = rows > 16LL * p.batch ? 2 : 1;
  p.bm = few ? 16 * mt : 128;
  // sequence b has ceil(new_b * group / bm) tiles per key/value head, of at most `room` positions
  const long long tiles = rows / p.bm + p.batch, room = p.max_pages * p.page_size;
  if (few) {
    p.step = kRowsStep;
    p.min_chunk = kRowsUnits;
    attention_rows_shape(p, mt);
    const int groups = p.hkv / p.hw;
    p.target = std::max(std::min(p.target, kRowsMost), groups);
    const long long units = (room + p.step - 1) / p.step;   // of a tile, at most
    const long long shares = units < p.target ? std::min<long long>(p.target / groups, (tiles * units + p.min_chunk - 1) / p.min_chunk)
                                              : p.target / groups;
    const long long grid = (shares + 7) / 8 * 8 * groups;
    if (grid > INT32_MAX) return hipErrorNotSupported;
    const hipError_t e = launch_attention_rows(p, mt, (unsigned)grid, stream);
    return e != hipSuccess || shares <= 1 ? e : launch_join(p, shares, stream);   // one share has all its tiles whole
  }
  p.step = kTileStep;
  p.min_chunk = kTileMinChunk;
  p.target = std::max(kTileTarget, p.hkv);
  // Items: at most target / hkv + tiles (a chunk is at least the work over the target),
  // and each tile has as many as the page table has room for. Workgroups past the last
  // item return.
  const long long chunks = (room + p.min_chunk - 1) / p.min_chunk;
  const long long items = std::min(tiles + p.target / p.hkv + 1, chunks < tiles + p.target ? tiles * chunks : (long long)INT64_MAX);
  if (items * p.hkv > INT32_MAX) return hipErrorNotSupported;
  const hipError_t e = launch_attention_tiles(p, (unsigned)(items * p.hkv), stream);
  // tiles that are cut have at least two slots each, of fewer than 2 target
  return e != hipSuccess || chunks <= 1 ? e : launch_join(p, std::min(tiles, (long long)(p.target / p.hkv + 1)), stream);
}

}  // namespace qg
