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
// ordering between the XCDs' caches within a kernel. It takes 3 to 4 us where nothing or
// little was cut, 6 to 11 us after a decode step of 64 sequences and 17 to 20 where large trees
// left cut tiles of 256 rows.
#include <algorithm>
#include <type_traits>

#include "attention_common.h"

namespace qg {

namespace {

constexpr int JT = 256;
// of 256 threads: a launch has less than 2^32 of those
constexpr long long kMostWorkgroups = (1ll << 24) - 1;
constexpr int kRowsMost = 512, kRowsStep = 32, kRowsHeads = 4;
// Items of the kernel for many rows, two per CU (one per CU: 1000 tokens after 32000 685 us
// against 517; four: eight prompts of 1 to 1024 tokens 54 us against 42, heads of 256 with a
// window 302 against 272, though e4m3 chunks with runs of 32 381 against 407), of at least
// 256 positions (128 or 512: level). A tile is cut only where it is longer than an even share
// of all tiles' positions, so batches of several prompts are not: of those eight, played
// through in launch order, the last workgroup ends after 16 blocks where the mean is 11.
constexpr int kTileTarget = 512, kTileMinChunk = 256, kTileStep = 64;
constexpr int kTreeRows = kTileTarget * 128;   // of all of a tree call's workgroups that run at once, at most

constexpr int dp_of(int64_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

}  // namespace

// A wave per row: its lanes take DP / 4 groups of four floats of 256 / DP parts at a
// time, eight such steps in flight, so that a row of up to 2048 / DP parts costs one
// memory latency after its record's.
template <int DP, bool TREE>
__global__ __launch_bounds__(JT) void attention_join_kernel(AttnArgs p, int parts, int rows_per_wg) {
  constexpr int LR = DP / 4, PH = 64 / LR;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x % p.hkv, at = blockIdx.x / p.hkv;
  const AttnRecord t = *attn_record(p, at / parts);
  if (at / parts >= *attn_record_count(p) || t.parts <= 1) return;   // (or written by the one that computed it)
  const int ns = t.parts;
  const long long slot_floats = attn_slot_floats(p.bm, DP);
  const float* slots = p.workspace + attn_header_floats(p.target);
  auto part_at = [&](int s) {
    return slots + (long long)((s == 0 ? t.first : t.next + (s - 1) * t.step) + h * t.head_step) * slot_floats;
  };
  const int d = lane % LR * 4, phase = lane / LR;
  const int r0 = at % parts * rows_per_wg, r1 = min(t.r_count, r0 + rows_per_wg);
  for (int r = r0 + wave; r < r1; r += JT / 64) {
    const int ml = p.bm * DP + 2 * r;   // a row's maximum and sum in a slot
    float top = -INFINITY;
    for (int s = lane; s < ns; s += 64) top = fmaxf(top, part_at(s)[ml]);
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
    const float base = top == -INFINITY ? 0.f : top;
    float4_t o;
    float sum;
    // KEEP: infinities and NaN stay, however small the part's share
    auto join = [&](auto keep) {
      constexpr bool KEEP = decltype(keep)::value;
      o = float4_t{0.f, 0.f, 0.f, 0.f};
      sum = 0.f;
      auto add = [&](auto steps, int s0) {   // parts s0, s0 + PH, ..: `steps` of them
        constexpr int U = decltype(steps)::value;
        float4_t x[U];
        float2_t m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float* from = part_at(min(s0 + u * PH, ns - 1));
          x[u] = *reinterpret_cast<const float4_t*>(from + (size_t)r * DP + d);
          m[u] = *reinterpret_cast<const float2_t*>(from + ml);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float f = __builtin_amdgcn_exp2f(m[u].x - base);
          if (s0 + u * PH < ns) {
            sum = __builtin_fmaf(m[u].y, f, sum);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[u][i], KEEP && !(fabsf(x[u][i]) < INFINITY) ? 1.f : f, o[i]);
          }
        }
      };
      if (ns <= 2 * PH) {
        add(std::integral_constant<int, 2>{}, phase);
      } else {
        for (int s0 = phase; s0 < ns; s0 += 8 * PH) add(std::integral_constant<int, 8>{}, s0);
      }
#pragma unroll
      for (int k = LR; k < 64; k <<= 1) {
        sum += __shfl_xor(sum, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], k);
      }
    };
    join(std::false_type{});
    if (__any(!(fabsf(o[0]) + fabsf(o[1]) + fabsf(o[2]) + fabsf(o[3]) < INFINITY))) join(std::true_type{});
    float inv = 1.f / sum;
    if (TREE && __any(sum == 0.f)) {   // the row sees nothing, or scores of -infinity alone (see seen_sum)
      bool sees = false;
      for (int s = lane; s < ns; s += 64) sees |= part_at(s)[ml + 1] != 0.f;
      inv = __any(sees) ? inv : 0.f;
    }
    const int row = t.r_first + r, token = over_group(p, row);
    uint16_t* to = p.out + ((size_t)(t.row0 + token) * p.hq + h * p.group + row - token * p.group) * p.d;
    if (phase == 0 && d < p.d)
      *reinterpret_cast<u32x2_t*>(to + d) = u32x2_t{f2bf2_rn(o[0] * inv, o[1] * inv), f2bf2_rn(o[2] * inv, o[3] * inv)};
  }
}

// cut: records, at most
static hipError_t launch_join(const AttnArgs& p, long long cut, hipStream_t stream) {
  const long long rows = std::min<long long>(p.bm, p.T * p.group);
  // a row per wave where that still is about one round of workgroups
  const int per_wg = cut * p.hkv * rows <= 64LL * p.num_cus ? 4 : 16;
  const long long parts = (rows + per_wg - 1) / per_wg;
  const dim3 grid((unsigned)(cut * parts * p.hkv));
  auto join = [&](auto of_64, auto of_128, auto of_256) {
    (p.d <= 64 ? of_64 : p.d <= 128 ? of_128 : of_256)<<<grid, JT, 0, stream>>>(p, (int)parts, per_wg);
  };
  if (p.tree) join(attention_join_kernel<64, true>, attention_join_kernel<128, true>, attention_join_kernel<256, true>);
  else join(attention_join_kernel<64, false>, attention_join_kernel<128, false>, attention_join_kernel<256, false>);
  return hipGetLastError();
}

static int log2_of(int64_t x) {
  int k = 0;
  while (((int64_t)1 << k) < x) ++k;
  return k;
}

// items of the kernel for many rows: a power of two, and at least one per head
static int tile_target(int64_t hkv) { return std::max(kTileTarget, 1 << log2_of(hkv)); }

int64_t attention_paged_workspace(int64_t T, int64_t batch, int64_t hq, int64_t hkv, int64_t d) {
  (void)T; (void)batch; (void)hq;
  // two slots per share and head
  const int64_t rt = std::max<int64_t>(kRowsMost, hkv), tt = tile_target(hkv);
  return std::max(attn_header_floats((int)rt) + 2 * kRowsHeads * rt * attn_slot_floats(32, dp_of(d)),
                  attn_header_floats((int)tt) + 2 * tt * attn_slot_floats(128, dp_of(d)));
}

// x / d for x < 2^31 as (umulhi(x, mul) + x) >> shift
static void divide_by(int d, uint32_t& mul, uint32_t& shift) {
  shift = log2_of(d);
  mul = (uint32_t)((((1ull << 32) * ((1ull << shift) - (uint64_t)d)) / (uint64_t)d) + 1);
}

// Sets how the work is cut: rows per tile, positions per unit.
static void set_shape(AttnArgs& p, int bm, int step) {
  p.bm = bm;
  p.bm_log2 = log2_of(bm);
  p.step = step;
  p.step_log2 = log2_of(step);
  // a tile has tokens t .. t + (bm - 1) / group + 1 at most, and starts up to step - 1 early
  const long long span = (long long)p.window + (bm - 1) / p.group + 1 + step;
  p.window_span = (int)std::min<long long>(span, INT32_MAX);
}

hipError_t launch_attention_paged(const AttnArgs& args, hipStream_t stream) {
  AttnArgs p = args;
  divide_by(p.page_size, p.div_mul, p.div_shift);
  divide_by(p.group, p.group_mul, p.group_shift);
  const long long rows = p.T * p.group;
  // By the batch's average, as the host knows no more. The kernel for few rows takes up to 16
  // rows per sequence and head (64 sequences of one token, 4 heads to one: bf16 204 us against
  // 264 in tiles of 128 rows, e4m3 123 against 331), and up to 32 where there are many
  // sequences (32 of 6 tokens: on 500 positions bf16 24 us against 30, e4m3 29 against 32; on
  // 4000 e4m3 84 against 110, but bf16 127 against 112). With fewer, each is cut into many
  // parts, whose records of 32 rows cost more than half-empty tiles (8 sequences on 4000: bf16
  // 48 us against 33, e4m3 47 against 37), except for e4m3 heads of 256, which the kernel
  // for many rows is slow at (81 us against 102, runs of 32 99 against 146; on 500 positions
  // 38 against 32). Beyond 32 rows it loses (32 sequences of 16 tokens on 4000: bf16 186 us
  // against 117, e4m3 134 against 114). A few long chunks among many single tokens go by the
  // average too: 256 tokens on 1000 and a chunk of 512 after 8000, bf16 863 us, 281 us as two calls.
  //
  // Trees have a kernel of their own for many rows, which on bf16 caches is the faster one from 17
  // rows on (32 trees of 6 tokens on 4000: 125 us against 129, 64 of 8 on 1000 55 against 70, of heads of
  // 64 33 against 49, heads of 256, 32 of 6 on 4000, 245 against 241), but not with 16 or fewer (32 of 4 on
  // 4000, without the remainders below: 121 against 112, heads of 256 212 against 205; heads of 64 57 against
  // 67), and on e4m3 where the other is (32 of 8 on 4000: 110 against 90; 8 of them 48 against 52; heads of
  // 256, 8 of 8, 117 against 94).
  const int mt = rows > 16LL * p.batch ? 2 : 1;
  const bool some = (!p.tree || p.fp8) && rows <= 32LL * p.batch && (4LL * p.batch * p.hkv > p.num_cus || (p.fp8 && p.d > 128));
  const bool few = mt == 1 || some;
  set_shape(p, few ? 16 * mt : 128, few ? kRowsStep : kTileStep);
  // sequence b has ceil(new_b * group / bm) tiles per key/value head, of at most `room` positions
  const long long tiles = rows / p.bm + p.batch, room = p.max_pages * p.page_size;
  if (few) {
    attention_rows_shape(p, mt);
    const int groups = p.hkv / p.hw;
    p.target = std::max(std::min(p.target, kRowsMost), groups);
    // pieces, at most: a wave per head (groups), or all waves on one head
    while ((room + p.step - 1) / p.step > INT32_MAX / tiles) set_shape(p, p.bm, 2 * p.step);   // units are counted in 32 bits
    const long long units = (room + p.step - 1) / p.step;   // of a tile, at most
    const long long wide = std::min<long long>(p.target / groups, tiles * units);
    const long long narrow = std::min<long long>(std::max(p.target / p.hkv, 1), tiles * units);
    const long long grid = std::max((wide + 7) / 8 * 8 * groups, (narrow + 7) / 8 * 8 * p.hkv);
    if (grid > kMostWorkgroups) return hipErrorNotSupported;
    const hipError_t e = (p.tree ? launch_attention_rows_tree : launch_attention_rows)(p, mt, (unsigned)grid, stream);
    const long long pieces = std::max(wide, narrow);
    return e != hipSuccess || pieces <= 1 ? e : launch_join(p, pieces, stream);   // one piece has all its tiles whole
  }
  if (p.tree) {
    // Tiles of 256 rows where 128 are not enough for most sequences: 32 trees of 64 tokens, 4 heads to one,
    // on up to 8191 positions 210 us against 244, 6 of 20 to 120 on up to 40000 (e4m3) 459 against 516.
    //
    // Up to 32 rows on bf16 caches: with the weights' remainders, as in the kernel for few rows. The error
    // against 64 bits is that of the result's rounding then, 1.66e-3 of the result (root mean square), without
    // them 2.33e-3; 32 trees of 6 on 4000 take 125 us against 122, 64 of 8 on 1000 55 against 53, heads of 64 33.5
    // against 30, of 256 245 against 211. With more rows they cost more and are left out, as in the other calls:
    // 32 of 32 on 4000 149 against 145, heads of 64 90 against 78, of 256 285 against 242; 32 of 64 213 against 170.
    const TreeTiles kind = rows > 128LL * p.batch ? TREE_TALL : rows > 32LL * p.batch ? TREE_MANY : TREE_FEW;
    attention_tree_shape(p, kind);
    p.target = std::max<int>(std::min<int>(p.target, kTreeRows / p.bm), p.hkv);   // the workspace's slots
    set_shape(p, p.bm, kTileStep);
    const long long tree_tiles = rows / p.bm + p.batch;
    while ((room + p.step - 1) / p.step > INT32_MAX / tree_tiles) set_shape(p, p.bm, 2 * p.step);   // units are counted in 32 bits
    const long long pieces = std::min<long long>(p.target / p.hkv, tree_tiles * ((room + p.step - 1) / p.step));
    const long long grid = (pieces + 7) / 8 * 8 * p.hkv;
    if (grid > kMostWorkgroups) return hipErrorNotSupported;
    const hipError_t e = launch_attention_tree(p, kind, (unsigned)grid, stream);
    return e != hipSuccess || pieces <= 1 ? e : launch_join(p, pieces, stream);
  }
  p.min_chunk = kTileMinChunk;
  p.target = tile_target(p.hkv);
  p.target_log2 = log2_of(p.target);
  // Items: at most target / hkv + tiles (a chunk is at least the work over the target),
  // and each tile has as many as the page table has room for. Workgroups past the last
  // item return.
  const long long chunks = (room + p.min_chunk - 1) / p.min_chunk;
  const long long items = std::min(tiles + p.target / p.hkv + 1, chunks < tiles + p.target ? tiles * chunks : (long long)INT64_MAX);
  if (items > kMostWorkgroups / p.hkv) return hipErrorNotSupported;
  const hipError_t e = launch_attention_tiles(p, (unsigned)(items * p.hkv), stream);
  // tiles that are cut have at least two slots each, of fewer than 2 target
  return e != hipSuccess || chunks <= 1 ? e : launch_join(p, std::min(tiles, (long long)(p.target / p.hkv + 1)), stream);
}

}  // namespace qg
