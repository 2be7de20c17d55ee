// Shared by the attention kernels over the paged cache: how a call's work is cut
// into items, e4m3 conversion, addresses of cache rows.
//
// A tile is BM consecutive (token, query head) rows of one sequence and one
// key/value head. Only the device knows the lengths, so every workgroup derives
// its share of the work from them, in one of two ways:
//
// Items (many rows): a tile's positions are cut into chunks, one item each, with W
// the sum over the tiles of the positions they cover:
//
//   chunk = max(min_chunk, W / target) rounded up to the kernel's step
//
// which gives about target + tiles items. A tile that is cut has fewer than
// 2 * positions / chunk items, so all of them together have fewer than 2 * target.
//
// Shares (few rows, and trees): the positions of all tiles, in units of `step`, form one line
// that is cut into pieces of equal length, one per workgroup (and group of hw heads),
// `target` workgroups in all, or fewer. A piece may hold the end of one tile, whole tiles, and the start of
// another, so every workgroup has the same amount to read, whatever the lengths.
//
// What a workgroup computes of a cut tile goes to the workspace, as does a record
// of the tile; a second launch joins the parts. Neither the parts nor the records
// grow with the batch or the lengths.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace qg {

typedef int i32x2v_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWideBlocks = 8;   // (see attn_share)
constexpr float kSlack = 8.f;    // log2 of how far a weight may exceed its row's reference

// Sums of values by weights of up to 2^8 may leave fp32's range where their mean, the
// result, does not. One pass is enough for accumulators below 2^116: those of four waves
// and 512 parts can be added without a thought. A row with larger ones is computed
// again (by the pass that selects values), its weights divided by a power of two that makes
// their sum over all positions at most 1/4, so that the sums, those of the other parts
// included, stay in range; the reference that goes with them says so.
//
// A weight's exponent is score * c - m in one rounding (c: scale and base), m the rounded
// product of the row's largest score: for that score it is m's rounding error, which no
// longer is about zero once scores pass 2^24, and takes all weights out of range from
// about 2^30 on. A row whose weights' sum has gone far from one is computed again with
// the product rounded in both places alike.
constexpr float kSumsMost = 0x1p116f;
constexpr int kRepeats = 3;   // runs of the pass that selects values: each row may change twice
// m: reference, sum: of the weights that go with it, of all positions (at least one where it
// is finite, but for that error)
__device__ __forceinline__ bool weights_off(float m, float sum) { return m > -INFINITY && !(sum > 0x1p-60f && sum < 0x1p60f); }
struct AttnRepeat {
  bool apart = false;         // exponents with the product rounded by itself
  int shift = 0;              // log2 of what the row's weights are divided by
  __device__ __forceinline__ float exponent(float score, float c, float m) const {
#pragma clang fp contract(off)
    const float x = score * c;
    return apart ? x - m : __builtin_fmaf(score, c, -m);
  }
  __device__ __forceinline__ float weight(float w) const { return __builtin_amdgcn_ldexpf(w, -shift); }
  __device__ __forceinline__ float reference(float m) const { return m + (float)shift; }
  // off: weights_off; large: some accumulator is not below kSumsMost. Whether the row has to
  // be computed again.
  __device__ __forceinline__ bool again(bool off, bool large, int positions) {
    if (off && !apart) {
      apart = true;
      return true;
    }
    if (!large || shift) return false;
    shift = 42 - __builtin_clz(positions);   // weights are 2^8 at most
    return true;
  }
};

// What one workgroup works on.
struct AttnItem {
  int b;            // sequence, -1 past the last item
  int tile;         // tile of the sequence's rows
  int split;        // chunk of the tile's positions
  int slots;        // workspace slot of (b, tile 0, head 0, split 0)
  int nsplit;       // chunks reserved per tile of this sequence
  int chunk;        // positions per chunk
  int row0, fresh, cached;   // the sequence's first row of q, new tokens, history
  int record;       // place of (b, tile) among the tiles of sequences with more than one chunk
};

// A cut tile, for the join: its rows, and where its parts lie. Part 0 of head h is
// slot first + h * head_step, part s > 0 slot next + (s - 1) * step + h * head_step.
struct AttnRecord {
  int parts;             // nothing to join below 2
  int row0, r_first, r_count;
  int first, next, step, head_step;
};

// What is the same in every lane, as the compiler cannot know where it comes from
// LDS or through a call.
__device__ __forceinline__ AttnItem uniform(AttnItem it) {
  it.b = __builtin_amdgcn_readfirstlane(it.b);
  it.tile = __builtin_amdgcn_readfirstlane(it.tile);
  it.split = __builtin_amdgcn_readfirstlane(it.split);
  it.slots = __builtin_amdgcn_readfirstlane(it.slots);
  it.nsplit = __builtin_amdgcn_readfirstlane(it.nsplit);
  it.chunk = __builtin_amdgcn_readfirstlane(it.chunk);
  it.row0 = __builtin_amdgcn_readfirstlane(it.row0);
  it.fresh = __builtin_amdgcn_readfirstlane(it.fresh);
  it.cached = __builtin_amdgcn_readfirstlane(it.cached);
  it.record = __builtin_amdgcn_readfirstlane(it.record);
  return it;
}
template <typename T>
__device__ __forceinline__ T* uniform(T* x) {
  const uint64_t a = reinterpret_cast<uint64_t>(x);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return reinterpret_cast<T*>((uint64_t)hi << 32 | lo);
}
// A condition that is the same in every lane, as a scalar one: an MFMA ignores the
// EXEC mask, so one that is meant to be skipped must be branched around.
__device__ __forceinline__ bool uniform(bool x) { return __builtin_amdgcn_readfirstlane((int)x) != 0; }

// The kernel's arguments, read again from where it got them, by scalar loads: for
// a function that is called, not inlined (a copy of them to pass would be written
// to memory by every lane, and what is loaded through an ordinary pointer would
// not count as the same in every lane).
typedef const __attribute__((address_space(4))) uint32_t* kernarg_t;
__device__ __forceinline__ AttnArgs reload_args(kernarg_t at) {
  static_assert(sizeof(AttnArgs) % 4 == 0, "whole words");
  const uint64_t a = (uint64_t)at;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  const kernarg_t from = (kernarg_t)((uint64_t)hi << 32 | lo);
  AttnArgs p;
  uint32_t w[sizeof(AttnArgs) / 4];
#pragma unroll
  for (int i = 0; i < (int)(sizeof(AttnArgs) / 4); ++i) w[i] = from[i];
  __builtin_memcpy(&p, w, sizeof(p));
  return p;
}

// The workspace: a count of records, the records, the slots. A slot holds a part's
// output rows, then their maxima and sums.
constexpr int kRecordInts = 8;
static_assert(sizeof(AttnRecord) == kRecordInts * 4, "a record's place in the workspace");
__host__ __device__ constexpr long long attn_header_floats(int target) { return (long long)kRecordInts * (target + 16); }
__host__ __device__ constexpr long long attn_slot_floats(int bm, int dp) { return (long long)bm * (dp + 2); }
__device__ __forceinline__ int* attn_record_count(const AttnArgs& p) { return reinterpret_cast<int*>(p.workspace); }
__device__ __forceinline__ AttnRecord* attn_record(const AttnArgs& p, int i) {
  return reinterpret_cast<AttnRecord*>(p.workspace + (size_t)kRecordInts * (i + 1));
}

// x / d for the divisor that (mul, shift) were made for; x < 2^31
__device__ __forceinline__ uint32_t fast_div(uint32_t x, uint32_t mul, uint32_t shift) {
  return (__umulhi(x, mul) + x) >> shift;
}
__device__ __forceinline__ int over_group(const AttnArgs& p, int x) { return (int)fast_div(x, p.group_mul, p.group_shift); }

// Tiles of a sequence, and the positions its longest tile may cover (window_span: the
// window and what a tile's tokens and the rounding of its start add to it).
__device__ __forceinline__ int attn_tiles(const AttnArgs& p, int fresh) { return (fresh * p.group + p.bm - 1) >> p.bm_log2; }
// In a tree every tile may see all drafted tokens, and up to `window` positions before them.
template <bool TREE>
__device__ __forceinline__ int attn_span(const AttnArgs& p, int len, int fresh) {
  if (TREE) return p.window ? (int)min((unsigned)len, (unsigned)p.window + (unsigned)fresh + (unsigned)p.step) : len;
  return p.window ? min(len, p.window_span) : len;
}

template <int NT>
struct AttnScan {
  unsigned long long cost[NT / 64];
  int items[NT / 64], slots[NT / 64], cuts[NT / 64];
  AttnItem found;
};

// Positions per chunk, from the sum over the tiles of the positions they cover
// (target is a power of two).
__device__ __forceinline__ int attn_chunk(const AttnArgs& p, unsigned long long cost) {
  const unsigned long long even = (cost * (unsigned)p.hkv + p.target - 1) >> p.target_log2;
  const int chunk = even < (unsigned long long)p.min_chunk ? p.min_chunk : even > INT32_MAX / 2 ? INT32_MAX / 2 : (int)even;
  return __builtin_amdgcn_readfirstlane((chunk + p.step - 1) & -p.step);
}
__device__ __forceinline__ int attn_chunks(int span, int chunk) { return span <= chunk ? 1 : (span + chunk - 1) / chunk; }

// Item `want` of each head; all NT threads call it. Items are ordered
// by sequence, then chunk, then tile (the last tiles, which see the most positions,
// first). Workgroup 0 also writes the workspace's count of records.
template <int NT>
__device__ __forceinline__ AttnItem attn_locate(const AttnArgs& p, int want, AttnScan<NT>& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (p.batch <= 64) {
    // every wave looks at all sequences, one per lane: no barrier. The longest sequences
    // come first, so that the last workgroups to start have the least to do.
    int row0 = 0, fresh = 0, len = -1;
    if (lane < p.batch) {
      row0 = (int)p.offs[lane];
      fresh = (int)p.offs[lane + 1] - row0;
      len = fresh + (int)p.cache_len[lane];
    }
    const int tiles = attn_tiles(p, fresh), span = attn_span<false>(p, len, fresh);
    unsigned long long all = lane < p.batch ? (unsigned long long)tiles * (unsigned)span : 0;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) all += __shfl_xor(all, d);
    const int chunk = attn_chunk(p, all);
    const int ns = tiles ? attn_chunks(span, chunk) : 0;
    int rank = lane < p.batch ? 0 : lane;
    for (int b = 0; b < p.batch; ++b) {
      const int other = __builtin_amdgcn_readlane(len, b);
      if (lane < p.batch) rank += other > len || (other == len && b < lane);
    }
    const int from = __builtin_amdgcn_ds_permute(4 * rank, lane);   // the sequence of this rank
    const int tl = __shfl(tiles, from), nl = __shfl(ns, from);
    const int items = tl * nl, cuts = nl > 1 ? tl : 0, slots = cuts * nl * p.hkv;
    int ii = items, is = slots, ic = cuts;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int vi = __shfl_up(ii, d), vs = __shfl_up(is, d), vc = __shfl_up(ic, d);
      if (lane >= d) { ii += vi; is += vs; ic += vc; }
    }
    if (blockIdx.x == 0 && tid == 63) *attn_record_count(p) = ic;
    const unsigned long long hit = __ballot(want < ii);
    AttnItem it{};
    it.b = -1;
    if (!hit) return it;
    const int at = __ffsll((long long)hit) - 1;
    auto of = [&](int x) { return __builtin_amdgcn_readlane(x, at); };
    const int local = want - of(ii - items), nt = of(tl);
    it.b = of(from);
    it.split = local / nt;
    it.tile = nt - 1 - (local - it.split * nt);
    it.slots = of(is - slots);
    it.nsplit = of(nl);
    it.chunk = chunk;
    it.row0 = __builtin_amdgcn_readlane(row0, it.b);
    it.fresh = __builtin_amdgcn_readlane(fresh, it.b);
    it.cached = __builtin_amdgcn_readlane(len, it.b) - it.fresh;
    it.record = of(ic - cuts) + it.tile;
    return uniform(it);
  }
  unsigned long long cost = 0;
  int row00 = 0, fresh0 = 0, len0 = 0;
  for (int b0 = 0; b0 < p.batch; b0 += NT) {
    const int b = b0 + tid;
    if (b < p.batch) {
      const int row0 = (int)p.offs[b], fresh = (int)p.offs[b + 1] - row0;
      const int len = fresh + (int)p.cache_len[b];
      if (b0 == 0) { row00 = row0; fresh0 = fresh; len0 = len; }
      cost += (unsigned long long)attn_tiles(p, fresh) * (unsigned)attn_span<false>(p, len, fresh);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) cost += __shfl_xor(cost, d);
  if (lane == 0) sh.cost[wave] = cost;
  if (tid == 0) sh.found.b = -1;
  __syncthreads();
  cost = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) cost += sh.cost[w];
  const int chunk = attn_chunk(p, cost);

  int base = 0, slot_base = 0, cut_base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += NT) {
    const int b = b0 + tid;
    int tiles = 0, ns = 0, row0 = row00, fresh = fresh0, len = len0;
    if (b < p.batch) {
      if (b0 > 0) {
        row0 = (int)p.offs[b];
        fresh = (int)p.offs[b + 1] - row0;
        len = fresh + (int)p.cache_len[b];
      }
      tiles = attn_tiles(p, fresh);
      if (tiles) ns = attn_chunks(attn_span<false>(p, len, fresh), chunk);
    }
    const int items = tiles * ns, cuts = ns > 1 ? tiles : 0, slots = cuts * ns * p.hkv;
    int ii = items, is = slots, ic = cuts;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int vi = __shfl_up(ii, d), vs = __shfl_up(is, d), vc = __shfl_up(ic, d);
      if (lane >= d) { ii += vi; is += vs; ic += vc; }
    }
    if (lane == 63) { sh.items[wave] = ii; sh.slots[wave] = is; sh.cuts[wave] = ic; }
    __syncthreads();
    int bi = base, bs = slot_base, bc = cut_base;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wave) { bi += sh.items[w]; bs += sh.slots[w]; bc += sh.cuts[w]; }
      base += sh.items[w];
      slot_base += sh.slots[w];
      cut_base += sh.cuts[w];
    }
    const int first = bi + ii - items;
    if (want >= first && want < bi + ii) {
      const int local = want - first, tile = tiles - 1 - local % tiles;
      sh.found = AttnItem{b, tile, local / tiles, bs + is - slots, ns, chunk, row0, fresh, len - fresh, bc + ic - cuts + tile};
    }
    __syncthreads();
    if (want < base && blockIdx.x > 0) break;
  }
  if (blockIdx.x == 0 && tid == 0) *attn_record_count(p) = cut_base;
  const AttnItem it = uniform(sh.found);
  return it;
}

// The rows and positions of a tile.
struct AttnTile {
  int r_first, r_count;   // rows of the sequence (token-major)
  int t_first, t_last;    // their tokens
  int begin, end;         // positions that some row sees: [begin, end); of a tree, lie within (see tree_narrow)
  int start;              // begin rounded down
};

// Drafted tokens of a sequence that its rows of the mask have a bit for.
__device__ __forceinline__ int tree_named(const AttnArgs& p, int fresh) { return min(fresh, 32 * p.tree_words); }

template <bool TREE>
__device__ __forceinline__ AttnTile attn_tile(const AttnArgs& p, const AttnItem& it) {
  AttnTile t;
  t.r_first = it.tile << p.bm_log2;
  t.r_count = min(it.fresh * p.group - t.r_first, p.bm);
  t.t_first = over_group(p, t.r_first);
  t.t_last = over_group(p, t.r_first + t.r_count - 1);
  if (TREE) {
    t.end = it.cached + tree_named(p, it.fresh);
    t.begin = p.window ? max(0, it.cached - p.window) : 0;
  } else {
    t.end = p.causal ? it.cached + t.t_last + 1 : it.cached + it.fresh;
    t.begin = p.window ? max(0, it.cached + t.t_first - p.window + 1) : 0;
  }
  t.start = t.begin & -p.step;   // so that the first unit, or chunk, holds a position that is seen (step: a power of two)
  return t;
}

// The low n bits, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u; }

// First position of the history that token `tok` of a tree sees.
__device__ __forceinline__ int tree_low(const AttnArgs& p, const AttnItem& it, int tok) {
  if (!p.window) return 0;
  const uint32_t* words = p.tree + (size_t)(it.row0 + tok) * p.tree_words;
  const int n = tree_named(p, it.fresh);
  int seen = 0;
  for (int w = 0; 32 * w < n; ++w) seen += __popc(words[w] & low_bits(n - 32 * w));
  return max(0, it.cached - max(p.window - seen, 0));
}

// Bit i: whether token `tok` of a tree, whose history begins at `lo`, sees position k0 + i,
// for positions below `end`.
__device__ __forceinline__ uint32_t tree_sees(const AttnArgs& p, const AttnItem& it, int tok, int lo, int k0, int end) {
  const uint32_t* words = p.tree + (size_t)(it.row0 + tok) * p.tree_words;
  const int at = k0 - it.cached, w = at >> 5, most = p.tree_words - 1;   // bit 0 is drafted token `at`
  const uint32_t x = words[min(max(w, 0), most)], y = words[min(max(w + 1, 0), most)];
  const uint64_t both = (uint64_t)(w >= 0 && w <= most ? x : 0u) | (uint64_t)(w + 1 >= 0 && w < most ? y : 0u) << 32;
  const uint32_t drafted = (uint32_t)(both >> (at & 31)) & ~low_bits(-at) & low_bits(min(tree_named(p, it.fresh), end - it.cached) - at);
  const uint32_t history = low_bits(min(it.cached, end) - k0) & ~low_bits(lo - k0);
  return drafted | history;
}

// A row of a tree whose weights sum to nothing is zeros where it sees nothing; where it sees positions,
// all of them with scores of -infinity, it has no softmax: 0 / 0. Wherever parts of a row are joined,
// the latter has a sum of 1, which counts for nothing beside its reference of -infinity, but tells the two apart.
__device__ __forceinline__ float seen_sum(float sum, bool seen) { return sum == 0.f && seen ? 1.f : sum; }
// what its sums are multiplied by; m: reference, sum: as seen_sum says
__device__ __forceinline__ float tree_factor(float m, float sum) { return sum == 0.f ? 0.f : 1.f / (m > -INFINITY ? sum : 0.f); }

// The line's cut into `pieces` shares: the first `extra` have one unit more than `each`.
struct AttnCut {
  uint32_t units, pieces, each, extra;
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * each + min(w, extra); }
  // the share that holds unit u
  __device__ __forceinline__ uint32_t of(uint32_t u) const {
    const uint32_t big = extra * (each + 1);
    return u < big ? u / (each + 1) : extra + (u - big) / each;
  }
};
// A workgroup's share: heads h .. h + hw - 1, units [at, end) of the line (piece w), of
// which `at` is unit `in_tile` of tile `tile` of sequence b; b is -1 where there is none.
struct AttnShare {
  AttnCut cut;
  int h, hw, w;
  uint32_t at, end;
  int b, tile, in_tile;
  int row0, fresh, cached;    // of sequence b
};
// units of each tile of a sequence
template <bool TREE>
__device__ __forceinline__ int attn_units(const AttnArgs& p, int len, int fresh) {
  return (attn_span<TREE>(p, len, fresh) + p.step - 1) >> p.step_log2;
}

template <int NT>
struct ShareScan {
  uint32_t part[NT / 64];
  AttnShare found;
};

// Workgroups go to the eight XCDs in turn: all heads of a piece to one of them, so that
// its L2 gets whole cache rows (and scale lines), not every eighth 256 bytes.
//
// LEAST: units of a share, at least, with one head per workgroup. In the kernel for few rows each wave
// takes blocks of its own, so a share has one for each; in the one for trees all waves work on one block,
// and shares of one are mostly the better ones (against one per wave, bf16: one tree of 13 tokens on 500 13.5
// us against 15.7, 4 of 64 on 1000 42 against 45, 32 of 64 without history 22 against 94, e4m3, 13 on 2000 18
// against 23; but 8 of 13 on 500 29.6 against 25.7).
template <int NT, bool TREE, int LEAST>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& p, ShareScan<NT>& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool one_wave = p.batch <= 64;   // every wave looks at all sequences, one per lane: no barrier
  const int me = one_wave ? lane : tid;
  // a thread's sequences; of up to NT, the prefix sum over them is the total as well
  uint32_t units0 = 0, all = 0;
  int row00 = 0, fresh0 = 0, len0 = 0;
  for (int b0 = 0; b0 < p.batch; b0 += NT) {
    const int b = b0 + me;
    if (b < p.batch) {
      const int row0 = (int)p.offs[b], fresh = (int)p.offs[b + 1] - row0;
      const int len = fresh + (int)p.cache_len[b];
      const uint32_t units = (uint32_t)(attn_tiles(p, fresh) * attn_units<TREE>(p, len, fresh));
      if (b0 == 0) { row00 = row0; fresh0 = fresh; len0 = len; units0 = units; }
      all += units;
    }
  }
  uint32_t incl = all;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  AttnShare s{};
  uint32_t before = 0;
  if (one_wave) {
    s.cut.units = __builtin_amdgcn_readlane(incl, 63);
  } else {
    if (lane == 63) sh.part[wave] = incl;
    if (tid == 0) sh.found.b = -1;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NT / 64; ++v) {
      if (v < wave) before += sh.part[v];
      s.cut.units += sh.part[v];
    }
  }
  s.cut.units = __builtin_amdgcn_readfirstlane(s.cut.units);
  // With much to read, a wave per head and neighbouring heads together (p.hw). With fewer
  // than kWideBlocks blocks per wave, all waves on one head: a quarter of the parts to
  // join (single tokens, bf16, one head against several: 8 sequences of 500 positions 12.7 us
  // against 15.0, 16 of 2000 36 against 34, 32 of 2000 51 against 54, 64 of 1 to 8192 214 against 204).
  const bool wide = (unsigned long long)s.cut.units * (p.hkv / p.hw) >= (unsigned long long)kWideBlocks * p.target;
  s.hw = wide ? p.hw : 1;
  const int groups = wide ? p.hkv / p.hw : p.hkv, least = wide ? 1 : LEAST;
  const uint32_t at8 = blockIdx.x / 8;
  s.h = at8 % groups * s.hw;
  s.w = at8 / groups * 8 + blockIdx.x % 8;
  s.cut.pieces = min((uint32_t)max(p.target / groups, 1), (s.cut.units + least - 1) / least);
  if (blockIdx.x == 0 && tid == 0) *attn_record_count(p) = s.cut.pieces;
  if (s.w >= s.cut.pieces) {
    s.b = -1;
    return s;
  }
  if (s.h == 0 && tid == 0) attn_record(p, s.w)->parts = 0;
  const uint32_t w = s.w;
  s.cut.each = s.cut.units / s.cut.pieces;
  s.cut.extra = s.cut.units % s.cut.pieces;
  s.at = s.cut.start(w);
  s.end = s.cut.start(w + 1);
  if (one_wave) {
    const int at = __ffsll((long long)__ballot(s.at < incl)) - 1;
    const uint32_t local = s.at - __builtin_amdgcn_readlane(incl - all, at);
    s.b = at;
    s.row0 = __builtin_amdgcn_readlane(row00, at);
    s.fresh = __builtin_amdgcn_readlane(fresh0, at);
    s.cached = __builtin_amdgcn_readlane(len0, at) - s.fresh;
    const uint32_t un = attn_units<TREE>(p, s.fresh + s.cached, s.fresh);
    s.tile = local < un ? 0 : local / un;
    s.in_tile = local - s.tile * un;
    return s;
  }
  auto look = [&](int b, uint32_t first, uint32_t units, int row0, int fresh, int len) {
    if (s.at >= first && s.at - first < units) {
      const uint32_t un = attn_units<TREE>(p, len, fresh), local = s.at - first;
      sh.found.b = b;
      sh.found.tile = local / un;
      sh.found.in_tile = local % un;
      sh.found.row0 = row0;
      sh.found.fresh = fresh;
      sh.found.cached = len - fresh;
    }
  };
  if (p.batch <= NT) {
    look(tid, before + incl - all, units0, row00, fresh0, len0);
    __syncthreads();
  } else {
    uint32_t base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += NT) {
      const int b = b0 + tid;
      int row0 = 0, fresh = 0, len = 0;
      uint32_t units = 0;
      if (b < p.batch) {
        row0 = (int)p.offs[b];
        fresh = (int)p.offs[b + 1] - row0;
        len = fresh + (int)p.cache_len[b];
        units = (uint32_t)(attn_tiles(p, fresh) * attn_units<TREE>(p, len, fresh));
      }
      uint32_t run = units;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(run, d);
        if (lane >= d) run += v;
      }
      __syncthreads();
      if (lane == 63) sh.part[wave] = run;
      __syncthreads();
      uint32_t first = base + run - units;
#pragma unroll
      for (int v = 0; v < NT / 64; ++v) {
        if (v < wave) first += sh.part[v];
        base += sh.part[v];
      }
      look(b, first, units, row0, fresh, len);
      __syncthreads();
      if (s.at < base) break;
    }
  }
  s.b = __builtin_amdgcn_readfirstlane(sh.found.b);
  s.tile = __builtin_amdgcn_readfirstlane(sh.found.tile);
  s.in_tile = __builtin_amdgcn_readfirstlane(sh.found.in_tile);
  s.row0 = __builtin_amdgcn_readfirstlane(sh.found.row0);
  s.fresh = __builtin_amdgcn_readfirstlane(sh.found.fresh);
  s.cached = __builtin_amdgcn_readfirstlane(sh.found.cached);
  s.cut.pieces = __builtin_amdgcn_readfirstlane(s.cut.pieces);
  s.cut.each = __builtin_amdgcn_readfirstlane(s.cut.each);
  s.cut.extra = __builtin_amdgcn_readfirstlane(s.cut.extra);
  s.at = s.cut.start(w);
  s.end = s.cut.start(w + 1);
  return s;
}

// The part of a share that lies in the tile it stands at: `take` units, positions [first, end)
// (none where the tile ends before its sequence's longest does), and the workspace's slot for
// them, -1 where they are the whole tile.
struct AttnPart {
  int take, first, end, slot;
};
template <bool TREE>
__device__ __forceinline__ AttnPart attn_part(const AttnArgs& p, const AttnShare& s, const AttnTile& t) {
  const int un = attn_units<TREE>(p, s.fresh + s.cached, s.fresh);   // the tile's units: [first_unit, first_unit + un)
  const uint32_t first_unit = s.at - s.in_tile;
  AttnPart part;
  part.take = min((int)(s.end - s.at), un - s.in_tile);
  // (a tile's first unit may begin with positions, and pages, that nobody sees)
  const int from = t.start + s.in_tile * p.step;
  part.first = max(from, t.begin & ~31);
  part.end = min(t.end, from + part.take * p.step);
  part.slot = -1;
  if (part.first >= part.end) return part;
  const uint32_t last_unit = first_unit + ((t.end - t.start + p.step - 1) >> p.step_log2) - 1;
  const uint32_t begin = s.cut.start(s.w);
  // a share's first part goes to its slot 2 w, its last to 2 w + 1; those between are whole tiles
  if (first_unit < begin || last_unit >= s.end) part.slot = (2 * s.w + (s.at == begin ? 0 : 1)) * p.hkv + s.h;
  if (first_unit < begin && s.h == 0 && threadIdx.x == 0) {
    const int w0 = s.cut.of(first_unit);
    if (s.w == w0 + 1) {                                       // the tile's second share describes it for the join
      const int first = 2 * w0 + (first_unit == s.cut.start(w0) ? 0 : 1);
      *attn_record(p, s.w) = AttnRecord{(int)s.cut.of(last_unit) - w0 + 1, s.row0, t.r_first, t.r_count, first * p.hkv,
                                        2 * s.w * p.hkv, 2 * p.hkv, 1};
    }
  }
  return part;
}
// On to the share's next tile, after `take` units of this one; false at its end.
__device__ __forceinline__ bool attn_next(const AttnArgs& p, AttnShare& s, int take) {
  s.at += take;
  if (s.at >= s.end) return false;
  s.in_tile = 0;
  if (++s.tile == attn_tiles(p, s.fresh)) {            // on to the next sequence that has tiles
    s.tile = 0;
    do {
      ++s.b;
      s.row0 = (int)p.offs[s.b];
      s.fresh = (int)p.offs[s.b + 1] - s.row0;
    } while (s.fresh == 0);
    s.cached = (int)p.cache_len[s.b];
  }
  return true;
}

// the largest of the wave's x
__device__ __forceinline__ int largest(int x) {
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true));    // lane ^ 1
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true));    // lane ^ 2
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true));   // 7 - lane of 8
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true));   // 15 - lane of 16
  return max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
             max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}

// What the rows of a tree's tile see lies in [begin, end): none of the history before `begin`, no
// drafted token from position `end` on; nothing at all where the two are equal. Every wave reads the
// mask for itself: a lane per token, words in turn.
struct TreeRange {
  int begin, end;
};
__device__ __forceinline__ TreeRange tree_range(const AttnArgs& p, const AttnItem& it, const AttnTile& t) {
  const int n = tree_named(p, it.fresh);
  int low = it.cached, top = 0;
  for (int tok = t.t_first + (int)(threadIdx.x & 63); tok <= t.t_last; tok += 64) {
    const uint32_t* words = p.tree + (size_t)(it.row0 + tok) * p.tree_words;
    int seen = 0;
#pragma unroll 4
    for (int w = 0; 32 * w < n; ++w) {
      const uint32_t x = words[w] & low_bits(n - 32 * w);
      seen += __popc(x);
      top = x ? 32 * w + 32 - __clz((int)x) : top;
    }
    low = min(low, p.window ? max(0, it.cached - max(p.window - seen, 0)) : 0);
  }
  return TreeRange{p.window ? it.cached - largest(it.cached - low) : 0, it.cached + largest(top)};
}

// A part of a tree's tile without the positions at its ends that no row sees: their pages need not
// exist. False where that leaves none.
__device__ __forceinline__ bool tree_narrow(const AttnArgs& p, const AttnItem& it, AttnTile& t, AttnPart& part) {
  if (p.window || part.end > it.cached) {   // (without a window, every row sees all of the history)
    const TreeRange seen = tree_range(p, it, t);
    t.begin = seen.begin;
    part.first = max(part.first, t.begin & ~31);
    part.end = min(part.end, seen.end);
  }
  return max(part.first, t.begin) < part.end;
}

// Rows of `heads` heads from h on that see nothing of a part: zeros, or (slot >= 0) a part without weight.
template <int NT, int DP>
__device__ __forceinline__ void store_unseen(const AttnArgs& p, const AttnItem& it, const AttnTile& t, int h, int heads, int slot) {
  for (int e = threadIdx.x; e < heads * t.r_count * (DP / 4); e += NT) {
    const int sub = e / (t.r_count * (DP / 4)), r = e / (DP / 4) % t.r_count, d = e % (DP / 4) * 4;
    if (slot < 0) {
      const int row = t.r_first + r, token = over_group(p, row);
      if (d < p.d)
        *reinterpret_cast<u32x2_t*>(p.out + ((size_t)(it.row0 + token) * p.hq + (h + sub) * p.group + row - token * p.group) * p.d + d) =
            u32x2_t{0, 0};
    } else {
      float* ws = p.workspace + attn_header_floats(p.target) + (size_t)(slot + sub) * attn_slot_floats(p.bm, DP);
      *reinterpret_cast<float4_t*>(ws + (size_t)r * DP + d) = float4_t{0.f, 0.f, 0.f, 0.f};
      if (d == 0) {
        ws[(size_t)p.bm * DP + 2 * r] = -INFINITY;
        ws[(size_t)p.bm * DP + 2 * r + 1] = 0.f;
      }
    }
  }
}

// four e4m3 codes -> four bf16 (exact)
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
  hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
}

// global_load_lds with a 64-bit address per lane: lane l's 16 (4) bytes land at
// LDS byte lds + 16 l (4 l), for the lanes that are active. The issuer counts its
// loads and waits for them with wait_loads.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_at(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(at) : "memory", "m0");
}
__device__ __forceinline__ void dma4_at(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(at) : "memory", "m0");
}
#pragma clang diagnostic pop

// Makes the compiler wait here for what it loads into x itself. Its waits count
// only the loads it knows of: left to the first use inside a loop, one would wait
// for the loop's direct-to-LDS loads as well, in every iteration.
__device__ __forceinline__ void arrived(u32x4_t& x) { asm volatile("" : "+v"(x)); }

// until at most N of this wave's vector-memory loads are in flight
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// until the loads of at most min(left, N) blocks of LB loads each are in flight
template <int LB, int N>
__device__ __forceinline__ void wait_blocks(int left) {
  if constexpr (N == 0) {
    wait_loads<0>();
  } else {
    if (left >= N) wait_loads<N * LB>();
    else wait_blocks<LB, N - 1>(left);
  }
}

// until this wave's LDS reads have returned (before a load into the same place)
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// LDS byte address, the same in every lane: the low half of a generic pointer into
// LDS (a cast of the pointer itself would first test it for null)
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(p));
}

// the larger of x and the other half-wave's x
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  const uint32_t a = r[0], b = r[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
// the larger of x in lanes l and l ^ 16
__device__ __forceinline__ float max_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  const uint32_t a = r[0], b = r[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// Where some values are infinities or NaN they enter a product of their own, with weights
// of one where the row sees the position: the result is theirs however small the weight
// (an infinity times a weight that has vanished would be NaN). finite(v): eight bf16 with
// zero in place of them.
__device__ __forceinline__ u32x4_t finite(u32x4_t v) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = v[i];
    r[i] = ((x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) | ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u);
  }
  return r;
}
// x where it is an infinity or NaN, else x * f
__device__ __forceinline__ float times(float x, float f) { return fabsf(x) < INFINITY ? x * f : x; }

// eight transposed bf16 rows x 16 columns: see the kernels for the lanes' order
__device__ __forceinline__ uint64_t lds_read_tr16(const void* p) {
  return __builtin_bit_cast(uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                          (__attribute__((address_space(3))) s16x4_t*)(const_cast<void*>(p))));
}
__device__ __forceinline__ uint64_t lds_read_tr8(const void* p) {
  return __builtin_bit_cast(uint64_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                          (__attribute__((address_space(3))) i32x2v_t*)(const_cast<void*>(p))));
}

// The pages of a tile's positions where page_size is a multiple of 16: 16 aligned
// positions lie in one page, whose id is a scalar load.
typedef const __attribute__((address_space(4))) uint32_t* page_list_t;
struct Row16 {
  size_t row;    // cache row (page, slot) of the first of 16 positions
  int pos;       // that position
};
// of positions pos0 .. pos0 + 15, or where all of these lie outside [begin, end) of 16
// others that do not (their pages may not exist)
__device__ __forceinline__ Row16 rows_of16(const AttnArgs& p, page_list_t pages, int pos0, int begin, int end) {
  const int x = min(max(pos0, begin & ~15), (end - 1) & ~15);
  const uint32_t pg = fast_div(x, p.div_mul, p.div_shift);
  return Row16{(size_t)pages[pg] * p.page_size + (x - pg * p.page_size), x};
}

// Sets what launch_attention_rows goes by: `target`, the workgroups that run at once,
// and `hw`, the heads per workgroup.
void attention_rows_shape(AttnArgs& p, int mt);
hipError_t launch_attention_rows(const AttnArgs& p, int mt, unsigned grid, hipStream_t stream);
hipError_t launch_attention_rows_tree(const AttnArgs& p, int mt, unsigned grid, hipStream_t stream);
hipError_t launch_attention_tiles(const AttnArgs& p, unsigned grid, hipStream_t stream);
// The same for trees with many rows: rows per tile, and workgroups that run at once. Tiles have 128
// rows: TREE_FEW with the weights' remainders on bf16 caches, TREE_TALL 256 where there are such instances.
enum TreeTiles { TREE_FEW, TREE_MANY, TREE_TALL };
void attention_tree_shape(AttnArgs& p, TreeTiles tiles);
hipError_t launch_attention_tree(const AttnArgs& p, TreeTiles tiles, unsigned grid, hipStream_t stream);

}  // namespace qg
