// Attention over the paged cache for many rows per key/value head (prompts and
// chunks of prompts), bound by the matrix cores.
//
//   s_i = scale * sum_d q[d] * k_i[d]          over the positions i a row sees
//   out = sum_i e^(s_i - m) v_i / sum_i e^(s_i - m)
//
// The rows of a tile are 128 consecutive (token, query head) pairs of one
// key/value head, token-major, so its pages are read once for all query heads
// that share them. Each of four waves owns 32 rows and computes the scores
// transposed, S^T = K Q^T with 32x32x16 MFMAs: a lane then holds scores of one
// row only, the running maximum and sum need one exchange with the other half of
// the wave, and the probabilities are already the B operand of O^T = V^T P^T (the
// key slots of that product come in the order the scores lie in, and the
// transposed reads of V name the same order). Keys and values pass through LDS,
// two blocks deep, as bf16: straight from memory (direct-to-LDS loads) or, from
// an e4m3 cache, through registers that convert the codes.
//
// The running maximum is a reference, not the maximum itself: the output
// accumulators are rescaled only when a row's scores exceed it by more than 2^8
// in weight, which after a row's first blocks hardly ever happens.
//
// Numbers: products of bf16 are summed in fp32; e4m3 codes enter as bf16
// (exact), a key's scale multiplies the fp32 partial score of its run and a
// value's scale its probability in fp32. Maximum, sum and output accumulators
// are fp32. The one rounding inside is that of the probabilities to bf16, which
// the MFMA takes (at most 2^-8 of each, as the output's own rounding).
//
// Measured (heads of 128, 32 on 8): a prompt of 8192 in 528 us, 1041 TFLOP/s over the
// pairs that see each other; 1000 tokens after a history of 32000 in 512 us, 1039 TFLOP/s
// (a large bf16 library product: 1.15 to 1.22 PFLOP/s); eight prompts of 1 to 1024 tokens
// 42 us. 64 rows per wave, which would halve the LDS reads, leaves one wave per SIMD
// and accumulators that the compiler moves in and out of AGPRs: 280 TFLOP/s.
// e4m3 caches reach 604 TFLOP/s (0.26 ms for eight chunks of 1 to 1024 tokens on up to
// 4096; runs of 64 0.32 ms, of 32 0.41): MFMA busy 25 %, VALU 36 %; codes wait in registers
// between a block's loads and its conversion, and a quarter of the time passes with
// workgroups that have ended (uncut tiles of unequal length). Page numbers looked up a
// block ahead did not shorten it (0.30 ms). Heads of 256 reach 449 TFLOP/s (e4m3 chunks
// 0.81 ms, runs of 64 1.04, of 32 1.27): 128 accumulators and 64 query registers leave
// one wave per SIMD, and nothing covers its LDS latencies (a ring of four blocks: 324 -> 355 us).
//
// A position that a row must not see takes a score of -infinity by selection.
// Its value row is still multiplied, by zero: where it holds an infinity or NaN
// the row's output would turn NaN. So a tile whose accumulators are not finite, or so
// large that sums of them may not be, is computed again with the values selected per
// token (and, where that does not help, other weights: AttnRepeat).
#pragma once

#include "attention_common.h"

namespace qg {

namespace {

constexpr int TPG = 1024;            // page table entries held in LDS at a time

// 16-byte chunk c of LDS row r (DP bf16 elements) lies at c ^ swz(r): the 16 rows of a
// read phase of the key fragments, and the 4 x 64 bytes of a transposed read of
// values, meet different banks
template <int DP>
__device__ __forceinline__ int swz_t(int r) {
  return DP >= 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
}

}  // namespace

// LDS of a workgroup of AW waves. KB: positions per block.
template <int DP, int GRAN, int AW, int KB>
struct AttnTileLds {
  static constexpr int R = GRAN > 0 ? DP / GRAN : 1;        // scale runs per head, at most
  __attribute__((aligned(16))) u32x4_t ring[2][2][KB * DP / 8];                                   // [block parity][keys, values]
  __attribute__((aligned(16))) float ring_s[GRAN > 0 ? 2 : 1][2][R][GRAN > 0 ? KB : 1];   // [keys, values][run][position]
  uint32_t pages[TPG];
  int w_off[AW];
  AttnScan<AW * 64> scan;
};

// What eight weights lose as the bf16 pairs r.
__device__ __forceinline__ u32x4_t remainders(const float (&w)[8], u32x4_t r) {
#pragma clang fp contract(off)   // the same remainder whatever the code around it: not one of an unrounded product
  u32x4_t rest;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t v = r[g];
    rest[g] = f2bf2_rn(w[2 * g] - bf2f((uint16_t)v), w[2 * g + 1] - bf2f((uint16_t)(v >> 16)));
  }
  return rest;
}

// A wave's rows: the result, or (slot >= 0) the part of it with its reference and sum (of a tree: seen_sum).
template <int DP, bool TREE>
__device__ __forceinline__ void store_tile(const AttnArgs& p, const AttnItem& it, const AttnTile& t, int h, int slot,
                                           const float16_t (&acc)[DP / 32], float m, float sum) {
  constexpr int ND = DP / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  float* ws = p.workspace + attn_header_floats(p.target) + (size_t)slot * attn_slot_floats(p.bm, DP);
  const int r = wave * 32 + col;
  if (r >= t.r_count) return;
  if (slot < 0) {
    const float inv = TREE ? tree_factor(m, sum) : 1.f / sum;
    const int row = t.r_first + r, token = over_group(p, row);
    uint16_t* to = p.out + ((size_t)(it.row0 + token) * p.hq + h * p.group + row - token * p.group) * p.d;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = n * 32 + 8 * g + 4 * half;
        if (d < p.d)
          *reinterpret_cast<u32x2_t*>(to + d) = u32x2_t{f2bf2_rn(acc[n][4 * g] * inv, acc[n][4 * g + 1] * inv),
                                                        f2bf2_rn(acc[n][4 * g + 2] * inv, acc[n][4 * g + 3] * inv)};
      }
  } else {
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4_t*>(ws + (size_t)r * DP + n * 32 + 8 * g + 4 * half) =
            float4_t{acc[n][4 * g], acc[n][4 * g + 1], acc[n][4 * g + 2], acc[n][4 * g + 3]};
    if (half == 0) {
      ws[(size_t)p.bm * DP + 2 * r] = m;
      ws[(size_t)p.bm * DP + 2 * r + 1] = sum;
    }
  }
}

// Positions [c_first, c_end) of one tile, which are all of them where `slot` is -1 and go to
// that slot of the workspace else. GRAN: head-dim elements per scale of an e4m3 cache, 0
// for bf16. SAFE: values are selected per token. Returns whether some row has to be computed
// again (without SAFE: sums are too large, infinities, NaN or zero; with it: as `rep`, the
// state of this lane's row, says), for the whole workgroup, and then has written nothing. REST (bf16): what
// the weights lose to bf16 is multiplied with the values too.
template <int DP, int GRAN, int AW, int KB, bool SAFE, bool TREE, bool REST>
__device__ __forceinline__ bool attend_tile(const AttnArgs& p, const AttnItem& it, const AttnTile& t, int h, int c_first, int c_end,
                                            int slot, AttnTileLds<DP, GRAN, AW, KB>& lds, AttnRepeat& rep) {
  constexpr bool FP8 = GRAN > 0;
  constexpr int NT = AW * 64;
  constexpr int NB = KB / 32;
  constexpr int NS = DP / 16;                 // MFMA steps of a score
  constexpr int ND = DP / 32;                 // 32-wide strips of the output
  constexpr int CH = DP / 8;                  // 16-byte chunks per LDS row
  constexpr int TILE = KB * CH;
  constexpr int LD = TILE / NT;               // direct loads per lane for the keys (or values) of a block
  constexpr int R = AttnTileLds<DP, GRAN, AW, KB>::R;
  constexpr int RS = FP8 ? GRAN / 16 : NS;    // MFMA steps per run
  constexpr int LC = FP8 ? DP / 16 : 1;       // e4m3: 16-code loads per row
  constexpr int LQ = FP8 ? KB * LC / NT : 0;  // e4m3: loads per thread for the keys (or values)
  constexpr int LS = FP8 ? (2 * KB * R + NT - 1) / NT : 0;   // scales per thread
  static_assert(LD >= 1 && (!FP8 || LQ >= 1), "a block is at least one load of every thread");
  auto& ring = lds.ring;
  auto& ring_s = lds.ring_s;
  auto& pages = lds.pages;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;

  const int rows = it.fresh * p.group;
  const int my_row = min(t.r_first + wave * 32 + col, rows - 1), tok = over_group(p, my_row);
  const int hi = p.causal ? it.cached + tok : it.cached + it.fresh - 1;
  const int lo = TREE ? tree_low(p, it, tok) : p.window ? it.cached + tok - p.window + 1 : 0;
  const uint16_t* q = p.q + ((size_t)(it.row0 + tok) * p.hq + h * p.group + my_row - tok * p.group) * p.d;
  u32x4_t qf[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int d = 16 * s + 8 * half;
    qf[s] = d < p.d ? *reinterpret_cast<const u32x4_t*>(q + d) : u32x4_t{0, 0, 0, 0};
  }
#pragma unroll
  for (int s = 0; s < NS; ++s) arrived(qf[s]);
  const float cs = p.scale * kLog2e;
  const int runs = FP8 ? p.d / (FP8 ? GRAN : 1) : 1;
  const int chunks = p.d / 8;                                 // chunks of an LDS row that exist
  if (chunks < CH) {                                          // the others are zero from here on
    for (int e = tid; e < 4 * TILE; e += NT) (&ring[0][0][0])[e] = u32x4_t{0, 0, 0, 0};
  }
  const size_t row_bytes = (size_t)p.hkv * p.d * (FP8 ? 1 : 2);   // a (page, slot) row
  const size_t plane_bytes = (size_t)p.pages * p.page_size * row_bytes;
  const char* keys = static_cast<const char*>(p.blocks) + 2 * p.layer * plane_bytes + (size_t)h * p.d * (FP8 ? 1 : 2);
  const size_t plane_scales = (size_t)p.pages * p.page_size * p.hkv * runs;
  const float* key_scales = FP8 ? p.scales + 2 * p.layer * plane_scales + (size_t)h * runs : nullptr;
  const uint32_t* my_pages = p.page_table + (size_t)it.b * p.max_pages;
  const int row_scales = p.hkv * runs;
  const bool by16 = p.page_size % 16 == 0;
  // Where this lane's loads of a block come from, within 16 positions of one page. bf16:
  // LDS position e = 64 (LD wave + k) + lane is row e / CH, chunk e % CH; e4m3: load k is
  // row (k NT + tid) / LC, codes 16 ((k NT + tid) % LC) .. + 15.
  constexpr int NV = FP8 ? LQ : LD;
  const int e0 = FP8 ? tid : wave * LD * 64 + lane, ek = FP8 ? NT : 64, er = FP8 ? LC : CH;
  uint32_t voff[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = e0 + k * ek, key = e / er, c = FP8 ? min(e % er * 16, p.d - 16) : ((e % er) ^ swz_t<DP>(key)) * 16;
    voff[k] = (key & 15) * (uint32_t)row_bytes + c;
  }

  float16_t acc[ND];
  float m = -INFINITY, l = 0.f;   // reference of the weights' exponents (base 2), this lane's share of their sum
  float sum;                      // the row's
  uint32_t seen = 0;              // in a tree: not 0 where the row has seen a position
  {
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][i] = 0.f;
    // as many positions at a time as the list of pages covers
    const int seg = by16 ? c_end - c_first : (int)min((long long)(c_end - c_first), (long long)(TPG - 1) * p.page_size / KB * KB);
    for (int s_first = c_first; s_first < c_end; s_first += seg) {
      const int s_end = min(c_end, s_first + seg);
      const int page0 = by16 ? 0 : fast_div(max(s_first, t.begin), p.div_mul, p.div_shift);
      if (!by16) {
        const int page1 = fast_div(s_end - 1, p.div_mul, p.div_shift);
        __syncthreads();
        for (int e = tid; e <= page1 - page0; e += NT) pages[e] = my_pages[page0 + e];
      }
      if (!by16 || chunks < CH) __syncthreads();

      // positions outside [begin, end) re-read one inside (their pages may not exist)
      auto row_of = [&](int pos) {
        const int x = min(max(pos, t.begin), s_end - 1);
        const uint32_t pg = fast_div(x, p.div_mul, p.div_shift);
        return (size_t)pages[pg - page0] * p.page_size + (x - pg * p.page_size);
      };
      // an offset of voff, for a position that is not in [begin, s_end)
      auto clamped = [&](const Row16& r, int k) {
        const int e = e0 + k * ek, key = e / er;
        const int x = min(max(r.pos + (key & 15), t.begin), s_end - 1) - r.pos;
        return voff[k] + (x - (key & 15)) * (uint32_t)row_bytes;
      };
      // bf16: block i on its way into ring[at]
      auto issue = [&](int i, int at) {
        const int first = s_first + KB * i;
        if (by16) {
          // a wave loads 16 positions (8 where a block has 32): one page
          const int mine = wave * (KB / AW) & ~15;
          const Row16 r = rows_of16(p, (page_list_t)my_pages, first + mine, t.begin, s_end);
          const char* kbase = uniform(keys + r.row * row_bytes);
          const char* vbase = uniform(kbase + plane_bytes);
          const bool inside = first + mine >= t.begin && first + mine + 16 <= s_end;
#pragma unroll
          for (int k = 0; k < LD; ++k) {
            const int e = (wave * LD + k) * 64;
            const uint32_t off = inside ? voff[k] : clamped(r, k);
            if (((e + lane) % CH ^ swz_t<DP>((e + lane) / CH)) < chunks) {
              dma16(kbase, off, lds_addr(&ring[at][0][e]));
              dma16(vbase, off, lds_addr(&ring[at][1][e]));
            }
          }
          return;
        }
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const int e = (wave * LD + k) * 64, key = (e + lane) / CH, c = (e + lane) % CH ^ swz_t<DP>(key);
          const char* src = keys + row_of(first + key) * row_bytes + c * 16;
          if (c < chunks) {
            dma16_at(src, lds_addr(&ring[at][0][e]));
            dma16_at(src + plane_bytes, lds_addr(&ring[at][1][e]));
          }
        }
      };
      // e4m3: block i into registers, and from there into ring[at]
      u32x4_t stage[2][FP8 ? LQ : 1];
      float stage_s[FP8 ? LS : 1];
      auto fetch = [&](int i) {
        const int first = s_first + KB * i;
        if (by16) {
          Row16 r[KB / 16];
#pragma unroll
          for (int g = 0; g < KB / 16; ++g) r[g] = rows_of16(p, (page_list_t)my_pages, first + 16 * g, t.begin, s_end);
          const bool inside = first >= t.begin && first + KB <= s_end;
#pragma unroll
          for (int k = 0; k < LQ; ++k) {
            constexpr int PER = 64 / LC;   // positions of a wave's load
            const int g = (k * (NT / LC) + wave * PER) >> 4;
            Row16 rk = r[0];
#pragma unroll
            for (int u = 1; u < KB / 16; ++u)
              if (g == u) rk = r[u];
            const char* base = uniform(keys + rk.row * row_bytes);
            const uint32_t off = inside ? voff[k] : clamped(rk, k);
            stage[0][k] = *reinterpret_cast<const u32x4_t*>(base + off);
            stage[1][k] = *reinterpret_cast<const u32x4_t*>(base + plane_bytes + off);
          }
#pragma unroll
          for (int k = 0; k < LS; ++k) {
            const int e = min(k * NT + tid, 2 * KB * R - 1), plane = e / (KB * R), run = e / KB % R, key = e % KB;
            Row16 rk = r[0];
#pragma unroll
            for (int u = 1; u < KB / 16; ++u)
              if (key >> 4 == u) rk = r[u];
            const int x = min(max(rk.pos + (key & 15), t.begin), s_end - 1) - rk.pos;
            stage_s[k] = key_scales[plane * plane_scales + (rk.row + x) * row_scales + min(run, runs - 1)];
          }
          return;
        }
#pragma unroll
        for (int k = 0; k < LQ; ++k) {
          const int e = k * NT + tid, key = e / LC, c = e % LC;
          const char* src = keys + row_of(first + key) * row_bytes + min(c * 16, p.d - 16);
          stage[0][k] = *reinterpret_cast<const u32x4_t*>(src);
          stage[1][k] = *reinterpret_cast<const u32x4_t*>(src + plane_bytes);
        }
#pragma unroll
        for (int k = 0; k < LS; ++k) {
          const int e = min(k * NT + tid, 2 * KB * R - 1), plane = e / (KB * R), run = e / KB % R, key = e % KB;
          stage_s[k] = key_scales[plane * plane_scales + row_of(first + key) * row_scales + min(run, runs - 1)];
        }
      };
      auto store = [&](int at) {
#pragma unroll
        for (int k = 0; k < LQ; ++k) {
          const int e = k * NT + tid, key = e / LC, c = e % LC;
          if (c * 16 >= p.d) continue;
#pragma unroll
          for (int plane = 0; plane < 2; ++plane) {
            uint32_t o[8];
#pragma unroll
            for (int g = 0; g < 4; ++g) e4m3x4_to_bf16(stage[plane][k][g], o[2 * g], o[2 * g + 1]);
            const int z = swz_t<DP>(key);
            ring[at][plane][key * CH + ((2 * c) ^ z)] = u32x4_t{o[0], o[1], o[2], o[3]};
            ring[at][plane][key * CH + ((2 * c + 1) ^ z)] = u32x4_t{o[4], o[5], o[6], o[7]};
          }
        }
#pragma unroll
        for (int k = 0; k < LS; ++k)
          if (k * NT + tid < 2 * KB * R) (&ring_s[at][0][0][0])[k * NT + tid] = stage_s[k];
      };

      const int blocks = (s_end - s_first + KB - 1) / KB;
      if constexpr (FP8) {
        fetch(0);
        store(0);
      } else {
        issue(0, 0);
      }
      int at = 0;
      for (int i = 0; i < blocks; ++i, at ^= 1) {
        if constexpr (!FP8) wait_loads<0>();
        __syncthreads();             // block i is in LDS; nobody reads the other half any more
        if (i + 1 < blocks) {
          if constexpr (FP8) fetch(i + 1);
          else issue(i + 1, at ^ 1);
        }
        const int k0 = s_first + KB * i;
        const u32x4_t* lk = ring[at][0];
        const char* lv = reinterpret_cast<const char*>(ring[at][1]);

        // Two workgroups share a CU (bf16, heads up to 128): the one at its MFMAs goes first, so
        // that the other's softmax fills in behind it instead of beside it (prompt of 8192:
        // 589 -> 569 us; with e4m3's longer softmax, or one workgroup per CU, it costs 1 to 6 %).
        constexpr bool FIRST = !FP8 && DP <= 128;
        if constexpr (FIRST) __builtin_amdgcn_s_setprio(1);
        // scores: register i of block nb holds position k0 + 32 nb + 8 (i / 4) + 4 half + i % 4
        float16_t sc[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int key = nb * 32 + col;
          float16_t part;
#pragma unroll
          for (int e = 0; e < 16; ++e) part[e] = 0.f;
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const u32x4_t kf = lk[key * CH + ((2 * s + half) ^ swz_t<DP>(key))];
            part = mfma32x32x16_bf16(kf, qf[s], part);
            if constexpr (FP8) {
              if ((s + 1) % RS == 0) {   // a run is complete: times the keys' scales
                const int run = (s + 1) / RS - 1;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  const float4_t ks = *reinterpret_cast<const float4_t*>(&ring_s[at][0][run][nb * 32 + 8 * g + 4 * half]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    sc[nb][4 * g + e] =
                        run == 0 ? part[4 * g + e] * ks[e] : __builtin_fmaf(part[4 * g + e], ks[e], sc[nb][4 * g + e]);
                    part[4 * g + e] = 0.f;
                  }
                }
                // Runs of one or two pairs of MFMAs: finished before the next run begins. Left
                // alone, the compiler keeps a set of partial scores per run and spills (eight
                // chunks of 1 to 1024 tokens, runs of 32: 2.37 -> 0.41 ms; of 64: 0.62 -> 0.33;
                // heads of 256: 4.36 -> 1.30, 1.44 -> 1.10). Runs of 128 have room for two
                // (heads of 256: 0.88 ms, and 0.95 in turn).
                if constexpr (R > 1 && GRAN < 128) {
                  asm volatile("" : "+v"(sc[nb]));
                  __builtin_amdgcn_sched_barrier(0);
                }
              }
            }
          }
          if constexpr (!FP8) sc[nb] = part;
        }
        if constexpr (FIRST) __builtin_amdgcn_s_setprio(0);
        // in a tree: the drafted tokens, and where windows begin, somewhere before them
        const bool masked = TREE ? uniform((p.window && k0 < min(it.cached, t.end - p.window)) || k0 < t.begin || k0 + KB > min(s_end, it.cached))
                                 : uniform((p.window && k0 < it.cached + t.t_last - p.window + 1) || k0 < t.begin ||
                                           k0 + KB > min(s_end, p.causal ? it.cached + t.t_first + 1 : t.end));
        uint32_t vis[TREE ? NB : 1];   // bit 8 (e / 4) + e % 4 of position e of 16 that the row sees
        if constexpr (TREE) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            vis[nb] = ~0u;
            if (masked) {
              vis[nb] = tree_sees(p, it, tok, lo, k0 + 32 * nb, s_end) >> (4 * half);
#pragma unroll
              for (int e = 0; e < 16; ++e) sc[nb][e] = vis[nb] >> (8 * (e / 4) + e % 4) & 1 ? sc[nb][e] : -INFINITY;
            }
            seen |= vis[nb];
          }
        } else if (masked) {
          // positions lo .. min(hi, s_end - 1), counted from lo
          const uint32_t seen = max(min(hi, s_end - 1) - lo + 1, 0), first = k0 + 4 * half - lo;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              sc[nb][e] = first + (nb * 32 + 8 * (e / 4) + e % 4) < seen ? sc[nb][e] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 16; ++e) mx = fmaxf(mx, sc[nb][e]);
        mx = max_halves(mx) * cs;
        const bool more = mx > m + kSlack;   // (-infinity: the row has seen nothing yet)
        if (__any(more)) {
          // only a row's own scores move its reference: its result is the same whatever the others see
          const float alpha = more ? __builtin_amdgcn_exp2f(m - mx) : 1.f;
          m = more ? mx : m;
          l *= alpha;
#pragma unroll
          for (int n = 0; n < ND; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[n][e] = SAFE ? times(acc[n][e], alpha) : acc[n][e] * alpha;
        }
        // a row that has seen nothing yet keeps -infinity; its weights are 0
        const float base = m == -INFINITY ? 0.f : m;
        float l_block = 0.f;
        uint32_t sees = 0;   // SAFE: bit 16 nb + e of positions whose weight is more than zero, be it too small for fp32
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (SAFE) sees |= (uint32_t)(sc[nb][e] > -INFINITY) << (16 * nb + e);
            sc[nb][e] = __builtin_amdgcn_exp2f(SAFE ? rep.exponent(sc[nb][e], cs, base) : __builtin_fmaf(sc[nb][e], cs, -base));
            if (SAFE) sc[nb][e] = rep.weight(sc[nb][e]);
            l_block += sc[nb][e];
          }
        l += l_block;

        // weights of 16 positions as the B operand, and REST's of them; key slots 0..3 are key0 + 0..3, 4..7 key0 + 8..11
        auto weights = [&](int nb, int ks, int run, u32x4_t& rest) {
          float w[8];
          const int key0 = nb * 32 + ks * 16 + 4 * half;
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = sc[nb][8 * ks + e];
          if constexpr (FP8) {   // times the value scales of the strip's run
            const float4_t v0 = *reinterpret_cast<const float4_t*>(&ring_s[at][1][run][key0]);
            const float4_t v1 = *reinterpret_cast<const float4_t*>(&ring_s[at][1][run][key0 + 8]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float v = e < 4 ? v0[e] : v1[e - 4];
              if (!SAFE) {
                w[e] *= v;
              } else {   // the scale of a position that the row does not see may be an infinity or NaN
                const int pos = k0 + key0 + e % 4 + 8 * (e / 4);
                const bool far = !(fabsf(v) < INFINITY) && (sees >> (16 * nb + 8 * ks + e) & 1);
                const bool hidden = TREE ? !(vis[TREE ? nb : 0] >> (16 * ks + 8 * (e / 4) + e % 4) & 1) : pos > hi || pos < lo || pos >= s_end;
                w[e] = hidden ? 0.f : far ? v : w[e] * v;
              }
            }
          }
          const u32x4_t r = {f2bf2_rn(w[0], w[1]), f2bf2_rn(w[2], w[3]), f2bf2_rn(w[4], w[5]), f2bf2_rn(w[6], w[7])};
          if constexpr (REST) rest = remainders(w, r);
          return r;
        };
        // V^T fragment of strip n: lane m of a 16-lane group names row m / 4 of four and
        // elements 4 (m % 4) .. + 3 of 16, and receives the four rows of column m
        auto values = [&](int nb, int ks, int n) {
          const int m16 = lane & 15, c0 = n * 32 + 16 * ((lane >> 4) & 1) + 4 * (m16 & 3);
          const int key = nb * 32 + ks * 16 + 4 * half + (m16 >> 2);
          const uint64_t w0 = lds_read_tr16(lv + (key * CH + ((c0 >> 3) ^ swz_t<DP>(key))) * 16 + (c0 & 7) * 2);
          const uint64_t w1 = lds_read_tr16(lv + ((key + 8) * CH + ((c0 >> 3) ^ swz_t<DP>(key + 8))) * 16 + (c0 & 7) * 2);
          return u32x4_t{(uint32_t)w0, (uint32_t)(w0 >> 32), (uint32_t)w1, (uint32_t)(w1 >> 32)};
        };
        // SAFE: the product of strip n's values vf with the weights, infinities and NaN apart
        auto product = [&](u32x4_t vf, u32x4_t pf, u32x4_t rest, int nb, int ks, float16_t sum) {
          uint32_t one[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) one[e] = sees >> (16 * nb + 8 * ks + e) & 1 ? 0x3F80u : 0u;
          const u32x4_t of = {one[0] | one[1] << 16, one[2] | one[3] << 16, one[4] | one[5] << 16, one[6] | one[7] << 16};
          const u32x4_t v = finite(vf);
          sum = mfma32x32x16_bf16(v, pf, sum);
          if constexpr (REST) sum = mfma32x32x16_bf16(v, rest, sum);
          return mfma32x32x16_bf16(vf ^ v, of, sum);
        };
        if constexpr (FIRST) __builtin_amdgcn_s_setprio(1);
        if (!SAFE || !masked) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              u32x4_t pf, rest = {};
#pragma unroll
              for (int n = 0; n < ND; ++n) {
                if (n == 0 || (FP8 && n * 32 % (FP8 ? GRAN : 1) == 0)) pf = weights(nb, ks, FP8 ? n * 32 / (FP8 ? GRAN : 1) : 0, rest);
                const u32x4_t vf = values(nb, ks, n);
                acc[n] = SAFE ? product(vf, pf, rest, nb, ks, acc[n]) : mfma32x32x16_bf16(vf, pf, acc[n]);
              }
            }
        } else {
          // token by token, with the values it does not see set to zero
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
              for (int n = 0; n < ND; ++n) {
                const u32x4_t vf = values(nb, ks, n);
                u32x4_t rest = {};
                const u32x4_t pf = weights(nb, ks, FP8 ? n * 32 / (FP8 ? GRAN : 1) : 0, rest);
#pragma unroll 1
                for (int tt = t.t_first; tt <= t.t_last; ++tt) {
                  const int t_hi = p.causal ? it.cached + tt : it.cached + it.fresh - 1;
                  const int t_lo = p.window ? it.cached + tt - p.window + 1 : 0;
                  const uint32_t t_vis = TREE ? tree_sees(p, it, tt, tree_low(p, it, tt), k0 + nb * 32, s_end) >> (16 * ks + 4 * half) : 0u;
                  uint32_t keep[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const int pos = k0 + nb * 32 + ks * 16 + 4 * half + e % 4 + 8 * (e / 4);
                    const bool kept = TREE ? t_vis >> (8 * (e / 4) + e % 4) & 1 : pos <= t_hi && pos >= t_lo && pos < s_end;
                    keep[e] = kept ? 0xFFFFu : 0u;
                  }
                  const u32x4_t vs = {vf.x & (keep[0] | keep[1] << 16), vf.y & (keep[2] | keep[3] << 16),
                                      vf.z & (keep[4] | keep[5] << 16), vf.w & (keep[6] | keep[7] << 16)};
                  const float16_t with = product(vs, pf, rest, nb, ks, acc[n]);
#pragma unroll
                  for (int e = 0; e < 16; ++e) acc[n][e] = tt == tok ? with[e] : acc[n][e];
                }
              }
        }
        if constexpr (FIRST) __builtin_amdgcn_s_setprio(0);
        if constexpr (FP8) {
          if (i + 1 < blocks) store(at ^ 1);
        }
      }
    }
    int off = 0;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) off |= !(fabsf(acc[n][e]) < kSumsMost);
    sum = l + __shfl_xor(l, 32);
    if (SAFE) off = rep.again(weights_off(m, sum), off | __shfl_xor(off, 32), t.end - t.start);
    else off |= weights_off(m, sum);
    off = __any(off);
    if (lane == 0) lds.w_off[wave] = off;
    __syncthreads();
    off = 0;
#pragma unroll
    for (int w = 0; w < AW; ++w) off |= lds.w_off[w];
    if (uniform(off != 0)) return true;   // a scalar branch: the accumulators are not live across the call behind it
  }

  if (TREE) sum = seen_sum(sum, (seen | __shfl_xor(seen, 32)) != 0);
  store_tile<DP, TREE>(p, it, t, h, slot, acc, SAFE ? rep.reference(m) : m, sum);
  return false;
}

// Called, not inlined: hardly ever taken, and its registers stay out of the kernel's.
template <int DP, int GRAN, int AW, int KB, bool TREE, bool REST>
__device__ __attribute__((noinline)) void attend_tile_safe(kernarg_t args, AttnItem it, int h, int c_first, int c_end, int slot,
                                                           AttnTileLds<DP, GRAN, AW, KB>* lds) {
  const AttnArgs p = reload_args(args);
  const AttnItem item = uniform(it);
  AttnTile t = attn_tile<TREE>(p, item);
  if (TREE && p.window) t.begin = tree_range(p, item, t).begin;
  AttnRepeat rep;
  for (int pass = 0; pass < kRepeats; ++pass)
    if (!attend_tile<DP, GRAN, AW, KB, true, TREE, REST>(p, item, t, __builtin_amdgcn_readfirstlane(h), __builtin_amdgcn_readfirstlane(c_first),
                                               __builtin_amdgcn_readfirstlane(c_end), __builtin_amdgcn_readfirstlane(slot), *lds, rep))
      return;
}

// A workgroup per item (see attn_locate): of a causal call, tiles and parts differ in length.
template <int DP, int GRAN>
__global__ __launch_bounds__(256, DP > 128 ? 1 : 2) void attention_tile_kernel(AttnArgs p) {
  constexpr int AW = 4, KB = DP > 128 ? 32 : 64;
  __shared__ AttnTileLds<DP, GRAN, AW, KB> lds;
  const int h = blockIdx.x % p.hkv;
  const AttnItem it = attn_locate<AW * 64>(p, blockIdx.x / p.hkv, lds.scan);
  if (it.b < 0) return;
  const AttnTile t = attn_tile<false>(p, it);
  const int c_first = t.start + it.split * it.chunk;          // this item's positions [c_first, c_end)
  const int c_end = min(t.end, c_first + it.chunk);
  if (c_first >= c_end) return;                               // the sequence's longer tiles need this chunk
  if (it.nsplit > 1 && it.split == 0 && h == 0 && threadIdx.x == 0) {   // one workgroup describes the tile for the join
    const int first = (it.slots + it.tile * p.hkv * it.nsplit);
    *attn_record(p, it.record) = AttnRecord{(t.end - t.start + it.chunk - 1) / it.chunk, it.row0, t.r_first, t.r_count,
                                            first, first + 1, 1, it.nsplit};
  }
  const int slot = t.end - t.start <= it.chunk ? -1 : it.slots + (it.tile * p.hkv + h) * it.nsplit + it.split;
  AttnRepeat none;
  if (attend_tile<DP, GRAN, AW, KB, false, false, false>(p, it, t, h, c_first, c_end, slot, lds, none))
    attend_tile_safe<DP, GRAN, AW, KB, false, false>((kernarg_t)__builtin_amdgcn_kernarg_segment_ptr(), it, h, c_first, c_end, slot, &lds);
}

}  // namespace qg
