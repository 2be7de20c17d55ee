// Attention over the paged cache for trees of drafted tokens with many rows per key/value
// head. The mathematics, tiles and fragments are those of the kernel for many rows
// (attention_tile_kernel.h); what differs:
//
//   * All tiles of a sequence see the same positions, so every workgroup takes an equal share
//     of all tiles' positions, as in the kernel for few rows.
//   * A tree of 64 tokens and 4 heads to one is 256 rows, two tiles of 128 that would read the
//     whole history twice. Eight waves take 256 rows at once: one read, and half the
//     conversions of e4m3 codes.
//   * The order of the instructions around the MFMAs is given (see PF).
//   * e4m3 codes arrive in LDS by direct loads, several blocks ahead, and are converted from
//     there by the lane that loaded them.
//   * Which drafted tokens a row sees is a word of bits per block; blocks of the history need none.
//
// What bounds it: within a block the MFMAs and the softmax in turn, over a call the ends of parts. 32
// trees of 64 tokens on 1 to 8191 positions (32 heads on 8 of 128, bf16, 139 GFLOP, 585 MB) take 208 us
// with the join of 17 to 20, 670 TFLOP/s. A block of 256 rows on 64 positions takes 1.9 us when its pages
// are in the caches (1136 TFLOP/s, the library's large product: 1373), 2.1 to 2.3 from HBM, so some 145 us of
// these are blocks; the start and end of a part take 8 to 13, and a workgroup has one to three of them: over
// the whole call the MFMAs are busy a third of the time. 6 trees of 20 to 120 on 8000 to 40000 (e4m3, runs of
// 64, 244 GFLOP): 460 us with the join, 530 TFLOP/s; the scales of two runs and the conversion are 210 vector
// instructions per wave and block beside the 230 of a bf16 cache, MFMAs busy 23 %, and a tree of more than 64
// tokens makes a second tile that reads and converts its whole history again.
// Tried: items of whole tiles and chunks instead of shares (bf16 232 us), two groups of waves that
// take turns at the MFMAs (204, e4m3 spills), fragments 6 or 8 ahead (level), tiles of 128 rows
// (244, e4m3 516, against 210 and 459).
#pragma once

#include <type_traits>

#include "attention_tile_kernel.h"

namespace qg {

// LDS of a workgroup of AW waves. ODD: page sizes that are no multiple of 16.
template <int DP, int GRAN, int AW, bool ODD>
struct AttnTreeLds {
  static constexpr bool FP8 = GRAN > 0;
  static constexpr int KB = DP > 128 || (FP8 && DP == 128 && AW == 4) ? 32 : 64;   // positions per block
  static constexpr int R = FP8 ? DP / GRAN : 1;             // scale runs per head, at most
  static constexpr bool ONE = AW == 8 || DP > 128;          // one workgroup per CU
  static constexpr int NST = FP8 ? 2 : ONE ? 4 : 2;         // blocks as bf16
  static constexpr int NRAW = 3, NSC = NRAW + 2;            // e4m3: blocks as codes, and their scales
  struct Blocks {
    __attribute__((aligned(16))) u32x4_t ring[NST][2][KB * DP / 8];                       // [block][keys, values]
    __attribute__((aligned(16))) u32x4_t raw[FP8 ? NRAW : 1][2][FP8 ? KB * DP / 16 : 1];
    __attribute__((aligned(16))) float scales[FP8 ? NSC : 1][FP8 ? 2 * R * KB : 4];       // [block][wave][keys, values][run][position]
  };
  union {
    Blocks b;
    AttnTileLds<DP, GRAN, AW, KB> safe;
  };
  uint32_t pages[ODD ? TPG : 1];
  int w_off[AW];
  ShareScan<AW * 64> share;
};

// Positions [c_first, c_end) of one tile, as attend_tile without SAFE; block by block and sum by
// sum as it does with it, so that rows which need no repetition come out alike.
//
// REST: what the weights lose to bf16 is multiplied with the values too (half as many MFMAs again; which
// calls have it is the launcher's choice).
template <int DP, int GRAN, int AW, bool ODD, bool REST>
__device__ __forceinline__ bool attend_tree(const AttnArgs& p, const AttnItem& it, const AttnTile& t, int h, int c_first, int c_end,
                                            int slot, AttnTreeLds<DP, GRAN, AW, ODD>& lds) {
  typedef AttnTreeLds<DP, GRAN, AW, ODD> Lds;
  constexpr bool FP8 = GRAN > 0;
  constexpr int NT = AW * 64, KB = Lds::KB, R = Lds::R, NST = Lds::NST, NRAW = Lds::NRAW, NSC = Lds::NSC;
  constexpr int NB = KB / 32;
  constexpr int NS = DP / 16;                 // MFMA steps of a score
  constexpr int ND = DP / 32;                 // 32-wide strips of the output
  constexpr int CH = DP / 8;                  // 16-byte chunks per LDS row
  constexpr int ROW = CH * 16, PLANE = KB * ROW, BLOCK = 2 * PLANE;   // bytes
  constexpr int PW = KB / AW;                 // positions that a wave loads
  constexpr int LC = FP8 ? DP / 16 : CH;      // 16-byte loads per cache row, and per lane and plane
  constexpr int LD = PW * LC / 64;
  constexpr int NSL = FP8 ? (PW * R + 63) / 64 : 0;        // loads of scales per plane
  constexpr int LB = 2 * LD + 2 * NSL;        // loads per block
  constexpr int RS = FP8 ? GRAN / 16 : NS;    // MFMA steps per run
  // Fragments read ahead of their MFMAs. Left to itself the compiler reads each right before its
  // MFMA and waits out the LDS latency every time.
  constexpr int PF = 4;
  static_assert(PW == 8 || PW == 16, "a wave's positions lie in one page");
  static_assert(LD >= 1 && LB * (FP8 ? NRAW : NST) < 64, "loads in flight that a wait can count");
  auto& ring = lds.b.ring;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const bool idle = wave * 32 >= t.r_count;   // rows of no token: such a wave moves blocks only

  const int rows = it.fresh * p.group;
  const int my_row = min(t.r_first + wave * 32 + col, rows - 1), tok = over_group(p, my_row);
  const int lo = tree_low(p, it, tok);
  const uint16_t* q = p.q + ((size_t)(it.row0 + tok) * p.hq + h * p.group + my_row - tok * p.group) * p.d;
  u32x4_t qf[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int d = 16 * s + 8 * half;
    qf[s] = d < p.d ? *reinterpret_cast<const u32x4_t*>(q + d) : u32x4_t{0, 0, 0, 0};
  }
  const float cs = p.scale * kLog2e;
  const int runs = FP8 ? p.d / (FP8 ? GRAN : 1) : 1;
  if (p.d < DP) {                             // chunks of an LDS row that do not exist are zero from here on
    for (int e = tid; e < NST * BLOCK / 16; e += NT) (&ring[0][0][0])[e] = u32x4_t{0, 0, 0, 0};
  }
  const uint32_t row_bytes = (uint32_t)(p.hkv * p.d * (FP8 ? 1 : 2));   // a (page, slot) row
  const size_t plane_bytes = (size_t)p.pages * p.page_size * row_bytes;
  const char* keys = static_cast<const char*>(p.blocks) + 2 * p.layer * plane_bytes + (size_t)h * p.d * (FP8 ? 1 : 2);
  const uint32_t row_scales = p.hkv * runs;
  const size_t plane_scales = (size_t)p.pages * p.page_size * row_scales;
  const float* key_scales = FP8 ? p.scales + 2 * p.layer * plane_scales + (size_t)h * runs : nullptr;
  const uint32_t* my_pages = p.page_table + (size_t)it.b * p.max_pages;
  // A wave's load k of a block: its row wpos(k) of PW, 16 bytes from byte wbyte(k) of the head's row on.
  // bf16: LDS chunk c of row r holds chunk c ^ swz(r) of the cache row.
  const int mine = wave * PW & ~15, place = wave * PW & 15;
  auto wpos = [&](int k) { return (k * 64 + lane) / LC; };
  auto wbyte = [&](int k) {
    const int c = (k * 64 + lane) % LC;
    return (FP8 ? c : c ^ swz_t<DP>(wave * PW + wpos(k))) * 16;
  };
  // its scale n of a plane: of the wave's position spos(n), run srun(n)
  auto spos = [&](int n) { return (n * 64 + lane) % PW; };
  auto srun = [&](int n) { return min((n * 64 + lane) / PW, runs - 1); };

  float16_t acc[ND];
  float m = -INFINITY, l = 0.f;   // reference of the weights' exponents (base 2), this lane's share of their sum
  uint32_t seen = 0;              // not 0 where the row has seen a position
  // A zero that the compiler does not know for one: it would let the accumulators share it with the
  // upper halves of addresses, and hold those in registers of 16 that it spills at every use.
  float none = 0.f;
  asm volatile("" : "+v"(none));
#pragma unroll
  for (int n = 0; n < ND; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[n][i] = none;
  // LDS addresses of this lane's first fragments, relative to their block: chunk 2 s + half of key row
  // col lies at ^ 32 s bytes, and of the values (rows 4 half + (lane & 15) / 4 of 16, and 8 behind)
  // strip n at ^ 64 n, the rows behind at ^ 32. All else is a constant offset.
  const uint32_t k_at = col * ROW + ((half ^ swz_t<DP>(col)) << 4);
  const int v_row = 4 * half + ((lane & 15) >> 2), v_chunk = 2 * ((lane >> 4) & 1) + ((lane & 2) >> 1);
  const uint32_t v_at = PLANE + v_row * ROW + ((v_chunk ^ swz_t<DP>(v_row)) << 4) + 8 * (lane & 1);
  char* const blocks_at = reinterpret_cast<char*>(&ring[0][0][0]);

  // as many positions at a time as the list of pages covers
  const int seg = !ODD ? c_end - c_first : (int)min((long long)(c_end - c_first), (long long)(TPG - 1) * p.page_size / KB * KB);
  for (int s_first = c_first; s_first < c_end; s_first += seg) {
    const int s_end = min(c_end, s_first + seg);
    const int page0 = !ODD ? 0 : fast_div(max(s_first, t.begin), p.div_mul, p.div_shift);
    if (ODD) {
      const int page1 = fast_div(s_end - 1, p.div_mul, p.div_shift);
      __syncthreads();
      for (int e = tid; e <= page1 - page0; e += NT) lds.pages[e] = my_pages[page0 + e];
    }
    if (ODD || p.d < DP) __syncthreads();

    // cache row of a position; positions outside [begin, s_end) take one inside (their pages may
    // not exist)
    auto row_of = [&](int pos) {
      const int x = min(max(pos, t.begin), s_end - 1);
      const uint32_t pg = fast_div(x, p.div_mul, p.div_shift);
      return (size_t)lds.pages[pg - page0] * p.page_size + (x - pg * p.page_size);
    };
    // The 16 positions that hold this wave's of the block to be loaded next: looked up a block ahead, as
    // the wait for a page's number would be the longest of a turn.
    Row16 ahead{};
    auto look = [&](int i) {
      if constexpr (!ODD) ahead = rows_of16(p, (page_list_t)my_pages, s_first + KB * i + mine, t.begin, s_end);
    };
    // block i (whose place `look` has found) on its way: bf16 into ring[at], codes into raw[at] and scales into scales[i % NSC]
    auto issue = [&](int i, int at) {
      const int first = s_first + KB * i + mine;   // of the 16 positions that hold this wave's
      char* const to = FP8 ? reinterpret_cast<char*>(&lds.b.raw[FP8 ? at : 0][0][0]) : blocks_at + at * BLOCK;
      constexpr int TO = FP8 ? KB * DP : PLANE;    // bytes of a plane there
      const uint32_t to_lds = lds_addr(to) + wave * LD * 1024;
      if constexpr (!ODD) {
        const Row16 r = ahead;
        look(i + 1);
        const char* kbase = uniform(keys + r.row * row_bytes);
        const char* vbase = uniform(kbase + plane_bytes);
        const bool inside = first >= t.begin && first + 16 <= s_end;
        // offset from the 16 positions' first row of the one to be read for place x of this wave's
        auto slot_of = [&](int x) { return inside ? place + x : min(max(r.pos + place + x, t.begin), s_end - 1) - r.pos; };
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const uint32_t off = slot_of(wpos(k)) * row_bytes + wbyte(k);
          if (wbyte(k) < p.d * (FP8 ? 1 : 2)) {
            dma16(kbase, off, to_lds + k * 1024);
            dma16(vbase, off, to_lds + TO + k * 1024);
          }
        }
        if constexpr (FP8) {
          const uint32_t s_lds = lds_addr(&lds.b.scales[i % NSC][wave * PW * 2 * R]);
#pragma unroll
          for (int n = 0; n < NSL; ++n) {
            const uint32_t off = (slot_of(spos(n)) * row_scales + srun(n)) * 4;
            const float* from = uniform(key_scales + r.row * row_scales);
            const bool on = n * 64 + lane < PW * R;
            dma4_lanes(from, off, s_lds + n * 256, on);
            dma4_lanes(uniform(from + plane_scales), off, s_lds + PW * R * 4 + n * 256, on);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const char* src = keys + row_of(first + place + wpos(k)) * row_bytes + wbyte(k);
          if (wbyte(k) < p.d * (FP8 ? 1 : 2)) {
            dma16_at(src, to_lds + k * 1024);
            dma16_at(src + plane_bytes, to_lds + TO + k * 1024);
          }
        }
        if constexpr (FP8) {
          const uint32_t s_lds = lds_addr(&lds.b.scales[i % NSC][wave * PW * 2 * R]);
#pragma unroll
          for (int n = 0; n < NSL; ++n)
            if (n * 64 + lane < PW * R) {
              const float* from = key_scales + row_of(first + place + spos(n)) * row_scales + srun(n);
              dma4_at(from, s_lds + n * 256);
              dma4_at(from + plane_scales, s_lds + PW * R * 4 + n * 256);
            }
        }
      }
    };
    // e4m3: this lane's codes of raw[from] as bf16 into ring[to]
    auto convert = [&](int from, int to) {
#pragma unroll
      for (int k = 0; k < LD; ++k) {
        const int e = (wave * LD + k) * 64 + lane, row = e / LC, c = e % LC;
        if (c * 16 >= p.d) continue;
#pragma unroll
        for (int plane = 0; plane < 2; ++plane) {
          const u32x4_t v = lds.b.raw[FP8 ? from : 0][plane][FP8 ? e : 0];
          uint32_t o[8];
#pragma unroll
          for (int g = 0; g < 4; ++g) e4m3x4_to_bf16(v[g], o[2 * g], o[2 * g + 1]);
          const int z = swz_t<DP>(row);
          ring[to][plane][row * CH + ((2 * c) ^ z)] = u32x4_t{o[0], o[1], o[2], o[3]};
          ring[to][plane][row * CH + ((2 * c + 1) ^ z)] = u32x4_t{o[4], o[5], o[6], o[7]};
        }
      }
    };

    const int blocks = (s_end - s_first + KB - 1) / KB;
    look(0);
    // a block's scores, then weights: register e of nb is position 32 nb + 8 (e / 4) + 4 half + e % 4
    typedef float16_t Scores[NB];

    // where a block lies: bf16 in ring[at], scales in scales[i % NSC]
    struct Place {
      uint32_t base, s_base;
    };
    auto place_of = [&](int i, int at) {
      Place x{(uint32_t)(at * BLOCK), (uint32_t)((i % NSC) * (2 * R * KB * 4) + 16 * half)};
      // computed here, for every block: addresses held across blocks would be too many registers
      asm volatile("" : "+v"(x.base), "+v"(x.s_base));
      return x;
    };
    // scales of 4 positions from `pos` on, of which 4 half is in s_base
    auto scale4 = [&](const Place& x, int plane, int run, int pos) {
      const int w = pos / PW, o = pos % PW;
      return *reinterpret_cast<const float4_t*>(reinterpret_cast<const char*>(&lds.b.scales[0][0]) + x.s_base +
                                                (((w * 2 + plane) * R + run) * PW + o) * 4);
    };
    // weights of 16 positions, and REST's of them; key slots 0..3 are key0 + 0..3, 4..7 key0 + 8..11
    auto weights = [&](const Scores& sc, const Place& x, int nb, int ks, int run, u32x4_t& rest) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = sc[nb][8 * ks + e];
      if constexpr (FP8) {   // times the value scales of the strip's run
        const float4_t v0 = scale4(x, 1, run, nb * 32 + ks * 16), v1 = scale4(x, 1, run, nb * 32 + ks * 16 + 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= e < 4 ? v0[e] : v1[e - 4];
      }
      const u32x4_t r = {f2bf2_rn(w[0], w[1]), f2bf2_rn(w[2], w[3]), f2bf2_rn(w[4], w[5]), f2bf2_rn(w[6], w[7])};
      if constexpr (REST) rest = remainders(w, r);
      return r;
    };
    // S^T = K Q^T of the block at x
    auto score = [&](Scores& sc, const Place& x) {
      constexpr int KS = NB * NS, G = KS / RS;     // MFMAs, runs of them (of one nb each)
      // bf16: the halves of a block in turn, as an MFMA waits for the sum that it adds to
      auto step_of = [&](int j) { return FP8 ? j % NS : j / NB; };
      auto half_of = [&](int j) { return FP8 ? j / NS : j % NB; };
      auto frag = [&](int j) {
        return *reinterpret_cast<const u32x4_t*>(blocks_at + ((x.base + k_at) ^ (32 * step_of(j))) + half_of(j) * 32 * ROW);
      };
      __builtin_amdgcn_s_setprio(1);
      u32x4_t f[PF];
      // A run's scales are applied behind the next run's MFMAs, so that nothing waits for its own.
      float16_t part[R > 2 ? 2 : 1];               // scores of runs behind the first
      float4_t ks[4];
      auto sums = [&](int g) -> float16_t& { return g % R == 0 ? sc[g / R] : part[R > 2 ? g & 1 : 0]; };
      auto scales = [&](int g) {
#pragma unroll
        for (int u = 0; u < 4; ++u) ks[u] = scale4(x, 0, g % R, g / R * 32 + 8 * u);
      };
      auto scaled = [&](int g) {
        float16_t& to = sc[g / R];
#pragma unroll
        for (int e = 0; e < 16; ++e) to[e] = g % R == 0 ? to[e] * ks[e >> 2][e & 3] : __builtin_fmaf(sums(g)[e], ks[e >> 2][e & 3], to[e]);
        asm volatile("" : "+v"(to));               // here, not where the scores are used: all runs' sums would be held until then
      };
#pragma unroll
      for (int j = 0; j < PF; ++j) f[j] = frag(j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int g = FP8 ? j / RS : half_of(j);
        float16_t& to = sums(g);
        if (step_of(j) % RS == 0) {
          if constexpr (FP8) {
            if (g > 0) scales(g - 1);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) to[e] = 0.f;
        }
        to = mfma32x32x16_bf16(f[j % PF], qf[step_of(j)], to);
        if (j + PF < KS) f[j % PF] = frag(j + PF);
        if (FP8 && j % RS == RS - 1 && g > 0) scaled(g - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (FP8) {
        scales(G - 1);
        scaled(G - 1);
      }
      __builtin_amdgcn_s_setprio(0);
    };
    // O^T += V^T P^T
    auto add_values = [&](const Scores& sc, const Place& x) {
      constexpr int VS = NB * 2 * ND;
      auto frag = [&](int j) {   // strip n of 16 positions (see attend_tile)
        const uint32_t at_n = (x.base + v_at) ^ (64 * (j % ND));
        const char* from = blocks_at + j / ND * 16 * ROW;
        const uint64_t w0 = lds_read_tr16(from + at_n), w1 = lds_read_tr16(from + (at_n ^ 32) + 8 * ROW);
        return u32x4_t{(uint32_t)w0, (uint32_t)(w0 >> 32), (uint32_t)w1, (uint32_t)(w1 >> 32)};
      };
      __builtin_amdgcn_s_setprio(1);
      u32x4_t f[PF], w, rest;
#pragma unroll
      for (int j = 0; j < PF; ++j) f[j] = frag(j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < VS; ++j) {
        const int n = j % ND;
        if (n == 0 || (FP8 && n * 32 % (FP8 ? GRAN : 1) == 0)) w = weights(sc, x, j / (2 * ND), j / ND % 2, FP8 ? n * 32 / (FP8 ? GRAN : 1) : 0, rest);
        acc[n] = mfma32x32x16_bf16(f[j % PF], w, acc[n]);
        if constexpr (REST) acc[n] = mfma32x32x16_bf16(f[j % PF], rest, acc[n]);
        if (j + PF < VS) f[j % PF] = frag(j + PF);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    };
    // Scores of the block from position k0 on to weights.
    auto soften = [&](Scores& sc, int k0) {
      // the drafted tokens, and where windows begin, somewhere before them
      const bool masked = uniform((p.window && k0 < min(it.cached, t.end - p.window)) || k0 < t.begin || k0 + KB > min(s_end, it.cached));
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t vis = tree_sees(p, it, tok, lo, k0 + 32 * nb, s_end) >> (4 * half);
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[nb][e] = vis >> (8 * (e / 4) + e % 4) & 1 ? sc[nb][e] : -INFINITY;
          seen |= vis;
        }
      } else {
        seen = 1;
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
          for (int e = 0; e < 16; ++e) acc[n][e] *= alpha;
      }
      // a row that has seen nothing yet keeps -infinity; its weights are 0
      const float ref = m == -INFINITY ? 0.f : m;
      float l_block = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          sc[nb][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[nb][e], cs, -ref));
          l_block += sc[nb][e];
        }
      l += l_block;
    };
    int raw = 0;                                   // e4m3: place of the codes to be converted next
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < NRAW; ++u)
        if (u < blocks) issue(u, u);
      wait_blocks<LB, NRAW - 1>(blocks - 1);
      convert(0, 0);
      wait_lds();
      if (NRAW < blocks) issue(NRAW, 0);
      raw = 1;
    } else {
#pragma unroll
      for (int u = 0; u < NST - 1; ++u)
        if (u < blocks) issue(u, u);
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) arrived(qf[n]);   // (with the first blocks, which are waited for next anyway)
    int at = 0;
    for (int i = 0; i < blocks; ++i, at = at + 1 == NST ? 0 : at + 1) {
      if constexpr (!FP8) wait_blocks<LB, NST - 2>(blocks - 1 - i);
      __syncthreads();             // block i is in LDS; nobody reads the one before any more
      auto load = [&]() {
        if constexpr (FP8) {
          if (i + 1 < blocks) {
            wait_blocks<LB, NRAW - 1>(blocks - 2 - i);
            convert(raw, at ^ 1);
            wait_lds();
            if (i + 1 + NRAW < blocks) issue(i + 1 + NRAW, raw);
            raw = raw + 1 == NRAW ? 0 : raw + 1;
          }
        } else {
          if (i + NST - 1 < blocks) issue(i + NST - 1, at == 0 ? NST - 1 : at - 1);
        }
      };
      if (idle) {
        load();
      } else {
        const Place x = place_of(i, at);
        Scores sc;
        score(sc, x);
        load();
        soften(sc, s_first + KB * i);
        add_values(sc, x);
      }
    }
  }
  int off = 0;
#pragma unroll
  for (int n = 0; n < ND; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) off |= !(fabsf(acc[n][e]) < kSumsMost);
  const float sum = l + __shfl_xor(l, 32);
  off |= weights_off(m, sum);
  off = __any(off);
  if (lane == 0) lds.w_off[wave] = off;
  __syncthreads();
  off = 0;
#pragma unroll
  for (int w = 0; w < AW; ++w) off |= lds.w_off[w];
  if (uniform(off != 0)) return true;   // a scalar branch: the accumulators are not live across the call behind it
  store_tile<DP, true>(p, it, t, h, slot, acc, m, seen_sum(sum, (seen | __shfl_xor(seen, 32)) != 0));
  return false;
}

// A workgroup per share (see attn_share).
template <int DP, int GRAN, int AW, bool ODD, bool REST>
__global__ __launch_bounds__(AW * 64, DP > 128 ? 1 : 2) void attention_tree_kernel(AttnArgs p) {
  __shared__ AttnTreeLds<DP, GRAN, AW, ODD> lds;
  AttnShare s = attn_share<AW * 64, true, 1>(p, lds.share);
  if (s.b < 0) return;
  while (true) {
    AttnItem it{};
    it.b = s.b;
    it.tile = s.tile;
    it.row0 = s.row0;
    it.fresh = s.fresh;
    it.cached = s.cached;
    AttnTile t = attn_tile<true>(p, it);
    AttnPart part = attn_part<true>(p, s, t);
    if (part.first < part.end) {
      if (!tree_narrow(p, it, t, part))
        store_unseen<AW * 64, DP>(p, it, t, s.h, 1, part.slot);
      else if (attend_tree<DP, GRAN, AW, ODD, REST>(p, it, t, s.h, part.first, part.end, part.slot, lds))
        attend_tile_safe<DP, GRAN, AW, AttnTreeLds<DP, GRAN, AW, ODD>::KB, true, REST>((kernarg_t)__builtin_amdgcn_kernarg_segment_ptr(), it, s.h, part.first, part.end, part.slot, &lds.safe);
    }
    if (!attn_next(p, s, part.take)) return;
    __syncthreads();   // the next part's loads overwrite what the last one's blocks were read from
  }
}

}  // namespace qg
