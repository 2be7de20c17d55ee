// Attention over the paged cache for few rows per key/value head (single tokens,
// drafted tokens): a stream over the cache, bound by HBM.
//
// A tile is 16 * MT (token, query head) rows. A workgroup takes an equal share of
// all tiles' positions, part by part; its waves take blocks of 32 positions in turn, each with its
// own ring of two blocks in LDS, filled by direct-to-LDS loads (no registers
// held, no barrier between the waves). Scores come transposed from 16x16x32
// MFMAs, S^T = K Q^T: a lane holds eight scores of one row, and they are, as they
// lie, the B operand of O^T = V^T P^T with the key slots in the order
// {4j .. 4j + 3, 16 + 4j .. 16 + 4j + 3} for lane quarter j; the transposed reads
// of V name its rows in that order.
//
// The MFMAs have time to spare here, so a probability enters as two bf16 (value
// and remainder): the result is that of fp32 probabilities, rounded once.
//
// Measured (heads of 128, 32 on 8, pages of 128): 64 sequences with 1 to 8192
// positions, 204 us on bf16 (5.4 TB/s of cache read; a contiguous read reaches 6.2) and
// 124 us on e4m3 (4.6 TB/s), runs of 32 147 us; heads of 256 (16 on 4) 220 us. The same
// without the arithmetic takes as long: what counts is how the cache is read. One head per
// workgroup, 256 or 128 bytes of each cache row: 222 and 141 us; rings of three or
// four blocks with the waves that fit then: 226 and 255, 146 and 144 (when those 204 and
// 124 were 207 and 125).
//
// Running maximum, e4m3 scales and what a row must not see are dealt with as in
// the kernel for many rows.
#include <algorithm>

#include "attention_common.h"

namespace qg {

namespace {

constexpr int RPG = 1024;   // page table entries held in LDS at a time (page sizes not a multiple of 16)

// LDS rows of CH 16-byte chunks: chunk c of row r lies at c ^ swz(r). A phase of
// transposed value reads takes 8 rows (bf16; 16 rows of e4m3) of one strip, which
// meet different banks; key fragments use the same order, so that one offset per
// lane serves both planes' loads.
template <int CH, bool FP8>
__device__ __forceinline__ int swz_r(int r) {
  if (!FP8) return CH >= 16 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
  return CH >= 16 ? (r & 7) | ((r >> 4) & 1) << 3 : CH == 8 ? ((r >> 1) & 3) | ((r >> 4) & 1) << 2 : ((r >> 2) & 1) | ((r >> 4) & 1) << 1;
}

template <int DP, int GRAN, int MT, int NW, int NST>
struct AttnRowsLds {
  static constexpr int TILE = 2 * DP * (GRAN > 0 ? 1 : 2);   // 16-byte chunks of a block's keys (or values)
  static constexpr int R = GRAN > 0 ? DP / GRAN : 1;          // scale runs per head, at most
  __attribute__((aligned(16))) u32x4_t ring[NW][NST][2][TILE];    // [wave][slot][keys, values]
  __attribute__((aligned(16))) float ring_s[GRAN > 0 ? NW : 1][NST][R][2][32];   // run scales [run][keys, values][position]
  uint32_t pages[RPG];
  float w_m[NW][16 * MT], w_l[NW][16 * MT];
  int w_off[NW];
  ShareScan<NW * 64> scan;
};

}  // namespace

// Positions [c_first, c_end) of one tile, which are all of them where `slot` is -1
// and go to that slot of the workspace else. GRAN: head-dim elements per scale of an
// e4m3 cache, 0 for bf16. SAFE: values are selected per token. Returns whether some
// row has to be computed again (without SAFE: sums are too large, infinities, NaN or
// zero; with it: as `rep`, the state of this lane's rows in this wave, says), for the
// whole workgroup, and then has written nothing.
template <int DP, int GRAN, int MT, int NW, int NST, bool SAFE>
__device__ __forceinline__ bool attend_rows(const AttnArgs& p, const AttnItem& it, int h0, int hw, int c_first, int c_end, int slot,
                                            AttnRowsLds<DP, GRAN, MT, NW, NST>& lds, AttnRepeat (&rep)[MT]) {
  constexpr bool FP8 = GRAN > 0;
  constexpr int ES = FP8 ? 1 : 2;              // bytes per cached element
  constexpr int CH = DP * ES / 16;             // chunks per LDS row
  constexpr int TILE = 32 * CH;
  constexpr int LD = TILE / 64;                // loads per lane for a block's keys (or values)
  constexpr int NS = DP / 32;                  // MFMA steps of a score
  constexpr int ND = DP / 16;                  // 16-wide strips of the output
  constexpr int R = FP8 ? DP / GRAN : 1;
  constexpr int RS = FP8 ? GRAN / 32 : NS;     // MFMA steps per run
  constexpr int NT = NW * 64;
  // floats per row of a wave's partial output in LDS
  constexpr int OS = 16 * MT * (DP + 4) * 4 <= NST * 2 * TILE * 16 ? DP + 4 : DP;
  static_assert(16 * MT * OS * 4 <= NST * 2 * TILE * 16, "a wave's partial output fits its ring");
  static_assert(LD >= 2, "a load covers 16 positions at most");
  constexpr int LB = 2 * LD + (FP8 ? R : 0);   // loads per block
  static_assert((NST - 1) * LB < 64, "loads in flight that a wait can count");
  auto& ring = lds.ring;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, j = lane >> 4;
  const int h = h0 + wave % hw, phase = wave / hw, phases = NW / hw;   // this wave's head and blocks
  const AttnTile t = attn_tile(p, it);

  // rows of this lane, one per 16-row tile
  const int rows = it.fresh * p.group;
  int tok[MT], hi[MT], lo[MT];
  u32x4_t qf[MT][NS];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = min(t.r_first + 16 * mt + col, rows - 1);
    tok[mt] = over_group(p, r);
    hi[mt] = p.causal ? it.cached + tok[mt] : it.cached + it.fresh - 1;
    lo[mt] = p.window ? it.cached + tok[mt] - p.window + 1 : 0;
    const uint16_t* q = p.q + ((size_t)(it.row0 + tok[mt]) * p.hq + h * p.group + r - tok[mt] * p.group) * p.d;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = 32 * s + 8 * j;
      qf[mt][s] = d < p.d ? *reinterpret_cast<const u32x4_t*>(q + d) : u32x4_t{0, 0, 0, 0};
    }
  }
  const int runs = FP8 ? p.d / (FP8 ? GRAN : 1) : 1;
  const int chunks = p.d * ES / 16;                           // chunks of a cache row that exist
  // head dims between p.d and DP: never loaded, zero from here on
  if (chunks < CH) {
    for (int e = tid; e < NW * NST * 2 * TILE; e += NT) (&ring[0][0][0][0])[e] = u32x4_t{0, 0, 0, 0};
  }
  const float cs = p.scale * kLog2e;
  const uint32_t row_bytes = (uint32_t)(p.hkv * p.d * ES);    // a (page, slot) row
  const size_t plane_bytes = (size_t)p.pages * p.page_size * row_bytes;
  const char* keys = static_cast<const char*>(p.blocks) + 2 * p.layer * plane_bytes + (size_t)h * p.d * ES;
  const int row_scales = p.hkv * runs;
  const size_t plane_scales = (size_t)p.pages * p.page_size * row_scales;
  const float* key_scales = FP8 ? p.scales + 2 * p.layer * plane_scales + (size_t)h * runs : nullptr;
  const uint32_t* my_pages = p.page_table + (size_t)it.b * p.max_pages;
  const bool by16 = p.page_size % 16 == 0;
  // this lane's places in a block: key e / CH, chunk e % CH of LDS position e = 64 k + lane
  uint32_t voff[LD];
  bool there[LD];
#pragma unroll
  for (int k = 0; k < LD; ++k) {
    const int e = k * 64 + lane, key = e / CH, c = e % CH ^ swz_r<CH, FP8>(key);
    voff[k] = (key & 15) * row_bytes + c * 16;
    there[k] = c < chunks;
  }

  float4_t acc[MT][ND];
  float m[MT], l[MT];     // reference of the weights' exponents (base 2), this lane's share of their sum
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = -INFINITY;
    l[mt] = 0.f;
#pragma unroll
    for (int n = 0; n < ND; ++n) acc[mt][n] = float4_t{0.f, 0.f, 0.f, 0.f};
  }
  // as many positions at a time as the list of pages covers
  const int seg = by16 ? c_end - c_first : (int)min((long long)(c_end - c_first), (long long)(RPG - 1) * p.page_size / (32 * NW) * (32 * NW));
  for (int s_first = c_first; s_first < c_end; s_first += seg) {
    const int s_end = min(c_end, s_first + seg);
    const int page0 = by16 ? 0 : fast_div(max(s_first, t.begin), p.div_mul, p.div_shift);
    if (!by16) {
      const int page1 = fast_div(s_end - 1, p.div_mul, p.div_shift);
      if (s_first > c_first) __syncthreads();
      for (int e = tid; e <= page1 - page0; e += NT) lds.pages[e] = my_pages[page0 + e];
    }
    if (!by16 || chunks < CH) __syncthreads();

    // cache row of a position; positions outside [begin, end) take one inside (their
    // pages may not exist)
    auto row_of = [&](int pos) {
      const int x = min(max(pos, t.begin), s_end - 1);
      const uint32_t pg = fast_div(x, p.div_mul, p.div_shift);
      return (size_t)lds.pages[pg - page0] * p.page_size + (x - pg * p.page_size);
    };
    // block i of the segment on its way into slot `at` of this wave's ring
    auto issue = [&](int i, int at) {
      wait_lds();
      const int first = s_first + 32 * i;
      if (by16) {
        Row16 r[2];
        const char* base[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          r[u] = rows_of16(p, (page_list_t)my_pages, first + 16 * u, t.begin, s_end);
          base[u] = uniform(keys + r[u].row * row_bytes);
        }
        const bool inside = first >= t.begin && first + 32 <= s_end;
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const int u = k >= LD / 2;
          uint32_t off = voff[k];
          if (!inside) {
            const int e = k * 64 + lane, key = e / CH;
            const int x = min(max(r[u].pos + (key & 15), t.begin), s_end - 1) - r[u].pos;
            off = x * row_bytes + (e % CH ^ swz_r<CH, FP8>(key)) * 16;
          }
          if (there[k]) {
            dma16(base[u], off, lds_addr(&ring[wave][at][0][k * 64]));
            dma16(uniform(base[u] + plane_bytes), off, lds_addr(&ring[wave][at][1][k * 64]));
          }
        }
        if constexpr (FP8) {
          const int u = (lane >> 4) & 1;
          const int x = min(max((u ? r[1].pos : r[0].pos) + col, t.begin), s_end - 1) - (u ? r[1].pos : r[0].pos);
          const float* src = key_scales + ((u ? r[1].row : r[0].row) + x) * row_scales + (lane >> 5) * plane_scales;
#pragma unroll
          for (int g = 0; g < R; ++g)   // the same number of loads whatever `runs`: wait_loads counts them
            dma4_at(src + min(g, runs - 1), lds_addr(&lds.ring_s[wave][at][g][0][0]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const int e = k * 64 + lane, key = e / CH;
          const char* src = keys + row_of(first + key) * row_bytes + (e % CH ^ swz_r<CH, FP8>(key)) * 16;
          if (there[k]) {
            dma16_at(src, lds_addr(&ring[wave][at][0][k * 64]));
            dma16_at(src + plane_bytes, lds_addr(&ring[wave][at][1][k * 64]));
          }
        }
        if constexpr (FP8) {
          const float* src = key_scales + row_of(first + (lane & 31)) * row_scales + (lane >> 5) * plane_scales;
#pragma unroll
          for (int g = 0; g < R; ++g) dma4_at(src + min(g, runs - 1), lds_addr(&lds.ring_s[wave][at][g][0][0]));
        }
      }
    };

    const int blocks = (s_end - s_first + 31) / 32;
    // NST - 1 blocks in flight besides the one in hand
    const int my_blocks = phase < blocks ? (blocks - phase + phases - 1) / phases : 0;
#pragma unroll
    for (int u = 0; u < NST - 1; ++u)
      if (u < my_blocks) issue(phase + u * phases, u);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < NS; ++s) arrived(qf[mt][s]);   // (with the first blocks, which are waited for next anyway)
    int at = 0, to = NST - 1;
    for (int n = 0; n < my_blocks; ++n, at = at + 1 == NST ? 0 : at + 1) {
      const int i = phase + n * phases;
      if (n + NST - 1 < my_blocks) {
        issue(i + (NST - 1) * phases, to);
        to = to + 1 == NST ? 0 : to + 1;
      }
      wait_blocks<LB, NST - 1>(my_blocks - 1 - n);
      const int k0 = s_first + 32 * i;
      const u32x4_t* lk = ring[wave][at][0];
      const char* lv = reinterpret_cast<const char*>(ring[wave][at][1]);
      const float(*ls)[2][32] = lds.ring_s[FP8 ? wave : 0][at];

      // scores: register i of sc[.][nb] is position k0 + 16 nb + 4 j + i
      float4_t sc[MT][2];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const int key = 16 * nb + col;
        float4_t part[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) part[mt] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          u32x4_t kf;
          if constexpr (FP8) {
            const int c = 2 * s + (j >> 1);
            const u32x2_t w = *reinterpret_cast<const u32x2_t*>(reinterpret_cast<const char*>(lk + key * CH + (c ^ swz_r<CH, FP8>(key))) + 8 * (j & 1));
            const uint32_t w0 = w.x, w1 = w.y;
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_bf16(w0, a0, a1);
            e4m3x4_to_bf16(w1, a2, a3);
            kf = u32x4_t{a0, a1, a2, a3};
          } else {
            kf = lk[key * CH + ((4 * s + j) ^ swz_r<CH, FP8>(key))];
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) part[mt] = mfma16x16x32_bf16(kf, qf[mt][s], part[mt]);
          if constexpr (FP8) {
            if ((s + 1) % RS == 0) {   // a run is complete: times the keys' scales
              const int run = (s + 1) / RS - 1;
              const float4_t ks = *reinterpret_cast<const float4_t*>(&ls[run][0][16 * nb + 4 * j]);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  sc[mt][nb][e] = run == 0 ? part[mt][e] * ks[e] : __builtin_fmaf(part[mt][e], ks[e], sc[mt][nb][e]);
                part[mt] = float4_t{0.f, 0.f, 0.f, 0.f};
                // each run finished before the next, as in the kernel for many rows (32
                // sequences of 6 tokens on 4000 positions, heads of 256: runs of 32
                // 627 -> 256 us, of 64 346 -> 215; heads of 128, runs of 32: 176 -> 111)
                if constexpr (MT > 1 && GRAN < 128) asm volatile("" : "+v"(sc[mt][nb]));
              }
              if constexpr (MT > 1 && GRAN < 128) __builtin_amdgcn_sched_barrier(0);
            }
          }
        }
        if constexpr (!FP8) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sc[mt][nb] = part[mt];
        }
      }
      const bool masked = uniform((p.window && k0 < it.cached + t.t_last - p.window + 1) || k0 < t.begin ||
                                  k0 + 32 > min(s_end, p.causal ? it.cached + t.t_first + 1 : t.end));
      uint32_t sees[MT];   // SAFE: bit e of positions whose weight is more than zero, be it too small for fp32
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        sees[mt] = 0;
        if (masked) {
          // positions lo .. min(hi, s_end - 1), counted from lo
          const uint32_t seen = max(min(hi[mt], s_end - 1) - lo[mt] + 1, 0), first = k0 + 4 * j - lo[mt];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sc[mt][e >> 2][e & 3] = first + (16 * (e >> 2) + (e & 3)) < seen ? sc[mt][e >> 2][e & 3] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, sc[mt][e >> 2][e & 3]);
        mx = max_halves(max_quarters(mx)) * cs;
        const bool more = mx > m[mt] + kSlack;   // (-infinity: the row has seen nothing yet)
        if (__any(more)) {
          // only a row's own scores move its reference: its result is the same whatever the others see
          const float alpha = more ? __builtin_amdgcn_exp2f(m[mt] - mx) : 1.f;
          m[mt] = more ? mx : m[mt];
          l[mt] *= alpha;
#pragma unroll
          for (int n = 0; n < ND; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][n][i] = SAFE ? times(acc[mt][n][i], alpha) : acc[mt][n][i] * alpha;
        }
        // a row that has seen nothing yet keeps -infinity; its weights are 0
        const float base = m[mt] == -INFINITY ? 0.f : m[mt];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x = sc[mt][e >> 2][e & 3];
          x = __builtin_amdgcn_exp2f(SAFE ? rep[mt].exponent(x, cs, base) : __builtin_fmaf(x, cs, -base));
          if (SAFE) {
            sees[mt] |= (uint32_t)(sc[mt][e >> 2][e & 3] > -INFINITY) << e;
            x = rep[mt].weight(x);
          }
          sc[mt][e >> 2][e & 3] = x;
          sum += x;
        }
        l[mt] += sum;
      }
      u32x4_t pf[MT][2];    // probabilities: value and remainder
      // SAFE: the product of a strip's values with row tile mt's weights, infinities and NaN apart
      auto product = [&](u32x4_t vf, int mt, float4_t sum) {
        uint32_t one[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) one[e] = sees[mt] >> e & 1 ? 0x3F80u : 0u;
        const u32x4_t of = {one[0] | one[1] << 16, one[2] | one[3] << 16, one[4] | one[5] << 16, one[6] | one[7] << 16};
        const u32x4_t v = finite(vf);
        return mfma16x16x32_bf16(vf ^ v, of, mfma16x16x32_bf16(v, pf[mt][1], mfma16x16x32_bf16(v, pf[mt][0], sum)));
      };
      auto split_p = [&](int mt, int run) {
#pragma clang fp contract(off)   // the same remainder whatever the code around it: not one of an unrounded product
        uint32_t a[4], b[4];
        float4_t vs[2];
        if constexpr (FP8) {   // times the value scales of the strip's run
          vs[0] = *reinterpret_cast<const float4_t*>(&ls[run][1][4 * j]);
          vs[1] = *reinterpret_cast<const float4_t*>(&ls[run][1][16 + 4 * j]);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int e = 2 * g + u;
            x[u] = sc[mt][e >> 2][e & 3];
            if constexpr (FP8) {
              const float v = vs[e >> 2][e & 3];
              if (!SAFE) {
                x[u] *= v;
              } else {   // the scale of a position that the row does not see may be an infinity or NaN
                const int pos = k0 + 16 * (e >> 2) + 4 * j + (e & 3);
                const bool far = !(fabsf(v) < INFINITY) && (sees[mt] >> e & 1);
                x[u] = pos > hi[mt] || pos < lo[mt] || pos >= s_end ? 0.f : far ? v : x[u] * v;
              }
            }
          }
          a[g] = f2bf2_rn(x[0], x[1]);
          float rest[2] = {x[0] - bf2f((uint16_t)a[g]), x[1] - bf2f((uint16_t)(a[g] >> 16))};
          if (FP8 && SAFE) {   // an infinite scale has no remainder
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (!(fabsf(rest[u]) < INFINITY)) rest[u] = 0.f;
          }
          b[g] = f2bf2_rn(rest[0], rest[1]);
        }
        pf[mt][0] = u32x4_t{a[0], a[1], a[2], a[3]};
        pf[mt][1] = u32x4_t{b[0], b[1], b[2], b[3]};
      };
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        if (n == 0 || (FP8 && n * 16 % (FP8 ? GRAN : 1) == 0)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) split_p(mt, FP8 ? n * 16 / (FP8 ? GRAN : 1) : 0);
        }
        u32x4_t vf;
        if constexpr (FP8) {
          // lane m of a 16-lane group names row m / 2 of eight and eight codes of 16
          const int r = (lane & 15) >> 1, key = (r < 4 ? r : 12 + r) + 4 * j;
          const uint64_t w = lds_read_tr8(lv + (key * CH + (n ^ swz_r<CH, FP8>(key))) * 16 + 8 * (lane & 1));
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_bf16((uint32_t)w, a0, a1);
          e4m3x4_to_bf16((uint32_t)(w >> 32), a2, a3);
          vf = u32x4_t{a0, a1, a2, a3};
        } else {
          // lane m of a 16-lane group names row m / 4 of four and elements 4 (m % 4) .. + 3 of 16
          const int k1 = 4 * j + ((lane & 15) >> 2), c = 2 * n + ((lane & 2) >> 1);
          const uint64_t w0 = lds_read_tr16(lv + (k1 * CH + (c ^ swz_r<CH, FP8>(k1))) * 16 + 8 * (lane & 1));
          const uint64_t w1 = lds_read_tr16(lv + ((k1 + 16) * CH + (c ^ swz_r<CH, FP8>(k1 + 16))) * 16 + 8 * (lane & 1));
          vf = u32x4_t{(uint32_t)w0, (uint32_t)(w0 >> 32), (uint32_t)w1, (uint32_t)(w1 >> 32)};
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (!SAFE) {
            acc[mt][n] = mfma16x16x32_bf16(vf, pf[mt][0], acc[mt][n]);
            acc[mt][n] = mfma16x16x32_bf16(vf, pf[mt][1], acc[mt][n]);
          } else if (!masked) {
            acc[mt][n] = product(vf, mt, acc[mt][n]);
          } else {
            // token by token, with the values it does not see set to zero
#pragma unroll 1
            for (int tt = t.t_first; tt <= t.t_last; ++tt) {
              const int t_hi = p.causal ? it.cached + tt : it.cached + it.fresh - 1;
              const int t_lo = p.window ? it.cached + tt - p.window + 1 : 0;
              uint32_t keep[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int pos = k0 + 16 * (e >> 2) + 4 * j + (e & 3);
                keep[e] = pos <= t_hi && pos >= t_lo && pos < s_end ? 0xFFFFu : 0u;
              }
              const uint32_t v0 = vf.x, v1 = vf.y, v2 = vf.z, v3 = vf.w;
              const u32x4_t vs = {v0 & (keep[0] | keep[1] << 16), v1 & (keep[2] | keep[3] << 16),
                                  v2 & (keep[4] | keep[5] << 16), v3 & (keep[6] | keep[7] << 16)};
              const float4_t with = product(vs, mt, acc[mt][n]);
              if (tt == tok[mt]) acc[mt][n] = with;
            }
          }
        }
      }
    }
  }
  int off = 0;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    int far = 0;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) far |= !(fabsf(acc[mt][n][i]) < kSumsMost);
    l[mt] += __shfl_xor(l[mt], 16);
    l[mt] += __shfl_xor(l[mt], 32);
    if (SAFE) {
      far |= __shfl_xor(far, 16);
      far |= __shfl_xor(far, 32);
      const float with = rep[mt].reference(m[mt]);
      far = rep[mt].again(weights_off(m[mt], l[mt]), far, t.end - t.start);
      m[mt] = with;
    } else {
      far |= weights_off(m[mt], l[mt]);
    }
    off |= far;
  }
  off = __any(off);
  if (lane == 0) lds.w_off[wave] = off;

  // the waves' results joined through LDS (their rings, which no load targets any more)
  float* mine = reinterpret_cast<float*>(&ring[wave][0][0][0]);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (j == 0) {
      lds.w_m[wave][16 * mt + col] = m[mt];
      lds.w_l[wave][16 * mt + col] = l[mt];
    }
#pragma unroll
    for (int n = 0; n < ND; ++n) *reinterpret_cast<float4_t*>(mine + (16 * mt + col) * OS + 16 * n + 4 * j) = acc[mt][n];
  }
  __syncthreads();
  off = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) off |= lds.w_off[w];
  if (off) {
    __syncthreads();   // before the rings are used again
    return true;
  }
  for (int e = tid; e < hw * t.r_count * (DP / 4); e += NT) {
    const int sub = e / (t.r_count * (DP / 4)), r = e / (DP / 4) % t.r_count, d = e % (DP / 4) * 4;
    float top = -INFINITY;
    for (int w = sub; w < NW; w += hw) top = fmaxf(top, lds.w_m[w][r]);
    const float base = top == -INFINITY ? 0.f : top;
    float4_t o = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
    for (int w = sub; w < NW; w += hw) {
      const float f = __builtin_amdgcn_exp2f(lds.w_m[w][r] - base);
      const float4_t x = *reinterpret_cast<const float4_t*>(reinterpret_cast<const float*>(&ring[w][0][0][0]) + r * OS + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = SAFE && !(fabsf(x[i]) < INFINITY) ? o[i] + x[i] : __builtin_fmaf(x[i], f, o[i]);
      sum = __builtin_fmaf(lds.w_l[w][r], f, sum);
    }
    if (slot < 0) {
      if (d < p.d) {
        const int row = t.r_first + r, token = over_group(p, row);
        const float inv = 1.f / sum;   // every row sees a position
        uint16_t* to = p.out + ((size_t)(it.row0 + token) * p.hq + (h0 + sub) * p.group + row - token * p.group) * p.d + d;
        *reinterpret_cast<u32x2_t*>(to) = u32x2_t{f2bf2_rn(o[0] * inv, o[1] * inv), f2bf2_rn(o[2] * inv, o[3] * inv)};
      }
    } else {
      float* ws = p.workspace + attn_header_floats(p.target) + (size_t)(slot + sub) * attn_slot_floats(16 * MT, DP);
      *reinterpret_cast<float4_t*>(ws + (size_t)r * DP + d) = o;
      if (d == 0) {
        ws[16 * MT * DP + 2 * r] = top;
        ws[16 * MT * DP + 2 * r + 1] = sum;
      }
    }
  }
  return false;
}

// Called, not inlined: hardly ever taken, and its registers stay out of the kernel's.
template <int DP, int GRAN, int MT, int NW, int NST>
__device__ __attribute__((noinline)) void attend_rows_safe(kernarg_t args, AttnItem it, int h, int hw, int c_first, int c_end,
                                                           int slot, AttnRowsLds<DP, GRAN, MT, NW, NST>* lds) {
  const AttnArgs p = reload_args(args);
  AttnRepeat rep[MT];
  for (int pass = 0; pass < kRepeats; ++pass)
    if (!attend_rows<DP, GRAN, MT, NW, NST, true>(p, uniform(it), __builtin_amdgcn_readfirstlane(h), __builtin_amdgcn_readfirstlane(hw),
                                                  __builtin_amdgcn_readfirstlane(c_first), __builtin_amdgcn_readfirstlane(c_end),
                                                  __builtin_amdgcn_readfirstlane(slot), *lds, rep))
      return;
}

// Workgroups per CU by LDS (160 KB), and the waves per SIMD that the registers are divided
// for: two where LDS has room for eight waves per CU (all heads of 64, e4m3 of 128), else one.
template <typename Lds>
constexpr int attn_resident(int nw) {
  const int by_lds = 163840 / (int)sizeof(Lds), by_registers = 8 / nw;
  return by_lds < by_registers ? by_lds : by_registers;
}
template <typename Lds>
constexpr int attn_waves(int nw) { return attn_resident<Lds>(nw) * nw >= 8 ? 2 : 1; }

template <int DP, int GRAN, int MT, int NW, int NST>
__global__ __launch_bounds__(NW * 64, (attn_waves<AttnRowsLds<DP, GRAN, MT, NW, NST>>(NW))) void attention_rows_kernel(AttnArgs p) {
  __shared__ AttnRowsLds<DP, GRAN, MT, NW, NST> lds;
  AttnShare s = attn_share<NW * 64>(p, lds.scan);
  if (s.b < 0) return;
  while (true) {
    AttnItem it{};
    it.b = s.b;
    it.tile = s.tile;
    it.row0 = s.row0;
    it.fresh = s.fresh;
    it.cached = s.cached;
    const AttnTile t = attn_tile(p, it);
    const int un = attn_units(p, s.fresh + s.cached);          // the tile's units: [first_unit, first_unit + un)
    const uint32_t first_unit = s.at - s.in_tile;
    const int take = min((int)(s.end - s.at), un - s.in_tile);
    // (a tile's first unit may begin with positions, and pages, that nobody sees)
    const int from = t.start + s.in_tile * p.step, c_first = max(from, t.begin & ~31), c_end = min(t.end, from + take * p.step);
    if (c_first < c_end) {                                     // a tile may end before its sequence's longest does
      const uint32_t last_unit = first_unit + ((t.end - t.start + p.step - 1) >> p.step_log2) - 1;
      const uint32_t begin = s.cut.start(s.w);
      // a share's first part goes to its slot 2 w, its last to 2 w + 1; those between are whole tiles
      const int slot = first_unit >= begin && last_unit < s.end ? -1 : (2 * s.w + (s.at == begin ? 0 : 1)) * p.hkv + s.h;
      if (first_unit < begin && s.h == 0 && threadIdx.x == 0) {
        const int w0 = s.cut.of(first_unit);
        if (s.w == w0 + 1) {                                     // the tile's second share describes it for the join
          const int first = 2 * w0 + (first_unit == s.cut.start(w0) ? 0 : 1);
          *attn_record(p, s.w) = AttnRecord{(int)s.cut.of(last_unit) - w0 + 1, it.row0, t.r_first, t.r_count, first * p.hkv,
                                            2 * s.w * p.hkv, 2 * p.hkv, 1};
        }
      }
      AttnRepeat none[MT];
      if (attend_rows<DP, GRAN, MT, NW, NST, false>(p, it, s.h, s.hw, c_first, c_end, slot, lds, none))
        attend_rows_safe<DP, GRAN, MT, NW, NST>((kernarg_t)__builtin_amdgcn_kernarg_segment_ptr(), it, s.h, s.hw, c_first, c_end, slot, &lds);
    }
    s.at += take;
    if (s.at >= s.end) return;
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
    __syncthreads();   // the next part's loads overwrite what the last one's join read
  }
}

namespace {

// f(kernel, waves per workgroup, workgroups per CU) of the instance that serves a call.
template <typename F>
void with_rows_kernel(const AttnArgs& p, int mt, F&& f) {
#define QG_ATTN(DP, GRAN, NW, NST)                                                                              \
  do {                                                                                                          \
    if (mt == 1) f(attention_rows_kernel<DP, GRAN, 1, NW, NST>, NW, attn_resident<AttnRowsLds<DP, GRAN, 1, NW, NST>>(NW)); \
    else f(attention_rows_kernel<DP, GRAN, 2, NW, NST>, NW, attn_resident<AttnRowsLds<DP, GRAN, 2, NW, NST>>(NW));         \
  } while (0)
  const int gran = p.fp8 ? p.gran : 0;
  if (p.d <= 64) {
    if (gran == 0) QG_ATTN(64, 0, 4, 2);
    else if (gran == 32) QG_ATTN(64, 32, 4, 2);
    else QG_ATTN(64, 64, 4, 2);
  } else if (p.d <= 128) {
    if (gran == 0) QG_ATTN(128, 0, 4, 2);
    else if (gran == 32) QG_ATTN(128, 32, 4, 2);
    else if (gran == 64) QG_ATTN(128, 64, 4, 2);
    else QG_ATTN(128, 128, 4, 2);
  } else {
    if (gran == 0) QG_ATTN(256, 0, 2, 2);
    else if (gran == 32) QG_ATTN(256, 32, 2, 2);
    else if (gran == 64) QG_ATTN(256, 64, 2, 2);
    else QG_ATTN(256, 128, 2, 2);
  }
#undef QG_ATTN
}

}  // namespace

void attention_rows_shape(AttnArgs& p, int mt) {
  with_rows_kernel(p, mt, [&](auto, int nw, int resident) {
    p.target = p.num_cus * resident;
    p.hw = nw;
    while (p.hkv % p.hw != 0) p.hw /= 2;
  });
}

hipError_t launch_attention_rows(const AttnArgs& p, int mt, unsigned grid, hipStream_t stream) {
  with_rows_kernel(p, mt, [&](auto kernel, int nw, int) { kernel<<<grid, nw * 64, 0, stream>>>(p); });
  return hipGetLastError();
}

}  // namespace qg
