// Attention over the paged cache for few rows per key/value head (single tokens,
// drafted tokens): a stream over the cache, bound by HBM.
//
// A tile is 16 * MT (token, query head) rows. A workgroup takes one chunk of one
// tile's positions; its waves take blocks of 32 positions in turn, each with its
// own ring of two blocks in LDS, filled by direct-to-LDS loads (no registers
// held, no barrier between the waves). Scores come transposed from 16x16x32
// MFMAs, S^T = K Q^T: a lane holds eight scores of one row, and they are, as they
// lie, the B operand of O^T = V^T P^T with the key slots in the order
// {4j .. 4j + 3, 16 + 4j .. 16 + 4j + 3} for lane quarter j; the transposed reads
// of V name its rows in that order.
//
// The MFMAs have time to spare here, so a probability enters as two bf16 (value
// and remainder): the result is that of fp32 probabilities, rounded once.
#include "attention_common.h"

namespace qg {

namespace {

constexpr int RPG = 1024;   // page table entries held in LDS at a time

// LDS rows of CH 16-byte chunks: chunk c of row r lies at c ^ swz(r). A read phase
// of key fragments takes 16 rows of one chunk column, a phase of transposed value
// reads 8 rows (bf16; 16 rows of e4m3) of one strip; both meet different banks.
template <int CH>
__device__ __forceinline__ int swz_rk(int r) {
  return CH >= 16 ? r & 15 : CH == 8 ? (r >> 1) & 7 : (r >> 2) & 3;
}
template <int CH, bool FP8>
__device__ __forceinline__ int swz_rv(int r) {
  if (!FP8) return CH >= 16 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
  return CH >= 16 ? (r & 7) | ((r >> 4) & 1) << 3 : CH == 8 ? ((r >> 1) & 3) | ((r >> 4) & 1) << 2 : ((r >> 2) & 1) | ((r >> 4) & 1) << 1;
}

}  // namespace

template <int DP, bool FP8, int MT, int NW>
__global__ __launch_bounds__(NW * 64) void attention_rows_kernel(AttnArgs p) {
  constexpr int ES = FP8 ? 1 : 2;              // bytes per cached element
  constexpr int CH = DP * ES / 16;             // chunks per LDS row
  constexpr int TILE = 32 * CH;                // chunks of a block's keys (or values)
  constexpr int LD = TILE / 64;                // loads per lane for them
  constexpr int NS = DP / 32;                  // MFMA steps of a score
  constexpr int ND = DP / 16;                  // 16-wide strips of the output
  constexpr int MAXR = FP8 ? DP / 32 : 1;
  constexpr int NT = NW * 64;
  // floats per row of a wave's partial output in LDS
  constexpr int OS = 16 * MT * (DP + 4) * 4 <= 4 * TILE * 16 ? DP + 4 : DP;
  static_assert(16 * MT * OS * 4 <= 4 * TILE * 16, "a wave's partial output fits its ring");
  __shared__ __attribute__((aligned(16))) u32x4_t ring[NW][2][2][TILE];      // [wave][block parity][keys, values]
  __shared__ __attribute__((aligned(16))) float ring_s[FP8 ? NW : 1][2][MAXR][2][32];   // run scales [run][keys, values][position]
  __shared__ uint32_t pages[RPG];
  __shared__ float w_m[NW][16 * MT], w_l[NW][16 * MT];
  __shared__ AttnScan<NT> scan;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, j = lane >> 4;
  const int h = blockIdx.x % p.hkv;
  const AttnItem it = attn_locate<NT, false>(p, blockIdx.x / p.hkv, scan);
  if (it.b < 0) return;
  const AttnTile t = attn_tile(p, it);
  const int c_first = t.start + it.split * it.chunk;          // this item's positions [c_first, c_end)
  const int c_end = min(t.end, c_first + it.chunk);
  if (c_first >= c_end) return;                               // the sequence's longer tiles need this chunk
  const bool alone = t.end - t.start <= it.chunk;

  // rows of this lane, one per 16-row tile
  const int rows = it.fresh * p.group;
  int tok[MT], hi[MT], lo[MT];
  u32x4_t qf[MT][NS];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = min(t.r_first + 16 * mt + col, rows - 1);
    tok[mt] = r / p.group;
    hi[mt] = p.causal ? it.cached + tok[mt] : it.cached + it.fresh - 1;
    lo[mt] = p.window ? it.cached + tok[mt] - p.window + 1 : 0;
    const uint16_t* q = p.q + ((size_t)(it.row0 + tok[mt]) * p.hq + h * p.group + r % p.group) * p.d;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = 32 * s + 8 * j;
      qf[mt][s] = d < p.d ? *reinterpret_cast<const u32x4_t*>(q + d) : u32x4_t{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int s = 0; s < NS; ++s) arrived(qf[mt][s]);
  const int runs = FP8 ? p.d / p.gran : 1;
  const int run_steps = FP8 ? p.gran / 32 : NS;
  const int chunks = p.d * ES / 16;                           // chunks of a cache row that exist
  // head dims between p.d and DP: never loaded, zero from here on
  if (chunks < CH) {
    for (int e = tid; e < NW * 4 * TILE; e += NT) (&ring[0][0][0][0])[e] = u32x4_t{0, 0, 0, 0};
  }
  const float cs = p.scale * kLog2e;
  const size_t row_bytes = (size_t)p.hkv * p.d * ES;          // a (page, slot) row
  const size_t plane_bytes = (size_t)p.pages * p.page_size * row_bytes;
  const char* keys = static_cast<const char*>(p.blocks) + 2 * p.layer * plane_bytes + (size_t)h * p.d * ES;
  const size_t plane_scales = (size_t)p.pages * p.page_size * p.hkv * runs;
  const float* key_scales = FP8 ? p.scales + 2 * p.layer * plane_scales + (size_t)h * runs : nullptr;
  const uint32_t* my_pages = p.page_table + (size_t)it.b * p.max_pages;

  float4_t acc[MT][ND];
  float m[MT], l[MT];
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = -INFINITY;
      l[mt] = 0.f;
#pragma unroll
      for (int n = 0; n < ND; ++n) acc[mt][n] = float4_t{0.f, 0.f, 0.f, 0.f};
    }
    // as many positions at a time as the list of pages covers
    const int seg = (int)min((long long)it.chunk, (long long)(RPG - 1) * p.page_size / (32 * NW) * (32 * NW));
    for (int s_first = c_first; s_first < c_end; s_first += seg) {
      const int s_end = min(c_end, s_first + seg);
      const int page0 = fast_div(max(s_first, t.begin), p.div_mul, p.div_shift);
      const int page1 = fast_div(s_end - 1, p.div_mul, p.div_shift);
      __syncthreads();
      for (int e = tid; e <= page1 - page0; e += NT) pages[e] = my_pages[page0 + e];
      __syncthreads();

      // block i of the segment into slot `at` of this wave's ring. Positions outside
      // [begin, end) re-read one inside (their pages may not exist).
      auto row_of = [&](int pos) {
        const int x = min(max(pos, t.begin), s_end - 1);
        const uint32_t pg = fast_div(x, p.div_mul, p.div_shift);
        return (size_t)pages[pg - page0] * p.page_size + (x - pg * p.page_size);
      };
      auto issue = [&](int i, int at) {
        wait_lds();
        const int first = s_first + 32 * i;
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const int e = k * 64 + lane, key = e / CH, c = e % CH;
          const size_t off = row_of(first + key) * row_bytes;
          const int ck = c ^ swz_rk<CH>(key), cv = c ^ swz_rv<CH, FP8>(key);
          if (ck < chunks) dma16_at(keys + off + ck * 16, lds_addr(&ring[wave][at][0][k * 64]));
          if (cv < chunks) dma16_at(keys + off + plane_bytes + cv * 16, lds_addr(&ring[wave][at][1][k * 64]));
        }
        if constexpr (FP8) {
          const size_t off = row_of(first + (lane & 31)) * (p.hkv * runs) + (lane >> 5) * plane_scales;
#pragma unroll
          for (int r = 0; r < MAXR; ++r)   // the same number of loads whatever `runs`: wait_loads counts them
            dma4_at(key_scales + off + min(r, runs - 1), lds_addr(&ring_s[wave][at][r][0][0]));
        }
      };

      const int blocks = (s_end - s_first + 31) / 32;
      if (wave < blocks) issue(wave, 0);
      int at = 0;
      for (int i = wave; i < blocks; i += NW, at ^= 1) {
        if (i + NW < blocks) {
          issue(i + NW, at ^ 1);
          wait_loads<2 * LD + (FP8 ? MAXR : 0)>();
        } else {
          wait_loads<0>();
        }
        const int k0 = s_first + 32 * i;
        const u32x4_t* lk = ring[wave][at][0];
        const char* lv = reinterpret_cast<const char*>(ring[wave][at][1]);
        const float(*ls)[2][32] = ring_s[FP8 ? wave : 0][at];

        // scores: register i of sc[.][nb] is position k0 + 16 nb + 4 j + i
        float4_t sc[MT][2];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          const int key = 16 * nb + col;
          float4_t part[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sc[mt][nb] = part[mt] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            u32x4_t kf;
            if constexpr (FP8) {
              const int c = 2 * s + (j >> 1);
              const u32x2_t w = *reinterpret_cast<const u32x2_t*>(reinterpret_cast<const char*>(lk + key * CH + (c ^ swz_rk<CH>(key))) + 8 * (j & 1));
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_bf16(w.x, a0, a1);
              e4m3x4_to_bf16(w.y, a2, a3);
              kf = u32x4_t{a0, a1, a2, a3};
            } else {
              kf = lk[key * CH + ((4 * s + j) ^ swz_rk<CH>(key))];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) part[mt] = mfma16x16x32_bf16(kf, qf[mt][s], part[mt]);
            if constexpr (FP8) {
              if ((s + 1) % run_steps == 0 && (s + 1) * 32 <= p.d) {   // a run is complete: times the keys' scales
                const float4_t ks = *reinterpret_cast<const float4_t*>(&ls[(s + 1) / run_steps - 1][0][16 * nb + 4 * j]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                  for (int i4 = 0; i4 < 4; ++i4) sc[mt][nb][i4] = __builtin_fmaf(part[mt][i4], ks[i4], sc[mt][nb][i4]);
                  part[mt] = float4_t{0.f, 0.f, 0.f, 0.f};
                }
              }
            }
          }
          if constexpr (!FP8) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) sc[mt][nb] = part[mt];
          }
        }
        const bool masked = (p.window && k0 < it.cached + t.t_last - p.window + 1) || k0 < t.begin ||
                            k0 + 32 > min(s_end, p.causal ? it.cached + t.t_first + 1 : t.end);
        u32x4_t pf[MT][2];    // probabilities: value and remainder
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (masked) {
            // positions lo .. min(hi, s_end - 1), counted from lo
            const uint32_t seen = max(min(hi[mt], s_end - 1) - lo[mt] + 1, 0), first = k0 + 4 * j - lo[mt];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sc[mt][e >> 2][e & 3] = first + (16 * (e >> 2) + (e & 3)) < seen ? sc[mt][e >> 2][e & 3] : -INFINITY;
          }
          float mx = m[mt];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = fmaxf(mx, sc[mt][e >> 2][e & 3]);
          mx = max_halves(max_quarters(mx));
          // a row that has seen nothing yet keeps m = -infinity; its probabilities are 0
          const float base = mx == -INFINITY ? 0.f : mx * cs;
          const float alpha = __builtin_amdgcn_exp2f((m[mt] == -INFINITY ? -INFINITY : m[mt] * cs) - base);
          m[mt] = mx;
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[mt][e >> 2][e & 3], cs, -base));
            sc[mt][e >> 2][e & 3] = x;
            sum += x;
          }
          l[mt] = l[mt] * alpha + sum;
#pragma unroll
          for (int n = 0; n < ND; ++n) acc[mt][n] *= alpha;
        }
        auto split_p = [&](int mt, int run) {
          uint32_t a[4], b[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x[2], y[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int e = 2 * g + u;
              x[u] = sc[mt][e >> 2][e & 3];
              if constexpr (FP8) {   // times the value's scale of this strip's run
                const int key = 16 * (e >> 2) + 4 * j + (e & 3);
                x[u] *= ls[run][1][key];
                const int pos = k0 + key;
                if (pass && (pos > hi[mt] || pos < lo[mt] || pos >= s_end)) x[u] = 0.f;   // the scale may be NaN
              }
            }
            a[g] = f2bf2_rn(x[0], x[1]);
            y[0] = x[0] - bf2f((uint16_t)a[g]);
            y[1] = x[1] - bf2f((uint16_t)(a[g] >> 16));
            b[g] = f2bf2_rn(y[0], y[1]);
          }
          pf[mt][0] = u32x4_t{a[0], a[1], a[2], a[3]};
          pf[mt][1] = u32x4_t{b[0], b[1], b[2], b[3]};
        };
        if constexpr (!FP8) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) split_p(mt, 0);
        }
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          if constexpr (FP8) {
            if (n * 16 % p.gran == 0 && n * 16 < p.d) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) split_p(mt, n * 16 / p.gran);
            }
          }
          u32x4_t vf;
          if constexpr (FP8) {
            // lane m of a 16-lane group names row m / 2 of eight and eight codes of 16
            const int r = (lane & 15) >> 1, key = (r < 4 ? r : 12 + r) + 4 * j;
            const uint64_t w = lds_read_tr8(lv + (key * CH + (n ^ swz_rv<CH, FP8>(key))) * 16 + 8 * (lane & 1));
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_bf16((uint32_t)w, a0, a1);
            e4m3x4_to_bf16((uint32_t)(w >> 32), a2, a3);
            vf = u32x4_t{a0, a1, a2, a3};
          } else {
            // lane m of a 16-lane group names row m / 4 of four and elements 4 (m % 4) .. + 3 of 16
            const int k1 = 4 * j + ((lane & 15) >> 2), c = 2 * n + ((lane & 2) >> 1);
            const uint64_t w0 = lds_read_tr16(lv + (k1 * CH + (c ^ swz_rv<CH, FP8>(k1))) * 16 + 8 * (lane & 1));
            const uint64_t w1 = lds_read_tr16(lv + ((k1 + 16) * CH + (c ^ swz_rv<CH, FP8>(k1 + 16))) * 16 + 8 * (lane & 1));
            vf = u32x4_t{(uint32_t)w0, (uint32_t)(w0 >> 32), (uint32_t)w1, (uint32_t)(w1 >> 32)};
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (pass == 0 || !masked) {
              acc[mt][n] = mfma16x16x32_bf16(vf, pf[mt][0], acc[mt][n]);
              // (an infinite value times a remainder would be NaN: the second pass goes without)
              if (pass == 0) acc[mt][n] = mfma16x16x32_bf16(vf, pf[mt][1], acc[mt][n]);
            } else {
              // token by token, with the values it does not see set to zero
              for (int tt = t.t_first; tt <= t.t_last; ++tt) {
                const int t_hi = p.causal ? it.cached + tt : it.cached + it.fresh - 1;
                const int t_lo = p.window ? it.cached + tt - p.window + 1 : 0;
                uint32_t keep[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int pos = k0 + 16 * (e >> 2) + 4 * j + (e & 3);
                  keep[e] = pos <= t_hi && pos >= t_lo && pos < s_end ? 0xFFFFu : 0u;
                }
                const u32x4_t vs = {vf.x & (keep[0] | keep[1] << 16), vf.y & (keep[2] | keep[3] << 16),
                                    vf.z & (keep[4] | keep[5] << 16), vf.w & (keep[6] | keep[7] << 16)};
                const float4_t with = mfma16x16x32_bf16(vs, pf[mt][0], acc[mt][n]);
                if (tt == tok[mt]) acc[mt][n] = with;
              }
            }
          }
        }
      }
    }
    int off = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) off |= !(fabsf(acc[mt][n][i]) < INFINITY);
    if (pass == 0 && !__syncthreads_or(off)) break;
  }

  // the waves' results joined through LDS (their rings, which no load targets any more)
  __syncthreads();
  float* mine = reinterpret_cast<float*>(&ring[wave][0][0][0]);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    l[mt] += __shfl_xor(l[mt], 16);
    l[mt] += __shfl_xor(l[mt], 32);
    if (j == 0) {
      w_m[wave][16 * mt + col] = m[mt] == -INFINITY ? -INFINITY : m[mt] * cs;
      w_l[wave][16 * mt + col] = l[mt];
    }
#pragma unroll
    for (int n = 0; n < ND; ++n) *reinterpret_cast<float4_t*>(mine + (16 * mt + col) * OS + 16 * n + 4 * j) = acc[mt][n];
  }
  __syncthreads();
  const int slot = it.slots + (it.tile * p.hkv + h) * it.nsplit + it.split;
  float* ws = p.workspace + (size_t)slot * attn_slot_floats(16 * MT, DP);
  for (int e = tid; e < t.r_count * (DP / 4); e += NT) {
    const int r = e / (DP / 4), d = e % (DP / 4) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, w_m[w][r]);
    const float base = top == -INFINITY ? 0.f : top;
    float4_t o = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = __builtin_amdgcn_exp2f(w_m[w][r] - base);
      const float4_t x = *reinterpret_cast<const float4_t*>(reinterpret_cast<const float*>(&ring[w][0][0][0]) + r * OS + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], f, o[i]);
      sum = __builtin_fmaf(w_l[w][r], f, sum);
    }
    if (alone) {
      if (d < p.d) {
        const int row = t.r_first + r;
        const float inv = 1.f / sum;   // every row sees a position
        uint16_t* to = p.out + ((size_t)(it.row0 + row / p.group) * p.hq + h * p.group + row % p.group) * p.d + d;
        *reinterpret_cast<u32x2_t*>(to) = u32x2_t{f2bf2_rn(o[0] * inv, o[1] * inv), f2bf2_rn(o[2] * inv, o[3] * inv)};
      }
    } else {
      *reinterpret_cast<float4_t*>(ws + (size_t)r * DP + d) = o;
      if (d == 0) {
        ws[16 * MT * DP + 2 * r] = top;
        ws[16 * MT * DP + 2 * r + 1] = sum;
      }
    }
  }
}

hipError_t launch_attention_rows(AttnArgs p, int mt, hipStream_t stream) {
  const long long tiles = p.T * p.group / p.bm + p.batch;
  // items: at most target + tiles (a chunk is at least the work over the target)
  const long long items = tiles + p.target / p.hkv + 1;
  if (items * p.hkv > INT32_MAX) return hipErrorNotSupported;
  const dim3 grid((unsigned)(items * p.hkv));
#define QG_ATTN(DP, FP8, MT, NW) attention_rows_kernel<DP, FP8, MT, NW><<<grid, NW * 64, 0, stream>>>(p)
#define QG_ATTN_MT(DP, FP8, NW)             \
  do {                                      \
    if (mt == 1) QG_ATTN(DP, FP8, 1, NW);   \
    else QG_ATTN(DP, FP8, 2, NW);           \
  } while (0)
  if (p.fp8) {
    if (p.d <= 64) QG_ATTN_MT(64, true, 4);
    else if (p.d <= 128) QG_ATTN_MT(128, true, 4);
    else QG_ATTN_MT(256, true, 2);
  } else {
    if (p.d <= 64) QG_ATTN_MT(64, false, 4);
    else if (p.d <= 128) QG_ATTN_MT(128, false, 2);
    else QG_ATTN_MT(256, false, 2);
  }
#undef QG_ATTN_MT
#undef QG_ATTN
  return hipGetLastError();
}

}  // namespace qg
