// Attention of ragged rows of new tokens over a paged KV cache (bf16, or e4m3
// codes with one f32 scale per run of head-dim elements).
//
// Token j of sequence b sits at position p = cache_lengths[b] + j. For query
// head h and its key/value head g = h / (Hq / Hkv)
//
//   s_i = scale * sum_d q[d] * k_i[d]          over the positions i it sees
//   out = sum_i e^(s_i - m) v_i / sum_i e^(s_i - m)
//
// The rows of a tile are the (token, query head) pairs of one key/value head,
// token-major, so a key/value head's pages are read once for all query heads
// that share it. Each wave owns 32 rows and computes the scores transposed,
// S^T = K Q^T with 32x32x16 MFMAs: a lane then holds scores of one row only, the
// running maximum and sum need one exchange with the other half of the wave, and
// the probabilities are already the B operand of O^T = V^T P^T (the key slots of
// that product come in the order the scores lie in, and the transposed reads of
// V name the same order).
//
// Numbers: products of bf16 are summed in fp32; e4m3 codes enter as bf16
// (exact), a key's scale multiplies the fp32 partial score of its run and a
// value's scale its probability in fp32. Maximum, sum and output accumulators
// are fp32. The one rounding inside is that of the probabilities to bf16, which
// the MFMA takes (at most 2^-8 of each, as the output's own rounding).
//
// A position that a row must not see takes a score of -infinity by selection.
// Its value row is still multiplied, by zero: where it holds an infinity or NaN
// the row's output would turn NaN. So a tile whose result is not finite is
// computed again with the values selected per token.
#include "attention_common.h"

namespace qg {

namespace {

constexpr int AW = 4;            // waves
constexpr int ABM = 32 * AW;     // rows per tile

// 16-byte chunk c of LDS row r (DP bf16 elements): the 16 rows of a read phase of
// the key fragments, and the 4 x 64 bytes of a transposed read of values, meet
// different banks
template <int DP>
__device__ __forceinline__ int swz_k(int r, int c) {
  return DP >= 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}
template <int DP>
__device__ __forceinline__ int swz_v(int r, int c) {
  return DP >= 128 ? c ^ (((r & 3) << 2) | ((r >> 2) & 3)) : c ^ (((r >> 1) & 1) << 2 | ((r >> 2) & 3));
}

struct Rows {
  int b, tile;          // sequence, tile of its rows
};

// tile t of the launch: sequences in order, ceil(new * group / ABM) tiles each
__device__ __forceinline__ Rows locate_rows(int t, const uint32_t* __restrict__ offs, int batch, int group) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int b0 = 0; b0 < batch; b0 += 64) {
    const int b = b0 + lane;
    int cnt = 0;
    if (b < batch) cnt = ((int)(offs[b + 1] - offs[b]) * group + ABM - 1) / ABM;
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const unsigned long long hit = __ballot(t < base + incl);
    if (hit) {
      const int first = __ffsll((long long)hit) - 1;
      const int excl = __shfl(incl - cnt, first);
      return Rows{__builtin_amdgcn_readfirstlane(b0 + first), __builtin_amdgcn_readfirstlane(t - base - excl)};
    }
    base += __shfl(incl, 63);
  }
  return Rows{-1, 0};
}

// 16 e4m3 codes -> 16 bf16 (exact)
__device__ __forceinline__ void e4m3_to_bf16(u32x4_t v, u32x4_t& lo, u32x4_t& hi) {
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[k], false);
    const float2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[k], true);
    o[2 * k] = f2bf2_rn(a.x, a.y);
    o[2 * k + 1] = f2bf2_rn(b.x, b.y);
  }
  lo = u32x4_t{o[0], o[1], o[2], o[3]};
  hi = u32x4_t{o[4], o[5], o[6], o[7]};
}

}  // namespace

template <int DP, bool FP8>
__global__ __launch_bounds__(AW * 64) void attention_tile_kernel(AttnArgs p) {
  constexpr int KB = DP > 128 ? 32 : 64;      // keys per step
  constexpr int NB = KB / 32;
  constexpr int NS = DP / 16;                 // MFMA steps of a score
  constexpr int ND = DP / 32;                 // 32-wide strips of the output
  constexpr int CH = DP / 8;                  // 16-byte chunks per LDS row
  constexpr int MAXR = FP8 ? DP / 32 : 1;     // scale runs per head, at most
  __shared__ __attribute__((aligned(16))) u32x4_t lds_k[KB * CH];
  __shared__ __attribute__((aligned(16))) u32x4_t lds_v[KB * CH];
  __shared__ __attribute__((aligned(16))) float lds_s[2][MAXR][KB];   // run scales of keys, values

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int h = blockIdx.x % p.hkv;
  const Rows loc = locate_rows(blockIdx.x / p.hkv, p.offs, p.batch, p.group);
  if (loc.b < 0) return;
  const int row0 = (int)p.offs[loc.b], fresh = (int)p.offs[loc.b + 1] - row0;
  const int cached = (int)p.cache_len[loc.b];
  const int rows = fresh * p.group;
  const int r_first = loc.tile * ABM, r_last = min(rows, r_first + ABM) - 1;
  const int t_first = r_first / p.group, t_last = r_last / p.group;   // tokens of the tile
  // positions that some row of the tile sees: [begin, end)
  const int end = p.causal ? cached + t_last + 1 : cached + fresh;
  const int begin = p.window ? max(0, cached + t_first - p.window + 1) : 0;

  // this lane's row
  const int r = r_first + wave * 32 + col;
  const bool valid = r < rows;
  const int tok = min(r, rows - 1) / p.group;
  const int head = h * p.group + min(r, rows - 1) % p.group;
  const int hi = p.causal ? cached + tok : cached + fresh - 1;        // last and first position it sees
  const int lo = p.window ? cached + tok - p.window + 1 : 0;
  const size_t row_at = ((size_t)(row0 + tok) * p.hq + head) * p.d;

  u32x4_t qf[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int d = 16 * s + 8 * half;
    qf[s] = u32x4_t{0, 0, 0, 0};
    if (d < p.d) qf[s] = *reinterpret_cast<const u32x4_t*>(p.q + row_at + d);
  }
  const float cs = p.scale * kLog2e;
  const int run_steps = FP8 ? p.gran / 16 : NS;
  const int runs = FP8 ? p.d / p.gran : 1;
  const long long cache_row = (long long)p.hkv * p.d;                 // elements of a (page, slot) row
  const long long plane_rows = p.pages * p.page_size;
  const uint32_t* __restrict__ my_pages = p.page_table + (size_t)loc.b * p.max_pages;
  // first and last token of the wave's rows (the safe pass goes token by token)
  const int wt_first = min(r_first + wave * 32, rows - 1) / p.group;
  const int wt_last = min(r_first + wave * 32 + 31, rows - 1) / p.group;

  float16_t acc[ND];
  float m, l;
  for (int pass = 0; pass < 2; ++pass) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][i] = 0.f;

    for (int k0 = begin / KB * KB; k0 < end; k0 += KB) {
      __syncthreads();
      // keys and values of positions k0 .. k0 + KB - 1; positions outside
      // [begin, end) re-read a position inside (their pages may not exist)
      constexpr int EL = FP8 ? 16 : 8;            // elements of a 16-byte load
      constexpr int LC = DP / EL;
      for (int e = tid; e < 2 * KB * LC; e += AW * 64) {
        const int plane = e / (KB * LC), key = e / LC % KB, c = e % LC;
        const int pos = min(max(k0 + key, begin), end - 1);
        const long long at = (((long long)p.layer * 2 + plane) * plane_rows + (long long)my_pages[pos / p.page_size] * p.page_size +
                              pos % p.page_size) * cache_row + (long long)h * p.d + c * EL;
        u32x4_t v = {0, 0, 0, 0};
        u32x4_t* dst = plane ? lds_v : lds_k;
        if constexpr (FP8) {
          if (c * EL < p.d) v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(p.blocks) + at);
          u32x4_t a, b;
          e4m3_to_bf16(v, a, b);
          dst[key * CH + (plane ? swz_v<DP>(key, 2 * c) : swz_k<DP>(key, 2 * c))] = a;
          dst[key * CH + (plane ? swz_v<DP>(key, 2 * c + 1) : swz_k<DP>(key, 2 * c + 1))] = b;
        } else {
          if (c * EL < p.d) v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p.blocks) + at);
          dst[key * CH + (plane ? swz_v<DP>(key, c) : swz_k<DP>(key, c))] = v;
        }
      }
      if constexpr (FP8) {
        for (int e = tid; e < 2 * KB * runs; e += AW * 64) {
          const int plane = e / (KB * runs), key = e / runs % KB, run = e % runs;
          const int pos = min(max(k0 + key, begin), end - 1);
          const long long at = (((long long)p.layer * 2 + plane) * plane_rows +
                                (long long)my_pages[pos / p.page_size] * p.page_size + pos % p.page_size) *
                                   (p.hkv * runs) + (long long)h * runs + run;
          lds_s[plane][run][key] = p.scales[at];
        }
      }
      __syncthreads();

      // scores: register i of block nb holds key 32 nb + 8 (i / 4) + 4 half + i % 4
      float16_t sc[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[nb][i] = 0.f;
        float16_t part = sc[nb];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const int key = nb * 32 + col;
          part = mfma32x32x16_bf16(lds_k[key * CH + swz_k<DP>(key, 2 * s + half)], qf[s], part);
          if constexpr (FP8) {
            if ((s + 1) % run_steps == 0 && (s + 1) * 16 <= p.d) {
              const int run = (s + 1) / run_steps - 1;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                sc[nb][i] += part[i] * lds_s[0][run][nb * 32 + 8 * (i / 4) + 4 * half + i % 4];
                part[i] = 0.f;
              }
            }
          }
        }
        if constexpr (!FP8) sc[nb] = part;
      }
      // positions a row does not see
      const bool masked = (p.window && k0 < cached + t_last - p.window + 1) ||
                          k0 + KB > (p.causal ? cached + t_first + 1 : end);
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int pos = k0 + nb * 32 + 8 * (i / 4) + 4 * half + i % 4;
            if (pos > hi || pos < lo) sc[nb][i] = -INFINITY;
          }
      }
      float mx = m;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[nb][i]);
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      // a row that has seen nothing yet keeps m = -infinity; its probabilities are 0
      const float base = mx == -INFINITY ? 0.f : mx * cs;
      const float alpha = __builtin_amdgcn_exp2f((m == -INFINITY ? -INFINITY : m * cs) - base);
      m = mx;
      float sum = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          sc[nb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[nb][i], cs, -base));
          sum += sc[nb][i];
        }
      l = l * alpha + sum;
#pragma unroll
      for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[n][i] *= alpha;

#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          u32x4_t pf = {f2bf2_rn(sc[nb][8 * ks], sc[nb][8 * ks + 1]), f2bf2_rn(sc[nb][8 * ks + 2], sc[nb][8 * ks + 3]),
                        f2bf2_rn(sc[nb][8 * ks + 4], sc[nb][8 * ks + 5]), f2bf2_rn(sc[nb][8 * ks + 6], sc[nb][8 * ks + 7])};
          const int key0 = nb * 32 + ks * 16 + 4 * half;   // slots 0..3: key0 + 0..3, slots 4..7: key0 + 8..11
          int run_at = -1;
#pragma unroll
          for (int n = 0; n < ND; ++n) {
            if constexpr (FP8) {   // probabilities times the value scales of this strip's run
              const int run = min(n * 32 / p.gran, runs - 1);
              if (run != run_at) {
                run_at = run;
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int key = key0 + e % 4 + 8 * (e / 4);
                  w[e] = sc[nb][8 * ks + e] * lds_s[1][run][key];
                  if (pass && (k0 + key > hi || k0 + key < lo)) w[e] = 0.f;   // the scale may be NaN
                }
                pf = u32x4_t{f2bf2_rn(w[0], w[1]), f2bf2_rn(w[2], w[3]), f2bf2_rn(w[4], w[5]), f2bf2_rn(w[6], w[7])};
              }
            }
            // lane m of a 16-lane group names row m / 4 and elements 4 (m % 4) .. + 3 of
            // 16 columns, and receives the four rows of column m
            const int m16 = lane & 15, c0 = n * 32 + 16 * ((lane >> 4) & 1) + 4 * (m16 & 3);
            uint32_t vw[4];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int key = key0 + 8 * g + (m16 >> 2);
              const char* at = reinterpret_cast<const char*>(lds_v + key * CH + swz_v<DP>(key, c0 >> 3)) + (c0 & 7) * 2;
              const s16x4_t t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4_t*)(const_cast<char*>(at)));
              const uint64_t u = __builtin_bit_cast(uint64_t, t);
              vw[2 * g] = (uint32_t)u;
              vw[2 * g + 1] = (uint32_t)(u >> 32);
            }
            const u32x4_t vf = {vw[0], vw[1], vw[2], vw[3]};
            if (pass == 0 || !masked) {
              acc[n] = mfma32x32x16_bf16(vf, pf, acc[n]);
            } else {
              for (int t = wt_first; t <= wt_last; ++t) {
                const int t_hi = p.causal ? cached + t : cached + fresh - 1, t_lo = p.window ? cached + t - p.window + 1 : 0;
                uint32_t keep[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int pos = k0 + key0 + e % 4 + 8 * (e / 4);
                  keep[e] = pos <= t_hi && pos >= t_lo ? 0xFFFFu : 0u;
                }
                const u32x4_t vs = {vw[0] & (keep[0] | keep[1] << 16), vw[1] & (keep[2] | keep[3] << 16),
                                    vw[2] & (keep[4] | keep[5] << 16), vw[3] & (keep[6] | keep[7] << 16)};
                const float16_t with = mfma32x32x16_bf16(vs, pf, acc[n]);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[n][i] = t == tok ? with[i] : acc[n][i];
              }
            }
          }
        }
      }
    }
    int off = 0;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) off |= !(fabsf(acc[n][i]) < INFINITY);
    if (pass == 0 && !__syncthreads_or(off)) break;
  }

  l += __shfl_xor(l, 32);
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // a NaN sum stays NaN
  if (valid) {
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = n * 32 + 8 * g + 4 * half;
        if (d < p.d) {
          u32x2_t o = {f2bf2_rn(acc[n][4 * g] * inv, acc[n][4 * g + 1] * inv),
                       f2bf2_rn(acc[n][4 * g + 2] * inv, acc[n][4 * g + 3] * inv)};
          *reinterpret_cast<u32x2_t*>(p.out + row_at + d) = o;
        }
      }
  }
}

hipError_t launch_attention_tiles(AttnArgs p, hipStream_t stream) {
  // sequence b has ceil(new_b * group / ABM) tiles per key/value head: at most
  // floor(T * group / ABM) + batch in all; workgroups past the last tile return
  const long long tiles = p.T * p.group / ABM + p.batch;
  if (tiles * p.hkv > INT32_MAX) return hipErrorNotSupported;
  const dim3 grid((unsigned)(tiles * p.hkv));
#define QG_ATTN(DP)                                                          \
  do {                                                                       \
    if (p.fp8) attention_tile_kernel<DP, true><<<grid, AW * 64, 0, stream>>>(p);  \
    else attention_tile_kernel<DP, false><<<grid, AW * 64, 0, stream>>>(p);       \
  } while (0)
  if (p.d <= 64) QG_ATTN(64);
  else if (p.d <= 128) QG_ATTN(128);
  else QG_ATTN(256);
#undef QG_ATTN
  return hipGetLastError();
}

}  // namespace qg
