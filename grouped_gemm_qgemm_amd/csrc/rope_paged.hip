// Rotary positions of the new tokens, and the cache's write: queries turned into q_out,
// keys turned and values as they are into their pages, bf16 or e4m3 with a scale per run.
//
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a) * amplitude,   a = position * f
//   s = amax / 448, code = e4m3(x / s)                              per run of G elements
//
// Bound by HBM: every element is read once and written once. A workgroup takes `tokens`
// tokens, more where a token has few heads. It finds their sequences and cache rows
// together, then the cosines and sines of their angles (R / 2 of them serve every head of a
// token), which pass through LDS. A thread then owns one chunk of 8 elements of a head, the
// same for every head and token it works on, and reads the partner chunk as well where pairs
// are R / 2 apart: from the cache line that another lane of its wave asked for anyway.
//
// 36900 tokens of 48 heads of 128 into e4m3 take 161 us, 5.2 TB/s read + written (a large copy:
// 5.1 to 5.4), eight prompts (3445 tokens, bf16) 17.7 us, 64 tokens 5.4 us on the GPU. A thread
// with the loads of one head in flight takes 167 us for the first of these, of two 173, of
// four 163; four tokens per workgroup take 162. Few heads: 32000 tokens of 9 heads of 128 46 us (two
// tokens per workgroup 79; 8 chunks of a thread instead of 6: 43), 41000 of 24 heads of 64 54 (81;
// 57), 18800 of 3 heads of 256 26 (42; 26), 64-bit angles being half of that: one of them serves
// two heads.
//
// Pairs R / 2 apart with R / 2 no multiple of 8 find their partners by eight loads of 2 bytes at the point
// of use: 36900 tokens of 40 heads of 72, bf16, 123 us, where pairs side by side take 83 (5.1 TB/s); 48 heads of
// 80 with R = 40 145, with R = 64 or 80 108.
//
// The angle a = position * f is a product of 31 and 24 bits, of which a far position keeps
// few behind the point: its reduction carries what each 64-bit product rounds away, so that
// every position's part of a turn is exact to fp32. From there on fp32 is enough.
#include <algorithm>

#include "paged_common.h"

namespace qg {

namespace {

constexpr int RT = 256;            // threads
constexpr int RTOK = 16;           // tokens per workgroup, at most
constexpr int RHEADS = 3;          // heads whose loads a thread has in flight
constexpr int RANGLES = 2048;      // angles per workgroup, at most (a token has up to 512)
constexpr int RWORK = 6;           // chunks of a thread that fill a workgroup's tokens
enum { PAIRS_APART = 0, PAIRS_ODD = 1, PAIRS_SIDE = 2 };   // R / 2 apart (a multiple of 8, or not), side by side

// t * f / (2 pi) less the nearest whole number
__device__ __forceinline__ float part_of_turn(double t, double f) {
  constexpr double kInv = 0.15915494309189535, kRest = -9.839338337591243e-18;   // 1 / (2 pi), and what that lacks
  const double a = t * f, a_rest = __builtin_fma(t, f, -a);
  const double n = a * kInv, n_rest = __builtin_fma(a, kInv, -n) + (a * kRest + a_rest * kInv);
  return (float)((n - rint(n)) + n_rest);
}

// largest magnitude, of which a scale is made; NaN elements do not count
__device__ __forceinline__ float largest8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}

// e4m3(x / s), nearest even; x / s may pass 448 where s is subnormal and was rounded. NaN's code is
// NaN, also where a run has no other elements but zeros, and the scale 0.
__device__ __forceinline__ float code_value(float x, float s) {
  const float v = s > 0.f ? x / s : x == x ? 0.f : x;
  return fabsf(v) > 448.f ? copysignf(448.f, v) : v;
}

__device__ __forceinline__ void unpack8(u32x4_t v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    x[2 * i] = bf2f((uint16_t)w);
    x[2 * i + 1] = bf2f((uint16_t)(w >> 16));
  }
}

// Cache rows and positions of this wave's tokens, wave, wave + 4, .. of the workgroup's: as
// owner_of, N of them at a time.
template <int N>
__device__ __forceinline__ void find(const RopeArgs& p, long long r0, long long rows, long long* s_row, double* s_pos) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int lo[N] = {}, n = p.kv.batch;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = lane * step;
    uint32_t x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = p.offs[min(lo[k] + at, p.kv.batch - 1)];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const bool below = at < n && lo[k] + at < p.kv.batch && x[k] <= (uint32_t)(r0 + wave + k * (RT / 64));
      lo[k] += max(__popcll(__ballot(below)) - 1, 0) * step;   // (offs[0] = 0: lane 0 always is)
    }
    n = step;
  }
  int b = lo[0];
#pragma unroll
  for (int k = 1; k < N; ++k) b = lane == k ? lo[k] : b;
  const int tok = wave + lane * (RT / 64);
  const long long r = r0 + tok;
  if (lane < N && r < rows) {
    const uint32_t at = p.kv.cache_len[b] + ((uint32_t)r - p.offs[b]);
    s_pos[tok] = p.positions ? (double)p.positions[r] : (double)at;
    s_row[tok] = p.k ? cache_row(p.kv, b, at) : 0;
  }
}

}  // namespace

// SHORT: a thread's turn of RHEADS heads is more than a token has.
template <bool FP8, int PAIRS, bool SHORT>
__global__ __launch_bounds__(RT) void rope_paged_kernel(RopeArgs p, int tokens) {
  __shared__ __attribute__((aligned(16))) float s_cos[RANGLES], s_sin[RANGLES];
  __shared__ long long s_row[RTOK];
  __shared__ double s_pos[RTOK];
  const int tid = threadIdx.x;
  const long long r0 = (long long)blockIdx.x * tokens;
  const int half = p.half, d = p.kv.d;
  const int angle = half > 0 ? tid % half : 0;
  const float freq = half > 0 ? p.inv_freq[angle] : 0.f;   // of this thread's first angle
  const long long rows = min((long long)p.offs[p.kv.batch], (long long)p.T);
  if (tokens > RT / 64) find<RTOK / (RT / 64)>(p, r0, min(rows, r0 + tokens), s_row, s_pos);
  else if (tid < 64 * tokens) find<1>(p, r0, rows, s_row, s_pos);
  const int count = (int)min((long long)tokens, rows - r0);   // (negative behind the last sequence)
  __syncthreads();
  for (int e = tid; e < count * half; e += RT) {
    const int t = e / half, i = e - t * half;
    float sn, cs;
    sincospif(2.f * part_of_turn(s_pos[t], (double)(e == tid ? freq : p.inv_freq[i])), &sn, &cs);
    s_cos[e] = cs * p.amplitude;
    s_sin[e] = sn * p.amplitude;
  }
  __syncthreads();

  const int ch = d >> 3, per = RT / ch;            // chunks of a head, heads at a time
  const int slot = tid / ch, c = tid - slot * ch;
  if (slot >= per) return;
  const int hq = p.q ? p.hq : 0, hkv = p.kv.hkv, heads = hq + (p.k ? 2 * hkv : 0);
  const int first = 8 * c;                         // this thread's elements: first .. first + 7
  const bool turned = first < 2 * half;
  const size_t plane = (size_t)p.kv.pages * p.kv.page_size * hkv;   // (page, slot, head) rows of a plane
  const int runs = FP8 ? d / p.kv.gran : 1, lanes = FP8 ? p.kv.gran >> 3 : 1;
  u32x4_t raw[RHEADS], other[RHEADS];
  float cs[8], sn[8];                              // of a token
  auto turn_by = [&](int t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int at;
      if (PAIRS == PAIRS_SIDE) at = (first + i) >> 1;
      else at = first + i < half ? first + i : first + i - half;
      const bool in = first + i < 2 * half;
      cs[i] = in ? s_cos[t * half + (in ? at : 0)] : 1.f;
      sn[i] = in ? s_sin[t * half + (in ? at : 0)] : 0.f;
      const bool second = PAIRS == PAIRS_SIDE ? i & 1 : first + i >= half;
      if (!second) sn[i] = -sn[i];
    }
  };
  auto load = [&](int u, long long r, int h) {
    const uint16_t* src = h < hq ? p.q + r * p.q_stride + (size_t)h * d
                          : h >= hq + hkv ? p.v + r * p.v_stride + (size_t)(h - hq - hkv) * d
                                          : p.k + r * p.k_stride + (size_t)(h - hq) * d;
    raw[u] = *reinterpret_cast<const u32x4_t*>(src + first);
    if (PAIRS == PAIRS_APART && turned && h < hq + hkv)
      other[u] = *reinterpret_cast<const u32x4_t*>(src + (first < half ? first + half : first - half));
  };
  auto finish = [&](int u, long long r, int h, long long row) {
    const bool is_q = h < hq, is_v = h >= hq + hkv;
    float x[8];
    unpack8(raw[u], x);
    if (turned && !is_v) {
      float y[8];                                  // the other element of each pair
      if (PAIRS == PAIRS_SIDE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
      } else if (PAIRS == PAIRS_APART) {
        unpack8(other[u], y);
      } else {
        const uint16_t* src = is_q ? p.q + r * p.q_stride + (size_t)h * d : p.k + r * p.k_stride + (size_t)(h - hq) * d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = first + i;
          y[i] = bf2f(src[e >= 2 * half ? e : e < half ? e + half : e - half]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = PAIRS == PAIRS_APART || first + i < 2 * half;
        x[i] = in ? __builtin_fmaf(x[i], cs[i], y[i] * sn[i]) : x[i];
      }
    }
    const size_t head_row = (2 * (size_t)p.layer + is_v) * plane + (size_t)row * hkv + (h - hq - (is_v ? hkv : 0));   // of a key or value
    if (is_q || !FP8) {
      const u32x4_t o = {f2bf2_rn(x[0], x[1]), f2bf2_rn(x[2], x[3]), f2bf2_rn(x[4], x[5]), f2bf2_rn(x[6], x[7])};
      uint16_t* to = is_q ? p.q_out + ((size_t)r * hq + h) * d : static_cast<uint16_t*>(p.kv.blocks) + head_row * d;
      *reinterpret_cast<u32x4_t*>(to + first) = o;
    } else {
      // the chunks of a run are neighbouring lanes, all of which are here
      float a = largest8(x);
      for (int k = 1; k < lanes; k <<= 1) a = fmaxf(a, __shfl_xor(a, k));
      const float s = a / 448.0f;
      uint32_t w[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t v = __builtin_amdgcn_cvt_pk_fp8_f32(code_value(x[4 * g], s), code_value(x[4 * g + 1], s), 0, false);
        w[g] = __builtin_amdgcn_cvt_pk_fp8_f32(code_value(x[4 * g + 2], s), code_value(x[4 * g + 3], s), v, true);
      }
      *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.kv.blocks) + head_row * d + first) = u32x2_t{w[0], w[1]};
      if ((c & (lanes - 1)) == 0) p.kv.scales[head_row * runs + first / p.kv.gran] = s;
    }
  };

  // the loads of several heads before the first of them is stored
  if constexpr (!SHORT) {                          // all of them of one token
    for (int t = 0; t < count; ++t) {
      const long long r = r0 + t, row = s_row[t];
      if (turned) turn_by(t);
      for (int h0 = slot; h0 < heads; h0 += RHEADS * per) {
#pragma unroll
        for (int u = 0; u < RHEADS; ++u) load(u, r, min(h0 + u * per, heads - 1));
#pragma unroll
        for (int u = 0; u < RHEADS; ++u) {
          if (h0 + u * per >= heads) break;
          finish(u, r, h0 + u * per, row);
        }
      }
    }
  } else {
    const int next_t = per / heads, next_h = per - next_t * heads;   // from one of a thread's heads to its next
    int t = slot / heads, h = slot - t * heads, held = -1;
    while (t < count) {
      int ts[RHEADS], hs[RHEADS];
#pragma unroll
      for (int u = 0; u < RHEADS; ++u) {
        ts[u] = t;
        hs[u] = h;
        load(u, r0 + min(t, count - 1), h);
        t += next_t;
        h += next_h;
        if (h >= heads) {
          h -= heads;
          ++t;
        }
      }
#pragma unroll
      for (int u = 0; u < RHEADS; ++u) {
        if (ts[u] >= count) break;
        if (turned && ts[u] != held) turn_by(held = ts[u]);
        finish(u, r0 + ts[u], hs[u], s_row[ts[u]]);
      }
    }
  }
}

template <bool FP8, int PAIRS>
static void launch(const RopeArgs& p, int tokens, bool few, hipStream_t stream) {
  const unsigned grid = (unsigned)((p.T + tokens - 1) / tokens);
  if (few) rope_paged_kernel<FP8, PAIRS, true><<<grid, RT, 0, stream>>>(p, tokens);
  else rope_paged_kernel<FP8, PAIRS, false><<<grid, RT, 0, stream>>>(p, tokens);
}

hipError_t launch_rope_paged(const RopeArgs& args, hipStream_t stream) {
  RopeArgs p = args;
  divide_pages(p.kv);
  // as many tokens as give every thread RWORK chunks, but four workgroups per CU
  const long long chunks = ((p.q ? p.hq : 0) + (p.k ? 2LL * p.kv.hkv : 0)) * (p.kv.d >> 3);   // of a token
  long long tokens_most = std::min<long long>(RTOK, (RWORK * RT + chunks / 2) / chunks);
  if (p.half > 0) tokens_most = std::min<long long>(tokens_most, RANGLES / p.half);
  const int tokens = (int)std::max<long long>(1, std::min<long long>(tokens_most, p.T / (4LL * p.num_cus)));
  // By token where one fills a turn of RHEADS heads (the first case above 161 us, else 176).
  const bool few = chunks < RHEADS * RT;
  const int pairs = p.interleaved ? PAIRS_SIDE : p.half % 8 == 0 ? PAIRS_APART : PAIRS_ODD;
#define QG_ROPE(FP8)                                                                                                   \
  do {                                                                                                                 \
    if (pairs == PAIRS_SIDE) launch<FP8, PAIRS_SIDE>(p, tokens, few, stream);                                            \
    else if (pairs == PAIRS_APART) launch<FP8, PAIRS_APART>(p, tokens, few, stream);                                     \
    else launch<FP8, PAIRS_ODD>(p, tokens, few, stream);                                                                 \
  } while (0)
  if (p.k && p.kv.fp8) QG_ROPE(true);
  else QG_ROPE(false);
#undef QG_ROPE
  return hipGetLastError();
}

}  // namespace qg
