// Rotary positions of the new tokens, and the cache's write: queries turned into q_out,
// keys turned and values as they are into their pages, bf16 or e4m3 with a scale per run.
//
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a) * amplitude,   a = position * f
//   s = amax / 448, code = e4m3(x / s)                              per run of G elements
//
// Bound by HBM: every element is read once and written once. A workgroup takes `tokens`
// tokens. One wave per token finds its sequence and cache row and the cosines and sines
// of its angles (R / 2 of them serve every head), which pass through LDS. A thread then
// owns one chunk of 8 elements of a head, the same for every head and token it works on,
// and reads the partner chunk as well where pairs are R / 2 apart: from the cache line that
// another lane of its wave asked for anyway.
//
// 36900 tokens of 48 heads into e4m3 take 160 us, 5.2 TB/s read + written (a large copy:
// 5.1 to 5.4), eight prompts (3445 tokens, bf16) 17.7 us, 64 tokens 5.4 us on the GPU. A thread
// with the loads of one head in flight takes 167 us for the first of these, of two 173, of
// four 163; four tokens per workgroup take 162 us.
//
// The angle a = position * f is a product of 31 and 24 bits, of which a far position keeps
// few behind the point: its reduction carries what each 64-bit product rounds away, so that
// every position's part of a turn is exact to fp32. From there on fp32 is enough.
#include "paged_common.h"

namespace qg {

namespace {

constexpr int RT = 256;            // threads
constexpr int RTOK = 2;            // tokens per workgroup, at most (a wave each to find its place)
constexpr int RHEADS = 3;          // heads whose loads a thread has in flight
constexpr int RHALF = 512;         // angles per token, at most
enum { PAIRS_APART = 0, PAIRS_ODD = 1, PAIRS_SIDE = 2 };   // R / 2 apart (a multiple of 8, or not), side by side

// t * f / (2 pi) less the nearest whole number
__device__ __forceinline__ float part_of_turn(double t, double f) {
  constexpr double kInv = 0.15915494309189535, kRest = -9.839338337591243e-18;   // 1 / (2 pi), and what that lacks
  const double a = t * f, a_rest = __builtin_fma(t, f, -a);
  const double n = a * kInv, n_rest = __builtin_fma(a, kInv, -n) + (a * kRest + a_rest * kInv);
  return (float)((n - rint(n)) + n_rest);
}

// what the calculation of codes divides by; NaN elements do not count
__device__ __forceinline__ float largest8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}

// e4m3(x / s), nearest even; x / s may pass 448 where s is subnormal and was rounded
__device__ __forceinline__ float code_value(float x, float s) {
  const float v = s > 0.f ? x / s : 0.f;
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

}  // namespace

template <bool FP8, int PAIRS>
__global__ __launch_bounds__(RT) void rope_paged_kernel(RopeArgs p, int tokens) {
  __shared__ __attribute__((aligned(16))) float s_cos[RTOK * RHALF], s_sin[RTOK * RHALF];
  __shared__ long long s_row[RTOK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const long long r0 = (long long)blockIdx.x * tokens;
  const int half = p.half, d = p.kv.d;
  if (wave < tokens) {
    const long long r = r0 + wave;
    const int b = r < p.T ? owner_of(p.offs, p.kv.batch, (uint32_t)r) : -1;
    long long row = -1;
    if (b >= 0) {
      const uint32_t at = p.kv.cache_len[b] + ((uint32_t)r - p.offs[b]);
      row = p.k ? cache_row(p.kv, b, at) : 0;
      const double t = p.positions ? (double)p.positions[r] : (double)at;
      for (int i = lane; i < half; i += 64) {
        float sn, cs;
        sincospif(2.f * part_of_turn(t, (double)p.inv_freq[i]), &sn, &cs);
        s_cos[wave * half + i] = cs * p.amplitude;
        s_sin[wave * half + i] = sn * p.amplitude;
      }
    }
    if (lane == 0) s_row[wave] = row;
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
  for (int t = 0; t < tokens; ++t) {
    const long long row = s_row[t];
    if (row < 0) continue;
    const long long r = r0 + t;
    float cs[8], sn[8];
    if (turned) {
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
    }
    for (int h0 = slot; h0 < heads; h0 += RHEADS * per) {
      // the loads of several heads before the first of them is stored
      u32x4_t raw[RHEADS], other[RHEADS];
#pragma unroll
      for (int u = 0; u < RHEADS; ++u) {
        const int h = min(h0 + u * per, heads - 1);
        const uint16_t* src = h < hq ? p.q + r * p.q_stride + (size_t)h * d
                              : h >= hq + hkv ? p.v + r * p.v_stride + (size_t)(h - hq - hkv) * d
                                              : p.k + r * p.k_stride + (size_t)(h - hq) * d;
        raw[u] = *reinterpret_cast<const u32x4_t*>(src + first);
        if (PAIRS == PAIRS_APART && turned && h < hq + hkv)
          other[u] = *reinterpret_cast<const u32x4_t*>(src + (first < half ? first + half : first - half));
      }
#pragma unroll
      for (int u = 0; u < RHEADS; ++u) {
        const int h = h0 + u * per;
        if (h >= heads) break;
        const bool is_q = h < hq, is_v = h >= hq + hkv;
        float x[8];
        unpack8(raw[u], x);
        if (turned && !is_v) {
          float y[8];                                // the other element of each pair
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
        if (is_q || !FP8) {
          const u32x4_t o = {f2bf2_rn(x[0], x[1]), f2bf2_rn(x[2], x[3]), f2bf2_rn(x[4], x[5]), f2bf2_rn(x[6], x[7])};
          uint16_t* to = is_q ? p.q_out + ((size_t)r * hq + h) * d
                              : static_cast<uint16_t*>(p.kv.blocks) +
                                    ((2 * (size_t)p.layer + is_v) * plane + (size_t)row * hkv + (h - hq - (is_v ? hkv : 0))) * d;
          *reinterpret_cast<u32x4_t*>(to + first) = o;
        } else {
          // the chunks of a run are neighbouring lanes, all of which are here
          float a = largest8(x);
          for (int k = 1; k < lanes; k <<= 1) a = fmaxf(a, __shfl_xor(a, k));
          const float s = a / 448.0f;
          const size_t head_row = (2 * (size_t)p.layer + is_v) * plane + (size_t)row * hkv + (h - hq - (is_v ? hkv : 0));
          uint32_t w[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t v = __builtin_amdgcn_cvt_pk_fp8_f32(code_value(x[4 * g], s), code_value(x[4 * g + 1], s), 0, false);
            w[g] = __builtin_amdgcn_cvt_pk_fp8_f32(code_value(x[4 * g + 2], s), code_value(x[4 * g + 3], s), v, true);
          }
          *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.kv.blocks) + head_row * d + first) = u32x2_t{w[0], w[1]};
          if ((c & (lanes - 1)) == 0) p.kv.scales[head_row * runs + first / p.kv.gran] = s;
        }
      }
    }
  }
}

hipError_t launch_rope_paged(const RopeArgs& args, hipStream_t stream) {
  RopeArgs p = args;
  divide_pages(p.kv);
  // two tokens per workgroup, one where that leaves CUs idle
  const int tokens = p.T >= 4LL * RTOK * p.num_cus ? RTOK : 1;
  const long long grid = (p.T + tokens - 1) / tokens;
  const int pairs = p.interleaved ? PAIRS_SIDE : p.half % 8 == 0 ? PAIRS_APART : PAIRS_ODD;
#define QG_ROPE(FP8)                                                                                               \
  do {                                                                                                             \
    if (pairs == PAIRS_SIDE) rope_paged_kernel<FP8, PAIRS_SIDE><<<(unsigned)grid, RT, 0, stream>>>(p, tokens);       \
    else if (pairs == PAIRS_APART) rope_paged_kernel<FP8, PAIRS_APART><<<(unsigned)grid, RT, 0, stream>>>(p, tokens); \
    else rope_paged_kernel<FP8, PAIRS_ODD><<<(unsigned)grid, RT, 0, stream>>>(p, tokens);                            \
  } while (0)
  if (p.k && p.kv.fp8) QG_ROPE(true);
  else QG_ROPE(false);
#undef QG_ROPE
  return hipGetLastError();
}

}  // namespace qg
