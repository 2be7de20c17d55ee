// Rows of a paged cache moved as they are: ranges read back as dense rows, and the
// accepted tokens of a draft tree moved together.
//
// Both are copies, bound by HBM, or by latency where they are small. Reading 379000 positions
// of 8 heads of 128 out of an e4m3 cache as bf16 (2.4 GB read and written) takes 456 us, 5.2
// TB/s, which is a large copy's rate; 1900 rows of a bf16 cache (16 MB) 6 us on the GPU.
// Three of eight tokens in 32 layers (0.5 MB) move in 3.5 us, paths of 64 sequences in an e4m3
// cache (39 MB) in 7.6 us: the lengths, the path, the page numbers and the rows in turn.
#include <algorithm>

#include "paged_common.h"

namespace qg {

namespace {

constexpr int CT = 256;          // threads
constexpr int CROWS = 64;        // rows per workgroup of a read, at most (a lane each to find them)
constexpr int CMOVES = 64;       // moves whose rows are found at a time
constexpr int CBATCH = 8;        // rows in flight per thread

// eight codes times their scale
__device__ __forceinline__ void decode8(u32x2_t w, float s, float (&x)[8]) {
  const uint32_t a = w.x, b = w.y;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t v = g ? b : a;
    const float2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
    x[4 * g] = lo.x * s;
    x[4 * g + 1] = lo.y * s;
    x[4 * g + 2] = hi.x * s;
    x[4 * g + 3] = hi.y * s;
  }
}

}  // namespace

// A workgroup takes some rows of one plane: one wave finds where they lie, then all copy
// chunks of 8 elements.
template <bool FP8, bool F32>
__global__ __launch_bounds__(CT) void kv_read_kernel(KvReadArgs p, int planes, int rows_per_wg) {
  __shared__ long long s_row[CROWS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int plane = planes == 2 ? blockIdx.x & 1 : p.out[0] ? 0 : 1;
  const long long r0 = (long long)(planes == 2 ? blockIdx.x >> 1 : blockIdx.x) * rows_per_wg;
  if (tid < 64) {
    const uint32_t rows = min(p.offs[p.kv.batch], (uint32_t)p.T);   // (offsets are not checked: no row behind the outputs)
    int b = owner_of(p.offs, p.kv.batch, (uint32_t)r0);
    const long long r = r0 + lane;
    if (lane < rows_per_wg) {
      long long row = -1;
      if (b >= 0 && r < rows) {
        if (p.offs[b + 1] <= (uint32_t)r) {   // behind the first row's sequence
          int hi = p.kv.batch;
          while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (p.offs[mid] <= (uint32_t)r) b = mid; else hi = mid;
          }
        }
        row = cache_row(p.kv, b, (p.first ? p.first[b] : 0) + ((uint32_t)r - p.offs[b]));
      }
      s_row[lane] = row;
    }
  }
  __syncthreads();
  const int width = p.kv.hkv * p.kv.d, ch = width >> 3;   // elements and chunks of a row
  const size_t base = (2 * (size_t)p.layer + plane) * p.kv.pages * p.kv.page_size;
  for (int e = tid; e < rows_per_wg * ch; e += CT) {
    const int i = e / ch, c = e - i * ch;
    const long long row = s_row[i];
    if (row < 0) continue;
    const size_t from = (base + row) * width + 8 * c, to = (size_t)(r0 + i) * width + 8 * c;
    if constexpr (!FP8 && !F32) {
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.out[plane]) + to) =
          *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p.kv.blocks) + from);
    } else {
      float x[8];
      if constexpr (FP8) {
        const float s = p.kv.scales[from / p.kv.gran];
        decode8(*reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(p.kv.blocks) + from), s, x);
      } else {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p.kv.blocks) + from);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t w = v[g];
          x[2 * g] = bf2f((uint16_t)w);
          x[2 * g + 1] = bf2f((uint16_t)(w >> 16));
        }
      }
      if constexpr (F32) {
        float* o = static_cast<float*>(p.out[plane]) + to;
        *reinterpret_cast<float4_t*>(o) = float4_t{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<float4_t*>(o + 4) = float4_t{x[4], x[5], x[6], x[7]};
      } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.out[plane]) + to) =
            u32x4_t{f2bf2_rn(x[0], x[1]), f2bf2_rn(x[2], x[3]), f2bf2_rn(x[4], x[5]), f2bf2_rn(x[6], x[7])};
      }
    }
  }
}

// A workgroup takes one sequence and some of its columns: a thread owns 16 bytes (of codes
// or values; 4 bytes of scales) of one layer and plane and moves them for the whole path
// in order, CBATCH rows read before the first of them is written. That is safe as a path is
// strictly increasing: what a later batch reads lies behind all that an earlier one writes.
__global__ __launch_bounds__(CT) void kv_keep_kernel(KvKeepArgs p, int wgs, uint32_t row16, uint32_t row4) {
  __shared__ long long s_from[CMOVES], s_to[CMOVES];
  __shared__ int s_moves;
  const int tid = threadIdx.x, lane = tid & 63;
  const int b = blockIdx.x / wgs, part = blockIdx.x - b * wgs;
  const int kept = (int)min((long long)p.kept[b], (long long)p.width);
  const uint32_t cached = p.kv.cache_len[b];
  const int32_t* path = p.path + (size_t)b * p.width;
  const size_t plane = (size_t)p.kv.pages * p.kv.page_size;
  const long long planes = 2 * p.kv.layers, columns = planes * ((long long)row16 + row4);
  for (int i0 = 0; i0 < kept; i0 += CMOVES) {
    if (i0 > 0) __syncthreads();
    if (tid < CMOVES) {
      const int i = i0 + lane, at = i < kept ? path[i] : -1;
      const bool moves = at > i;
      const unsigned long long who = __ballot(moves);
      if (moves) {
        const int n = __popcll(who & ((1ull << lane) - 1));
        s_from[n] = cache_row(p.kv, b, cached + at);
        s_to[n] = cache_row(p.kv, b, cached + i);
      }
      if (lane == 0) s_moves = __popcll(who);
    }
    __syncthreads();
    const int moves = s_moves;
    for (long long e = (long long)part * CT + tid; e < columns; e += (long long)wgs * CT) {
      if (e < planes * row16) {
        const long long l = e / row16;
        u32x4_t* base = static_cast<u32x4_t*>(p.kv.blocks) + (size_t)l * plane * row16 + (e - l * row16);
        for (int m = 0; m < moves; m += CBATCH) {
          u32x4_t x[CBATCH];
#pragma unroll
          for (int k = 0; k < CBATCH; ++k)
            if (m + k < moves) x[k] = base[(size_t)s_from[m + k] * row16];
#pragma unroll
          for (int k = 0; k < CBATCH; ++k)
            if (m + k < moves) base[(size_t)s_to[m + k] * row16] = x[k];
        }
      } else {
        const long long f = e - planes * row16, l = f / row4;
        float* base = p.kv.scales + (size_t)l * plane * row4 + (f - l * row4);
        for (int m = 0; m < moves; m += CBATCH) {
          float x[CBATCH];
#pragma unroll
          for (int k = 0; k < CBATCH; ++k)
            if (m + k < moves) x[k] = base[(size_t)s_from[m + k] * row4];
#pragma unroll
          for (int k = 0; k < CBATCH; ++k)
            if (m + k < moves) base[(size_t)s_to[m + k] * row4] = x[k];
        }
      }
    }
  }
}

hipError_t launch_kv_read(const KvReadArgs& args, hipStream_t stream) {
  KvReadArgs p = args;
  divide_pages(p.kv);
  const int planes = (p.out[0] ? 1 : 0) + (p.out[1] ? 1 : 0);
  const int ch = p.kv.hkv * p.kv.d >> 3;
  // Eight chunks of codes per thread, or four of values, and two workgroups per CU. With 16 rows always,
  // 465000 rows of one head of 128 took 113 us out of e4m3 (now 79) and 106 out of bf16 (95), 483 of
  // 16 heads of 256 17 (8).
  const long long most = std::min<long long>(CROWS, p.T * planes / (2 * p.num_cus));
  const long long want = std::max<long long>(1, std::min<long long>(most, (p.kv.fp8 ? 8 : 4) * CT / ch));
  const int rows = (int)std::max<long long>(want, p.T * planes >> 23);   // (a launch has less than 2^32 threads)
  const unsigned grid = (unsigned)((p.T + rows - 1) / rows * planes);
  if (p.kv.fp8) {
    if (p.f32) kv_read_kernel<true, true><<<grid, CT, 0, stream>>>(p, planes, rows);
    else kv_read_kernel<true, false><<<grid, CT, 0, stream>>>(p, planes, rows);
  } else {
    if (p.f32) kv_read_kernel<false, true><<<grid, CT, 0, stream>>>(p, planes, rows);
    else kv_read_kernel<false, false><<<grid, CT, 0, stream>>>(p, planes, rows);
  }
  return hipGetLastError();
}

hipError_t launch_kv_keep(const KvKeepArgs& args, hipStream_t stream) {
  KvKeepArgs p = args;
  divide_pages(p.kv);
  const int width = p.kv.hkv * p.kv.d;
  const uint32_t row16 = (uint32_t)(width * (p.kv.fp8 ? 1 : 2) / 16), row4 = p.kv.fp8 ? width / p.kv.gran : 0;
  const long long columns = 2 * p.kv.layers * ((long long)row16 + row4);
  // a column per thread, but no more than some eight rounds of workgroups
  const long long want = (columns + CT - 1) / CT, most = (64LL * p.num_cus + p.kv.batch - 1) / p.kv.batch;
  const int wgs = (int)(want < most ? want : most);
  kv_keep_kernel<<<(unsigned)(wgs * p.kv.batch), CT, 0, stream>>>(p, wgs, row16, row4);
  return hipGetLastError();
}

}  // namespace qg
