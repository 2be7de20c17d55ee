// The kernel for many rows: instances for attention_ragged_paged.
#include "attention_tile_kernel.h"

namespace qg {

hipError_t launch_attention_tiles(const AttnArgs& p, unsigned grid, hipStream_t stream) {
#define QG_ATTN(DP, GRAN) attention_tile_kernel<DP, GRAN><<<grid, 256, 0, stream>>>(p)
  const int gran = p.fp8 ? p.gran : 0;
  if (p.d <= 64) {
    if (gran == 0) QG_ATTN(64, 0);
    else if (gran == 32) QG_ATTN(64, 32);
    else QG_ATTN(64, 64);
  } else if (p.d <= 128) {
    if (gran == 0) QG_ATTN(128, 0);
    else if (gran == 32) QG_ATTN(128, 32);
    else if (gran == 64) QG_ATTN(128, 64);
    else QG_ATTN(128, 128);
  } else {
    if (gran == 0) QG_ATTN(256, 0);
    else if (gran == 32) QG_ATTN(256, 32);
    else if (gran == 64) QG_ATTN(256, 64);
    else QG_ATTN(256, 128);
  }
#undef QG_ATTN
  return hipGetLastError();
}

}  // namespace qg
