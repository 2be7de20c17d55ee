// The kernel for few rows: instances for attention_ragged_paged.
#include "attention_rows_kernel.h"

namespace qg {

void attention_rows_shape(AttnArgs& p, int mt) {
  with_rows_kernel<false>(p, mt, [&](auto, int nw, int resident) {
    p.target = p.num_cus * resident;
    p.hw = nw;
    while (p.hkv % p.hw != 0) p.hw /= 2;
  });
}

hipError_t launch_attention_rows(const AttnArgs& p, int mt, unsigned grid, hipStream_t stream) {
  with_rows_kernel<false>(p, mt, [&](auto kernel, int nw, int) { kernel<<<grid, nw * 64, 0, stream>>>(p); });
  return hipGetLastError();
}

}  // namespace qg
