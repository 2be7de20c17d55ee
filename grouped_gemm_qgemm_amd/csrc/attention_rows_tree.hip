// The kernel for few rows: instances for attention_tree_ragged_paged (the same shapes).
#include "attention_rows_kernel.h"

namespace qg {

hipError_t launch_attention_rows_tree(const AttnArgs& p, int mt, unsigned grid, hipStream_t stream) {
  with_rows_kernel<true>(p, mt, [&](auto kernel, int nw, int) { kernel<<<grid, nw * 64, 0, stream>>>(p); });
  return hipGetLastError();
}

}  // namespace qg
