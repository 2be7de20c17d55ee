// The kernel for many rows: instances for attention_tree_ragged_paged.
#include "attention_tile_kernel.h"

namespace qg {

hipError_t launch_attention_tiles_tree(const AttnArgs& p, unsigned grid, hipStream_t stream) {
  return launch_tiles<true>(p, grid, stream);
}

}  // namespace qg
