// The kernel for many rows: instances for attention_tree_ragged_paged.
#include "attention_tree_kernel.h"

namespace qg {

namespace {

// f(kernel, waves per workgroup, workgroups per CU) of the instance that serves a call. Tiles of 256 rows
// (TREE_TALL) are for heads of 65 to 128 on pages of a multiple of 16: with heads of 64 they lose (32 trees of
// 64 tokens on 1 to 8191 positions, bf16, 151 us against 145; their e4m3 blocks are too small for eight waves to
// load), and for heads of 256 LDS has no room for the blocks of 64 positions that eight waves need. On other
// pages they would win (pages of 20: those trees with heads of 128 218 us against 250, 6 of 20 to 120 on up
// to 40000, e4m3, 435 against 500), but pages that are no multiple of 16 are not given an instance more.
template <typename F>
void with_tree_kernel(const AttnArgs& p, TreeTiles tiles, F&& f) {
#define QG_ATTN_REST(DP, GRAN, REST)                                                                               \
  do {                                                                                                             \
    if (odd) f(attention_tree_kernel<DP, GRAN, 4, true, REST>, 4, AttnTreeLds<DP, GRAN, 4, true>::ONE ? 1 : 2);      \
    else f(attention_tree_kernel<DP, GRAN, 4, false, REST>, 4, AttnTreeLds<DP, GRAN, 4, false>::ONE ? 1 : 2);        \
  } while (0)
#define QG_ATTN(DP, GRAN)                                               \
  do {                                                                  \
    if constexpr (GRAN == 0) {                                          \
      if (tiles == TREE_FEW) {                                          \
        QG_ATTN_REST(DP, GRAN, true);                                   \
        break;                                                          \
      }                                                                 \
    }                                                                   \
    QG_ATTN_REST(DP, GRAN, false);                                      \
  } while (0)
#define QG_ATTN_TALL(GRAN)                                                                    \
  do {                                                                                        \
    if (tiles == TREE_TALL && !odd) f(attention_tree_kernel<128, GRAN, 8, false, false>, 8, 1); \
    else QG_ATTN(128, GRAN);                                                                  \
  } while (0)
  const bool odd = p.page_size % 16 != 0;
  const int gran = p.fp8 ? p.gran : 0;
  if (p.d <= 64) {
    if (gran == 0) QG_ATTN(64, 0);
    else if (gran == 32) QG_ATTN(64, 32);
    else QG_ATTN(64, 64);
  } else if (p.d <= 128) {
    if (gran == 0) QG_ATTN_TALL(0);
    else if (gran == 32) QG_ATTN_TALL(32);
    else if (gran == 64) QG_ATTN_TALL(64);
    else QG_ATTN_TALL(128);
  } else {
    if (gran == 0) QG_ATTN(256, 0);
    else if (gran == 32) QG_ATTN(256, 32);
    else if (gran == 64) QG_ATTN(256, 64);
    else QG_ATTN(256, 128);
  }
#undef QG_ATTN_REST
#undef QG_ATTN
#undef QG_ATTN_TALL
}

}  // namespace

void attention_tree_shape(AttnArgs& p, TreeTiles tiles) {
  with_tree_kernel(p, tiles, [&](auto, int nw, int resident) {
    p.bm = 32 * nw;
    p.target = p.num_cus * resident;
  });
}

hipError_t launch_attention_tree(const AttnArgs& p, TreeTiles tiles, unsigned grid, hipStream_t stream) {
  with_tree_kernel(p, tiles, [&](auto kernel, int nw, int) { kernel<<<grid, nw * 64, 0, stream>>>(p); });
  return hipGetLastError();
}

}  // namespace qg
