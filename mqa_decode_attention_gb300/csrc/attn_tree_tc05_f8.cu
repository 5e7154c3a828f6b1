// attn_tree_tc05_kernel over a fp8 e5m2 cache (a translation unit of its own: they compile side by side).
#include "attn_tree_tc05.cuh"

namespace mqa {

cudaError_t launch_tree_tc05_f8(const TreeParams& p, int tiles, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tq, cudaStream_t stream) {
  return launch_tree_tc05_dt<kDtypeF8>(p, tiles, ctas, tk, tv, tq, stream);
}

}  // namespace mqa
