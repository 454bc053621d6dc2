// Attention of a group's many rows, a few of each sequence, over its prefix (paged_attn_tiles.cuh): a unit of its own, as the
// kernels take long to compile.
#include "paged_attn_tiles.cuh"

namespace gk {

gk_status launch_shared_fine(gk_ctx* ctx, const AttnArgs& a) { return launch_tiles<PREFIX, true>(ctx, a); }

}  // namespace gk
