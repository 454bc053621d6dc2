// Attention of many rows over shared prefixes, and over what follows them, on the tensor cores (paged_attn_tiles.cuh).
#include "paged_attn_tiles.cuh"

namespace gk {

gk_status launch_shared_tiles(gk_ctx* ctx, const AttnArgs& a, int part) {
    if (part == PREFIX) return a.fine ? launch_shared_fine(ctx, a) : launch_tiles<PREFIX>(ctx, a);
    return launch_tiles<OWN>(ctx, a);
}

gk_status launch_shared_expand(gk_ctx* ctx, const AttnArgs& a) { return launch_expand<PREFIX>(ctx, a); }

}  // namespace gk
