// Attention of chunks of new tokens over the paged cache, on the tensor cores (tcgen05).
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order). The kernel: paged_attn_tiles.cuh.
#include "paged_attn_tiles.cuh"

namespace gk {

gk_status launch_attn_tiles(gk_ctx* ctx, const AttnArgs& a) { return launch_tiles<WHOLE>(ctx, a); }

}  // namespace gk
