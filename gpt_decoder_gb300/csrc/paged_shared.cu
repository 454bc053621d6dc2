// Attention of a batch whose sequences share prefixes: the entry point.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
#include <algorithm>

#include "paged_attn.cuh"

using namespace gk;

extern "C" gk_status gk_paged_attn_shared(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y,
                                          int64_t ldy, float* lse, const int32_t* q_start, int B, const int32_t* group_start,
                                          const int32_t* prefix_len, int n_groups, int H, int64_t rows, int max_q, int max_group_q,
                                          float scale) {
    if (!ctx) return GK_ERR_ARG;
    GK_REQUIRE(ctx, group_start && prefix_len, GK_ERR_ARG, "gk_paged_attn_shared: null pointer");
    GK_REQUIRE(ctx, n_groups >= 1 && n_groups <= 65535 && max_group_q >= 1, GK_ERR_ARG, "gk_paged_attn_shared: bad groups");
    if (cache && cache->Hkv > 0 && H > 0 && rows > 0)
        GK_REQUIRE(ctx, std::min<int64_t>(max_group_q, rows) * (H / cache->Hkv) < (1ll << 30), GK_ERR_UNSUPPORTED,
                   "gk_paged_attn_shared: groups of %d rows of %d heads a key / value head", max_group_q, H / cache->Hkv);
    return gk_paged_attn(ctx, cache, dtype, q, ldq, y, ldy, lse, q_start, B, H, rows, max_q, scale);
}
