// The paged key / value cache as kernels see it, and the checks its entry points share.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (one key and value row per position).
#pragma once

#include "launch.cuh"

namespace gk {

// gk_paged_kv with the sizes kernels use; every index it leads to is checked before use.
struct Pages {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    const int32_t* table;
    const int32_t* kv_len;
    int64_t n_pages, ld_table;
    int Hkv, hs, page_log2;
    int capacity;  // positions the table has room for: max_pages * page_size (below 2^30)
};

// Refuse what no kernel could run on; fill `p`.
inline gk_status check_pages(gk_ctx* ctx, const char* what, const gk_paged_kv* c, const int32_t* q_start, int B,
                             int64_t rows, Pages* p) {
    if (!ctx) return GK_ERR_ARG;
    int dev = -1;
    GK_REQUIRE(ctx, cudaGetDevice(&dev) == cudaSuccess && dev == ctx->device, GK_ERR_ARG,
               "%s: the context's device is not current", what);
    GK_REQUIRE(ctx, c && c->k && c->v && c->page_table && c->kv_len && q_start, GK_ERR_ARG, "%s: null pointer", what);
    GK_REQUIRE(ctx, c->dtype == GK_BF16 || c->dtype == GK_I8, GK_ERR_ARG, "%s: cache dtype %d", what, c->dtype);
    GK_REQUIRE(ctx, c->dtype == GK_BF16 || (c->k_scale && c->v_scale), GK_ERR_ARG, "%s: 8-bit pages need scales", what);
    GK_REQUIRE(ctx, c->n_pages >= 1 && c->Hkv >= 1 && c->max_pages >= 1 && c->ld_table >= c->max_pages, GK_ERR_ARG,
               "%s: bad cache sizes", what);
    GK_REQUIRE(ctx, B >= 1 && B <= 65535 && rows >= 0 && rows < (1ll << 31), GK_ERR_ARG, "%s: bad batch", what);
    int lg = 0;
    while ((1 << lg) < c->page_size && lg < 9) ++lg;
    GK_REQUIRE(ctx, c->page_size >= 16 && lg <= 8 && (1 << lg) == c->page_size, GK_ERR_UNSUPPORTED,
               "%s: page size %d (16, 32, 64, 128 or 256)", what, c->page_size);
    GK_REQUIRE(ctx, c->hs >= 16 && c->hs <= 128 && c->hs % 16 == 0, GK_ERR_UNSUPPORTED,
               "%s: head size %d (a multiple of 16 up to 128)", what, c->hs);
    GK_REQUIRE(ctx, c->Hkv <= 65535 && (int64_t)c->max_pages * c->page_size < (1ll << 30) &&
               c->n_pages < (1ll << 31) / c->Hkv / c->page_size,
               GK_ERR_UNSUPPORTED, "%s: cache too large", what);
    GK_REQUIRE(ctx, aligned16(c->k) && aligned16(c->v) && aligned16(c->k_scale) && aligned16(c->v_scale), GK_ERR_ALIGN,
               "%s: cache arrays must be 16-byte aligned", what);
    p->k = c->k;
    p->v = c->v;
    p->k_scale = c->dtype == GK_I8 ? c->k_scale : nullptr;
    p->v_scale = c->dtype == GK_I8 ? c->v_scale : nullptr;
    p->table = c->page_table;
    p->kv_len = c->kv_len;
    p->n_pages = c->n_pages;
    p->ld_table = c->ld_table;
    p->Hkv = c->Hkv;
    p->hs = c->hs;
    p->page_log2 = lg;
    p->capacity = c->max_pages * c->page_size;
    return GK_OK;
}

// The sequence that token row r belongs to, or -1, by the whole warp: each round compares 32 of
// q_start's entries at once, so a batch of up to 31 takes one round trip and one of 1023 two.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ q_start, int B, int r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B + 1;
    while (n > 1) {
        const int step = (n + 31) >> 5, i = lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < n && __ldg(q_start + lo + i) <= r);
        if (!m) return -1;
        const int c = 31 - __clz(m);
        lo += c * step;
        n = min(step, n - c * step);
    }
    return lo < B ? lo : -1;
}

}  // namespace gk
