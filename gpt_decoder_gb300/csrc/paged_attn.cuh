// Internal interface of the attention over the paged cache: the arguments its kernels share, and
// the partial results of sequences split over the GPU.
#pragma once

#include "paged.cuh"

namespace gk {

struct AttnArgs {
    Pages p;
    const __nv_bfloat16* q;
    __nv_bfloat16* y;
    float* lse;  // may be null
    const int32_t* q_start;
    int64_t ldq, ldy;
    int B, H, G, rows, max_q;  // G = H / Hkv heads share a key / value head
    float scale_log2;          // scale * log2(e): scores are kept in powers of two
    // a sequence of kv keys is cut into pieces of split_keys(kv) keys, at most `splits` of them;
    // with splits > 1 piece s of row r, head h leaves its weighted sum of values (not divided) in
    // part_o[(r * H + h) * splits + s][hs] and its reference and sum of weights in part_ml
    int splits, min_split;
    int clustered;  // the pieces are the blocks of one cluster, which joins them itself
    float* part_o;
    float2* part_ml;
    // 8-bit codes laid out as bf16 for the tile kernel, or null: of key / value heads head0 ..
    // head0 + heads - 1, which one launch takes (0 .. Hkv - 1 without)
    int head0, heads;
    __nv_bfloat16* expanded_k;
    __nv_bfloat16* expanded_v;
    int64_t expanded_rows;
    int* err;
    CodeMasks masks;
    __host__ __device__ int split_keys(int kv) const {
        const int even = (kv + splits - 1) / splits;
        return max(min_split, (even + 127) & ~127);
    }
};

// Join the pieces of every (row, head).
gk_status launch_attn_join(gk_ctx* ctx, const AttnArgs& a);
// Sequences with at most 64 query rows per key / value head (32 where pages are bf16).
gk_status launch_attn_few(gk_ctx* ctx, const AttnArgs& a);
// Any number of rows, for heads head0 .. head0 + heads - 1, in tiles of 128 on the tensor cores (tcgen05).
gk_status launch_attn_tiles(gk_ctx* ctx, const AttnArgs& a);

}  // namespace gk
