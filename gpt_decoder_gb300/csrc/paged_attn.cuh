// Internal interface of the attention over the paged cache: the arguments its kernels share, the partial
// results of sequences split over the GPU, and what a block works on where sequences share prefixes.
#pragma once

#include "paged.cuh"

namespace gk {

// What the "sequences" of a launch are: whole sequences; the shared prefixes, each with the rows of its group's
// sequences; or what follows the prefix in each sequence.
enum { WHOLE, PREFIX, OWN };

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
    // shared prefixes: groups of sequences (of `sequences` in all); B and max_q are those of the launch. A row's parts
    // are `slots`, this launch's from slot0 on; the prefixes' are split by prefix_splits and prefix_min.
    const int32_t* group_start;
    const int32_t* prefix_len;
    int n_groups, sequences, max_group, slots, slot0, prefix_splits, prefix_min;
    bool fine;        // PREFIX in tiles: weights as two bf16 parts
    int2* row_parts;  // [rows]: pieces of the prefix and of a row's own keys; (0, 0): the row is left as it was
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
    __host__ __device__ static int split_keys(int kv, int splits, int min_split) {
        const int even = (kv + splits - 1) / splits;
        return max(min_split, (even + 127) & ~127);
    }
    __host__ __device__ int split_keys(int kv) const { return split_keys(kv, splits, min_split); }
};

// The first row and the number of rows of a group's sequences; false: it cannot be.
__device__ __forceinline__ bool group_rows(const AttnArgs& a, int g, int& s0, int& n) {
    const int first = __ldg(a.group_start + g), end = __ldg(a.group_start + g + 1);
    n = 0;
    if (first >= end) return true;
    if (first < 0 || end > a.sequences) return false;
    s0 = __ldg(a.q_start + first);
    const int s1 = __ldg(a.q_start + end);
    n = s1 - s0;
    return s0 >= 0 && s1 <= a.rows && n <= a.max_group;
}
// The part of a group's prefix that there is room for.
__device__ __forceinline__ int prefix_of(const AttnArgs& a, int g) { return min(max(__ldg(a.prefix_len + g), 0), a.p.capacity); }
// The prefix that sequence b shares, by the whole warp: 0 unless all of its rows lie behind it.
__device__ __forceinline__ int shared_by(const AttnArgs& a, int b, int n, int kv_all) {
    const int g = find_sequence(a.group_start, a.n_groups, b);
    const int prefix = g < 0 ? 0 : prefix_of(a, g);
    return kv_all - n >= prefix ? prefix : 0;
}

// The rows and keys of a launch's sequence b: rows s0 .. s0 + n - 1, row i seeing the positions from `from` to
// min(kv - 1, kv_all - n + i) in row `table` of the page table.
struct Rows {
    int s0, n, kv_all, kv, from, table;
};
template <int PART>
__device__ __forceinline__ bool rows_of(const AttnArgs& a, int b, Rows& r) {
    r.table = b;
    r.from = 0;
    bool fits;
    if constexpr (PART == PREFIX) {
        fits = group_rows(a, b, r.s0, r.n);
        if (fits && r.n <= 0) return false;
    } else {
        r.s0 = a.q_start[b];
        const int s1 = a.q_start[b + 1];
        r.n = s1 - r.s0;
        if (r.n <= 0) return false;
        fits = r.n <= a.max_q && r.s0 >= 0 && s1 <= a.rows;
    }
    if (!fits) {
        if (threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
        return false;
    }
    if constexpr (PART == PREFIX) {
        r.table = __ldg(a.group_start + b);
        r.kv = prefix_of(a, b);
        r.kv_all = r.kv + r.n;  // every row lies behind it (rows of sequences that do not are not joined with it)
        if (__ldg(a.prefix_len + b) > a.p.capacity && threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
        return r.kv > 0;
    } else {
        r.kv_all = max(a.p.kv_len[b], 0);
        r.kv = min(r.kv_all, a.p.capacity);
        if (r.kv_all > a.p.capacity && threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
        if constexpr (PART == OWN) r.from = shared_by(a, b, r.n, r.kv_all);
        return true;
    }
}
// Pieces are cut from a whole tile of 128 on.
__device__ __forceinline__ int first_tile(int from) { return from & ~127; }

// Leave for the join what the rows of a sequence consist of (in the launch of own keys, by a block a sequence that has
// no other work: the loads that it takes follow on each other).
__device__ __forceinline__ void leave_row_parts(const AttnArgs& a, int b) {
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1], n = s1 - s0;
    int2 parts = make_int2(0, 0);
    if (n > 0 && n <= a.max_q && s0 >= 0 && s1 <= a.rows) {
        const int kv_all = max(a.p.kv_len[b], 0), kv = min(kv_all, a.p.capacity), g = find_sequence(a.group_start, a.n_groups, b);
        int prefix = 0, gs, gn;
        const bool there = g < 0 || group_rows(a, g, gs, gn);
        if (g >= 0) prefix = prefix_of(a, g);
        if (kv_all - n < prefix) prefix = 0;
        if (there) {
            const int keys = kv - first_tile(prefix), piece = a.split_keys(keys);
            const int first = AttnArgs::split_keys(prefix, a.prefix_splits, a.prefix_min);
            parts = make_int2((prefix + first - 1) / first, max(1, (keys + piece - 1) / piece));
        }
    }
    for (int r = max(s0, 0) + threadIdx.x; r < min(s1, a.rows); r += blockDim.x) a.row_parts[r] = parts;
}

// Refuse what no kernel could run on; fill `a` with the arguments.
gk_status check_attn(gk_ctx* ctx, const char* what, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y, int64_t ldy,
                     float* lse, const int32_t* q_start, int B, int H, int64_t rows, int max_q, float scale, AttnArgs* a);
// Join the pieces of every (row, head).
gk_status launch_attn_join(gk_ctx* ctx, const AttnArgs& a);
// Sequences with at most 64 query rows per key / value head (32 where pages are bf16).
gk_status launch_attn_few(gk_ctx* ctx, const AttnArgs& a);
// Any number of rows, for heads head0 .. head0 + heads - 1, in tiles of 128 on the tensor cores (tcgen05).
gk_status launch_attn_tiles(gk_ctx* ctx, const AttnArgs& a);
// The same for the prefixes of groups (PREFIX) or what follows them (OWN), which leave parts; prefixes in tiles with
// weights of 16 bits where a.fine.
gk_status launch_shared_few(gk_ctx* ctx, const AttnArgs& a, int part);
gk_status launch_shared_tiles(gk_ctx* ctx, const AttnArgs& a, int part);
gk_status launch_shared_fine(gk_ctx* ctx, const AttnArgs& a);
// 8-bit codes of the prefixes as bf16, before the tiles that take them.
gk_status launch_shared_expand(gk_ctx* ctx, const AttnArgs& a);

}  // namespace gk
