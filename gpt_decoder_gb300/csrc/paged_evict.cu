// Cutting sequences of the paged cache to a budget: their tokens of most attention weight move to other pages.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the cache that grows by a row a token; here it is held to a size).
//
// Two launches. Select: per sequence and key / value head the n-th largest mass by its bits, eight at a time
// (a histogram of the digit among what still matches), then one walk in order that writes down the positions
// that stay. Move: those rows, with scales and mass, a tile of tokens a block.
#include <math.h>

#include <algorithm>

#include "paged.cuh"

namespace gk {
namespace {

struct EvictArgs {
    Pages from, to;
    const float* mass;
    float* to_mass;
    const int32_t* first;  // may be null
    int budget, recent;
    int32_t* new_len;
    int32_t* kept;
    int* err;
};

// What a sequence has: tokens in all, the first ones that stay, and those behind them.
struct Cut {
    int kv, first, behind;
};
__device__ __forceinline__ Cut cut_of(const EvictArgs& a, int b) {
    Cut c;
    c.kv = min(max(a.from.kv_len[b], 0), a.from.capacity);
    c.first = a.first ? min(max(a.first[b], 0), c.kv) : 0;
    c.behind = c.kv - c.first;
    return c;
}

// Unsigned integers in the order of the numbers; a NaN is the least of them, and both zeros are one.
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The row (token of this head) at a position, or -1.
__device__ __forceinline__ int64_t row_at(const Pages& p, int b, int hk, int pos) {
    if (pos >= p.capacity) return -1;
    const int id = __ldg(p.table + b * p.ld_table + (pos >> p.page_log2));
    if (id < 0 || id >= p.n_pages) return -1;
    return (((int64_t)id * p.Hkv + hk) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
}

constexpr int SELECT = 1024;

__global__ void __launch_bounds__(SELECT) evict_select_kernel(const EvictArgs a) {
    __shared__ int s_hist[256];
    __shared__ uint2 s_warp[SELECT / 32];
    __shared__ int s_digit, s_left;
    wait_for_earlier_kernels();
    const int b = blockIdx.y, hk = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Cut c = cut_of(a, b);
    int32_t* kept = a.kept + ((int64_t)b * a.from.Hkv + hk) * a.budget;
    if (hk == 0 && tid == 0) {
        a.new_len[b] = c.first + min(c.behind, a.budget);
        if (a.from.kv_len[b] > a.from.capacity) report(a.err, GK_ERR_INDEX);
    }
    if (c.behind <= a.budget) {
        for (int i = tid; i < a.budget; i += SELECT) kept[i] = i < c.behind ? c.first + i : -1;
        return;
    }
    const int need = a.budget - a.recent, n = c.behind - a.recent;  // the heaviest `need` of n: 0 <= need < n
    auto key = [&](int i) {
        const int64_t r = row_at(a.from, b, hk, c.first + i);
        if (r < 0) report(a.err, GK_ERR_INDEX);
        return ordered(r < 0 ? -INFINITY : a.mass[r]);
    };
    uint32_t top = 0;  // the digits found so far
    int left = need;   // how many of the keys that match them stay
    for (int shift = 24; shift >= 0 && need; shift -= 8) {
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += SELECT) {
            const uint32_t k = key(i);
            if (shift == 24 || k >> (shift + 8) == top >> (shift + 8)) atomicAdd(&s_hist[k >> shift & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int d = 255, sum = 0;
            while (d > 0 && sum + s_hist[d] < left) sum += s_hist[d--];
            s_digit = d;
            s_left = left - sum;
        }
        __syncthreads();
        top |= (uint32_t)s_digit << shift;
        left = s_left;
        __syncthreads();
    }
    // in order: keys above `top`, and the first `left` of those equal to it
    uint2 base = make_uint2(0, 0);  // (above, equal) before this round
    for (int i0 = 0; i0 < n && need; i0 += SELECT) {
        const int i = i0 + tid;
        const uint32_t k = i < n ? key(i) : 0;
        const bool more = i < n && k > top, same = i < n && k == top;
        const unsigned m = __ballot_sync(0xffffffffu, more), e = __ballot_sync(0xffffffffu, same);
        if (lane == 0) s_warp[warp] = make_uint2(__popc(m), __popc(e));
        __syncthreads();
        uint2 at = base;
        for (int w = 0; w < SELECT / 32; ++w) {
            const uint2 x = s_warp[w];
            if (w < warp) at.x += x.x, at.y += x.y;
            base.x += x.x, base.y += x.y;
        }
        const unsigned below = (1u << lane) - 1;
        at.x += __popc(m & below), at.y += __popc(e & below);
        if (more || (same && (int)at.y < left)) kept[at.x + min((int)at.y, left)] = c.first + i;
        __syncthreads();
    }
    for (int i = tid; i < a.recent; i += SELECT) kept[need + i] = c.kv - a.recent + i;
}

// A block moves TOKENS of the kept tokens, and its share of the first ones: 16-byte pieces of keys and values.
constexpr int MOVE = 256, TOKENS = 64;
__global__ void __launch_bounds__(MOVE) evict_move_kernel(const EvictArgs a) {
    __shared__ int64_t s_from[TOKENS], s_to[TOKENS];
    wait_for_earlier_kernels();
    const int b = blockIdx.z, hk = blockIdx.y, tid = threadIdx.x;
    const Cut c = cut_of(a, b);
    const int32_t* kept = a.kept + ((int64_t)b * a.from.Hkv + hk) * a.budget;
    const int row_bytes = a.from.hs * (a.from.k_scale ? 1 : 2), per = row_bytes >> 4;
    const bool one_pool = a.from.k == a.to.k;
    auto tile = [&](int at, int n, bool listed) {  // new positions at .. at + n - 1
        __syncthreads();
        if (tid < n) {
            const int pos = at + tid, old = listed ? kept[pos - c.first] : pos;
            const int64_t from = row_at(a.from, b, hk, old), to = row_at(a.to, b, hk, pos);
            if (from < 0 || to < 0) report(a.err, GK_ERR_INDEX);
            s_to[tid] = to < 0 || (one_pool && to == from) ? -1 : to;
            s_from[tid] = from;
        }
        __syncthreads();
        for (int x = tid; x < n * per; x += MOVE) {
            const int i = x / per, d = (x - i * per) << 4;
            const int64_t from = s_from[i], to = s_to[i];
            if (to < 0) continue;
            uint4 k = make_uint4(0, 0, 0, 0), v = k;
            if (from >= 0) {
                k = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.from.k) + from * row_bytes + d);
                v = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.from.v) + from * row_bytes + d);
            }
            *reinterpret_cast<uint4*>(static_cast<char*>(a.to.k) + to * row_bytes + d) = k;
            *reinterpret_cast<uint4*>(static_cast<char*>(a.to.v) + to * row_bytes + d) = v;
        }
        if (tid < n && s_to[tid] >= 0) {
            const int64_t from = s_from[tid], to = s_to[tid];
            a.to_mass[to] = from < 0 ? 0.f : a.mass[from];
            if (a.from.k_scale) {
                a.to.k_scale[to] = from < 0 ? 0.f : a.from.k_scale[from];
                a.to.v_scale[to] = from < 0 ? 0.f : a.from.v_scale[from];
            }
        }
    };
    const int stay = min(c.behind, a.budget);
    for (int at = blockIdx.x * TOKENS; at < stay; at += gridDim.x * TOKENS) tile(c.first + at, min(TOKENS, stay - at), true);
    for (int at = blockIdx.x * TOKENS; at < c.first; at += gridDim.x * TOKENS) tile(at, min(TOKENS, c.first - at), false);
}

}  // namespace
}  // namespace gk

using namespace gk;

extern "C" gk_status gk_paged_evict(gk_ctx* ctx, const gk_paged_kv* cache, const float* mass, const gk_paged_kv* to, float* to_mass,
                                    const int32_t* first, int budget, int recent, int32_t* new_len, int32_t* kept, int B) {
    if (!ctx) return GK_ERR_ARG;
    EvictArgs a{};
    GK_REQUIRE(ctx, cache && to && mass && to_mass && new_len && kept, GK_ERR_ARG, "gk_paged_evict: null pointer");
    GK_TRY(check_pages(ctx, "gk_paged_evict", cache, new_len, B, 0, &a.from));
    gk_paged_kv t = *to;
    t.kv_len = new_len;
    GK_TRY(check_pages(ctx, "gk_paged_evict", &t, new_len, B, 0, &a.to));
    GK_REQUIRE(ctx, to->dtype == cache->dtype && to->Hkv == cache->Hkv && to->page_size == cache->page_size && to->hs == cache->hs,
               GK_ERR_ARG, "gk_paged_evict: the two caches differ");
    GK_REQUIRE(ctx, budget >= 1 && budget <= 1 << 30 && recent >= 0 && recent <= budget, GK_ERR_ARG, "gk_paged_evict: budget %d, recent %d",
               budget, recent);
    GK_REQUIRE(ctx, aligned16(mass) && aligned16(to_mass), GK_ERR_ALIGN, "gk_paged_evict: mass must be 16-byte aligned");
    const uintptr_t x = (uintptr_t)new_len, y = (uintptr_t)cache->kv_len, len = (uintptr_t)B * sizeof(int32_t);
    GK_REQUIRE(ctx, x + len <= y || y + len <= x, GK_ERR_ARG, "gk_paged_evict: new_len overlaps the old lengths");
    a.mass = mass;
    a.to_mass = to_mass;
    a.first = first;
    a.budget = budget;
    a.recent = recent;
    a.new_len = new_len;
    a.kept = kept;
    a.err = ctx->d_err;
    GK_TRY(launch_dependent(ctx, "paged_evict_select", evict_select_kernel, dim3((unsigned)a.from.Hkv, (unsigned)B), dim3(SELECT), 0, 1, a));
    const int64_t tiles = cdiv(std::min(budget, a.from.capacity), TOKENS);
    return launch_dependent(ctx, "paged_evict_move", evict_move_kernel, dim3((unsigned)tiles, (unsigned)a.from.Hkv, (unsigned)B), dim3(MOVE), 0, 1, a);
}
