// Cutting sequences of the paged cache to a budget: their tokens of most attention weight move to other pages.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the cache that grows by a row a token; here it is held to a size).
//
// Two launches. Select: a cluster of blocks per sequence and key / value head holds the head's masses in shared memory, as
// integers that order like them (a table wider than its blocks can hold, 49152 positions each and up to eight blocks where
// sequences are few, has them read again each time), and finds the n-th largest by its bits: three digits of 11, 11 and
// 10 bits, for each a histogram of what still matches, summed over the cluster through distributed shared memory. Then each
// warp counts what stays of its stretch of positions and walks it, so the positions come out in order without a sort: keys
// above the n-th, and the first of those equal to it. Move: those rows, with scales and mass, a tile of tokens a block.
// The bytes of what moves bound it where there are many: 48 sequences of up to 8191 tokens to 2064, 8 heads of 128, bf16:
// 128 us, 5.9 TB/s (0.89 of a copy), the selection 15 of them; 3 of up to 65536 to 8256 52 us, 19 the selection (a chain:
// page ids, masses, three digits at about 2.5 us, the walk). One of 1100 to 516, 12 heads of 64: 9.1 us, two launches. Clusters
// and shared memory go by the table's width: with tables of 65536 positions the 48 take 136 us, the one 17.
#include <math.h>

#include <algorithm>
#include <initializer_list>

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

constexpr int SELECT = 512, SELECT_WARPS = SELECT / 32, BINS = 2048, MAX_CLUSTER = 8;
constexpr int HELD = 48 * 1024;  // masses that a block can hold

// `each`: positions of a block, a multiple of 128. HOLD: they are kept in shared memory (else read again each time).
template <bool HOLD>
__global__ void __launch_bounds__(SELECT) evict_select_kernel(const EvictArgs a, int each_most) {
    extern __shared__ __align__(16) uint32_t s_keys[];
    __shared__ __align__(16) uint32_t s_hist[3][BINS], s_total[BINS / 2];
    __shared__ uint32_t s_share[3];
    __shared__ uint2 s_warp[SELECT_WARPS], s_mine;
    __shared__ uint32_t s_sum[SELECT_WARPS];
    __shared__ int s_digit, s_left;
    wait_for_earlier_kernels();
    const int blocks = gridDim.x, rank = blockIdx.x, b = blockIdx.z, hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Cut c = cut_of(a, b);
    int32_t* kept = a.kept + ((int64_t)b * a.from.Hkv + hk) * a.budget;
    if (hk == 0 && rank == 0 && tid == 0) {
        a.new_len[b] = c.first + min(c.behind, a.budget);
        if (a.from.kv_len[b] > a.from.capacity) report(a.err, GK_ERR_INDEX);
    }
    if (c.behind <= a.budget) {  // (all blocks of the cluster)
        for (int i = rank * SELECT + tid; i < a.budget; i += blocks * SELECT) kept[i] = i < c.behind ? c.first + i : -1;
        return;
    }
    const int need = a.budget - a.recent, end = c.kv - a.recent;  // the heaviest `need` of positions first .. end - 1
    for (int i = rank * SELECT + tid; i < a.recent; i += blocks * SELECT) kept[need + i] = end + i;
    if (need == 0) return;
    auto barrier = [&]() {
        __syncwarp();
        if (blocks > 1) cluster_barrier();
        else __syncthreads();
    };

    // this block's positions p0 .. p0 + each - 1, four at a time (they share a page); 0: not one to choose from
    const int base = c.first & ~127, each = min(each_most, ((end - base + blocks - 1) / blocks + 127) & ~127), p0 = base + rank * each;
    bool missing = false;
    auto row4 = [&](int i) -> int64_t {
        if (i >= each || p0 + i >= end) return -1;
        const int64_t r = row_at(a.from, b, hk, p0 + i);
        missing |= r < 0;
        return r;
    };
    auto mass4 = [&](int64_t r) {
        return r >= 0 ? *reinterpret_cast<const float4*>(a.mass + r) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    };
    auto keys4 = [&](int i, const float4& m) {
        const int pos = p0 + i;
        return make_uint4(pos >= c.first && pos < end ? ordered(m.x) : 0, pos + 1 >= c.first && pos + 1 < end ? ordered(m.y) : 0,
                          pos + 2 >= c.first && pos + 2 < end ? ordered(m.z) : 0, pos + 3 >= c.first && pos + 3 < end ? ordered(m.w) : 0);
    };
    auto load4 = [&](int i) { return keys4(i, mass4(row4(i))); };
    for (int i = tid; i < 3 * BINS; i += SELECT) (&s_hist[0][0])[i] = 0;
    if (tid < 3) s_share[tid] = 0;
    if (HOLD) {
        constexpr int AHEAD = 4;  // page ids, then masses, of this many places on their way together
        for (int i0 = tid * 4; i0 < each; i0 += AHEAD * SELECT * 4) {
            int64_t r[AHEAD];
            float4 m[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) r[u] = row4(i0 + u * SELECT * 4);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) m[u] = mass4(r[u]);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = i0 + u * SELECT * 4;
                if (i < each) *reinterpret_cast<uint4*>(s_keys + i) = keys4(i, m[u]);
            }
        }
    }
    __syncthreads();
    uint32_t top = 0;  // the digits found so far
    int left = need;   // how many of the keys that match them stay
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid * 4; i < each; i += SELECT * 4) {
            const uint4 k4 = HOLD ? *reinterpret_cast<const uint4*>(s_keys + i) : load4(i);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k[e] && (pass == 0 || k[e] >> (shift + bits) == top >> (shift + bits))) atomicAdd(&s_hist[pass][k[e] >> shift & ((1 << bits) - 1)], 1u);
        }
        barrier();
        // four bins a thread, from the highest down: which of them holds the left-th key
        static_assert(SELECT * 4 == BINS, "four bins a thread");
        int first_bin = BINS - 4 - 4 * tid;
        uint4 h = make_uint4(0, 0, 0, 0);
        uint32_t higher = 0;  // keys in the bins of higher shares
        if (blocks == 1) {
            h = *reinterpret_cast<const uint4*>(&s_hist[pass][first_bin]);
        } else {
            // each block sums a share of the bins over the cluster; then all look at the share that holds the key (all bins
            // of all blocks read by each took 3 to 5 us a digit, 8 blocks)
            const int share = BINS / blocks;
            if (tid * 4 < share) {
                for (int r = 0; r < blocks; ++r) {
                    const uint4 x = load_cluster_u32x4(&s_hist[pass][rank * share + tid * 4], r);
                    h.x += x.x, h.y += x.y, h.z += x.z, h.w += x.w;
                }
                *reinterpret_cast<uint4*>(s_total + tid * 4) = h;
                uint32_t sum = h.x + h.y + h.z + h.w;
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) atomicAdd(&s_share[pass], sum);
            }
            barrier();
            uint32_t n[MAX_CLUSTER];
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) n[r] = r < blocks ? load_cluster_u32(&s_share[pass], r) : 0;
            int owner = MAX_CLUSTER - 1;
#pragma unroll
            for (int r = MAX_CLUSTER - 1; r > 0; --r)
                if (owner == r && higher + n[r] < (uint32_t)left) higher += n[r], owner = r - 1;
            first_bin = owner * share + share - 4 - 4 * tid;
            h = tid * 4 < share ? load_cluster_u32x4(s_total + share - 4 - 4 * tid, owner) : make_uint4(0, 0, 0, 0);
        }
        const uint32_t mine = h.x + h.y + h.z + h.w;
        uint32_t run = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += y;
        }
        if (lane == 31) s_sum[warp] = run;
        __syncthreads();
        uint32_t before = higher + run - mine;  // keys in higher bins
        for (int w = 0; w < warp; ++w) before += s_sum[w];
        if (before < (uint32_t)left && before + mine >= (uint32_t)left) {
            const uint32_t n[4] = {h.w, h.z, h.y, h.x};
            int d = 0;
            while (d < 3 && before + n[d] < (uint32_t)left) before += n[d++];
            s_digit = first_bin + 3 - d;
            s_left = left - (int)before;
        }
        __syncthreads();
        top |= (uint32_t)s_digit << shift;
        left = s_left;
    }
    if (missing) report(a.err, GK_ERR_INDEX);
    // each warp's stretch of the block: what stays of it, and where it goes
    const int stretch = ((each + SELECT_WARPS - 1) / SELECT_WARPS + 127) & ~127, w0 = min(warp * stretch, each), w1 = min(w0 + stretch, each);
    uint2 n = make_uint2(0, 0);  // keys above `top`, and equal to it
    for (int i = w0 + lane * 4; i < w1; i += 128) {
        const uint4 k = HOLD ? *reinterpret_cast<const uint4*>(s_keys + i) : load4(i);
        n.x += (k.x > top) + (k.y > top) + (k.z > top) + (k.w > top);
        n.y += (k.x == top) + (k.y == top) + (k.z == top) + (k.w == top);
    }
    for (int o = 16; o > 0; o >>= 1) n.x += __shfl_xor_sync(0xffffffffu, n.x, o), n.y += __shfl_xor_sync(0xffffffffu, n.y, o);
    if (lane == 0) s_warp[warp] = n;
    __syncthreads();
    uint2 at = make_uint2(0, 0), all = at;
    for (int w = 0; w < SELECT_WARPS; ++w) {
        const uint2 x = s_warp[w];
        if (w < warp) at.x += x.x, at.y += x.y;
        all.x += x.x, all.y += x.y;
    }
    if (blocks > 1) {
        if (tid == 0) s_mine = all;
        barrier();
        for (int r = 0; r < rank; ++r) at.x += load_cluster_u32(&s_mine.x, r), at.y += load_cluster_u32(&s_mine.y, r);
    }
    for (int i = w0; i < w1; i += 128) {
        const uint4 k4 = HOLD ? *reinterpret_cast<const uint4*>(s_keys + i + lane * 4) : load4(i + lane * 4);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        // the lane's four keys follow those of the lanes below it
        uint32_t above = 0, same = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) above += k[e] > top, same += k[e] == top;
        uint32_t both = above | same << 16;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, both, o);
            if (lane >= o) both += y;
        }
        uint32_t x = at.x + (both & 0xffff) - above, y = at.y + (both >> 16) - same;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k[e] > top || (k[e] == top && (int)y < left)) kept[x + min((int)y, left)] = p0 + i + lane * 4 + e;
            x += k[e] > top, y += k[e] == top;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, both, 31);
        at.x += total & 0xffff, at.y += total >> 16;
    }
    if (blocks > 1) barrier();  // no block ends while another reads its words
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
    // (an array of both beside one that is not: a page id would name other places in the one than in the other, and what is
    // read of the shared one may be written)
    const bool same = cache->k == to->k;
    GK_REQUIRE(ctx, (cache->v == to->v) == same && (mass == to_mass) == same &&
               (!a.from.k_scale || ((cache->k_scale == to->k_scale) == same && (cache->v_scale == to->v_scale) == same)),
               GK_ERR_ARG, "gk_paged_evict: one pool has one set of arrays, and two have two");
    GK_REQUIRE(ctx, budget >= 1 && budget <= 1 << 30 && recent >= 0 && recent <= budget, GK_ERR_ARG, "gk_paged_evict: budget %d, recent %d",
               budget, recent);
    GK_REQUIRE(ctx, aligned16(mass) && aligned16(to_mass), GK_ERR_ALIGN, "gk_paged_evict: mass must be 16-byte aligned");
    const uintptr_t x = (uintptr_t)new_len, len = (uintptr_t)B * sizeof(int32_t);
    for (const int32_t* read : {cache->kv_len, first})
        GK_REQUIRE(ctx, !read || x + len <= (uintptr_t)read || (uintptr_t)read + len <= x, GK_ERR_ARG,
                   "gk_paged_evict: new_len overlaps the old lengths or first");
    a.mass = mass;
    a.to_mass = to_mass;
    a.first = first;
    a.budget = budget;
    a.recent = recent;
    a.new_len = new_len;
    a.kept = kept;
    a.err = ctx->d_err;
    // Blocks of a cluster: of about 4096 positions each while they fit the GPU at once, four an SM (48 sequences of up to 8191,
    // 8 heads: one block a head 129.3 us with the moving, two 135.6).
    int blocks = 1;
    while (blocks < MAX_CLUSTER && a.from.capacity > 4096 * blocks && (int64_t)a.from.Hkv * B * blocks * 2 <= 4 * (int64_t)ctx->num_sms) blocks *= 2;
    const int each = (int)((cdiv(a.from.capacity, blocks) + 255) & ~int64_t(127));
    const dim3 grid((unsigned)blocks, (unsigned)a.from.Hkv, (unsigned)B);
    if (each <= HELD) {
        GK_TRY((allow_shared<evict_select_kernel<true>>(ctx, "gk_paged_evict", HELD * sizeof(uint32_t))));
        GK_TRY(launch_dependent(ctx, "paged_evict_select", evict_select_kernel<true>, grid, dim3(SELECT), each * sizeof(uint32_t), blocks, a, each));
    } else {
        GK_TRY(launch_dependent(ctx, "paged_evict_select", evict_select_kernel<false>, grid, dim3(SELECT), 0, blocks, a, each));
    }
    // A block a tile of the budget. The first tokens move too, and only the device knows their number: where a table has room
    // for more of them than for a few budgets, eight blocks an SM (first 8192 and a budget of 256, 8 sequences, 8 heads of 128:
    // 58 us, 145 with the budget's blocks alone; one sequence of 1100 with a budget of 512 would take 9.3 instead of 9.1).
    int64_t tiles = cdiv(std::min(budget, a.from.capacity), TOKENS);
    if (first && a.from.capacity / 4 > budget) tiles = std::max(tiles, std::min(cdiv(a.from.capacity, TOKENS), cdiv(8 * (int64_t)ctx->num_sms, (int64_t)a.from.Hkv * B)));
    return launch_dependent(ctx, "paged_evict_move", evict_move_kernel, dim3((unsigned)tiles, (unsigned)a.from.Hkv, (unsigned)B), dim3(MOVE), 0, 1, a);
}
