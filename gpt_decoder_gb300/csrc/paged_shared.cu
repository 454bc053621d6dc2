// Attention of a batch whose sequences share prefixes: the entry point, the kernel for few rows (paged_attn_few.cuh) over
// prefixes and what follows them, and the joining of a row's parts.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// A softmax over two sets of keys is joined from each set's reference m, sum l and weighted values o (not divided):
// y = (o_1 2^(m_1 - m) + o_2 2^(m_2 - m)) / (l_1 2^(m_1 - m) + l_2 2^(m_2 - m)), m the larger. So a group's prefix is
// attended as one sequence that holds the rows of all of its sequences (they lie next to each other): with S sequences its
// bytes are read once instead of S times, and the rows that meet a key are S times as many, which is what the tensor
// cores need. Then each sequence attends to its own keys. Both are the kernels of gk_paged_attn, launched beside each
// other (Branch, launch.cuh).
// Measured: a token of 64 sequences behind 16384 shared 8-bit keys and up to 1024 own ones, 32 heads over 8 of 128: 82 us
// (gk_paged_attn 361): 23 to lay the codes out as bf16, beside the own keys, 49 the prefix in tiles of 128 rows (8 key tiles a
// block at its softmax warps' rate for codes and weights in two parts, and 15 to begin and end), 10 the join; bf16 pages 63
// (539). 7 groups of up to 16 sequences behind up to 8100 keys, 12 heads of 64, bf16: 43 us, 3.0 TB/s (121): blocks of few
// tiles, a third of their time the loads that lead to the first key; 8 bits 33 (119). Chunks of 256 behind 16384 keys, 12
// sequences a group: 717 (784), as own keys fill the SMs that the prefixes' last wave leaves; the tensor cores' part bounds
// both. 8 bits, 256 MB of workspace: 1049 (3431, whose codes have no room as bf16).
#include <math.h>

#include <algorithm>

#include "paged_attn_few.cuh"

namespace gk {
namespace {

template <int PART>
gk_status launch_few(gk_ctx* ctx, const AttnArgs& a) {
    if (a.p.hs <= 64) return a.p.k_scale ? few<64, true, PART>(ctx, a) : few<64, false, PART>(ctx, a);
    return a.p.k_scale ? few<128, true, PART>(ctx, a) : few<128, false, PART>(ctx, a);
}

// A row and head: four dims a lane, the prefix's pieces and then its own keys'; with more than eight pieces 2, 4 or 8
// warps of the block share them and add their sums in shared memory.
constexpr int JOIN_WARPS = 8;
__host__ __device__ constexpr int join_log2(int slots) { return slots <= 8 ? 0 : slots <= 16 ? 1 : slots <= 32 ? 2 : 3; }
__global__ void __launch_bounds__(JOIN_WARPS * 32) shared_join_kernel(const AttnArgs a) {
    __shared__ float4 s_o[JOIN_WARPS][32];
    __shared__ float s_l[JOIN_WARPS];
    wait_for_earlier_kernels();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = join_log2(a.slots), share = 1 << lg, sub = warp & (share - 1);
    const int64_t out = (int64_t)blockIdx.x * (JOIN_WARPS >> lg) + (warp >> lg);
    const int r = (int)(out / a.H), h = (int)(out - (int64_t)r * a.H);
    int2 parts = make_int2(0, 0);
    if (r < a.rows && r >= a.q_start[0] && r < a.q_start[a.B]) parts = a.row_parts[r];
    // (held to what there is, whatever a q_start that does not ascend has left)
    const int first = min(max(parts.x, 0), a.slot0), pieces = first + min(max(parts.y, 0), a.slots - a.slot0), skip = a.slot0 - first;
    const int per = a.p.hs >> 2;
    float top = -INFINITY;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (pieces) {
        const float2* ml = a.part_ml + out * a.slots;
        const float4* po = reinterpret_cast<const float4*>(a.part_o + out * a.slots * a.p.hs) + min(lane, per - 1);
        auto place = [&](int s) { return s < first ? s : s + skip; };
        // the first eight of the warp's values are on their way while the references are looked through
        constexpr int AHEAD = 8;
        float4 v[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (sub + u * share < pieces) v[u] = po[place(sub + u * share) * per];
        const float2 mine = lane < pieces ? ml[place(lane)] : make_float2(-INFINITY, 0.f);
        top = mine.x;
        for (int s = lane + 32; s < pieces; s += 32) top = fmaxf(top, ml[place(s)].x);
        top = warp_max(top);
        auto add = [&](const float2& x, const float4& v) {
            // a piece in which the row sees nothing has sum 0 (or NaN, which stays) and no reference; its values are
            // zeros. A factor that underflows still multiplies: what is not finite stays so.
            const float c = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : ex2(x.x - top);
            l += x.y * c;
            o.x += v.x * c, o.y += v.y * c, o.z += v.z * c, o.w += v.w * c;
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int s = sub + u * share;
            if (s >= pieces) break;
            float2 x;
            if (s < 32) x = make_float2(__shfl_sync(0xffffffffu, mine.x, s), __shfl_sync(0xffffffffu, mine.y, s));
            else x = ml[place(s)];
            add(x, v[u]);
        }
#pragma unroll 4
        for (int s = sub + AHEAD * share; s < pieces; s += share) add(ml[place(s)], po[place(s) * per]);
    }
    if (lg) {
        s_o[warp][lane] = o;
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (sub) return;
        for (int w = 1; w < share; ++w) {
            const float4 v = s_o[warp + w][lane];
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            l += s_l[warp + w];
        }
    }
    if (!pieces) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane < per)
        *reinterpret_cast<uint2*>(a.y + (int64_t)r * a.ldy + h * a.p.hs + lane * 4) = make_uint2(pack(o.x * inv, o.y * inv), pack(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[out] = l == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(l)) * 0.6931471805599453f;
}

// Up to this many rows of a key / value head take the few-rows kernel (as for gk_paged_attn).
bool is_few(const AttnArgs& a, int64_t rows) { return rows <= (a.p.k_scale ? 64 : 32); }

// Pieces of the prefixes' `units` (groups, heads, pairs of row tiles). Few rows: four or sixteen blocks an SM, as
// for gk_paged_attn, but pieces of 512 where there are some groups (7 of up to 8100 keys, 12 heads of 64: 43.1 us against
// 47.7 with pieces of 256). Tiles: one wave, pieces of 256 at least.
void split_prefixes(gk_ctx* ctx, bool few, int64_t units, int capacity, int64_t* splits, int* least) {
    const bool alone = units < ctx->num_sms / 2;
    *least = !few ? 256 : alone ? 128 : 512;
    *splits = cdiv((!few ? 1 : alone ? 4 : 16) * (int64_t)ctx->num_sms, units);
    *splits = std::max<int64_t>(1, std::min(*splits, cdiv(capacity, *least)));
}
// And of what follows them: mostly short, so pieces of 256 and two of them at most once they fill the GPU (64 sequences of
// up to 1024 own keys, 8 heads: two pieces 82.2 us in all, five 86.0, five of 1024 91.1; 54 sequences 43.1, 44.8, 48.0).
void split_own(gk_ctx* ctx, bool few, int64_t units, int capacity, int64_t* splits, int* least) {
    *least = few ? (units < ctx->num_sms / 2 ? 128 : 256) : 1024;
    *splits = few ? std::max<int64_t>(2, cdiv(4 * (int64_t)ctx->num_sms, units)) : cdiv((int64_t)ctx->num_sms, units);
    *splits = std::max<int64_t>(1, std::min(*splits, cdiv(capacity, *least)));
}

}  // namespace

gk_status launch_shared_few(gk_ctx* ctx, const AttnArgs& a, int part) {
    return part == PREFIX ? launch_few<PREFIX>(ctx, a) : launch_few<OWN>(ctx, a);
}

}  // namespace gk

using namespace gk;

extern "C" gk_status gk_paged_attn_shared(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y,
                                          int64_t ldy, float* lse, const int32_t* q_start, int B, const int32_t* group_start,
                                          const int32_t* prefix_len, int n_groups, int H, int64_t rows, int max_q, int max_group_q,
                                          float scale) {
    AttnArgs a{};
    GK_TRY(check_attn(ctx, "gk_paged_attn_shared", cache, dtype, q, ldq, y, ldy, lse, q_start, B, H, rows, max_q, scale, &a));
    GK_REQUIRE(ctx, group_start && prefix_len, GK_ERR_ARG, "gk_paged_attn_shared: null pointer");
    GK_REQUIRE(ctx, n_groups >= 1 && n_groups <= 65535 && max_group_q >= 1, GK_ERR_ARG, "gk_paged_attn_shared: bad groups");
    GK_REQUIRE(ctx, std::min<int64_t>(max_group_q, rows) * a.G < (1ll << 30), GK_ERR_UNSUPPORTED,
               "gk_paged_attn_shared: groups of %d rows of %d heads a key / value head", max_group_q, a.G);
    if (rows == 0) return GK_OK;
    // Sharing costs two launches, a branch and a join, and wins from about 1000 positions on for a token of many sequences, from
    // more for wide heads and for chunks. Tables of 4096 positions, prefixes of 250 / 1000 / 2000 / 3900, a token of one group
    // (against each sequence alone): 12 heads of 64, bf16, 16 sequences 12.5 / 12.5 / 13.6 / 15.9 us (11 / 21 / 22 / 37), 64 of
    // them 17 / 18 / 21 / 25 (19 / 38 / 55 / 93); 32 heads over 8 of 128, 8 bits, 16 of them 21 / 21 / 21 / 24 (13 / 19 / 26 / 39),
    // 64 39 / 40 / 42 / 44 (20 / 42 / 63 / 101); 2 sequences 11 to 13.5 (6 to 10), which win from 16000 on (16.6 against 20). 16
    // chunks of 256 behind 1000, 32 heads over 8 of 128, bf16: 193 (100), 8 bits 211 (133); behind 8000 494 (942). The lengths are
    // on the device; the table's width bounds them, and one border stands for all of these.
    if (a.p.capacity < 2048 || 2 * (int64_t)n_groups > B) return gk_paged_attn(ctx, cache, dtype, q, ldq, y, ldy, lse, q_start, B, H, rows, max_q, scale);
    a.group_start = group_start;
    a.prefix_len = prefix_len;
    a.n_groups = n_groups;
    a.sequences = B;
    a.max_group = (int)std::min<int64_t>(max_group_q, rows);
    a.heads = a.p.Hkv;

    const int64_t group_rows = (int64_t)a.max_group * a.G, own_rows = (int64_t)a.max_q * a.G, per = rows * H * (a.p.hs * 4 + 8);
    const size_t info = ((size_t)rows * sizeof(int2) + 15) & ~size_t(15);
    const bool prefix_few = is_few(a, group_rows), own_few = is_few(a, own_rows);
    char* ws = static_cast<char*>(ctx->ws);
    size_t room = ctx->ws_bytes;
    AttnArgs p = a;  // the prefixes' launch
    // A sequence's rows keep the 16 bits of weights that gk_paged_attn gives them, however many rows the group has (64 samples
    // behind 16384 keys: 82.1 us, with bf16 weights 77.9 and 0.0023 of the result off 64 bits instead of y's own 0.0016).
    p.fine = own_few && !prefix_few;
    p.B = n_groups;
    p.max_q = a.max_group;
    int64_t prefix_splits, own_splits;
    const int64_t pairs = prefix_few ? 1 : cdiv(group_rows, 256);  // blocks a prefix and head
    split_prefixes(ctx, prefix_few, (int64_t)n_groups * a.p.Hkv * pairs, a.p.capacity, &prefix_splits, &p.min_split);
    split_own(ctx, own_few, (int64_t)B * a.p.Hkv * (own_few ? 1 : cdiv(own_rows, 256)), a.p.capacity, &own_splits, &a.min_split);
    if (room < info + 2 * per) return gk_paged_attn(ctx, cache, dtype, q, ldq, y, ldy, lse, q_start, B, H, rows, max_q, scale);
    if (!prefix_few && a.p.k_scale && (a.p.hs > 64 || group_rows > 512)) {
        // 8-bit codes laid out as bf16 first, as in gk_paged_attn: of the prefixes, all heads or a few at a time, in what the
        // rows' parts leave of the workspace. (64 samples behind 15300 keys, 8 heads of 128: 81 us with 96 MB; 64 MB hold 21
        // parts of the rows but not the codes beside them, which are then unpacked on the way: 96 us, each sequence alone 338.)
        const int64_t parts = info + std::min<int64_t>(512, prefix_splits + own_splits) * per, left = std::max<int64_t>(0, (int64_t)room - parts);
        const int64_t er = (int64_t)n_groups * cdiv(a.p.capacity, 128) * 128, bytes = er * a.p.hs * 2;  // of a head
        const int64_t fit = std::min<int64_t>(a.p.Hkv, left / (2 * bytes));
        const int64_t turns = fit ? cdiv(a.p.Hkv, fit) : 0, heads = fit ? cdiv(a.p.Hkv, turns) : 0;
        if (fit && er * heads < (1ll << 31) && (turns == 1 || 2 * heads * n_groups * pairs >= ctx->num_sms)) {
            p.heads = (int)heads;
            p.expanded_k = reinterpret_cast<__nv_bfloat16*>(ws);
            p.expanded_v = reinterpret_cast<__nv_bfloat16*>(ws + bytes * heads);
            p.expanded_rows = er * heads;
            ws += 2 * bytes * heads;
            room -= 2 * (size_t)(bytes * heads);
            split_prefixes(ctx, prefix_few, n_groups * heads * pairs, a.p.capacity, &prefix_splits, &p.min_split);
        }
    }
    const int64_t slots = std::min<int64_t>(512, (int64_t)((room - info) / per));
    prefix_splits = std::min(prefix_splits, std::max<int64_t>(1, slots * prefix_splits / (prefix_splits + own_splits)));
    own_splits = std::min(own_splits, slots - prefix_splits);
    p.splits = (int)prefix_splits;
    a.splits = (int)own_splits;
    a.prefix_splits = p.splits;
    a.prefix_min = p.min_split;
    a.slots = p.slots = p.splits + a.splits;
    a.slot0 = p.splits;
    a.row_parts = reinterpret_cast<int2*>(ws);
    a.part_o = p.part_o = reinterpret_cast<float*>(ws + info);
    a.part_ml = p.part_ml = reinterpret_cast<float2*>(a.part_o + rows * H * a.slots * a.p.hs);
    // The own keys' launch beside the prefixes': neither reads what the other writes, and each by itself leaves much of the
    // GPU idle (one after the other: 64 samples, then with weights of one part, 82.5 us, 7 groups 44.7, chunks 806; side by
    // side 77.6, 43.1, 714).
    const bool expanded = p.expanded_k && p.heads == a.p.Hkv;
    Branch own(ctx);
    GK_TRY(own.fork());
    if (expanded) GK_TRY(launch_shared_expand(ctx, p));
    if (prefix_few) {
        GK_TRY(launch_shared_few(ctx, p, PREFIX));
    } else {
        for (; p.head0 < a.p.Hkv; p.head0 += p.heads) {
            p.heads = std::min(p.heads, a.p.Hkv - p.head0);
            if (p.expanded_k && !expanded) GK_TRY(launch_shared_expand(ctx, p));
            GK_TRY(launch_shared_tiles(ctx, p, PREFIX));
        }
    }
    GK_TRY(own.run([&] { return own_few ? launch_shared_few(ctx, a, OWN) : launch_shared_tiles(ctx, a, OWN); }));
    GK_TRY(own.join());
    return launch_dependent(ctx, "paged_shared_join", shared_join_kernel, dim3((unsigned)cdiv(rows * H, JOIN_WARPS >> join_log2(a.slots))),
                            dim3(JOIN_WARPS * 32), 0, 1, a);
}
