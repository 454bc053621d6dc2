// Attention of a few new tokens over the paged cache (decoding): the entry point, the kernel for few rows (
// up to 64 query rows per key / value head, 32 of bf16 pages), and the joining of split sequences.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// y_i = sum_j p_ij v_j with p_ij = 2^(s_ij - m_i) / l_i, s = scale log2(e) q k. One pass over the
// keys with a running reference m (moved, and o and l rescaled, only when a score passes it by more than
// 8, so weights stay below 2^8) and sum l.
//
// With few rows the bytes of the cache are what counts, so each is read once, straight into
// registers in the order that the matrix instructions take, with no shared memory between: the
// products are computed transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16), with 16
// keys (dims) as the rows and 8 query rows as the columns, so that one decoded token with up to 8
// heads a key / value head wastes nothing. The elements that a thread holds of a K row are 16
// contiguous bytes; Q is loaded in the same order, so the permutation of the summed index cancels.
// Of V it holds 16 bytes of four keys, paired by byte permutes. (tcgen05 takes its operands from
// shared memory in tiles of 128 rows: at these few rows it would compute 16 times what is needed
// and every byte would make the trip through shared memory.)
//   rows per key / value head: all H / Hkv heads of all n queries; row i is query i / G, head i % G.
//   A warp takes 8 or 16 rows (NT = 1, 2) and every KG-th tile of 16 keys; more rows are 2 or 4
//   warps of the block next to each other, which read the same keys (L1 serves all but one of them).
// 8-bit codes become bf16 exactly (|code| < 2^7): (code & 0x7f | 0x4300) is 128 + the low bits, and
// (code & 0x80 | 0x4300) is 128 or 256, so their difference is the code. The key's scale multiplies
// the score, the value's scale the weight.
// Weights are split into two bf16 parts (hi + lo: 16 significant bits), so the result carries no
// rounding but the output's.
// Measured: 48 sequences of up to 8191 keys, 32 query heads over 8 of 128, one token each: bf16 pages 111 us, 5.5
// TB/s of the cache's bytes (0.82 of a copy); 8-bit ones 87 us, 3.6 TB/s (0.53): no pipe is full (ALU 43%, issue
// 41%, DRAM 49%), the 12 warps an SM that the registers leave do not cover the loads' latency beside unpacking
// (four instructions a pair of codes). One token over 777 keys of 12 heads: 5.3 us from the host; 8.1 where the
// table has room for 131072 positions, as the pieces then go by that and are joined by a second launch.
#include <math.h>

#include <algorithm>

#include "paged_attn_few.cuh"

namespace gk {
namespace {

// A warp per (row, head) and up to eight pieces, four dims a lane, its pieces' loads in flight together;
// with more pieces 2, 4 or 8 warps of the block share them and add their sums in shared memory.
constexpr int JOIN_WARPS = 8;
__host__ __device__ constexpr int join_log2(int splits) { return splits <= 8 ? 0 : splits <= 16 ? 1 : splits <= 32 ? 2 : 3; }
__global__ void __launch_bounds__(JOIN_WARPS * 32) attn_join_kernel(const AttnArgs a) {
    __shared__ float4 s_o[JOIN_WARPS][32];
    __shared__ float s_l[JOIN_WARPS];
    wait_for_earlier_kernels();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = join_log2(a.splits), share = 1 << lg, sub = warp & (share - 1);
    const int64_t out = (int64_t)blockIdx.x * (JOIN_WARPS >> lg) + (warp >> lg);
    const int r = (int)(out / a.H), h = (int)(out - (int64_t)r * a.H);
    int pieces = 0;
    if (r < a.rows) {
        const int b = find_sequence(a.q_start, a.B, r);
        if (b >= 0) {
            const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
            if (s0 >= 0 && r >= s0 && r < s1 && s1 - s0 <= a.max_q && s1 <= a.rows) {
                const int kv = min(max(a.p.kv_len[b], 0), a.p.capacity);
                pieces = kv <= 0 ? 1 : (kv + a.split_keys(kv) - 1) / a.split_keys(kv);
            }
        }
    }
    const int per = a.p.hs >> 2;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, top = -INFINITY;
    if (pieces) {
        const float2* ml = a.part_ml + out * a.splits;
        const float4* po = reinterpret_cast<const float4*>(a.part_o + out * a.splits * a.p.hs) + min(lane, per - 1);
        for (int s = lane; s < pieces; s += 32) top = fmaxf(top, ml[s].x);
        top = warp_max(top);
#pragma unroll 8
        for (int s = sub; s < pieces; s += share) {
            const float2 x = ml[s];
            const float4 v = po[s * per];
            // (as in join_cluster)
            const float c = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : ex2(x.x - top);
            l += x.y * c;
            o.x += v.x * c, o.y += v.y * c, o.z += v.z * c, o.w += v.w * c;
        }
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

}  // namespace

// Refuse what no kernel could run on; fill `a` with the arguments.
gk_status check_attn(gk_ctx* ctx, const char* what, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y, int64_t ldy,
                     float* lse, const int32_t* q_start, int B, int H, int64_t rows, int max_q, float scale, AttnArgs* a) {
    GK_TRY(check_pages(ctx, what, cache, q_start, B, rows, &a->p));
    GK_REQUIRE(ctx, q && y, GK_ERR_ARG, "%s: null pointer", what);
    GK_REQUIRE(ctx, dtype == GK_BF16, GK_ERR_UNSUPPORTED, "%s: dtype %d (GK_BF16 only)", what, dtype);
    a->scale_log2 = scale * 1.4426950408889634f;
    GK_REQUIRE(ctx, H >= 1 && H <= 65535 && H % a->p.Hkv == 0 && max_q >= 1 && scale > 0.f && isfinite(a->scale_log2), GK_ERR_ARG,
               "%s: bad argument", what);
    GK_REQUIRE(ctx, ldq >= (int64_t)H * a->p.hs && ldy >= (int64_t)H * a->p.hs, GK_ERR_ARG, "%s: row stride", what);
    GK_REQUIRE(ctx, aligned16(q) && aligned16(y) && ldq % 8 == 0 && ldy % 8 == 0, GK_ERR_ALIGN,
               "%s: rows must be 16-byte aligned with strides a multiple of 8", what);
    GK_REQUIRE(ctx, std::min<int64_t>(max_q, rows) * (H / a->p.Hkv) < (1ll << 30), GK_ERR_UNSUPPORTED,
               "%s: %d rows of %d heads a key / value head", what, max_q, H / a->p.Hkv);
    a->q = static_cast<const __nv_bfloat16*>(q);
    a->y = static_cast<__nv_bfloat16*>(y);
    a->lse = lse;
    a->q_start = q_start;
    a->ldq = ldq;
    a->ldy = ldy;
    a->B = B;
    a->H = H;
    a->G = H / a->p.Hkv;
    a->rows = (int)rows;
    a->max_q = (int)std::min<int64_t>(max_q, rows);
    a->err = ctx->d_err;
    return GK_OK;
}

gk_status launch_attn_join(gk_ctx* ctx, const AttnArgs& a) {
    return launch_dependent(ctx, "paged_attn_join", attn_join_kernel, dim3((unsigned)cdiv((int64_t)a.rows * a.H, JOIN_WARPS >> join_log2(a.splits))),
                            dim3(JOIN_WARPS * 32), 0, 1, a);
}

gk_status launch_attn_few(gk_ctx* ctx, const AttnArgs& a) {
    if (a.p.hs <= 64) return a.p.k_scale ? few<64, true, WHOLE>(ctx, a) : few<64, false, WHOLE>(ctx, a);
    return a.p.k_scale ? few<128, true, WHOLE>(ctx, a) : few<128, false, WHOLE>(ctx, a);
}

}  // namespace gk

using namespace gk;

extern "C" gk_status gk_paged_attn(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y,
                                   int64_t ldy, float* lse, const int32_t* q_start, int B, int H, int64_t rows, int max_q,
                                   float scale) {
    AttnArgs a{};
    GK_TRY(check_attn(ctx, "gk_paged_attn", cache, dtype, q, ldq, y, ldy, lse, q_start, B, H, rows, max_q, scale, &a));
    if (rows == 0) return GK_OK;
    const int64_t R = (int64_t)a.max_q * a.G, per = rows * H * (a.p.hs * 4 + 8);
    // Up to 64 rows of 8-bit pages, 32 of bf16 ones, take the few-rows kernel. (48 sequences, kv up to 4000, 8
    // key / value heads of 128, 64 rows: 8-bit 224 us against 429 in tiles; bf16 221 against 121, and with 32
    // rows 126 against 129.)
    const bool few = R <= (a.p.k_scale ? 64 : 32);
    a.heads = a.p.Hkv;
    char* ws = static_cast<char*>(ctx->ws);
    size_t room = ctx->ws_bytes;
    if (!few && a.p.k_scale && (a.p.hs > 64 || R > 512)) {
        // Codes to bf16 once, in the workspace. Unpacking on the way is the slower the longer the rows: 2
        // sequences, kv up to 16384, 8 heads of 128 take 69 against 98 us at 68 rows and 79 against 128 at
        // 256; with heads of 64 (3 sequences, 12 heads) 512 rows take 80 against 74 us and 700 106 against 109.
        // If not all heads have room (three quarters, the rest is for pieces), a few of them at a time, while
        // a launch still fills half the GPU.
        const int64_t er = (int64_t)B * cdiv(a.p.capacity, 128) * 128, bytes = er * a.p.hs * 2;  // of a head
        const int64_t fit = (int64_t)(room / 2) >= bytes * a.p.Hkv ? a.p.Hkv : (int64_t)(room / 8 * 3) / bytes;
        const int64_t turns = fit ? cdiv(a.p.Hkv, fit) : 0, heads = fit ? cdiv(a.p.Hkv, turns) : 0;
        if (fit && er * heads < (1ll << 31) && (turns == 1 || 2 * heads * B * cdiv(R, 256) >= ctx->num_sms)) {
            a.heads = (int)heads;
            a.expanded_k = reinterpret_cast<__nv_bfloat16*>(ws);
            a.expanded_v = reinterpret_cast<__nv_bfloat16*>(ws + bytes * heads);
            a.expanded_rows = er * heads;
            ws += 2 * bytes * heads;
            room -= 2 * (size_t)(bytes * heads);
        }
    }
    const int64_t units = (int64_t)B * a.heads * (few ? 1 : cdiv(R, 256));
    int64_t splits;
    if (few) {
        // Pieces that give the GPU one wave of blocks (four an SM), or for batches that come near to filling it
        // by themselves four waves, which even out sequences of unequal lengths; short pieces where there are
        // few. (Sequences of up to 8191 over 8 heads of 128, 4 / 16 blocks an SM: 4 of them 17.8 / 23.3 us, 16
        // 45 / 39, 48 105 / 94. Least pieces of 128 / 256 / 1024: 16 of them 39 / 37 / -, 48 96 / 94 / 88; one
        // of 777 9.3 / 9.6 / 10.7.)
        const bool alone = units < ctx->num_sms / 2;
        a.min_split = alone ? 128 : units < ctx->num_sms ? 256 : 1024;
        splits = cdiv((alone ? 4 : 16) * (int64_t)ctx->num_sms, units);
    } else {
        // One wave: more blocks cost more to join than they even out (chunks of 1000 over 8100 keys with one /
        // two / four waves: 86 / 85 / 99 us); pieces of 1024 (100 rows of one sequence: 27.6 us, 512 33.9).
        a.min_split = 1024;
        splits = cdiv((int64_t)ctx->num_sms, units);
    }
    splits = std::min<int64_t>(splits, cdiv(a.p.capacity, a.min_split));
    // With few pieces of few sequences the blocks of a cluster join them, without a second launch (one token
    // over 777 keys 6.5 us, 9.9 with it; 3000 keys 8.7 / 10.2, 4000 10.0 / 10.4, 8000, whose pieces are long
    // then, 14.5 / 12.0; 48 sequences of up to 8191, whose blocks wait for each other, 122 / 93).
    const bool cluster = few && units < ctx->num_sms / 2;
    if (cluster && a.p.capacity <= 4096) splits = std::min<int64_t>(splits, MAX_CLUSTER);
    a.clustered = cluster && splits > 1 && splits <= MAX_CLUSTER;
    if (!a.clustered) splits = std::min<int64_t>(splits, std::min<int64_t>(256, (int64_t)(room / per)));
    a.splits = (int)std::max<int64_t>(1, splits);
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * H * a.splits * a.p.hs);
    if (few) {
        GK_TRY(launch_attn_few(ctx, a));
    } else {
        for (; a.head0 < a.p.Hkv; a.head0 += a.heads) {
            a.heads = std::min(a.heads, a.p.Hkv - a.head0);
            GK_TRY(launch_attn_tiles(ctx, a));
        }
    }
    return a.splits > 1 && !a.clustered ? launch_attn_join(ctx, a) : GK_OK;
}
