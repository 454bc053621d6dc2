// Attention of new tokens over the paged cache.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// One warp per (token row, head): the keys one after the other, each lane four elements of the
// head, with a running maximum m and sum l of the softmax (o and l rescaled when m moves).
#include <math.h>

#include "paged.cuh"

namespace gk {
namespace {

constexpr int THREADS = 128;

struct AttnArgs {
    Pages p;
    const __nv_bfloat16* q;
    __nv_bfloat16* y;
    float* lse;
    const int32_t* q_start;
    int64_t ldq, ldy;
    int B, H, rows, max_q;
    float scale;
    int* err;
};

template <bool Q8>
__global__ void __launch_bounds__(THREADS) paged_attn_kernel(AttnArgs a) {
    const int64_t w = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int r = (int)(w / a.H), h = (int)(w % a.H);
    if (r >= a.rows) return;
    const int b = find_sequence(a.q_start, a.B, r);
    if (b < 0) return;
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
    if (r < s0 || r >= s1) return;
    if (s1 - s0 > a.max_q) {
        report(a.err, GK_ERR_INDEX);
        return;
    }
    const int hs = a.p.hs, d = lane * 4;
    const bool has = d < hs;
    int64_t last = (int64_t)a.p.kv_len[b] - s1 + r;
    if (last >= a.p.capacity) {
        report(a.err, GK_ERR_INDEX);
        last = a.p.capacity - 1;
    }
    const int hk = h / (a.H / a.p.Hkv);
    float qv[4] = {}, o[4] = {}, m = -INFINITY, l = 0.f;
    if (has)
        for (int i = 0; i < 4; ++i) qv[i] = __bfloat162float(a.q[r * a.ldq + h * hs + d + i]) * a.scale;
    const int mask = (1 << a.p.page_log2) - 1;
    for (int j = 0; j <= last; ++j) {
        const int id = a.p.table[b * a.p.ld_table + (j >> a.p.page_log2)];
        if (id < 0 || id >= a.p.n_pages) {
            report(a.err, GK_ERR_INDEX);
            continue;
        }
        const int64_t vec = ((int64_t)id * a.p.Hkv + hk << a.p.page_log2) + (j & mask), at = vec * hs + d;
        float s = 0.f, vv[4] = {};
        for (int i = 0; i < 4; ++i)
            if (has) {
                if (Q8) {
                    s = fmaf(qv[i], (float)static_cast<const int8_t*>(a.p.k)[at + i], s);
                    vv[i] = (float)static_cast<const int8_t*>(a.p.v)[at + i] * a.p.v_scale[vec];
                } else {
                    s = fmaf(qv[i], __bfloat162float(static_cast<const __nv_bfloat16*>(a.p.k)[at + i]), s);
                    vv[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.p.v)[at + i]);
                }
            }
        s = warp_sum(s);
        if (Q8) s *= a.p.k_scale[vec];
        const float mn = fmaxf(m, s), c = m == mn ? 1.f : expf(m - mn), e = s == -INFINITY && mn == s ? 0.f : expf(s - mn);
        m = mn;
        l = l * c + e;
        for (int i = 0; i < 4; ++i) o[i] = o[i] * c + e * vv[i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (has)
        for (int i = 0; i < 4; ++i) a.y[r * a.ldy + h * hs + d + i] = __float2bfloat16_rn(o[i] * inv);
    if (a.lse && lane == 0) a.lse[(int64_t)r * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace gk

using namespace gk;

extern "C" gk_status gk_paged_attn(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y,
                                   int64_t ldy, float* lse, const int32_t* q_start, int B, int H, int64_t rows, int max_q,
                                   float scale) {
    AttnArgs a{};
    GK_TRY(check_pages(ctx, "gk_paged_attn", cache, q_start, B, rows, &a.p));
    GK_REQUIRE(ctx, q && y, GK_ERR_ARG, "gk_paged_attn: null pointer");
    GK_REQUIRE(ctx, dtype == GK_BF16, GK_ERR_UNSUPPORTED, "gk_paged_attn: dtype %d (GK_BF16 only)", dtype);
    GK_REQUIRE(ctx, H >= 1 && H % a.p.Hkv == 0 && max_q >= 1 && isfinite(scale), GK_ERR_ARG, "gk_paged_attn: bad argument");
    GK_REQUIRE(ctx, ldq >= (int64_t)H * a.p.hs && ldy >= (int64_t)H * a.p.hs, GK_ERR_ARG, "gk_paged_attn: row stride");
    GK_REQUIRE(ctx, aligned16(q) && aligned16(y) && ldq % 8 == 0 && ldy % 8 == 0, GK_ERR_ALIGN,
               "gk_paged_attn: rows must be 16-byte aligned with strides a multiple of 8");
    if (rows == 0) return GK_OK;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.y = static_cast<__nv_bfloat16*>(y);
    a.lse = lse;
    a.q_start = q_start;
    a.ldq = ldq;
    a.ldy = ldy;
    a.B = B;
    a.H = H;
    a.rows = (int)rows;
    a.max_q = max_q;
    a.scale = scale;
    a.err = ctx->d_err;
    const unsigned grid = (unsigned)cdiv(rows * H, THREADS / 32);
    if (a.p.k_scale) paged_attn_kernel<true><<<grid, THREADS, 0, ctx->stream>>>(a);
    else paged_attn_kernel<false><<<grid, THREADS, 0, ctx->stream>>>(a);
    return launched(ctx, "paged_attn");
}
