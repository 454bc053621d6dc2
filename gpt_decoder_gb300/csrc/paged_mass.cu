// The attention weight that cached tokens receive: the column sums of the softmax whose rows gk_paged_attn computes.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// mass_j = sum over rows i that see j of 2^(s_ij - l_i), s = scale log2(e) q k, l = lse log2(e): with the rows' log sums
// known a key needs nothing of the other keys. A warp takes a key and walks the rows, four dims a lane.
#include <math.h>

#include <algorithm>

#include "paged.cuh"

namespace gk {
namespace {

struct MassArgs {
    Pages p;
    const __nv_bfloat16* q;
    int64_t ldq;
    const float* lse;
    const float* old;  // may be null, or `mass`
    float* mass;
    float decay, scale_log2;
    const int32_t* first;  // may be null
    const int32_t* q_start;
    int B, H, G, rows, max_q;
    int* err;
};

constexpr int WARPS = 8;

__global__ void __launch_bounds__(WARPS * 32) mass_kernel(const MassArgs a) {
    wait_for_earlier_kernels();
    const int b = blockIdx.z, hk = blockIdx.y, lane = threadIdx.x & 31, hs = a.p.hs;
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1], n = s1 - s0;
    if (n <= 0) return;
    if (n > a.max_q || s0 < 0 || s1 > a.rows) {
        if (threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
        return;
    }
    const int kv_all = max(a.p.kv_len[b], 0), kv = min(kv_all, a.p.capacity);
    if (kv_all > a.p.capacity && threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
    const int first = a.first ? min(max(a.first[b], 0), kv) : 0;
    for (int j = first + blockIdx.x * WARPS + (threadIdx.x >> 5); j < kv; j += gridDim.x * WARPS) {
        const int id = __ldg(a.p.table + b * a.p.ld_table + (j >> a.p.page_log2));
        if (id < 0 || id >= a.p.n_pages) {
            if (lane == 0) report(a.err, GK_ERR_INDEX);
            continue;
        }
        const int64_t row = (((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (j & ((1 << a.p.page_log2) - 1));
        float k[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (lane * 4 + e < hs)
                k[e] = a.p.k_scale ? (float)static_cast<const int8_t*>(a.p.k)[row * hs + lane * 4 + e]
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(a.p.k)[row * hs + lane * 4 + e]);
        const float f = a.scale_log2 * (a.p.k_scale ? a.p.k_scale[row] : 1.f);
        float sum = 0.f;
        for (int i = max(0, j - (kv_all - n)); i < n; ++i)
            for (int h = hk * a.G; h < (hk + 1) * a.G; ++h) {
                const __nv_bfloat16* q = a.q + (int64_t)(s0 + i) * a.ldq + h * hs + lane * 4;
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (lane * 4 + e < hs) s += k[e] * __bfloat162float(q[e]);
                s = warp_sum(s);
                const float l = a.lse[(int64_t)(s0 + i) * a.H + h];
                if (l != -INFINITY) sum += exp2f(s * f - l * 1.4426950408889634f);
            }
        if (lane == 0) a.mass[row] = sum + (a.old && j < kv_all - n ? a.decay * a.old[row] : 0.f);
    }
}

}  // namespace
}  // namespace gk

using namespace gk;

extern "C" gk_status gk_paged_mass(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, const float* lse,
                                   const float* old, float decay, float* mass, const int32_t* first, const int32_t* q_start, int B, int H,
                                   int64_t rows, int max_q, float scale) {
    MassArgs a{};
    GK_TRY(check_pages(ctx, "gk_paged_mass", cache, q_start, B, rows, &a.p));
    GK_REQUIRE(ctx, q && lse && mass, GK_ERR_ARG, "gk_paged_mass: null pointer");
    GK_REQUIRE(ctx, dtype == GK_BF16, GK_ERR_UNSUPPORTED, "gk_paged_mass: dtype %d (GK_BF16 only)", dtype);
    a.scale_log2 = scale * 1.4426950408889634f;
    GK_REQUIRE(ctx, H >= 1 && H <= 65535 && H % a.p.Hkv == 0 && max_q >= 1 && scale > 0.f && isfinite(a.scale_log2) && decay >= 0.f && isfinite(decay),
               GK_ERR_ARG, "gk_paged_mass: bad argument");
    GK_REQUIRE(ctx, ldq >= (int64_t)H * a.p.hs, GK_ERR_ARG, "gk_paged_mass: row stride");
    GK_REQUIRE(ctx, aligned16(q) && ldq % 8 == 0 && aligned16(old) && aligned16(mass), GK_ERR_ALIGN,
               "gk_paged_mass: rows and masses must be 16-byte aligned, strides a multiple of 8");
    GK_REQUIRE(ctx, std::min<int64_t>(max_q, rows) * (H / a.p.Hkv) < (1ll << 30), GK_ERR_UNSUPPORTED,
               "gk_paged_mass: %d rows of %d heads a key / value head", max_q, H / a.p.Hkv);
    if (rows == 0) return GK_OK;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.ldq = ldq;
    a.lse = lse;
    a.old = old;
    a.mass = mass;
    a.decay = decay;
    a.first = first;
    a.q_start = q_start;
    a.B = B;
    a.H = H;
    a.G = H / a.p.Hkv;
    a.rows = (int)rows;
    a.max_q = (int)std::min<int64_t>(max_q, rows);
    a.err = ctx->d_err;
    const int64_t blocks = std::min<int64_t>(cdiv(a.p.capacity, WARPS), cdiv(16 * (int64_t)ctx->num_sms, (int64_t)a.p.Hkv * B) + 8);
    return launch_dependent(ctx, "paged_mass", mass_kernel, dim3((unsigned)blocks, (unsigned)a.p.Hkv, (unsigned)B), dim3(WARPS * 32), 0, 1, a);
}
