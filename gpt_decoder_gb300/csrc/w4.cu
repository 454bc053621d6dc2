// Linear layers with 4-bit weights: quantising them, and products for a few rows.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Loading weights
// into our classes" (a Linear's weight is [in, out]; here each output's K codes lie together).
#include <math.h>

#include "common.cuh"

namespace gk {
namespace {

// One thread per (output, group): the group's largest magnitude, the bf16 scale, the codes.
__global__ void quant_w4_kernel(const float* __restrict__ W, int64_t ldw, int transW, uint8_t* __restrict__ Wq,
                                __nv_bfloat16* __restrict__ scales, int group, int64_t K, int64_t M) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, G = K / group;
    if (i >= M * G) return;
    const int64_t m = i % M, g = i / M;  // neighbouring threads: neighbouring outputs
    const float* w = transW ? W + m * ldw + g * group : W + g * group * ldw + m;
    const int64_t step = transW ? 1 : ldw;
    float most = 0.f, z = 0.f;
    for (int k = 0; k < group; ++k) {
        const float x = w[k * step];
        most = fmaxf(most, fabsf(x));
        z += x * 0.f;  // NaN as soon as one is infinite or NaN
    }
    const bool odd = z != z;
    const __nv_bfloat16 sb = __float2bfloat16_rn(odd ? NAN : most / 7.f);
    const float s = __bfloat162float(sb);
    uint8_t* out = Wq + m * (K / 2) + g * (group / 2);
    for (int k = 0; k < group; k += 2) {
        uint32_t c[2];
        for (int e = 0; e < 2; ++e) {
            const float t = s > 0.f && !odd ? rintf(w[(k + e) * step] / s) : 0.f;
            c[e] = (uint32_t)(8 + (int)fminf(fmaxf(t, -7.f), 7.f));
        }
        out[k / 2] = (uint8_t)(c[0] | (c[1] << 4));
    }
    scales[m * G + g] = sb;
}

// One warp per (output, row).
__global__ void matvec_w4_kernel(const __nv_bfloat16* __restrict__ X, int64_t ldx, const uint8_t* __restrict__ Wq,
                                 const __nv_bfloat16* __restrict__ scales, int group, const float* __restrict__ bias,
                                 const float* residual, int64_t ldr, void* Y, int64_t ldy, int y_f32, int64_t K,
                                 int64_t M) {
    const int64_t m = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5), n = blockIdx.y;
    const int lane = threadIdx.x & 31;
    if (m >= M) return;
    float s = 0.f;
    for (int64_t i = lane; i < K / 2; i += 32) {
        const int c = Wq[m * (K / 2) + i];
        const float w = __bfloat162float(scales[m * (K / group) + 2 * i / group]);
        const float t = (float)((c & 15) - 8) * __bfloat162float(X[n * ldx + 2 * i]) +
                        (float)((c >> 4) - 8) * __bfloat162float(X[n * ldx + 2 * i + 1]);
        s = fmaf(t, w, s);
    }
    s = warp_sum(s);
    if (lane == 0) {
        if (bias) s += bias[m];
        if (residual) s += residual[n * ldr + m];
        if (y_f32) static_cast<float*>(Y)[n * ldy + m] = s;
        else static_cast<__nv_bfloat16*>(Y)[n * ldy + m] = __float2bfloat16_rn(s);
    }
}

gk_status check_w4(gk_ctx* ctx, const char* what, const void* Wq, const void* scales, int group, int64_t K, int64_t M) {
    if (!ctx) return GK_ERR_ARG;
    int dev = -1;
    GK_REQUIRE(ctx, cudaGetDevice(&dev) == cudaSuccess && dev == ctx->device, GK_ERR_ARG,
               "%s: the context's device is not current", what);
    GK_REQUIRE(ctx, Wq && scales, GK_ERR_ARG, "%s: null pointer", what);
    GK_REQUIRE(ctx, group == 32 || group == 64 || group == 128, GK_ERR_UNSUPPORTED, "%s: group %d (32, 64 or 128)", what,
               group);
    GK_REQUIRE(ctx, K >= 1 && M >= 1 && K % group == 0, GK_ERR_ARG, "%s: K must be a positive multiple of the group", what);
    GK_REQUIRE(ctx, K < (1ll << 24) && M < (1ll << 31), GK_ERR_UNSUPPORTED, "%s: sizes too large", what);
    GK_REQUIRE(ctx, aligned16(Wq) && (reinterpret_cast<uintptr_t>(scales) & 1) == 0, GK_ERR_ALIGN, "%s: misaligned weights",
               what);
    return GK_OK;
}

}  // namespace
}  // namespace gk

using namespace gk;

extern "C" {

gk_status gk_quant_w4(gk_ctx* ctx, const float* W, int64_t ldw, int transW, uint8_t* Wq, uint16_t* scales, int group,
                      int64_t K, int64_t M) {
    GK_TRY(check_w4(ctx, "gk_quant_w4", Wq, scales, group, K, M));
    GK_REQUIRE(ctx, W && ldw >= (transW ? K : M), GK_ERR_ARG, "gk_quant_w4: bad argument");
    const int64_t blocks = cdiv(M * (K / group), 256);
    GK_REQUIRE(ctx, blocks < (1ll << 31), GK_ERR_UNSUPPORTED, "gk_quant_w4: sizes too large");
    quant_w4_kernel<<<(unsigned)blocks, 256, 0, ctx->stream>>>(W, ldw, transW, Wq,
                                                               reinterpret_cast<__nv_bfloat16*>(scales), group, K, M);
    return launched(ctx, "quant_w4");
}

gk_status gk_matvec_w4(gk_ctx* ctx, int dtype, const void* X, int64_t ldx, const uint8_t* Wq, const uint16_t* scales,
                       int group, const float* bias, const float* residual, int64_t ldr, void* Y, int64_t ldy, int y_dtype,
                       int64_t N, int64_t K, int64_t M) {
    GK_TRY(check_w4(ctx, "gk_matvec_w4", Wq, scales, group, K, M));
    GK_REQUIRE(ctx, dtype == GK_BF16, GK_ERR_UNSUPPORTED, "gk_matvec_w4: dtype %d (GK_BF16 only)", dtype);
    GK_REQUIRE(ctx, y_dtype == GK_F32 || y_dtype == GK_BF16, GK_ERR_ARG, "gk_matvec_w4: y_dtype %d", y_dtype);
    GK_REQUIRE(ctx, X && Y && N >= 0 && ldx >= K && ldy >= M && (!residual || ldr >= M), GK_ERR_ARG,
               "gk_matvec_w4: bad argument");
    GK_REQUIRE(ctx, residual != Y || (y_dtype == GK_F32 && ldr == ldy), GK_ERR_ARG,
               "gk_matvec_w4: residual may alias only a float32 Y of its stride");
    GK_REQUIRE(ctx, N <= 32, GK_ERR_UNSUPPORTED, "gk_matvec_w4: %lld rows (up to 32)", (long long)N);
    GK_REQUIRE(ctx, aligned16(X) && ldx % 8 == 0, GK_ERR_ALIGN, "gk_matvec_w4: X must be 16-byte aligned, ldx a multiple of 8");
    if (N == 0) return GK_OK;
    matvec_w4_kernel<<<dim3((unsigned)cdiv(M, 8), (unsigned)N), 256, 0, ctx->stream>>>(
        static_cast<const __nv_bfloat16*>(X), ldx, Wq, reinterpret_cast<const __nv_bfloat16*>(scales), group, bias, residual,
        ldr, Y, ldy, y_dtype == GK_F32, K, M);
    return launched(ctx, "matvec_w4");
}

}  // extern "C"
