// Linear layers with 4-bit weights: quantising them, and products for a few rows.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Loading weights
// into our classes" (a Linear's weight is [in, out]; here each output's K codes lie together).
#include <math.h>

#include "launch.cuh"

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

// Y = X W^T for a few rows, bound by the weights' bytes: every code is read once, straight into the
// registers that the matrix instruction takes (mma.sync m16n8k16: 16 outputs by 8 rows of X; with
// tcgen05's tiles of 128 rows most of the product would be of nothing, and the codes would have
// to be unpacked into shared memory first).
//   A warp takes MT tiles of 16 outputs and, of each, U groups of K at a time: a lane loads
// group / 32 words (8 codes each) of outputs g and g + 8 at once, so four lanes cover a group's
// codes of a row; the next U groups are in flight while U are multiplied. A word's codes become bf16 pairs by masks:
// (w >> 4 i) & 0x000f000f | 0x43004300 is 128 + code, exactly, and 136 taken off leaves code - 8. The pairs
// are codes (i, i + 4); X's elements are paired the same way by byte permutes, once for all MT tiles.
//   The products of a group are summed by the matrix instruction and then scaled in float32. The 8
// warps of a block share the K groups, the blocks of a cluster share them again when there are few
// outputs; sums are joined in shared memory in a fixed order.
constexpr int W4_WARPS = 8;

struct W4Args {
    const __nv_bfloat16* x;
    const uint8_t* w;
    const __nv_bfloat16* scales;
    const float* bias;
    const float* residual;
    void* y;
    int64_t ldx, ldr, ldy;
    int N, K, M, y_f32, slices;  // slices: blocks (one cluster) that share a tile's K
};

__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes i and i + 4 of a word, as bf16 (code - 8).
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int i) {
    const uint32_t a = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u, b = 0x43084308u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
}

template <int LW>
struct Words {
    uint32_t w[LW];
};
template <int LW>
__device__ __forceinline__ Words<LW> load_words(const uint8_t* p) {
    Words<LW> r;
    if constexpr (LW == 4) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
    } else if constexpr (LW == 2) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
        r.w[0] = u.x, r.w[1] = u.y;
    } else {
        r.w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
    return r;
}

// LW: words of a group per lane (group / 32). NT: tiles of 8 rows. MT: tiles of 16 outputs per warp.
template <int LW, int NT, int MT>
__global__ void __launch_bounds__(W4_WARPS * 32, NT * MT == 8 ? 1 : 2) matvec_w4_kernel(const W4Args a) {
    constexpr int G = 32 * LW, U = LW == 4 ? 2 : LW == 2 ? 4 : 8;
    __shared__ float part[W4_WARPS][NT * 8][MT * 16 + 1];
    wait_for_earlier_kernels();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.x / a.slices, slice = blockIdx.x - tile * a.slices;
    const int m0 = tile * MT * 16, groups = a.K / G;
    const uint8_t* wp[MT][2];
    const __nv_bfloat16* sp[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // outputs past M read the last one's weights and are not stored
            const int64_t m = min(m0 + mt * 16 + h * 8 + g, a.M - 1);
            wp[mt][h] = a.w + m * (a.K / 2) + t * 4 * LW;
            sp[mt][h] = a.scales + m * groups;
        }
    const __nv_bfloat16* xp[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xp[nt] = a.x + (int64_t)min(nt * 8 + g, a.N - 1) * a.ldx + t * 8 * LW;
    float sum[MT][NT][4] = {};
    struct Step {
        Words<LW> w[U][MT][2];
        float s[U][MT][2];
    };
    auto load = [&](Step& to, int g0) {  // groups past the last read the last one's, and are not used
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int gi = min(g0 + u, groups - 1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) to.w[u][mt][h] = load_words<LW>(wp[mt][h] + (int64_t)gi * (G / 2));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int gi = min(g0 + u, groups - 1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) to.s[u][mt][h] = __bfloat162float(sp[mt][h][gi]);
        }
    };
    auto multiply = [&](const Step& now, int g0, int u) {
        float acc[MT][NT][4] = {};
#pragma unroll
        for (int j = 0; j < LW; ++j) {
            uint32_t b[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(xp[nt] + (g0 + u) * G + j * 8));
                b[nt][0] = __byte_perm(v.x, v.z, 0x5410), b[nt][1] = __byte_perm(v.x, v.z, 0x7632);
                b[nt][2] = __byte_perm(v.y, v.w, 0x5410), b[nt][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint32_t w0 = now.w[u][mt][0].w[j], w1 = now.w[u][mt][1].w[j];
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const uint32_t a0 = w4_pair(w0, i), a1 = w4_pair(w1, i), a2 = w4_pair(w0, i + 1), a3 = w4_pair(w1, i + 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) w4_mma(acc[mt][nt], a0, a1, a2, a3, b[nt][i], b[nt][i + 1]);
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[mt][nt][e] = fmaf(acc[mt][nt][e], now.s[u][mt][e >> 1], sum[mt][nt][e]);
    };
    // the next step's codes are on their way while this step is multiplied
    const int stride = a.slices * W4_WARPS * U;
    int g0 = (slice * W4_WARPS + warp) * U;
    Step step[2];
    auto turn = [&](const Step& now, Step& next) {
        if (g0 + stride < groups) load(next, g0 + stride);
        if (g0 + U <= groups) {
#pragma unroll
            for (int u = 0; u < U; ++u) multiply(now, g0, u);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (g0 + u < groups) multiply(now, g0, u);
        }
        g0 += stride;
    };
    if (g0 < groups) load(step[0], g0);
    while (g0 < groups) {
        turn(step[0], step[1]);
        if (g0 < groups) turn(step[1], step[0]);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[warp][nt * 8 + 2 * t + (e & 1)][mt * 16 + g + (e >> 1) * 8] = sum[mt][nt][e];
    __syncthreads();
    constexpr int OUT = NT * 8 * MT * 16;
    if (a.slices > 1) {  // this block's sum, for the cluster
        for (int i = threadIdx.x; i < OUT; i += W4_WARPS * 32) {
            const int n = i / (MT * 16), m = i - n * (MT * 16);
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < W4_WARPS; ++w) v += part[w][n][m];
            part[0][n][m] = v;
        }
        cluster_barrier();
    }
    for (int i = slice * (W4_WARPS * 32) + threadIdx.x; i < OUT; i += a.slices * W4_WARPS * 32) {
        const int n = i / (MT * 16), m = i - n * (MT * 16);
        float v = 0.f;
        if (a.slices > 1) {
            for (int r = 0; r < a.slices; ++r) v += load_cluster(&part[0][n][m], r);
        } else {
#pragma unroll
            for (int w = 0; w < W4_WARPS; ++w) v += part[w][n][m];
        }
        if (n >= a.N || m0 + m >= a.M) continue;
        if (a.bias) v += a.bias[m0 + m];
        if (a.residual) v += a.residual[n * a.ldr + m0 + m];
        if (a.y_f32) static_cast<float*>(a.y)[n * a.ldy + m0 + m] = v;
        else static_cast<__nv_bfloat16*>(a.y)[n * a.ldy + m0 + m] = __float2bfloat16_rn(v);
    }
    if (a.slices > 1) cluster_barrier();  // no block leaves while another reads its sums
}

template <int LW, int NT, int MT>
gk_status run_w4(gk_ctx* ctx, W4Args& a) {
    const int64_t tiles = cdiv(a.M, MT * 16);
    const int groups = a.K / (32 * LW), turns = (int)cdiv(groups, W4_WARPS * (LW == 4 ? 2 : LW == 2 ? 4 : 8));
    a.slices = 1;  // a cluster shares K while that adds blocks that have work and fit the GPU once
    while (a.slices < 8 && tiles * a.slices * 2 <= 2 * ctx->num_sms && a.slices * 2 <= turns) a.slices *= 2;
    return launch_dependent(ctx, "matvec_w4", matvec_w4_kernel<LW, NT, MT>, dim3((unsigned)(tiles * a.slices)),
                            dim3(W4_WARPS * 32), 0, a.slices, a);
}

// Two tiles of outputs per warp halve the reads of X (from L1) once there are enough tiles for
// two blocks an SM all the same.
template <int LW, int NT>
gk_status run_w4_tiles(gk_ctx* ctx, W4Args& a) {
    return a.M >= 32 * 2 * ctx->num_sms ? run_w4<LW, NT, 2>(ctx, a) : run_w4<LW, NT, 1>(ctx, a);
}

template <int LW>
gk_status run_w4_rows(gk_ctx* ctx, W4Args& a) {
    if (a.N <= 8) return run_w4_tiles<LW, 1>(ctx, a);
    return a.N <= 16 ? run_w4_tiles<LW, 2>(ctx, a) : run_w4_tiles<LW, 4>(ctx, a);
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
    W4Args a{static_cast<const __nv_bfloat16*>(X), Wq, reinterpret_cast<const __nv_bfloat16*>(scales), bias, residual, Y,
             ldx, ldr, ldy, (int)N, (int)K, (int)M, y_dtype == GK_F32, 1};
    return group == 128 ? run_w4_rows<4>(ctx, a) : group == 64 ? run_w4_rows<2>(ctx, a) : run_w4_rows<1>(ctx, a);
}

}  // extern "C"
