// Linear layers with 4-bit weights: quantising them, and products for a few rows.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Loading weights
// into our classes" (a Linear's weight is [in, out]; here each output's K codes lie together).
#include <math.h>

#include <algorithm>

#include "launch.cuh"

namespace gk {
namespace {

// One thread per (output, group): the group's largest magnitude, the bf16 scale, the codes. It runs once a weight: the
// simplest form was kept. 8192 x 28672 from [K, M] 0.95 ms, 1.1 TB/s (0.16 of a copy: weights read twice, codes stored
// a byte at a time), from [M, K] 2.4 ms (0.07: each thread walks a row of its own).
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

// Y = X W^T for a few rows, bound by the weights' bytes: every code is read once and multiplied on
// mma.sync m16n8k16 (16 outputs by 8 rows of X; with tcgen05's tiles of 128 rows most of the product
// would be of nothing).
//   A warp takes MT tiles of 16 outputs and of K every 8th piece of 256 (128 bytes of a row): whole lines
// by cp.async into a ring of its own in shared memory, SLOTS - 1 pieces ahead, running on from one tile of
// outputs to the block's next, so that a warp waits for nobody but the memory. The ring's
// 16-byte chunks are swizzled by the row, so that the words of 8 rows come from 32 different banks.
//   A word's codes become bf16 pairs by masks: (w >> 4 i) & 0x000f000f | 0x43004300 is 128 + code, exactly,
// and 136 taken off leaves code - 8. The pairs are codes (i, i + 4); X's elements are paired the same
// way by byte permutes, once for all MT tiles. The four lanes of a row hold neighbouring words, so X is
// read 64 bytes a row at a time (from L1).
//   The products of a group are summed by the matrix instruction and then scaled in float32. The 8
// warps of a block share K, the blocks of a cluster share it again when there are few outputs; sums
// are joined in shared memory in a fixed order.
// Measured: K = 8192, M = 28672, groups of 128: 1 / 5 / 8 / 16 / 17 / 32 rows 33.5 / 35.7 / 38 / 46 / 76 / 81 us, 5 of
// them 3.4 TB/s of the codes and scales (0.50 of a copy). No pipe is full (5 rows: ALU 56%, issue 52%, DRAM 41%): a
// shift, a logic instruction and a subtraction a pair of codes, on 16 warps an SM (eight above 16 rows) that wait for
// X and the weights' words. One row of a small layer 4.7 us from the host, 2.6 in a graph.
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
    CodeMasks masks;
};

__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes i and i + 4 of a word, as bf16 (code - 8).
__device__ __forceinline__ uint32_t w4_pair(const CodeMasks& k, uint32_t w, int i) {
    const uint32_t a = and_or(w >> (4 * i), k.low4, k.bf16_128);
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&k.bf16_136));
    return *reinterpret_cast<const uint32_t*>(&d);
}

constexpr int PIECE = 256;  // codes of a row that a warp takes at a time

template <int NT, int MT>
struct W4Shared {
    static constexpr int SLOTS = NT == 4 ? 4 : 3;
    static constexpr int SLOT = MT * 16 * (PIECE / 2), RING = W4_WARPS * SLOTS * SLOT;
    static constexpr int ROW = MT * 16 + 1;
    static constexpr int BYTES = RING + W4_WARPS * NT * 8 * ROW * 4;
};

// LW: words (8 codes) of a group per lane: group / 32. NT: tiles of 8 rows. MT: tiles of 16 outputs per warp.
template <int LW, int NT, int MT>
__global__ void __launch_bounds__(W4_WARPS * 32, NT == 4 ? 1 : 2) matvec_w4_kernel(const W4Args a) {
    using S = W4Shared<NT, MT>;
    constexpr int GPP = 8 / LW;  // groups of a piece
    extern __shared__ __align__(128) uint8_t w4_smem[];
    float(*part)[NT * 8][S::ROW] = reinterpret_cast<float(*)[NT * 8][S::ROW]>(w4_smem + S::RING);
    wait_for_earlier_kernels();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int slice = blockIdx.x % a.slices, groups = a.K / (32 * LW), row_bytes = a.K / 2;
    const int tiles = (a.M + MT * 16 - 1) / (MT * 16), hop = gridDim.x / a.slices;
    const int pieces = (a.K + PIECE - 1) / PIECE, stride = a.slices * W4_WARPS, first = slice * W4_WARPS + warp;
    uint8_t* ring = w4_smem + warp * S::SLOTS * S::SLOT;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    const __nv_bfloat16* xp[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xp[nt] = a.x + (int64_t)min(nt * 8 + g, a.N - 1) * a.ldx + t * 8;

    // send for piece p of a tile's rows; outputs past M read the last one's, bytes past a row's end are zeros
    auto send = [&](int slot, int tile, int p) {
#pragma unroll
        for (int i = 0; i < MT * 4; ++i) {
            const int r = i * 4 + (lane >> 3), c = lane & 7, at = p * (PIECE / 2) + c * 16;
            const uint8_t* src = a.w + (int64_t)min(tile * MT * 16 + r, a.M - 1) * row_bytes + (at < row_bytes ? at : 0);
            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(
                             ring_at + slot * S::SLOT + r * 128 + ((c ^ (r & 7)) << 4)),
                         "l"(src), "r"(at < row_bytes ? 16 : 0)
                         : "memory");
        }
    };
    // the piece's scales, read one piece ahead
    struct Scales {
        __nv_bfloat16 s[MT][2][GPP];
    };
    const bool vector = groups % GPP == 0 && (reinterpret_cast<uintptr_t>(a.scales) & (2 * GPP - 1)) == 0;
    auto load_scales = [&](Scales& to, int tile, int p) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const __nv_bfloat16* sp = a.scales + (int64_t)min(tile * MT * 16 + mt * 16 + h * 8 + g, a.M - 1) * groups + p * GPP;
                if (vector) {
                    if constexpr (GPP == 2) *reinterpret_cast<uint32_t*>(to.s[mt][h]) = __ldg(reinterpret_cast<const uint32_t*>(sp));
                    else if constexpr (GPP == 4) *reinterpret_cast<uint2*>(to.s[mt][h]) = __ldg(reinterpret_cast<const uint2*>(sp));
                    else *reinterpret_cast<uint4*>(to.s[mt][h]) = __ldg(reinterpret_cast<const uint4*>(sp));
                } else {
#pragma unroll
                    for (int u = 0; u < GPP; ++u) to.s[mt][h][u] = sp[min(u, groups - 1 - p * GPP)];
                }
            }
    };
    // the next piece of this warp's walk over (tile, piece)
    auto step_on = [&](int& tile, int& p) {
        p += stride;
        if (p >= pieces) p = first, tile += hop;
    };
    int tile = blockIdx.x / a.slices, sent_tile = tile, sent_p = first;  // sent: the next piece to send for
    const bool works = first < pieces;
    int slot = 0, sent_slot = 0;
#pragma unroll
    for (int i = 0; i < S::SLOTS - 1; ++i) {
        if (works && sent_tile < tiles) {
            send(sent_slot, sent_tile, sent_p);
            step_on(sent_tile, sent_p);
        }
        sent_slot = sent_slot + 1 == S::SLOTS ? 0 : sent_slot + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    Scales sc;
    if (works && tile < tiles) load_scales(sc, tile, first);
    for (; tile < tiles; tile += hop) {
        float sum[MT][NT][4] = {};
        for (int p = first; p < pieces; p += stride) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::SLOTS - 2) : "memory");
            __syncwarp();  // every lane's part of the piece is there, and the slot sent for next has been read
            if (sent_tile < tiles) {
                send(sent_slot, sent_tile, sent_p);
                step_on(sent_tile, sent_p);
            }
            sent_slot = sent_slot + 1 == S::SLOTS ? 0 : sent_slot + 1;
            asm volatile("cp.async.commit_group;" ::: "memory");
            const Scales now = sc;
            {
                int tn = tile, pn = p;
                step_on(tn, pn);
                if (tn < tiles) load_scales(sc, tn, pn);
            }
            const uint8_t* rows = ring + slot * S::SLOT + t * 4;
            slot = slot + 1 == S::SLOTS ? 0 : slot + 1;
#pragma unroll
            for (int u = 0; u < GPP; ++u) {
                if (p * GPP + u >= groups) break;
                float acc[MT][NT][4] = {};
#pragma unroll
                for (int j = 0; j < LW; ++j) {
                    const int q = u * LW + j;
                    uint32_t b[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4*>(xp[nt] + p * PIECE + q * 32));
                        b[nt][0] = __byte_perm(v.x, v.z, 0x5410), b[nt][1] = __byte_perm(v.x, v.z, 0x7632);
                        b[nt][2] = __byte_perm(v.y, v.w, 0x5410), b[nt][3] = __byte_perm(v.y, v.w, 0x7632);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(rows + (mt * 16 + g) * 128 + ((q ^ g) << 4));
                        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(rows + (mt * 16 + 8 + g) * 128 + ((q ^ g) << 4));
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const uint32_t a0 = w4_pair(a.masks, w0, i), a1 = w4_pair(a.masks, w1, i), a2 = w4_pair(a.masks, w0, i + 1), a3 = w4_pair(a.masks, w1, i + 1);
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
                        for (int e = 0; e < 4; ++e) sum[mt][nt][e] = fmaf(acc[mt][nt][e], __bfloat162float(now.s[mt][e >> 1][u]), sum[mt][nt][e]);
            }
        }
        __syncthreads();  // the tile before has been written
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[warp][nt * 8 + 2 * t + (e & 1)][mt * 16 + g + (e >> 1) * 8] = sum[mt][nt][e];
        __syncthreads();
        constexpr int OUT = NT * 8 * MT * 16;
        const int m0 = tile * MT * 16;
        if (a.slices > 1) {  // this block's sum, for the cluster
            for (int i = threadIdx.x; i < OUT; i += W4_WARPS * 32) {
                const int n = i / (MT * 16), m = i - n * (MT * 16);
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < W4_WARPS; ++w) v += part[w][n][m];
                part[0][n][m] = v;
            }
            __syncwarp();
            cluster_barrier();
        }
        for (int i = slice * (W4_WARPS * 32) + threadIdx.x; i < min(OUT, a.N * MT * 16); i += a.slices * W4_WARPS * 32) {
            const int n = i / (MT * 16), m = i - n * (MT * 16);
            float v = 0.f;
            if (a.slices > 1) {
                for (int r = 0; r < a.slices; ++r) v += load_cluster(&part[0][n][m], r);
            } else {
#pragma unroll
                for (int w = 0; w < W4_WARPS; ++w) v += part[w][n][m];
            }
            if (m0 + m >= a.M) continue;
            if (a.bias) v += a.bias[m0 + m];
            if (a.residual) v += a.residual[n * a.ldr + m0 + m];
            if (a.y_f32) static_cast<float*>(a.y)[n * a.ldy + m0 + m] = v;
            else static_cast<__nv_bfloat16*>(a.y)[n * a.ldy + m0 + m] = __float2bfloat16_rn(v);
        }
        if (a.slices > 1) {  // no block goes on while another reads its sums
            __syncwarp();
            cluster_barrier();
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int LW, int NT, int MT>
gk_status run_w4(gk_ctx* ctx, W4Args& a) {
    constexpr int BYTES = W4Shared<NT, MT>::BYTES;
    GK_TRY((allow_shared<matvec_w4_kernel<LW, NT, MT>>(ctx, "gk_matvec_w4", BYTES)));
    const int64_t tiles = cdiv(a.M, MT * 16), turns = cdiv(a.K, PIECE * W4_WARPS), wave = (NT == 4 ? 1 : 2) * ctx->num_sms;
    a.slices = 1;  // a cluster shares K while that adds blocks that have work and fit the GPU once
    while (a.slices < 8 && tiles * a.slices * 2 <= wave && a.slices * 2 <= turns) a.slices *= 2;
    return launch_dependent(ctx, "matvec_w4", matvec_w4_kernel<LW, NT, MT>, dim3((unsigned)(std::min(tiles, wave) * a.slices)),
                            dim3(W4_WARPS * 32), BYTES, a.slices, a);
}

// Two tiles of outputs per warp halve the reads of X (from L1) once there are three such pairs for two
// SMs: K = 8192, two tiles against one: M = 5000 12.3 / 10.6 us, 8192 12.3 / 13.1 (16 rows 15.4 / 18.0), 28672
// 36.4 / 37.4 (16 rows 47 / 53).
template <int LW, int NT>
gk_status run_w4_tiles(gk_ctx* ctx, W4Args& a) {
    return a.M >= 48 * ctx->num_sms ? run_w4<LW, NT, 2>(ctx, a) : run_w4<LW, NT, 1>(ctx, a);
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
    GK_REQUIRE(ctx, K < (1ll << 24) && M < (1ll << 30), GK_ERR_UNSUPPORTED, "%s: sizes too large", what);
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
             ldx, ldr, ldy, (int)N, (int)K, (int)M, y_dtype == GK_F32, 1, {}};
    return group == 128 ? run_w4_rows<4>(ctx, a) : group == 64 ? run_w4_rows<2>(ctx, a) : run_w4_rows<1>(ctx, a);
}

}  // extern "C"
