// Writing tokens into the paged cache, quantising them to 8 bits on the way, and reading them back.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (each step appends its key and value rows).
//
// Both are one pass over the rows and bound by DRAM: a token's head vector of hs elements is held
// by hs / 8 lanes (rounded up to a power of two), 16 bytes of bf16 each; its largest magnitude is
// an exchange among those lanes, and nothing is read twice. A block takes a few token rows: each
// row's sequence and page are looked up once by a warp, then all the block's threads go through
// the rows' 2 Hkv vectors.
#include "paged.cuh"

namespace gk {
namespace {

constexpr int THREADS = 256, MAX_RPB = 8;

// Where a block's rows are kept: the page's first row-of-head element is added per head.
struct Place {
    int page;   // >= 0; -1: padding (a negative position); -2: refused; -3: no sequence
    int row;    // row of the page
};

__device__ __forceinline__ Place find_place(const Pages& p, const int32_t* __restrict__ q_start, int B, int r, int* err) {
    Place at{-3, 0};
    const int b = find_sequence(q_start, B, r);
    if (b < 0) return at;
    const int s0 = __ldg(q_start + b), s1 = __ldg(q_start + b + 1), kv = __ldg(p.kv_len + b);
    if (r < s0 || r >= s1) return at;  // q_start does not ascend here
    const int64_t pos = (int64_t)kv - s1 + r;
    if (pos < 0) {
        at.page = -1;
        return at;
    }
    at.page = -2;
    if (pos < p.capacity) {
        const int id = __ldg(p.table + b * p.ld_table + (pos >> p.page_log2));
        if (id >= 0 && id < p.n_pages) at.page = id;
        at.row = (int)pos & ((1 << p.page_log2) - 1);
    }
    if (at.page == -2 && (threadIdx.x & 31) == 0) report(err, GK_ERR_INDEX);
    return at;
}

template <typename S>
__device__ __forceinline__ void load8(const S* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename S, bool Q8>
__global__ void __launch_bounds__(THREADS)
    paged_write_kernel(Pages p, const S* __restrict__ k, int64_t ldk, const S* __restrict__ v, int64_t ldv,
                       const int32_t* __restrict__ q_start, int B, int rows, int rpb, int lpv_log2, int* err) {
    __shared__ Place at[MAX_RPB];
    const int warp = threadIdx.x >> 5, r0 = blockIdx.x * rpb;
    if (warp < rpb && r0 + warp < rows) {
        const Place a = find_place(p, q_start, B, r0 + warp, err);
        if ((threadIdx.x & 31) == 0) at[warp] = a;
    }
    __syncthreads();
    const int n = min(rpb, rows - r0), per = 2 * p.Hkv;
    const int lpv = 1 << lpv_log2, part = threadIdx.x & (lpv - 1);
    const bool has = part * 8 < p.hs;
    // the loop bound is the same for all lanes of a vector, but not of a warp: a vector's lanes
    // exchange under their own mask
    const unsigned mask = lpv == 32 ? 0xffffffffu : ((1u << lpv) - 1) << ((threadIdx.x & 31) & ~(lpv - 1));
    for (int it = threadIdx.x >> lpv_log2; it < n * per; it += THREADS >> lpv_log2) {
        const int rr = it / per, h2 = it - rr * per;
        const Place a = at[rr];
        if (a.page < 0) continue;
        const bool is_v = h2 >= p.Hkv;
        const int h = is_v ? h2 - p.Hkv : h2;
        const S* src = (is_v ? v + (r0 + rr) * ldv : k + (r0 + rr) * ldk) + h * p.hs + part * 8;
        float x[8] = {};
        if (has) load8(src, x);
        const int64_t vec = ((int64_t)a.page * p.Hkv + h << p.page_log2) + a.row;
        const int64_t o = vec * p.hs + part * 8;
        if (Q8) {
            float m = 0.f, z = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m = fmaxf(m, fabsf(x[i]));
                z += x[i] * 0.f;  // NaN as soon as one is infinite or NaN
            }
            for (int s = lpv >> 1; s > 0; s >>= 1) {
                m = fmaxf(m, __shfl_xor_sync(mask, m, s));
                z += __shfl_xor_sync(mask, z, s);
            }
            const bool odd = z != z, none = !(m >= 0x1p-100f);
            const float inv = odd || none ? 0.f : 127.f / m;
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = odd ? 0 : max(-127, min(127, __float2int_rn(x[i] * inv)));
                w[i >> 2] |= ((uint32_t)c & 0xffu) << (8 * (i & 3));
            }
            if (has) *reinterpret_cast<uint2*>(static_cast<int8_t*>(is_v ? p.v : p.k) + o) = make_uint2(w[0], w[1]);
            if (part == 0) (is_v ? p.v_scale : p.k_scale)[vec] = odd ? __int_as_float(0x7fffffff) : none ? 0.f : m / 127.f;
        } else if (has) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.v : p.k) + o) = pack8(x);
        }
    }
}

template <typename D, bool Q8>
__global__ void __launch_bounds__(THREADS)
    paged_read_kernel(Pages p, D* __restrict__ k, int64_t ldk, D* __restrict__ v, int64_t ldv,
                      const int32_t* __restrict__ q_start, int B, int rows, int rpb, int lpv_log2, int* err) {
    __shared__ Place at[MAX_RPB];
    const int warp = threadIdx.x >> 5, r0 = blockIdx.x * rpb;
    if (warp < rpb && r0 + warp < rows) {
        const Place a = find_place(p, q_start, B, r0 + warp, err);
        if ((threadIdx.x & 31) == 0) at[warp] = a;
    }
    __syncthreads();
    const int n = min(rpb, rows - r0), per = 2 * p.Hkv;
    const int part = threadIdx.x & ((1 << lpv_log2) - 1);
    if (part * 8 >= p.hs) return;
    for (int it = threadIdx.x >> lpv_log2; it < n * per; it += THREADS >> lpv_log2) {
        const int rr = it / per, h2 = it - rr * per;
        const Place a = at[rr];
        if (a.page == -3) continue;
        const bool is_v = h2 >= p.Hkv;
        const int h = is_v ? h2 - p.Hkv : h2;
        float x[8] = {};
        if (a.page >= 0) {
            const int64_t vec = ((int64_t)a.page * p.Hkv + h << p.page_log2) + a.row;
            const int64_t o = vec * p.hs + part * 8;
            if (Q8) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(is_v ? p.v : p.k) + o));
                const float s = (is_v ? p.v_scale : p.k_scale)[vec];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t w = i < 4 ? u.x : u.y;
                    x[i] = (float)(int8_t)(w >> (8 * (i & 3))) * s;
                }
            } else {
                load8(static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + o, x);
            }
        }
        D* dst = (is_v ? v + (r0 + rr) * ldv : k + (r0 + rr) * ldk) + h * p.hs + part * 8;
        if constexpr (sizeof(D) == 4) {
            __stcs(reinterpret_cast<float4*>(dst), make_float4(x[0], x[1], x[2], x[3]));
            __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
            __stcs(reinterpret_cast<uint4*>(dst), pack8(x));
        }
    }
}

gk_status check_rows(gk_ctx* ctx, const char* what, const Pages& p, int dtype, const void* k, int64_t ldk, const void* v,
                     int64_t ldv) {
    GK_REQUIRE(ctx, k && v, GK_ERR_ARG, "%s: null pointer", what);
    GK_REQUIRE(ctx, dtype == GK_F32 || dtype == GK_BF16, GK_ERR_ARG, "%s: dtype %d", what, dtype);
    GK_REQUIRE(ctx, ldk >= (int64_t)p.Hkv * p.hs && ldv >= (int64_t)p.Hkv * p.hs, GK_ERR_ARG, "%s: row stride", what);
    GK_REQUIRE(ctx, aligned16(k) && aligned16(v) && ldk % 8 == 0 && ldv % 8 == 0, GK_ERR_ALIGN,
               "%s: rows must be 16-byte aligned with strides a multiple of 8", what);
    return GK_OK;
}

}  // namespace
}  // namespace gk

using namespace gk;

// Rows per block: eight (a warp looks each up) once that still fills the GPU, else one.
#define ROWS_AND_LANES                                                     \
    const int rpb = rows >= (int64_t)MAX_RPB * 4 * ctx->num_sms ? MAX_RPB : 1; \
    int lpv = 1;                                                           \
    while ((8 << lpv) < p.hs) ++lpv;                                       \
    const unsigned grid = (unsigned)cdiv(rows, rpb);

extern "C" {

gk_status gk_paged_write(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* k, int64_t ldk, const void* v,
                         int64_t ldv, const int32_t* q_start, int B, int64_t rows) {
    Pages p;
    GK_TRY(check_pages(ctx, "gk_paged_write", cache, q_start, B, rows, &p));
    GK_TRY(check_rows(ctx, "gk_paged_write", p, dtype, k, ldk, v, ldv));
    if (rows == 0) return GK_OK;
    ROWS_AND_LANES
#define WRITE(S, Q8)                                                                                           \
    paged_write_kernel<S, Q8><<<grid, THREADS, 0, ctx->stream>>>(p, static_cast<const S*>(k), ldk,              \
                                                                 static_cast<const S*>(v), ldv, q_start, B, (int)rows, \
                                                                 rpb, lpv, ctx->d_err)
    if (dtype == GK_F32) {
        if (p.k_scale) WRITE(float, true);
        else WRITE(float, false);
    } else {
        if (p.k_scale) WRITE(__nv_bfloat16, true);
        else WRITE(__nv_bfloat16, false);
    }
#undef WRITE
    return launched(ctx, "paged_write");
}

gk_status gk_paged_read(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, void* k, int64_t ldk, void* v, int64_t ldv,
                        const int32_t* q_start, int B, int64_t rows) {
    Pages p;
    GK_TRY(check_pages(ctx, "gk_paged_read", cache, q_start, B, rows, &p));
    GK_TRY(check_rows(ctx, "gk_paged_read", p, dtype, k, ldk, v, ldv));
    if (rows == 0) return GK_OK;
    ROWS_AND_LANES
#define READ(D, Q8)                                                                                                 \
    paged_read_kernel<D, Q8><<<grid, THREADS, 0, ctx->stream>>>(p, static_cast<D*>(k), ldk, static_cast<D*>(v), ldv, \
                                                                q_start, B, (int)rows, rpb, lpv, ctx->d_err)
    if (dtype == GK_F32) {
        if (p.k_scale) READ(float, true);
        else READ(float, false);
    } else {
        if (p.k_scale) READ(__nv_bfloat16, true);
        else READ(__nv_bfloat16, false);
    }
#undef READ
    return launched(ctx, "paged_read");
}

}  // extern "C"
