// Writing tokens into the paged cache, quantising them to 8 bits on the way, and reading them back.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (each step appends its key and value rows).
//
// Both are one pass over the rows and bound by DRAM: a token's head vector of hs elements is held
// by hs / 16 lanes (rounded up to a power of two), 16 elements each; its largest magnitude is
// an exchange among those lanes, and nothing is read twice. A block takes a few token rows: each
// row's sequence and page are looked up once by a warp, then all the block's threads go through
// the rows' 2 Hkv vectors.
// Measured: reading back 16 sequences of up to 16384 8-bit tokens of 8 heads of 128 as bf16 111 us, 6.2 TB/s
// (0.91 of a copy), of bf16 pages 136 us, 6.7 TB/s (0.99); storing 7 chunks of up to 4096 of them 22.6 us, 4.2 TB/s
// (0.62; issue 69%: the quantiser's instructions in less than two waves of blocks), reading those back 19.1, 5.0 TB/s
// (0.74), of bf16 pages 23.5 (0.79) and 22.0 (0.84). A few rows cost their launches: 4 us to read 333 rows.
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

// Sixteen values as a thread holds them.
struct Float16 {
    float x[16];
};
__device__ __forceinline__ Float16 load16(const float* p) {
    Float16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + i);
        r.x[4 * i] = a.x, r.x[4 * i + 1] = a.y, r.x[4 * i + 2] = a.z, r.x[4 * i + 3] = a.w;
    }
    return r;
}
__device__ __forceinline__ Float16 load16(const __nv_bfloat16* p) {
    Float16 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
            r.x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    return r;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) __stcs(reinterpret_cast<float4*>(p) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(pack(x[8 * i], x[8 * i + 1]), pack(x[8 * i + 2], x[8 * i + 3]),
                                                           pack(x[8 * i + 4], x[8 * i + 5]), pack(x[8 * i + 6], x[8 * i + 7])));
}

// The block's rows and the thread's part of their vectors, the same for writing and reading: 2^lanes_log2
// neighbouring threads hold a head vector, 16 elements each; a pass of the loop covers one row's 2 Hkv
// vectors (keys, then values) or THREADS >> lanes_log2 of them.
template <typename F>
__device__ __forceinline__ void each_vector(const Pages& p, const int32_t* __restrict__ q_start, int B, int rows, int rpb,
                                            int lanes_log2, int* err, F&& visit) {
    __shared__ Place at[MAX_RPB];
    const int warp = threadIdx.x >> 5, r0 = blockIdx.x * rpb;
    if (warp < rpb && r0 + warp < rows) {
        const Place a = find_place(p, q_start, B, r0 + warp, err);
        if ((threadIdx.x & 31) == 0) at[warp] = a;
    }
    __syncthreads();
    const int n = min(rpb, rows - r0), per = 2 * p.Hkv, step = THREADS >> lanes_log2;
    const int first = threadIdx.x >> lanes_log2;
    int rr = first / per, h = first - rr * per;  // row of the block, vector of the row
    const int d_row = step / per, d_h = step - d_row * per;
    while (rr < n) {
        const Place a = at[rr];
        const bool is_v = h >= p.Hkv;
        const int head = is_v ? h - p.Hkv : h;
        visit(r0 + rr, a, is_v, head, ((int64_t)a.page * p.Hkv + head << p.page_log2) + a.row);
        rr += d_row;
        h += d_h;
        if (h >= per) h -= per, ++rr;
    }
}

// Eight blocks an SM, at a few spilled words: the last wave is fuller (7 chunks of up to 4096, with their reading:
// six blocks 41.0 us, eight 39.1; from float32 62.2 / 59.8).
template <typename S, bool Q8>
__global__ void __launch_bounds__(THREADS, 8)
    paged_write_kernel(Pages p, const S* __restrict__ k, int64_t ldk, const S* __restrict__ v, int64_t ldv,
                       const int32_t* __restrict__ q_start, int B, int rows, int rpb, int lanes_log2, int* err) {
    wait_for_earlier_kernels();
    const int lanes = 1 << lanes_log2, part = (threadIdx.x & (lanes - 1)) * 16;
    const bool has = part < p.hs;
    // a vector's threads exchange under their own mask: a warp's vectors may end in different passes
    const unsigned mask = ((1u << lanes) - 1) << ((threadIdx.x & 31) & ~(lanes - 1));
    each_vector(p, q_start, B, rows, rpb, lanes_log2, err, [&](int r, const Place& a, bool is_v, int head, int64_t vec) {
        if (a.page < 0) return;
        const S* src = (is_v ? v + r * ldv : k + r * ldk) + head * p.hs + part;
        Float16 f = {};
        if (has) f = load16(src);
        const int64_t o = vec * p.hs + part;
        if (Q8) {
            // as bit patterns magnitudes compare like the numbers, infinities and NaN above all
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = max(most, __float_as_uint(f.x[i]) & 0x7fffffffu);
            for (int s = lanes >> 1; s > 0; s >>= 1) most = max(most, __shfl_xor_sync(mask, most, s));
            const float m = __uint_as_float(most);
            const bool odd = most >= 0x7f800000u, none = odd || m < 0x1p-100f;
            const float inv = 127.f / m;
            // x * inv is at most 127 (1 + 2^-23): adding 1.5 x 2^23 rounds it to a whole number, ties to
            // even, whose two's complement is the sum's low byte
            uint32_t c[16], w[4];
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i] = __float_as_uint(__fadd_rn(__fmul_rn(f.x[i], inv), 12582912.f));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = none ? 0u : __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
            if (has) *reinterpret_cast<uint4*>(static_cast<int8_t*>(is_v ? p.v : p.k) + o) = make_uint4(w[0], w[1], w[2], w[3]);
            if (part == 0) (is_v ? p.v_scale : p.k_scale)[vec] = odd ? __int_as_float(0x7fffffff) : none ? 0.f : m / 127.f;
        } else if (has) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v : p.k) + o;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                reinterpret_cast<uint4*>(dst)[i] = make_uint4(pack(f.x[8 * i], f.x[8 * i + 1]), pack(f.x[8 * i + 2], f.x[8 * i + 3]),
                                                              pack(f.x[8 * i + 4], f.x[8 * i + 5]), pack(f.x[8 * i + 6], f.x[8 * i + 7]));
        }
    });
}

template <typename D, bool Q8>
__global__ void __launch_bounds__(THREADS)
    paged_read_kernel(Pages p, D* __restrict__ k, int64_t ldk, D* __restrict__ v, int64_t ldv,
                      const int32_t* __restrict__ q_start, int B, int rows, int rpb, int lanes_log2, int* err) {
    wait_for_earlier_kernels();
    const int part = (threadIdx.x & ((1 << lanes_log2) - 1)) * 16;
    each_vector(p, q_start, B, rows, rpb, lanes_log2, err, [&](int r, const Place& a, bool is_v, int head, int64_t vec) {
        if (a.page == -3 || part >= p.hs) return;
        Float16 f = {};
        if (a.page >= 0) {
            const int64_t o = vec * p.hs + part;
            if (Q8) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(is_v ? p.v : p.k) + o));
                const float s = (is_v ? p.v_scale : p.k_scale)[vec];
                const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
#pragma unroll
                for (int i = 0; i < 16; ++i)  // 2^23 + code + 128 by bytes, exactly
                    f.x[i] = (__uint_as_float(__byte_perm(w[i >> 2], 0x4b000000u, 0x7440 | (i & 3))) - 8388736.f) * s;
            } else {
                f = load16(static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + o);
            }
        }
        store16((is_v ? v + r * ldv : k + r * ldk) + head * p.hs + part, f.x);
    });
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

// Rows per block: eight (a warp looks each up) once that is a block an SM, else one. (Stores of 7
// sequences' up to 600 / 1200 / 4096 rows, eight a block against one: 13.6 / 14.7, 16.8 / 23.0, 40.9 / 61.5 us.)
#define ROWS_AND_LANES                                                     \
    const int rpb = rows >= (int64_t)MAX_RPB * ctx->num_sms ? MAX_RPB : 1; \
    int lanes = 0;                                                         \
    while ((16 << lanes) < p.hs) ++lanes;                                  \
    const unsigned grid = (unsigned)cdiv(rows, rpb);

extern "C" {

gk_status gk_paged_write(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* k, int64_t ldk, const void* v,
                         int64_t ldv, const int32_t* q_start, int B, int64_t rows) {
    Pages p;
    GK_TRY(check_pages(ctx, "gk_paged_write", cache, q_start, B, rows, &p));
    GK_TRY(check_rows(ctx, "gk_paged_write", p, dtype, k, ldk, v, ldv));
    if (rows == 0) return GK_OK;
    ROWS_AND_LANES
#define WRITE(S, Q8)                                                                                                     \
    return launch_dependent(ctx, "paged_write", paged_write_kernel<S, Q8>, dim3(grid), dim3(THREADS), 0, 1, p,            \
                            static_cast<const S*>(k), ldk, static_cast<const S*>(v), ldv, q_start, B, (int)rows, rpb, lanes, \
                            ctx->d_err)
    if (dtype == GK_F32) {
        if (p.k_scale) WRITE(float, true);
        else WRITE(float, false);
    } else {
        if (p.k_scale) WRITE(__nv_bfloat16, true);
        else WRITE(__nv_bfloat16, false);
    }
#undef WRITE
}

gk_status gk_paged_read(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, void* k, int64_t ldk, void* v, int64_t ldv,
                        const int32_t* q_start, int B, int64_t rows) {
    Pages p;
    GK_TRY(check_pages(ctx, "gk_paged_read", cache, q_start, B, rows, &p));
    GK_TRY(check_rows(ctx, "gk_paged_read", p, dtype, k, ldk, v, ldv));
    if (rows == 0) return GK_OK;
    ROWS_AND_LANES
#define READ(D, Q8)                                                                                                  \
    return launch_dependent(ctx, "paged_read", paged_read_kernel<D, Q8>, dim3(grid), dim3(THREADS), 0, 1, p,          \
                            static_cast<D*>(k), ldk, static_cast<D*>(v), ldv, q_start, B, (int)rows, rpb, lanes, ctx->d_err)
    if (dtype == GK_F32) {
        if (p.k_scale) READ(float, true);
        else READ(float, false);
    } else {
        if (p.k_scale) READ(__nv_bfloat16, true);
        else READ(__nv_bfloat16, false);
    }
#undef READ
}

}  // extern "C"
