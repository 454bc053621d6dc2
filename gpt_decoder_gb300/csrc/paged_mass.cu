// The attention weight that cached tokens receive: the column sums of the softmax whose rows gk_paged_attn computes.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// mass_j = sum over rows i that see j of 2^(s_ij - l_i), s = scale log2(e) q k, l = lse log2(e): with the rows' log sums
// known a key needs nothing of the other keys, and nothing is joined. Both kernels compute the scores transposed,
// S^T = K Q^T, so that a key's sum stays with the thread (or the four lanes) that holds its row.
//   Few rows: a warp takes tiles of 16 keys straight from the cache into the registers of mma.sync m16n8k16 (as the
//   attention of few rows does), its rows eight at a time from shared memory, which holds them in operand order.
//   Tiles: a block holds 256 keys in shared memory (8-bit codes as bf16, once) and walks the rows in pairs of tiles of
//   128, which TMA brings (a box of whole queries of the heads that share the keys); D = K Q^T (tcgen05, M = 128 keys, N
//   = 256 rows, so that the keys' trip through shared memory serves twice the rows) into tensor memory, a buffer for each
//   half of the keys: one is computed while the other is summed. Sixteen warps, a thread a key and one tile's rows of a
//   pair, read the scores and add their weights. A key's factor f (scale log2(e), times its own scale for codes) is
//   its thread's. The rows' log sums would be a broadcast load for every element (four wavefronts of shared memory for
//   four of them, which is all that the operands leave): they are one more 16-deep step of the product instead, of 1 / f
//   and -l in three bf16 parts each, so that D = s / f - l / f and the weight is 2^(f D).
// Measured: 48 sequences of up to 8191 8-bit keys, 8 heads of 128, a token of 32 heads each: 37 us, 4.3 TB/s (0.65 of a
// copy; ALU 55%, issue 51%: the unpacking's instructions); bf16 pages 52 us, 5.9 TB/s (0.88). Two chunks of up to 2048 rows
// behind 16384 keys, 32 heads over 8 of 128: 287 us, 1.19 PFLOP/s (0.60 of a dense product; tensor pipe 60%, exponentials
// 55% of their pipe): some 35 us are the blocks' beginnings (one of 256 keys an SM at a time), the rest waits that sixteen
// warps do not cover. (128 rows a product and two buffers: 340 us, the operands' trips through shared memory; a broadcast load of
// the log sums: 358; eight warps: 409.) Chunks of up to 1000, 12 heads of 64, 8 bits: 43 us, a third of it beginnings.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "paged_mma.cuh"
#include "tcgen05.cuh"

namespace gk {
namespace {

using namespace tc;

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
    int tile_heads, tile_queries;  // a tile of rows: this many heads of this many queries, 128 at most
    int* err;
    CodeMasks masks;
};

// The sequence that a block works on.
struct Span {
    int s0, n, kv_all, kv, first;
};
__device__ __forceinline__ bool span_of(const MassArgs& a, int b, Span& s) {
    s.s0 = a.q_start[b];
    const int s1 = a.q_start[b + 1];
    s.n = s1 - s.s0;
    if (s.n <= 0) return false;
    if (s.n > a.max_q || s.s0 < 0 || s1 > a.rows) {
        if (threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
        return false;
    }
    s.kv_all = max(a.p.kv_len[b], 0);
    s.kv = min(s.kv_all, a.p.capacity);
    if (s.kv_all > a.p.capacity && threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
    s.first = a.first ? min(max(a.first[b], 0), s.kv) : 0;
    return s.first < s.kv;
}

// ------------------------------------------------------------------------------------- few rows
constexpr int WARPS = 4;

// HSP: head size rounded up to 64 or 128 (the rest reads as zeros). NT: tiles of 8 rows.
template <int HSP, bool Q8, int NT>
__global__ void __launch_bounds__(WARPS * 32) mass_few_kernel(const MassArgs a) {
    constexpr int KC = Q8 ? HSP / 64 : HSP / 32;  // 16-byte pieces of a K row per thread
    __shared__ uint2 s_q[NT][HSP / 16][32];       // B operands, in the order of the K registers
    __shared__ float2 s_l[NT][4];                 // columns 2t, 2t + 1: log sums, in powers of two
    __shared__ int2 s_last[NT][4];                // and the last positions that they see
    wait_for_earlier_kernels();
    const int b = blockIdx.z, hk = blockIdx.y, hs = a.p.hs;
    Span s;
    if (!span_of(a, b, s)) return;
    const int tile0 = s.first >> 4, tiles = ((s.kv + 15) >> 4) - tile0;
    if ((int)blockIdx.x * WARPS >= tiles) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int R = s.n * a.G;

    for (int x = warp; x < NT * (HSP / 32); x += WARPS) {  // eight rows' 32 dims
        const int nt = x / (HSP / 32), c = x - nt * (HSP / 32), i = nt * 8 + g;
        const int d = Q8 ? ((c >> 1) * 4 + t) * 16 + (c & 1) * 8 : (c * 4 + t) * 8;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (i < R && d < hs)
            u = *reinterpret_cast<const uint4*>(a.q + (int64_t)(s.s0 + i / a.G) * a.ldq + (hk * a.G + i % a.G) * hs + d);
        if (Q8) {
            s_q[nt][2 * c][lane] = make_uint2(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.x, u.y, 0x7632));
            s_q[nt][2 * c + 1][lane] = make_uint2(__byte_perm(u.z, u.w, 0x5410), __byte_perm(u.z, u.w, 0x7632));
        } else {
            s_q[nt][2 * c][lane] = make_uint2(u.x, u.y);
            s_q[nt][2 * c + 1][lane] = make_uint2(u.z, u.w);
        }
    }
    for (int i = threadIdx.x; i < NT * 8; i += WARPS * 32) {
        const float l = i < R ? a.lse[(int64_t)(s.s0 + i / a.G) * a.H + hk * a.G + i % a.G] : -INFINITY;
        // a row without weight sees nothing
        reinterpret_cast<float*>(s_l)[i] = l * 1.4426950408889634f;
        reinterpret_cast<int*>(s_last)[i] = l == -INFINITY ? -1 : s.kv_all - s.n + i / a.G;
    }
    __syncthreads();

    const int row_bytes = hs * (Q8 ? 1 : 2), step = gridDim.x * WARPS;
    int k_at[KC];  // the thread's places in a tile; dims past hs: the row's last 16 bytes (Q is zero there)
#pragma unroll
    for (int c = 0; c < KC; ++c) k_at[c] = g * row_bytes + min((c * 4 + t) * 16, row_bytes - 16);
    int j = blockIdx.x * WARPS + warp;
    int ids = 0;
    bool bad_page = false;
    unsigned refused = 0;  // of the 32 tiles looked up last
    int round = 0;
    auto tile_row = [&](int j) -> int64_t {  // the first row of the tile's part of its page
        if ((round & 31) == 0) {             // 32 tiles' page ids at once, one per lane
            const int mine = j + lane * step;
            ids = 0;
            bool bad = false;
            if (mine < tiles) {
                ids = __ldg(a.p.table + b * a.p.ld_table + ((tile0 + mine) * 16 >> a.p.page_log2));
                if (ids < 0 || ids >= a.p.n_pages) {
                    ids = 0;
                    bad = bad_page = true;
                }
            }
            refused = __ballot_sync(0xffffffffu, bad);
        }
        const int id = __shfl_sync(0xffffffffu, ids, round & 31);
        const int pos = (tile0 + j) * 16;
        ++round;
        return (((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
    };
    uint4 kr[2][KC];
    float ks[2] = {1.f, 1.f};
    auto load_k = [&](int64_t row) {
        const char* base = static_cast<const char*>(a.p.k) + row * row_bytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int c = 0; c < KC; ++c) kr[h][c] = __ldg(reinterpret_cast<const uint4*>(base + (k_at[c] + h * 8 * row_bytes)));
            if (Q8) ks[h] = __ldg(a.p.k_scale + row + h * 8 + g);
        }
    };
    int64_t row = 0;
    bool off = false;
    if (j < tiles) {
        row = tile_row(j);
        off = refused & 1;
        load_k(row);
    }
    for (; j < tiles; j += step) {
        const int pos = (tile0 + j) * 16 + g;  // and pos + 8
        const int64_t here = row;
        const bool none = off;
        float old[2] = {0.f, 0.f};
        const bool mine = t < 2 && !none && pos + t * 8 < s.kv && pos + t * 8 >= s.first;  // lane t = 0, 1 of a row's four: key pos, pos + 8
        if (mine && a.old && pos + t * 8 < s.kv_all - s.n) old[0] = a.old[here + g + t * 8];
        float sc[NT][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const uint32_t x[2][4] = {{kr[0][c].x, kr[0][c].y, kr[0][c].z, kr[0][c].w}, {kr[1][c].x, kr[1][c].y, kr[1][c].z, kr[1][c].w}};
            if (Q8) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t a0 = codes02(a.masks, x[0][w]), a1 = codes02(a.masks, x[1][w]), a2 = codes02(a.masks, x[0][w] >> 8), a3 = codes02(a.masks, x[1][w] >> 8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 q = s_q[nt][4 * c + w][lane];
                        mma(sc[nt], a0, a1, a2, a3, q.x, q.y);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 q = s_q[nt][2 * c + e][lane];
                        mma(sc[nt], x[0][2 * e], x[1][2 * e], x[0][2 * e + 1], x[1][2 * e + 1], q.x, q.y);
                    }
            }
        }
        float f[2] = {a.scale_log2, a.scale_log2};
        if (Q8) f[0] *= ks[0], f[1] *= ks[1];
        if (j + step < tiles) {  // the next keys are on their way
            row = tile_row(j + step);
            off = refused >> ((round - 1) & 31) & 1;
            load_k(row);
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 l = s_l[nt][t];
            const int2 last = s_last[nt][t];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = ex2(fmaf(sc[nt][e], f[e >> 1], -(e & 1 ? l.y : l.x)));
                sum[e >> 1] += pos + (e >> 1) * 8 <= (e & 1 ? last.y : last.x) ? p : 0.f;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        }
        if (mine) a.mass[here + g + t * 8] = (t ? sum[1] : sum[0]) + a.decay * old[0];
    }
    if (bad_page) report(a.err, GK_ERR_INDEX);
}

// ---------------------------------------------------------------------------------------- tiles
constexpr int KEYS = 256, RT = 128, THREADS = 640, SUM_WARPS = 16;
constexpr uint32_t HALF = 128 * 128;  // 128 rows of 64 bf16
constexpr uint32_t STEP = 128 * 32;   // 128 rows of one 16-deep step
constexpr int PAIR = 2;               // tiles of rows a product
constexpr uint64_t WAIT_NS = 1000000000ull;
constexpr float LEAST_F = 0x1p-60f;    // a smaller factor (of codes): no score at all
constexpr float NO_WEIGHT = -0x1p60f;  // instead of -l: 1 / f times it is finite

template <int HSP>
struct Layout {
    static constexpr int HALVES = HSP / 64, STAGES = HSP == 64 ? 4 : 2;
    static constexpr uint32_t TILE = HALVES * HALF;
    static constexpr uint32_t Q = 2 * TILE, KX = Q + STAGES * PAIR * TILE, QX = KX + 2 * STEP, JOIN = QX + STAGES * PAIR * STEP, BARS = JOIN + KEYS * 4,
                              BYTES = BARS + 256 + 1024;
};

// (x, y) *= (s, s); (x, y) += (a, b): two float32 operations an instruction.
__device__ __forceinline__ void mul2(uint32_t& x, uint32_t& y, float s) {
    asm("{\n\t.reg .b64 v, f;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 f, {%2, %2};\n\tmul.rn.f32x2 v, v, f;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(s));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
// Barrier of `n` threads (id 1 ..; 0 is __syncthreads).
__device__ __forceinline__ void named_bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// x as three bf16 parts (24 significant bits; what is not finite is all in the first).
struct Parts {
    uint32_t p[3];
};
__device__ __forceinline__ Parts parts_of(float x) {
    Parts r;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(x);
        r.p[i] = __bfloat16_as_ushort(h);
        const float rest = x - __bfloat162float(h);
        x = isfinite(rest) ? rest : 0.f;
    }
    return r;
}
// Six products whose sum is a b: slots of the 16-deep step (the other ten are zeros).
__device__ __forceinline__ uint4 slots_a(const Parts& a) { return make_uint4(a.p[0] | a.p[0] << 16, a.p[0] | a.p[1] << 16, a.p[1] | a.p[2] << 16, 0); }
__device__ __forceinline__ uint4 slots_b(const Parts& b) { return make_uint4(b.p[0] | b.p[1] << 16, b.p[2] | b.p[0] << 16, b.p[1] | b.p[0] << 16, 0); }

template <int HSP, bool Q8>
__global__ void __launch_bounds__(THREADS, 1) mass_tiles_kernel(const MassArgs a, const __grid_constant__ CUtensorMap tm_q) {
    using L = Layout<HSP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = smem;  // [2 halves of the keys][halves of the dims]
    uint8_t* sQ = smem + L::Q;
    uint8_t* sKx = smem + L::KX;  // [2]: the step of 1 / f
    uint8_t* sQx = smem + L::QX;  // [stages]: and of -l
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t* q_full = bars;       // [4]
    uint64_t* q_empty = bars + 4;  // [4]
    uint64_t* s_full = bars + 8;   // [2 halves of the keys]
    uint64_t* s_free = bars + 12;  // [2] (an arrival per warp)
    uint64_t* bar_drain = bars + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);
    wait_for_earlier_kernels();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hs = a.p.hs;
    const int b = blockIdx.z, hk = blockIdx.y;
    Span s;
    if (!span_of(a, b, s)) return;
    const int k0 = (s.first & ~(KEYS - 1)) + blockIdx.x * KEYS;
    if (k0 >= s.kv) return;
    const bool on[2] = {k0 + RT > s.first, k0 + RT < s.kv};  // halves with a key to weigh
    // tiles of rows, from the first that sees a key of the block on
    const int parts = (a.G + a.tile_heads - 1) / a.tile_heads, seen_from = max(0, max(k0, s.first) - (s.kv_all - s.n));
    const int block0 = min(seen_from, s.n) / a.tile_queries, n_tiles = ((s.n + a.tile_queries - 1) / a.tile_queries - block0) * parts;
    const int cols = a.tile_heads * a.tile_queries, n_pairs = (n_tiles + PAIR - 1) / PAIR;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 8);
        }
        mbar_init(bar_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == SUM_WARPS + 1) tmem_alloc(tmem_slot, 512);
    for (int x = tid; x < L::STAGES * PAIR * RT; x += THREADS)
        *reinterpret_cast<uint4*>(sQx + x / RT * STEP + swizzled32(x % RT, 1)) = make_uint4(0, 0, 0, 0);
    // rows that no box of TMA fills: zeros, whose log sum gives them no weight
    for (int x = tid; x < L::STAGES * PAIR * L::HALVES * (RT - cols) * 8; x += THREADS) {
        const int t = x / ((RT - cols) * 8), r = cols + x % ((RT - cols) * 8) / 8;
        *reinterpret_cast<uint4*>(sQ + t * HALF + swizzled(r, x & 7)) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;
    auto factor = [&](int64_t row) {  // of a key's score; 0: it has none
        const float f = Q8 ? a.scale_log2 * __ldg(a.p.k_scale + row) : a.scale_log2;
        return Q8 && fabsf(f) < LEAST_F ? 0.f : f;
    };
    if (warp < SUM_WARPS) {
        // the block's keys as bf16, while the first rows are on their way; past the end, before the first, on refused
        // pages and without a score zeros
        bool bad_page = false;
        constexpr int CH = Q8 ? HSP / 16 : HSP / 8;  // 16-byte pieces of a row
#pragma unroll 4
        for (int x = tid; x < KEYS * CH; x += SUM_WARPS * 32) {
            const int r = x / CH, c = x - r * CH, pos = k0 + r;
            uint4 u = make_uint4(0, 0, 0, 0);
            float f = 1.f;
            if (pos < s.kv && pos >= s.first) {
                const int id = __ldg(a.p.table + b * a.p.ld_table + (pos >> a.p.page_log2));
                if (id >= 0 && id < a.p.n_pages) {
                    const int64_t row = (((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
                    if (c * 16 < hs * (Q8 ? 1 : 2))
                        u = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.p.k) + row * (hs * (Q8 ? 1 : 2)) + c * 16));
                    f = factor(row);
                    if (f == 0.f) u = make_uint4(0, 0, 0, 0), f = 1.f;
                } else {
                    bad_page = true;
                }
            }
            uint8_t* tile = sK + (r >> 7) * L::TILE;
            if (Q8) {
                const uint4 lo = make_uint4(codes_pair(a.masks, u.x, 0), codes_pair(a.masks, u.x, 1), codes_pair(a.masks, u.y, 0), codes_pair(a.masks, u.y, 1));
                const uint4 hi = make_uint4(codes_pair(a.masks, u.z, 0), codes_pair(a.masks, u.z, 1), codes_pair(a.masks, u.w, 0), codes_pair(a.masks, u.w, 1));
                *reinterpret_cast<uint4*>(tile + (c >> 2) * HALF + swizzled(r & 127, 2 * (c & 3))) = lo;
                *reinterpret_cast<uint4*>(tile + (c >> 2) * HALF + swizzled(r & 127, 2 * (c & 3) + 1)) = hi;
            } else {
                *reinterpret_cast<uint4*>(tile + (c >> 3) * HALF + swizzled(r & 127, c & 7)) = u;
            }
            if (c == 0) {
                *reinterpret_cast<uint4*>(sKx + (r >> 7) * STEP + swizzled32(r & 127, 0)) = slots_a(parts_of(1.f / f));
                *reinterpret_cast<uint4*>(sKx + (r >> 7) * STEP + swizzled32(r & 127, 1)) = make_uint4(0, 0, 0, 0);
            }
        }
        if (bad_page) report(a.err, GK_ERR_INDEX);
        fence_proxy_async_smem();
    }
    if (warp != SUM_WARPS) named_bar_sync(3, (SUM_WARPS + 3) * 32);  // the keys are there

    if (warp == SUM_WARPS) {  // rows by TMA, log sums by lanes (four each)
        int in_flight = -1, q0 = block0 * a.tile_queries, h0 = 0;  // of the next tile that is sent for
        int ql = q0, hl = 0;                                       // and whose log sums are read
        int query[4], head[4];  // of the lane's rows (lane, lane + 32, ..), from the tile's first
        float l[PAIR][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = lane + e * 32;
            query[e] = c < cols ? c / a.tile_heads : 1 << 30;
            head[e] = c % a.tile_heads;
        }
        auto next = [&](int& q, int& h) {
            h += a.tile_heads;
            if (h >= a.G) h = 0, q += a.tile_queries;
        };
        auto load_l = [&]() {
#pragma unroll
            for (int t = 0; t < PAIR; ++t) {  // (past the last tile: no query is left)
                const float* src = a.lse + (int64_t)(s.s0 + ql) * a.H + hk * a.G + hl;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    l[t][e] = query[e] < s.n - ql && head[e] < a.G - hl ? __ldg(src + (int64_t)query[e] * a.H + head[e]) : INFINITY;
                next(ql, hl);
            }
        };
        if (n_tiles > 0) load_l();
        for (int i = 0; i < n_pairs; ++i) {
            const int st = i % L::STAGES;
            if (!__all_sync(0xffffffffu, mbar_wait(&q_empty[st], i / L::STAGES & 1 ^ 1, nullptr, WAIT_NS))) {
                failed = true;
                break;
            }
#pragma unroll
            for (int t = 0; t < PAIR; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<uint4*>(sQx + (st * PAIR + t) * STEP + swizzled32(lane + e * 32, 0)) =
                        slots_b(parts_of(isinf(l[t][e]) ? NO_WEIGHT : l[t][e] * -1.4426950408889634f));
            fence_proxy_async_smem();
            __syncwarp();
            const int here = min(PAIR, n_tiles - i * PAIR);
            if (lane == 0) mbar_expect_tx(&q_full[st], (uint32_t)(L::HALVES * 128 * cols * here));
            for (int t = 0; t < here; ++t) {
                if (lane == 0)
                    for (int h = 0; h < L::HALVES; ++h)
                        tma_load_3d(&tm_q, &q_full[st], sQ + st * PAIR * L::TILE + (h * PAIR + t) * HALF, h * 64, hk * a.G + h0, s.s0 + q0);
                next(q0, h0);
            }
            in_flight = i;
            if (i + 1 < n_pairs) load_l();
        }
        if (failed)  // the copies in flight land before the block ends
            for (int i = max(0, in_flight - L::STAGES + 1); i <= in_flight; ++i) mbar_wait(&q_full[i % L::STAGES], i / L::STAGES & 1, nullptr, WAIT_NS / 5);
    } else if (warp == SUM_WARPS + 1) {
        const uint32_t id = instr_desc_bf16(false, false, 128, PAIR * RT);
        const uint64_t k_d = smem_desc(saddr(sK), 16, 1024), q_d = smem_desc(saddr(sQ), 16, 1024);
        const uint64_t kx_d = smem_desc32(saddr(sKx)), qx_d = smem_desc32(saddr(sQx));
        const int steps = hs >> 4;
        bool ok = true;
        for (int i = 0; ok && i < n_pairs; ++i) {
            const int st = i % L::STAGES;
            ok = __all_sync(0xffffffffu, mbar_wait(&q_full[st], i / L::STAGES & 1, nullptr, WAIT_NS));
            for (int g = 0; g < 2 && ok; ++g) {
                if (!on[g]) continue;
                ok = __all_sync(0xffffffffu, mbar_wait(&s_free[g], i & 1 ^ 1, nullptr, WAIT_NS));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t d = tmem + g * 256;
                    for (int kk = 0; kk < steps; ++kk) {
                        const uint32_t half = (kk >> 2) * HALF, at = (kk & 3) * 32;
                        umma_bf16(d, desc_add(k_d, g * L::TILE + half + at), desc_add(q_d, st * PAIR * L::TILE + PAIR * half + at), id, kk > 0);
                    }
                    // (last: the sums before it are cut at the size of the scores, not of the log sums)
                    umma_bf16(d, desc_add(kx_d, g * STEP), desc_add(qx_d, st * PAIR * STEP), id, 1);
                    umma_commit(&s_full[g]);
                }
                __syncwarp();
            }
            if (ok) {
                if (elect_one()) umma_commit(&q_empty[st]);
                __syncwarp();
            }
        }
        if (n_tiles > 0) {  // everything issued is complete before the block ends
            if (elect_one()) {
                umma_commit(bar_drain);
                mbar_wait(bar_drain, 0, nullptr, ok ? WAIT_NS : WAIT_NS / 5);
            }
            __syncwarp();
        }
        if (!ok) failed = true;
    } else if (warp < SUM_WARPS && on[warp >> 3]) {
        const int g = warp >> 3, side = warp >> 2 & 1, pos = k0 + g * RT + (warp & 3) * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * 256 + side * RT;
        int64_t row = -1;
        if (pos >= s.first && pos < s.kv) {
            const int id = __ldg(a.p.table + b * a.p.ld_table + (pos >> a.p.page_log2));
            if (id >= 0 && id < a.p.n_pages) row = (((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
        }
        float f = row >= 0 ? factor(row) : 1.f;
        if (f == 0.f) f = 1.f;
        const float before = row >= 0 && a.old && pos < s.kv_all - s.n ? a.old[row] : 0.f;
        // of the tile's columns: the first that sees the key, and the end of the rows (the tile's heads of the
        // sequence's queries, or where a query's heads fill tiles by themselves the rest of them)
        int lo = (max(0, pos - (s.kv_all - s.n)) - block0 * a.tile_queries) * a.tile_heads, part = 0;
        int left = s.n - block0 * a.tile_queries;  // queries
        auto next = [&]() {
            if (++part == parts) part = 0, lo -= cols, left -= a.tile_queries;
        };
        if (side) next();  // this thread's tiles are every other one
        float total = 0.f;
        for (int i = 0; i < n_pairs; ++i) {
            if (!__all_sync(0xffffffffu, mbar_wait(&s_full[g], i & 1, nullptr, WAIT_NS))) {
                failed = true;
                break;
            }
            tc_fence_after();
            const int hi = parts > 1 ? (left > 0 ? min(cols, a.G - part * a.tile_heads) : 0) : min(cols, max(0, min(left, RT)) * a.tile_heads);
            const bool some = __any_sync(0xffffffffu, lo > 0) || hi < cols;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            // 32 columns at a time: with four warps a scheduler the others cover the load
            auto weights = [&](auto masked) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[32];
                    tmem_ld32_nowait(lane_addr + c * 32, w);
                    tmem_wait_ld_only();
                    reg_fence32(w);
                    if (c == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_free[g]);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        mul2(w[e], w[e + 1], f);
                        mul2(w[e + 2], w[e + 3], f);
                        float p[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            p[x] = ex2_hw(__uint_as_float(w[e + x]));
                            if (decltype(masked)::value && (c * 32 + e + x < lo || c * 32 + e + x >= hi)) p[x] = 0.f;
                        }
                        add2(sum[0], sum[1], p[0], p[1]);
                        add2(sum[2], sum[3], p[2], p[3]);
                    }
                }
            };
            if (some) weights(std::true_type{});
            else weights(std::false_type{});
            total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            next();
            next();
        }
        // the two halves of a key's rows join
        float* other = reinterpret_cast<float*>(smem + L::JOIN) + g * RT + (warp & 3) * 32 + lane;
        if (side) *other = total;
        named_bar_sync(1 + g, 256);
        if (!failed && !side && row >= 0) a.mass[row] = total + *other + a.decay * before;
    }
    if (failed) report(a.err, GK_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == SUM_WARPS + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HSP, bool Q8>
gk_status launch(gk_ctx* ctx, MassArgs& a) {
    const int64_t R = (int64_t)a.max_q * a.G;
    const unsigned Hkv = (unsigned)a.p.Hkv, B = (unsigned)a.B;
    if (R <= 64) {
        // Four tiles of keys a warp, more where the blocks would be over 32 an SM (48 sequences of up to 8191 8-bit keys, 8
        // heads of 128: 8 / 16 / 32 / 64 blocks an SM 44 / 40 / 37 / 40.5 us; two or three tiles on their way at a time, 42 / 46).
        const int64_t each = 4 * WARPS * 16, most = cdiv(32 * (int64_t)ctx->num_sms, (int64_t)Hkv * B);
        const unsigned x = (unsigned)std::max<int64_t>(1, std::min(cdiv(a.p.capacity, each), most));
#define FEW(NT) return launch_dependent(ctx, "paged_mass", mass_few_kernel<HSP, Q8, NT>, dim3(x, Hkv, B), dim3(WARPS * 32), 0, 1, a)
        if (R <= 8) FEW(1);
        if (R <= 16) FEW(2);
        if (R <= 32) FEW(4);
        FEW(8);
#undef FEW
    }
    GK_TRY((allow_shared<mass_tiles_kernel<HSP, Q8>>(ctx, "gk_paged_mass", Layout<HSP>::BYTES)));
    a.tile_heads = std::min(a.G, RT);
    a.tile_queries = RT / a.tile_heads;
    CUtensorMap map{};
    GK_REQUIRE(ctx, make_map_3d(&map, a.q, a.p.hs, a.H, a.p.hs, a.rows, a.ldq, a.tile_heads, a.tile_queries), GK_ERR_CUDA,
               "gk_paged_mass: tensor map");
    return launch_dependent(ctx, "paged_mass_tiles", mass_tiles_kernel<HSP, Q8>, dim3((unsigned)cdiv(a.p.capacity, KEYS), Hkv, B),
                            dim3(THREADS), Layout<HSP>::BYTES, 1, a, map);
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
    GK_REQUIRE(ctx, H >= 1 && H <= 65535 && H % a.p.Hkv == 0 && max_q >= 1 && scale > 0.f && isfinite(scale) && decay >= 0.f && isfinite(decay),
               GK_ERR_ARG, "gk_paged_mass: bad argument");
    GK_REQUIRE(ctx, scale >= 0x1p-50f && scale <= 0x1p50f, GK_ERR_UNSUPPORTED, "gk_paged_mass: scale %g (2^-50 to 2^50)", (double)scale);
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
    const bool small = a.p.hs <= 64;
    if (a.p.k_scale) return small ? launch<64, true>(ctx, a) : launch<128, true>(ctx, a);
    return small ? launch<64, false>(ctx, a) : launch<128, false>(ctx, a);
}
