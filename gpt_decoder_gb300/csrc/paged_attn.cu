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

#include "paged_attn.cuh"

namespace gk {
namespace {

constexpr int WARPS = 4;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D += A B, bf16 operands, float32 accumulators: A 16x16, B 16x8.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose an 8x8 matrix of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
// The codes in bytes 0 and 2 of x as a pair of bf16.
__device__ __forceinline__ uint32_t codes02(const CodeMasks& k, uint32_t x) {
    const uint32_t a = and_or(x, k.low7, k.bf16_128), b = and_or(x, k.sign, k.bf16_128);
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
}
// Zero the infinities and NaN of a bf16 pair; true if there were any.
__device__ __forceinline__ bool drop_odd(uint32_t& x) {
    const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
    if (lo) x &= 0xffff0000u;
    if (hi) x &= 0x0000ffffu;
    return lo || hi;
}

// Join the pieces that the blocks of a cluster hold in shared memory: two dims a thread, over all of the
// cluster's threads, every piece's words on their way at once.
constexpr int MAX_CLUSTER = 8;
__device__ __forceinline__ void join_cluster(const AttnArgs& a, int s0, int hk, int R, int kv, int split, const float* o, int ld,
                                             const float2* ml) {
    __syncwarp();
    cluster_barrier();
    const int piece = a.split_keys(kv), pieces = max(1, (kv + piece - 1) / piece), hs = a.p.hs, per = hs >> 1;
    for (int x = split * WARPS * 32 + threadIdx.x; x < R * per; x += a.splits * WARPS * 32) {
        const int r = x / per, d = (x - r * per) * 2;
        float m[MAX_CLUSTER], w[MAX_CLUSTER], v[MAX_CLUSTER][2], top = -INFINITY, l = 0.f, y[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < MAX_CLUSTER; ++s) {
            const int from = min(s, pieces - 1);
            m[s] = load_cluster(&ml[r].x, from), w[s] = load_cluster(&ml[r].y, from);
            v[s][0] = load_cluster(o + r * ld + d, from), v[s][1] = load_cluster(o + r * ld + d + 1, from);
        }
#pragma unroll
        for (int s = 0; s < MAX_CLUSTER; ++s)
            if (s < pieces) top = fmaxf(top, m[s]);
#pragma unroll
        for (int s = 0; s < MAX_CLUSTER; ++s) {
            // a piece in which the row sees nothing has sum 0 (or NaN, which stays) and no reference; its values are
            // zeros. A factor that underflows still multiplies: what is not finite stays so.
            const float c = m[s] == -INFINITY ? (w[s] == 0.f ? 0.f : 1.f) : ex2(m[s] - top);
            if (s < pieces) l += w[s] * c, y[0] += v[s][0] * c, y[1] += v[s][1] * c;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int query = r / a.G, h = hk * a.G + r % a.G;
        *reinterpret_cast<uint32_t*>(a.y + (int64_t)(s0 + query) * a.ldy + h * hs + d) = pack(y[0] * inv, y[1] * inv);
        if (a.lse && d == 0)
            a.lse[(int64_t)(s0 + query) * a.H + h] = l == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(l)) * 0.6931471805599453f;
    }
    __syncwarp();
    cluster_barrier();  // no block ends while another reads its words
}

// HSP: head size rounded up to 64 or 128 (the rest reads as zeros). NT: tiles of 8 rows per warp.
// KG: warps that share the keys; WARPS / KG groups of rows.
template <int HSP, bool Q8, int NT, int KG>
__global__ void __launch_bounds__(WARPS * 32) attn_few_kernel(const AttnArgs a) {
    constexpr int KC = Q8 ? HSP / 64 : HSP / 32;  // 16-byte pieces of a K row per thread
    constexpr int VC = Q8 ? 1 : HSP / 64;         // and of a V row (8-bit, HSP = 64: 8 bytes)
    constexpr int MT = HSP / 16;                  // tiles of 16 dims
    constexpr int ROWS = NT * 8 * (WARPS / KG);
    __shared__ float s_o[KG][ROWS][HSP + 4];
    __shared__ float2 s_ml[KG][ROWS];
    __shared__ float2 s_join[ROWS];  // clustered: the piece's reference and sum, its weighted values in s_o[0]
    __shared__ int s_odd;
    wait_for_earlier_kernels();

    const int b = blockIdx.y, hk = blockIdx.x / a.splits, split = blockIdx.x - hk * a.splits;
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1], n = s1 - s0;
    if (n <= 0) return;
    if (n > a.max_q || s0 < 0 || s1 > a.rows) {
        if (threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
        return;
    }
    const int kv_all = max(a.p.kv_len[b], 0), kv = min(kv_all, a.p.capacity);
    if (kv_all > a.p.capacity && threadIdx.x == 0) report(a.err, GK_ERR_INDEX);
    const int R = n * a.G, hs = a.p.hs;
    const int piece = a.split_keys(kv), k_begin = split * piece, k_end = min(kv, k_begin + piece);
    if (split > 0 && k_begin >= kv) {
        if (a.clustered) join_cluster(a, s0, hk, R, kv, split, &s_o[0][0][0], HSP + 4, s_join);
        return;
    }

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kg = warp % KG, row0 = (warp / KG) * NT * 8;
    if (threadIdx.x == 0) s_odd = 0;

    // Q in the order of the K registers; rows past R are zeros
    uint32_t q[NT][HSP / 8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int i = row0 + nt * 8 + g;
        const __nv_bfloat16* src = a.q + (int64_t)(s0 + i / a.G) * a.ldq + (hk * a.G + i % a.G) * hs;
#pragma unroll
        for (int c = 0; c < HSP / 32; ++c) {
            const int d = Q8 ? ((c >> 1) * 4 + t) * 16 + (c & 1) * 8 : (c * 4 + t) * 8;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (i < R && d < hs) u = *reinterpret_cast<const uint4*>(src + d);
            if (Q8) {
                q[nt][4 * c] = __byte_perm(u.x, u.y, 0x5410);
                q[nt][4 * c + 1] = __byte_perm(u.x, u.y, 0x7632);
                q[nt][4 * c + 2] = __byte_perm(u.z, u.w, 0x5410);
                q[nt][4 * c + 3] = __byte_perm(u.z, u.w, 0x7632);
            } else {
                q[nt][4 * c] = u.x, q[nt][4 * c + 1] = u.y, q[nt][4 * c + 2] = u.z, q[nt][4 * c + 3] = u.w;
            }
        }
    }
    // the last position that each of this thread's score columns sees (kv_all - n + query)
    int last[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = row0 + nt * 8 + 2 * t + e;
            last[nt][e] = i < R ? min(kv - 1, kv_all - n + i / a.G) : -1;
        }
    const int clear = kv_all - n;  // keys up to this position are seen by every row

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
    }

    // Every load is of a row that exists: a refused page's keys are read from page 0 and masked, and
    // dims past hs from the row's last 16 bytes (Q is zero there, and such dims of the result are not
    // stored). The offsets from a tile's first row are the thread's own, once.
    const int esz = Q8 ? 1 : 2, row_bytes = hs * esz;
    uint4 kr[2][KC], vr[4][VC];
    float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
    int k_at[KC], v_at[VC];
#pragma unroll
    for (int c = 0; c < KC; ++c) k_at[c] = g * row_bytes + min((c * 4 + t) * 16, row_bytes - 16);
#pragma unroll
    for (int c = 0; c < VC; ++c)
        v_at[c] = 2 * t * row_bytes + (Q8 && HSP == 64 ? min(g * 8, row_bytes - 8) : min((c * 8 + g) * 16, row_bytes - 16));
    const int tiles = (k_end - k_begin + 15) >> 4;
    const int mine = tiles > kg ? (tiles - kg + KG - 1) / KG : 0;
    int ids = 0;
    bool bad_page = false;
    unsigned refused = 0;  // of the 32 tiles looked up last
    // the first row (token of this key / value head) of the tile's part of its page
    auto tile_row = [&](int j) -> int64_t {
        if ((j & 31) == 0) {  // 32 tiles' page ids at once, one per lane
            const int pos = k_begin + (kg + KG * (j + lane)) * 16;
            ids = 0;
            bool bad = false;
            if (j + lane < mine) {
                ids = __ldg(a.p.table + b * a.p.ld_table + (pos >> a.p.page_log2));
                if (ids < 0 || ids >= a.p.n_pages) {
                    ids = 0;
                    bad = true;
                }
            }
            bad_page |= bad;
            refused = __ballot_sync(0xffffffffu, bad);
        }
        // bf16 rows of more than 64: the next tile's keys and values (16 rows of its page) are sent for to L2, as
        // a warp's own loads leave too little on its way (48 sequences of heads of 128 124 -> 113 us, 200 of them
        // 127 -> 117, one token 7.3 -> 7.5; not with 8 bits, 89 -> 92, nor heads of 64 in pages of 16, 13.6 -> 14.9)
        if constexpr (!Q8 && HSP == 128) {
            if (lane == (j & 31) + 1 && j + 1 < mine) {
                const int pos = k_begin + (kg + KG * (j + 1)) * 16;
                const int64_t at = ((((int64_t)ids * a.p.Hkv + hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1))) * row_bytes;
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(a.p.k) + at), "r"(16 * row_bytes));
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(a.p.v) + at), "r"(16 * row_bytes));
            }
        }
        const int id = __shfl_sync(0xffffffffu, ids, j & 31);
        const int pos = k_begin + (kg + KG * j) * 16;
        return (((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
    };
    auto load_k = [&](int64_t row) {
        const char* base = static_cast<const char*>(a.p.k) + row * row_bytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int c = 0; c < KC; ++c) kr[h][c] = __ldg(reinterpret_cast<const uint4*>(base + (k_at[c] + h * 8 * row_bytes)));
            if (Q8) ks[h] = __ldg(a.p.k_scale + row + h * 8 + g);
        }
    };
    auto load_v = [&](int64_t row) {
        const char* base = static_cast<const char*>(a.p.v) + row * row_bytes;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const char* src = base + (v_at[c] + ((x >> 1) * 8 + (x & 1)) * row_bytes);
                if (Q8 && HSP == 64) {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
                    vr[x][c] = make_uint4(u.x, u.y, 0, 0);
                } else {
                    vr[x][c] = __ldg(reinterpret_cast<const uint4*>(src));
                }
            }
        if (Q8)
#pragma unroll
            for (int h = 0; h < 2; ++h) vs[h] = __ldg(a.p.v_scale + row + h * 8 + g);
    };

    int64_t row = 0;
    if (mine > 0) {
        row = tile_row(0);
        load_k(row);
        load_v(row);
    }
    bool odd = false;
    for (int j = 0; j < mine; ++j) {
        const int pos = k_begin + (kg + KG * j) * 16;
        // S^T = K Q^T: keys g, g + 8 by rows 2t, 2t + 1
        float s[NT][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const uint32_t x[2][4] = {{kr[0][c].x, kr[0][c].y, kr[0][c].z, kr[0][c].w}, {kr[1][c].x, kr[1][c].y, kr[1][c].z, kr[1][c].w}};
            if (Q8) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t a0 = codes02(a.masks, x[0][w]), a1 = codes02(a.masks, x[1][w]), a2 = codes02(a.masks, x[0][w] >> 8), a3 = codes02(a.masks, x[1][w] >> 8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(s[nt], a0, a1, a2, a3, q[nt][8 * c + 2 * w], q[nt][8 * c + 2 * w + 1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma(s[nt], x[0][2 * e], x[1][2 * e], x[0][2 * e + 1], x[1][2 * e + 1], q[nt][4 * c + 2 * e], q[nt][4 * c + 2 * e + 1]);
            }
        }
        float f[2] = {a.scale_log2, a.scale_log2}, vsc[2] = {vs[0], vs[1]};
        if (Q8) f[0] *= ks[0], f[1] *= ks[1];
        const bool off = refused >> (j & 31) & 1;  // on a refused page: not visible
        if (j + 1 < mine) {  // the next keys are on their way while this tile is finished
            row = tile_row(j + 1);
            load_k(row);
        }
        const bool part = pos + 15 > clear || pos + 16 > kv || off;  // some key some row does not see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] *= f[e >> 1];
        if (part) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (off || pos + g + (e >> 1) * 8 > last[nt][e & 1]) s[nt][e] = -INFINITY;
        }
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) move |= fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + 8.f;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[nt][e], s[nt][e + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    if (x > m[nt][e]) {
                        const float c = ex2(m[nt][e] - x);  // 0 while the row was empty
                        m[nt][e] = x;
                        l[nt][e] *= c;
#pragma unroll
                        for (int i = 0; i < MT; ++i) o[nt][i][e] *= c, o[nt][i][e + 2] *= c;
                    }
                }
        }
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ref = m[nt][e & 1];
                p[e] = ex2(s[nt][e] - (ref == -INFINITY ? 0.f : ref));
                l[nt][e & 1] += p[e];
                if (Q8) p[e] *= vsc[e >> 1];
            }
            if (Q8 && part) {  // an unseen key's scale may be anything
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (s[nt][e] == -INFINITY) p[e] = 0.f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t hi = pack(p[2 * h], p[2 * h + 1]);
                const uint32_t lo = pack(p[2 * h] - __uint_as_float(hi << 16), p[2 * h + 1] - __uint_as_float(hi & 0xffff0000u));
                ph[nt][h] = transpose8(hi);
                pl[nt][h] = transpose8(lo);
            }
        }
        if (!Q8 && part) {
            // values of keys past the end are not the cache's: zeros. An infinity or NaN that only
            // later rows see must not meet the earlier rows' zero weights: all of the tile's are taken
            // out here, and put back at the end for the rows that see them.
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const bool none = off || pos + (x >> 1) * 8 + 2 * t + (x & 1) >= kv;
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    if (none) vr[x][c] = make_uint4(0, 0, 0, 0);
                    odd |= drop_odd(vr[x][c].x) | drop_odd(vr[x][c].y) | drop_odd(vr[x][c].z) | drop_odd(vr[x][c].w);
                }
            }
        }
        // O^T += V^T P^T: dims by rows
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int w = 0; w < (Q8 && HSP == 64 ? 2 : 4); ++w) {
                uint32_t x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = w == 0 ? vr[k][c].x : w == 1 ? vr[k][c].y : w == 2 ? vr[k][c].z : vr[k][c].w;
                if (Q8) {
                    const uint32_t y0 = __byte_perm(x[0], x[1], 0x5410), y1 = __byte_perm(x[0], x[1], 0x7632);
                    const uint32_t z0 = __byte_perm(x[2], x[3], 0x5410), z1 = __byte_perm(x[2], x[3], 0x7632);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t y = half ? y1 : y0, z = half ? z1 : z0;
                        const uint32_t a0 = codes02(a.masks, y), a1 = codes02(a.masks, y >> 8), a2 = codes02(a.masks, z), a3 = codes02(a.masks, z >> 8);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma(o[nt][2 * w + half], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                            mma(o[nt][2 * w + half], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                        }
                    }
                } else {
                    const uint32_t a0 = __byte_perm(x[0], x[1], 0x5410), a1 = __byte_perm(x[0], x[1], 0x7632);
                    const uint32_t a2 = __byte_perm(x[2], x[3], 0x5410), a3 = __byte_perm(x[2], x[3], 0x7632);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(o[nt][4 * c + w], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                        mma(o[nt][4 * c + w], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                    }
                }
            }
        if (j + 1 < mine) load_v(row);
    }
    if (bad_page) report(a.err, GK_ERR_INDEX);

    // join the warps that shared the keys: the largest reference of each row, then the scaled sums
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
            if (g == 0) s_ml[kg][row0 + nt * 8 + 2 * t + e] = make_float2(m[nt][e], l[nt][e]);
        }
    __syncthreads();
    if (odd) s_odd = 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row0 + nt * 8 + 2 * t + e;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < KG; ++w) top = fmaxf(top, s_ml[w][r].x);
            const float c = m[nt][e] == -INFINITY ? (l[nt][e] == 0.f ? 0.f : 1.f) : ex2(m[nt][e] - top);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the dim of tile i's row g + 8 h, as V was dealt out
                    const int d = Q8 ? (HSP == 64 ? g * 8 : g * 16) + 2 * i + h : (i >> 2) * 64 + g * 8 + 2 * (i & 3) + h;
                    s_o[kg][r][d] = o[nt][i][e + 2 * h] * c;  // (c = 0 too: what is not finite stays so)
                }
        }
    __syncthreads();
    // write: a piece's sum for the join, or the result. Values that are not finite were taken out of every tile from
    // the one that holds key clear + 1 or the end on, keys before it in that tile among them.
    const int per = hs >> 3, odd_from = s_odd ? max(k_begin, min(clear + 1, kv) & ~15) : 0x7fffffff;
    for (int x = threadIdx.x; x < R * per; x += WARPS * 32) {
        const int r = x / per, d = (x - r * per) * 8;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < KG; ++w) top = fmaxf(top, s_ml[w][r].x);
#pragma unroll
        for (int w = 0; w < KG; ++w) {
            const float2 ml = s_ml[w][r];
            sum += ml.x == -INFINITY ? ml.y : ml.y * ex2(ml.x - top);  // (an empty part's sum is 0, or NaN)
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = s_o[0][r][d + e];
#pragma unroll
            for (int w = 1; w < KG; ++w) v[e] += s_o[w][r][d + e];
        }
        const int query = r / a.G, h = hk * a.G + r % a.G;
        for (int j = odd_from; j < k_end && j <= kv_all - n + query; ++j) {  // rare: see above
            const int id = a.p.table[b * a.p.ld_table + (j >> a.p.page_log2)];
            if (id < 0 || id >= a.p.n_pages) continue;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.p.v) +
                                       ((((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (j & ((1 << a.p.page_log2) - 1))) * hs + d;
            for (int e = 0; e < 8; ++e) {
                const float y = __bfloat162float(src[e]);
                if (!isfinite(y)) v[e] += y;
            }
        }
        const int64_t out = (int64_t)(s0 + query) * a.H + h;
        if (a.clustered) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s_o[0][r][d + e] = v[e];  // (this thread's own words)
            if (d == 0) s_join[r] = make_float2(top, sum);
        } else if (a.splits > 1) {
            float* dst = a.part_o + (out * a.splits + split) * hs + d;
            *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (d == 0) a.part_ml[out * a.splits + split] = make_float2(top, sum);
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint4*>(a.y + (int64_t)(s0 + query) * a.ldy + h * hs + d) =
                make_uint4(pack(v[0] * inv, v[1] * inv), pack(v[2] * inv, v[3] * inv), pack(v[4] * inv, v[5] * inv), pack(v[6] * inv, v[7] * inv));
            if (a.lse && d == 0) a.lse[out] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * 0.6931471805599453f;
        }
    }
    if (a.clustered) join_cluster(a, s0, hk, R, kv, split, &s_o[0][0][0], HSP + 4, s_join);
}

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

template <int HSP, bool Q8>
gk_status few(gk_ctx* ctx, const AttnArgs& a) {
    const int64_t R = (int64_t)a.max_q * a.G;
    const dim3 grid((unsigned)(a.p.Hkv * a.splits), (unsigned)a.B), block(WARPS * 32);
#define FEW(NT, KG) return launch_dependent(ctx, "paged_attn", attn_few_kernel<HSP, Q8, NT, KG>, grid, block, 0, a.clustered ? a.splits : 1, a)
    if (R <= 8) FEW(1, 4);
    if (R <= 16) FEW(2, 4);
    if constexpr (Q8)
        if (R > 32) FEW(2, 1);
    FEW(2, 2);
#undef FEW
}

}  // namespace

gk_status launch_attn_join(gk_ctx* ctx, const AttnArgs& a) {
    return launch_dependent(ctx, "paged_attn_join", attn_join_kernel, dim3((unsigned)cdiv((int64_t)a.rows * a.H, JOIN_WARPS >> join_log2(a.splits))),
                            dim3(JOIN_WARPS * 32), 0, 1, a);
}

gk_status launch_attn_few(gk_ctx* ctx, const AttnArgs& a) {
    if (a.p.hs <= 64) return a.p.k_scale ? few<64, true>(ctx, a) : few<64, false>(ctx, a);
    return a.p.k_scale ? few<128, true>(ctx, a) : few<128, false>(ctx, a);
}

}  // namespace gk

using namespace gk;

extern "C" gk_status gk_paged_attn(gk_ctx* ctx, const gk_paged_kv* cache, int dtype, const void* q, int64_t ldq, void* y,
                                   int64_t ldy, float* lse, const int32_t* q_start, int B, int H, int64_t rows, int max_q,
                                   float scale) {
    AttnArgs a{};
    GK_TRY(check_pages(ctx, "gk_paged_attn", cache, q_start, B, rows, &a.p));
    GK_REQUIRE(ctx, q && y, GK_ERR_ARG, "gk_paged_attn: null pointer");
    GK_REQUIRE(ctx, dtype == GK_BF16, GK_ERR_UNSUPPORTED, "gk_paged_attn: dtype %d (GK_BF16 only)", dtype);
    a.scale_log2 = scale * 1.4426950408889634f;
    GK_REQUIRE(ctx, H >= 1 && H <= 65535 && H % a.p.Hkv == 0 && max_q >= 1 && scale > 0.f && isfinite(a.scale_log2), GK_ERR_ARG,
               "gk_paged_attn: bad argument");
    GK_REQUIRE(ctx, ldq >= (int64_t)H * a.p.hs && ldy >= (int64_t)H * a.p.hs, GK_ERR_ARG, "gk_paged_attn: row stride");
    GK_REQUIRE(ctx, aligned16(q) && aligned16(y) && ldq % 8 == 0 && ldy % 8 == 0, GK_ERR_ALIGN,
               "gk_paged_attn: rows must be 16-byte aligned with strides a multiple of 8");
    GK_REQUIRE(ctx, std::min<int64_t>(max_q, rows) * (H / a.p.Hkv) < (1ll << 30), GK_ERR_UNSUPPORTED,
               "gk_paged_attn: %d rows of %d heads a key / value head", max_q, H / a.p.Hkv);
    if (rows == 0) return GK_OK;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.y = static_cast<__nv_bfloat16*>(y);
    a.lse = lse;
    a.q_start = q_start;
    a.ldq = ldq;
    a.ldy = ldy;
    a.B = B;
    a.H = H;
    a.G = H / a.p.Hkv;
    a.rows = (int)rows;
    a.max_q = (int)std::min<int64_t>(max_q, rows);
    a.err = ctx->d_err;
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
