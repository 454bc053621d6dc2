// The kernel of attention of few rows over the paged cache (its mathematics and layout: paged_attn.cu), for whole
// sequences, shared prefixes and what follows them.
#pragma once

#include <math.h>

#include "paged_attn.cuh"
#include "paged_mma.cuh"

namespace gk {

constexpr int MAX_CLUSTER = 8;

namespace {

constexpr int WARPS = 4;

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
// Zero the infinities and NaN of a bf16 pair; true if there were any.
__device__ __forceinline__ bool drop_odd(uint32_t& x) {
    const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
    if (lo) x &= 0xffff0000u;
    if (hi) x &= 0x0000ffffu;
    return lo || hi;
}

// Join the pieces that the blocks of a cluster hold in shared memory: two dims a thread, over all of the
// cluster's threads, every piece's words on their way at once.
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
template <int HSP, bool Q8, int NT, int KG, int PART>
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
    if (PART == OWN && hk == a.p.Hkv) return leave_row_parts(a, b);
    Rows rows;
    if (!rows_of<PART>(a, b, rows)) return;
    const int s0 = rows.s0, n = rows.n, kv_all = rows.kv_all, kv = rows.kv, from = rows.from, tb = rows.table;
    const int R = n * a.G, hs = a.p.hs;
    const int base = first_tile(from), piece = a.split_keys(kv - base), start = base + split * piece, k_end = min(kv, start + piece);
    const int k_begin = PART == OWN ? max(start, from & ~15) : start;  // (from lies in the first piece)
    if (split > 0 && start >= kv) {
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
                ids = __ldg(a.p.table + tb * a.p.ld_table + (pos >> a.p.page_log2));
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
        const bool part = pos + 15 > clear || pos + 16 > kv || off || (PART == OWN && pos < from);  // some key some row does not see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] *= f[e >> 1];
        if (part) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (off || pos + g + (e >> 1) * 8 > last[nt][e & 1] || (PART == OWN && pos + g + (e >> 1) * 8 < from)) s[nt][e] = -INFINITY;
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
                const int at = pos + (x >> 1) * 8 + 2 * t + (x & 1);
                const bool none = off || at >= kv || (PART == OWN && at < from);
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
    // the one that holds key clear + 1 or the end on, keys before it in that tile among them. (Own keys behind a prefix:
    // from the tile in which it ends too, so all are gone through; those that were in the sums count twice.)
    const int per = hs >> 3, odd_from = !s_odd ? 0x7fffffff : PART == OWN ? max(k_begin, from) : max(k_begin, min(clear + 1, kv) & ~15);
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
            const int id = a.p.table[tb * a.p.ld_table + (j >> a.p.page_log2)];
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
        } else if (PART != WHOLE || a.splits > 1) {
            const int64_t slot = PART == WHOLE ? out * a.splits + split : out * a.slots + a.slot0 + split;
            float* dst = a.part_o + slot * hs + d;
            *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (d == 0) a.part_ml[slot] = make_float2(top, sum);
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint4*>(a.y + (int64_t)(s0 + query) * a.ldy + h * hs + d) =
                make_uint4(pack(v[0] * inv, v[1] * inv), pack(v[2] * inv, v[3] * inv), pack(v[4] * inv, v[5] * inv), pack(v[6] * inv, v[7] * inv));
            if (a.lse && d == 0) a.lse[out] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * 0.6931471805599453f;
        }
    }
    if (a.clustered) join_cluster(a, s0, hk, R, kv, split, &s_o[0][0][0], HSP + 4, s_join);
}

template <int HSP, bool Q8, int PART>
gk_status few(gk_ctx* ctx, const AttnArgs& a) {
    const int64_t R = (int64_t)a.max_q * a.G;
    const dim3 grid((unsigned)(a.p.Hkv * a.splits + (PART == OWN)), (unsigned)a.B), block(WARPS * 32);
#define FEW(NT, KG) return launch_dependent(ctx, "paged_attn", attn_few_kernel<HSP, Q8, NT, KG, PART>, grid, block, 0, a.clustered ? a.splits : 1, a)
    if (R <= 8) FEW(1, 4);
    if (R <= 16) FEW(2, 4);
    if constexpr (Q8)
        if (R > 32) FEW(2, 1);
    FEW(2, 2);
#undef FEW
}

}  // namespace
}  // namespace gk
