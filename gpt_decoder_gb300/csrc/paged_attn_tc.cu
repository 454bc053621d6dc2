// Attention of chunks of new tokens over the paged cache, on the tensor cores (tcgen05).
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// A block takes two tiles of 128 query rows of one key / value head (the H / Hkv heads that share it
// side by side: row i is query i / G, head i % G, so its keys are read once for all of them) and
// walks the keys in tiles of 128:
//   S = Q K^T   (M = 128 rows, N = 128 keys, K = head size) into tensor memory;
//   softmax     a thread per row: P = 2^(s - m) with s in powers of two, as bf16 over S in tensor
//               memory; the reference m moves (and O is rescaled there) only when the row's maximum
//               passes it by more than 8;
//   O += P V    (N = head size, K = 128 keys), accumulated in tensor memory.
// The two tiles take turns: while one group of four warps turns its S into P, the tensor core
// computes the other's products. Warps 8-11 bring the keys: pages lie anywhere, so rows are
// gathered, 16 bytes a thread, into the 128-byte-swizzled layouts that the MMAs read; bf16 pages
// by cp.async (zero-filled past the end), 8-bit pages through registers, where the codes become bf16
// (exactly). Codes carry no scale into the products: the key's scale multiplies the score and
// the value's scale the weight, both from shared memory. Warp 12 issues the MMAs.
// K and V have rings of their own (a K tile is free once both S are there, a V tile after both
// products), of three tiles each for head sizes up to 64 and two for 128.
// Registers: 512 threads at 128; the softmax warpgroups take 176 each, the copying one 104, the
// MMA warp's 48.
// All mbarrier waits are bounded (timeout -> GK_ERR_TIMEOUT in the error word).
#include <algorithm>

#include "paged_attn.cuh"
#include "tcgen05.cuh"

namespace gk {
namespace {

using namespace tc;

constexpr int QT = 128, KT = 128, THREADS = 512;
constexpr uint32_t HALF = 128 * 128;  // 128 rows of 64 bf16
constexpr uint64_t WAIT_NS = 1000000000ull;

template <int HSP>
struct Layout {
    static constexpr int HALVES = HSP / 64, STAGES = HSP == 64 ? 3 : 2;
    static constexpr uint32_t TILE = HALVES * HALF;
    static constexpr uint32_t K = 2 * TILE, V = K + STAGES * TILE, SCALES = V + STAGES * TILE;
    static constexpr uint32_t BARS = SCALES + 2 * 4 * KT * 4;  // [4 tiles][k, v][128 keys]
    static constexpr uint32_t BYTES = BARS + 512 + 1024;
};

// Byte offset of the 16 bytes at chunk c (of 8) of row r in a 128-byte-swizzled half tile.
__device__ __forceinline__ uint32_t swizzled(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
// Codes 0 and 1 (or 2 and 3) of a word as a pair of bf16: 128 + the low seven bits, less 128 or 256.
__device__ __forceinline__ uint32_t codes_pair(uint32_t w, int second) {
    const uint32_t x = __byte_perm(w, 0, second ? 0x4342 : 0x4140);
    const uint32_t a = (x & 0x007f007fu) | 0x43004300u, b = (x & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ bool drop_odd2(uint32_t& x) {  // infinities and NaN of a bf16 pair become zeros
    const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
    if (lo) x &= 0xffff0000u;
    if (hi) x &= 0x0000ffffu;
    return lo || hi;
}

// What one block works on.
struct Item {
    int b, hk, split, s0, n, R, row0;  // rows row0 .. row0 + 255 of R
    int kv_all, kv, k_begin, k_end;    // keys k_begin .. k_end - 1 of this piece
    int t0, t1;                        // key tiles that some row of each query tile sees
    __device__ __forceinline__ int tiles(int g) const { return g ? t1 : t0; }
    __device__ __forceinline__ int last(int row, int G) const { return min(kv - 1, kv_all - n + row / G); }
};

template <int HSP, bool Q8>
__global__ void __launch_bounds__(THREADS, 1) attn_tiles_kernel(const AttnArgs a) {
    using L = Layout<HSP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;           // [2 tiles][halves]
    uint8_t* sK = smem + L::K;    // [stages][halves]
    uint8_t* sV = smem + L::V;
    float* s_ks = reinterpret_cast<float*>(smem + L::SCALES);  // [4][128]: scale of the scores per key
    float* s_vs = s_ks + 4 * KT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t* q_full = bars;         // [2] tile's rows are there (128 arrivals)
    uint64_t* k_full = bars + 2;     // [3] (128)
    uint64_t* k_empty = bars + 5;    // [3]
    uint64_t* v_full = bars + 8;     // [3] (128)
    uint64_t* v_empty = bars + 11;   // [3]
    uint64_t* c_full = bars + 14;    // [4] the tile's scales and refused pages are there (128)
    uint64_t* bar_s = bars + 18;     // [2] S_g is there
    uint64_t* bar_p = bars + 20;     // [2] P_g is there (128)
    uint64_t* bar_o = bars + 22;     // [2] O_g is complete
    uint64_t* bar_drain = bars + 24;
    volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(bars + 25);  // [4] 16-key groups on refused pages
    volatile int* s_odd = reinterpret_cast<volatile int*>(bars + 27);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 28);
    wait_for_earlier_kernels();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Item it;
    {
        const int pairs = gridDim.x / a.splits;
        const int pair = pairs - 1 - blockIdx.x / a.splits;  // the last rows see the most keys: first
        it.split = blockIdx.x % a.splits;
        it.b = blockIdx.z;
        it.hk = blockIdx.y;
        it.s0 = a.q_start[it.b];
        const int s1 = a.q_start[it.b + 1];
        it.n = s1 - it.s0;
        if (it.n <= 0) return;
        if (it.n > a.max_q || it.s0 < 0 || s1 > a.rows) {
            if (tid == 0) report(a.err, GK_ERR_INDEX);
            return;
        }
        it.R = it.n * a.G;
        it.row0 = pair * 2 * QT;
        if (it.row0 >= it.R) return;
        it.kv_all = max(a.p.kv_len[it.b], 0);
        it.kv = min(it.kv_all, a.p.capacity);
        if (it.kv_all > a.p.capacity && tid == 0) report(a.err, GK_ERR_INDEX);
        const int piece = a.split_keys(it.kv);
        it.k_begin = it.split * piece;
        it.k_end = min(it.kv, it.k_begin + piece);
        if (it.split > 0 && it.k_begin >= it.kv) return;
        auto seen_tiles = [&](int first) {
            const int rows = min(QT, it.R - first);
            const int seen = rows > 0 ? min(it.k_end, it.last(first + rows - 1, a.G) + 1) : 0;
            return seen > it.k_begin ? (seen - it.k_begin + KT - 1) / KT : 0;
        };
        it.t0 = seen_tiles(it.row0);
        it.t1 = seen_tiles(it.row0 + QT);
    }
    const int n_kv = max(it.t0, it.t1);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 128);
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_p[i], 128);
            mbar_init(&bar_o[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&k_full[i], 128);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 128);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&c_full[i], 128);
        mbar_init(bar_drain, 1);
        *s_odd = 0;
        for (int i = 0; i < 4; ++i) s_bad[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int hs = a.p.hs;
    bool failed = false;

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 12) {
            const uint32_t id_s = instr_desc_bf16(false, false, 128, 128);
            const uint32_t id_o = instr_desc_bf16(false, true, 128, HSP);
            const uint64_t q_d = smem_desc(saddr(sQ), 16, 1024), k_d = smem_desc(saddr(sK), 16, 1024);
            const uint64_t v_d = smem_desc(saddr(sV), HALF, 1024);
            bool ok = true, issued = false;
            uint32_t stage = 0, phase = 0;  // of tile j
            auto scores = [&](int g, uint32_t st) {
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HSP / 16; ++kk) {
                        const uint32_t at = (kk >> 2) * HALF + (kk & 3) * 32;
                        umma_bf16(tmem + g * 128, desc_add(q_d, g * L::TILE + at), desc_add(k_d, st * L::TILE + at), id_s, kk > 0);
                    }
                    umma_commit(&bar_s[g]);
                }
                __syncwarp();
                issued = true;
            };
            if (n_kv > 0) ok = __all_sync(0xffffffffu, mbar_wait(&k_full[0], 0, nullptr, WAIT_NS));
            for (int g = 0; g < 2 && ok; ++g)
                if (it.tiles(g) > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&q_full[g], 0, nullptr, WAIT_NS));
                    if (!ok) break;
                    tc_fence_after();
                    scores(g, 0);
                }
            if (ok && n_kv > 0) {
                if (elect_one()) umma_commit(&k_empty[0]);
                __syncwarp();
            }
            for (int j = 0; ok && j < n_kv; ++j) {
                const uint32_t sn = stage + 1 == L::STAGES ? 0 : stage + 1, pn = sn ? phase : phase ^ 1;
                bool have_v = false, have_k = false;
                for (int g = 0; g < 2 && ok; ++g) {
                    if (j >= it.tiles(g)) continue;
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar_p[g], j & 1, nullptr, WAIT_NS));
                    if (ok && !have_v) ok = __all_sync(0xffffffffu, mbar_wait(&v_full[stage], phase, nullptr, WAIT_NS));
                    if (!ok) break;
                    have_v = true;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            umma_bf16_ts(tmem + 256 + g * HSP, tmem + g * 128 + kk * 8, desc_add(v_d, stage * L::TILE + kk * 2048),
                                         id_o, (j > 0 || kk > 0) ? 1u : 0u);
                        if (j == it.tiles(g) - 1) umma_commit(&bar_o[g]);
                    }
                    __syncwarp();
                    if (j + 1 < it.tiles(g)) {
                        if (!have_k) ok = __all_sync(0xffffffffu, mbar_wait(&k_full[sn], pn, nullptr, WAIT_NS));
                        if (!ok) break;
                        have_k = true;
                        tc_fence_after();
                        scores(g, sn);
                    }
                }
                if (!ok) break;
                if (elect_one()) {  // these tiles are free once the products issued so far are complete
                    umma_commit(&v_empty[stage]);
                    if (j + 1 < n_kv) umma_commit(&k_empty[sn]);
                }
                __syncwarp();
                stage = sn;
                phase = pn;
            }
            // everything issued is complete before the block ends
            if (issued) {
                if (elect_one()) {
                    umma_commit(bar_drain);
                    mbar_wait(bar_drain, 0, nullptr, ok ? WAIT_NS : WAIT_NS / 5);
                }
                __syncwarp();
            }
            if (!ok) failed = true;
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        const int p = tid - 256;
        const int tpr = Q8 ? HSP / 16 : 8;  // threads a row (bf16: a 128-byte half of it)
        const int clear = it.kv_all - it.n + it.row0 / a.G;  // every row sees the keys up to here
        // this thread's rows of a unit are (p / tpr) + i * (128 / tpr)
        constexpr int PASSES = Q8 ? HSP / 16 : 8;
        uint4 buf[2][Q8 ? PASSES : 1];
        bool ok = true, bad_page = false, odd = false;
        int ids = -1;  // lane i < 8: the page of keys 16 i .. of the tile, or -1
        auto look_up = [&](int j) {
            const int pos = it.k_begin + j * KT + (lane & 7) * 16;
            ids = -1;
            if (pos < it.k_end) {
                ids = __ldg(a.p.table + it.b * a.p.ld_table + (pos >> a.p.page_log2));
                if (ids < 0 || ids >= a.p.n_pages) {
                    ids = -1;
                    bad_page = true;
                }
            }
        };
        // the token row of key r of tile j, or -1 where there is none to read
        auto token = [&](int j, int r) -> int64_t {
            const int id = __shfl_sync(0xffffffffu, ids, r >> 4);
            const int pos = it.k_begin + j * KT + r;
            if (id < 0 || pos >= it.k_end) return -1;
            return (((int64_t)id * a.p.Hkv + it.hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
        };
        auto load8 = [&](int j, const void* pages, uint4 (&to)[Q8 ? PASSES : 1]) {  // codes into registers
            if constexpr (Q8) {
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int64_t row = token(j, p / tpr + i * (128 / tpr));
                    const int d = (p % tpr) * 16;
                    to[i] = make_uint4(0, 0, 0, 0);
                    if (row >= 0 && d < hs) to[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(pages) + row * hs + d));
                }
            }
        };
        auto put8 = [&](uint8_t* tile, const uint4 (&from)[Q8 ? PASSES : 1]) {
            if constexpr (Q8) {
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int r = p / tpr + i * (128 / tpr), c = p % tpr, half = c >> 2;
                    const uint4 x = from[i];
                    const uint4 lo = make_uint4(codes_pair(x.x, 0), codes_pair(x.x, 1), codes_pair(x.y, 0), codes_pair(x.y, 1));
                    const uint4 hi = make_uint4(codes_pair(x.z, 0), codes_pair(x.z, 1), codes_pair(x.w, 0), codes_pair(x.w, 1));
                    // the two halves' threads store even and odd chunks in turn: no bank conflicts
                    *reinterpret_cast<uint4*>(tile + half * HALF + swizzled(r, 2 * (c & 3) + half)) = half ? hi : lo;
                    *reinterpret_cast<uint4*>(tile + half * HALF + swizzled(r, 2 * (c & 3) + (half ^ 1))) = half ? lo : hi;
                }
            }
        };
        auto copy16 = [&](int j, const void* pages, uint8_t* tile) {  // bf16 rows by cp.async
            const uint32_t base = saddr(tile);
#pragma unroll
            for (int h = 0; h < L::HALVES; ++h)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = p / 8 + i * 16, c = p % 8, d = h * 64 + c * 8;
                    const int64_t row = token(j, r);
                    const bool real = row >= 0 && d < hs;
                    cp_async16(base + h * HALF + swizzled(r, c), static_cast<const __nv_bfloat16*>(pages) + (real ? row * hs + d : 0), real);
                }
        };
        auto copy16_checked = [&](int j, const void* pages, uint8_t* tile) {  // V where some row must not see an odd value
            for (int h = 0; h < L::HALVES; ++h)
#pragma unroll 4
                for (int i = 0; i < 8; ++i) {
                    const int r = p / 8 + i * 16, c = p % 8, d = h * 64 + c * 8;
                    const int64_t row = token(j, r);
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row >= 0 && d < hs) x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages) + row * hs + d));
                    odd |= drop_odd2(x.x) | drop_odd2(x.y) | drop_odd2(x.z) | drop_odd2(x.w);
                    *reinterpret_cast<uint4*>(tile + h * HALF + swizzled(r, c)) = x;
                }
        };
        auto scales = [&](int j) {  // thread p: key p of the tile; and which groups of 16 lie on refused pages
            const int64_t row = token(j, p);
            if constexpr (Q8) {
                s_ks[(j & 3) * KT + p] = row >= 0 ? a.p.k_scale[row] * a.scale_log2 : 0.f;
                s_vs[(j & 3) * KT + p] = row >= 0 ? a.p.v_scale[row] : 0.f;
            }
            const unsigned bad = __ballot_sync(0xffffffffu, lane < 8 && ids < 0 && it.k_begin + j * KT + lane * 16 < it.k_end);
            if (p == 0) s_bad[j & 3] = bad;
            mbar_arrive(&c_full[j & 3]);
        };
        uint32_t stage = 0, phase = 0;
        // bf16: a unit (K or V of a tile) is announced when the same kind's unit LAG tiles later has been
        // issued. One tile less than the ring holds: that later unit waits only for products that
        // come before those that need this one.
        constexpr int LAG = L::STAGES - 1;
        auto landed = [&](uint64_t* full) {
            asm volatile("cp.async.wait_group %0;" ::"n"(2 * LAG) : "memory");
            fence_proxy_async_smem();
            mbar_arrive(&full[stage + 1 == L::STAGES ? 0 : stage + 1]);
        };
        if (n_kv > 0) {
            look_up(0);
            load8(0, a.p.k, buf[0]);
            load8(0, a.p.v, buf[1]);
        }
        for (int j = 0; j < n_kv && ok; ++j) {
            ok = mbar_wait(&k_empty[stage], phase ^ 1, nullptr, WAIT_NS);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            const int id_now = ids;
            if constexpr (Q8) {
                put8(sK + stage * L::TILE, buf[0]);
                scales(j);
                if (j + 1 < n_kv) {
                    look_up(j + 1);
                    load8(j + 1, a.p.k, buf[0]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&k_full[stage]);
            } else {
                copy16(j, a.p.k, sK + stage * L::TILE);
                asm volatile("cp.async.commit_group;" ::: "memory");
                scales(j);
                if (j >= LAG) landed(k_full);
            }
            ok = mbar_wait(&v_empty[stage], phase ^ 1, nullptr, WAIT_NS);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            if constexpr (Q8) {
                put8(sV + stage * L::TILE, buf[1]);
                if (j + 1 < n_kv) load8(j + 1, a.p.v, buf[1]);
                fence_proxy_async_smem();
                mbar_arrive(&v_full[stage]);
            } else {
                ids = id_now;
                if (it.k_begin + j * KT + KT - 1 > clear) {
                    copy16_checked(j, a.p.v, sV + stage * L::TILE);
                    if (odd) *s_odd = 1;
                } else {
                    copy16(j, a.p.v, sV + stage * L::TILE);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (j + 1 < n_kv) look_up(j + 1);
                if (j >= LAG) landed(v_full);
            }
            if (++stage == L::STAGES) stage = 0, phase ^= 1;
        }
        if constexpr (!Q8) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (ok && n_kv > 0) {
                fence_proxy_async_smem();
                for (int i = max(0, n_kv - LAG); i < n_kv; ++i) {
                    mbar_arrive(&k_full[i % L::STAGES]);
                    mbar_arrive(&v_full[i % L::STAGES]);
                }
            }
        }
        if (bad_page) report(a.err, GK_ERR_INDEX);
        if (!ok) failed = true;
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int g = warp >> 2, rr = (warp & 3) * 32 + lane;
        const int row = it.row0 + g * QT + rr, my_kt = it.tiles(g);
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_addr + 256 + g * HSP;
        const bool mine = row < it.R;
        const int query = row / a.G, h = it.hk * a.G + row % a.G;
        if (my_kt > 0) {  // this thread's row of Q
            const __nv_bfloat16* src = a.q + (int64_t)(it.s0 + query) * a.ldq + h * hs;
#pragma unroll
            for (int c = 0; c < HSP / 8; ++c) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (mine && c * 8 < hs) x = __ldg(reinterpret_cast<const uint4*>(src + c * 8));
                *reinterpret_cast<uint4*>(sQ + g * L::TILE + (c >> 3) * HALF + swizzled(rr, c & 7)) = x;
            }
            fence_proxy_async_smem();
            mbar_arrive(&q_full[g]);
        }
        const int last = mine ? min(it.last(row, a.G), it.k_end - 1) : -1;
        const float sl2 = a.scale_log2;
        float m_ref = -INFINITY, l = 0.f;
        for (int j = 0; j < my_kt; ++j) {
            if (!__all_sync(0xffffffffu, mbar_wait(&c_full[j & 3], (j >> 2) & 1, nullptr, WAIT_NS) &&
                                             mbar_wait(&bar_s[g], j & 1, nullptr, WAIT_NS))) {
                failed = true;
                break;
            }
            tc_fence_after();
            uint32_t sv[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_nowait(lane_addr + g * 128 + c * 32, sv[c]);
            tmem_wait_ld_only();
#pragma unroll
            for (int c = 0; c < 4; ++c) reg_fence32(sv[c]);
            const float4* ks4 = reinterpret_cast<const float4*>(s_ks + (j & 3) * KT);
            const float4* vs4 = reinterpret_cast<const float4*>(s_vs + (j & 3) * KT);
            if constexpr (Q8) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 k4 = ks4[c * 8 + i];
                        sv[c][4 * i] = __float_as_uint(__uint_as_float(sv[c][4 * i]) * k4.x);
                        sv[c][4 * i + 1] = __float_as_uint(__uint_as_float(sv[c][4 * i + 1]) * k4.y);
                        sv[c][4 * i + 2] = __float_as_uint(__uint_as_float(sv[c][4 * i + 2]) * k4.z);
                        sv[c][4 * i + 3] = __float_as_uint(__uint_as_float(sv[c][4 * i + 3]) * k4.w);
                    }
            }
            const int lim = last - (it.k_begin + j * KT) + 1;  // keys i < lim are seen
            const uint32_t bad = s_bad[j & 3];
            const bool part = __any_sync(0xffffffffu, lim < KT) || bad;
            if (part) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c * 32 + i >= lim || (bad >> (c * 2 + (i >> 4)) & 1)) sv[c][i] = 0xff800000u;
            }
            float mx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = __uint_as_float(sv[0][e]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(sv[c][i]));
            const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
            const float m_new = fmaxf(m_ref, Q8 ? mt : mt * sl2);
            float corr = 1.f;
            const bool rescale = m_new > m_ref + 8.f;
            if (rescale) {
                corr = ex2_hw(m_ref - m_new);  // 0 while the row was empty
                l *= corr;
                m_ref = m_new;
            }
            const float ref = m_ref == -INFINITY ? 0.f : m_ref;  // (a row that has seen nothing yet)
            float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t pw[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float s = __uint_as_float(sv[c][4 * e + x]);
                        p[x] = ex2_hw(Q8 ? s - ref : fmaf(s, sl2, -ref));
                        ps[x] += p[x];
                    }
                    if constexpr (Q8) {
                        const float4 v4 = vs4[c * 8 + e];
                        const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x)  // (an unseen key's scale may be anything)
                            p[x] = part && sv[c][4 * e + x] == 0xff800000u ? 0.f : p[x] * v[x];
                    }
                    pw[2 * e] = pack2(p[0], p[1]);
                    pw[2 * e + 1] = pack2(p[2], p[3]);
                }
                tmem_st16(lane_addr + g * 128 + c * 16, pw);
            }
            l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
            if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
                for (int c = 0; c < HSP / 32; ++c) {
                    uint32_t ov[32];
                    tmem_ld32_nowait(o_addr + c * 32, ov);
                    tmem_wait_ld_only();
                    reg_fence32(ov);
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * corr);
                    tmem_st32(o_addr + c * 32, ov);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar_p[g]);
        }
        if (!failed && my_kt > 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bar_o[g], 0, nullptr, WAIT_NS))) failed = true;
            tc_fence_after();
        }
        if (!failed) {
            const int64_t out = (int64_t)(it.s0 + query) * a.H + h;
            const float inv = a.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const int odd_from = !Q8 && *s_odd ? max(it.k_begin, it.kv_all - it.n + it.row0 / a.G + 1) : 0x7fffffff;
#pragma unroll
            for (int c = 0; c < HSP / 32; ++c) {
                uint32_t ov[32];
                if (my_kt > 0) {
                    tmem_ld32_nowait(o_addr + c * 32, ov);
                    tmem_wait_ld_only();
                    reg_fence32(ov);
                }
                if (mine) {
#pragma unroll
                for (int i = 0; i < 32; ++i) ov[i] = my_kt > 0 && l != 0.f ? __float_as_uint(__uint_as_float(ov[i]) * inv) : 0u;
                for (int j = odd_from; j <= last; ++j) {  // rare: infinities and NaN that were taken out of V, where they are seen
                    const int id = a.p.table[it.b * a.p.ld_table + (j >> a.p.page_log2)];
                    if (id < 0 || id >= a.p.n_pages) continue;
                    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.p.v) +
                                               ((((int64_t)id * a.p.Hkv + it.hk) << a.p.page_log2) + (j & ((1 << a.p.page_log2) - 1))) * hs + c * 32;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float y = c * 32 + i < hs ? __bfloat162float(src[i]) : 0.f;
                        if (!isfinite(y)) ov[i] = __float_as_uint(__uint_as_float(ov[i]) + y);
                    }
                }
                if (a.splits > 1) {
                    float* dst = a.part_o + (out * a.splits + it.split) * hs + c * 32;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (c * 32 + i < hs) *reinterpret_cast<uint4*>(dst + i) = make_uint4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
                } else {
                    __nv_bfloat16* dst = a.y + (int64_t)(it.s0 + query) * a.ldy + h * hs + c * 32;
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (c * 32 + i < hs)
                            *reinterpret_cast<uint4*>(dst + i) =
                                make_uint4(pack2(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1])), pack2(__uint_as_float(ov[i + 2]), __uint_as_float(ov[i + 3])),
                                           pack2(__uint_as_float(ov[i + 4]), __uint_as_float(ov[i + 5])), pack2(__uint_as_float(ov[i + 6]), __uint_as_float(ov[i + 7])));
                }
                }
                __syncwarp();
            }
            if (mine) {
                if (a.splits > 1) a.part_ml[out * a.splits + it.split] = make_float2(m_ref, l);
                else if (a.lse) a.lse[out] = l == 0.f ? -INFINITY : ((m_ref == -INFINITY ? 0.f : m_ref) + log2f(l)) * 0.6931471805599453f;
            }
        }
    }
    if (failed) report(a.err, GK_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HSP, bool Q8>
gk_status tiles(gk_ctx* ctx, const AttnArgs& a) {
    if (cudaFuncSetAttribute(attn_tiles_kernel<HSP, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<HSP>::BYTES) !=
        cudaSuccess) {
        cudaGetLastError();
        return fail(ctx, GK_ERR_CUDA, "gk_paged_attn: shared memory");
    }
    const int64_t pairs = cdiv((int64_t)a.max_q * a.G, 2 * QT);
    return launch_dependent(ctx, "paged_attn_tiles", attn_tiles_kernel<HSP, Q8>,
                            dim3((unsigned)(pairs * a.splits), (unsigned)a.p.Hkv, (unsigned)a.B), dim3(THREADS), Layout<HSP>::BYTES, 1, a);
}

}  // namespace

gk_status launch_attn_tiles(gk_ctx* ctx, const AttnArgs& a) {
    if (a.p.hs <= 64) return a.p.k_scale ? tiles<64, true>(ctx, a) : tiles<64, false>(ctx, a);
    return a.p.k_scale ? tiles<128, true>(ctx, a) : tiles<128, false>(ctx, a);
}

}  // namespace gk
