// Attention of chunks of new tokens over the paged cache, on the tensor cores (tcgen05).
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// A block takes two tiles of 128 query rows of one key / value head (the H / Hkv heads that share it
// side by side: row i is query i / G, head i % G, so its keys are read once for all of them) and
// walks the keys in tiles of 128:
//   S = Q K^T   (M = 128 rows, N = 128 keys, K = head size) into tensor memory;
//   softmax     a thread per row: P = 2^(s - m) with s in powers of two, as bf16 over S in tensor
//               memory (an operand of the product has 16 bits; 2^-8 of a weight at most, as y's own
//               rounding, where a second part would double the products; sums of weights stay float32);
//               the reference m moves (and O is rescaled there) only when the row's maximum passes it
//               by more than 8;
//   O += P V    (N = head size, K = 128 keys), accumulated in tensor memory.
// Head sizes up to 64 leave room there for P beside S: the next S is computed as soon as the scores of
// this one have been read, under the softmax. With 128 P lies over S, and the next S waits for P V.
// The two tiles take turns: while one group of four warps turns its S into P, the tensor core
// computes the other's products. Warp 8 sends for the keys by TMA, a box per page (pages lie anywhere).
// 8-bit codes become bf16 (exactly) first: in one pass into the workspace, if it has room (for all heads or a few
// at a time) and heads are wide or rows many; else on the way, by warps 8-11. Codes carry no scale into the products: the key's scale multiplies the score and
// the value's scale the weight, both from shared memory. Warp 12 issues the MMAs.
// K and V have rings of their own (a K tile is free once both S are there, a V tile after both
// products), of three tiles each for head sizes up to 64 and two for 128.
// Registers: 512 threads at 128; the softmax warpgroups take 184 each, the copying one 96, the MMA warp's
// 48 (where the copying one unpacks codes: 176, 104, 48).
// All mbarrier waits are bounded (timeout -> GK_ERR_TIMEOUT in the error word).
// Measured: two chunks of up to 2048 tokens behind 16384 keys, 32 heads over 8 of 128: bf16 pages 494 us, 1.07
// PFLOP/s (0.55 of a dense product); 8-bit ones 670 us with the pass that expands them (1980 unpacked on the way):
// the softmax warps bound both, by a thread's 128 exponentials, maxima and packing a tile, for 8 bits by two more
// products a score. Three chunks of up to 1000 over 8100 keys, 12 heads of 64: 85 us (half the products a tile for
// the same softmax). Key tiles that two groups of blocks read side by side come from L2.
#include <algorithm>
#include <type_traits>

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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
// Codes 0 and 1 (or 2 and 3) of a word as a pair of bf16: 128 + the low seven bits, less 128 or 256.
__device__ __forceinline__ uint32_t codes_pair(const CodeMasks& k, uint32_t w, int second) {
    const uint32_t x = __byte_perm(w, 0, second ? 0x4342 : 0x4140);
    const uint32_t a = and_or(x, k.low7, k.bf16_128), b = and_or(x, k.sign, k.bf16_128);
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ bool drop_odd2(uint32_t& x) {  // infinities and NaN of a bf16 pair become zeros
    const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
    if (lo) x &= 0xffff0000u;
    if (hi) x &= 0x0000ffffu;
    return lo || hi;
}

// Two float32 operations an instruction: (x, y) = (x s + t, y s + t); (x, y) += (a, b); (x, y) *= (a, b).
__device__ __forceinline__ void fma2(uint32_t& x, uint32_t& y, float s, float t) {
    asm("{\n\t.reg .b64 v, a, b;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %3};\n\t"
        "fma.rn.f32x2 v, v, a, b;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(s), "f"(t));
}
__device__ __forceinline__ void add2(uint32_t& x, uint32_t& y, float a, float b) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void mul2(uint32_t& x, uint32_t& y, float a, float b) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tmul.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(a), "f"(b));
}

__device__ __forceinline__ uint32_t test_phase(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(saddr(bar)), "r"(parity)
        : "memory");
    return ok;
}
// Wait for a phase: polled at first (try_wait suspends the thread, and its wake-up takes longer than most
// of the waits here), then bounded by the clock.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint64_t limit) {
#pragma unroll 1
    for (int i = 0; i < 4096; ++i)
        if (test_phase(bar, parity)) return true;
    return mbar_wait(bar, parity, nullptr, limit);
}
// Several at once: even a test of a completed phase takes hundreds of cycles behind the softmax warps' traffic
// with the tensor memory, so the tests are sent together. (b and c only where asked.)
__device__ __forceinline__ bool wait_phases(uint64_t* a, uint32_t pa, bool has_b, uint64_t* b, uint32_t pb, bool has_c, uint64_t* c,
                                            uint32_t pc, uint64_t limit) {
#pragma unroll 1
    for (int i = 0; i < 4096; ++i) {
        const uint32_t x = test_phase(a, pa), y = test_phase(has_b ? b : a, has_b ? pb : pa);
        const uint32_t z = test_phase(has_c ? c : a, has_c ? pc : pa);
        if (x & y & z) return true;
    }
    return mbar_wait(a, pa, nullptr, limit) && (!has_b || mbar_wait(b, pb, nullptr, limit)) && (!has_c || mbar_wait(c, pc, nullptr, limit));
}

// Rows that a sequence takes per head once expanded: whole tiles of keys.
__device__ __forceinline__ int expanded_rows(const Pages& p, int b) {
    return (min(max(__ldg(p.kv_len + b), 0), p.capacity) + KT - 1) / KT * KT;
}

// What one block works on.
struct Item {
    int b, hk, split, s0, n, R, row0;  // rows row0 .. row0 + 255 of R
    int kv_all, kv, k_begin, k_end;    // keys k_begin .. k_end - 1 of this piece
    int t0, t1;                        // key tiles that some row of each query tile sees
    __device__ __forceinline__ int tiles(int g) const { return g ? t1 : t0; }
    __device__ __forceinline__ int last(int row, int G) const { return min(kv - 1, kv_all - n + row / G); }
};

// Where the keys come from: bf16 pages, by TMA; 8-bit pages, unpacked by warps 8-11; or 8-bit codes
// already laid out as bf16 in the workspace (expand_kernel), by TMA.
enum { PAGES16, PAGES8, EXPANDED };
constexpr uint32_t ODD_SCALES = 1u << 31;  // beside a tile's refused groups: some value's scale is not finite

template <int HSP, int FROM>
__global__ void __launch_bounds__(THREADS, 1)
    attn_tiles_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    constexpr bool Q8 = FROM != PAGES16;
    using L = Layout<HSP>;
    constexpr bool EARLY = HSP == 64;  // the next S before P V
    constexpr uint32_t P_AT = EARLY ? 384 : 0, P_STEP = EARLY ? 64 : 128;  // tensor memory columns of P_g
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;           // [2 tiles][halves]
    uint8_t* sK = smem + L::K;    // [stages][halves]
    uint8_t* sV = smem + L::V;
    float* s_ks = reinterpret_cast<float*>(smem + L::SCALES);  // [4][128]: scale of the scores per key
    float* s_vs = s_ks + 4 * KT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t* q_full = bars;         // [2] tile's rows are there (one arrival per warp)
    uint64_t* k_full = bars + 2;     // [3]
    uint64_t* k_empty = bars + 5;    // [3]
    uint64_t* v_full = bars + 8;     // [3]
    uint64_t* v_empty = bars + 11;   // [3]
    uint64_t* c_full = bars + 14;    // [4] the tile's scales and refused pages are there
    uint64_t* bar_s = bars + 18;     // [2] S_g is there
    uint64_t* bar_p = bars + 20;     // [2] P_g is there (one arrival per warp)
    uint64_t* bar_o = bars + 22;     // [2] O_g is complete
    uint64_t* bar_drain = bars + 24;
    volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(bars + 25);  // [4] 16-key groups on refused pages
    volatile int* s_odd = reinterpret_cast<volatile int*>(bars + 27);  // where values were taken out of V first
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 28);
    uint64_t* s_free = bars + 29;    // [2] early S: S_g has been read (one arrival per warp)
    uint64_t* bar_pv = bars + 31;    // [2] early S: P_g V is complete
    wait_for_earlier_kernels();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Item it;
    {
        const int pairs = gridDim.x / a.splits;
        // the last rows see the most keys: first; and pairs that read the same keys next to each other
        const int pair = pairs - 1 - blockIdx.x % pairs;
        it.split = blockIdx.x / pairs;
        it.b = blockIdx.z;
        it.hk = a.head0 + blockIdx.y;
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
            mbar_init(&q_full[i], 4);
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_p[i], 4);
            mbar_init(&bar_o[i], 1);
            mbar_init(&s_free[i], 4);
            mbar_init(&bar_pv[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&c_full[i], 1);
        mbar_init(bar_drain, 1);
        *s_odd = 0x7fffffff;
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
            if (n_kv > 0) ok = __all_sync(0xffffffffu, wait_phase(&k_full[0], 0, WAIT_NS));
            for (int g = 0; g < 2 && ok; ++g)
                if (it.tiles(g) > 0) {
                    ok = __all_sync(0xffffffffu, wait_phase(&q_full[g], 0, WAIT_NS));
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
                const bool next_a = j + 1 < it.t0, next_b = j + 1 < it.t1;
                if constexpr (EARLY) {
                    if (next_a || next_b) {
                        ok = __all_sync(0xffffffffu, wait_phases(&k_full[sn], pn, next_a, &s_free[0], j & 1, next_b, &s_free[1], j & 1,
                                                                 WAIT_NS));
                        if (!ok) break;
                        tc_fence_after();
                        if (next_a) scores(0, sn);
                        if (next_b) scores(1, sn);
                        if (elect_one()) umma_commit(&k_empty[sn]);
                        __syncwarp();
                    }
                }
                bool first = true;
                for (int g = 0; g < 2 && ok; ++g) {
                    if (j >= it.tiles(g)) continue;
                    // the first group's wait takes V, and the next K, with it
                    ok = __all_sync(0xffffffffu, wait_phases(&bar_p[g], j & 1, first, &v_full[stage], phase,
                                                             !EARLY && first && j + 1 < n_kv, &k_full[sn], pn, WAIT_NS));
                    if (!ok) break;
                    first = false;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            umma_bf16_ts(tmem + 256 + g * HSP, tmem + P_AT + g * P_STEP + kk * 8, desc_add(v_d, stage * L::TILE + kk * 2048),
                                         id_o, (j > 0 || kk > 0) ? 1u : 0u);
                        if (EARLY) umma_commit(&bar_pv[g]);
                        if (j == it.tiles(g) - 1) umma_commit(&bar_o[g]);
                    }
                    __syncwarp();
                    if (!EARLY && j + 1 < it.tiles(g)) scores(g, sn);
                }
                if (!ok) break;
                if (elect_one()) {  // these tiles are free once the products issued so far are complete
                    umma_commit(&v_empty[stage]);
                    if (!EARLY && j + 1 < n_kv) umma_commit(&k_empty[sn]);
                }
                __syncwarp();
                stage = sn;
                phase = pn;
            }
            // everything issued is complete before the block ends
            if (issued) {
                if (elect_one()) {
                    umma_commit(bar_drain);
                    wait_phase(bar_drain, 0, ok ? WAIT_NS : WAIT_NS / 5);
                }
                __syncwarp();
            }
            if (!ok) failed = true;
        }
    } else if (warp >= 8) {
        if constexpr (FROM == PAGES8) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        const int row_bytes = FROM == PAGES8 ? hs : 2 * hs;
        const int clear = it.kv_all - it.n + it.row0 / a.G;  // every row sees the keys up to here
        bool ok = true, bad_page = false, odd = false, odd_tile = false;
        int ids = 0;  // lane i < 8: the page of keys 16 i .. of the tile
        bool bad = false;
        auto look_up = [&](int j) {
            const int pos = it.k_begin + j * KT + (lane & 7) * 16;
            ids = 0;
            bad = false;
            if (pos < it.k_end) {
                ids = __ldg(a.p.table + it.b * a.p.ld_table + (pos >> a.p.page_log2));
                if (ids < 0 || ids >= a.p.n_pages) {
                    ids = 0;
                    bad = bad_page = true;
                }
            }
        };
        // keys of a group of 16 lie together in a page: the first one's row
        auto group_row = [&](int j, int grp) -> int64_t {
            const int id = __shfl_sync(0xffffffffu, ids, grp);
            const int pos = it.k_begin + j * KT + grp * 16;
            return (((int64_t)id * a.p.Hkv + it.hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
        };
        // the scales of tile j, four keys a lane, read one tile ahead; then they and the refused pages are
        // left for the softmax
        float4 ks_next = make_float4(0.f, 0.f, 0.f, 0.f), vs_next = ks_next;
        auto load_scales = [&](int j) {
            if constexpr (Q8) {
                const int64_t row = group_row(j, lane >> 2) + (lane & 3) * 4;
                ks_next = vs_next = make_float4(0.f, 0.f, 0.f, 0.f);
                if (lane * 4 < it.k_end - (it.k_begin + j * KT)) {  // (a page's rows past the end exist)
                    ks_next = __ldg(reinterpret_cast<const float4*>(a.p.k_scale + row));
                    vs_next = __ldg(reinterpret_cast<const float4*>(a.p.v_scale + row));
                }
            }
        };
        auto leave_scales = [&](int j, unsigned refused) {
            if constexpr (Q8) {
                const float c = a.scale_log2;
                reinterpret_cast<float4*>(s_ks + (j & 3) * KT)[lane] = make_float4(ks_next.x * c, ks_next.y * c, ks_next.z * c, ks_next.w * c);
                reinterpret_cast<float4*>(s_vs + (j & 3) * KT)[lane] = vs_next;
            }
            const bool odd = !(isfinite(vs_next.x) && isfinite(vs_next.y) && isfinite(vs_next.z) && isfinite(vs_next.w));
            if (Q8 && __any_sync(0xffffffffu, odd)) refused |= ODD_SCALES;
            if (lane == 0) s_bad[j & 3] = refused;
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[j & 3]);
        };
        if constexpr (FROM != PAGES8) {
            // Warp 8 sends for the tiles: whole boxes of a page's rows (EXPANDED: the tile's 128 rows) by TMA.
            // Tiles of V that hold keys some row must not see, or past the end, or on refused pages, it copies
            // itself: what is not finite or not there becomes zeros (and is put back at the end for the rows that see
            // it, from the first key on of the first tile that lost any). EXPANDED tiles are finite, and zeros past the
            // end. (Chunks of 1000 take 85.2 us so, 86.7 with only the keys cleared that some row must not see.)
            const int box = FROM == EXPANDED ? KT : min(KT, 1 << a.p.page_log2);
            int64_t base_row = 0;  // EXPANDED: this head's first row
            if constexpr (FROM == EXPANDED) {
                int64_t sum = 0;
                for (int i = lane; i < it.b; i += 32) sum += expanded_rows(a.p, i);
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                base_row = sum * a.heads + (int64_t)(it.hk - a.head0) * expanded_rows(a.p, it.b) + it.k_begin;
            }
            int in_flight_k = -1, in_flight_v = -1;
            if (warp == 8 && n_kv > 0) {
                look_up(0);
                load_scales(0);
            }
            for (int j = 0; warp == 8 && j < n_kv; ++j) {
                const uint32_t stage = j % L::STAGES, phase = (j / L::STAGES) & 1;
                const unsigned refused = __ballot_sync(0xffffffffu, lane < 8 && bad);
                const bool checked = FROM == PAGES16 && (refused || it.k_begin + j * KT + KT - 1 > min(clear, it.k_end - 1));
                const int left = it.k_end - (it.k_begin + j * KT);  // keys r < left exist
                const int row = (int)(FROM == EXPANDED ? base_row + (int64_t)j * KT : group_row(j, (lane & 7) * box >> 4));
                ok = __all_sync(0xffffffffu, wait_phase(&k_empty[stage], phase ^ 1, WAIT_NS));
                if (!ok) break;
                leave_scales(j, refused);
                auto send = [&](const CUtensorMap* map, uint8_t* tile, uint64_t* full) {
                    if (lane == 0) mbar_expect_tx(full, L::TILE);
                    __syncwarp();
                    if (lane < KT / box)
                        for (int h = 0; h < L::HALVES; ++h) tma_load_2d(map, full, tile + h * HALF + lane * box * 128, h * 64, row);
                    __syncwarp();
                };
                send(&tm_k, sK + stage * L::TILE, &k_full[stage]);
                in_flight_k = j;
                ok = __all_sync(0xffffffffu, wait_phase(&v_empty[stage], phase ^ 1, WAIT_NS));
                if (!ok) break;
                if (!checked) {
                    send(&tm_v, sV + stage * L::TILE, &v_full[stage]);
                } else {
                    uint8_t* tile = sV + stage * L::TILE;
                    for (int grp = 0; grp < 8; ++grp) {
                        const char* src = static_cast<const char*>(a.p.v) + group_row(j, grp) * row_bytes;
                        const bool none = refused >> grp & 1;
#pragma unroll
                        for (int i = 0; i < 4 * L::HALVES; ++i) {
                            const int r = i / L::HALVES * 4 + lane / 8, c = (i % L::HALVES) * 8 + lane % 8;
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (!none && grp * 16 + r < left && c * 8 < hs) x = __ldg(reinterpret_cast<const uint4*>(src + r * row_bytes + c * 16));
                            odd |= drop_odd2(x.x) | drop_odd2(x.y) | drop_odd2(x.z) | drop_odd2(x.w);
                            *reinterpret_cast<uint4*>(tile + (c >> 3) * HALF + swizzled(grp * 16 + r, c & 7)) = x;
                        }
                    }
                    if (!odd_tile && __any_sync(0xffffffffu, odd)) {
                        odd_tile = true;
                        if (lane == 0) *s_odd = it.k_begin + j * KT;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_full[stage]);
                }
                in_flight_v = j;
                if (j + 1 < n_kv) {
                    look_up(j + 1);
                    load_scales(j + 1);
                }
            }
            if (!ok && warp == 8) {  // the copies in flight land before the block ends
                for (int j = max(0, in_flight_k - L::STAGES + 1); j <= in_flight_k; ++j) wait_phase(&k_full[j % L::STAGES], (j / L::STAGES) & 1, WAIT_NS / 5);
                for (int j = max(0, in_flight_v - L::STAGES + 1); j <= in_flight_v; ++j) wait_phase(&v_full[j % L::STAGES], (j / L::STAGES) & 1, WAIT_NS / 5);
            }
        } else {
            // each warp brings whole tiles: warps 8 and 10 those of K in turn, 9 and 11 those of V
            const bool is_v = warp & 1;
            const char* pages = static_cast<const char*>(is_v ? a.p.v : a.p.k);
            uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
            int j = (warp - 8) >> 1;
            if (j < n_kv) {
                look_up(j);
                if (!is_v) load_scales(j);
            }
            for (; j < n_kv; j += 2) {
                const uint32_t stage = j % L::STAGES, phase = (j / L::STAGES) & 1;
                const unsigned refused = __ballot_sync(0xffffffffu, lane < 8 && bad);
                // (K too waits for the V tile that far back: its scales' places have been read then)
                ok = __all_sync(0xffffffffu, wait_phase(&empty[stage], phase ^ 1, WAIT_NS) && (is_v || wait_phase(&v_empty[stage], phase ^ 1, WAIT_NS)));
                if (!ok) break;
                uint8_t* tile = (is_v ? sV : sK) + stage * L::TILE;
                if (!is_v) leave_scales(j, refused);
                // lane: 16 codes of a row, 128 / HSP * 4 rows a pass; loads run AHEAD passes ahead (rows of 128: eight 429 us
                // against 568 with four, 48 sequences of 64 rows; of 64: 98 against 88)
                constexpr int TPR = HSP / 16, RPP = 32 / TPR, PASSES = KT / RPP;
                const int c = lane % TPR, half = c >> 2, r_in = lane / TPR;
                const int at = min(c * 16, row_bytes - 16);  // (dims past hs: Q is zero there, and they are not stored)
                constexpr int AHEAD = HSP == 64 ? 4 : 8;
                uint4 x[AHEAD];
                auto load = [&](int i) {
                    const int r = i * RPP + r_in;
                    const int64_t row = group_row(j, (i * RPP) >> 4) + (r & 15);
                    uint4 v;  // (volatile: kept this far ahead of its use)
                    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "l"(pages + row * row_bytes + at));
                    return v;
                };
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) x[i] = load(i);
#pragma unroll AHEAD
                for (int i = 0; i < PASSES; ++i) {
                    const uint4 now = x[i & (AHEAD - 1)];
                    if (i + AHEAD < PASSES) x[i & (AHEAD - 1)] = load(i + AHEAD);
                    const int r = i * RPP + r_in;
                    const uint4 lo = make_uint4(codes_pair(a.masks, now.x, 0), codes_pair(a.masks, now.x, 1), codes_pair(a.masks, now.y, 0), codes_pair(a.masks, now.y, 1));
                    const uint4 hi = make_uint4(codes_pair(a.masks, now.z, 0), codes_pair(a.masks, now.z, 1), codes_pair(a.masks, now.w, 0), codes_pair(a.masks, now.w, 1));
                    // the two halves' threads store even and odd chunks in turn: no bank conflicts
                    *reinterpret_cast<uint4*>(tile + half * HALF + swizzled(r, 2 * (c & 3) + half)) = half ? hi : lo;
                    *reinterpret_cast<uint4*>(tile + half * HALF + swizzled(r, 2 * (c & 3) + (half ^ 1))) = half ? lo : hi;
                }
                if (j + 2 < n_kv) {
                    look_up(j + 2);
                    if (!is_v) load_scales(j + 2);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[stage]);
            }
        }
        if (bad_page) report(a.err, GK_ERR_INDEX);
        if (!ok) failed = true;
    } else {
        if constexpr (FROM == PAGES8) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[g]);
        }
        const int last = mine ? min(it.last(row, a.G), it.k_end - 1) : -1;
        const float sl2 = a.scale_log2;
        float m_ref = -INFINITY, l = 0.f;
        for (int j = 0; j < my_kt; ++j) {
            if (!__all_sync(0xffffffffu, wait_phases(&bar_s[g], j & 1, true, &c_full[j & 3], (j >> 2) & 1, false, nullptr, 0, WAIT_NS))) {
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
            if constexpr (EARLY) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[g]);
            }
            const int lim = last - (it.k_begin + j * KT) + 1;  // keys i < lim are seen
            const uint32_t bad = s_bad[j & 3];
            const bool part = __any_sync(0xffffffffu, lim < KT) || (bad & 0xff);
            if constexpr (Q8) {
                const float4* ks4 = reinterpret_cast<const float4*>(s_ks + (j & 3) * KT);
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 k4 = ks4[c * 8 + i];
                        mul2(sv[c][4 * i], sv[c][4 * i + 1], k4.x, k4.y);
                        mul2(sv[c][4 * i + 2], sv[c][4 * i + 3], k4.z, k4.w);
                    }
            }
            if (part) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c * 32 + i >= lim || (bad >> (c * 2 + (i >> 4)) & 1)) sv[c][i] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(sv[0][e]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) mx[i & 3] = fmaxf(fmaxf(mx[i & 3], __uint_as_float(sv[c][2 * i])), __uint_as_float(sv[c][2 * i + 1]));
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float m_new = fmaxf(m_ref, Q8 ? mt : mt * sl2);
            float corr = 1.f;
            const bool rescale = m_new > m_ref + 8.f;
            if (rescale) {
                corr = ex2_hw(m_ref - m_new);  // 0 while the row was empty
                l *= corr;
                m_ref = m_new;
            }
            if constexpr (EARLY) {  // P and O are free once the products before are complete
                if (j > 0 && !__all_sync(0xffffffffu, wait_phase(&bar_pv[g], (j - 1) & 1, WAIT_NS))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
            }
            const float ref = m_ref == -INFINITY ? 0.f : m_ref;  // (a row that has seen nothing yet)
            uint32_t ps[4] = {0, 0, 0, 0};  // two pairs of running sums
            const float4* vs4 = reinterpret_cast<const float4*>(s_vs + (j & 3) * KT);
            // weights of the row's 128 keys into tensor memory; `odd`: a value's scale is not finite, and keys that are
            // not seen must be kept from it
            auto weights = [&](auto odd) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pw[16];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t* w = &sv[c][4 * e];
                        const float one = Q8 ? 1.f : sl2;
                        fma2(w[0], w[1], one, -ref);
                        fma2(w[2], w[3], one, -ref);
                        float p[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) p[x] = ex2_hw(__uint_as_float(w[x]));
                        add2(ps[0], ps[1], p[0], p[1]);
                        add2(ps[2], ps[3], p[2], p[3]);
                        if constexpr (Q8) {
                            const float4 v4 = vs4[c * 8 + e];
                            uint32_t y[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) y[x] = __float_as_uint(p[x]);
                            mul2(y[0], y[1], v4.x, v4.y);
                            mul2(y[2], y[3], v4.z, v4.w);
#pragma unroll
                            for (int x = 0; x < 4; ++x) p[x] = decltype(odd)::value && w[x] == 0xff800000u ? 0.f : __uint_as_float(y[x]);
                        }
                        pw[2 * e] = pack2(p[0], p[1]);
                        pw[2 * e + 1] = pack2(p[2], p[3]);
                    }
                    tmem_st16(lane_addr + P_AT + g * P_STEP + c * 16, pw);
                }
            };
            if (Q8 && (bad & ODD_SCALES)) weights(std::true_type{});
            else weights(std::false_type{});
            l += (__uint_as_float(ps[0]) + __uint_as_float(ps[1])) + (__uint_as_float(ps[2]) + __uint_as_float(ps[3]));
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_p[g]);
        }
        if (!failed && my_kt > 0) {
            if (!__all_sync(0xffffffffu, wait_phase(&bar_o[g], 0, WAIT_NS))) failed = true;
            tc_fence_after();
        }
        if (!failed) {
            const int64_t out = (int64_t)(it.s0 + query) * a.H + h;
            const float inv = a.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const int odd_from = Q8 ? 0x7fffffff : *s_odd;
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
                // rare: infinities and NaN that were taken out of V, where they are seen (twice in tiles that kept theirs)
                for (int j = odd_from; j <= last; ++j) {
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

// The codes of every sequence's heads head0 .. as bf16 rows, heads apart: sequence b's head head0 + h at row
// (sum of expanded_rows before b) * heads + h * expanded_rows(b), zeros past its end and on refused pages.
// One pass, a block per 64 positions of a head.
__global__ void __launch_bounds__(256) expand_kernel(const AttnArgs a, __nv_bfloat16* k_out, __nv_bfloat16* v_out) {
    wait_for_earlier_kernels();
    const int b = blockIdx.z, hk = a.head0 + blockIdx.y, len = expanded_rows(a.p, b), p0 = blockIdx.x * 64;
    if (p0 >= len) return;
    const int lane = threadIdx.x & 31, kv = min(max(a.p.kv_len[b], 0), a.p.capacity), hs = a.p.hs;
    int64_t base = 0;
    for (int i = lane; i < b; i += 32) base += expanded_rows(a.p, i);
    for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
    base = base * a.heads + (int64_t)blockIdx.y * len;
    const int per = hs >> 4;
    for (int i = threadIdx.x; i < 64 * per; i += 256) {
        const int pos = p0 + i / per, d = (i % per) * 16;
        const int id = pos < kv ? __ldg(a.p.table + b * a.p.ld_table + (pos >> a.p.page_log2)) : -1;
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (id >= 0 && id < a.p.n_pages) {
            const int64_t at = ((((int64_t)id * a.p.Hkv + hk) << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1))) * hs + d;
            x[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.p.k) + at));
            x[1] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.p.v) + at));
        }
        const int64_t out = (base + pos) * hs + d;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint4* dst = reinterpret_cast<uint4*>((e ? v_out : k_out) + out);
            dst[0] = make_uint4(codes_pair(a.masks, x[e].x, 0), codes_pair(a.masks, x[e].x, 1), codes_pair(a.masks, x[e].y, 0), codes_pair(a.masks, x[e].y, 1));
            dst[1] = make_uint4(codes_pair(a.masks, x[e].z, 0), codes_pair(a.masks, x[e].z, 1), codes_pair(a.masks, x[e].w, 0), codes_pair(a.masks, x[e].w, 1));
        }
    }
}

template <int HSP, int FROM>
gk_status tiles(gk_ctx* ctx, const AttnArgs& a, const __nv_bfloat16* k, const __nv_bfloat16* v, int64_t rows, int box) {
    GK_TRY((allow_shared<attn_tiles_kernel<HSP, FROM>>(ctx, "gk_paged_attn", Layout<HSP>::BYTES)));
    CUtensorMap mk{}, mv{};
    if (FROM != PAGES8)
        GK_REQUIRE(ctx, make_map(&mk, k, a.p.hs, rows, a.p.hs, box) && make_map(&mv, v, a.p.hs, rows, a.p.hs, box), GK_ERR_CUDA,
                   "gk_paged_attn: tensor map");
    const int64_t pairs = cdiv((int64_t)a.max_q * a.G, 2 * QT);
    return launch_dependent(ctx, "paged_attn_tiles", attn_tiles_kernel<HSP, FROM>,
                            dim3((unsigned)(pairs * a.splits), (unsigned)a.heads, (unsigned)a.B), dim3(THREADS), Layout<HSP>::BYTES, 1, a,
                            mk, mv);
}

}  // namespace

gk_status launch_attn_tiles(gk_ctx* ctx, const AttnArgs& a) {
    const bool small = a.p.hs <= 64;
    if (a.expanded_k) {
        const int64_t rows = a.expanded_rows;
        GK_TRY(launch_dependent(ctx, "paged_attn_expand", expand_kernel, dim3((unsigned)cdiv(a.p.capacity, 128) * 2, (unsigned)a.heads, (unsigned)a.B),
                                dim3(256), 0, 1, a, a.expanded_k, a.expanded_v));
        return small ? tiles<64, EXPANDED>(ctx, a, a.expanded_k, a.expanded_v, rows, KT)
                     : tiles<128, EXPANDED>(ctx, a, a.expanded_k, a.expanded_v, rows, KT);
    }
    if (a.p.k_scale) return small ? tiles<64, PAGES8>(ctx, a, nullptr, nullptr, 0, 0) : tiles<128, PAGES8>(ctx, a, nullptr, nullptr, 0, 0);
    const int64_t rows = (a.p.n_pages * a.p.Hkv) << a.p.page_log2;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(a.p.k), *v = static_cast<const __nv_bfloat16*>(a.p.v);
    const int box = std::min(KT, 1 << a.p.page_log2);
    return small ? tiles<64, PAGES16>(ctx, a, k, v, rows, box) : tiles<128, PAGES16>(ctx, a, k, v, rows, box);
}

}  // namespace gk
