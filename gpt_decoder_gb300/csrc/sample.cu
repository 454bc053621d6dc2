// Filtered sampling: one token per row of logits, from given uniform numbers.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Temperature and
// top-k" (the k-th largest logit is the threshold, ties with it kept).
//
// A cluster of blocks takes a row: each block reads its slice of the logits once, into shared
// memory, and the rest happens on chip. Every filter is a threshold on the logit. A row is
//   the largest logit (a maximum over the cluster);
//   a histogram of the logits, by count (top-k) or by weight (top-p), over 1024 steps of 1/22 in log2 of the
//     weight, which gives the step where the count or share is reached;
//   the logits up to that step. If they are at most 512, they are brought together in one block, which
//     finds the exact thresholds and the pick by comparing each with all the others.
//   Else (flat rows, no filter, very many equal logits): the thresholds from the logits of the
//     decisive step in the same way, or by histograms of the 32-bit keys that order floats, 1024 parts at
//     a time; then the kept weights' sums by warp, and the pick in the warp's part where it falls. The
//     kept logits are packed before their weights are taken, so that dropped ones cost no exponential.
// Weights are integers, round(2^45 exp((l - max) / T)): sums are exact, and no order of adding
// matters to the result. (Float64 runs at 1/64 of the float32 rate here, and float32 sums over a
// vocabulary would move picks: a share of 1e-7 of the weight, at 50257 tokens, falls between two
// roundings every few hundred rows.) The exponential is taken with pairs of floats:
//   z = (max - l) log2(e) / T as a pair, z = n + i / 512 + f with |f| <= 2^-10;
//   2^-z = 2^-n T (1 + e), T = 2^(-i / 512) from a table (in units of 2^-48, and as a pair), and
//   e = -g + g^2/2 - g^3/6 + g^4/24, g = f ln 2, its first term as a pair;
// T e goes to units of 2^-48 in two steps of 32 bits. Off by at most 1.6 x 2^-45 in all.
// Measured: 192 rows of 50257 float32 with filters of every kind 91 us (0.42 TB/s: the histograms' shared-memory
// atomics, the exponentials, and waits at barriers: a block's slice is a power of two, so that of four blocks the
// last holds 1105 of 50257 logits and waits for the others); one row with top-k 13.5 us, two walks over the slice
// with four barriers of the cluster and about a dozen of the block between them.
#include <math.h>

#include "launch.cuh"

namespace gk {
namespace {

constexpr int THREADS = 512, BINS = 1024, LIST = THREADS, POWERS = 512, MAX_V = 1 << 18;
constexpr uint64_t ONE = 1ull << 45;  // the largest weight: up to 2^18 tokens sum below 2^63

// round(2^63 * 2^(-i / 32)) and round(2^63 * 2^(-j / 1024))
__device__ const uint64_t POW2_32[32] = {
    0x8000000000000000ull, 0x7d41d96db915019dull, 0x7a92be8a92436616ull, 0x77f25ccdee6d7ae6ull,
    0x75606373ee921c97ull, 0x72dc8373be41a454ull, 0x70666f76154a7089ull, 0x6dfddbcbed791babull,
    0x6ba27e656b4eb57aull, 0x69540ec8f895722dull, 0x6712460a8fc24072ull, 0x64dcdec3371793d1ull,
    0x62b39508aa836d6full, 0x6096266533384a2bull, 0x5e8451cfac061b5full, 0x5c7dd7a3b17dcf75ull,
    0x5a827999fcef3242ull, 0x5891fac0e95612c8ull, 0x56ac1f752150a563ull, 0x54d0ad5a753e077cull,
    0x52ff6b54d8a89c75ull, 0x513821818624b40cull, 0x4f7a993048d088d7ull, 0x4dc69cdceaa72a9cull,
    0x4c1bf828c6dc54b8ull, 0x4a7a77d47f7b84b1ull, 0x48e1e9b9d588e19bull, 0x47521cc5a2e6a9e0ull,
    0x45cae0f1f545eb73ull, 0x444c0740496d4294ull, 0x42d561b3e6243d8aull, 0x4166c34c5615d0ecull};
__device__ const uint64_t POW2_1024[32] = {
    0x8000000000000000ull, 0x7fe9d3a8e07bf086ull, 0x7fd3ab290e46d769ull, 0x7fbd867fdf0acb3bull,
    0x7fa765aca88f6453ull, 0x7f9148aec0b9b7b1ull, 0x7f7b2f857d8c51e5ull, 0x7f651a30352731eeull,
    0x7f4f08ae3dc7c426ull, 0x7f38fafeedc8dd26ull, 0x7f22f1219ba2b4aeull, 0x7f0ceb159deae091ull,
    0x7ef6e8da4b544f9aull, 0x7ee0ea6efaaf4479ull, 0x7ecaefd302e950afull, 0x7eb4f905bb0d4f78ull,
    0x7e9f06067a4360baull, 0x7e8916d497d0e3f4ull, 0x7e732b6f6b18732aull, 0x7e5d43d64b99ddd7ull,
    0x7e47600890f223deull, 0x7e31800592db7078ull, 0x7e1ba3cca92d152cull, 0x7e05cb5d2bdb84beull,
    0x7deff6b672f84e24ull, 0x7dda25d7d6b2177full, 0x7dc458c0af549908ull, 0x7dae8f7055489813ull,
    0x7d98c9e62113e1faull, 0x7d8308216b594720ull, 0x7d6d4a218cd895e5ull, 0x7d578fe5de6e95a0ull};

// Unsigned keys in the order of the floats (-0 is made +0); NaN lowest.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
constexpr uint32_t KEY_NINF = 0x007fffffu;  // key of -inf: candidates are above it

struct SampleArgs {
    const void* logits;
    int64_t ld;
    int V, cluster, run_log2;  // blocks per row; elements per thread, a power of two
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* next;
    float* prob;
};

struct Hist {
    uint32_t count[BINS], lo[BINS], hi[BINS];  // weights as 32 low bits and the rest
    uint32_t part_lo[32], part_hi[32];         // sums of every 32 bins
};

struct Shared {
    uint64_t pow_fix[POWERS];  // 2^(-i / 512) in units of 2^-48
    float2 pow_pair[POWERS];   // and as 24 bits and the rest
    Hist hist[2];
    uint64_t red_w[THREADS / 32];
    uint32_t red_c[THREADS / 32];
    uint32_t range[2][2];   // exchange: the largest and smallest key (two sets in turn)
    uint64_t sum;           // exchange: this block's kept weight
    float c_hi, c_lo, z_max;  // the row's numbers that one thread takes in float64 (a slow pipe here)
    uint64_t least, asked;
    uint32_t n_list;        // exchange: this block's candidates, their keys and indices
    uint32_t list_k[LIST];
    int32_t list_i[LIST];
    uint32_t all_k[LIST];   // the cluster's
    int32_t all_i[LIST];
    uint64_t all_w[LIST];
    uint32_t chosen;
    uint32_t packed[THREADS / 32][64];
    int bin;                // the step where the wanted count or weight is reached, or -1
    uint64_t above, upto;   // and what lies in the steps before it, and with it
};

// What a row's weights need.
struct Scale {
    float largest, half_max, c_hi, c_lo;
    bool flat, peak;  // every finite logit has weight one; only the largest has any
};

// (max - l) log2(e) / T to float32: the same everywhere, and never larger for a larger l.
__device__ __forceinline__ float distance(const Scale& s, float l) { return fmaf(-0.5f, l, s.half_max) * s.c_hi; }

__device__ __forceinline__ uint64_t weight(const Shared& sh, const Scale& s, float l) {
    if (l == s.largest) return ONE;
    if (!(l > -INFINITY) || s.peak) return 0;
    if (s.flat) return ONE;
    // (max - l) / 2 as a pair of floats (halves: the difference cannot overflow), times 2 log2(e) / T
    const float a = s.half_max, b = -0.5f * l, d = a + b, bb = d - a;
    const float err = (a - (d - bb)) + (b - bb);
    const float z = d * s.c_hi;
    if (!(z < 47.f)) return 0;
    const float z_lo = fmaf(d, s.c_hi, -z) + fmaf(d, s.c_lo, err * s.c_hi);
    const float m = fmaf(z, 512.f, 12582912.f);  // 1.5 x 2^23: the sum's low bits are round(512 z)
    const int k = __float_as_int(m) & 0x3fffff, n = k >> 9;
    const float f = fmaf(m - 12582912.f, -1.f / 512.f, z);
    const float ln2_hi = 0x1.62e43p-1f, ln2_lo = -0x1.05c61p-29f;
    const float g = f * ln2_hi, g_lo = fmaf(f, ln2_hi, -g) + fmaf(f, ln2_lo, z_lo * ln2_hi);
    const float e = fmaf(g, g_lo, fmaf(g * g, fmaf(g, fmaf(g, 1.f / 24.f, -1.f / 6.f), 0.5f), -g_lo));
    const float2 t = sh.pow_pair[k & 511];
    const float p = -t.x * g;
    const float lo = fmaf(-t.x, g, -p) + fmaf(t.x, e, -t.y * g);
    const int hi30 = __float2int_rn(p * 0x1p30f);
    const int lo48 = __float2int_rn((lo + fmaf((float)-hi30, 0x1p-30f, p)) * 0x1p48f);
    const int64_t w = (int64_t)sh.pow_fix[k & 511] + (int64_t)hi30 * (1 << 18) + lo48;
    const int shift = 3 + n;
    return (uint64_t)(w + (1ll << (shift - 1))) >> shift;
}

__device__ __forceinline__ void row_barrier(int cluster) {
    __syncwarp();
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
}
__device__ __forceinline__ uint32_t peer_u32(const uint32_t* p, int rank, int cluster) {
    return cluster > 1 ? load_cluster_u32(p, rank) : *p;
}

// The word at p in every block of the cluster (0 past its size): all reads are on their way at once.
constexpr int MAX_CLUSTER = 8;
__device__ __forceinline__ void peers(uint32_t (&v)[MAX_CLUSTER], const uint32_t* p, int cluster) {
#pragma unroll
    for (int q = 0; q < MAX_CLUSTER; ++q) v[q] = q < cluster ? peer_u32(p, q, cluster) : 0;
}
__device__ __forceinline__ uint64_t peers_sum(const uint32_t* p, int cluster) {
    uint32_t v[MAX_CLUSTER];
    peers(v, p, cluster);
    uint64_t s = 0;
#pragma unroll
    for (int q = 0; q < MAX_CLUSTER; ++q) s += v[q];
    return s;
}

// floor(x * all) for 0 <= x < 1 (exact down to x = 2^-40), and whether anything was cut off.
__device__ __forceinline__ uint64_t part_of(float x, uint64_t all, bool* cut) {
    const uint32_t b = __float_as_uint(x);
    const int shift = (int)(b >> 23) - 86;  // x = mantissa * 2^(exponent - 150), in units of 2^-64
    const uint64_t m = (b & 0x7fffffu) | 0x800000u;
    const uint64_t fix = shift >= 0 ? m << shift : shift > -24 ? m >> -shift : 0;
    *cut = fix * all != 0;
    return __umul64hi(fix, all);
}
// A whole running sum exceeds u * all when it exceeds this; u >= 1 or NaN: the last kept.
__device__ __forceinline__ uint64_t needed(float u, uint64_t all) {
    bool cut;
    return u <= 0.f ? 0 : u < 1.f ? part_of(u, all, &cut) : all - 1;
}
// What the share p < 1 of a whole is reached with.
__device__ __forceinline__ uint64_t share(float p, uint64_t all) {
    bool cut;
    if (!(p > 0.f)) return 1;
    const uint64_t w = part_of(p, all, &cut);
    return max((uint64_t)1, w + (cut ? 1 : 0));
}

// Sums of every 32 bins, a warp two of them, before the cluster's barrier.
__device__ __forceinline__ void sum_parts(Hist& h, bool weigh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int part = warp * 2 + e, b = part * 32 + lane;
        uint64_t v = weigh ? ((uint64_t)h.hi[b] << 32) + h.lo[b] : h.count[b];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) h.part_lo[part] = (uint32_t)v, h.part_hi[part] = (uint32_t)(v >> 32);
    }
}
__device__ __forceinline__ uint64_t warp_inclusive(uint64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += x;
    }
    return v;
}

// After it: the first bin (ascending: descending logits) at which the cluster's counts (or weights) reach
// `want`, or the share p of them all, `have` before bin 0. One warp adds the parts' sums of all the
// blocks, then the 32 bins of the part where it is reached; the answers are left in sh.
__device__ __forceinline__ void search(Shared& sh, const Hist& h, int cluster, bool weigh, uint64_t want, bool of_share, float p, uint64_t have) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        uint64_t s = have + warp_inclusive((peers_sum(&h.part_hi[lane], cluster) << 32) + peers_sum(&h.part_lo[lane], cluster));
        if (of_share) want = share(p, __shfl_sync(0xffffffffu, s, 31));
        const unsigned m = __ballot_sync(0xffffffffu, s >= want);
        const int part = m ? __ffs(m) - 1 : 31, b = part * 32 + lane;
        uint64_t before = __shfl_sync(0xffffffffu, s, max(part - 1, 0));
        if (part == 0) before = have;
        s = before + warp_inclusive(weigh ? (peers_sum(&h.hi[b], cluster) << 32) + peers_sum(&h.lo[b], cluster) : peers_sum(&h.count[b], cluster));
        const unsigned m2 = __ballot_sync(0xffffffffu, s >= want);
        const int at = m2 ? __ffs(m2) - 1 : 31;
        const uint64_t upto = __shfl_sync(0xffffffffu, s, at), above = __shfl_sync(0xffffffffu, s, max(at - 1, 0));
        if (lane == 0) {
            sh.bin = m ? part * 32 + at : -1;
            sh.above = at ? above : before;
            sh.upto = upto;
            sh.asked = want;
        }
    }
    __syncthreads();
}

// Exclusive prefix of v over the block's threads, and the block's total.
__device__ __forceinline__ uint64_t block_prefix(Shared& sh, uint64_t v, uint64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t incl = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) sh.red_w[warp] = incl;
    __syncthreads();
    const uint64_t w = warp_inclusive(lane < THREADS / 32 ? sh.red_w[lane] : 0);
    *total = __shfl_sync(0xffffffffu, w, 31);
    const uint64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return (warp ? before : 0) + incl - v;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) sample_rows_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    float* x = reinterpret_cast<float*>(smem + sizeof(Shared));
    wait_for_earlier_kernels();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cl = a.cluster;
    const int r = blockIdx.x / cl, rank = blockIdx.x - r * cl, run = 1 << a.run_log2;
    const int slice = THREADS << a.run_log2, base = rank * slice, n = max(0, min(slice, a.V - base));
    const T* src = static_cast<const T*>(a.logits) + (int64_t)r * a.ld + base;
    {
        const uint64_t w = (__umul64hi(POW2_32[tid >> 4], POW2_1024[(tid & 15) * 2]) + (1 << 13)) >> 14;
        sh.pow_fix[tid] = w;
        sh.pow_pair[tid] = make_float2((float)(uint32_t)(w >> 24) * 0x1p-24f, (float)(uint32_t)(w & 0xffffff) * 0x1p-48f);
    }
    const float t = a.temperature ? a.temperature[r] : 1.f, u = a.u[r];
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;

    if (tid == 64) {
        const double c = 2.0 * 1.4426950408889634074 / (double)t;
        sh.c_hi = (float)c;
        sh.c_lo = (float)(c - (double)sh.c_hi);
        sh.least = min_p > 0.f ? max((uint64_t)1, (uint64_t)ceil((double)ONE * fmin((double)min_p, 1.0))) : 1;
        // a distance well past min_p's needs no weight
        sh.z_max = min_p > 0.f ? fminf(46.f, 0.01f - log2f(fminf(min_p, 1.f))) : 46.f;
    }
    // the slice into shared memory, and its largest key
    uint32_t most = 0;
    auto put = [&](int i, float v) {
        x[i] = v;
        most = max(most, key_of(v));
    };
    constexpr int VEC = 16 / sizeof(T);
    const int lead = min(n, (int)((-(reinterpret_cast<uintptr_t>(src) / sizeof(T))) & (VEC - 1)));
    if (tid < lead) put(tid, load_as_f32(src + tid));
    const int vecs = (n - lead) / VEC;
#pragma unroll 8
    for (int i = tid; i < vecs; i += THREADS) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src + lead) + i);
        const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = lead + i * VEC + e * (VEC / 4);
            if constexpr (sizeof(T) == 4) {
                put(at, __uint_as_float(c[e]));
            } else {
                put(at, __uint_as_float(c[e] << 16));
                put(at + 1, __uint_as_float(c[e] & 0xffff0000u));
            }
        }
    }
    const int tail = lead + vecs * VEC + tid;
    if (tail < n) put(tail, load_as_f32(src + tail));
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) sh.red_c[warp] = most;
    __syncthreads();
    if (warp == 0) {
        most = __reduce_max_sync(0xffffffffu, lane < THREADS / 32 ? sh.red_c[lane] : 0);
        if (lane == 0) sh.range[0][0] = most;
    }
    row_barrier(cl);
    uint32_t top = 0, got[MAX_CLUSTER];
    peers(got, &sh.range[0][0], cl);
#pragma unroll
    for (int q = 0; q < MAX_CLUSTER; ++q) top = max(top, got[q]);
    if (top <= KEY_NINF) {  // nothing to pick
        if (rank == 0 && tid == 0) {
            a.next[r] = -1;
            if (a.prob) a.prob[r] = 0.f;
        }
        row_barrier(cl);  // no block leaves while another reads its shared memory
        return;
    }
    const float largest = value_of(top);
    const bool greedy = !(t > 0.f);
    Scale sc;
    sc.largest = largest;
    sc.half_max = 0.5f * largest;
    sc.c_hi = sh.c_hi;
    sc.c_lo = sh.c_lo;
    sc.peak = greedy || isinf(largest) || isinf(sc.c_hi);
    sc.flat = sc.c_hi == 0.f;

    // this warp's part of the slice, 32 neighbours a turn
    const int w0 = warp * 32 * run, turns = (max(0, min(32 * run, n - w0)) + 31) >> 5;
    auto each = [&](auto&& f) {  // (index in the slice, logit; -inf past its end), four loads at a time
        for (int i = 0; i < turns; i += 4) {
            float l[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = w0 + (i + q) * 32 + lane;
                l[q] = i + q < turns && e < n ? x[e] : -INFINITY;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) f(w0 + (i + q) * 32 + lane, l[q]);
        }
    };
    uint32_t low = greedy ? top : KEY_NINF + 1;  // the threshold so far, as a key and as a logit
    float low_l = value_of(low);
    auto raise = [&](uint32_t key) {
        low = key;
        low_l = value_of(key);
    };
    const uint64_t least = sh.least;
    auto step_of = [&](float l) {
        const float z = distance(sc, l);
        return l == largest ? 0 : z < 46.5f ? (int)(z * 22.f) : BINS - 1;
    };
    auto add_weight = [&](Hist& h, int b, uint64_t w) {
        const uint32_t lo = (uint32_t)w, old = atomicAdd(&h.lo[b], lo);
        const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
        if (hi) atomicAdd(&h.hi[b], hi);
    };
    int turn = 0;  // of the two histograms and exchange words
    // the cluster's kept logits of some steps into all_k, all_i (`keep_here`, at most LIST): how many, and their range
    auto gather = [&](int step_from, int step_to, uint32_t* k_lo, uint32_t* k_hi, bool keep_here) -> uint32_t {
        uint32_t kmax = 0, kmin = 0xffffffffu;
        uint32_t* ex = sh.range[turn & 1];
        if (tid == 0) ex[0] = 0, ex[1] = 0xffffffffu, sh.n_list = 0, sh.chosen = 0;
        __syncthreads();
        each([&](int e, float l) {
            if (!(l >= low_l)) return;
            const int step = step_of(l);
            if (step < step_from || step > step_to) return;
            const uint32_t key = key_of(l);
            kmax = max(kmax, key), kmin = min(kmin, key);
            const uint32_t at = atomicAdd(&sh.n_list, 1u);
            if (at < LIST) sh.list_k[at] = key, sh.list_i[at] = base + e;
        });
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        if (lane == 0 && kmax) atomicMax(&ex[0], kmax), atomicMin(&ex[1], kmin);
        row_barrier(cl);
        uint32_t many = 0, at = tid;
        int owner = -1;
        uint32_t hi[MAX_CLUSTER], lo[MAX_CLUSTER], m[MAX_CLUSTER];
        peers(hi, &ex[0], cl);
        peers(lo, &ex[1], cl);
        peers(m, &sh.n_list, cl);
        *k_hi = 0;
        *k_lo = 0xffffffffu;
#pragma unroll
        for (int q = 0; q < MAX_CLUSTER; ++q) {
            if (q >= cl) continue;
            *k_hi = max(*k_hi, hi[q]), *k_lo = min(*k_lo, lo[q]);
            if (owner < 0 && tid < many + m[q]) owner = q, at = tid - many;
            many += m[q];
        }
        ++turn;
        if (many <= LIST && keep_here && owner >= 0) {
            sh.all_k[tid] = peer_u32(&sh.list_k[at], owner, cl);
            sh.all_i[tid] = (int32_t)peer_u32(reinterpret_cast<const uint32_t*>(&sh.list_i[at]), owner, cl);
        }
        return many;
    };
    // the largest kept key at which the sum of the candidates' weights (or their number) after `have` reaches
    // `want`; all_w is set
    auto decide = [&](uint32_t many, bool weigh, uint64_t have, uint64_t want) {
        if (tid == 0) sh.chosen = 0;
        __syncthreads();
        if (tid < many && sh.all_k[tid] >= low) {
            const uint32_t key = sh.all_k[tid];
            uint64_t sum = have;
            for (uint32_t i = 0; i < many; ++i)
                if (sh.all_k[i] >= key) sum += weigh ? sh.all_w[i] : 1;
            if (sum >= want) atomicMax(&sh.chosen, key);
        }
        __syncthreads();
        raise(sh.chosen);
        __syncthreads();
    };
    auto clear = [&](Hist& h) {
        for (int b = tid; b < BINS; b += THREADS) h.count[b] = h.lo[b] = h.hi[b] = 0;
        __syncthreads();
    };
    // where the kept logits' number reaches `want`, or their weight top_p's share, over the steps of weight
    auto histogram = [&](bool weigh, uint64_t want) {
        Hist& h = sh.hist[turn++ & 1];
        clear(h);
        each([&](int, float l) {
            if (!(l >= low_l)) return;
            const int b = step_of(l);
            if (!weigh) atomicAdd(&h.count[b], 1u);
            else if (b < BINS - 1) add_weight(h, b, weight(sh, sc, l));
        });
        __syncthreads();
        sum_parts(h, weigh);
        row_barrier(cl);
        search(sh, h, cl, weigh, want, weigh, top_p, 0);
        return sh.asked;
    };
    // the exact threshold inside a step too full to be compared pairwise: histograms of keys
    auto refine = [&](bool weigh, uint64_t want, uint64_t have, uint32_t k_lo, uint32_t k_hi) {
        const int bits = 32 - __clz((int)(k_hi - k_lo));
        uint32_t shift = bits > 10 ? (uint32_t)(bits - 10) : 0;
        while (true) {
            Hist& h = sh.hist[turn++ & 1];
            clear(h);
            for (int i = 0; i < turns; ++i) {
                const int e = w0 + i * 32 + lane;
                if (e >= n) continue;
                const float l = x[e];
                const uint32_t key = key_of(l);
                if (key > k_hi || key < k_lo || key < low) continue;
                const uint32_t b = (k_hi - key) >> shift;
                if (b >= BINS) continue;
                if (weigh) add_weight(h, b, weight(sh, sc, l));
                else atomicAdd(&h.count[b], 1u);
            }
            __syncthreads();
            sum_parts(h, weigh);
            row_barrier(cl);
            search(sh, h, cl, weigh, want, false, 0.f, have);
            const int bin = sh.bin;
            have = sh.above;
            __syncthreads();
            if (bin < 0) return;
            k_hi -= (uint32_t)bin << shift;
            if (shift == 0) {
                raise(k_hi);
                return;
            }
            shift = shift > 10 ? shift - 10 : 0;
        }
    };

    bool by_k = !greedy && top_k > 0 && top_k < a.V, by_p = !greedy && top_p < 1.f;
    if (by_k || by_p) {
        const bool weigh = !by_k;
        uint64_t want = histogram(weigh, (uint64_t)top_k);
        const int bin = sh.bin;
        const uint64_t above = sh.above;
        __syncthreads();
        // reached nowhere, or among weights of zero only: every weight stays
        bool decided = bin < 0 || bin == BINS - 1;
        if (decided && by_k) by_k = false;
        if (decided && weigh) by_p = false;
        if (!decided) {
            uint32_t k_lo, k_hi;
            // how many logits lie up to the step: by count it is known, by weight it shows
            uint32_t many = by_k && sh.upto > LIST ? LIST + 1 : gather(0, bin, &k_lo, &k_hi, rank == 0);
            if (many <= LIST) {
                // one block has all that can be picked
                if (rank == 0) {
                    if (tid < many) sh.all_w[tid] = weight(sh, sc, value_of(sh.all_k[tid]));
                    if (tid == 0) sh.bin = 0;
                    __syncthreads();
                    if (by_k) decide(many, false, 0, (uint64_t)top_k);
                    if (by_p) {
                        if (by_k) {
                            uint64_t all = tid < many && sh.all_k[tid] >= low ? sh.all_w[tid] : 0;
                            block_prefix(sh, all, &all);
                            want = share(top_p, all);
                        }
                        decide(many, true, 0, want);
                    }
                    const bool in = tid < many && sh.all_k[tid] >= low && sh.all_w[tid] >= least;
                    const uint64_t own = in ? sh.all_w[tid] : 0;
                    __syncthreads();
                    if (tid < many) sh.all_w[tid] = own;
                    uint64_t all = own;
                    block_prefix(sh, all, &all);  // (and every all_w is written)
                    const uint64_t need = needed(u, all);
                    if (own) {
                        const int32_t index = sh.all_i[tid];
                        uint64_t before = 0;
                        for (uint32_t i = 0; i < many; ++i)
                            if (sh.all_i[i] < index) before += sh.all_w[i];
                        if (before <= need && before + own > need) {
                            a.next[r] = index;
                            if (a.prob) a.prob[r] = (float)((double)own / (double)all);
                        }
                    }
                }
                row_barrier(cl);  // no block leaves while another reads its shared memory
                return;
            }
            row_barrier(cl);  // the other blocks have read this one's candidates
            many = gather(bin, bin, &k_lo, &k_hi, true);
            if (k_hi == k_lo) {
                raise(k_hi);
            } else if (many <= LIST) {
                if (weigh && tid < many) sh.all_w[tid] = weight(sh, sc, value_of(sh.all_k[tid]));
                decide(many, weigh, above, want);
            } else {
                refine(weigh, want, above, k_lo, k_hi);
            }
            __syncthreads();
        }
        if (by_p && !weigh) {  // top-p of what top-k left, where that is many
            want = histogram(true, 0);
            const int bin = sh.bin;
            const uint64_t above = sh.above;
            __syncthreads();
            if (bin >= 0 && bin < BINS - 1) {
                uint32_t k_lo, k_hi;
                const uint32_t many = gather(bin, bin, &k_lo, &k_hi, true);
                if (k_hi == k_lo) {
                    raise(k_hi);
                } else if (many <= LIST) {
                    if (tid < many) sh.all_w[tid] = weight(sh, sc, value_of(sh.all_k[tid]));
                    decide(many, true, above, want);
                } else {
                    refine(true, want, above, k_lo, k_hi);
                }
                __syncthreads();
            }
        }
    }

    // sums of the kept weights in index order: the warp's part (its kept logits packed, 32 at a time), the
    // block's, the cluster's
    const float z_max = sh.z_max;
    auto kept = [&](float l) -> uint64_t {
        if (!(l >= low_l)) return 0;
        const uint64_t w = weight(sh, sc, l);
        return w >= least ? w : 0;
    };
    uint64_t own = 0;
    uint32_t* packed = sh.packed[warp];
    int held = 0;
    each([&](int, float l) {
        const bool in = l >= low_l && (l == largest || sc.flat || (!sc.peak && distance(sc, l) <= z_max + 0.5f));
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (m == 0) return;
        if (in) packed[held + __popc(m & ((1u << lane) - 1))] = __float_as_uint(l);
        held += __popc(m);
        __syncwarp();
        if (held >= 32) {
            own += kept(__uint_as_float(packed[lane]));
            held -= 32;
            const uint32_t next = lane < held ? packed[32 + lane] : 0;
            __syncwarp();
            if (lane < held) packed[lane] = next;
            __syncwarp();
        }
    });
    if (lane < held) own += kept(__uint_as_float(packed[lane]));
    for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
    __syncthreads();
    if (lane == 0) sh.red_w[warp] = own;
    __syncthreads();
    uint64_t here = lane < THREADS / 32 ? sh.red_w[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) here += __shfl_xor_sync(0xffffffffu, here, o);
    if (tid == 0) sh.sum = here;
    row_barrier(cl);
    uint64_t all = here, before = 0;
    if (cl > 1) {
        all = 0;
        uint32_t hi[MAX_CLUSTER], lo[MAX_CLUSTER];
        peers(lo, reinterpret_cast<const uint32_t*>(&sh.sum), cl);
        peers(hi, reinterpret_cast<const uint32_t*>(&sh.sum) + 1, cl);
#pragma unroll
        for (int q = 0; q < MAX_CLUSTER; ++q) {
            const uint64_t v = ((uint64_t)hi[q] << 32) + lo[q];
            if (q < rank) before += v;
            all += v;
        }
        row_barrier(cl);  // no block leaves while another reads its shared memory
    }
    const uint64_t need = greedy ? 0 : needed(u, all);
    if (here == 0 || need < before || need >= before + here) return;  // another block's
    int part = 0;  // the warp in whose part it falls: its elements are dealt to the whole block
    while (part < THREADS / 32 - 1 && before + sh.red_w[part] <= need) before += sh.red_w[part++];
    const int per = (32 * run + THREADS - 1) / THREADS, i0 = part * 32 * run + tid * per;
    const int i1 = min(min(n, (part + 1) * 32 * run), i0 + per);
    own = 0;
    for (int i = i0; i < i1; ++i) own += kept(x[i]);
    uint64_t total;
    before += block_prefix(sh, own, &total);
    if (own && before <= need && before + own > need) {  // one thread
        for (int i = i0; i < i1; ++i) {
            const uint64_t w = kept(x[i]);
            before += w;
            if (before > need) {
                a.next[r] = base + i;
                if (a.prob) a.prob[r] = greedy ? 1.f : (float)((double)w / (double)all);
                break;
            }
        }
    }
}

}  // namespace
}  // namespace gk

using namespace gk;

extern "C" gk_status gk_sample_rows(gk_ctx* ctx, int dtype, const void* logits, int64_t ld, int64_t rows, int V,
                                    const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                                    const float* min_p, int32_t* next, float* prob) {
    if (!ctx) return GK_ERR_ARG;
    int dev = -1;
    GK_REQUIRE(ctx, cudaGetDevice(&dev) == cudaSuccess && dev == ctx->device, GK_ERR_ARG,
               "gk_sample_rows: the context's device is not current");
    GK_REQUIRE(ctx, dtype == GK_F32 || dtype == GK_BF16, GK_ERR_ARG, "gk_sample_rows: dtype %d", dtype);
    GK_REQUIRE(ctx, logits && u && next && V >= 1 && ld >= V && rows >= 0 && rows < (1ll << 28), GK_ERR_ARG,
               "gk_sample_rows: bad argument");
    GK_REQUIRE(ctx, V <= MAX_V, GK_ERR_UNSUPPORTED, "gk_sample_rows: vocabulary of %d (up to 262144)", V);
    GK_REQUIRE(ctx, reinterpret_cast<uintptr_t>(logits) % (dtype == GK_F32 ? 4 : 2) == 0, GK_ERR_ALIGN,
               "gk_sample_rows: misaligned logits");
    if (rows == 0) return GK_OK;
    SampleArgs a{logits, ld, V, 1, 0, u, temperature, top_k, top_p, min_p, next, prob};
    // blocks per row: as many as the GPU takes at once, while each still has 8 elements a thread; and enough that a
    // thread has at most 32 (113 KB of shared memory, two blocks an SM), or 64 for the largest rows. (Rows of 50257
    // in 2 / 4 / 8 blocks, top-k: one 23 / 17 / 14 us, 32 25 / 18 / 18, 64 25 / 22 / 33; mixed filters: 32 39 / 25 / 22,
    // 64 71 / 52 / 50, 192 105 / 86 / 110.)
    while (a.cluster < MAX_CLUSTER && (V > a.cluster * (THREADS * 32) ||
                             (rows * a.cluster * 2 <= 2 * ctx->num_sms && V >= a.cluster * 2 * THREADS * 8)))
        a.cluster *= 2;
    while (((int64_t)a.cluster * THREADS << a.run_log2) < V) ++a.run_log2;
    const size_t smem = sizeof(Shared) + ((size_t)THREADS << a.run_log2) * sizeof(float);
    constexpr size_t most = sizeof(Shared) + (MAX_V / MAX_CLUSTER) * sizeof(float);
    const bool f32 = dtype == GK_F32;
    GK_TRY(f32 ? allow_shared<sample_rows_kernel<float>>(ctx, "gk_sample_rows", most)
               : allow_shared<sample_rows_kernel<__nv_bfloat16>>(ctx, "gk_sample_rows", most));
    return launch_dependent(ctx, "sample_rows", f32 ? sample_rows_kernel<float> : sample_rows_kernel<__nv_bfloat16>, dim3((unsigned)(rows * a.cluster)), dim3(THREADS), smem, a.cluster, a);
}
