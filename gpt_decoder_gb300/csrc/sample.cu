// Filtered sampling: one token per row of logits, from given uniform numbers.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Temperature and
// top-k" (the k-th largest logit is the threshold, ties with it kept).
//
// A cluster of blocks takes a row: each block reads its slice of the logits once, into shared
// memory, and the rest happens on chip. Every filter is a threshold on the logit, so a row is
//   the largest logit (a maximum over the cluster),
//   top-k's threshold, then top-p's: a histogram of the kept logits, by count or by weight, over 1024 steps of
//     1/22 in log2 of the weight; then the logits of the step where the count or share is reached
//     are compared with each other, or, if over 512, cut by histograms of the 32-bit keys that
//     order floats, 1024 parts at a time, down to one key,
//   the kept weights' running sum in index order, and the pick by the thread in whose run it falls.
// Weights are integers, round(2^45 exp((l - max) / T)): sums are exact, and no order of adding
// matters to the result. (Float64 runs at 1/64 of the float32 rate here, and float32 sums over a
// vocabulary would move picks: a share of 1e-7 of the weight, at 50257 tokens, falls between two
// roundings every few hundred rows.) The exponential is taken in fixed point:
//   z = (max - l) log2(e) / T as a pair of floats, then in units of 2^-52: n + i/32 + j/1024 + r;
//   2^-z = 2^-n 2^(-i/32) 2^(-j/1024) (1 - g + g^2/2 - g^3/6 + g^4/24), g = r ln 2 < 2^-10.5,
// the two factors from tables of 32 (64 bits each), g to 64 bits, the later terms (below 2^-22) in float32:
// off by at most 1.5 x 2^-45 in all.
#include <math.h>

#include "launch.cuh"

namespace gk {
namespace {

constexpr int THREADS = 512, BINS = 1024, LIST = THREADS;
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
constexpr uint64_t LN2 = 0xb17217f7d1cf79acull;  // ln 2 in units of 2^-64

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
};

struct Shared {
    uint64_t pow32[32], pow1024[32];
    Hist hist[2];
    uint64_t red_w[THREADS / 32];
    uint32_t red_c[THREADS / 32];
    uint32_t range[2][2];   // exchange: the largest and smallest key (two sets in turn)
    uint64_t sum;           // exchange: this block's kept weight
    uint32_t n_list;        // exchange: this block's candidates
    uint32_t list[LIST], all_k[LIST];  // their keys; the cluster's keys and weights
    uint64_t all_w[LIST];
    uint32_t chosen;
    int bin;                // the step where the wanted count or weight is reached, or -1
    uint64_t above;         // and what lies in the steps before it
};

// What a row's weights need.
struct Scale {
    float half_max, c_hi, c_lo;
    bool flat, peak;  // every finite logit has weight one; only the largest has any
};

__device__ __forceinline__ float log2_distance(const Scale& s, float l, float* low) {
    // (max - l) / 2 as a pair of floats (halves: the difference cannot overflow), times 2 log2(e) / T
    const float a = s.half_max, b = -0.5f * l, d = a + b, bb = d - a;
    const float e = (a - (d - bb)) + (b - bb);
    const float z = d * s.c_hi;
    *low = fmaf(d, s.c_hi, -z) + fmaf(d, s.c_lo, e * s.c_hi);
    return z;
}

__device__ __forceinline__ uint64_t weight(const Shared& sh, const Scale& s, uint32_t key, uint32_t top, float l) {
    if (key == top) return ONE;
    if (key <= KEY_NINF || s.peak) return 0;
    if (s.flat) return ONE;
    float low;
    const float z = log2_distance(s, l, &low);
    if (!(z < 47.f)) return 0;
    // z in units of 2^-52 by its bits, and the low part by a 32-bit conversion (units of 2^-46: 64-bit
    // conversions run on the float64 pipe)
    const uint32_t bits = __float_as_uint(z);
    const int up = (int)(bits >> 23) - 98;
    const uint64_t whole = (bits & 0x7fffffu) | 0x800000u;
    const int64_t f = max((int64_t)0, (int64_t)(up >= 0 ? whole << up : up > -24 ? whole >> -up : 0) + ((int64_t)__float2int_rn(low * 0x1p46f) << 6));
    const int n = (int)(f >> 52);
    if (n >= 47) return 0;
    const uint64_t t = __umul64hi(sh.pow32[(f >> 47) & 31], sh.pow1024[(f >> 42) & 31]);  // 2^62 and below
    const uint64_t g = __umul64hi((uint64_t)f << 22, LN2);                                // units of 2^-74
    const float gf = (float)(uint32_t)(g >> 32) * 0x1p-42f;
    const float q = gf * gf * 0.5f * fmaf(gf * (-1.f / 3.f), fmaf(gf, -0.25f, 1.f), 1.f);
    const uint64_t less = (g >> 10) - ((uint64_t)__float2uint_rn(q * 0x1p53f) << 11);  // 1 - e^-g in units of 2^-64
    const uint64_t w = t - __umul64hi(t, less);
    const int shift = 17 + n;
    return (w + (1ull << (shift - 1))) >> shift;
}

__device__ __forceinline__ void row_barrier(int cluster) {
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
}
__device__ __forceinline__ uint32_t peer_u32(const uint32_t* p, int rank, int cluster) {
    return cluster > 1 ? load_cluster_u32(p, rank) : *p;
}

// The first bin (ascending: descending logits) at which the counts (or weights) of all the
// cluster's blocks reach `want`, `have` before bin 0; what lies before the bin is left in sh.
__device__ void find_bin(Shared& sh, const Hist& mine, int cluster, bool weigh, uint64_t want, uint64_t have) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t v[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int b = threadIdx.x * 2 + e;
        for (int r = 0; r < cluster; ++r) {
            if (weigh) v[e] += ((uint64_t)peer_u32(&mine.hi[b], r, cluster) << 32) + peer_u32(&mine.lo[b], r, cluster);
            else v[e] += peer_u32(&mine.count[b], r, cluster);
        }
    }
    uint64_t incl = v[0] + v[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sh.red_w[warp] = incl;
    if (threadIdx.x == 0) sh.bin = -1;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += sh.red_w[w];
    incl += have;
    const uint64_t mid = incl - v[1], before = mid - v[0];
    if (before < want && incl >= want) {  // one thread at most
        const bool second = mid < want;
        sh.bin = threadIdx.x * 2 + (second ? 1 : 0);
        sh.above = second ? mid : before;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(THREADS) sample_rows_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    float* x = reinterpret_cast<float*>(smem + sizeof(Shared));  // thread i's run at i * (run + 1): no bank conflicts
    wait_for_earlier_kernels();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cl = a.cluster;
    const int r = blockIdx.x / cl, rank = blockIdx.x - r * cl, lg = a.run_log2, run = 1 << lg;
    const int slice = THREADS << lg, base = rank * slice, n = max(0, min(slice, a.V - base));
    const T* src = static_cast<const T*>(a.logits) + (int64_t)r * a.ld + base;
    if (tid < 32) sh.pow32[tid] = POW2_32[tid], sh.pow1024[tid] = POW2_1024[tid];
    const float t = a.temperature ? a.temperature[r] : 1.f, u = a.u[r];
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;

    // the slice into shared memory, and its largest key
    uint32_t most = 0;
    auto put = [&](int i, float v) {
        x[i + (i >> lg)] = v;
        most = max(most, key_of(v));
    };
    constexpr int VEC = 16 / sizeof(T);
    const int lead = min(n, (int)((-(reinterpret_cast<uintptr_t>(src) / sizeof(T))) & (VEC - 1)));
    if (tid < lead) put(tid, load_as_f32(src + tid));
    const int vecs = (n - lead) / VEC;
#pragma unroll 4
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
    if (tid == 0) {
        for (int w = 1; w < THREADS / 32; ++w) most = max(most, sh.red_c[w]);
        sh.range[0][0] = most;
    }
    row_barrier(cl);
    uint32_t top = 0;
    for (int q = 0; q < cl; ++q) top = max(top, peer_u32(&sh.range[0][0], q, cl));
    const bool empty = top <= KEY_NINF;
    if (empty) {
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
    const double c = 2.0 * 1.4426950408889634074 / (double)t;
    sc.half_max = 0.5f * largest;
    sc.c_hi = (float)c;
    sc.c_lo = (float)(c - (double)sc.c_hi);
    sc.peak = greedy || isinf(largest) || isinf(sc.c_hi);
    sc.flat = sc.c_hi == 0.f;

    const int i0 = min(tid << lg, n), mine = min(run, n - i0);
    const float* xr = x + tid * (run + 1);
    uint32_t low = greedy ? top : KEY_NINF + 1;  // the threshold so far
    int turn = 0;
    // raise `low` to the largest key that keeps `want` tokens, or the share p of the weight, of those kept now
    auto select = [&](bool weigh, uint64_t want, float p) {
        uint32_t k_hi = 0, k_lo = 0, shift = 0;  // the range of keys under the bins, once below the steps of weight
        int step = -1;
        uint64_t have = 0;
        auto step_of = [&](uint32_t key, float l) {
            if (key == top || sc.flat) return 0;
            float lo;
            const float z = sc.peak ? INFINITY : log2_distance(sc, l, &lo);
            return z < 46.5f ? (int)(z * 22.f) : BINS - 1;
        };
        for (int level = 0;; ++level) {
            Hist& h = sh.hist[turn & 1];
            for (int b = tid; b < BINS; b += THREADS) h.count[b] = h.lo[b] = h.hi[b] = 0;
            __syncthreads();
            for (int i = 0; i < mine; ++i) {
                const float l = xr[i];
                const uint32_t key = key_of(l);
                if (key < low) continue;
                int b;
                if (level == 0) {
                    b = step_of(key, l);
                } else {
                    if (key > k_hi || key < k_lo) continue;  // (steps are ranges of keys)
                    const uint32_t d = (k_hi - key) >> shift;
                    if (d >= BINS) continue;
                    b = (int)d;
                }
                if (weigh) {
                    const uint64_t w = weight(sh, sc, key, top, l);
                    const uint32_t lo = (uint32_t)w, old = atomicAdd(&h.lo[b], lo);
                    const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
                    if (hi) atomicAdd(&h.hi[b], hi);
                } else {
                    atomicAdd(&h.count[b], 1u);
                }
            }
            row_barrier(cl);
            if (weigh && level == 0) {  // the share of the whole
                uint64_t all = 0;
                for (int b = tid; b < BINS; b += THREADS)
                    for (int q = 0; q < cl; ++q) all += ((uint64_t)peer_u32(&h.hi[b], q, cl) << 32) + peer_u32(&h.lo[b], q, cl);
                for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
                if (lane == 0) sh.red_w[warp] = all;
                __syncthreads();
                all = 0;
                for (int w = 0; w < THREADS / 32; ++w) all += sh.red_w[w];
                want = p > 0.f ? max((uint64_t)1, (uint64_t)ceil((double)p * (double)all)) : 1;
                __syncthreads();
            }
            find_bin(sh, h, cl, weigh, want, have);
            ++turn;
            const int bin = sh.bin;
            if (bin >= 0) have = sh.above;
            if (bin < 0) return;  // there are fewer: all stay
            if (level == 0) {
                if (bin == BINS - 1) return;  // reached among weights of zero: all others stay
                step = bin;
                // the logits of this step, over the cluster: usually few enough that each is compared with
                // all the others
                uint32_t kmax = 0, kmin = 0xffffffffu;
                uint32_t* ex = sh.range[turn & 1];
                if (tid == 0) ex[0] = 0, ex[1] = 0xffffffffu, sh.n_list = 0, sh.chosen = 0;
                __syncthreads();
                for (int i = 0; i < mine; ++i) {
                    const uint32_t key = key_of(xr[i]);
                    if (key < low || step_of(key, xr[i]) != step) continue;
                    kmax = max(kmax, key), kmin = min(kmin, key);
                    const uint32_t at = atomicAdd(&sh.n_list, 1u);
                    if (at < LIST) sh.list[at] = key;
                }
                kmax = __reduce_max_sync(0xffffffffu, kmax);
                kmin = __reduce_min_sync(0xffffffffu, kmin);
                if (lane == 0 && kmax) atomicMax(&ex[0], kmax), atomicMin(&ex[1], kmin);
                row_barrier(cl);
                k_hi = 0;
                k_lo = 0xffffffffu;
                uint32_t many = 0, at = tid;
                int from = -1;
                for (int q = 0; q < cl; ++q) {
                    k_hi = max(k_hi, peer_u32(&ex[0], q, cl)), k_lo = min(k_lo, peer_u32(&ex[1], q, cl));
                    const uint32_t m = peer_u32(&sh.n_list, q, cl);
                    if (from < 0 && tid < many + m) from = q, at = tid - many;
                    many += m;
                }
                if (k_hi == k_lo) {
                    low = k_hi;
                    return;
                }
                if (many <= LIST) {
                    if (from >= 0) {
                        const uint32_t key = peer_u32(&sh.list[at], from, cl);
                        sh.all_k[tid] = key;
                        sh.all_w[tid] = weigh ? weight(sh, sc, key, top, value_of(key)) : 1;
                    }
                    __syncthreads();
                    if (from >= 0) {
                        const uint32_t key = sh.all_k[tid];
                        uint64_t sum = have;
                        for (uint32_t i = 0; i < many; ++i)
                            if (sh.all_k[i] >= key) sum += sh.all_w[i];
                        if (sum >= want) atomicMax(&sh.chosen, key);
                    }
                    __syncthreads();
                    low = sh.chosen;
                    return;
                }
                const int bits = 32 - __clz((int)(k_hi - k_lo));
                shift = bits > 10 ? (uint32_t)(bits - 10) : 0;
            } else {
                k_hi -= (uint32_t)bin << shift;
                if (shift == 0) {
                    low = k_hi;
                    return;
                }
                shift = shift > 10 ? shift - 10 : 0;
            }
            __syncthreads();
        }
    };
    if (!greedy) {
        if (top_k > 0 && top_k < a.V) select(false, (uint64_t)top_k, 0.f);
        if (top_p < 1.f) select(true, 0, top_p);
    }
    const uint64_t least = min_p > 0.f ? max((uint64_t)1, (uint64_t)ceil((double)ONE * fmin((double)min_p, 1.0))) : 1;
    auto kept = [&](float l) -> uint64_t {
        const uint32_t key = key_of(l);
        if (key < low) return 0;
        const uint64_t w = weight(sh, sc, key, top, l);
        return w >= least ? w : 0;
    };
    // running sums in index order: the thread's, the block's, the cluster's
    uint64_t own = 0;
    for (int i = 0; i < mine; ++i) own += kept(xr[i]);
    uint64_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sh.red_w[warp] = incl;
    __syncthreads();
    uint64_t before = incl - own, all = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh.red_w[w];
        all += sh.red_w[w];
    }
    if (tid == 0) sh.sum = all;
    row_barrier(cl);
    if (cl > 1) {
        all = 0;
        for (int q = 0; q < cl; ++q) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&sh.sum);
            const uint64_t v = ((uint64_t)peer_u32(p + 1, q, cl) << 32) + peer_u32(p, q, cl);
            if (q < rank) before += v;
            all += v;
        }
        row_barrier(cl);  // no block leaves while another reads its shared memory
    }
    // a whole running sum exceeds u * all when it exceeds its floor; u >= 1 or NaN: the last kept
    const double ua = (double)u * (double)all;
    const uint64_t need = greedy ? 0 : ua < (double)all ? min((uint64_t)fmax(ua, 0.0), all - 1) : all - 1;
    if (own && before <= need && before + own > need) {  // one thread of the cluster
        for (int i = 0; i < mine; ++i) {
            const uint64_t w = kept(xr[i]);
            before += w;
            if (before > need) {
                a.next[r] = base + i0 + i;
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
    GK_REQUIRE(ctx, V <= 1 << 18, GK_ERR_UNSUPPORTED, "gk_sample_rows: vocabulary of %d (up to 262144)", V);
    GK_REQUIRE(ctx, reinterpret_cast<uintptr_t>(logits) % (dtype == GK_F32 ? 4 : 2) == 0, GK_ERR_ALIGN,
               "gk_sample_rows: misaligned logits");
    if (rows == 0) return GK_OK;
    SampleArgs a{logits, ld, V, 1, 0, u, temperature, top_k, top_p, min_p, next, prob};
    // blocks per row: as many as fill the GPU, while each still has 8 elements a thread; and enough that a
    // thread has at most 32 (98 KB of shared memory, two blocks an SM), or 64 for the largest rows
    while (a.cluster < 8 && (V > a.cluster * (THREADS * 32) ||
                             (rows * a.cluster * 2 <= 4 * ctx->num_sms && V >= a.cluster * 2 * THREADS * 8)))
        a.cluster *= 2;
    while (((int64_t)a.cluster * THREADS << a.run_log2) < V) ++a.run_log2;
    const size_t smem = sizeof(Shared) + (size_t)THREADS * ((1 << a.run_log2) + 1) * sizeof(float);
    auto kernel = dtype == GK_F32 ? sample_rows_kernel<float> : sample_rows_kernel<__nv_bfloat16>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return fail(ctx, GK_ERR_CUDA, "gk_sample_rows: shared memory");
    }
    return launch_dependent(ctx, "sample_rows", kernel, dim3((unsigned)(rows * a.cluster)), dim3(THREADS), smem, a.cluster, a);
}
