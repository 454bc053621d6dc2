// Filtered sampling: one token per row of logits, from given uniform numbers.
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Temperature and
// top-k" (the k-th largest logit is the threshold, ties with it kept).
//
// Every filter is a threshold on the logit: top-k and top-p find theirs by bisection over the
// 32-bit keys that order floats, counting (or weighing) the logits at or above a key. Weights are
// integers, round(2^45 exp((l - max) / T)), so sums are exact and no order of adding matters.
#include <math.h>

#include "common.cuh"

namespace gk {
namespace {

constexpr int THREADS = 1024;
constexpr double ONE = 35184372088832.0;  // 2^45: up to 2^18 tokens sum below 2^63

// Unsigned keys in the order of the floats (-0 below +0 is made equal first); NaN lowest.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
constexpr uint32_t KEY_NINF = 0x007fffffu;  // key of -inf: candidates are above it

struct SampleArgs {
    const void* logits;
    int64_t ld;
    int V;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* next;
    float* prob;
};

__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* red) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint64_t t = 0;
    for (int w = 0; w < THREADS / 32; ++w) t += red[w];
    return t;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) sample_rows_kernel(SampleArgs a) {
    __shared__ uint64_t red[THREADS / 32];
    __shared__ uint32_t kmax;
    __shared__ int first;
    const int r = blockIdx.x, V = a.V;
    const T* x = static_cast<const T*>(a.logits) + (int64_t)r * a.ld;
    if (threadIdx.x == 0) kmax = 0, first = 0x7fffffff;
    __syncthreads();
    uint32_t mine = 0;
    for (int i = threadIdx.x; i < V; i += THREADS) mine = max(mine, key_of(load_as_f32(x + i)));
    atomicMax(&kmax, mine);
    __syncthreads();
    const uint32_t top = kmax;
    if (top <= KEY_NINF) {
        if (threadIdx.x == 0) {
            a.next[r] = -1;
            if (a.prob) a.prob[r] = 0.f;
        }
        return;
    }
    const float lmax = __uint_as_float((top & 0x80000000u) ? top & 0x7fffffffu : ~top);
    const float t = a.temperature ? a.temperature[r] : 1.f;
    const bool greedy = !(t > 0.f);
    auto weight = [&](uint32_t key, float l) -> uint64_t {
        if (key <= KEY_NINF) return 0;
        if (key == top) return (uint64_t)ONE;
        if (greedy || lmax == INFINITY) return 0;
        return (uint64_t)llrint(ONE * exp(((double)l - (double)lmax) / (double)t));
    };
    uint32_t low = greedy ? top : KEY_NINF + 1;  // the threshold so far
    // the largest threshold that keeps at least `want` (tokens, or their weight) of those from `from`
    auto bisect = [&](uint32_t from, bool weigh, uint64_t want) {
        uint32_t lo = from, hi = top;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            uint64_t s = 0;
            for (int i = threadIdx.x; i < V; i += THREADS) {
                const float l = load_as_f32(x + i);
                const uint32_t k = key_of(l);
                if (k >= mid) s += weigh ? weight(k, l) : 1;
            }
            if (block_sum(s, red) >= want) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    auto total = [&]() {
        uint64_t s = 0;
        for (int i = threadIdx.x; i < V; i += THREADS) {
            const float l = load_as_f32(x + i);
            const uint32_t k = key_of(l);
            if (k >= low) s += weight(k, l);
        }
        return block_sum(s, red);
    };
    if (!greedy) {
        const int k = a.top_k ? a.top_k[r] : 0;
        if (k > 0 && k < V) low = bisect(low, false, (uint64_t)k);
        const float p = a.top_p ? a.top_p[r] : 1.f;
        if (p < 1.f) low = bisect(low, true, p > 0.f ? (uint64_t)ceil((double)p * (double)total()) : 1);
    }
    const float mp = a.min_p ? a.min_p[r] : 0.f;
    const uint64_t least = mp > 0.f ? (uint64_t)ceil(ONE * fmin((double)mp, 1.0)) : 1;
    // contiguous ranges per thread: exclusive sums in index order
    const int per = (V + THREADS - 1) / THREADS, i0 = min(V, (int)threadIdx.x * per), i1 = min(V, i0 + per);
    auto kept = [&](int i) -> uint64_t {
        const float l = load_as_f32(x + i);
        const uint32_t k = key_of(l);
        if (k < low) return 0;
        const uint64_t w = weight(k, l);
        return w >= least ? w : 0;
    };
    uint64_t s = 0;
    for (int i = i0; i < i1; ++i) s += kept(i);
    uint64_t incl = s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    uint64_t before = 0, all = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += red[w];
        all += red[w];
    }
    before += incl - s;
    // a whole running sum exceeds u * all when it exceeds its floor; u >= 1 or NaN: the last kept
    const double ua = (double)a.u[r] * (double)all;
    const uint64_t need = greedy ? 0 : ua < (double)all ? min((uint64_t)fmax(ua, 0.0), all - 1) : all - 1;
    uint64_t run = before;
    if (s && before + s > need)
        for (int i = i0; i < i1; ++i) {
            const uint64_t w = kept(i);
            run += w;
            if (w && run > need) {
                atomicMin(&first, i);
                break;
            }
        }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.next[r] = first;
        if (a.prob) a.prob[r] = greedy ? 1.f : (float)((double)kept(first) / (double)all);
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
    GK_REQUIRE(ctx, logits && u && next && V >= 1 && ld >= V && rows >= 0 && rows < (1ll << 31), GK_ERR_ARG,
               "gk_sample_rows: bad argument");
    GK_REQUIRE(ctx, V <= 1 << 18, GK_ERR_UNSUPPORTED, "gk_sample_rows: vocabulary of %d (up to 262144)", V);
    if (rows == 0) return GK_OK;
    SampleArgs a{logits, ld, V, u, temperature, top_k, top_p, min_p, next, prob};
    if (dtype == GK_F32) sample_rows_kernel<float><<<(unsigned)rows, THREADS, 0, ctx->stream>>>(a);
    else sample_rows_kernel<__nv_bfloat16><<<(unsigned)rows, THREADS, 0, ctx->stream>>>(a);
    return launched(ctx, "sample_rows");
}
