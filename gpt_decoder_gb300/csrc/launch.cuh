// Launches of the serving kernels: as programmatic dependents of the kernel before them on the
// stream, alone or in clusters, and the cluster's barrier and shared-memory reads.
#pragma once

#include <atomic>

#include "common.cuh"

namespace gk {

// Let `Kernel` have up to `bytes` (always the same) of dynamic shared memory on the context's device. The
// setting lasts, so it is made once a device (it takes the host about as long as a launch).
template <auto Kernel>
gk_status allow_shared(gk_ctx* ctx, const char* what, size_t bytes) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = ctx->device < 64 ? 1ull << ctx->device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return GK_OK;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
        cudaGetLastError();
        return fail(ctx, GK_ERR_CUDA, "%s: shared memory", what);
    }
    done.fetch_or(bit, std::memory_order_relaxed);
    return GK_OK;
}

// Every thread of `kernel` begins with wait_for_earlier_kernels, so only the launch overlaps the
// earlier kernel's end. cluster: blocks along x that form one cluster (1: none).
template <typename... KArgs, typename... Args>
gk_status launch_dependent(gk_ctx* ctx, const char* what, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           int cluster, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx->stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(ctx, GK_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
    }
    return launched(ctx, what);
}

// A branch of a call's launches, beside those on the context's stream: what run() launches comes after all that was on
// the stream when the branch was made, and what is launched after join() after both. Events fork and join it, so that it can be
// captured with the stream; a call that fails on the way joins all the same.
class Branch {
public:
    explicit Branch(gk_ctx* ctx) : ctx_(ctx), main_(ctx->stream) {}
    Branch(const Branch&) = delete;
    Branch& operator=(const Branch&) = delete;
    ~Branch() { join(); }
    gk_status fork() {
        if (cudaEventRecord(ctx_->forked, main_) != cudaSuccess || cudaStreamWaitEvent(ctx_->side, ctx_->forked, 0) != cudaSuccess) return failed("fork");
        open_ = true;
        return GK_OK;
    }
    template <typename F>
    gk_status run(F launches) {
        ctx_->stream = ctx_->side;
        const gk_status s = launches();
        ctx_->stream = main_;
        return s;
    }
    gk_status join() {
        if (!open_) return GK_OK;
        open_ = false;
        if (cudaEventRecord(ctx_->joined, ctx_->side) != cudaSuccess || cudaStreamWaitEvent(main_, ctx_->joined, 0) != cudaSuccess) return failed("join");
        return GK_OK;
    }

private:
    gk_status failed(const char* what) {
        return fail(ctx_, GK_ERR_CUDA, "%s of a call's launches: %s", what, cudaGetErrorString(cudaGetLastError()));
    }
    gk_ctx* ctx_;
    cudaStream_t main_;
    bool open_ = false;
};

__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// (a & b) | c in one instruction. Only one operand of it can be a constant in the code: kernels that unpack
// codes take their masks as arguments (CodeMasks), which stay in registers.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
struct CodeMasks {
    uint32_t bf16_128 = 0x43004300u;  // 128 as a pair of bf16: seven low bits added to it are exact
    uint32_t low7 = 0x007f007fu, sign = 0x00800080u;   // 8-bit codes
    uint32_t low4 = 0x000f000fu, bf16_136 = 0x43084308u;  // 4-bit codes
};

// Every thread of every block of the cluster arrives, then waits (release / acquire).
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at this block's shared-memory address p, read from block `rank` of the cluster. (No memory
// clobber, so that several such reads are on their way at once: a barrier before them orders them.)
__device__ __forceinline__ uint32_t load_cluster_u32(const void* p, int rank) {
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
// Four words (16-byte aligned) of block `rank`.
__device__ __forceinline__ uint4 load_cluster_u32x4(const void* p, int rank) {
    uint32_t at;
    uint4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ float load_cluster(const float* p, int rank) { return __uint_as_float(load_cluster_u32(p, rank)); }

}  // namespace gk
