// block_mma.cuh -- what the block-scaled tensor-core kernels (block_gemm.cu,
// block_gated.cu) share: tile sizes, the tensor-memory layout of the E8M0 kernels, and
// their launches.
#pragma once

#include <atomic>

#include "block.cuh"
#include "once_per_device.h"

namespace fp8k {

constexpr int BM = 128, BN = 256, BK = 128;   // a CTA's rows, the pair's columns, a k-block
constexpr int HALF = BM * BK;                 // bytes of a CTA's A (or B) slice of one k-block

// Tensor memory of the E8M0 pair kernels.
constexpr int MX_ACC1 = 224;       // first column of the second accumulator
constexpr int MX_SF = 480;         // first column of the scales
constexpr int MX_SF_STRIDE = 16;   // columns per stage of scales: 4 for A, 8 for B

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) &
                                       ~static_cast<uintptr_t>(1023));
}

// Named barrier of n threads that tells all of them whether pred held for each.
__device__ __forceinline__ bool barrier_and(int id, int n, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(id), "r"(n), "r"(static_cast<uint32_t>(pred))
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// attr must have room for two attributes: the cluster shape and PDL.
inline cudaLaunchConfig_t cluster_config(dim3 grid, int threads, size_t smem, int cluster,
                                         cudaLaunchAttribute *attr, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// The pair kernel's shared-memory limit is set and the number of CTA pairs that
// can be resident at once is found on a device's first call.
template <typename Args>
struct PairKernel {
    void (*kernel)(Args);
    int threads;
    size_t smem;
    SmemLimit limit;
    OncePerDevice once;
    std::atomic<int> slots[kDeviceSlots] = {};

    cudaError_t init(int sm_count, int *slots_here) {
        int device = 0;
        const cudaError_t err = once.run([this, sm_count](int dev) {
            cudaError_t e = limit.allow(kernel, smem);
            if (e != cudaSuccess) return e;
            cudaLaunchAttribute attr[2];
            cudaLaunchConfig_t cfg =
                cluster_config(dim3(sm_count & ~1), threads, smem, 2, attr, nullptr);
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            slots[dev] = n;
            return e;
        }, &device);
        *slots_here = slots[device];
        return err;
    }
};

}  // namespace fp8k
