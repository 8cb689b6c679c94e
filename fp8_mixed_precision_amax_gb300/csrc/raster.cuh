// raster.cuh -- the order in which the persistent GEMM kernels (gemm.cu, block_gemm.cu)
// visit output tiles.
#pragma once

#include <cstdint>

namespace fp8k {

// Tiles are walked down groups of group_m row-blocks: tile -> (row-block mb,
// column-block nb).
__device__ __forceinline__ void tile_coords(int tile, int tiles_m, int tiles_n, int group_m,
                                            int &mb, int &nb) {
    const int group = tile / (group_m * tiles_n);
    const int first_m = group * group_m;
    const int gm = min(tiles_m - first_m, group_m);
    const int in = tile - group * group_m * tiles_n;
    mb = first_m + in % gm;
    nb = in / gm;
}

// When one operand is small enough to stay in L2, walk so that it does and the
// other streams through once: all row-blocks at a time when A is the smaller (A
// resident), two row-blocks when B is (B resident).  When neither fits: groups
// of kGroupM row-blocks when A is the smaller, so that the larger B is walked
// fewer times, and of kGroupMSmall otherwise, which keeps more of B in L2 from
// one group's waves to the next.  (Per-tensor GEMM, 70B-shaped layer, DRAM bytes per
// launch: fprop 1.10 GB with 16 against 1.47 GB with 8; the grouped backward 3.85 GB
// with 8 and 8 against 4.51 GB with 16 and 16.  The block-scaled kernels' times do not
// tell them apart, the tensor pipe and the power limit bind first: E8M0 scales, 8192 x
// 28672 x 8192 1120 us with 16, 1130 to 1144 with 8; 28672 x 8192 x 8192 1265 to 1299
// with either.)
constexpr int kGroupM = 16, kGroupMSmall = 8;
constexpr int64_t kResidentBytes = 48 << 20;   // an operand this small is kept in L2

inline int raster_group(int64_t a_bytes, int64_t b_bytes, int tiles_m) {
    if (a_bytes <= b_bytes && a_bytes <= kResidentBytes) return tiles_m;
    if (b_bytes < a_bytes && b_bytes <= kResidentBytes) return 2;
    return a_bytes < b_bytes ? kGroupM : kGroupMSmall;
}

}  // namespace fp8k
