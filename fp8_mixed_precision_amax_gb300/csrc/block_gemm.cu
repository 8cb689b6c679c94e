// block_gemm.cu -- FP8 matrix product with a scale for each block of 128, on the
// sm_103a tcgen05 tensor cores:
//   D[i][j] = bf16_rne( sum over k-blocks b of sA(i, b) * sB(j, b) * dot_b ),
//   dot_b = sum over the block's 128 columns of A[i][c] * B[j][c]   (fp32)
// A is [M][K], B [N][K], both contiguous along K; sA and sB belong to one row
// or to 128 rows, and are E8M0 bytes or floats.  Three kernels:
//
//   mx    E8M0 scales, many rows: the tensor cores take the scales themselves
//         (kind::mxf8f6f4), so a tile's sums stay in TMEM over all of K;
//   f32   float scales, many rows: each k-block's dot_b goes from TMEM into
//         register sums, times its scale;
//   few   few rows (tokens being decoded): the rows of B, the weights, take the
//         instruction's 128-row side and the tokens its columns, and K is split
//         over a cluster whose CTAs join their sums in shared memory.
//
// Every wait is bounded.
#include <atomic>
#include <cstdint>

#include "block.cuh"
#include "once_per_device.h"
#include "raster.cuh"

namespace fp8k {

namespace {

__device__ unsigned g_block_gemm_error_flags = 0;

constexpr int BM = 128, BN = 256, BK = 128;   // a CTA's rows, the pair's columns, a k-block
constexpr int HALF = BM * BK;                 // bytes of a CTA's A (or B) slice of one k-block
constexpr int EPI_COLS = 64;                  // output columns staged at a time (128 B of BF16)
constexpr int EPI_BUF = 32 * EPI_COLS * 2;    // a warp's staging buffer: 32 rows x 128 B

__device__ __forceinline__ void raise_error(volatile int *abort_flag) {
    atomicOr(&g_block_gemm_error_flags, kErrWaitTimeout);
    *abort_flag = 1;
}

// One row's float scales along K, fetched four k-blocks ahead, four at a time.
// (Fetched one block ahead, each block waited for L2.)
struct ScaleStream {
    const float *row;
    int num_kb;
    bool vec;        // four floats are one 16-byte load
    float ahead[4];  // the next group
    float cur[4];    // scales from the current k-block on

    __device__ __forceinline__ void fetch(int group) {
        const int kb = 4 * group;
        if (kb >= num_kb) return;
        if (vec) {
            const float4 u = reinterpret_cast<const float4 *>(row)[group];
            ahead[0] = u.x, ahead[1] = u.y, ahead[2] = u.z, ahead[3] = u.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) ahead[i] = kb + i < num_kb ? row[kb + i] : 0.0f;
        }
    }
    __device__ __forceinline__ void take() {
#pragma unroll
        for (int i = 0; i < 4; ++i) cur[i] = ahead[i];
    }
    __device__ __forceinline__ void shift() { cur[0] = cur[1], cur[1] = cur[2], cur[2] = cur[3]; }
    // from k-block kb0 on, up to `blocks`
    __device__ __forceinline__ void start(const BlockView &v, int64_t r, int kb0, int blocks) {
        row = static_cast<const float *>(v.scales) + (v.block_rows == 1 ? r : r >> 7) * v.ld_s;
        vec = ((reinterpret_cast<uintptr_t>(v.scales) | static_cast<uintptr_t>(4 * v.ld_s)) & 15u) == 0;
        num_kb = blocks;
        fetch(kb0 >> 2);
        if (kb0 & 3) {
            take();
            for (int i = 0; i < (kb0 & 3); ++i) shift();
            fetch((kb0 >> 2) + 1);
        }
    }
    // the scale of k-block kb; called for each in turn
    __device__ __forceinline__ float next(int kb) {
        if ((kb & 3) == 0) {
            take();
            fetch((kb >> 2) + 1);
        }
        const float s = cur[0];
        shift();
        return s;
    }
};

// ------------------------------------------------------- pair kernels: common --
// Two CTAs on two SMs (a cluster) share each 256 x 256 tile (cta_group::2): each
// loads its own 128 rows of A and 128 of the 256 rows of B, and the even CTA
// issues MMAs that read both CTAs' shared memory and write both CTAs' TMEM.

// The tiles of the last, partial wave are cut into four pieces by columns where that many
// pairs would have nothing to do otherwise (4096 x 11008 has 9 waves of 76 pairs and 4
// tiles: 16 pieces).  Each sum is the same.
constexpr int kPieces = 4;

struct PairArgs {
    CUtensorMap mapA, mapB, mapD;
    CUtensorMap mapBPart;   // mapB with the rows of a piece
    BlockView A, B;
    __nv_bfloat16 *D;
    int64_t M, N, ldd;
    bool tma_d;     // D's rows are 16-byte aligned: store by TMA
    bool pairs_d;   // D's rows are 4-byte aligned
    int tiles_m, tiles_n, num_items, num_kb, group_m;
    int whole;   // items from this one on are pieces
    uint32_t idesc, idesc_part;
};

struct Item {
    int64_t row0;   // of the pair's 256 rows of D
    int64_t col0;
    int width;      // columns: 256, of a piece 64
};

__device__ __forceinline__ Item item_at(const PairArgs &a, int item) {
    const bool part = item >= a.whole;
    const int tile = part ? a.whole + (item - a.whole) / kPieces : item;
    int mb, nb;
    tile_coords(tile, a.tiles_m, a.tiles_n, a.group_m, mb, nb);
    Item t;
    t.row0 = static_cast<int64_t>(mb) * 2 * BM;
    t.width = part ? BN / kPieces : BN;
    t.col0 = static_cast<int64_t>(nb) * BN + (part ? (item - a.whole) % kPieces * t.width : 0);
    return t;
}

// The producer warp: A and B slices of every k-block of the pair's tiles.
template <int STAGES>
__device__ __forceinline__ void produce(const PairArgs &a, uint32_t rank, int unit, int num_units,
                                        uint32_t sA, uint32_t sB, uint32_t full0, uint32_t empty0,
                                        volatile int *abort_flag) {
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int item = unit; ok && item < a.num_items; item += num_units) {
        const Item t = item_at(a, item);
        const int32_t arow = static_cast<int32_t>(t.row0) + static_cast<int32_t>(rank) * BM;
        const int32_t brow = static_cast<int32_t>(t.col0) + static_cast<int32_t>(rank) * (t.width / 2);
        const CUtensorMap *mapB = t.width == BN ? &a.mapB : &a.mapBPart;
        const uint32_t bytes = 2 * HALF + t.width * BK;
        for (int kb = 0; kb < a.num_kb; ++kb) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag))) {
                if ((threadIdx.x & 31) == 0) raise_error(abort_flag);
                ok = false;
                break;
            }
            if (elect_one()) {
                // both CTAs' halves complete on the even CTA's barrier
                const uint32_t fb = full0 + 8 * stage, fb0 = mapa_shared(fb, 0);
                if (rank == 0) mbar_arrive_expect_tx(fb, bytes);
                tma_load_2d_pair(sA + stage * HALF, &a.mapA, fb0, kb * BK, arow);
                tma_load_2d_pair(sB + stage * HALF, mapB, fb0, kb * BK, brow);
            }
            __syncwarp();
            ++issued;
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    if (ok) {
        // every stage's last release is signalled from the even SM: it must have
        // arrived before this CTA exits
        for (int i = 0; i < STAGES; ++i) {
            mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag);
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (rank == 0) {
        // let the copies already issued land before the CTA exits
        for (int i = 0; i < STAGES && issued > 0; ++i, --issued) {
            stage = stage == 0 ? STAGES - 1 : stage - 1;
            if (stage == STAGES - 1) phase ^= 1u;
            mbar_wait(full0 + 8 * stage, phase, nullptr, 100000000ull);
        }
    }
}

// A warp's 32 rows x 64 columns of BF16 to D at (row0, col0) from its staging buffer,
// where 16-byte chunk j of row r sits at j ^ (r mod 8): the 128-byte swizzle of D's
// tensor map.  Rows of D that TMA cannot address, and chunks of 32 columns, go out with
// each warp instruction along one row.
__device__ __forceinline__ void store_chunk(const PairArgs &a, uint32_t sbuf, int64_t row0,
                                            int64_t col0, int cols = EPI_COLS) {
    const int lane = threadIdx.x & 31;
    // a TMA store clips at 16-byte steps: a chunk that ends inside one goes the other way
    if (a.tma_d && cols == EPI_COLS && (col0 + EPI_COLS <= a.N || a.N % 8 == 0)) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (row0 < a.M && col0 < a.N)   // boxes wholly outside D are skipped
                tma_store_2d(&a.mapD, sbuf, static_cast<int32_t>(col0), static_cast<int32_t>(row0));
            bulk_commit_group();
        }
        return;
    }
    __syncwarp();
    const int64_t c = col0 + 2 * lane, end = min(a.N, col0 + cols);
    const int rows = row0 >= a.M ? 0 : a.M - row0 < 32 ? static_cast<int>(a.M - row0) : 32;
    for (int r = 0; r < rows; ++r) {
        uint32_t w;
        asm volatile("ld.shared.b32 %0, [%1];"
                     : "=r"(w)
                     : "r"(sbuf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + ((lane & 3) << 2))
                     : "memory");
        uint16_t *d = reinterpret_cast<uint16_t *>(a.D + (row0 + r) * a.ldd + c);
        if (a.pairs_d && c + 1 < end) {
            *reinterpret_cast<uint32_t *>(d) = w;
        } else {
            if (c < end) d[0] = static_cast<uint16_t>(w);
            if (c + 1 < end) d[1] = static_cast<uint16_t>(w >> 16);
        }
    }
    __syncwarp();
    if (lane == 0) bulk_commit_group();   // an empty one: each chunk is one group
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) &
                                       ~static_cast<uintptr_t>(1023));
}

// ------------------------------------------------------------------ mx kernel --
// Warps: 0 TMA, 1 MMA, 4-7 scales, 8-11 epilogue (2 and 3 idle: tcgen05.st and .ld
// reach the lane quarter of the warp's number mod 4).
//
// TMEM (512 columns): a 256-column accumulator fills half, and two of them leave no
// room for scales.  So the two overlap: tile i uses columns 0-255 or 224-479 in turn.
// The epilogue reads the shared 32 columns first and then lets the next tile's MMAs
// start, which costs them one 64-column read (an eighth of the epilogue) instead of
// all of it.  Columns 480-511 hold two stages of scales: the word of lane l, column
// j is row 32 j + l's four E8M0 bytes of k-blocks 4 g .. 4 g + 3 (4 columns for the
// CTA's rows of A, 8 for the tile's rows of B, the same in all four lane quarters);
// the MMAs of k-block 4 g + b name byte b in their descriptor.  A block of 128 is
// four of the instruction's blocks of 32 with the same scale.
//
// Bound by the tensor pipe, and in back-to-back calls by the power limit: 8192 x 11008 x
// 4096 takes 218 us (3390 TFLOP/s), 8192 x 28672 x 8192 1067 us (3610).

constexpr int MX_STAGES = 6;
constexpr int MX_THREADS = 384;
constexpr int MX_ACC1 = 224;       // first column of the second accumulator
constexpr int MX_SF = 480;         // first column of the scales
constexpr int MX_SF_STRIDE = 16;   // columns per stage of scales: 4 for A, 8 for B
constexpr int MX_BARS = 2 * MX_STAGES + 2 + 1 + 4 + 1;
constexpr size_t MX_SMEM = 1024 + MX_STAGES * 2 * HALF + 4 * 2 * EPI_BUF + MX_BARS * 8 + 16;

__global__ void __launch_bounds__(MX_THREADS, 1)
    block_gemm_mx_kernel(const __grid_constant__ PairArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sA = smem_u32(smem), sB = sA + MX_STAGES * HALF;
    const uint32_t sD = sB + MX_STAGES * HALF;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + MX_STAGES * 2 * HALF + 4 * 2 * EPI_BUF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + MX_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();   // 0 = the CTA that issues MMAs
    const int unit = static_cast<int>(blockIdx.x >> 1), num_units = static_cast<int>(gridDim.x >> 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * MX_STAGES;
    const uint32_t accf0 = empty0 + 8 * MX_STAGES, acce = accf0 + 16;
    const uint32_t sff0 = acce + 8, sfe0 = sff0 + 16, drain = sfe0 + 16;

    if (threadIdx.x == 0) {
        for (int s = 0; s < MX_STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(sff0 + 8 * b, 8);   // four scale warps of each CTA
            mbar_init(sfe0 + 8 * b, 1);
        }
        mbar_init(acce, 8);               // four epilogue warps of each CTA
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&a.mapA);
        prefetch_tmap(&a.mapB);
        if (a.tma_d) prefetch_tmap(&a.mapD);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();   // both CTAs' barriers exist before any remote signal
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        produce<MX_STAGES>(a, rank, unit, num_units, sA, sB, full0, empty0, abort_flag);
    } else if (warp == 1) {
        if (rank == 0) {
            int stage = 0, sf = 0, it = 0;
            uint32_t phase = 0, sf_phase = 0;
            bool ok = true, any = false;
            for (int item = unit; ok && item < a.num_items; item += num_units, ++it) {
                const uint32_t idesc0 = item < a.whole ? a.idesc : a.idesc_part;
                // the previous tile's epilogue has read the columns the two share
                const bool freed =
                    it == 0 || mbar_wait(acce, static_cast<uint32_t>(it - 1) & 1u, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, freed)) {
                    if (lane == 0) raise_error(abort_flag);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + ((it & 1) ? MX_ACC1 : 0);
                for (int kb = 0; kb < a.num_kb; ++kb) {
                    const bool last = kb == a.num_kb - 1;
                    const bool go = ((kb & 3) != 0 || mbar_wait(sff0 + 8 * sf, sf_phase, abort_flag)) &&
                                    mbar_wait(full0 + 8 * stage, phase, abort_flag);
                    if (!__all_sync(0xFFFFFFFFu, go)) {
                        if (lane == 0) raise_error(abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t sfa = tmem + MX_SF + sf * MX_SF_STRIDE, sfb = sfa + 4;
                        const uint32_t idesc = idesc0 | static_cast<uint32_t>(kb & 3) << 4 |
                                               static_cast<uint32_t>(kb & 3) << 29;
                        const uint64_t ad = smem_desc_sw128(sA + stage * HALF);
                        const uint64_t bd = smem_desc_sw128(sB + stage * HALF);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)   // 32 bytes on: 2 in the descriptors' unit
                            mma_mxf8_pair(d, ad + 2 * k, bd + 2 * k, idesc, sfa, sfb, (kb | k) != 0);
                        mma_commit_pair(empty0 + 8 * stage, 0x3);
                        if ((kb & 3) == 3 || last) mma_commit_pair(sfe0 + 8 * sf, 0x3);
                        if (last) mma_commit_pair(accf0 + 8 * (it & 1), 0x3);
                    }
                    __syncwarp();
                    any = true;
                    if (++stage == MX_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (((kb & 3) == 3 || last) && ++sf == 2) {
                        sf = 0;
                        sf_phase ^= 1u;
                    }
                }
            }
            if (!ok && any) {
                // wait (bounded) for the MMAs in flight before TMEM is freed
                if (elect_one()) mma_commit_pair(drain, 0x1);
                __syncwarp();
                mbar_wait(drain, 0, nullptr, 100000000ull);
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // scales: every lane fetches its word of each 32 rows; rows past the end
        // repeat the last one (their codes are zeros and their results are not stored)
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + MX_SF;
        const uint8_t *pa = static_cast<const uint8_t *>(a.A.scales);
        const uint8_t *pb = static_cast<const uint8_t *>(a.B.scales);
        int sf = 0;
        uint32_t sf_phase = 0;
        bool ok = true;
        for (int item = unit; ok && item < a.num_items; item += num_units) {
            const Item t = item_at(a, item);
            const uint8_t *ra[4], *rb[8];   // of a piece the first B words are used
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t r = min(t.row0 + rank * BM + 32 * j + lane, a.M - 1);
                ra[j] = pa + (a.A.block_rows == 1 ? r : r >> 7) * a.A.ld_s;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t r = min(t.col0 + 32 * j + lane, a.N - 1);
                rb[j] = pb + (a.B.block_rows == 1 ? r : r >> 7) * a.B.ld_s;
            }
            for (int kb = 0; kb < a.num_kb; kb += 4) {
                uint32_t wa[4], wb[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) wa[j] = *reinterpret_cast<const uint32_t *>(ra[j] + kb);
#pragma unroll
                for (int j = 0; j < 8; ++j) wb[j] = *reinterpret_cast<const uint32_t *>(rb[j] + kb);
                const bool got = mbar_wait(sfe0 + 8 * sf, sf_phase ^ 1u, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    if (lane == 0) raise_error(abort_flag);
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_store_4cols(lane_base + sf * MX_SF_STRIDE, wa[0], wa[1], wa[2], wa[3]);
                tmem_store_8cols(lane_base + sf * MX_SF_STRIDE + 4, wb);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(sff0 + 8 * sf, 0));
                if (++sf == 2) {
                    sf = 0;
                    sf_phase ^= 1u;
                }
            }
        }
        // the last releases come from the even SM: let them arrive
        for (int i = 0; ok && i < 2; ++i) {
            mbar_wait(sfe0 + 8 * sf, sf_phase ^ 1u, abort_flag);
            if (++sf == 2) {
                sf = 0;
                sf_phase ^= 1u;
            }
        }
    } else if (warp >= 8) {
        const int q = warp & 3;   // TMEM lane quarter
        uint32_t chunk = 0;       // chunks staged so far (selects the buffer)
        int it = 0;
        for (int item = unit; item < a.num_items; item += num_units, ++it) {
            const Item tile = item_at(a, item);
            const bool got = mbar_wait(accf0 + 8 * (it & 1), static_cast<uint32_t>(it >> 1) & 1u, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) {
                if (lane == 0) raise_error(abort_flag);
                break;
            }
            tc_fence_after();
            const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + ((it & 1) ? MX_ACC1 : 0);
            const int64_t row0 = tile.row0 + rank * BM + q * 32;
            const int chunks_here = tile.width / EPI_COLS;
#pragma unroll 1
            for (int i = 0; i < chunks_here; ++i) {
                const int c = (it & 1) ? i : chunks_here - 1 - i;   // the shared columns first
                uint32_t r[2][32];
                tmem_load_32cols(t + c * EPI_COLS, r[0]);
                tmem_load_32cols(t + c * EPI_COLS + 32, r[1]);
                if (i == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(acce, 0));
                }
                uint32_t packed[32];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        packed[16 * h + j] = pack2<__nv_bfloat16>(__uint_as_float(r[h][2 * j]),
                                                                  __uint_as_float(r[h][2 * j + 1]));
                // this buffer's previous store (two chunks back) has read it
                if (lane == 0) bulk_wait_group_read<1>();
                __syncwarp();
                const uint32_t sbuf = sD + (q * 2 + (chunk & 1)) * EPI_BUF;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_shared_v4(sbuf + lane * 128 + ((j ^ (lane & 7)) << 4), packed[4 * j],
                                 packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                store_chunk(a, sbuf, row0, tile.col0 + c * EPI_COLS);
                ++chunk;
            }
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();   // the other SM is done with this CTA's memory
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
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

// ----------------------------------------------------------------- f32 kernel --
// Warps: 0 TMA, 1 MMA (2 and 3 idle), 4-11 sums: warp w has lane quarter w mod 4 and
// half (w - 4) / 4 of the item's columns, 128 sums per thread.  Each k-block's MMAs
// start a fresh accumulator in one of two TMEM buffers; while one is summed the other
// is computed.  Of the launch's 384 x 168 registers the first four warps hand back
// 96 each per thread and the eight summing warps take 48 more: 128 x 72 + 256 x 216.
//
// The scales of four k-blocks at a time go through shared memory.  A thread reads the
// accumulator as 16 lanes x 256 bits: it holds 4 rows and 32 columns of the warp's
// 32 x 128, so that it needs 4 scales of A and 32 of B.  (With one row per thread,
// it needs 128 of B, and their 128 x 32 lanes x 4 bytes from shared memory took twice
// the MMAs' time.)  PER_ROW: B has one scale per row; otherwise the 128 columns of a
// warp share one.
//
// Bound by TMEM: MMAs that accumulate and the sums' reads share it, and a k-block takes
// some 1300 cycles where its MMAs alone take 512.  8192 x 11008 x 4096 with tiles of B:
// 465 us, 1590 TFLOP/s; 4096 x 11008 x 8192 with a scale per row of B, which costs each
// sum a multiplication more: 512 us, 1440 TFLOP/s.

constexpr int FS_STAGES = 5;
constexpr int FS_THREADS = 384;
constexpr int FS_REGS_CONTROL = 72, FS_REGS_SUMS = 216;
static_assert(128 * FS_REGS_CONTROL + 256 * FS_REGS_SUMS <= FS_THREADS * 168, "register split");
constexpr int FS_BARS = 2 * FS_STAGES + 4 + 1;
// B's scales of a k-block: per half of the columns and lane class (columns 8 j + 2 c,
// + 1 of class c) 32 floats, padded by 16 bytes so that the four classes' reads fall
// into different banks.
constexpr int FS_CLASS = 36, FS_SB = 8 * FS_CLASS;
constexpr size_t FS_SMEM = 1024 + FS_STAGES * 2 * HALF + 8 * EPI_BUF + 8 * (FS_SB + BM) * 4 +
                           FS_BARS * 8 + 16;

// 16 lanes x 32 columns of a k-block's dot products, times their scales onto the sums; h / 2
// is the group of 32 columns, h mod 2 the half of the lanes.  LAST: the accumulator has
// been read.
template <bool PER_ROW>
__device__ __forceinline__ void add_step(int h, bool last, uint32_t t, const float *sbk,
                                         const uint64_t (&sa2)[4], uint64_t (&sb2)[4],
                                         uint32_t freed, uint64_t (&sum)[4][16]) {
    uint32_t v[16];
    tmem_load_16x256b_x4(t + (h >> 1) * 32 + (static_cast<uint32_t>(h & 1) << 20), v);
    if (PER_ROW && (h & 1) == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(sbk + (h >> 1) * 8 + 4 * j);
            sb2[2 * j] = u.x, sb2[2 * j + 1] = u.y;
        }
    }
    tmem_wait_16cols(v);
    if (last) {
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive_cluster_relaxed(mapa_shared(freed, 0));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t x = f32x2_pack(__uint_as_float(v[4 * j + 2 * i]),
                                          __uint_as_float(v[4 * j + 2 * i + 1]));
            const uint64_t s1 = sa2[2 * (h & 1) + i];
            uint64_t &to = sum[2 * (h & 1) + i][4 * (h >> 1) + j];
            to = f32x2_fma(x, PER_ROW ? f32x2_mul(s1, sb2[j]) : s1, to);
        }
    }
}

// A warp's share of a k-block: 128 columns, or 32 of a piece.
template <bool PER_ROW>
__device__ __forceinline__ void add_block(uint32_t t, const float *sbk, const uint64_t (&sa2)[4],
                                          uint32_t freed, bool whole, uint64_t (&sum)[4][16]) {
    uint64_t sb2[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) add_step<PER_ROW>(h, false, t, sbk, sa2, sb2, freed, sum);
    if (whole) {
#pragma unroll
        for (int h = 2; h < 8; ++h) add_step<PER_ROW>(h, h == 7, t, sbk, sa2, sb2, freed, sum);
    } else {
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive_cluster_relaxed(mapa_shared(freed, 0));
    }
}

template <bool PER_ROW>
__global__ void __launch_bounds__(FS_THREADS, 1)
    block_gemm_f32_kernel(const __grid_constant__ PairArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sA = smem_u32(smem), sB = sA + FS_STAGES * HALF;
    const uint32_t sD = sB + FS_STAGES * HALF;
    float *sbs = reinterpret_cast<float *>(smem + FS_STAGES * 2 * HALF + 8 * EPI_BUF);   // [8][FS_SB]
    float *sas = sbs + 8 * FS_SB;                                                        // [8][BM]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sas + 8 * BM);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + FS_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int unit = static_cast<int>(blockIdx.x >> 1), num_units = static_cast<int>(gridDim.x >> 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * FS_STAGES;
    const uint32_t accf0 = empty0 + 8 * FS_STAGES, acce0 = accf0 + 16, drain = acce0 + 16;

    if (threadIdx.x == 0) {
        for (int s = 0; s < FS_STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, 16);   // eight warps of each CTA
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&a.mapA);
        prefetch_tmap(&a.mapB);
        if (a.tma_d) prefetch_tmap(&a.mapD);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FS_REGS_CONTROL));
        if (warp == 0) {
            produce<FS_STAGES>(a, rank, unit, num_units, sA, sB, full0, empty0, abort_flag);
        } else if (warp == 1 && rank == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, any = false;
            for (int item = unit; ok && item < a.num_items; item += num_units) {
                const uint32_t idesc = item < a.whole ? a.idesc : a.idesc_part;
                for (int kb = 0; kb < a.num_kb; ++kb) {
                    const bool go = mbar_wait(acce0 + 8 * acc, acc_phase ^ 1u, abort_flag) &&
                                    mbar_wait(full0 + 8 * stage, phase, abort_flag);
                    if (!__all_sync(0xFFFFFFFFu, go)) {
                        if (lane == 0) raise_error(abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = smem_desc_sw128(sA + stage * HALF);
                        const uint64_t bd = smem_desc_sw128(sB + stage * HALF);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            mma_f8f6f4_pair(tmem + acc * BN, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                        mma_commit_pair(empty0 + 8 * stage, 0x3);
                        mma_commit_pair(accf0 + 8 * acc, 0x3);
                    }
                    __syncwarp();
                    any = true;
                    if (++stage == FS_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
            }
            if (!ok && any) {
                if (elect_one()) mma_commit_pair(drain, 0x1);
                __syncwarp();
                mbar_wait(drain, 0, nullptr, 100000000ull);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FS_REGS_SUMS));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int et = threadIdx.x - 128;   // 0..255: the column (and row) whose scales it fetches
        const uint32_t sbuf = sD + (warp - 4) * EPI_BUF;
        const int my_cols = half * 4 * FS_CLASS + (lane & 3) * FS_CLASS;
        const int my_row = q * 32 + (lane >> 2);
        uint32_t n = 0;   // k-blocks so far: accumulator n mod 2
        bool ok = true;
        for (int item = unit; ok && item < a.num_items; item += num_units) {
            const int hw = item < a.whole ? 128 : 32;   // columns of a half of the item
            const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * hw;
            const int own_col = (et >= hw ? 4 * FS_CLASS : 0) + ((et >> 1) & 3) * FS_CLASS +
                                ((et & (hw - 1)) >> 3) * 2 + (et & 1);
            const bool has_col = et < 2 * hw;
            // rows and columns past the end repeat the last one
            ScaleStream fa, fb;
            {
                const Item tile = item_at(a, item);
                if (et < BM) fa.start(a.A, min(tile.row0 + rank * BM + et, a.M - 1), 0, a.num_kb);
                fb.start(a.B, min(tile.col0 + et, a.N - 1), 0, a.num_kb);
            }
            uint64_t sum[4][16];   // [row lane / 4 + 8 i][columns 8 j + 2 (lane mod 4), + 1]
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[i][j] = 0;
#pragma unroll 1
            for (int kb = 0; kb < a.num_kb; ++kb) {
                if ((kb & 3) == 0) {
                    // the scales of four k-blocks; they are written over eight blocks
                    // later, with a barrier in between
                    if (et < BM) {
                        fa.take();
                        fa.fetch((kb >> 2) + 1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sas[((kb & 7) + i) * BM + et] = fa.cur[i];
                    }
                    fb.take();
                    fb.fetch((kb >> 2) + 1);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (has_col) sbs[((kb & 7) + i) * FS_SB + own_col] = fb.cur[i];
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
                const float *sbk = sbs + (kb & 7) * FS_SB + my_cols;
                const float *sak = sas + (kb & 7) * BM + my_row;
                const bool got = mbar_wait(accf0 + 8 * (n & 1), (n >> 1) & 1u, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    if (lane == 0) raise_error(abort_flag);
                    ok = false;   // goes on to this tile's end, where all agree to stop
                }
                uint64_t sa2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sa2[i] = splat_f32x2(PER_ROW ? sak[8 * i] : __fmul_rn(sak[8 * i], sbk[0]));
                if (ok) {
                    tc_fence_after();
                    add_block<PER_ROW>(t0 + (n & 1) * BN, sbk, sa2, acce0 + 8 * (n & 1), item < a.whole, sum);
                }
                ++n;
            }
            // all have read the last scales before the next tile's are written, and all
            // go on or none: a warp alone in the next tile's barriers would stay there
            ok = barrier_and(1, 256, ok);
            if (ok) {
                const Item tile = item_at(a, item);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c * EPI_COLS >= hw) break;
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float lo, hi;
                            f32x2_unpack(sum[i][8 * c + j], lo, hi);
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(
                                             sbuf + ((lane >> 2) + 8 * i) * 128 +
                                             ((j ^ (lane >> 2)) << 4) + (lane & 3) * 4),
                                         "r"(pack2<__nv_bfloat16>(lo, hi))
                                         : "memory");
                        }
                    }
                    store_chunk(a, sbuf, tile.row0 + rank * BM + q * 32, tile.col0 + half * hw + c * EPI_COLS,
                                min(hw, EPI_COLS));
                }
            }
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ----------------------------------------------------------------- few kernel --
// A CTA computes 128 rows of B (weights) times NT rows of A (tokens) over its share
// of the k-blocks; gridDim.x CTAs, a cluster, share a tile's k-blocks.  Warps: 0 TMA,
// 1 MMA, the others (thread = weight row) by the scales' type:
//   E8M0 (MX): four warps bring the scales to TMEM as in the mx kernel, and the sums
//        back from it at the end;
//   float: as in the f32 kernel, each warp with one lane quarter and, of eight warps,
//        half of the tokens (16 tokens: four warps and all of them), with several
//        accumulators, so that the MMAs run ahead of the sums.
// Shared memory and TMEM allow two CTAs per SM, so that one's start and end overlap the
// other's loads.  One SM alone reads some 65 GB/s whatever its ring holds, so K is split
// until all SMs read: 1 x 4096 x 4096 took 13.4 us unsplit and 6.8 in 8 parts (5.5 since
// the MMA warp issues as one).  The join costs more with more tokens: 128 x 11008 x 4096
// takes 18.9 us unsplit and 19.1 in 3 parts, and a tile of 128 tokens is not split.

template <int NT, bool MX>
struct Few {
    static constexpr int X_STAGE = NT * BK;
    static constexpr int STAGES = NT <= 32 ? 5 : NT <= 64 ? 4 : 3;
    static constexpr int ACCS = MX ? 1 : NT <= 32 ? 8 : 256 / NT;
    static constexpr int MOST_SPLITS = 8;
    static constexpr int WARPS = MX || NT <= 16 ? 4 : 8;   // beside TMA and MMA
    static constexpr int THREADS = 64 + 32 * WARPS;
    static constexpr int COLS = NT * 4 / WARPS;            // tokens per warp
    static constexpr int SF = NT;                          // MX: first TMEM column of the scales,
    static constexpr int SF_STRIDE = 8;                    // per stage 4 for weights, 4 for tokens
    static constexpr int TMEM = MX ? 2 * NT : ACCS * NT;   // columns, a power of two of at least 32
    static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 4 + 1;
    static constexpr size_t SMEM =
        1024 + STAGES * (HALF + X_STAGE) + 2 * NT * 4 + NUM_BARS * 8 + 16;
    static_assert(STAGES * (HALF + X_STAGE) >= NT * 128 * 4, "the sums fit where the tiles were");
    static_assert(!MX || SF + 2 * SF_STRIDE <= TMEM, "the scales fit");
};

struct FewArgs {
    CUtensorMap mapW, mapX;   // B's rows (128 x 128 boxes) and A's (128 x NT)
    BlockView W, X;
    __nv_bfloat16 *D;
    int64_t M, N, ldd;
    int num_kb;
    uint32_t idesc;
};

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int NT, bool MX>
__global__ void __launch_bounds__(Few<NT, MX>::THREADS, NT <= 64 ? 2 : 1)
    block_gemm_few_kernel(const __grid_constant__ FewArgs a) {
    using C = Few<NT, MX>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sW = smem_u32(smem), sX = sW + C::STAGES * HALF;
    float *sxs = reinterpret_cast<float *>(smem + C::STAGES * (HALF + C::X_STAGE));   // [2][NT]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sxs + 2 * NT);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t accf0 = empty0 + 8 * C::STAGES, acce0 = accf0 + 8 * C::ACCS;
    const uint32_t sff0 = acce0 + 8 * C::ACCS, sfe0 = sff0 + 16, drain = sfe0 + 16;
    const int splits = static_cast<int>(gridDim.x), split = static_cast<int>(blockIdx.x);
    const int kb0 = static_cast<int>(static_cast<int64_t>(a.num_kb) * split / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(a.num_kb) * (split + 1) / splits);
    const int32_t wrow0 = static_cast<int32_t>(blockIdx.y) * 128;
    const int32_t xrow0 = static_cast<int32_t>(blockIdx.z) * NT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < C::ACCS; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, C::WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sff0 + 8 * b, 4);
            mbar_init(sfe0 + 8 * b, 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&a.mapW);
        prefetch_tmap(&a.mapX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    const int q = warp & 3, part = (warp - 2) >> 2;   // lane quarter, share of the tokens
    uint64_t sum[C::COLS / 2] = {};                   // pairs of tokens
    bool ok = true;
    if (warp == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag))) {
                if (lane == 0) raise_error(abort_flag);
                ok = false;
                break;
            }
            if (elect_one()) {
                const uint32_t fb = full0 + 8 * stage;
                mbar_arrive_expect_tx(fb, HALF + C::X_STAGE);
                tma_load_2d(sW + stage * HALF, &a.mapW, fb, kb * BK, wrow0);
                tma_load_2d(sX + stage * C::X_STAGE, &a.mapX, fb, kb * BK, xrow0);
            }
            __syncwarp();
            ++issued;
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {
            // let the copies already issued land before the CTA exits
            for (int i = 0; i < C::STAGES && issued > 0; ++i, --issued) {
                stage = stage == 0 ? C::STAGES - 1 : stage - 1;
                if (stage == C::STAGES - 1) phase ^= 1u;
                mbar_wait(full0 + 8 * stage, phase, nullptr, 100000000ull);
            }
        }
    } else if (warp == 1) {
        int stage = 0, acc = 0, sf = 0;
        uint32_t phase = 0, acc_phase = 0, sf_phase = 0;
        bool any = false;
        for (int kb = kb0; kb < kb1; ++kb) {
            // MX: a stage of scales holds those of four k-blocks, from a multiple of 4 on
            const bool first = MX ? kb == kb0 || (kb & 3) == 0 : true;
            const uint32_t ready = MX ? sff0 + 8 * sf : acce0 + 8 * acc;
            const bool go = (!first || mbar_wait(ready, MX ? sf_phase : acc_phase ^ 1u, abort_flag)) &&
                            mbar_wait(full0 + 8 * stage, phase, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, go)) {
                if (lane == 0) raise_error(abort_flag);
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t wd = smem_desc_sw128(sW + stage * HALF);
                const uint64_t xd = smem_desc_sw128(sX + stage * C::X_STAGE);
#pragma unroll
                for (int k = 0; k < BK / 32; ++k) {   // 32 bytes on: 2 in the descriptors' unit
                    if constexpr (MX) {
                        const uint32_t id = static_cast<uint32_t>(kb & 3);
                        mma_mxf8(tmem, wd + 2 * k, xd + 2 * k, a.idesc | id << 4 | id << 29,
                                 tmem + C::SF + sf * C::SF_STRIDE, tmem + C::SF + sf * C::SF_STRIDE + 4,
                                 kb != kb0 || k != 0);
                    } else {
                        mma_f8f6f4(tmem + acc * NT, wd + 2 * k, xd + 2 * k, a.idesc, k != 0);
                    }
                }
                mma_commit(empty0 + 8 * stage);
                if (MX && (kb & 3) == 3) mma_commit(sfe0 + 8 * sf);
                if (!MX) mma_commit(accf0 + 8 * acc);
                if (MX && kb == kb1 - 1) mma_commit(accf0);
            }
            __syncwarp();
            any = true;
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if (MX && (kb & 3) == 3 && ++sf == 2) {
                sf = 0;
                sf_phase ^= 1u;
            }
            if (!MX && ++acc == C::ACCS) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (!ok && any) {
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            mbar_wait(drain, 0, nullptr, 100000000ull);
        }
    } else if constexpr (MX) {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        // rows past the end repeat the last one
        const uint8_t *pw[4], *px[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t w = min(static_cast<int64_t>(wrow0) + 32 * j + lane, a.N - 1);
            const int64_t x = min(static_cast<int64_t>(xrow0) + 32 * j + lane, a.M - 1);
            pw[j] = static_cast<const uint8_t *>(a.W.scales) + (a.W.block_rows == 1 ? w : w >> 7) * a.W.ld_s;
            px[j] = static_cast<const uint8_t *>(a.X.scales) + (a.X.block_rows == 1 ? x : x >> 7) * a.X.ld_s;
        }
        uint32_t ww[4], wx[4] = {0, 0, 0, 0};
        auto fetch = [&](int kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ww[j] = *reinterpret_cast<const uint32_t *>(pw[j] + kb);
                if (32 * j < NT) wx[j] = *reinterpret_cast<const uint32_t *>(px[j] + kb);
            }
        };
        int sf = 0;
        uint32_t sf_phase = 0;
        if (kb0 < kb1) fetch(kb0 & ~3);
        for (int kb = kb0 & ~3; kb < kb1; kb += 4) {
            const uint32_t sw[4] = {ww[0], ww[1], ww[2], ww[3]}, sx[4] = {wx[0], wx[1], wx[2], wx[3]};
            if (kb + 4 < kb1) fetch(kb + 4);
            const bool got = mbar_wait(sfe0 + 8 * sf, sf_phase ^ 1u, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) {
                if (lane == 0) raise_error(abort_flag);
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t at = lanes + C::SF + sf * C::SF_STRIDE;
            tmem_store_4cols(at, sw[0], sw[1], sw[2], sw[3]);
            tmem_store_4cols(at + 4, sx[0], sx[1], sx[2], sx[3]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sff0 + 8 * sf);
            if (++sf == 2) {
                sf = 0;
                sf_phase ^= 1u;
            }
        }
        const bool got = kb0 < kb1 && ok && mbar_wait(accf0, 0, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
            if (lane == 0 && kb0 < kb1) raise_error(abort_flag);
            ok = false;
        }
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < NT / 16; ++h) {
                uint32_t r[16];
                tmem_load_16cols(lanes + h * 16, r);
                tmem_wait_16cols(r);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    sum[8 * h + c] = f32x2_pack(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
            }
            tc_fence_before();
        }
    } else {
        const int et = threadIdx.x - 64;
        const int64_t w = min(static_cast<int64_t>(wrow0) + q * 32 + lane, a.N - 1);
        const int64_t x = min(static_cast<int64_t>(xrow0) + et, a.M - 1);
        int acc = 0;
        uint32_t acc_phase = 0;
        ScaleStream fw, fx;
        fw.start(a.W, w, kb0, kb1);
        fx.start(a.X, x, kb0, kb1);
#pragma unroll 1
        for (int kb = kb0; kb < kb1; ++kb) {
            const float sw = fw.next(kb), sx_own = fx.next(kb);
            float *sx = sxs + ((kb - kb0) & 1) * NT;
            if (et < NT) sx[et] = sx_own;
            // a buffer is written again only after the next block's barrier
            asm volatile("bar.sync 1, %0;" ::"n"(32 * C::WARPS) : "memory");
            const bool got = mbar_wait(accf0 + 8 * acc, acc_phase, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) {
                if (lane == 0) raise_error(abort_flag);
                ok = false;   // the others give up in the same wait
            }
            if (ok) {
                tc_fence_after();
                const uint32_t t =
                    tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * NT + part * C::COLS;
                uint32_t r[2][16];
                tmem_load_16cols(t, r[0]);
                const uint64_t sw2 = splat_f32x2(sw);
#pragma unroll
                for (int h = 0; h < C::COLS / 16; ++h) {
                    tmem_wait_16cols(r[h & 1]);
                    if (h < C::COLS / 16 - 1) {
                        tmem_load_16cols(t + (h + 1) * 16, r[(h + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acce0 + 8 * acc);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const ulonglong2 s2 = *reinterpret_cast<const ulonglong2 *>(
                            sx + part * C::COLS + 16 * h + 4 * c);
                        const uint32_t *v = r[h & 1] + 4 * c;
                        uint64_t *to = sum + 8 * h + 2 * c;
                        to[0] = f32x2_fma(f32x2_pack(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                          f32x2_mul(sw2, s2.x), to[0]);
                        to[1] = f32x2_fma(f32x2_pack(__uint_as_float(v[2]), __uint_as_float(v[3])),
                                          f32x2_mul(sw2, s2.y), to[1]);
                    }
                }
            }
            if (++acc == C::ACCS) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    const int tokens = a.M - xrow0 < NT ? static_cast<int>(a.M - xrow0) : NT;
    const int r = q * 32 + lane;
    const int64_t n = static_cast<int64_t>(wrow0) + r;
    __nv_bfloat16 *d = a.D + static_cast<int64_t>(xrow0) * a.ldd + n;
    if (splits == 1) {
        if (warp >= 2 && ok && n < a.N) {
#pragma unroll
            for (int c = 0; c < C::COLS / 2; ++c) {
                const int token = part * C::COLS + 2 * c;
                float lo, hi;
                f32x2_unpack(sum[c], lo, hi);
                if (token < tokens) d[token * a.ldd] = __float2bfloat16_rn(lo);
                if (token + 1 < tokens) d[(token + 1) * a.ldd] = __float2bfloat16_rn(hi);
            }
        }
    } else {
        // sums [token][weight row] in the shared memory that held the tiles: all MMAs
        // that read it are done
        float *red = reinterpret_cast<float *>(smem);
        __syncthreads();
        if (warp >= 2) {
#pragma unroll
            for (int c = 0; c < C::COLS / 2; ++c) {
                const int token = part * C::COLS + 2 * c;
                float lo, hi;
                f32x2_unpack(sum[c], lo, hi);
                if (token < tokens) red[token * 128 + r] = lo;
                if (token + 1 < tokens) red[(token + 1) * 128 + r] = hi;
            }
        }
        __syncwarp();
        cluster_sync();
        // CTA k of the cluster joins tokens k, k + splits, ...  A read from another SM
        // takes about a microsecond, so those of four tokens and all splits go out
        // together.  (Writing the sums to the joining SM's memory instead is as fast for
        // 16 tokens and slower for more; bulk copies are slower throughout.)
        if (warp >= 2 && n < a.N) {
            constexpr int U = 4;
            const int step = splits * (C::WARPS / 4);
            for (int c0 = split + part * splits; c0 < tokens; c0 += U * step) {
                float v[U][C::MOST_SPLITS];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < C::MOST_SPLITS; ++k)
                        v[u][k] = k < splits && c0 + u * step < tokens
                                      ? ld_shared_cluster(mapa_shared(
                                            smem_u32(red + (c0 + u * step) * 128 + r),
                                            static_cast<uint32_t>(k)))
                                      : 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float s = 0.0f;   // in the order of the splits
#pragma unroll
                    for (int k = 0; k < C::MOST_SPLITS; ++k) s = __fadd_rn(s, v[u][k]);
                    if (c0 + u * step < tokens) d[(c0 + u * step) * a.ldd] = __float2bfloat16_rn(s);
                }
            }
        }
        __syncwarp();
        cluster_sync();   // the others have read this CTA's sums
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// --------------------------------------------------------------------- host --

// attr must have room for two attributes: the cluster shape and PDL.
cudaLaunchConfig_t cluster_config(dim3 grid, int threads, size_t smem, int cluster,
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
struct PairKernel {
    void (*kernel)(PairArgs);
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
PairKernel g_mx{block_gemm_mx_kernel, MX_THREADS, MX_SMEM};
PairKernel g_f32_tiles{block_gemm_f32_kernel<false>, FS_THREADS, FS_SMEM};
PairKernel g_f32_rows{block_gemm_f32_kernel<true>, FS_THREADS, FS_SMEM};

template <int NT, bool MX>
cudaError_t launch_few(const BlockView &A, const BlockView &B, const MatView &D, int sm_count,
                       cudaStream_t st, const char **what) {
    using C = Few<NT, MX>;
    FewArgs a;
    if (!encode_tmap_2d(&a.mapW, B.codes, false, B.cols, B.rows, BK, 128, true, B.ld) ||
        !encode_tmap_2d(&a.mapX, A.codes, false, A.cols, A.rows, BK, NT, true, A.ld)) {
        *what = "cuTensorMapEncodeTiled failed for an operand";
        return cudaErrorInvalidValue;
    }
    a.W = B;
    a.X = A;
    a.D = static_cast<__nv_bfloat16 *>(D.data);
    a.M = D.rows;
    a.N = D.cols;
    a.ldd = D.ld;
    a.num_kb = static_cast<int>((A.cols + BK - 1) / BK);
    const uint32_t fw = static_cast<uint32_t>(B.fmt), fx = static_cast<uint32_t>(A.fmt);
    a.idesc = MX ? idesc_mxf8(fw, fx, 128, NT, 0) : idesc_f8(fw, fx, 128, NT);
    static SmemLimit limit;
    const cudaError_t attr_err = limit.allow(block_gemm_few_kernel<NT, MX>, C::SMEM);
    if (attr_err != cudaSuccess) return attr_err;
    const int64_t tw = (D.cols + 127) / 128, tx = (D.rows + NT - 1) / NT;
    // as many CTAs as run at once, two per SM, with at least two k-blocks each
    int64_t splits = 2 * sm_count / (tw * tx);
    if (NT > 64 && tw * tx > sm_count / 2) splits = 1;   // the join costs more than it saves
    if (splits > a.num_kb / 2) splits = a.num_kb / 2;
    if (splits > C::MOST_SPLITS) splits = C::MOST_SPLITS;
    if (splits < 1) splits = 1;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg =
        cluster_config(dim3(static_cast<unsigned>(splits), static_cast<unsigned>(tw), static_cast<unsigned>(tx)),
                       C::THREADS, C::SMEM,
                       static_cast<int>(splits), attr, st);
    return cudaLaunchKernelEx(&cfg, block_gemm_few_kernel<NT, MX>, a);
}

template <bool MX>
cudaError_t launch_few_any(const BlockView &A, const BlockView &B, const MatView &D, int sm_count,
                           cudaStream_t st, const char **what) {
    if (D.rows <= 16) return launch_few<16, MX>(A, B, D, sm_count, st, what);
    if (D.rows <= 32) return launch_few<32, MX>(A, B, D, sm_count, st, what);
    if (D.rows <= 64) return launch_few<64, MX>(A, B, D, sm_count, st, what);
    return launch_few<128, MX>(A, B, D, sm_count, st, what);
}

// The few kernel takes up to kFewRows rows of A, and more as long as its 128 x 128 tiles, four
// to a 256 x 256 tile, run at once: one for each SM.  On 152 SMs that is up to 38 tiles.  Float
// scales, K = 4096, M x N, few and pair kernel in us: 256 x 8192 (32 tiles) 26.0 and 28.3, 256
// x 9728 (38) 26.0 and 28.6, 256 x 10240 (40) 49.8 and 28.7; 256 x 4096 (16) 23.1 and 20.1.  E8M0
// scales: 13.9 and 13.3, at 38 tiles 20.4 and 19.2, at 1024 x 2048 (32) 18.6 and 14.9: there the
// pair kernel is ahead throughout, and the rule is the float scales'.
constexpr int64_t kFewRows = 128;
int64_t few_tiles(int sm_count) { return sm_count / 4; }
constexpr int64_t kFewCols = int64_t(65535) * 128;   // of D in one launch: tiles count in gridDim.y
constexpr int kMxPieceWaves = 6;

// The columns of D from c on, at most n of them, and the rows of B that give them.
void take_columns(BlockView &B, MatView &D, int64_t c, int64_t n) {
    B.codes += c * B.ld;
    B.scales = static_cast<uint8_t *>(B.scales) + c / B.block_rows * B.ld_s * (B.scale_f32 ? 4 : 1);
    D.data = static_cast<__nv_bfloat16 *>(D.data) + c;
    B.rows = D.cols = D.cols - c < n ? D.cols - c : n;
}

}  // namespace

cudaError_t launch_block_gemm(const BlockView &A, const BlockView &B, const MatView &D,
                              int sm_count, cudaStream_t st, const char **what) {
    if (D.rows == 0 || D.cols == 0) return cudaSuccess;
    if (A.cols == 0) return cudaMemset2DAsync(D.data, D.ld * 2, 0, D.cols * 2, D.rows, st);
    if (D.rows <= kFewRows && D.cols > kFewCols) {
        for (int64_t c = 0; c < D.cols; c += kFewCols) {
            BlockView part = B;
            MatView to = D;
            take_columns(part, to, c, kFewCols);
            const cudaError_t e = launch_block_gemm(A, part, to, sm_count, st, what);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    const bool mx = A.scale_f32 == 0;
    PairKernel &pk = mx ? g_mx : B.block_rows == 1 ? g_f32_rows : g_f32_tiles;
    const int64_t pair_tiles = ((D.rows + 255) / 256) * ((D.cols + 255) / 256);
    int slots = 0;
    if (D.rows > kFewRows && pair_tiles > few_tiles(sm_count)) {
        const cudaError_t e = pk.init(sm_count, &slots);
        if (e != cudaSuccess) return e;
    }
    if (slots < 1)
        return mx ? launch_few_any<true>(A, B, D, sm_count, st, what)
                  : launch_few_any<false>(A, B, D, sm_count, st, what);
    PairArgs a;
    a.tma_d = (reinterpret_cast<uintptr_t>(D.data) & 15u) == 0 && D.ld % 8 == 0;
    a.pairs_d = (reinterpret_cast<uintptr_t>(D.data) & 3u) == 0 && D.ld % 2 == 0;
    if (!encode_tmap_2d(&a.mapA, A.codes, false, A.cols, A.rows, BK, BM, true, A.ld) ||
        !encode_tmap_2d(&a.mapB, B.codes, false, B.cols, B.rows, BK, BN / 2, true, B.ld)) {
        *what = "cuTensorMapEncodeTiled failed for an operand";
        return cudaErrorInvalidValue;
    }
    if (a.tma_d && !encode_tmap_2d(&a.mapD, D.data, true, D.cols, D.rows, EPI_COLS, 32, true, D.ld)) {
        *what = "cuTensorMapEncodeTiled failed for the output";
        return cudaErrorInvalidValue;
    }
    a.A = A;
    a.B = B;
    a.D = static_cast<__nv_bfloat16 *>(D.data);
    a.M = D.rows;
    a.N = D.cols;
    a.ldd = D.ld;
    a.tiles_m = static_cast<int>((D.rows + 2 * BM - 1) / (2 * BM));
    a.tiles_n = static_cast<int>((D.cols + BN - 1) / BN);
    // The last wave in pieces.  With float scales it always pays (4096 x 11008 x 8192, 9
    // waves: 512 us, whole 530; 2304 x 2560 x 4096: 45.3 and 52.5).  The mx kernel runs into the power limit where there are
    // many waves, and the pairs that idle in the last one cost nothing (2304 x 2560 x 4096,
    // 1.2 waves: 25.7 us, whole 28.0; 4 waves 58.7 and 60.0; 8 waves 106.3 and 105.3).
    const int num_tiles = a.tiles_m * a.tiles_n, rest = num_tiles % slots;
    const bool pieces = kPieces * rest <= slots && (!mx || num_tiles < kMxPieceWaves * slots);
    a.whole = pieces ? num_tiles - rest : num_tiles;
    a.num_items = a.whole + (num_tiles - a.whole) * kPieces;
    a.num_kb = static_cast<int>((A.cols + BK - 1) / BK);
    a.group_m = raster_group(D.rows * A.cols, D.cols * A.cols, a.tiles_m);
    const uint32_t fa = static_cast<uint32_t>(A.fmt), fb = static_cast<uint32_t>(B.fmt);
    const auto idesc = [&](int n) {
        return mx ? idesc_mxf8(fa, fb, 2 * BM, n, 0) : idesc_f8(fa, fb, 2 * BM, n);
    };
    a.idesc = idesc(BN);
    a.idesc_part = idesc(BN / kPieces);
    if (!encode_tmap_2d(&a.mapBPart, B.codes, false, B.cols, B.rows, BK, BN / 2 / kPieces, true, B.ld)) {
        *what = "cuTensorMapEncodeTiled failed for an operand";
        return cudaErrorInvalidValue;
    }
    const int units = a.num_items < slots ? a.num_items : slots;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(dim3(2 * units), pk.threads, pk.smem, 2, attr, st);
    return cudaLaunchKernelEx(&cfg, pk.kernel, a);
}

cudaError_t read_and_clear_block_gemm_error_flag(unsigned *flags) {
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_block_gemm_error_flags, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_block_gemm_error_flags, &zero, sizeof(unsigned));
}

}  // namespace fp8k
