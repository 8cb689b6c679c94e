// block_gemm.cu -- FP8 matrix product with a scale for each block of 128, on the
// sm_103a tcgen05 tensor cores:
//   D[i][j] = bf16_rne( sum over k-blocks b of sA(i, b) * sB(j, b) * dot_b ),
//   dot_b = sum over the block's 128 columns of A[i][c] * B[j][c]   (fp32)
// A is [M][K], B [N][K], both contiguous along K; sA and sB belong to one row
// or to 128 rows, and are E8M0 bytes or floats.
//
// One CTA per SM, persistent over 128 x 128 output tiles:
//   warp 0     TMA producer: 128-byte-swizzled 128-deep slices of A and B;
//   warp 1     issues tcgen05.mma: each k-block's four MMAs start a fresh
//              accumulator in one of two TMEM buffers;
//   warps 2-5  read each finished dot_b from TMEM and add it, times its scale,
//              to sums in registers; after the last k-block they round and
//              store the tile.
// Every wait is bounded.
#include <cstdint>
#include <mutex>

#include "block.cuh"

namespace fp8k {

namespace {

__device__ unsigned g_block_gemm_error_flags = 0;

constexpr int BM = 128, BN = 128, BK = 128;
constexpr int STAGES = 6;
constexpr int NUM_THREADS = 192;
constexpr int A_STAGE = BM * BK, B_STAGE = BN * BK;
constexpr int TMEM_COLS = 2 * BN;
constexpr int NUM_BARS = 2 * STAGES + 4 + 1;
constexpr size_t SMEM =
    1024 + STAGES * (A_STAGE + B_STAGE) + 2 * BN * sizeof(float) + NUM_BARS * 8 + 16;

struct Args {
    CUtensorMap mapA, mapB;
    BlockView A, B;
    __nv_bfloat16 *D;
    int64_t M, N, ldd;
    bool vecd;
    int tiles_n, num_tiles, num_kb;
    uint32_t idesc;
};

__device__ __forceinline__ void raise_error(volatile int *abort_flag) {
    atomicOr(&g_block_gemm_error_flags, kErrWaitTimeout);
    *abort_flag = 1;
}

__global__ void __launch_bounds__(NUM_THREADS, 1) block_gemm_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sA = smem;
    uint8_t *sB = smem + STAGES * A_STAGE;
    float *sbs = reinterpret_cast<float *>(sB + STAGES * B_STAGE);   // [2][BN] scales of B
    uint64_t *bars = reinterpret_cast<uint64_t *>(sbs + 2 * BN);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
    const uint32_t accf0 = smem_u32(bars + 2 * STAGES), acce0 = smem_u32(bars + 2 * STAGES + 2);
    const uint32_t drain_bar = smem_u32(bars + 2 * STAGES + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, 4);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&a.mapA);
        prefetch_tmap(&a.mapB);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < a.num_tiles; tile += gridDim.x) {
                const int mb = tile / a.tiles_n, nb = tile % a.tiles_n;
                for (int kb = 0; kb < a.num_kb; ++kb) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
                        raise_error(abort_flag);
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * stage;
                    mbar_arrive_expect_tx(fb, A_STAGE + B_STAGE);
                    tma_load_2d(smem_u32(sA + stage * A_STAGE), &a.mapA, fb, kb * BK, mb * BM);
                    tma_load_2d(smem_u32(sB + stage * B_STAGE), &a.mapB, fb, kb * BK, nb * BN);
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // let the copies already issued land before the CTA exits
                for (int i = 0; i < STAGES && issued > 0; ++i, --issued) {
                    stage = stage == 0 ? STAGES - 1 : stage - 1;
                    if (stage == STAGES - 1) phase ^= 1u;
                    mbar_wait(full0 + 8 * stage, phase, nullptr, 100000000ull);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, any = false;
            for (int tile = blockIdx.x; ok && tile < a.num_tiles; tile += gridDim.x) {
                for (int kb = 0; kb < a.num_kb; ++kb) {
                    if (!mbar_wait(acce0 + 8 * acc, acc_phase ^ 1u, abort_flag) ||
                        !mbar_wait(full0 + 8 * stage, phase, abort_flag)) {
                        raise_error(abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(sA + stage * A_STAGE);
                    const uint32_t b0 = smem_u32(sB + stage * B_STAGE);
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_f8f6f4(tmem_base + acc * BN, smem_desc_sw128(a0 + 32 * k),
                                   smem_desc_sw128(b0 + 32 * k), a.idesc, k != 0);
                    mma_commit(empty0 + 8 * stage);
                    mma_commit(accf0 + 8 * acc);
                    any = true;
                    if (++stage == STAGES) {
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
                mma_commit(drain_bar);
                mbar_wait(drain_bar, 0, nullptr, 100000000ull);
            }
        }
    } else {
        const int q = warp & 3;             // TMEM lane quarter this warp may access
        const int et = threadIdx.x - 64;    // 0..127: the column whose scale this thread fetches
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < a.num_tiles; tile += gridDim.x) {
            const int mb = tile / a.tiles_n, nb = tile % a.tiles_n;
            const int64_t row = static_cast<int64_t>(mb) * BM + q * 32 + lane;
            const int64_t col = static_cast<int64_t>(nb) * BN + et;
            const int64_t ra = row < a.M ? row / a.A.block_rows : 0;
            const int64_t rb = col < a.N ? col / a.B.block_rows : 0;
            float sum[BN];
#pragma unroll
            for (int c = 0; c < BN; ++c) sum[c] = 0.0f;
            float sa_next = load_scale(a.A, ra, 0), sb_next = load_scale(a.B, rb, 0);
#pragma unroll 1
            for (int kb = 0; kb < a.num_kb; ++kb) {
                const float sa = sa_next;
                float *sb = sbs + (kb & 1) * BN;
                sb[et] = sb_next;
                if (kb + 1 < a.num_kb) {
                    sa_next = load_scale(a.A, ra, kb + 1);
                    sb_next = load_scale(a.B, rb, kb + 1);
                }
                // the other buffer is written only after this barrier of the next block
                asm volatile("bar.sync 1, 128;" ::: "memory");
                const bool got = mbar_wait(accf0 + 8 * acc, acc_phase, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    if (lane == 0) raise_error(abort_flag);
                    ok = false;
                    // the barrier's other warps see the abort flag in their own wait
                }
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int h = 0; h < BN / 32; ++h) {
                        uint32_t r[32];
                        tmem_load_32cols(tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                             acc * BN + h * 32,
                                         r);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            sum[h * 32 + c] = __fmaf_rn(__uint_as_float(r[c]),
                                                        __fmul_rn(sa, sb[h * 32 + c]),
                                                        sum[h * 32 + c]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acce0 + 8 * acc);
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");   // all have read the last scales
            if (ok && row < a.M) {
                __nv_bfloat16 *d = a.D + row * a.ldd;
                const int64_t c0 = static_cast<int64_t>(nb) * BN;
#pragma unroll
                for (int c = 0; c < BN; c += 8) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = sum[c + i];
                    if (c0 + c < a.N)
                        store_row<__nv_bfloat16, 8>(d, c0 + c, a.N, a.vecd, v);
                }
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

}  // namespace

cudaError_t launch_block_gemm(const BlockView &A, const BlockView &B, const MatView &D,
                              int sm_count, cudaStream_t st, const char **what) {
    if (D.rows == 0 || D.cols == 0) return cudaSuccess;
    if (A.cols == 0)
        return cudaMemset2DAsync(D.data, D.ld * 2, 0, D.cols * 2, D.rows, st);
    Args a;
    if (!encode_tmap_2d(&a.mapA, A.codes, false, A.cols, A.rows, BK, BM, true, A.ld) ||
        !encode_tmap_2d(&a.mapB, B.codes, false, B.cols, B.rows, BK, BN, true, B.ld)) {
        *what = "cuTensorMapEncodeTiled failed for an operand";
        return cudaErrorInvalidValue;
    }
    a.A = A;
    a.B = B;
    a.D = static_cast<__nv_bfloat16 *>(D.data);
    a.M = D.rows;
    a.N = D.cols;
    a.ldd = D.ld;
    a.vecd = (reinterpret_cast<uintptr_t>(D.data) & 15u) == 0 && D.ld % 8 == 0;
    a.tiles_n = static_cast<int>((D.cols + BN - 1) / BN);
    a.num_tiles = static_cast<int>((D.rows + BM - 1) / BM) * a.tiles_n;
    a.num_kb = static_cast<int>((A.cols + BK - 1) / BK);
    a.idesc = idesc_f8(static_cast<uint32_t>(A.fmt), static_cast<uint32_t>(B.fmt), BM, BN);
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    std::call_once(once, [] {
        attr = cudaFuncSetAttribute(block_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(SMEM));
    });
    if (attr != cudaSuccess) return attr;
    const int grid = a.num_tiles < sm_count ? a.num_tiles : sm_count;
    return launch_pdl(block_gemm_kernel, dim3(grid), dim3(NUM_THREADS), SMEM, st, a);
}

cudaError_t read_and_clear_block_gemm_error_flag(unsigned *flags) {
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_block_gemm_error_flags, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_block_gemm_error_flags, &zero, sizeof(unsigned));
}

}  // namespace fp8k
