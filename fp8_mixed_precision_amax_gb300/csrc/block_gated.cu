// block_gated.cu -- the gated feed-forward product, forward and backward, on the sm_103a
// tcgen05 tensor cores: both projections, SiLU and the product in one kernel, and the
// way back through them in one.  E8M0 scales, one for each block of 128.
//
// Forward, A [M][K] and B [2F][K] = [gate rows | value rows]:
//   g = A . B[0 : F]^T,  u = A . B[F : 2F]^T   (fp32, in TMEM),
//   a = g / (1 + exp(-g)) * u,  block quantized into a8 [M][F]; [g | u] into h8 [M][2F]
// Backward, A = dy [M][K] and B [F][K], with g and u from h8 and s = 1 / (1 + exp(-g)):
//   da = A . B^T  (fp32, in TMEM),
//   dg = da * u * s * (1 + g * (1 - s)),  du = da * (g * s),
//   [dg | du] block quantized into dh8 [M][2F] and, transposed, dh8t [2F][M]; the
//   forward's a again, transposed, into a8t [F][M]
// Neither h = [g | u] nor da is rounded to 16 bits or written on the way.
//
// 8192 x 4096 -> 11008 with h kept: forward 454 us = 3250 TFLOP/s, tensor pipe 75 % active, bound by
// the MMAs and the exposed start and end (sustained, as the power limit takes the clock down,
// 497 us); backward 384 us, bound by the elementwise part, some 75 instructions an element at 49
// % of the issue slots, until K is about 3500, and from there on by the MMAs' operand reads and the
// elementwise part's passes through shared memory, which slow each other down (K = 256, 2048,
// 4096, 8192: 326, 360, 384, 603 us).
//
// Two CTAs on two SMs (a cluster) share each tile of 256 rows of A and 256 rows of B
// (cta_group::2): each loads its own 128 rows of either, and the even CTA issues the
// MMAs, whose 256 sums for each of a CTA's 128 rows fill half of its TMEM.  Forward:
// the even CTA's rows of B are gates and the odd one's the values that belong to them, so
// that columns j and 128 + j of a tile make one a, and a tile is one block of a wide.
// Backward: 256 columns of da, two blocks.
//
// Warps: the first ones (8 forward, 16 backward) do the elementwise part of one tile while
// the next one's MMAs run; then TMA, MMA, two idle ones, and four that bring scales to TMEM.
// The latter eight hand back registers, and the elementwise warps take them.
//
// TMEM: as in the matrix product of block_gemm.cu the two accumulators overlap by 32 columns
// (0-255 and 224-479), and columns 480-511 hold two stages of scales.  The elementwise
// warps read the shared columns first and then let the next tile's MMAs start.
//
// Every wait is bounded.
#include <cstdint>

#include "block_mma.cuh"
#include "error_flag.h"
#include "raster.cuh"

namespace fp8k {

namespace {

__device__ unsigned g_gated_error_flags = 0;

__device__ __forceinline__ void raise_error(volatile int *abort_flag) {
    atomicOr(&g_gated_error_flags, kErrWaitTimeout);
    *abort_flag = 1;
}

struct GatedArgs {
    CUtensorMap mapA, mapB;
    CUtensorMap mapBHalf;         // mapB with half the rows
    CUtensorMap map_a8, map_h8;   // forward: 32 rows of a block
    BlockView A, B;
    int64_t M, F;
    int64_t b_second;   // from the even CTA's first row of B to the odd one's
    int tile_cols;      // columns of a or da in a tile
    int tiles_m, tiles_n, num_items, num_kb, group_m;
    int whole;          // items from this one on are halves of tiles (backward: a block of da)
    uint32_t idesc, idesc_half;
    BlockView a8, h8;              // forward: outputs (h8's codes may be null); backward: h8 is read
    BlockView dh8, dh8t, a8t;      // backward: outputs, codes null: not wanted
};

struct Tile {
    int64_t row0, col0;   // of the pair's 256 rows; of the columns of a or da
    bool half;
};
__device__ __forceinline__ Tile tile_at(const GatedArgs &a, int item) {
    const bool half = item >= a.whole, own = a.tile_cols == kTile;   // own: of a tile's width
    const int tile = half && !own ? a.whole + (item - a.whole) / 2 : item;
    int mb, nb;
    tile_coords(tile, a.tiles_m, a.tiles_n, a.group_m, mb, nb);
    return Tile{static_cast<int64_t>(mb) * 2 * BM,
                static_cast<int64_t>(nb) * a.tile_cols + (half && !own ? (item - a.whole) % 2 * kTile : 0), half};
}

// What the elementwise warps of a CTA share.
template <bool BWD>
struct GatedShared;
template <>
struct GatedShared<false> {
    uint8_t codes[4][3][32 * kTile];   // [lane quarter][a, gate, value]: 32 rows, in TMA's 128-byte swizzle
    float3 row_max[2][2][BM];          // [tile mod 2][half of the columns][row]
};
template <>
struct GatedShared<true> {
    float da[kTile * kTile];
    uint8_t codes[3][kTile * kTile];   // d gate, d value, a: by columns
    uint32_t max[3][kTile];            // column maxima; 0 between their uses
    float inv[3][kTile];
};

// Registers: of the launch's, which are equal for all warps, the control warps keep
// REGS_CONTROL per thread and the elementwise warps have REGS_ELEMENTS.
template <bool BWD>
struct Gated {
    static constexpr int STAGES = BWD ? 3 : 5;
    static constexpr int WARPS = BWD ? 16 : 8;   // elementwise ones
    static constexpr int THREADS = 32 * (WARPS + 8);
    static constexpr int REGS_CONTROL = BWD ? 48 : 64, REGS_ELEMENTS = BWD ? 96 : 192;
    static constexpr int REGS_LAUNCH = 65536 / THREADS / 8 * 8;
    static_assert(256 * REGS_CONTROL + 32 * WARPS * REGS_ELEMENTS <= THREADS * REGS_LAUNCH, "register split");
    static constexpr int NUM_BARS = 2 * STAGES + 2 + 1 + 4 + 1;
    static constexpr size_t SMEM =
        1024 + STAGES * 2 * HALF + sizeof(GatedShared<BWD>) + NUM_BARS * 8 + 16;
    static_assert(SMEM <= 227 * 1024, "shared memory of an SM");
};

// ------------------------------------------------------------ TMA, MMA, scales --

template <int STAGES>
__device__ __forceinline__ void gated_produce(const GatedArgs &a, uint32_t rank, int unit, int num_units,
                                              uint32_t sA, uint32_t sB, uint32_t full0, uint32_t empty0,
                                              volatile int *abort_flag) {
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int tile = unit; ok && tile < a.num_items; tile += num_units) {
        const Tile t = tile_at(a, tile);
        const int32_t arow = static_cast<int32_t>(t.row0 + rank * BM);
        const int32_t brow = static_cast<int32_t>(t.col0 + rank * (t.half ? BM / 2 : a.b_second));
        const CUtensorMap *mapB = t.half ? &a.mapBHalf : &a.mapB;
        const uint32_t bytes = t.half ? 3 * HALF : 4 * HALF;
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

// The even CTA's MMA warp.
template <int STAGES>
__device__ __forceinline__ void gated_mma(const GatedArgs &a, int unit, int num_units, uint32_t tmem, uint32_t sA,
                                          uint32_t sB, uint32_t full0, uint32_t empty0, uint32_t accf0,
                                          uint32_t acce, uint32_t sff0, uint32_t sfe0, uint32_t drain,
                                          volatile int *abort_flag) {
    const int lane = threadIdx.x & 31;
    int stage = 0, sf = 0, it = 0;
    uint32_t phase = 0, sf_phase = 0;
    bool ok = true, any = false;
    for (int tile = unit; ok && tile < a.num_items; tile += num_units, ++it) {
        // the previous tile's shared columns have been read
        const bool freed = it == 0 || mbar_wait(acce, static_cast<uint32_t>(it - 1) & 1u, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, freed)) {
            if (lane == 0) raise_error(abort_flag);
            ok = false;
            break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ((it & 1) ? MX_ACC1 : 0), idesc0 = tile < a.whole ? a.idesc : a.idesc_half;
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
            if (++stage == STAGES) {
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

// The scale warps: every lane fetches its word (four k-blocks) of each 32 rows; rows past the
// end repeat the last one (their codes are zeros and their results are not stored).
__device__ __forceinline__ void gated_scales(const GatedArgs &a, uint32_t rank, int unit, int num_units,
                                             uint32_t tmem, uint32_t sff0, uint32_t sfe0,
                                             volatile int *abort_flag) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + MX_SF;
    int sf = 0;
    uint32_t sf_phase = 0;
    bool ok = true;
    for (int tile = unit; ok && tile < a.num_items; tile += num_units) {
        const Tile t = tile_at(a, tile);
        const uint8_t *pa = static_cast<const uint8_t *>(a.A.scales), *pb = static_cast<const uint8_t *>(a.B.scales);
        const int sa = a.A.block_rows == 1 ? 0 : 7, sb = a.B.block_rows == 1 ? 0 : 7;
        const unsigned ra = static_cast<unsigned>(t.row0 + rank * BM + lane), most_a = static_cast<unsigned>(a.M - 1);
        const unsigned rb = static_cast<unsigned>(t.col0 + lane), most_b = static_cast<unsigned>(a.B.rows - 1);
        const unsigned second = static_cast<unsigned>(a.b_second);
        for (int kb = 0; kb < a.num_kb; kb += 4) {
            uint32_t wa[4], wb[8];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wa[j] = *reinterpret_cast<const uint32_t *>(pa + row_at(min(ra + 32 * j, most_a) >> sa, a.A.ld_s) + kb);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                wb[j] = *reinterpret_cast<const uint32_t *>(
                    pb + row_at(min(rb + (j >> 2) * second + 32 * (j & 3), most_b) >> sb, a.B.ld_s) + kb);
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
}

// ------------------------------------------------------------ elementwise parts --

__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    return f32x2_pack(__uint_as_float(lo), __uint_as_float(hi));
}
// max over finite magnitudes in place of one that came out infinite
template <int N>
__device__ __forceinline__ float finite_max(const uint64_t (&v)[N], float m) {
#pragma unroll
    for (int i = 0; i < N; ++i) m = absmax3(m, without_inf(v[i]));
    return m;
}
template <int N>
__device__ __forceinline__ float block_max(const uint64_t (&v)[N], float m0) {
    float m = m0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = absmax3(m, v[i]);
    return is_inf(m) ? finite_max(v, m0) : m;
}
__device__ __forceinline__ uint64_t silu_times(uint64_t g, uint64_t u) {
    float g0, g1;
    f32x2_unpack(g, g0, g1);
    return f32x2_mul(f32x2_mul(g, sigmoid2(g0, g1)), u);
}

// 16 columns of gate and value of this lane's row, the columns that two accumulators share
// from `keep` (which half of this warp's columns they are: gate's first or value's last).
__device__ __forceinline__ void gate_value16(uint32_t t, int c, const uint32_t (&keep)[32], bool keep_g,
                                             bool keep_u, uint64_t (&g)[8], uint64_t (&u)[8]) {
    uint32_t rg[16], ru[16];
    tmem_load_16cols(t + 16 * c, rg);
    tmem_load_16cols(t + BM + 16 * c, ru);
    tmem_wait_16cols(rg);
    tmem_wait_16cols(ru);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (c < 2) rg[i] = keep_g ? keep[16 * (c & 1) + i] : rg[i];
        if (c >= 2) ru[i] = keep_u ? keep[16 * (c & 1) + i] : ru[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i] = pair_of(rg[2 * i], rg[2 * i + 1]);
        u[i] = pair_of(ru[2 * i], ru[2 * i + 1]);
    }
}

// 16 values of this lane's row as codes, its 16-byte chunk `at` of 32 staged rows
template <int FMT>
__device__ __forceinline__ void stage_codes16(uint32_t rows, int at, const uint64_t *v, float inv) {
    const int lane = threadIdx.x & 31;
    const uint64_t inv2 = splat_f32x2(inv);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = encode4<FMT>(f32x2_mul(v[2 * i], inv2), f32x2_mul(v[2 * i + 1], inv2));
    st_shared_v4(rows + lane * kTile + ((at ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void quarter_sync(int q) { asm volatile("bar.sync %0, 64;" ::"r"(2 + q) : "memory"); }

// AFMT, HFMT: formats of a8 and h8.
template <int AFMT, int HFMT>
__device__ __forceinline__ void gated_fwd_tile(const GatedArgs &a, GatedShared<false> &sm, const Tile &tile,
                                               uint32_t rank, int it, uint32_t tmem, uint32_t acce0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, half = warp >> 2;
    const bool odd = it & 1;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t t = lanes + (odd ? MX_ACC1 : 0) + 64 * half;
    // shared by the two accumulators: value's last 32 columns, or gate's first 32
    const bool keep_g = odd && half == 0, keep_u = !odd && half == 1;
    uint32_t keep[32];
    if (keep_g || keep_u) tmem_load_32cols(lanes + MX_ACC1, keep);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster_relaxed(acce0);

    uint64_t av[32];
    float ma = 0.0f, mg = 0.0f, mu = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint64_t g[8], u[8], o[8];
        gate_value16(t, c, keep, keep_g, keep_u, g, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) av[8 * c + i] = o[i] = silu_times(g[i], u[i]);
        ma = block_max(o, ma);
        mg = block_max(g, mg);
        mu = block_max(u, mu);
    }
    // the other half of the row's block is the partner warp's
    const int r = 32 * q + lane;
    sm.row_max[it & 1][half][r] = make_float3(ma, mg, mu);
    if (half == 0 && lane == 0) bulk_wait_group_read<0>();   // the staged rows before these have left
    __syncwarp();
    quarter_sync(q);
    const float3 other = sm.row_max[it & 1][half ^ 1][r];
    const uint32_t ba = scale_byte<AFMT>(__float_as_uint(fmaxf(ma, other.x)));
    const uint32_t bg = scale_byte<HFMT>(__float_as_uint(fmaxf(mg, other.y)));
    const uint32_t bu = scale_byte<HFMT>(__float_as_uint(fmaxf(mu, other.z)));
    const int64_t row0 = tile.row0 + rank * BM + 32 * q, row = row0 + lane;
    const bool keep_h = a.h8.codes != nullptr;
    if (row < a.M && half == 0) {
        store_scale(a.a8, row, tile.col0 / kTile, ba);
        if (keep_h) {
            store_scale(a.h8, row, tile.col0 / kTile, bg);
            store_scale(a.h8, row, (a.F + tile.col0) / kTile, bu);
        }
    }
    const uint32_t to = smem_u32(sm.codes[q]);
#pragma unroll
    for (int c = 0; c < 4; ++c) stage_codes16<AFMT>(to, 4 * half + c, av + 8 * c, scale_inverse(ba));
    if (keep_h) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint64_t g[8], u[8];
            gate_value16(t, c, keep, keep_g, keep_u, g, u);
            stage_codes16<HFMT>(to + 32 * kTile, 4 * half + c, g, scale_inverse(bg));
            stage_codes16<HFMT>(to + 2 * 32 * kTile, 4 * half + c, u, scale_inverse(bu));
        }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    quarter_sync(q);
    if (half == 0 && lane == 0 && row0 < a.M) {
        const int32_t x = static_cast<int32_t>(tile.col0), y = static_cast<int32_t>(row0);
        tma_store_2d(&a.map_a8, to, x, y);
        if (keep_h) {
            tma_store_2d(&a.map_h8, to + 32 * kTile, x, y);
            tma_store_2d(&a.map_h8, to + 2 * 32 * kTile, x + static_cast<int32_t>(a.F), y);
        }
        bulk_commit_group();
    }
}

// gate or value of 4 columns from their codes
__device__ __forceinline__ void decode_pairs(uint32_t w, int fmt, float scale, uint64_t (&v)[2]) {
    float f[4];
    decode4(w, fmt, f);
    const uint64_t s2 = splat_f32x2(scale);
    v[0] = f32x2_mul(f32x2_pack(f[0], f[1]), s2);
    v[1] = f32x2_mul(f32x2_pack(f[2], f[3]), s2);
}

// Backward, a block of 128 columns of da.  It goes through shared memory from TMEM's layout
// (a lane is a row) to one in which warp w of 16 has the 8 rows from 8 w on and lane l
// columns 4 l .. 4 l + 3: a row's maximum is then one warp reduction, a column's is taken over a
// thread's 8 rows first, and rows of h8 and dh8 are read and written 128 bytes at a time.
// Everything is computed twice from da and the codes, for the maxima and again for the
// results: kept, the three results of a tile are most of an SM's registers, and code for
// fewer warps with more of them is too long for the instruction cache.  (8192 x 4096 -> 11008:
// 384 us; with a row per lane throughout 676; with 8 warps that keep two of the three 467.)
struct BlockCodes {   // of h8, for this lane's 4 columns of its warp's 8 rows, two rows at a time
    const uint8_t *at_g, *at_u;   // gate's and value's codes of the next two rows
    int rows;                     // of the 8, that there are
    uint32_t scale;               // lanes 0 .. 7: the rows' scales of gate; lanes 8 .. 15: of value
    uint32_t g[2], u[2];

    __device__ __forceinline__ void start(const GatedArgs &a, int64_t row0, int64_t col0) {
        const int lane = threadIdx.x & 31;
        const int64_t r0 = row0 + (threadIdx.x >> 5) * kTileRows;
        at_g = a.h8.codes + r0 * a.h8.ld + col0 + 4 * lane;
        at_u = at_g + a.F;
        rows = a.M - r0 >= kTileRows ? kTileRows : static_cast<int>(a.M - r0);
        scale = lane < 16 && (lane & 7) < rows
                    ? fetch_scale(a.h8, r0 + (lane & 7), (lane < 8 ? col0 : a.F + col0) / kTile)
                    : 0u;
        fetch(a, 0);
    }
    // rows i and i + 1, each call the next two
    __device__ __forceinline__ void fetch(const GatedArgs &a, int i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool in = i + k < rows;
            g[k] = in ? *reinterpret_cast<const uint32_t *>(at_g) : 0u;
            u[k] = in ? *reinterpret_cast<const uint32_t *>(at_u) : 0u;
            at_g += a.h8.ld, at_u += a.h8.ld;
        }
    }
    __device__ __forceinline__ void rewind(const GatedArgs &a) {
        at_g -= kTileRows * a.h8.ld, at_u -= kTileRows * a.h8.ld;
        fetch(a, 0);
    }
};

// 4 codes as fp32, exactly
__device__ __forceinline__ void decode_pairs(uint32_t w, int fmt, uint64_t (&v)[2]) {
    float f[4];
    decode4(w, fmt, f);
    v[0] = f32x2_pack(f[0], f[1]);
    v[1] = f32x2_pack(f[2], f[3]);
}

// d gate, d value and a of a row of the warp's, from its codes
template <int HFMT>
struct RowValues {
    uint64_t dg[2], du[2], a[2];

    __device__ __forceinline__ RowValues(const float *da, int i, uint32_t gc, uint32_t uc, float scale) {
        const int lane = threadIdx.x & 31, r = kTileRows * (threadIdx.x >> 5) + i;
        const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(&da[r * kTile + ((lane ^ (r & 31)) << 2)]);
        const float sg = __shfl_sync(0xFFFFFFFFu, scale, i), su = __shfl_sync(0xFFFFFFFFu, scale, 8 + i);
        const uint64_t sg2 = splat_f32x2(sg), sl2 = splat_f32x2(__fmul_rn(sg, -1.44269504f)), su2 = splat_f32x2(su);
        const uint64_t one2 = splat_f32x2(1.0f), quarter2 = splat_f32x2(0.25f);
        uint64_t cg[2], cu[2];
        decode_pairs(gc, HFMT, cg);
        decode_pairs(uc, HFMT, cu);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            // sigmoid2, with the logarithm's factor in the scale
            float e0, e1, q0, q1;
            f32x2_unpack(f32x2_mul(cg[p], sl2), e0, e1);
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e0));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e1));
            f32x2_unpack(f32x2_fma(f32x2_pack(e0, e1), quarter2, quarter2), q0, q1);
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(q0));
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(q1));
            const uint64_t s = f32x2_mul(f32x2_pack(q0, q1), quarter2);
            const uint64_t gs = f32x2_mul(f32x2_mul(cg[p], sg2), s), u = f32x2_mul(cu[p], su2), dp = p ? d.y : d.x;
            a[p] = f32x2_mul(gs, u);
            du[p] = f32x2_mul(dp, gs);
            // s (1 + g (1 - s))
            dg[p] = f32x2_mul(f32x2_mul(dp, u), f32x2_fma(gs, f32x2_sub(one2, s), s));
        }
    }
};

// The largest magnitudes: of this lane's columns over the warp's rows, and lane i's of row i.
struct Maxima {
    float col[3][4];
    uint32_t row_g, row_u;

    // FINITE: infinities do not count
    template <int HFMT, bool FINITE>
    __device__ __forceinline__ void take(const GatedArgs &a, const float *da, BlockCodes &h, float scale) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < 3; ++k) col[k][0] = col[k][1] = col[k][2] = col[k][3] = 0.0f;
        row_g = row_u = 0;
#pragma unroll 1
        for (int i = 0; i < kTileRows; i += 2) {
            const uint32_t g[2] = {h.g[0], h.g[1]}, u[2] = {h.u[0], h.u[1]};
            if (i + 2 < kTileRows)
                h.fetch(a, i + 2);
            else
                h.rewind(a);   // for the next pass
            RowValues<HFMT> r[2] = {{da, i, g[0], u[0], scale}, {da, i + 1, g[1], u[1], scale}};
            if constexpr (FINITE) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        r[k].dg[p] = without_inf(r[k].dg[p]);
                        r[k].du[p] = without_inf(r[k].du[p]);
                        r[k].a[p] = without_inf(r[k].a[p]);
                    }
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                columns(0, p, r[0].dg[p], r[1].dg[p]);
                columns(1, p, r[0].du[p], r[1].du[p]);
                columns(2, p, r[0].a[p], r[1].a[p]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t mg = row(r[k].dg), mu = row(r[k].du);
                if (lane == i + k) row_g = mg, row_u = mu;
            }
        }
    }
    __device__ __forceinline__ void columns(int k, int p, uint64_t a, uint64_t b) {
        float x, y, z, w;
        f32x2_unpack(a, x, y);
        f32x2_unpack(b, z, w);
        col[k][2 * p] = absmax3(col[k][2 * p], x, z);
        col[k][2 * p + 1] = absmax3(col[k][2 * p + 1], y, w);
    }
    static __device__ __forceinline__ uint32_t row(const uint64_t (&v)[2]) {
        return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(absmax3(absmax3(0.0f, v[0]), v[1])));
    }
    __device__ __forceinline__ bool infinite() const {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < 3; ++k) m = fmaxf(m, fmaxf(fmaxf(col[k][0], col[k][1]), fmaxf(col[k][2], col[k][3])));
        return is_inf(m);
    }
};

// Two rows' codes of this lane's 4 columns: word p has columns 2 p and 2 p + 1, 16 bits each.
template <int FMT>
__device__ __forceinline__ void encode_columns2(const uint64_t (&a)[2], const uint64_t (&b)[2], const float *inv,
                                                uint32_t (&w)[2]) {
    const ulonglong2 inv2 = *reinterpret_cast<const ulonglong2 *>(inv + 4 * (threadIdx.x & 31));
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float a0, a1, b0, b1;
        f32x2_unpack(f32x2_mul(a[p], p ? inv2.y : inv2.x), a0, a1);
        f32x2_unpack(f32x2_mul(b[p], p ? inv2.y : inv2.x), b0, b1);
        w[p] = encode4<FMT>(f32x2_pack(a0, b0), f32x2_pack(a1, b1));
    }
}
// Four rows' into a tile whose row is a column of 128 bytes; word n of column c (rows 4 n ..
// 4 n + 3) is kept at place n ^ (c >> 2), so that a warp's lanes write to 32 banks.
__device__ __forceinline__ void put_columns4(uint8_t *codes, int n, const uint32_t (&a)[2], const uint32_t (&b)[2]) {
    const int lane = threadIdx.x & 31;
    uint32_t *to = reinterpret_cast<uint32_t *>(codes) + 4 * lane * (kTile / 4) + (n ^ lane);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        to[2 * p * (kTile / 4)] = __byte_perm(a[p], b[p], 0x5410);
        to[(2 * p + 1) * (kTile / 4)] = __byte_perm(a[p], b[p], 0x7632);
    }
}

// The tile's columns as rows of o from first_row on, 8 threads each.
__device__ __forceinline__ void put_tile(const BlockView &o, int64_t first_row, int64_t row0, int64_t M,
                                         const uint8_t *codes) {
    const int k = threadIdx.x & 7, c0 = threadIdx.x >> 3;
    const int64_t left = M - (row0 + 16 * k);
    uint8_t *p = o.codes + (first_row + c0) * o.ld + row0 + 16 * k;
#pragma unroll
    for (int i = 0; i < 2; ++i, p += 64 * o.ld) {
        const int c = c0 + 64 * i, x = c >> 2;   // words 4 k .. 4 k + 3 are a block of four, in another order
        uint4 u = *reinterpret_cast<const uint4 *>(codes + c * kTile + ((k ^ (x >> 2)) << 4));
        if (x & 1) u = make_uint4(u.y, u.x, u.w, u.z);
        if (x & 2) u = make_uint4(u.z, u.w, u.x, u.y);
        if (left >= 16) {
            *reinterpret_cast<uint4 *>(p) = u;
        } else if (left > 0) {
            store_code_word(p, u.x, left);
            store_code_word(p + 4, u.y, left - 4);
            store_code_word(p + 8, u.z, left - 8);
            store_code_word(p + 12, u.w, left - 12);
        }
    }
}

__device__ __forceinline__ void elements_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

// h: the block's codes; `first`: the block that holds the columns shared by the two accumulators.
// FMT, AFMT, HFMT: formats of dh8 / dh8t, of a8t and of h8.  next: called once h is done with.
template <int FMT, int AFMT, int HFMT, typename Next>
__device__ __forceinline__ void gated_bwd_block(const GatedArgs &a, GatedShared<true> &sm, BlockCodes &h,
                                                int64_t row0, int64_t col0, bool first, uint32_t t, uint32_t acce0,
                                                Next next) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, part = warp >> 2;
    const bool want_t = a.dh8t.codes != nullptr, want_a = a.a8t.codes != nullptr, want_r = a.dh8.codes != nullptr;
    // (the block before has been read from da; its codes may still be on their way out, and the
    // next ones come three barriers later)
    // 16-byte chunk k of a row of da is kept at place k ^ (row mod 32): no bank twice, either way
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t d[16];
        tmem_load_16cols(t + 32 * part + 16 * k, d);
        tmem_wait_16cols(d);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(&sm.da[(32 * q + lane) * kTile + (((8 * part + 4 * k + j) ^ lane) << 2)]) =
                make_uint4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
    }
    if (first) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acce0);
    }
    elements_sync();
    const float scale = fetched_scale(a.h8, h.scale);
    Maxima m;
    m.take<HFMT, false>(a, sm.da, h, scale);
    if (__any_sync(0xFFFFFFFFu, m.infinite())) m.take<HFMT, true>(a, sm.da, h, scale);
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm volatile("red.shared::cta.max.u32 [%0], %1;" ::"r"(smem_u32(&sm.max[k][4 * lane + j])),
                         "r"(__float_as_uint(m.col[k][j]))
                         : "memory");
    elements_sync();
    if (threadIdx.x < 3 * kTile) {
        const int k = threadIdx.x / kTile, c = threadIdx.x % kTile;
        const uint32_t byte = k == 2 ? scale_byte<AFMT>(sm.max[k][c]) : scale_byte<FMT>(sm.max[k][c]);
        sm.max[k][c] = 0;
        sm.inv[k][c] = scale_inverse(byte);
        if (row0 < a.M) {
            if (k < 2 && want_t) store_scale(a.dh8t, (k ? a.F : 0) + col0 + c, row0 / kTile, byte);
            if (k == 2 && want_a) store_scale(a.a8t, col0 + c, row0 / kTile, byte);
        }
    }
    elements_sync();
    const int64_t r0 = row0 + kTileRows * warp;
    const uint32_t bg = scale_byte<FMT>(m.row_g), bu = scale_byte<FMT>(m.row_u);
    if (want_r && lane < kTileRows && lane < h.rows) {
        store_scale(a.dh8, r0 + lane, col0 / kTile, bg);
        store_scale(a.dh8, r0 + lane, (a.F + col0) / kTile, bu);
    }
    const float ig = scale_inverse(bg), iu = scale_inverse(bu);
    uint8_t *pg = a.dh8.codes + r0 * a.dh8.ld + col0 + 4 * lane, *pu = pg + a.F;
#pragma unroll 1
    for (int i = 0; i < kTileRows; i += 4) {
        uint32_t w[3][2][2];   // [d gate, d value, a][two rows]
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int at = i + 2 * n;
            const uint32_t g[2] = {h.g[0], h.g[1]}, u[2] = {h.u[0], h.u[1]};
            if (at + 2 < kTileRows) h.fetch(a, at + 2);
            const RowValues<HFMT> r[2] = {{sm.da, at, g[0], u[0], scale}, {sm.da, at + 1, g[1], u[1], scale}};
            if (want_r) {
#pragma unroll
                for (int k = 0; k < 2; ++k, pg += a.dh8.ld, pu += a.dh8.ld) {
                    const uint64_t g2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, ig, at + k));
                    const uint64_t u2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, iu, at + k));
                    const uint32_t wg = encode4<FMT>(f32x2_mul(r[k].dg[0], g2), f32x2_mul(r[k].dg[1], g2));
                    const uint32_t wu = encode4<FMT>(f32x2_mul(r[k].du[0], u2), f32x2_mul(r[k].du[1], u2));
                    if (at + k < h.rows) {
                        *reinterpret_cast<uint32_t *>(pg) = wg;
                        *reinterpret_cast<uint32_t *>(pu) = wu;
                    }
                }
            }
            encode_columns2<FMT>(r[0].dg, r[1].dg, sm.inv[0], w[0][n]);
            encode_columns2<FMT>(r[0].du, r[1].du, sm.inv[1], w[1][n]);
            encode_columns2<AFMT>(r[0].a, r[1].a, sm.inv[2], w[2][n]);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) put_columns4(sm.codes[k], 2 * warp + i / 4, w[k][0], w[k][1]);
    }
    next();
    elements_sync();
    if (want_t) {
        put_tile(a.dh8t, col0, row0, a.M, sm.codes[0]);
        put_tile(a.dh8t, a.F + col0, row0, a.M, sm.codes[1]);
    }
    if (want_a) put_tile(a.a8t, col0, row0, a.M, sm.codes[2]);
}

// F0, F1, F2: formats of a8 and h8, or of dh8 / dh8t, a8t and h8.
template <bool BWD, int F0, int F1, int F2>
__global__ void __launch_bounds__(Gated<BWD>::THREADS, 1) gated_pair_kernel(const __grid_constant__ GatedArgs a) {
    using C = Gated<BWD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sA = smem_u32(smem), sB = sA + C::STAGES * HALF;
    GatedShared<BWD> &sm = *reinterpret_cast<GatedShared<BWD> *>(smem + C::STAGES * 2 * HALF);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::STAGES * 2 * HALF + sizeof(GatedShared<BWD>));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();   // 0 = the CTA that issues MMAs
    const int unit = static_cast<int>(blockIdx.x >> 1), num_units = static_cast<int>(gridDim.x >> 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t accf0 = empty0 + 8 * C::STAGES, acce = accf0 + 16;
    const uint32_t sff0 = acce + 8, sfe0 = sff0 + 16, drain = sfe0 + 16;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(sff0 + 8 * b, 8);   // four scale warps of each CTA
            mbar_init(sfe0 + 8 * b, 1);
        }
        mbar_init(acce, 2 * C::WARPS);    // the elementwise warps of both CTAs
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&a.mapA);
        prefetch_tmap(&a.mapB);
    }
    if constexpr (BWD) {
        if (threadIdx.x < 3 * kTile) sm.max[threadIdx.x / kTile][threadIdx.x % kTile] = 0;
    }
    if (warp == C::WARPS + 1) {
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

    if (warp >= C::WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONTROL));
        const int role = warp - C::WARPS;
        if (role == 0)
            gated_produce<C::STAGES>(a, rank, unit, num_units, sA, sB, full0, empty0, abort_flag);
        else if (role == 1 && rank == 0)
            gated_mma<C::STAGES>(a, unit, num_units, tmem, sA, sB, full0, empty0, accf0, acce, sff0, sfe0, drain,
                                 abort_flag);
        else if (role >= 4)
            gated_scales(a, rank, unit, num_units, tmem, sff0, sfe0, abort_flag);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_ELEMENTS));
        const uint32_t acce0 = mapa_shared(acce, 0);
        int it = 0;
        BlockCodes h;   // backward: of the next block, while this one is in work
        // the columns of block j of the CTA's n-th tile (F: it has none): of two blocks the one with
        // the columns that two accumulators share comes first
        const auto col_of = [&](const Tile &tile, int n, int j) {
            if (tile.half) return j == 0 ? tile.col0 : a.F;
            return tile.col0 + ((n & 1) == j ? kTile : 0);
        };
        auto fetch = [&](int item, int n, int j) {
            if (item >= a.num_items) return;
            const Tile tile = tile_at(a, item);
            const int64_t c = col_of(tile, n, j);
            if (c < a.F) h.start(a, tile.row0 + rank * BM, c);
        };
        if constexpr (BWD) fetch(unit, 0, 0);
        for (int i = unit; i < a.num_items; i += num_units, ++it) {
            const Tile tile = tile_at(a, i);
            const bool got = mbar_wait(accf0 + 8 * (it & 1), static_cast<uint32_t>(it >> 1) & 1u, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got) && lane == 0) raise_error(abort_flag);
            // all go on or none: a warp alone in a tile's barriers would stay there
            if (!barrier_and(1, 32 * C::WARPS, got)) break;
            tc_fence_after();
            if constexpr (BWD) {
                const uint32_t t = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + ((it & 1) ? MX_ACC1 : 0);
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    const int64_t col0 = col_of(tile, it, j);
                    if (col0 >= a.F) {
                        if (j == 0) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster_relaxed(acce0);
                            fetch(i, it, 1);
                        } else {
                            fetch(i + num_units, it + 1, 0);
                        }
                        continue;
                    }
                    gated_bwd_block<F0, F1, F2>(a, sm, h, tile.row0 + rank * BM, col0, j == 0,
                                            t + static_cast<uint32_t>(col0 - tile.col0), acce0, [&] {
                                                if (j == 0)
                                                    fetch(i, it, 1);
                                                else
                                                    fetch(i + num_units, it + 1, 0);
                                            });
                }
                tc_fence_before();
            } else {
                gated_fwd_tile<F0, F1>(a, sm, tile, rank, it, tmem, acce0);
            }
        }
        if (!BWD && lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();   // the other SM is done with this CTA's memory
    if (warp == C::WARPS + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ----------------------------------------------------------------- few kernel --
// Forward of few tokens (being decoded, or one wave of tiles): a CTA computes one block of 128
// columns of a for NT tokens over its share of the k-blocks; the block's 128 gate rows of B and
// its 128 value rows take the instruction's 128-row side, one after the other, and the tokens its
// columns.  gridDim.x CTAs, a cluster, share a block's k-blocks: one SM alone reads too slowly for
// the weights of a token.  Their sums [token][gate, value][column] meet in shared memory, and
// the warps of CTA k of the cluster join, activate and quantize tokens k, k + splits, ..., a token
// each at a time.
// Warps: 0 TMA, 1 MMA, 2-9 the sums (thread = weight row; warps w and w + 4 have the same TMEM
// lanes, one gate, the other value), of which 2-5 bring the scales to TMEM before.

template <int NT>
struct GatedFew {
    static constexpr int X_STAGE = NT * BK, STAGE = 2 * HALF + X_STAGE;
    static constexpr int STAGES = NT <= 32 ? 3 : NT <= 64 ? 5 : 4;
    static constexpr int CTAS = NT <= 32 ? 2 : 1;       // per SM
    static constexpr int MOST_SPLITS = 8;
    static constexpr int THREADS = 320;
    static constexpr int SF = 2 * NT, SF_STRIDE = 16;   // TMEM: scales, per stage gate 4, value 4, tokens 4
    static constexpr int TMEM = NT <= 16 ? 64 : 4 * NT;
    static constexpr int NUM_BARS = 2 * STAGES + 1 + 4 + 1;
    static constexpr size_t SMEM = 1024 + STAGES * STAGE + NUM_BARS * 8 + 16;
    static_assert(STAGES * STAGE >= NT * 256 * 4, "the sums fit where the tiles were");
    static_assert(SF + 2 * SF_STRIDE <= TMEM, "the scales fit");
};

struct GatedFewArgs {
    CUtensorMap mapW, mapX;   // B's rows (128 x 128 boxes) and A's (128 x NT)
    BlockView W, X, a8, h8;
    int64_t M, F;
    int num_kb;
    uint32_t idesc;
};

// A block of a row by a warp, 4 columns per lane.
template <int FMT>
__device__ __forceinline__ void quantize_block4(const uint64_t (&v)[2], const BlockView &o, int64_t row, int64_t col0) {
    const int lane = threadIdx.x & 31;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(block_max(v, 0.0f)));
    const uint32_t byte = scale_byte<FMT>(m);
    const uint64_t inv2 = splat_f32x2(scale_inverse(byte));
    *reinterpret_cast<uint32_t *>(o.codes + row * o.ld + col0 + 4 * lane) =
        encode4<FMT>(f32x2_mul(v[0], inv2), f32x2_mul(v[1], inv2));
    if (lane == 0) store_scale(o, row, col0 / kTile, byte);
}
__device__ __forceinline__ float4 ld_shared_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The sums of up to S splits to results: a warp has T tokens at a time, a lane four columns of
// their block.
template <int S, int T, int AFMT, int HFMT>
__device__ __forceinline__ void gated_join(const GatedFewArgs &a, uint32_t sums, int split, int splits, int64_t token0,
                                           int tokens, int64_t col0) {
    const uint32_t red = sums + 16 * (threadIdx.x & 31);
    const int first = T * static_cast<int>((threadIdx.x >> 5) - 2);
    for (int i0 = first; split + i0 * splits < tokens; i0 += 8 * T) {
        float4 pg[T][S], pu[T][S];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int n = split + (i0 + i) * splits;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                pg[i][k] = pu[i][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (k < splits && n < tokens) {
                    const uint32_t at = mapa_shared(red + n * 1024, static_cast<uint32_t>(k));
                    pg[i][k] = ld_shared_cluster4(at);
                    pu[i][k] = ld_shared_cluster4(at + 512);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int n = split + (i0 + i) * splits;
            if (n >= tokens) break;
            uint64_t g[2] = {}, u[2] = {}, v[2];
#pragma unroll
            for (int k = 0; k < S; ++k) {   // in the order of the splits
                g[0] = f32x2_add(g[0], f32x2_pack(pg[i][k].x, pg[i][k].y));
                g[1] = f32x2_add(g[1], f32x2_pack(pg[i][k].z, pg[i][k].w));
                u[0] = f32x2_add(u[0], f32x2_pack(pu[i][k].x, pu[i][k].y));
                u[1] = f32x2_add(u[1], f32x2_pack(pu[i][k].z, pu[i][k].w));
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) v[p] = silu_times(g[p], u[p]);
            const int64_t row = token0 + n;
            quantize_block4<AFMT>(v, a.a8, row, col0);
            if (a.h8.codes != nullptr) {
                quantize_block4<HFMT>(g, a.h8, row, col0);
                quantize_block4<HFMT>(u, a.h8, row, a.F + col0);
            }
        }
    }
}

// Bound by the weights' bytes: 1 x 4096 -> 11008 16.9 us = 5.3 TB/s of them, 0.79 of a copy's rate;
// 64 tokens 20 us, 128 with h kept 27.8.
template <int NT, int AFMT, int HFMT>
__global__ void __launch_bounds__(GatedFew<NT>::THREADS, GatedFew<NT>::CTAS)
    gated_few_kernel(const __grid_constant__ GatedFewArgs a) {
    using C = GatedFew<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t sW = smem_u32(smem), sX = sW + C::STAGES * 2 * HALF;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::STAGES * C::STAGE);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t accf = empty0 + 8 * C::STAGES, sff0 = accf + 8, sfe0 = sff0 + 16, drain = sfe0 + 16;
    const int splits = static_cast<int>(gridDim.x), split = static_cast<int>(blockIdx.x);
    const int kb0 = static_cast<int>(static_cast<int64_t>(a.num_kb) * split / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(a.num_kb) * (split + 1) / splits);
    const int64_t col0 = static_cast<int64_t>(blockIdx.y) * kTile, token0 = static_cast<int64_t>(blockIdx.z) * NT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(accf, 1);
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

    const int q = warp & 3, r = 32 * q + lane;   // lane quarter and weight row of a sums warp
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
                const uint32_t fb = full0 + 8 * stage, to = sW + stage * 2 * HALF;
                mbar_arrive_expect_tx(fb, C::STAGE);
                tma_load_2d(to, &a.mapW, fb, kb * BK, static_cast<int32_t>(col0));
                tma_load_2d(to + HALF, &a.mapW, fb, kb * BK, static_cast<int32_t>(a.F + col0));
                tma_load_2d(sX + stage * C::X_STAGE, &a.mapX, fb, kb * BK, static_cast<int32_t>(token0));
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
        int stage = 0, sf = 0;
        uint32_t phase = 0, sf_phase = 0;
        bool any = false;
        for (int kb = kb0; kb < kb1; ++kb) {
            // a stage of scales holds those of four k-blocks, from a multiple of 4 on
            const bool first = kb == kb0 || (kb & 3) == 0;
            const bool go = (!first || mbar_wait(sff0 + 8 * sf, sf_phase, abort_flag)) &&
                            mbar_wait(full0 + 8 * stage, phase, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, go)) {
                if (lane == 0) raise_error(abort_flag);
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t gd = smem_desc_sw128(sW + stage * 2 * HALF), ud = smem_desc_sw128(sW + stage * 2 * HALF + HALF);
                const uint64_t xd = smem_desc_sw128(sX + stage * C::X_STAGE);
                const uint32_t id = static_cast<uint32_t>(kb & 3), idesc = a.idesc | id << 4 | id << 29;
                const uint32_t sfg = tmem + C::SF + sf * C::SF_STRIDE, sfx = sfg + 8;
#pragma unroll
                for (int k = 0; k < BK / 32; ++k) {   // 32 bytes on: 2 in the descriptors' unit
                    mma_mxf8(tmem, gd + 2 * k, xd + 2 * k, idesc, sfg, sfx, kb != kb0 || k != 0);
                    mma_mxf8(tmem + NT, ud + 2 * k, xd + 2 * k, idesc, sfg + 4, sfx, kb != kb0 || k != 0);
                }
                mma_commit(empty0 + 8 * stage);
                if ((kb & 3) == 3) mma_commit(sfe0 + 8 * sf);
                if (kb == kb1 - 1) mma_commit(accf);
            }
            __syncwarp();
            any = true;
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if ((kb & 3) == 3 && ++sf == 2) {
                sf = 0;
                sf_phase ^= 1u;
            }
        }
        if (!ok && any) {
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            mbar_wait(drain, 0, nullptr, 100000000ull);
        }
    } else {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        if (warp < 6) {
            // scales; rows past the end repeat the last one
            const uint8_t *pw = static_cast<const uint8_t *>(a.W.scales), *px = static_cast<const uint8_t *>(a.X.scales);
            const int sw = a.W.block_rows == 1 ? 0 : 7, sx = a.X.block_rows == 1 ? 0 : 7;
            uint32_t wg[4], wu[4], wx[4] = {0, 0, 0, 0};
            auto fetch = [&](int kb) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned g = static_cast<unsigned>(col0) + 32 * j + lane, u = static_cast<unsigned>(a.F) + g;
                    wg[j] = *reinterpret_cast<const uint32_t *>(pw + row_at(g >> sw, a.W.ld_s) + kb);
                    wu[j] = *reinterpret_cast<const uint32_t *>(pw + row_at(u >> sw, a.W.ld_s) + kb);
                    const unsigned x = min(static_cast<unsigned>(token0) + 32 * j + lane, static_cast<unsigned>(a.M - 1));
                    if (32 * j < NT) wx[j] = *reinterpret_cast<const uint32_t *>(px + row_at(x >> sx, a.X.ld_s) + kb);
                }
            };
            int sf = 0;
            uint32_t sf_phase = 0;
            if (kb0 < kb1) fetch(kb0 & ~3);
            for (int kb = kb0 & ~3; kb < kb1; kb += 4) {
                uint32_t g[4], u[4], x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] = wg[j], u[j] = wu[j], x[j] = wx[j];
                if (kb + 4 < kb1) fetch(kb + 4);
                const bool got = mbar_wait(sfe0 + 8 * sf, sf_phase ^ 1u, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    if (lane == 0) raise_error(abort_flag);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = lanes + C::SF + sf * C::SF_STRIDE;
                tmem_store_4cols(at, g[0], g[1], g[2], g[3]);
                tmem_store_4cols(at + 4, u[0], u[1], u[2], u[3]);
                tmem_store_4cols(at + 8, x[0], x[1], x[2], x[3]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sff0 + 8 * sf);
                if (++sf == 2) {
                    sf = 0;
                    sf_phase ^= 1u;
                }
            }
        }
        const bool got = kb0 < kb1 && ok && mbar_wait(accf, 0, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
            if (lane == 0 && kb0 < kb1) raise_error(abort_flag);
            ok = false;
        }
        if (ok) {
            // all MMAs that read the tiles are done: the sums take their place
            tc_fence_after();
            const int part = warp < 6 ? 0 : 1;   // gate, value
            float *red = reinterpret_cast<float *>(smem) + part * kTile + r;
#pragma unroll
            for (int h = 0; h < NT / 16; ++h) {
                uint32_t v[16];
                tmem_load_16cols(lanes + part * NT + h * 16, v);
                tmem_wait_16cols(v);
#pragma unroll
                for (int c = 0; c < 16; ++c) red[(16 * h + c) * 256] = __uint_as_float(v[c]);
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
        const int tokens = a.M - token0 < NT ? static_cast<int>(a.M - token0) : NT;
        if (splits == 1)
            gated_join<1, 4, AFMT, HFMT>(a, smem_u32(smem), split, splits, token0, tokens, col0);
        else if (splits <= 4)
            gated_join<4, 2, AFMT, HFMT>(a, smem_u32(smem), split, splits, token0, tokens, col0);
        else
            gated_join<8, 1, AFMT, HFMT>(a, smem_u32(smem), split, splits, token0, tokens, col0);
    }
    __syncwarp();
    cluster_sync();   // the others have read this CTA's sums
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// --------------------------------------------------------------------- host --

template <bool BWD, int F0, int F1, int F2 = 0>
cudaError_t launch_pair(GatedArgs &a, int sm_count, cudaStream_t st, const char **what) {
    static PairKernel<GatedArgs> pk{gated_pair_kernel<BWD, F0, F1, F2>, Gated<BWD>::THREADS, Gated<BWD>::SMEM};
    int slots = 0;
    const cudaError_t e = pk.init(sm_count, &slots);
    if (e != cudaSuccess) return e;
    if (slots < 1) {
        *what = "no pair of SMs can hold the kernel";
        return cudaErrorInvalidConfiguration;
    }
    const BlockView &A = a.A, &B = a.B;
    if (!encode_tmap_2d(&a.mapA, A.codes, false, A.cols, A.rows, BK, BM, true, A.ld) ||
        !encode_tmap_2d(&a.mapB, B.codes, false, B.cols, B.rows, BK, BM, true, B.ld)) {
        *what = "cuTensorMapEncodeTiled failed for an operand";
        return cudaErrorInvalidValue;
    }
    if (!BWD && (!encode_tmap_2d(&a.map_a8, a.a8.codes, false, a.F, a.M, kTile, 32, true, a.a8.ld) ||
                 (a.h8.codes != nullptr &&
                  !encode_tmap_2d(&a.map_h8, a.h8.codes, false, 2 * a.F, a.M, kTile, 32, true, a.h8.ld)))) {
        *what = "cuTensorMapEncodeTiled failed for an output";
        return cudaErrorInvalidValue;
    }
    a.b_second = BWD ? BM : a.F;
    a.tile_cols = BWD ? BN : BM;
    a.tiles_m = static_cast<int>((a.M + 2 * BM - 1) / (2 * BM));
    a.tiles_n = static_cast<int>((a.F + a.tile_cols - 1) / a.tile_cols);
    a.whole = a.num_items = a.tiles_m * a.tiles_n;
    if (BWD) {
        // The last wave in halves (a block of da each) where there are pairs for them, or only
        // blocks where a pair has fewer of them in a row then: the elementwise part of one takes
        // some 9 us.  (1537 x 1031 -> 2688, 77 tiles or 147 blocks: 25.3 us in blocks, 33.2 with the last
        // wave in halves, 35.3 in whole tiles.)
        const int rest = a.whole % slots, waves = a.whole / slots;
        const int64_t blocks = a.tiles_m * (a.F / kTile);
        if ((blocks + slots - 1) / slots < 2 * waves + (rest == 0 ? 0 : 2 * rest <= slots ? 1 : 2)) {
            a.tile_cols = kTile;
            a.tiles_n = static_cast<int>(a.F / kTile);
            a.whole = 0;
            a.num_items = static_cast<int>(blocks);
        } else if (2 * rest <= slots) {
            a.whole -= rest;
            a.num_items += rest;
        }
        if (!encode_tmap_2d(&a.mapBHalf, B.codes, false, B.cols, B.rows, BK, BM / 2, true, B.ld)) {
            *what = "cuTensorMapEncodeTiled failed for an operand";
            return cudaErrorInvalidValue;
        }
    }
    a.num_kb = static_cast<int>((A.cols + BK - 1) / BK);
    a.group_m = raster_group(A.rows * A.cols, B.rows * B.cols, a.tiles_m);
    a.idesc = idesc_mxf8(static_cast<uint32_t>(A.fmt), static_cast<uint32_t>(B.fmt), 2 * BM, BN, 0);
    a.idesc_half = idesc_mxf8(static_cast<uint32_t>(A.fmt), static_cast<uint32_t>(B.fmt), 2 * BM, BN / 2, 0);
    const int units = a.num_items < slots ? a.num_items : slots;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(dim3(2 * units), Gated<BWD>::THREADS, Gated<BWD>::SMEM, 2, attr, st);
    return cudaLaunchKernelEx(&cfg, gated_pair_kernel<BWD, F0, F1, F2>, a);
}

template <int FMT, int AFMT>
cudaError_t launch_bwd_formats(GatedArgs &a, int sm_count, cudaStream_t st, const char **what) {
    return a.h8.fmt == 0 ? launch_pair<true, FMT, AFMT, 0>(a, sm_count, st, what)
                         : launch_pair<true, FMT, AFMT, 1>(a, sm_count, st, what);
}

template <int NT, int AFMT, int HFMT>
cudaError_t launch_gated_few(const GatedArgs &g, int sm_count, cudaStream_t st, const char **what) {
    using C = GatedFew<NT>;
    GatedFewArgs a{};
    if (!encode_tmap_2d(&a.mapW, g.B.codes, false, g.B.cols, g.B.rows, BK, BM, true, g.B.ld) ||
        !encode_tmap_2d(&a.mapX, g.A.codes, false, g.A.cols, g.A.rows, BK, NT, true, g.A.ld)) {
        *what = "cuTensorMapEncodeTiled failed for an operand";
        return cudaErrorInvalidValue;
    }
    a.W = g.B, a.X = g.A, a.a8 = g.a8, a.h8 = g.h8;
    a.M = g.M, a.F = g.F;
    a.num_kb = static_cast<int>((g.A.cols + BK - 1) / BK);
    a.idesc = idesc_mxf8(static_cast<uint32_t>(g.B.fmt), static_cast<uint32_t>(g.A.fmt), BM, NT, 0);
    static SmemLimit limit;
    const cudaError_t err = limit.allow(gated_few_kernel<NT, AFMT, HFMT>, C::SMEM);
    if (err != cudaSuccess) return err;
    const int64_t tf = g.F / kTile, tx = (g.M + NT - 1) / NT;
    // as many CTAs as the SMs have places for, with at least two k-blocks each.  A cluster stays
    // within a GPC, so that not all places can be used: with one CTA an SM 152 SMs run 36 clusters
    // of 4 at once, 28 of 5, 23 of 6, and 15 of 7 or 8.  Those beyond are a second wave (256 x 4096 ->
    // 1024, 16 clusters of 8: 19.3 us; 512 tokens, 32 of 4: 11.8).
    int64_t splits = static_cast<int64_t>(C::CTAS) * sm_count / (tf * tx);
    if (splits > a.num_kb / 2) splits = a.num_kb / 2;
    if (splits > C::MOST_SPLITS) splits = C::MOST_SPLITS;
    if (splits < 1) splits = 1;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg =
        cluster_config(dim3(static_cast<unsigned>(splits), static_cast<unsigned>(tf), static_cast<unsigned>(tx)),
                       C::THREADS, C::SMEM, static_cast<int>(splits), attr, st);
    return cudaLaunchKernelEx(&cfg, gated_few_kernel<NT, AFMT, HFMT>, a);
}

// The few kernel takes up to 128 tokens, and more as long as they are so few pair tiles that
// most SMs would idle, an eighth of the SMs' number.  M x K -> F with h kept, few and pair kernel in us:
// 128 x 4096 -> 11008 27.8 and 34.2, 128 x 1000 -> 2688 9.2 and 9.4; 512 x 4096 -> 1024 (16
// pair tiles) 11.8 and 15.7, 129 x 4096 -> 1024 (8) 11.8 and 15.4, 256 x 4096 -> 2048 (16) 12.2 and 17.5;
// 256 x 1000 -> 2688 (21) 10.1 and 9.4, 600 x 1024 -> 1024 (24) 9.4 and 9.2, 777 x 1000 -> 2688
// (84) 15.9 and 13.1.  The rule does not see the second wave of clusters, and takes the slower
// kernel where there is one with work: 200 x 4096 -> 1024 16.8 and 15.4, 256 x 4096 -> 1024 19.3
// and 15.5, 256 x 1000 -> 2432 (19; 38 clusters of 4) 17.2 and 9.4.
constexpr int64_t kFewTokens = 128;

template <int AFMT, int HFMT>
cudaError_t launch_fwd_formats(GatedArgs &a, int sm_count, cudaStream_t st, const char **what) {
    const int64_t tf = a.F / kTile;
    if (tf <= 65535) {   // tiles count in gridDim.y
        if (a.M <= 16) return launch_gated_few<16, AFMT, HFMT>(a, sm_count, st, what);
        if (a.M <= 32) return launch_gated_few<32, AFMT, HFMT>(a, sm_count, st, what);
        if (a.M <= 64) return launch_gated_few<64, AFMT, HFMT>(a, sm_count, st, what);
        if (a.M <= kFewTokens || tf * ((a.M + 255) / 256) <= sm_count / 8)
            return launch_gated_few<128, AFMT, HFMT>(a, sm_count, st, what);
    }
    return launch_pair<false, AFMT, HFMT>(a, sm_count, st, what);
}

}  // namespace

cudaError_t launch_gated_fwd(const BlockView &A, const BlockView &B, const BlockView &a8, const BlockView &h8,
                             int sm_count, cudaStream_t st, const char **what) {
    if (A.rows == 0 || B.rows == 0) return cudaSuccess;
    GatedArgs a{};
    a.A = A, a.B = B, a.a8 = a8, a.h8 = h8;
    a.M = A.rows, a.F = B.rows / 2;
    const int hfmt = h8.codes != nullptr ? h8.fmt : 0;
    if (a8.fmt == 0)
        return hfmt == 0 ? launch_fwd_formats<0, 0>(a, sm_count, st, what)
                         : launch_fwd_formats<0, 1>(a, sm_count, st, what);
    return hfmt == 0 ? launch_fwd_formats<1, 0>(a, sm_count, st, what)
                     : launch_fwd_formats<1, 1>(a, sm_count, st, what);
}

cudaError_t launch_gated_bwd(const BlockView &A, const BlockView &B, const BlockView &h8, const BlockView &dh8,
                             const BlockView &dh8t, const BlockView &a8t, int sm_count, cudaStream_t st,
                             const char **what) {
    if (A.rows == 0 || B.rows == 0) return cudaSuccess;
    GatedArgs a{};
    a.A = A, a.B = B, a.h8 = h8, a.dh8 = dh8, a.dh8t = dh8t, a.a8t = a8t;
    a.M = A.rows, a.F = B.rows;
    const int fmt = dh8.codes != nullptr ? dh8.fmt : dh8t.codes != nullptr ? dh8t.fmt : 0;
    const int afmt = a8t.codes != nullptr ? a8t.fmt : 0;
    if (fmt == 0)
        return afmt == 0 ? launch_bwd_formats<0, 0>(a, sm_count, st, what)
                         : launch_bwd_formats<0, 1>(a, sm_count, st, what);
    return afmt == 0 ? launch_bwd_formats<1, 0>(a, sm_count, st, what)
                     : launch_bwd_formats<1, 1>(a, sm_count, st, what);
}

cudaError_t read_and_clear_gated_error_flag(unsigned *flags) {
    return take_error_flags(&g_gated_error_flags, flags);
}

}  // namespace fp8k
