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
// Two CTAs on two SMs (a cluster) share each tile of 256 rows of A and 256 rows of B
// (cta_group::2): each loads its own 128 rows of either, and the even CTA issues the
// MMAs, whose 256 sums for each of a CTA's 128 rows fill half of its TMEM.  Forward:
// the even CTA's rows of B are gates and the odd one's the values that belong to them, so
// that columns j and 128 + j of a tile make one a, and a tile is one block of a wide.
// Backward: 256 columns of da, two blocks.
//
// Warps: 0 TMA, 1 MMA (2 and 3 idle), 4-7 scales, 8-15 the elementwise part (warp w has the
// TMEM lanes 32 (w mod 4) .. + 31, a row of the tile each, and half of the columns of a
// block), of one tile while the next one's MMAs run.  Of the launch's 512 x 128 registers
// the first eight warps hand back 64 each per thread and the other eight take them.
//
// TMEM: as in the matrix product of block_gemm.cu the two accumulators overlap by 32 columns
// (0-255 and 224-479), and columns 480-511 hold two stages of scales.  The elementwise
// warps read the shared columns first and then let the next tile's MMAs start.
//
// Every wait is bounded.
#include <cstdint>

#include "block_mma.cuh"
#include "raster.cuh"

namespace fp8k {

namespace {

__device__ unsigned g_gated_error_flags = 0;

__device__ __forceinline__ void raise_error(volatile int *abort_flag) {
    atomicOr(&g_gated_error_flags, kErrWaitTimeout);
    *abort_flag = 1;
}

constexpr int GP_THREADS = 512;
constexpr int GP_REGS_CONTROL = 64, GP_REGS_ELEMENTS = 192;
static_assert(256 * GP_REGS_CONTROL + 256 * GP_REGS_ELEMENTS <= GP_THREADS * 128, "register split");

struct GatedArgs {
    CUtensorMap mapA, mapB;
    BlockView A, B;
    int64_t M, F;
    int64_t b_second;   // from the even CTA's first row of B to the odd one's
    int tile_cols;      // columns of a or da in a tile
    int tiles_m, tiles_n, num_tiles, num_kb, group_m;
    uint32_t idesc;
    BlockView a8, h8;              // forward: outputs (h8's codes may be null); backward: h8 is read
    BlockView dh8, dh8t, a8t;      // backward: outputs, codes null: not wanted
};

struct Tile {
    int64_t row0, col0;   // of the pair's 256 rows; of the columns of a or da
};
__device__ __forceinline__ Tile tile_at(const GatedArgs &a, int tile) {
    int mb, nb;
    tile_coords(tile, a.tiles_m, a.tiles_n, a.group_m, mb, nb);
    return Tile{static_cast<int64_t>(mb) * 2 * BM, static_cast<int64_t>(nb) * a.tile_cols};
}

// What the elementwise warps of a CTA share.
template <bool BWD>
struct GatedShared;
template <>
struct GatedShared<false> {
    float3 row_max[2][2][BM];   // [tile mod 2][half of the columns][row]: of a, gate, value
};
template <>
struct GatedShared<true> {
    uint8_t codes[3][kTile * kTile];   // [d gate, d value, a][column][row]
    uint32_t col_max[3][4][kTile];     // [..][lane quarter][column]
    float inv[3][kTile];
    float2 row_max[2][BM];             // [half of the columns][row]: of d gate, d value
};

template <bool BWD>
struct Gated {
    static constexpr int STAGES = BWD ? 5 : 6;
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
    for (int tile = unit; ok && tile < a.num_tiles; tile += num_units) {
        const Tile t = tile_at(a, tile);
        const int32_t arow = static_cast<int32_t>(t.row0 + rank * BM);
        const int32_t brow = static_cast<int32_t>(t.col0 + rank * a.b_second);
        for (int kb = 0; kb < a.num_kb; ++kb) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag))) {
                if ((threadIdx.x & 31) == 0) raise_error(abort_flag);
                ok = false;
                break;
            }
            if (elect_one()) {
                // both CTAs' halves complete on the even CTA's barrier
                const uint32_t fb = full0 + 8 * stage, fb0 = mapa_shared(fb, 0);
                if (rank == 0) mbar_arrive_expect_tx(fb, 4 * HALF);
                tma_load_2d_pair(sA + stage * HALF, &a.mapA, fb0, kb * BK, arow);
                tma_load_2d_pair(sB + stage * HALF, &a.mapB, fb0, kb * BK, brow);
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
    for (int tile = unit; ok && tile < a.num_tiles; tile += num_units, ++it) {
        // the previous tile's shared columns have been read
        const bool freed = it == 0 || mbar_wait(acce, static_cast<uint32_t>(it - 1) & 1u, abort_flag);
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
                const uint32_t idesc = a.idesc | static_cast<uint32_t>(kb & 3) << 4 |
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
    for (int tile = unit; ok && tile < a.num_tiles; tile += num_units) {
        const Tile t = tile_at(a, tile);
        const uint8_t *ra[4], *rb[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = min(t.row0 + rank * BM + 32 * j + lane, a.M - 1);
            ra[j] = static_cast<const uint8_t *>(a.A.scales) + (a.A.block_rows == 1 ? r : r >> 7) * a.A.ld_s;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t r = min(t.col0 + (j >> 2) * a.b_second + 32 * (j & 3) + lane, a.B.rows - 1);
            rb[j] = static_cast<const uint8_t *>(a.B.scales) + (a.B.block_rows == 1 ? r : r >> 7) * a.B.ld_s;
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

// 16 values of a row to 16 bytes of codes
template <int FMT>
__device__ __forceinline__ void store_codes16(uint8_t *p, const uint64_t *v, float inv) {
    const uint64_t inv2 = splat_f32x2(inv);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = encode4<FMT>(f32x2_mul(v[2 * i], inv2), f32x2_mul(v[2 * i + 1], inv2));
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// AFMT, HFMT: formats of a8 and h8.
template <int AFMT, int HFMT>
__device__ __forceinline__ bool gated_fwd_tile(const GatedArgs &a, GatedShared<false> &sm, const Tile &tile,
                                               uint32_t rank, int it, uint32_t tmem, uint32_t acce0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, half = (warp - 8) >> 2;
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
    asm volatile("bar.sync %0, 64;" ::"r"(2 + q) : "memory");
    const float3 other = sm.row_max[it & 1][half ^ 1][r];
    const uint32_t ba = scale_byte<AFMT>(__float_as_uint(fmaxf(ma, other.x)));
    const uint32_t bg = scale_byte<HFMT>(__float_as_uint(fmaxf(mg, other.y)));
    const uint32_t bu = scale_byte<HFMT>(__float_as_uint(fmaxf(mu, other.z)));
    const int64_t row = tile.row0 + rank * BM + r;
    const bool in = row < a.M, keep_h = a.h8.codes != nullptr;
    if (in && half == 0) {
        store_scale(a.a8, row, tile.col0 / kTile, ba);
        if (keep_h) {
            store_scale(a.h8, row, tile.col0 / kTile, bg);
            store_scale(a.h8, row, (a.F + tile.col0) / kTile, bu);
        }
    }
    if (in) {
        uint8_t *p = a.a8.codes + row * a.a8.ld + tile.col0 + 64 * half;
#pragma unroll
        for (int c = 0; c < 4; ++c) store_codes16<AFMT>(p + 16 * c, av + 8 * c, scale_inverse(ba));
    }
    if (keep_h) {
        uint8_t *p = a.h8.codes + row * a.h8.ld + tile.col0 + 64 * half;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint64_t g[8], u[8];
            gate_value16(t, c, keep, keep_g, keep_u, g, u);
            if (in) {
                store_codes16<HFMT>(p + 16 * c, g, scale_inverse(bg));
                store_codes16<HFMT>(p + a.F + 16 * c, u, scale_inverse(bu));
            }
        }
    }
    tc_fence_before();
    return true;
}

// gate and value of 4 columns from their codes
__device__ __forceinline__ void decode_pairs(uint32_t w, int fmt, uint64_t scale2, uint64_t (&v)[2]) {
    float f[4];
    decode4(w, fmt, f);
    v[0] = f32x2_mul(f32x2_pack(f[0], f[1]), scale2);
    v[1] = f32x2_mul(f32x2_pack(f[2], f[3]), scale2);
}
__device__ __forceinline__ uint32_t word_of(const uint4 (&u)[4], int i) {
    const uint4 &v = u[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
}

// The largest magnitudes of 4 columns over the warp's rows; column k's goes to lane k0 + k.
__device__ __forceinline__ void column_max4(const uint64_t (&v)[2], bool inf, int k0, uint32_t &mine) {
    const int lane = threadIdx.x & 31;
    float x[4];
    f32x2_unpack(inf ? without_inf(v[0]) : v[0], x[0], x[1]);
    f32x2_unpack(inf ? without_inf(v[1]) : v[1], x[2], x[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(absmax3(0.0f, x[k], x[k])));
        if (lane == k0 + k) mine = m;
    }
}

// 4 columns' codes of this lane's row into a tile kept by columns
template <int FMT>
__device__ __forceinline__ void put_columns4(uint8_t *codes, const uint64_t (&v)[2], const float4 &inv) {
    const uint32_t w = encode4<FMT>(f32x2_mul(v[0], f32x2_pack(inv.x, inv.y)), f32x2_mul(v[1], f32x2_pack(inv.z, inv.w)));
#pragma unroll
    for (int k = 0; k < 4; ++k) codes[k * kTile] = static_cast<uint8_t>(w >> (8 * k));
}

// One block of 128 columns of da; `first`: the one that holds the columns shared by the two
// accumulators.  FMT, AFMT: formats of dh8 / dh8t and of a8t.
template <int FMT, int AFMT>
__device__ __forceinline__ void gated_bwd_block(const GatedArgs &a, GatedShared<true> &sm, int64_t row0, int64_t col0,
                                                bool first, uint32_t t, uint32_t acce0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, half = (warp - 8) >> 2;
    const int et = threadIdx.x - 256, r = 32 * q + lane;
    const int64_t row = row0 + r;
    const bool in = row < a.M;
    const bool want_t = a.dh8t.codes != nullptr, want_a = a.a8t.codes != nullptr, want_r = a.dh8.codes != nullptr;
    uint4 gc[4], uc[4];
    float sg = 0.0f, su = 0.0f;
    auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < 4; ++i) gc[i] = uc[i] = make_uint4(0, 0, 0, 0);
        if (in) {
            const uint8_t *p = a.h8.codes + row * a.h8.ld + col0 + 64 * half;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                gc[i] = reinterpret_cast<const uint4 *>(p)[i];
                uc[i] = reinterpret_cast<const uint4 *>(p + a.F)[i];
            }
        }
    };
    if (in) {
        sg = load_scale(a.h8, row, col0 / kTile);
        su = load_scale(a.h8, row, (a.F + col0) / kTile);
    }
    fetch();
    const uint64_t sg2 = splat_f32x2(sg), su2 = splat_f32x2(su), one2 = splat_f32x2(1.0f);
    uint64_t dg[32], du[32];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t v[16];
        tmem_load_16cols(t + 64 * half + 16 * c, v);
        tmem_wait_16cols(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) du[8 * c + i] = pair_of(v[2 * i], v[2 * i + 1]);   // da for now
    }
    if (first) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acce0);
    }
    float mg = 0.0f, mu = 0.0f;
    uint32_t mine[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) {   // 4 columns at a time
        uint64_t g[2], u[2], av[2];
        decode_pairs(word_of(gc, i), a.h8.fmt, sg2, g);
        decode_pairs(word_of(uc, i), a.h8.fmt, su2, u);
        float m = 0.0f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float g0, g1;
            f32x2_unpack(g[p], g0, g1);
            const uint64_t s = sigmoid2(g0, g1), gs = f32x2_mul(g[p], s), d = du[2 * i + p];
            av[p] = f32x2_mul(gs, u[p]);
            dg[2 * i + p] = f32x2_mul(f32x2_mul(f32x2_mul(d, u[p]), s), f32x2_fma(g[p], f32x2_sub(one2, s), one2));
            du[2 * i + p] = f32x2_mul(d, gs);
            m = absmax3(absmax3(absmax3(m, av[p]), dg[2 * i + p]), du[2 * i + p]);
        }
        const bool inf = is_inf(m);
        const uint64_t dgp[2] = {dg[2 * i], dg[2 * i + 1]}, dup[2] = {du[2 * i], du[2 * i + 1]};
        mg = block_max(dgp, mg);
        mu = block_max(dup, mu);
        if (want_t) {
            column_max4(dgp, inf, (4 * i) & 31, mine[0]);
            column_max4(dup, inf, (4 * i) & 31, mine[1]);
        }
        if (want_a) column_max4(av, inf, (4 * i) & 31, mine[2]);
        if ((i & 7) == 7) {
#pragma unroll
            for (int k = 0; k < 3; ++k) sm.col_max[k][q][64 * half + 4 * (i & 8) + lane] = mine[k];
        }
    }
    sm.row_max[half][r] = make_float2(mg, mu);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    for (int i = et; i < 3 * kTile; i += 256) {
        const int k = i / kTile, c = i % kTile;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = max(m, sm.col_max[k][w][c]);
        const uint32_t byte = k == 2 ? scale_byte<AFMT>(m) : scale_byte<FMT>(m);
        sm.inv[k][c] = scale_inverse(byte);
        if (row0 < a.M) {
            if (k < 2 && want_t) store_scale(a.dh8t, (k ? a.F : 0) + col0 + c, row0 / kTile, byte);
            if (k == 2 && want_a) store_scale(a.a8t, col0 + c, row0 / kTile, byte);
        }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (want_r && in) {
        const float2 other = sm.row_max[half ^ 1][r];
        const uint32_t bg = scale_byte<FMT>(__float_as_uint(fmaxf(mg, other.x)));
        const uint32_t bu = scale_byte<FMT>(__float_as_uint(fmaxf(mu, other.y)));
        if (half == 0) {
            store_scale(a.dh8, row, col0 / kTile, bg);
            store_scale(a.dh8, row, (a.F + col0) / kTile, bu);
        }
        uint8_t *p = a.dh8.codes + row * a.dh8.ld + col0 + 64 * half;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            store_codes16<FMT>(p + 16 * c, dg + 8 * c, scale_inverse(bg));
            store_codes16<FMT>(p + a.F + 16 * c, du + 8 * c, scale_inverse(bu));
        }
    }
    if (want_t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int c = 64 * half + 4 * i;
            const uint64_t dgp[2] = {dg[2 * i], dg[2 * i + 1]}, dup[2] = {du[2 * i], du[2 * i + 1]};
            put_columns4<FMT>(&sm.codes[0][c * kTile + r], dgp, *reinterpret_cast<const float4 *>(&sm.inv[0][c]));
            put_columns4<FMT>(&sm.codes[1][c * kTile + r], dup, *reinterpret_cast<const float4 *>(&sm.inv[1][c]));
        }
    }
    if (want_a) {
        fetch();   // again: kept, they would not fit beside dg and du
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int c = 64 * half + 4 * i;
            uint64_t g[2], u[2];
            decode_pairs(word_of(gc, i), a.h8.fmt, sg2, g);
            decode_pairs(word_of(uc, i), a.h8.fmt, su2, u);
            const uint64_t av[2] = {silu_times(g[0], u[0]), silu_times(g[1], u[1])};
            put_columns4<AFMT>(&sm.codes[2][c * kTile + r], av, *reinterpret_cast<const float4 *>(&sm.inv[2][c]));
        }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    // the columns leave as rows of 128 bytes, 8 threads each
    const int k = et & 7, c0 = et >> 3;
    const int64_t left = a.M - (row0 + 16 * k);
    auto store = [&](const BlockView &o, int64_t first_row, const uint8_t *codes) {
        uint8_t *p = o.codes + (first_row + c0) * o.ld + row0 + 16 * k;
#pragma unroll
        for (int i = 0; i < kTile / 32; ++i, p += 32 * o.ld) {
            const uint4 u = *reinterpret_cast<const uint4 *>(codes + (c0 + 32 * i) * kTile + 16 * k);
            if (left >= 16) {
                *reinterpret_cast<uint4 *>(p) = u;
            } else if (left > 0) {
                store_code_word(p, u.x, left);
                store_code_word(p + 4, u.y, left - 4);
                store_code_word(p + 8, u.z, left - 8);
                store_code_word(p + 12, u.w, left - 12);
            }
        }
    };
    if (want_t) {
        store(a.dh8t, col0, sm.codes[0]);
        store(a.dh8t, a.F + col0, sm.codes[1]);
    }
    if (want_a) store(a.a8t, col0, sm.codes[2]);
}

// F0, F1: formats of a8 and h8, or of dh8 / dh8t and a8t.
template <bool BWD, int F0, int F1>
__global__ void __launch_bounds__(GP_THREADS, 1) gated_pair_kernel(const __grid_constant__ GatedArgs a) {
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
        mbar_init(acce, 16);              // eight elementwise warps of each CTA
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&a.mapA);
        prefetch_tmap(&a.mapB);
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

    if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(GP_REGS_CONTROL));
        if (warp == 0)
            gated_produce<C::STAGES>(a, rank, unit, num_units, sA, sB, full0, empty0, abort_flag);
        else if (warp == 1 && rank == 0)
            gated_mma<C::STAGES>(a, unit, num_units, tmem, sA, sB, full0, empty0, accf0, acce, sff0, sfe0, drain,
                                 abort_flag);
        else if (warp >= 4)
            gated_scales(a, rank, unit, num_units, tmem, sff0, sfe0, abort_flag);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(GP_REGS_ELEMENTS));
        const uint32_t acce0 = mapa_shared(acce, 0);
        int it = 0;
        for (int i = unit; i < a.num_tiles; i += num_units, ++it) {
            const Tile tile = tile_at(a, i);
            const bool got = mbar_wait(accf0 + 8 * (it & 1), static_cast<uint32_t>(it >> 1) & 1u, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got) && lane == 0) raise_error(abort_flag);
            // all go on or none: a warp alone in a tile's barriers would stay there
            if (!barrier_and(1, 256, got)) break;
            tc_fence_after();
            if constexpr (BWD) {
                const uint32_t t = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + ((it & 1) ? MX_ACC1 : 0);
                const int64_t row0 = tile.row0 + rank * BM;
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    const int b = (it & 1) ? j : 1 - j;   // the shared columns' block first
                    if (tile.col0 + b * kTile < a.F) {
                        gated_bwd_block<F0, F1>(a, sm, row0, tile.col0 + b * kTile, j == 0, t + b * kTile, acce0);
                    } else if (j == 0) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_relaxed(acce0);
                    }
                }
                tc_fence_before();
            } else {
                gated_fwd_tile<F0, F1>(a, sm, tile, rank, it, tmem, acce0);
            }
        }
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

// --------------------------------------------------------------------- host --

template <bool BWD, int F0, int F1>
cudaError_t launch_pair(GatedArgs &a, int sm_count, cudaStream_t st, const char **what) {
    static PairKernel<GatedArgs> pk{gated_pair_kernel<BWD, F0, F1>, GP_THREADS, Gated<BWD>::SMEM};
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
    a.b_second = BWD ? BM : a.F;
    a.tile_cols = BWD ? BN : BM;
    a.tiles_m = static_cast<int>((a.M + 2 * BM - 1) / (2 * BM));
    a.tiles_n = static_cast<int>((a.F + a.tile_cols - 1) / a.tile_cols);
    a.num_tiles = a.tiles_m * a.tiles_n;
    a.num_kb = static_cast<int>((A.cols + BK - 1) / BK);
    a.group_m = raster_group(A.rows * A.cols, B.rows * B.cols, a.tiles_m);
    a.idesc = idesc_mxf8(static_cast<uint32_t>(A.fmt), static_cast<uint32_t>(B.fmt), 2 * BM, BN, 0);
    const int units = a.num_tiles < slots ? a.num_tiles : slots;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(dim3(2 * units), GP_THREADS, Gated<BWD>::SMEM, 2, attr, st);
    return cudaLaunchKernelEx(&cfg, gated_pair_kernel<BWD, F0, F1>, a);
}

template <bool BWD>
cudaError_t launch_pair_formats(GatedArgs &a, int f0, int f1, int sm_count, cudaStream_t st, const char **what) {
    if (f0 == 0)
        return f1 == 0 ? launch_pair<BWD, 0, 0>(a, sm_count, st, what) : launch_pair<BWD, 0, 1>(a, sm_count, st, what);
    return f1 == 0 ? launch_pair<BWD, 1, 0>(a, sm_count, st, what) : launch_pair<BWD, 1, 1>(a, sm_count, st, what);
}

}  // namespace

cudaError_t launch_gated_fwd(const BlockView &A, const BlockView &B, const BlockView &a8, const BlockView &h8,
                             int sm_count, cudaStream_t st, const char **what) {
    if (A.rows == 0 || B.rows == 0) return cudaSuccess;
    GatedArgs a{};
    a.A = A, a.B = B, a.a8 = a8, a.h8 = h8;
    a.M = A.rows, a.F = B.rows / 2;
    return launch_pair_formats<false>(a, a8.fmt, h8.codes != nullptr ? h8.fmt : 0, sm_count, st, what);
}

cudaError_t launch_gated_bwd(const BlockView &A, const BlockView &B, const BlockView &h8, const BlockView &dh8,
                             const BlockView &dh8t, const BlockView &a8t, int sm_count, cudaStream_t st,
                             const char **what) {
    if (A.rows == 0 || B.rows == 0) return cudaSuccess;
    GatedArgs a{};
    a.A = A, a.B = B, a.h8 = h8, a.dh8 = dh8, a.dh8t = dh8t, a.a8t = a8t;
    a.M = A.rows, a.F = B.rows;
    const int fmt = dh8.codes != nullptr ? dh8.fmt : dh8t.codes != nullptr ? dh8t.fmt : 0;
    return launch_pair_formats<true>(a, fmt, a8t.codes != nullptr ? a8t.fmt : 0, sm_count, st, what);
}

cudaError_t read_and_clear_gated_error_flag(unsigned *flags) {
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_gated_error_flags, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_gated_error_flags, &zero, sizeof(unsigned));
}

}  // namespace fp8k
