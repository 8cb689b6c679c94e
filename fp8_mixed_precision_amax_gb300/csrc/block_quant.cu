// block_quant.cu -- block-scaled quantization of a matrix, of its transpose and
// of what a backward pass computes from an input kept in 8 bits: LayerNorm's
// output again, and SwiGLU forward and backward.  The formulas are in
// include/fp8amax.h; block.cuh has the scale rule and the tile's layout.
//
// Each value is read once and each result written once.  What has to be written
// transposed goes tile by tile (128 x 128, one block wide both ways), the rest row by
// row.  HBM is the floor; the instructions per element bind before it where much is
// computed of each.
#include <cstdint>

#include "block.cuh"
#include "once_per_device.h"

namespace fp8k {

namespace {

// ----------------------------------------------------------- quantization --

template <typename T>
struct QuantSmem {
    uint8_t in[2][kTile * kTile * sizeof(T)];
    ColsSmem cols;
    uint32_t red[2][16];
};

// Both ways or the transpose alone; also tiles row-major.  Two CTAs per SM, so that one's
// barriers fall into the other's work: 8192 x 4096 BF16 both ways 24 us, 5.6 TB/s of the
// bytes it must move (0.83 of a copy's rate); 1000 x 2731 fp32 in tiles 9.4 us, a latency.
template <typename T, int FMT, bool TILE>
__global__ void __launch_bounds__(kTileThreads, sizeof(T) == 4 ? 1 : 2)
    block_quantize_kernel(const T *__restrict__ x, int64_t rows, int64_t cols, int64_t ld, bool vec,
                          const BlockView q, const BlockView qt, unsigned tiles_r,
                          unsigned tiles_c) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    QuantSmem<T> &sm = *reinterpret_cast<QuantSmem<T> *>(smem_raw);
    const int part = (threadIdx.x >> 5) * kTileRows * kTile * static_cast<int>(sizeof(T));
    pdl_wait();
    pdl_trigger();
    TileWalk walk(tiles_r, tiles_c);
    unsigned row0, col0;
    walk.origin(row0, col0);
    fetch_rows<sizeof(T)>(smem_u32(sm.in[0]) + part, x, ld, rows, cols, vec, row0, col0);
    cp_async_commit();
    int stage = 0;
    for (bool more = true; more; stage ^= 1) {
        unsigned next_row0 = 0, next_col0 = 0;
        walk.next();
        more = walk.there();
        __syncwarp();   // the warp has read this part of the other stage
        if (more) {
            walk.origin(next_row0, next_col0);
            fetch_rows<sizeof(T)>(smem_u32(sm.in[stage ^ 1]) + part, x, ld, rows, cols, vec,
                                  next_row0, next_col0);
        }
        cp_async_commit();
        cp_async_wait<1>();
        __syncwarp();
        TileValues v;
#pragma unroll
        for (int r = 0; r < kTileRows; ++r) staged4<T>(sm.in[stage] + part, r, v[r]);
        int byte = -1;
        if constexpr (TILE) byte = static_cast<int>(scale_byte<FMT>(tile_max(v, sm.red[stage])));
        if (qt.codes != nullptr) {
            ulonglong2 inv;
            if constexpr (TILE) {
                if (threadIdx.x == 0) store_scale(qt, col0 / kTile, row0 / kTile, byte);
                inv.x = inv.y = splat_f32x2(scale_inverse(byte));
            } else {
                cols_max(v, sm.cols);
                __syncthreads();
                if (threadIdx.x < kTile) cols_scale<FMT>(threadIdx.x, sm.cols, qt, row0, col0);
                __syncthreads();
                inv = cols_inv(sm.cols);
            }
            cols_codes<FMT>(v, inv, sm.cols);
        }
        if (q.codes != nullptr) tile_rows<FMT>(v, q, row0, col0, byte);
        if (qt.codes != nullptr) {
            __syncthreads();
            cols_store(sm.cols, qt, row0, col0);
            // with tiles, nothing else keeps the next codes from overtaking these reads
            if constexpr (TILE) __syncthreads();
        }
        row0 = next_row0, col0 = next_col0;
    }
}

// One warp per 1024 columns of a row, 8 per lane and step of 256.  8192 x 4096 to BF16:
// 23.4 us, 4.3 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) block_dequantize_kernel(const BlockView q, T *__restrict__ out,
                                                               int64_t ld, bool vec) {
    pdl_wait();
    pdl_trigger();
    const int64_t segs = (q.cols + 1023) / 1024;
    const int64_t total = q.rows * segs;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); s < total;
         s += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t row = s / segs, c0 = (s % segs) * 1024 + 8 * (threadIdx.x & 31);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t c = c0 + 256 * k;
            if (c >= q.cols) break;
            float v[8];
            load_codes<8>(q.codes + row * q.ld, c, q.cols, q.fmt,
                          load_scale(q, row / q.block_rows, c >> 7), v);
            store_row<T, 8>(out + row * ld, c, q.cols, vec, v);
        }
    }
}

// ------------------------------------------------ LayerNorm's output again --

// gamma or beta at columns c .. c + 3 as packed pairs; 0 past the row.  One branch on the
// type, so that the loads are on their way together.
__device__ __forceinline__ void load_param4(const void *p, int type, int64_t c, int64_t cols,
                                            uint64_t (&v)[2]) {
    const bool vec = (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && c + 4 <= cols;
    float f[4];
    if (type == kTypeF32)
        load_row<float, 4>(static_cast<const float *>(p), c, cols, vec, f);
    else if (type == kTypeBF16)
        load_row<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(p), c, cols, vec, f);
    else
        load_row<__half, 4>(static_cast<const __half *>(p), c, cols, vec, f);
    v[0] = f32x2_pack(f[0], f[1]);
    v[1] = f32x2_pack(f[2], f[3]);
}

struct RecomputeSmem {
    uint8_t in[2][kTile * kTile];
    ColsSmem cols;
};

// The forward's formula on the codes, so the same roundings.  8192 x 4096: 21.5 us, bound
// by instructions; reading and writing alone is 10.  (With scalar arithmetic, a bound on
// every element and the rows' statistics fetched when needed: 32.)
template <int FMT>
__global__ void __launch_bounds__(kTileThreads, 2)
    ln_recompute_kernel(const BlockView x8, const void *__restrict__ gamma,
                        const void *__restrict__ beta, int wtype, const float *__restrict__ mean,
                        const float *__restrict__ rstd, const BlockView yt, unsigned tiles_r,
                        unsigned tiles_c) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    RecomputeSmem &sm = *reinterpret_cast<RecomputeSmem *>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp * kTileRows * kTile;
    pdl_wait();
    pdl_trigger();
    TileWalk walk(tiles_r, tiles_c);
    unsigned row0, col0;
    walk.origin(row0, col0);
    fetch_rows<1>(smem_u32(sm.in[0]) + part, x8.codes, x8.ld, x8.rows, up16(x8.cols), true, row0, col0);
    cp_async_commit();
    // lane r: row r's scale and statistics, a tile ahead
    uint32_t sc_next = 0;
    float mu_next = 0.0f, rs_next = 0.0f;
    auto fetch_stats = [&](unsigned r0, unsigned c0) {
        const unsigned row = r0 + warp * kTileRows + (lane & 7);
        if (row < x8.rows) {
            sc_next = fetch_scale(x8, row, c0 / kTile);
            mu_next = mean[row], rs_next = rstd[row];
        }
    };
    fetch_stats(row0, col0);
    int stage = 0;
    for (bool more = true; more; stage ^= 1) {
        unsigned next_row0 = 0, next_col0 = 0;
        walk.next();
        more = walk.there();
        __syncwarp();
        if (more) {
            walk.origin(next_row0, next_col0);
            fetch_rows<1>(smem_u32(sm.in[stage ^ 1]) + part, x8.codes, x8.ld, x8.rows, up16(x8.cols),
                          true, next_row0, next_col0);
        }
        cp_async_commit();
        const float sc = fetched_scale(x8, sc_next), nmu = -mu_next, rs = rs_next;
        if (more) fetch_stats(next_row0, next_col0);
        uint64_t g[2], b[2];
        load_param4(gamma, wtype, col0 + 4 * lane, x8.cols, g);
        load_param4(beta, wtype, col0 + 4 * lane, x8.cols, b);
        cp_async_wait<1>();
        __syncwarp();
        // columns past the end may hold anything: they are rows of yt that are not stored
        TileValues v;
#pragma unroll
        for (int r = 0; r < kTileRows; ++r) {
            const uint64_t s2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, sc, r));
            const uint64_t nm2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, nmu, r));
            const uint64_t rs2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, rs, r));
            float f[4];
            decode4(*reinterpret_cast<const uint32_t *>(sm.in[stage] + part + r * kTile + lane * 4), x8.fmt, f);
#pragma unroll
            for (int p = 0; p < 2; ++p)
                v[r][p] = f32x2_fma(f32x2_mul(f32x2_fma(f32x2_pack(f[2 * p], f[2 * p + 1]), s2, nm2), rs2),
                                    g[p], b[p]);
        }
        if (row0 + kTile > x8.rows) {
#pragma unroll
            for (int r = 0; r < kTileRows; ++r)
                if (row0 + warp * kTileRows + r >= x8.rows) v[r][0] = v[r][1] = 0;
        }
        cols_max(v, sm.cols);
        __syncthreads();
        if (threadIdx.x < kTile) cols_scale<FMT>(threadIdx.x, sm.cols, yt, row0, col0);
        __syncthreads();
        cols_codes<FMT>(v, cols_inv(sm.cols), sm.cols);
        __syncthreads();
        cols_store(sm.cols, yt, row0, col0);
        row0 = next_row0, col0 = next_col0;
    }
}

// ----------------------------------------------------------------- SwiGLU --

// 1 / (1 + exp(-x)) of a pair to a few units in the last place and |x| 2^-24: 0 for -inf, 1
// for +inf.  The instructions that flush subnormal numbers serve here: exp(-x) below 2^-126
// is nothing beside 1, and the reciprocal is taken of a quarter of 1 + exp(-x), so that it
// stays a normal number as long as exp(-x) is finite (x > -88.7) and the last product gives
// the result below 2^-126 that a block of such gates is made of: its scale may be as small
// as 2^-127.  (SwiGLU's backward at 8192 x 11008: 178.5 us; 176 without the quarter, where
// such a block comes out as zeros, and 189.5 with the reciprocal that keeps subnormal numbers.)
__device__ __forceinline__ uint64_t sigmoid2(float x, float y) {
    float s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(i ? y : x, -1.44269504f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(__fmaf_rn(e, 0.25f, 0.25f)));
    }
    return f32x2_mul(f32x2_pack(s[0], s[1]), splat_f32x2(0.25f));
}

// 8 lanes per block of 128 columns of a row, four blocks per warp.  8192 x 11008 BF16
// with h kept: 127 us, where reading and writing alone is 93; 777 x 2688 4.1 and 2.2.  (16
// lanes per block, with twice the exchanges and scales per value: 146 and 4.4, but 2.2 for
// one token of 11008, here 2.7.)
template <typename T>
__global__ void __launch_bounds__(256) swiglu_fwd_kernel(const T *__restrict__ h, int64_t M, int64_t F,
                                                         int64_t ld, bool vec, const BlockView a8,
                                                         const BlockView h8) {
    pdl_wait();
    pdl_trigger();
    const unsigned per_row = static_cast<unsigned>(F / 128);
    const int64_t total = M * per_row, step = static_cast<int64_t>(gridDim.x) * 32;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 5) * 4; w < total;
         w += step) {
        // the warp's later quarters may be past the end: they repeat the first one's block
        int64_t blk = w + ((threadIdx.x >> 3) & 3);
        if (blk >= total) blk = w;
        // a division of 32 bits where that is enough
        const int64_t row = total >> 32 ? blk / per_row : static_cast<uint32_t>(blk) / per_row;
        const int64_t c = (blk - row * per_row) * 128 + 16 * (threadIdx.x & 7);
        float g[16], u[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            load_row<T, 8>(h + row * ld, c + 8 * k, 2 * F, vec, *reinterpret_cast<float(*)[8]>(g + 8 * k));
            load_row<T, 8>(h + row * ld, F + c + 8 * k, 2 * F, vec, *reinterpret_cast<float(*)[8]>(u + 8 * k));
        }
        uint64_t g2[8], u2[8], a2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g2[i] = f32x2_pack(g[2 * i], g[2 * i + 1]);
            u2[i] = f32x2_pack(u[2 * i], u[2 * i + 1]);
            const uint64_t s = sigmoid2(g[2 * i], g[2 * i + 1]);
            a2[i] = f32x2_mul(f32x2_mul(g2[i], s), u2[i]);
        }
        RowWriter out;
        out.start(a8, row, c);
        out.put(a8, a2, 0, 16);
        if (h8.codes != nullptr) {
            out.start(h8, row, c);
            out.put(h8, g2, 0, 16);
            out.start(h8, row, F + c);
            out.put(h8, u2, 0, 16);
        }
    }
}

template <typename T>
struct SwigluSmem {
    // two stages of float da would not fit beside the rest
    static constexpr int kStages = sizeof(T) == 4 ? 1 : 2;
    uint8_t da[kStages][kTile * kTile * sizeof(T)];
    uint8_t gate[kStages][kTile * kTile], value[kStages][kTile * kTile];
    ColsSmem cols[3];   // d gate, d value, the output
};

// The three results of a tile in registers at once: 192 KB of the SM's 256, so one CTA
// per SM.  Bound by issue slots (59 %; some 46 instructions per element of da) and the three
// barriers of a tile: 8192 x 11008 BF16 178.5 us, 4.5 TB/s (0.67 of a copy's rate).
template <typename T, int FMT, int AFMT, int HFMT>
__global__ void __launch_bounds__(kTileThreads, 1)
    swiglu_bwd_kernel(const T *__restrict__ da, int64_t M, int64_t F, int64_t ld, bool vec,
                      const BlockView h8, const BlockView dh8, const BlockView dh8t,
                      const BlockView a8t, unsigned tiles_r, unsigned tiles_c) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SwigluSmem<T> &sm = *reinterpret_cast<SwigluSmem<T> *>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp * kTileRows * kTile;
    constexpr int kSize = static_cast<int>(sizeof(T));
    constexpr int kStages = SwigluSmem<T>::kStages;
    pdl_wait();
    pdl_trigger();
    TileWalk walk(tiles_r, tiles_c);
    unsigned row0, col0;
    walk.origin(row0, col0);
    auto fetch = [&](int stage, unsigned r0, unsigned c0) {
        fetch_rows<kSize>(smem_u32(sm.da[stage]) + part * kSize, da, ld, M, F, vec, r0, c0);
        fetch_rows<1>(smem_u32(sm.gate[stage]) + part, h8.codes, h8.ld, M, F, true, r0, c0);
        fetch_rows<1>(smem_u32(sm.value[stage]) + part, h8.codes + F, h8.ld, M, F, true, r0, c0);
    };
    // lanes 0 .. 7: the rows' scales of gate; lanes 8 .. 15: of value
    auto scale_of = [&](unsigned r0, unsigned c0) {
        const unsigned row = r0 + warp * kTileRows + (lane & 7);
        return lane < 16 && row < M ? fetch_scale(h8, row, (c0 + (lane < 8 ? 0 : F)) / kTile) : 0u;
    };
    fetch(0, row0, col0);
    cp_async_commit();
    uint32_t sc_next = scale_of(row0, col0);
    int stage = 0;
    for (bool more = true; more;) {
        const float sc = fetched_scale(h8, sc_next);
        unsigned next_row0 = 0, next_col0 = 0;
        walk.next();
        more = walk.there();
        if (more) {
            walk.origin(next_row0, next_col0);
            sc_next = scale_of(next_row0, next_col0);
        }
        if constexpr (kStages == 2) {
            __syncwarp();   // the warp has read its part of the other stage
            if (more) fetch(stage ^ 1, next_row0, next_col0);
            cp_async_commit();
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncwarp();
        TileValues dg, du, a;
        const uint64_t one2 = splat_f32x2(1.0f);
#pragma unroll
        for (int r = 0; r < kTileRows; ++r) {
            uint64_t d[2], g[2], u[2];
            staged4<T>(sm.da[stage] + part * kSize, r, d);
            staged_codes4(sm.gate[stage] + part, r, HFMT, __shfl_sync(0xFFFFFFFFu, sc, r), g);
            staged_codes4(sm.value[stage] + part, r, HFMT, __shfl_sync(0xFFFFFFFFu, sc, r + 8), u);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float g0, g1;
                f32x2_unpack(g[p], g0, g1);
                const uint64_t s = sigmoid2(g0, g1);
                const uint64_t gs = f32x2_mul(g[p], s);
                a[r][p] = f32x2_mul(gs, u[p]);
                du[r][p] = f32x2_mul(d[p], gs);
                dg[r][p] = f32x2_mul(f32x2_mul(f32x2_mul(d[p], u[p]), s),
                                     f32x2_fma(g[p], f32x2_sub(one2, s), one2));
            }
        }
        if constexpr (kStages == 1) {
            __syncwarp();
            if (more) fetch(0, next_row0, next_col0);
            cp_async_commit();
        }
        const bool t_dh = dh8t.codes != nullptr, t_a = a8t.codes != nullptr;
        if (t_dh) {
            cols_max(dg, sm.cols[0]);
            cols_max(du, sm.cols[1]);
        }
        if (t_a) cols_max(a, sm.cols[2]);
        __syncthreads();
        const int c = threadIdx.x & (kTile - 1);
        if (threadIdx.x < kTile) {
            if (t_dh) cols_scale<FMT>(c, sm.cols[0], dh8t, row0, col0);
        } else if (threadIdx.x < 2 * kTile) {
            if (t_dh) cols_scale<FMT>(c, sm.cols[1], dh8t, row0, static_cast<unsigned>(F) + col0);
        } else if (threadIdx.x < 3 * kTile) {
            if (t_a) cols_scale<AFMT>(c, sm.cols[2], a8t, row0, col0);
        }
        __syncthreads();
        if (t_dh) {
            cols_codes<FMT>(dg, cols_inv(sm.cols[0]), sm.cols[0]);
            cols_codes<FMT>(du, cols_inv(sm.cols[1]), sm.cols[1]);
        }
        if (t_a) cols_codes<AFMT>(a, cols_inv(sm.cols[2]), sm.cols[2]);
        if (dh8.codes != nullptr) {
            tile_rows<FMT>(dg, dh8, row0, col0, -1);
            tile_rows<FMT>(du, dh8, row0, static_cast<unsigned>(F) + col0, -1);
        }
        __syncthreads();
        if (t_dh) {
            cols_store(sm.cols[0], dh8t, row0, col0);
            cols_store(sm.cols[1], dh8t, row0, static_cast<unsigned>(F) + col0);
        }
        if (t_a) cols_store(sm.cols[2], a8t, row0, col0);
        row0 = next_row0, col0 = next_col0;
        if constexpr (kStages == 2) stage ^= 1;
    }
}

// Rows whose N-element vectors are aligned.
bool rows_vec(const MatView &m, int n) {
    const int64_t bytes = (m.type == kTypeF32 ? 4 : 2) * n;
    const int64_t al = bytes < 16 ? bytes : 16;
    return reinterpret_cast<uintptr_t>(m.data) % al == 0 &&
           (m.ld * (m.type == kTypeF32 ? 4 : 2)) % al == 0;
}

unsigned capped(int64_t n, int64_t cap) { return static_cast<unsigned>(n < cap ? n : cap); }

unsigned tiles_of(int64_t n) { return static_cast<unsigned>((n + kTile - 1) / kTile); }

// A persistent tile kernel with `per_sm` CTAs per SM, its shared-memory limit set on a
// device's first launch.
template <auto KERNEL, typename Smem, typename... Args>
cudaError_t launch_tiles(int per_sm, int64_t rows, int64_t cols, int sm_count, cudaStream_t st,
                         Args... args) {
    static SmemLimit limit;
    const cudaError_t err = limit.allow(KERNEL, sizeof(Smem));
    if (err != cudaSuccess) return err;
    const unsigned r = tiles_of(rows), c = tiles_of(cols);
    const dim3 grid(capped(static_cast<int64_t>(r) * c, static_cast<int64_t>(sm_count) * per_sm));
    return launch_pdl(KERNEL, grid, dim3(kTileThreads), sizeof(Smem), st, args..., r, c);
}

template <typename T, int FMT, bool TILE>
cudaError_t quantize_tiles(const MatView &x, const BlockView &q, const BlockView &qt, int sm_count,
                           cudaStream_t st) {
    return launch_tiles<block_quantize_kernel<T, FMT, TILE>, QuantSmem<T>>(
        sizeof(T) == 4 ? 1 : 2, x.rows, x.cols, sm_count, st, static_cast<const T *>(x.data), x.rows,
        x.cols, x.ld, rows_vec(x, static_cast<int>(16 / sizeof(T))), q, qt);
}

template <typename T>
cudaError_t quantize_typed(const MatView &x, const BlockView &q, const BlockView &qt, int fmt,
                           bool tile, int sm_count, cudaStream_t st) {
    if (fmt == 0)
        return tile ? quantize_tiles<T, 0, true>(x, q, qt, sm_count, st)
                    : quantize_tiles<T, 0, false>(x, q, qt, sm_count, st);
    return tile ? quantize_tiles<T, 1, true>(x, q, qt, sm_count, st)
                : quantize_tiles<T, 1, false>(x, q, qt, sm_count, st);
}

}  // namespace

cudaError_t launch_block_quantize(const MatView &x, const BlockView &q, const BlockView &qt,
                                  int sm_count, cudaStream_t st) {
    if (x.rows == 0 || x.cols == 0) return cudaSuccess;
    const BlockView &any = q.codes != nullptr ? q : qt;
    const bool tile = any.block_rows != 1;
    if (x.type == kTypeF32) return quantize_typed<float>(x, q, qt, any.fmt, tile, sm_count, st);
    if (x.type == kTypeBF16) return quantize_typed<__nv_bfloat16>(x, q, qt, any.fmt, tile, sm_count, st);
    return quantize_typed<__half>(x, q, qt, any.fmt, tile, sm_count, st);
}

cudaError_t launch_block_dequantize(const BlockView &q, const MatView &out, int sm_count,
                                    cudaStream_t st) {
    if (q.rows == 0 || q.cols == 0) return cudaSuccess;
    const int64_t segs = q.rows * ((q.cols + 1023) / 1024);
    const dim3 grid(capped((segs + 7) / 8, static_cast<int64_t>(sm_count) * 64));
    const bool vec = rows_vec(out, 8);
    if (out.type == kTypeF32)
        return launch_pdl(block_dequantize_kernel<float>, grid, dim3(256), 0, st, q,
                          static_cast<float *>(out.data), out.ld, vec);
    if (out.type == kTypeBF16)
        return launch_pdl(block_dequantize_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, q,
                          static_cast<__nv_bfloat16 *>(out.data), out.ld, vec);
    return launch_pdl(block_dequantize_kernel<__half>, grid, dim3(256), 0, st, q,
                      static_cast<__half *>(out.data), out.ld, vec);
}

cudaError_t launch_ln_recompute(const BlockView &x8, const void *gamma, const void *beta, int wtype,
                                const float *mean, const float *rstd, const BlockView &yt,
                                int sm_count, cudaStream_t st) {
    if (x8.rows == 0 || x8.cols == 0) return cudaSuccess;
    if (yt.fmt == 0)
        return launch_tiles<ln_recompute_kernel<0>, RecomputeSmem>(2, x8.rows, x8.cols, sm_count, st,
                                                                   x8, gamma, beta, wtype, mean, rstd, yt);
    return launch_tiles<ln_recompute_kernel<1>, RecomputeSmem>(2, x8.rows, x8.cols, sm_count, st, x8,
                                                               gamma, beta, wtype, mean, rstd, yt);
}

cudaError_t launch_swiglu_fwd(const MatView &h, const BlockView &a8, const BlockView &h8,
                              int sm_count, cudaStream_t st) {
    if (h.rows == 0 || h.cols == 0) return cudaSuccess;
    const int64_t F = h.cols / 2;
    const dim3 grid(capped((h.rows * (F / 128) + 31) / 32, static_cast<int64_t>(sm_count) * 64));
    const bool vec = rows_vec(h, 8);
    if (h.type == kTypeF32)
        return launch_pdl(swiglu_fwd_kernel<float>, grid, dim3(256), 0, st,
                          static_cast<const float *>(h.data), h.rows, F, h.ld, vec, a8, h8);
    if (h.type == kTypeBF16)
        return launch_pdl(swiglu_fwd_kernel<__nv_bfloat16>, grid, dim3(256), 0, st,
                          static_cast<const __nv_bfloat16 *>(h.data), h.rows, F, h.ld, vec, a8, h8);
    return launch_pdl(swiglu_fwd_kernel<__half>, grid, dim3(256), 0, st,
                      static_cast<const __half *>(h.data), h.rows, F, h.ld, vec, a8, h8);
}

namespace {
template <typename T, int FMT, int AFMT>
cudaError_t swiglu_bwd_tiles(const MatView &da, const BlockView &h8, const BlockView &dh8,
                             const BlockView &dh8t, const BlockView &a8t, int sm_count,
                             cudaStream_t st) {
    const T *p = static_cast<const T *>(da.data);
    const bool vec = rows_vec(da, static_cast<int>(16 / sizeof(T)));
    if (h8.fmt == 0)
        return launch_tiles<swiglu_bwd_kernel<T, FMT, AFMT, 0>, SwigluSmem<T>>(
            1, da.rows, da.cols, sm_count, st, p, da.rows, da.cols, da.ld, vec, h8, dh8, dh8t, a8t);
    return launch_tiles<swiglu_bwd_kernel<T, FMT, AFMT, 1>, SwigluSmem<T>>(
        1, da.rows, da.cols, sm_count, st, p, da.rows, da.cols, da.ld, vec, h8, dh8, dh8t, a8t);
}

template <typename T>
cudaError_t swiglu_bwd_typed(const MatView &da, const BlockView &h8, const BlockView &dh8,
                             const BlockView &dh8t, const BlockView &a8t, int sm_count,
                             cudaStream_t st) {
    const int fmt = dh8.codes != nullptr ? dh8.fmt : dh8t.fmt;
    const int afmt = a8t.codes != nullptr ? a8t.fmt : 0;
    if (fmt == 0)
        return afmt == 0 ? swiglu_bwd_tiles<T, 0, 0>(da, h8, dh8, dh8t, a8t, sm_count, st)
                         : swiglu_bwd_tiles<T, 0, 1>(da, h8, dh8, dh8t, a8t, sm_count, st);
    return afmt == 0 ? swiglu_bwd_tiles<T, 1, 0>(da, h8, dh8, dh8t, a8t, sm_count, st)
                     : swiglu_bwd_tiles<T, 1, 1>(da, h8, dh8, dh8t, a8t, sm_count, st);
}
}  // namespace

cudaError_t launch_swiglu_bwd(const MatView &da, const BlockView &h8, const BlockView &dh8,
                              const BlockView &dh8t, const BlockView &a8t, int sm_count,
                              cudaStream_t st) {
    if (da.rows == 0 || da.cols == 0) return cudaSuccess;
    if (da.type == kTypeF32) return swiglu_bwd_typed<float>(da, h8, dh8, dh8t, a8t, sm_count, st);
    if (da.type == kTypeBF16)
        return swiglu_bwd_typed<__nv_bfloat16>(da, h8, dh8, dh8t, a8t, sm_count, st);
    return swiglu_bwd_typed<__half>(da, h8, dh8, dh8t, a8t, sm_count, st);
}

}  // namespace fp8k
