// block_quant.cu -- block-scaled quantization of a matrix, of its transpose and
// of what a backward pass computes from an input kept in 8 bits: LayerNorm's
// output again, and SwiGLU forward and backward.  The formulas are in
// include/fp8amax.h; block.cuh has the scale rule and the tile's layout.
//
// All are bound by HBM.  What has to be written transposed goes tile by tile
// (128 x 128, one block wide both ways), the rest row by row.
#include <cstdint>

#include "block.cuh"

namespace fp8k {

namespace {

// The CTA's tile: tiles are numbered along the rows of tiles.
__device__ __forceinline__ void tile_origin(int64_t cols, int64_t &row0, int64_t &col0) {
    const unsigned per_row = static_cast<unsigned>((cols + kTile - 1) / kTile);
    row0 = static_cast<int64_t>(blockIdx.x / per_row) * kTile;
    col0 = static_cast<int64_t>(blockIdx.x % per_row) * kTile;
}

// ----------------------------------------------------------- quantization --

template <typename T, int FMT, bool TILE>
__global__ void __launch_bounds__(kTileThreads, 2)
    block_quantize_kernel(const T *__restrict__ x, int64_t rows, int64_t cols, int64_t ld, bool vec,
                          const BlockView q, const BlockView qt) {
    __shared__ __align__(16) TileSmem sm;
    __shared__ uint32_t red[16];
    pdl_wait();
    pdl_trigger();
    int64_t row0, col0;
    tile_origin(cols, row0, col0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float v[kTileRows][4];
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        const int64_t row = row0 + warp * kTileRows + r;
        if (row < rows) {
            load_row<T, 4>(x + row * ld, col0 + 4 * lane, cols, vec, v[r]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = 0.0f;
        }
    }
    int byte = -1;
    if constexpr (TILE) byte = static_cast<int>(scale_byte<FMT>(tile_max(v, red)));
    if (q.codes != nullptr) tile_rows<FMT>(v, q, row0, col0, byte);
    if (qt.codes != nullptr) tile_cols<FMT>(v, qt, row0, col0, byte, sm);
}

// One warp per 1024 columns of a row, 8 per lane and step of 256.
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

__global__ void __launch_bounds__(kTileThreads, 2)
    ln_recompute_kernel(const BlockView x8, const void *__restrict__ gamma,
                        const void *__restrict__ beta, int wtype, const float *__restrict__ mean,
                        const float *__restrict__ rstd, const BlockView yt) {
    __shared__ __align__(16) TileSmem sm;
    pdl_wait();
    pdl_trigger();
    int64_t row0, col0;
    tile_origin(x8.cols, row0, col0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = col0 + 4 * lane;
    float g[4], b[4], v[kTileRows][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool in = c + j < x8.cols;
        g[j] = in ? load_any(gamma, wtype, c + j) : 0.0f;
        b[j] = in ? load_any(beta, wtype, c + j) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        const int64_t row = row0 + warp * kTileRows + r;
        if (row < x8.rows) {
            load_codes<4>(x8.codes + row * x8.ld, c, x8.cols, x8.fmt,
                          load_scale(x8, row, col0 / kTile), v[r]);
            const float mu = mean[row], rs = rstd[row];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[r][j] = c + j < x8.cols
                              ? __fadd_rn(__fmul_rn(__fmul_rn(__fsub_rn(v[r][j], mu), rs), g[j]), b[j])
                              : 0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = 0.0f;
        }
    }
    if (yt.fmt == 0)
        tile_cols<0>(v, yt, row0, col0, -1, sm);
    else
        tile_cols<1>(v, yt, row0, col0, -1, sm);
}

// ----------------------------------------------------------------- SwiGLU --

// 1 / (1 + exp(-x)) to a few units in the last place: 0 for -inf, 1 for +inf.
__device__ __forceinline__ float sigmoid(float x) {
    return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-x)));
}

// Quantizes 8 consecutive columns per lane; 16 lanes hold a block of 128.
template <int FMT>
__device__ __forceinline__ void emit_full8(const float (&v)[8], const BlockView &q, int64_t row,
                                           int64_t c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_abs_bits(v[i]));
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const uint32_t byte = scale_byte<FMT>(m);
    const float inv = scale_inverse(byte);
    if ((threadIdx.x & 15) == 0) store_scale(q, row, c >> 7, byte);
    *reinterpret_cast<uint2 *>(q.codes + row * q.ld + c) =
        make_uint2(encode4<FMT>(v[0], v[1], v[2], v[3], inv),
                   encode4<FMT>(v[4], v[5], v[6], v[7], inv));
}

// 16 lanes per block of 128 columns of a row, two blocks per warp.
template <typename T>
__global__ void __launch_bounds__(256) swiglu_fwd_kernel(const T *__restrict__ h, int64_t M, int64_t F,
                                                         int64_t ld, bool vec, const BlockView a8,
                                                         const BlockView h8) {
    pdl_wait();
    pdl_trigger();
    const int64_t per_row = F / 128, total = M * per_row;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 16;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 5) * 2; w < total;
         w += step) {
        // the warp's second half may be past the end: it repeats the first half's block
        int64_t blk = w + ((threadIdx.x >> 4) & 1);
        if (blk >= total) blk = w;
        const int64_t row = blk / per_row, c = (blk % per_row) * 128 + 8 * (threadIdx.x & 15);
        float g[8], u[8], a[8];
        load_row<T, 8>(h + row * ld, c, 2 * F, vec, g);
        load_row<T, 8>(h + row * ld, F + c, 2 * F, vec, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = __fmul_rn(__fmul_rn(g[i], sigmoid(g[i])), u[i]);
        if (a8.fmt == 0)
            emit_full8<0>(a, a8, row, c);
        else
            emit_full8<1>(a, a8, row, c);
        if (h8.codes != nullptr) {
            if (h8.fmt == 0) {
                emit_full8<0>(g, h8, row, c);
                emit_full8<0>(u, h8, row, F + c);
            } else {
                emit_full8<1>(g, h8, row, c);
                emit_full8<1>(u, h8, row, F + c);
            }
        }
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kTileThreads, 1)
    swiglu_bwd_kernel(const T *__restrict__ da, int64_t M, int64_t F, int64_t ld, bool vec,
                      const BlockView h8, const BlockView dh8, const BlockView dh8t,
                      const BlockView a8t) {
    __shared__ __align__(16) TileSmem sm;
    pdl_wait();
    pdl_trigger();
    int64_t row0, col0;
    tile_origin(F, row0, col0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = col0 + 4 * lane;
    float dg[kTileRows][4], du[kTileRows][4], a[kTileRows][4];
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        const int64_t row = row0 + warp * kTileRows + r;
        if (row < M) {
            float d[4], g[4], u[4];
            load_row<T, 4>(da + row * ld, c, F, vec, d);
            load_codes<4>(h8.codes + row * h8.ld, c, h8.cols, h8.fmt,
                          load_scale(h8, row, col0 / kTile), g);
            load_codes<4>(h8.codes + row * h8.ld, F + c, h8.cols, h8.fmt,
                          load_scale(h8, row, (F + col0) / kTile), u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float s = sigmoid(g[j]), gs = __fmul_rn(g[j], s);
                a[r][j] = __fmul_rn(gs, u[j]);
                du[r][j] = __fmul_rn(d[j], gs);
                dg[r][j] = __fmul_rn(__fmul_rn(__fmul_rn(d[j], u[j]), s),
                                     __fmaf_rn(g[j], __fsub_rn(1.0f, s), 1.0f));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[r][j] = du[r][j] = dg[r][j] = 0.0f;
        }
    }
    if (dh8.codes != nullptr) {
        tile_rows<FMT>(dg, dh8, row0, col0, -1);
        tile_rows<FMT>(du, dh8, row0, F + col0, -1);
    }
    if (dh8t.codes != nullptr) {
        tile_cols<FMT>(dg, dh8t, row0, col0, -1, sm);
        __syncthreads();
        tile_cols<FMT>(du, dh8t, row0, F + col0, -1, sm);
        __syncthreads();
    }
    if (a8t.codes != nullptr) {
        if (a8t.fmt == 0)
            tile_cols<0>(a, a8t, row0, col0, -1, sm);
        else
            tile_cols<1>(a, a8t, row0, col0, -1, sm);
    }
}

// Rows whose N-element vectors are aligned.
bool rows_vec(const MatView &m, int n) {
    const int64_t bytes = (m.type == kTypeF32 ? 4 : 2) * n;
    const int64_t al = bytes < 16 ? bytes : 16;
    return reinterpret_cast<uintptr_t>(m.data) % al == 0 &&
           (m.ld * (m.type == kTypeF32 ? 4 : 2)) % al == 0;
}

dim3 tile_grid(int64_t rows, int64_t cols) {
    return dim3(static_cast<unsigned>(((cols + kTile - 1) / kTile) * ((rows + kTile - 1) / kTile)));
}

template <typename T>
cudaError_t quantize_typed(const MatView &x, const BlockView &q, const BlockView &qt, int fmt,
                           bool tile, cudaStream_t st) {
    const dim3 grid = tile_grid(x.rows, x.cols), block(kTileThreads);
    const T *p = static_cast<const T *>(x.data);
    const bool vec = rows_vec(x, 4);
    auto k = fmt == 0 ? (tile ? block_quantize_kernel<T, 0, true> : block_quantize_kernel<T, 0, false>)
                      : (tile ? block_quantize_kernel<T, 1, true> : block_quantize_kernel<T, 1, false>);
    return launch_pdl(k, grid, block, 0, st, p, x.rows, x.cols, x.ld, vec, q, qt);
}

unsigned capped(int64_t n, int64_t cap) { return static_cast<unsigned>(n < cap ? n : cap); }

}  // namespace

cudaError_t launch_block_quantize(const MatView &x, const BlockView &q, const BlockView &qt,
                                  cudaStream_t st) {
    if (x.rows == 0 || x.cols == 0) return cudaSuccess;
    const BlockView &any = q.codes != nullptr ? q : qt;
    const bool tile = any.block_rows != 1;
    if (x.type == kTypeF32) return quantize_typed<float>(x, q, qt, any.fmt, tile, st);
    if (x.type == kTypeBF16) return quantize_typed<__nv_bfloat16>(x, q, qt, any.fmt, tile, st);
    return quantize_typed<__half>(x, q, qt, any.fmt, tile, st);
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
                                cudaStream_t st) {
    if (x8.rows == 0 || x8.cols == 0) return cudaSuccess;
    return launch_pdl(ln_recompute_kernel, tile_grid(x8.rows, x8.cols), dim3(kTileThreads), 0, st, x8,
                      gamma, beta, wtype, mean, rstd, yt);
}

cudaError_t launch_swiglu_fwd(const MatView &h, const BlockView &a8, const BlockView &h8,
                              int sm_count, cudaStream_t st) {
    if (h.rows == 0 || h.cols == 0) return cudaSuccess;
    const int64_t F = h.cols / 2;
    const dim3 grid(capped((h.rows * (F / 128) + 15) / 16, static_cast<int64_t>(sm_count) * 64));
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
template <typename T>
cudaError_t swiglu_bwd_typed(const MatView &da, const BlockView &h8, const BlockView &dh8,
                             const BlockView &dh8t, const BlockView &a8t, cudaStream_t st) {
    const int fmt = dh8.codes != nullptr ? dh8.fmt : dh8t.fmt;
    auto k = fmt == 0 ? swiglu_bwd_kernel<T, 0> : swiglu_bwd_kernel<T, 1>;
    return launch_pdl(k, tile_grid(da.rows, da.cols), dim3(kTileThreads), 0, st,
                      static_cast<const T *>(da.data), da.rows, da.cols, da.ld, rows_vec(da, 4), h8,
                      dh8, dh8t, a8t);
}
}  // namespace

cudaError_t launch_swiglu_bwd(const MatView &da, const BlockView &h8, const BlockView &dh8,
                              const BlockView &dh8t, const BlockView &a8t, cudaStream_t st) {
    if (da.rows == 0 || da.cols == 0) return cudaSuccess;
    if (da.type == kTypeF32) return swiglu_bwd_typed<float>(da, h8, dh8, dh8t, a8t, st);
    if (da.type == kTypeBF16) return swiglu_bwd_typed<__nv_bfloat16>(da, h8, dh8, dh8t, a8t, st);
    return swiglu_bwd_typed<__half>(da, h8, dh8, dh8t, a8t, st);
}

}  // namespace fp8k
