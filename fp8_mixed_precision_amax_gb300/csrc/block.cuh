// block.cuh -- device code shared by the block-scaled kernels (block_quant.cu,
// layernorm.cu): loads and stores of 16- and 32-bit rows, a block's
// power-of-two scale, and the quantization of a 128 x 128 tile both ways.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace fp8k {

// ---------------------------------------------------- elements and vectors --

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Two packed 16-bit elements (lo first) to fp32 and back.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// N consecutive elements (N = 4 or 8) from p, which is aligned to N elements.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 f = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = f.x;
            v[4 * i + 1] = f.y;
            v[4 * i + 2] = f.z;
            v[4 * i + 3] = f.w;
        }
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = unpack2<T>(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        if constexpr (N == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// N elements of a row at column c; columns from `cols` on give 0.  vec: the
// row is aligned so that N elements at a multiple of N are one vector.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T *row, int64_t c, int64_t cols, bool vec,
                                         float (&v)[N]) {
    if (vec && c + N <= cols) {
        load_vec<T, N>(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = c + i < cols ? to_f32(row[c + i]) : 0.0f;
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_row(T *row, int64_t c, int64_t cols, bool vec,
                                          const float (&v)[N]) {
    if (vec && c + N <= cols) {
        store_vec<T, N>(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < cols) row[c + i] = from_f32<T>(v[i]);
    }
}

// gamma or beta (type known at run time) at column c.
__device__ __forceinline__ float load_any(const void *p, int type, int64_t c) {
    if (type == kTypeF32) return static_cast<const float *>(p)[c];
    if (type == kTypeBF16) return to_f32(static_cast<const __nv_bfloat16 *>(p)[c]);
    return to_f32(static_cast<const __half *>(p)[c]);
}

// ------------------------------------------------------------ block scales --

// |x| as bits, 0 for infinities and NaN: the unsigned maximum of these is the
// largest finite magnitude.
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
    return a < 0x7F800000u ? a : 0u;
}

// E8M0 byte of a block: e + 127 for the smallest e >= -127 with amax <= fmax 2^e.
// Both formats' fmax is 1.75 2^t (t = 8 or 15).  With amax = f 2^p, 1 <= f < 2, e is
// p - t if f <= 1.75 and p - t + 1 otherwise, and the biased exponent field of
// amax is p + 127.  A subnormal amax (field 0) gives byte 0, as it should.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - (FMT == 0 ? 8 : 15) +
                  ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(max(e, 0));
}
// 2^-(byte - 127) for a byte of scale_byte (at most 247, so never subnormal)
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127); 255 is NaN
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FC00000u)
                        : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

__device__ __forceinline__ void store_scale(const BlockView &q, int64_t rb, int64_t cb,
                                            uint32_t byte) {
    if (q.scale_f32)
        static_cast<float *>(q.scales)[rb * q.ld_s + cb] = scale_value(byte);
    else
        static_cast<uint8_t *>(q.scales)[rb * q.ld_s + cb] = static_cast<uint8_t>(byte);
}
__device__ __forceinline__ float load_scale(const BlockView &q, int64_t rb, int64_t cb) {
    if (q.scale_f32) return static_cast<const float *>(q.scales)[rb * q.ld_s + cb];
    return scale_value(static_cast<const uint8_t *>(q.scales)[rb * q.ld_s + cb]);
}

// Four FP8 codes (a word) to fp32, exactly (by way of FP16, which holds both formats).
__device__ __forceinline__ void decode4(uint32_t w, int fmt, float (&v)[4]) {
    uint32_t h0, h1;
    if (fmt == 0) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(h0), "=r"(h1) : "r"(w));
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, a;\n\t"
            "cvt.rn.f16x2.e5m2x2 %1, b;\n\t}"
            : "=r"(h0), "=r"(h1) : "r"(w));
    }
    const float2 f0 = unpack2<__half>(h0), f1 = unpack2<__half>(h1);
    v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
}

// N codes (4 or 8) of a row at column c (a multiple of N), times the scale;
// columns from `cols` on give 0.  Code rows are 16-byte aligned and end at a
// multiple of 16, so the whole vector is always readable.
template <int N>
__device__ __forceinline__ void load_codes(const uint8_t *row, int64_t c, int64_t cols, int fmt,
                                           float scale, float (&v)[N]) {
    if (c >= cols) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
        return;
    }
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        float f[4];
        decode4(reinterpret_cast<const uint32_t *>(row + c)[k], fmt, f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[4 * k + i] = c + 4 * k + i < cols ? __fmul_rn(f[i], scale) : 0.0f;
    }
}

template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
    return cvt2_fp8<FMT>(__fmul_rn(a, inv), __fmul_rn(b, inv)) |
           (cvt2_fp8<FMT>(__fmul_rn(c, inv), __fmul_rn(d, inv)) << 16);
}

// bytes [0, n) of a word of codes to p (4-byte aligned)
__device__ __forceinline__ void store_code_word(uint8_t *p, uint32_t w, int64_t n) {
    if (n >= 4) {
        *reinterpret_cast<uint32_t *>(p) = w;
    } else {
        for (int i = 0; i < n; ++i) p[i] = static_cast<uint8_t>(w >> (8 * i));
    }
}

// ----------------------------------------------------------- tile kernels --
//
// A CTA of 512 threads holds a 128 x 128 tile in fp32 registers: warp w has
// rows 8 w .. 8 w + 7, lane l columns 4 l .. 4 l + 3, so v[r][j] is row
// 8 w + r, column 4 l + j.  Elements outside the matrix are 0: they leave
// every maximum as it is.  A row's maximum is one warp reduction; a column's
// is taken over a thread's 8 rows and then over the 16 warps in shared memory.

constexpr int kTile = 128;
constexpr int kTileThreads = 512;
constexpr int kTileRows = 8;   // rows per warp

struct TileSmem {
    uint32_t colmax[16][kTile];   // per warp: a column's maximum over the warp's rows
    uint8_t codes[kTile * kTile]; // transposed codes [column][row], swizzled (see tile_cols)
};

// The tile's own maximum (block_rows 128), the same in every thread.
__device__ __forceinline__ uint32_t tile_max(const float (&v)[kTileRows][4], uint32_t *red) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < kTileRows; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, finite_abs_bits(v[r][j]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red[threadIdx.x & 15];
    return __reduce_max_sync(0xFFFFFFFFu, m);
}

// Row-major codes and scales of the tile at (row0, col0).  tile_byte < 0: one
// scale per row; otherwise the whole tile's.
template <int FMT>
__device__ __forceinline__ void tile_rows(const float (&v)[kTileRows][4], const BlockView &q,
                                          int64_t row0, int64_t col0, int tile_byte) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = col0 + 4 * lane;
    if (tile_byte >= 0 && threadIdx.x == 0)
        store_scale(q, row0 / kTile, col0 / kTile, static_cast<uint32_t>(tile_byte));
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        const int64_t row = row0 + warp * kTileRows + r;
        uint32_t byte = static_cast<uint32_t>(tile_byte);
        if (tile_byte < 0) {
            const uint32_t m = max(max(finite_abs_bits(v[r][0]), finite_abs_bits(v[r][1])),
                                   max(finite_abs_bits(v[r][2]), finite_abs_bits(v[r][3])));
            byte = scale_byte<FMT>(__reduce_max_sync(0xFFFFFFFFu, m));
        }
        if (row >= q.rows) continue;   // the same for the whole warp
        if (tile_byte < 0 && lane == 0) store_scale(q, row, col0 / kTile, byte);
        const uint32_t w = encode4<FMT>(v[r][0], v[r][1], v[r][2], v[r][3], scale_inverse(byte));
        if (c < q.cols) store_code_word(q.codes + row * q.ld + c, w, q.cols - c);
    }
}

// The transpose of the tile: qt's rows are the tile's columns.  The codes go
// through shared memory: column c's 128 bytes are row c of `codes`, in chunks of
// 16 bytes (two warps' 8 rows each).  Chunk k is kept at place
// k ^ ((c >> 2) & 7), its halves swapped when bit 5 of c is set: the lanes of a
// warp write 8 bytes each to columns 4 apart, and half a warp then covers all
// banks once.  Called by all threads; begins with the caller's shared memory free.
template <int FMT>
__device__ __forceinline__ void tile_cols(const float (&v)[kTileRows][4], const BlockView &qt,
                                          int64_t row0, int64_t col0, int tile_byte,
                                          TileSmem &sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float inv[4];
    if (tile_byte < 0) {
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = 0;
#pragma unroll
            for (int r = 0; r < kTileRows; ++r) m[j] = max(m[j], finite_abs_bits(v[r][j]));
        }
        *reinterpret_cast<uint4 *>(&sm.colmax[warp][4 * lane]) = make_uint4(m[0], m[1], m[2], m[3]);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&sm.colmax[w][4 * lane]);
            m[0] = max(m[0], o.x), m[1] = max(m[1], o.y), m[2] = max(m[2], o.z),
            m[3] = max(m[3], o.w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t byte = scale_byte<FMT>(m[j]);
            inv[j] = scale_inverse(byte);
            const int64_t c = col0 + 4 * lane + j;
            if (warp == 0 && c < qt.rows) store_scale(qt, c, row0 / kTile, byte);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) inv[j] = scale_inverse(static_cast<uint32_t>(tile_byte));
        if (threadIdx.x == 0)
            store_scale(qt, col0 / kTile, row0 / kTile, static_cast<uint32_t>(tile_byte));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = 4 * lane + j;
        const uint32_t lo = encode4<FMT>(v[0][j], v[1][j], v[2][j], v[3][j], inv[j]);
        const uint32_t hi = encode4<FMT>(v[4][j], v[5][j], v[6][j], v[7][j], inv[j]);
        const int at = c * kTile + (((warp >> 1) ^ ((c >> 2) & 7)) << 4) +
                       (((warp & 1) ^ ((c >> 5) & 1)) << 3);
        *reinterpret_cast<uint2 *>(&sm.codes[at]) = make_uint2(lo, hi);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTile * kTile / 16 / kTileThreads; ++i) {
        const int idx = threadIdx.x + i * kTileThreads;
        const int c = idx >> 3, k = idx & 7;
        if (col0 + c >= qt.rows) continue;
        uint4 u = *reinterpret_cast<const uint4 *>(&sm.codes[c * kTile + ((k ^ ((c >> 2) & 7)) << 4)]);
        if ((c >> 5) & 1) u = make_uint4(u.z, u.w, u.x, u.y);
        const int64_t r = row0 + 16 * k;
        uint8_t *p = qt.codes + (col0 + c) * qt.ld + r;
        if (r + 16 <= qt.cols) {
            *reinterpret_cast<uint4 *>(p) = u;
        } else {
            store_code_word(p, u.x, qt.cols - r);
            store_code_word(p + 4, u.y, qt.cols - r - 4);
            store_code_word(p + 8, u.z, qt.cols - r - 8);
            store_code_word(p + 12, u.w, qt.cols - r - 12);
        }
    }
}

}  // namespace fp8k
