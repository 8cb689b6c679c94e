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

// ------------------------------------------------- rows of any alignment --
//
// A thread's 8 elements of a row whose start has any alignment, by 16-byte accesses
// alone.  Only 16-byte blocks that hold an element of the row are touched (such a
// block never leaves the allocation, which starts and ends on wider boundaries).
// A warp's lanes hold consecutive groups of 8, so that a store can hand the end of
// one lane's group to the next lane, whose 16-byte blocks it completes.

// Bytes [off, off + 4 N) of the words in w: off in 0 .. 15, even.
template <int N, int WORDS>
__device__ __forceinline__ void shift_words(const uint32_t (&w)[WORDS], uint32_t off, uint32_t (&out)[N]) {
    static_assert(WORDS >= N + 4, "a whole block more than the result");
    uint32_t a[N + 2], b[N + 1];
    const uint32_t pick = off & 2u ? 0x5432u : 0x3210u;
#pragma unroll
    for (int i = 0; i < N + 2; ++i) a[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < N + 1; ++i) b[i] = off & 4u ? a[i + 1] : a[i];
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __byte_perm(b[i], b[i + 1], pick);
}

template <typename T>
struct RawRow8 {
    static constexpr int kWords = 2 * static_cast<int>(sizeof(T));   // of 8 elements
    uint32_t w[kWords + 4];

    // the blocks that hold columns c .. c + 7 of the row
    __device__ __forceinline__ void load(const T *row, int64_t c, int64_t cols) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row + c);
        const uintptr_t end = reinterpret_cast<uintptr_t>(row + cols), base = p & ~uintptr_t(15);
#pragma unroll
        for (int i = 0; i < kWords / 4 + 1; ++i) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (base + 16 * i < end && (i < kWords / 4 || base != p))
                u = *reinterpret_cast<const uint4 *>(base + 16 * i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
    // the same blocks from a copy in shared memory: `at` is the first one's address
    __device__ __forceinline__ void load_shared(const uint8_t *at, bool more) {
#pragma unroll
        for (int i = 0; i < kWords / 4 + 1; ++i) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (i < kWords / 4 || more) u = *reinterpret_cast<const uint4 *>(at + 16 * i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
    // the 8 elements as packed pairs; columns from cols on are 0
    __device__ __forceinline__ void get(const T *row, int64_t c, int64_t cols, uint64_t (&v)[4]) const {
        get(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u), static_cast<int>(cols - c), v);
    }
    // off: the row start's distance from a 16-byte boundary; left: columns from the first on
    __device__ __forceinline__ void get(uint32_t off, int left, uint64_t (&v)[4]) const {
        uint32_t x[kWords];
        if (off == 0) {   // the same for the whole row: 8 elements are whole blocks
#pragma unroll
            for (int i = 0; i < kWords; ++i) x[i] = w[i];
        } else {
            shift_words<kWords, kWords + 4>(w, off, x);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = f32x2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            } else {
                const float2 f = unpack2<T>(x[i]);
                v[i] = f32x2_pack(f.x, f.y);
            }
        }
        if (left < 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                f32x2_unpack(v[i], lo, hi);
                v[i] = f32x2_pack(2 * i < left ? lo : 0.0f, 2 * i + 1 < left ? hi : 0.0f);
            }
        }
    }
};

// N (8 or 16) elements of a row that starts on a 16-byte boundary and is a multiple of N
// elements long.
template <typename T, int N>
struct RawVec {
    static constexpr int kBlocks = N * static_cast<int>(sizeof(T)) / 16;
    uint4 u[kBlocks];

    __device__ __forceinline__ void load(const T *row, int64_t c, int64_t cols) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
            u[i] = c < cols ? reinterpret_cast<const uint4 *>(row + c)[i] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(const T *, int64_t, int64_t, uint64_t (&v)[N / 2]) const {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[2 * i] = f32x2_pack(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
                v[2 * i + 1] = f32x2_pack(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
            } else {
                const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack2<T>(w[k]);
                    v[4 * i + k] = f32x2_pack(f.x, f.y);
                }
            }
        }
    }
    static __device__ __forceinline__ void store(T *row, int64_t c, int64_t cols,
                                                 const uint64_t (&v)[N / 2]) {
        if (c >= cols) return;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            uint4 q;
            float a, b, d, e;
            if constexpr (sizeof(T) == 4) {
                f32x2_unpack(v[2 * i], a, b);
                f32x2_unpack(v[2 * i + 1], d, e);
                q = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(d),
                               __float_as_uint(e));
            } else {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f32x2_unpack(v[4 * i + k], a, b);
                    w[k] = pack2<T>(a, b);
                }
                q = make_uint4(w[0], w[1], w[2], w[3]);
            }
            reinterpret_cast<uint4 *>(row + c)[i] = q;
        }
    }
};

// Stores the pairs to columns c .. c + 7 (those below cols).  All lanes of the warp
// take part, lane l + 1 with the columns after lane l's.
template <typename T>
__device__ __forceinline__ void store_row8(T *row, int64_t c, int64_t cols, const uint64_t (&v)[4]) {
    constexpr int kWords = 2 * static_cast<int>(sizeof(T)), kBlocks = kWords / 4;
    const int lane = threadIdx.x & 31;
    uint32_t w[kWords + 8];   // the lane before's last block, this lane's words, room to shift
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f32x2_unpack(v[i], lo, hi);
        if constexpr (sizeof(T) == 4) {
            w[4 + 2 * i] = __float_as_uint(lo), w[5 + 2 * i] = __float_as_uint(hi);
        } else {
            w[4 + i] = pack2<T>(lo, hi);
        }
    }
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
    uint8_t *p = reinterpret_cast<uint8_t *>(row + c);
    const bool full = c + 8 <= cols;
    if (off == 0) {
        if (full) {
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                reinterpret_cast<uint4 *>(p)[i] =
                    make_uint4(w[4 + 4 * i], w[5 + 4 * i], w[6 + 4 * i], w[7 + 4 * i]);
            return;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __shfl_up_sync(0xFFFFFFFFu, w[kWords + i], 1);
            w[kWords + 4 + i] = 0;
        }
        uint32_t x[kWords + 4];   // whole blocks from the one that holds p on
        shift_words<kWords + 4, kWords + 8>(w, 16u - off, x);
        if (full) {
            uint32_t *at = reinterpret_cast<uint32_t *>(p - off);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)   // block 0 starts in the lane before
                if (i > 0 || lane > 0)
                    reinterpret_cast<uint4 *>(at)[i] =
                        make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            if (lane == 0) {   // nobody before: the part of block 0 from p on
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    if (4 * j >= off) at[j] = x[j];
                    else if (sizeof(T) == 2 && 4 * j + 2 == off)
                        reinterpret_cast<uint16_t *>(at)[2 * j + 1] = static_cast<uint16_t>(x[j] >> 16);
            }
            if (lane == 31 || c + 16 > cols) {   // nobody after: the beginning of the last block
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    if (4 * j + 4 <= off) at[kWords + j] = x[kWords + j];
                    else if (sizeof(T) == 2 && 4 * j + 2 == off)
                        reinterpret_cast<uint16_t *>(at)[2 * (kWords + j)] = static_cast<uint16_t>(x[kWords + j]);
            }
            return;
        }
    }
    // a group that the row's end cuts
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (c + i < cols) {
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(p)[i] = w[4 + i];
            else
                reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[4 + i / 2] >> (16 * (i & 1)));
        }
    }
}

// row * ld, both below 2^31, in one instruction
__device__ __forceinline__ int64_t row_at(unsigned row, int64_t ld) {
    return static_cast<int64_t>(static_cast<uint64_t>(row) * static_cast<uint32_t>(ld));
}

// ------------------------------------------------------------ block scales --

// E8M0 byte of a block: e + 127 for the smallest e >= -127 with amax <= fmax 2^e.
// Both formats' fmax is 1.75 2^t (t = 8 or 15).  With amax = f 2^p, 1 <= f < 2, e is
// p - t if f <= 1.75 and p - t + 1 otherwise, and the biased exponent field of
// amax is p + 127.  A subnormal amax (field 0) gives byte 0, as it should.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    // adding 0x1FFFFF carries into the exponent exactly when the fraction is above .75
    const int e = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - (FMT == 0 ? 8 : 15);
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

// Scale of row-block rb, column-block cb (rb and the row stride below 2^31).
__device__ __forceinline__ int64_t scale_at(const BlockView &q, int64_t rb, int64_t cb) {
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(rb)) *
                                static_cast<uint32_t>(q.ld_s)) + cb;
}
__device__ __forceinline__ void store_scale(const BlockView &q, int64_t rb, int64_t cb,
                                            uint32_t byte) {
    if (q.scale_f32)
        static_cast<float *>(q.scales)[scale_at(q, rb, cb)] = scale_value(byte);
    else
        static_cast<uint8_t *>(q.scales)[scale_at(q, rb, cb)] = static_cast<uint8_t>(byte);
}
// A scale on its way, and its value: apart, so that a scale can be fetched ahead of its
// use (the first instruction on a loaded value waits for it).
__device__ __forceinline__ uint32_t fetch_scale(const BlockView &q, int64_t rb, int64_t cb) {
    if (q.scale_f32) return static_cast<const uint32_t *>(q.scales)[scale_at(q, rb, cb)];
    return static_cast<const uint8_t *>(q.scales)[scale_at(q, rb, cb)];
}
__device__ __forceinline__ float fetched_scale(const BlockView &q, uint32_t raw) {
    return q.scale_f32 ? __uint_as_float(raw) : scale_value(raw);
}
__device__ __forceinline__ float load_scale(const BlockView &q, int64_t rb, int64_t cb) {
    return fetched_scale(q, fetch_scale(q, rb, cb));
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

// Four values (two packed pairs) to a word of four codes.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(uint64_t ab, uint64_t cd) {
    float a, b, c, d;
    f32x2_unpack(ab, a, b);
    f32x2_unpack(cd, c, d);
    uint32_t w;
    if constexpr (FMT == 0)
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
            : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
            : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// max(m, |a|, |b|) in one instruction; NaN does not count.  m is not NaN.
__device__ __forceinline__ float absmax3(float m, float a, float b) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float absmax3(float m, uint64_t ab) {
    float a, b;
    f32x2_unpack(ab, a, b);
    return absmax3(m, a, b);
}
__device__ __forceinline__ bool is_inf(float m) { return m == __uint_as_float(0x7F800000u); }
// the pair with 0 in place of infinities: what a maximum that came out infinite is
// taken over again
__device__ __forceinline__ uint64_t without_inf(uint64_t ab) {
    float a, b;
    f32x2_unpack(ab, a, b);
    return f32x2_pack(is_inf(fabsf(a)) ? 0.0f : a, is_inf(fabsf(b)) ? 0.0f : b);
}

// bytes [0, n) of a word of codes to p (4-byte aligned)
__device__ __forceinline__ void store_code_word(uint8_t *p, uint32_t w, int64_t n) {
    if (n >= 4) {
        *reinterpret_cast<uint32_t *>(p) = w;
    } else {
        for (int i = 0; i < n; ++i) p[i] = static_cast<uint8_t>(w >> (8 * i));
    }
}

// One row's block-scaled output by lanes that hold 2 P = 8 or 16 consecutive columns
// each: 64 / P lanes hold a block of 128.  Addresses are kept for this thread's columns
// and moved from row to row.
struct RowWriter {
    uint8_t *code;     // of this thread's first column
    uint8_t *scale;

    __device__ __forceinline__ void start(const BlockView &q, int64_t row, int64_t c) {
        code = q.codes + row_at(static_cast<unsigned>(row), q.ld) + c;
        scale = static_cast<uint8_t *>(q.scales) +
                (row_at(static_cast<unsigned>(row), q.ld_s) + (c >> 7)) * (q.scale_f32 ? 4 : 1);
    }
    __device__ __forceinline__ void move(const BlockView &q, unsigned rows) {
        code += row_at(rows, q.ld);
        scale += row_at(rows, q.ld_s) * (q.scale_f32 ? 4 : 1);
    }
    // All lanes of the warp take part; `left` columns of the row are from the values'
    // first on (0 or less: none; the values there are 0).  at: columns past the
    // thread's first.
    template <int P>
    __device__ __forceinline__ void put(const BlockView &q, const uint64_t (&v)[P], int at, int left) const {
        if (q.fmt != 0)
            put_as<1>(q, v, at, left);
        else
            put_as<0>(q, v, at, left);
    }
    template <int FMT, int P>
    __device__ __forceinline__ void put_as(const BlockView &q, const uint64_t (&v)[P], int at, int left) const {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) m = absmax3(m, v[i]);
        if (is_inf(m)) {
            m = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) m = absmax3(m, without_inf(v[i]));
        }
#pragma unroll
        for (int o = 32 / P; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const uint32_t byte = scale_byte<FMT>(__float_as_uint(m));
        const uint64_t inv2 = splat_f32x2(scale_inverse(byte));
        uint32_t w[P / 2];
#pragma unroll
        for (int i = 0; i < P / 2; ++i)
            w[i] = encode4<FMT>(f32x2_mul(v[2 * i], inv2), f32x2_mul(v[2 * i + 1], inv2));
        if (left <= 0) return;
        if ((threadIdx.x & (64 / P - 1)) == 0) {
            if (q.scale_f32)
                *reinterpret_cast<float *>(scale + (at >> 7) * 4) = scale_value(byte);
            else
                scale[at >> 7] = static_cast<uint8_t>(byte);
        }
        if (left >= 2 * P) {
            if constexpr (P == 8)
                *reinterpret_cast<uint4 *>(code + at) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint2 *>(code + at) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) store_code_word(code + at + 4 * i, w[i], left - 4 * i);
        }
    }
};

// ----------------------------------------------------------- tile kernels --
//
// Persistent CTAs of 512 threads hold one 128 x 128 tile at a time in fp32 registers:
// warp w has rows 8 w .. 8 w + 7, lane l columns 4 l .. 4 l + 3 as two packed
// pairs, so v[r][p] is row 8 w + r, columns 4 l + 2 p, + 1.  Elements outside the
// matrix are 0: they leave every maximum as it is.  While a tile is worked on, each
// warp's rows of the CTA's next tile are already on their way into shared memory
// (cp.async, waited for by that warp alone).  Rows that are not 16-byte aligned are not:
// the warp copies them element by element before it goes on, 32 loads one after the other.
//
// A row's maximum is one warp reduction.  A column's is taken over a thread's 8
// rows, then over the 16 warps by one thread per column.  The transposed codes go
// through shared memory and leave in rows of 128 bytes.

constexpr int kTile = 128;
constexpr int kTileThreads = 512;
constexpr int kTileRows = 8;   // rows per warp

using TileValues = uint64_t[kTileRows][2];

// A CTA's walk over the tiles of a matrix of tiles_r x tiles_c, gridDim.x apart.  Four
// rows of tiles are walked side by side, column by column, so that the neighbours whose
// scales share a word (four tiles down, four tiles across) and whose transposed rows
// continue each other are in flight together.
struct TileWalk {
    unsigned t, tiles, group, in, tiles_r, per_group;

    __device__ __forceinline__ TileWalk(unsigned rows, unsigned cols)
        : t(blockIdx.x), tiles(rows * cols), group(0), in(blockIdx.x), tiles_r(rows), per_group(4 * cols) {
        wrap();
    }
    __device__ __forceinline__ void wrap() {
        while (in >= per_group) in -= per_group, ++group;
    }
    __device__ __forceinline__ bool there() const { return t < tiles; }
    __device__ __forceinline__ void next() {
        t += gridDim.x, in += gridDim.x;
        wrap();
    }
    __device__ __forceinline__ void origin(unsigned &row0, unsigned &col0) const {
        const unsigned rows = min(4u, tiles_r - 4 * group);
        const unsigned r = rows == 4 ? in & 3 : in % rows, c = rows == 4 ? in >> 2 : in / rows;
        row0 = (4 * group + r) * kTile;
        col0 = c * kTile;
    }
};

__host__ __device__ constexpr int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// This warp's 8 rows x 128 columns of elements of SIZE bytes at (row0, col0) into
// its part of a stage (rows of 128 * SIZE bytes); outside the matrix: zeros.  vec:
// rows are 16-byte aligned; otherwise elements are copied one by one.
template <int SIZE>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const void *base, int64_t ld, int64_t rows,
                                           int64_t cols, bool vec, unsigned row0, unsigned col0) {
    constexpr int kPerRow = kTile * SIZE / 16;   // 16-byte chunks
    constexpr int kElems = 16 / SIZE;
    constexpr int kStep = 32 / kPerRow;          // rows per instruction of the warp
    const int lane = threadIdx.x & 31;
    const unsigned first = row0 + (threadIdx.x >> 5) * kTileRows;
    const uint8_t *p = static_cast<const uint8_t *>(base);
    if (vec) {
        const int r0 = lane / kPerRow, k = lane % kPerRow;
        const unsigned c = col0 + k * kElems;
        const uint8_t *src = p + (row_at(first + r0, ld) + c) * SIZE;
        const uint32_t to = dst + r0 * kTile * SIZE + k * 16;
        if (row0 + kTile <= rows && col0 + kTile <= cols) {
#pragma unroll
            for (int i = 0; i < kTileRows / kStep; ++i, src += kStep * ld * SIZE)
                cp_async16(to + i * kStep * kTile * SIZE, src, 16);
        } else {
            const int64_t left = (cols - static_cast<int64_t>(c)) * SIZE;
            const uint32_t bytes = left <= 0 ? 0u : left < 16 ? static_cast<uint32_t>(left) : 16u;
#pragma unroll
            for (int i = 0; i < kTileRows / kStep; ++i, src += kStep * ld * SIZE) {
                const uint32_t n = first + r0 + i * kStep < rows ? bytes : 0u;
                cp_async16(to + i * kStep * kTile * SIZE, n ? src : p, n);
            }
        }
    } else {
        for (int idx = lane; idx < kTileRows * kTile; idx += 32) {
            const int r = idx / kTile, k = idx % kTile;
            const bool in = first + r < rows && col0 + k < cols;
            const uint8_t *src = p + (row_at(first + r, ld) + col0 + k) * SIZE;
            const uint32_t at = dst + idx * SIZE;
            if constexpr (SIZE == 4) {
                const uint32_t w = in ? *reinterpret_cast<const uint32_t *>(src) : 0u;
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
            } else {
                const uint16_t w = in ? *reinterpret_cast<const uint16_t *>(src) : uint16_t(0);
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(w) : "memory");
            }
        }
    }
}

// Row r's four elements of this lane from a warp's part of a stage.
template <typename T>
__device__ __forceinline__ void staged4(const uint8_t *part, int r, uint64_t (&v)[2]) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 4) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(part + r * 512 + lane * 16);
        v[0] = u.x, v[1] = u.y;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(part + r * 256 + lane * 8);
        const float2 a = unpack2<T>(u.x), b = unpack2<T>(u.y);
        v[0] = f32x2_pack(a.x, a.y), v[1] = f32x2_pack(b.x, b.y);
    }
}
// The same of FP8 codes, times the row's scale.
__device__ __forceinline__ void staged_codes4(const uint8_t *part, int r, int fmt, float scale,
                                              uint64_t (&v)[2]) {
    float f[4];
    decode4(*reinterpret_cast<const uint32_t *>(part + r * 128 + (threadIdx.x & 31) * 4), fmt, f);
    const uint64_t s2 = splat_f32x2(scale);
    v[0] = f32x2_mul(f32x2_pack(f[0], f[1]), s2);
    v[1] = f32x2_mul(f32x2_pack(f[2], f[3]), s2);
}

// Lane r (0 .. 7): the bits of row r's largest finite magnitude.
__device__ __forceinline__ uint32_t row_maxima(const TileValues &v) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0;
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        const float m = absmax3(absmax3(0.0f, v[r][0]), v[r][1]);
        const uint32_t row = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
        if (lane == r) mine = row;
    }
    if (__any_sync(0xFFFFFFFFu, mine == 0x7F800000u)) {
#pragma unroll 1
        for (int r = 0; r < kTileRows; ++r) {
            float m = 0.0f;
#pragma unroll
            for (int k = 0; k < kTileRows; ++k)
                if (k == r) m = absmax3(absmax3(0.0f, without_inf(v[k][0])), without_inf(v[k][1]));
            const uint32_t row = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
            if (lane == r) mine = row;
        }
    }
    return mine;
}

// The tile's own maximum (block_rows 128), the same in every thread.  One barrier;
// red is not written again before another one.
__device__ __forceinline__ uint32_t tile_max(const TileValues &v, uint32_t *red) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, row_maxima(v));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, red[threadIdx.x & 15]);
}

// Row-major codes and scales of the tile at (row0, col0).  tile_byte < 0: one
// scale per row; otherwise the whole tile's.
template <int FMT>
__device__ __forceinline__ void tile_rows(const TileValues &v, const BlockView &q, unsigned row0,
                                          unsigned col0, int tile_byte) {
    const int lane = threadIdx.x & 31;
    const unsigned first = row0 + (threadIdx.x >> 5) * kTileRows, c = col0 + 4 * lane;
    uint32_t byte = static_cast<uint32_t>(tile_byte);   // lane r: of row r
    if (tile_byte < 0) {
        byte = scale_byte<FMT>(row_maxima(v));
        if (lane < kTileRows && first + lane < q.rows) store_scale(q, first + lane, col0 / kTile, byte);
    } else if (threadIdx.x == 0) {
        store_scale(q, row0 / kTile, col0 / kTile, byte);
    }
    const float inv = scale_inverse(byte);
    uint8_t *p = q.codes + row_at(first, q.ld) + c;
    if (row0 + kTile <= q.rows && col0 + kTile <= q.cols) {
#pragma unroll
        for (int r = 0; r < kTileRows; ++r, p += q.ld) {
            const uint64_t inv2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, inv, r));
            *reinterpret_cast<uint32_t *>(p) =
                encode4<FMT>(f32x2_mul(v[r][0], inv2), f32x2_mul(v[r][1], inv2));
        }
    } else {
#pragma unroll
        for (int r = 0; r < kTileRows; ++r, p += q.ld) {
            const uint64_t inv2 = splat_f32x2(__shfl_sync(0xFFFFFFFFu, inv, r));
            const uint32_t code = encode4<FMT>(f32x2_mul(v[r][0], inv2), f32x2_mul(v[r][1], inv2));
            if (first + r < q.rows && c < q.cols) store_code_word(p, code, q.cols - c);
        }
    }
}

// Transposition, in steps with a barrier between each two:
//   cols_max     per warp and column, the maximum over the warp's rows;
//   cols_scale   one thread per column: its scale, to memory and, inverted, to inv;
//   cols_codes   codes into `codes`: column c's 128 bytes are its row c, in
//                chunks of 16 bytes (two warps' 8 rows each); chunk k is kept at place
//                k ^ ((c >> 2) & 7), its halves swapped when bit 5 of c is set: the
//                lanes of a warp write 8 bytes each to columns 4 apart, and half a warp
//                then covers all banks once;
//   cols_store   the tile's columns as rows of qt.
struct ColsSmem {
    uint32_t max[16][kTile];
    float inv[kTile];
    uint8_t codes[kTile * kTile];
};

__device__ __forceinline__ void cols_max(const TileValues &v, ColsSmem &sm) {
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto take = [&](int r, uint64_t a0, uint64_t a1, uint64_t b0, uint64_t b1) {
        float x, y, z, w;
        f32x2_unpack(a0, x, y);
        f32x2_unpack(b0, z, w);
        m[0] = absmax3(m[0], x, z);
        m[1] = absmax3(m[1], y, w);
        f32x2_unpack(a1, x, y);
        f32x2_unpack(b1, z, w);
        m[2] = absmax3(m[2], x, z);
        m[3] = absmax3(m[3], y, w);
    };
#pragma unroll
    for (int r = 0; r < kTileRows; r += 2) take(r, v[r][0], v[r][1], v[r + 1][0], v[r + 1][1]);
    if (is_inf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])))) {
        m[0] = m[1] = m[2] = m[3] = 0.0f;
#pragma unroll
        for (int r = 0; r < kTileRows; r += 2)
            take(r, without_inf(v[r][0]), without_inf(v[r][1]), without_inf(v[r + 1][0]),
                 without_inf(v[r + 1][1]));
    }
    *reinterpret_cast<float4 *>(&sm.max[threadIdx.x >> 5][4 * (threadIdx.x & 31)]) =
        make_float4(m[0], m[1], m[2], m[3]);
}

// thread c (0 .. 127) of the caller's choice
template <int FMT>
__device__ __forceinline__ void cols_scale(int c, ColsSmem &sm, const BlockView &qt, unsigned row0,
                                           unsigned col0) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) m = max(m, sm.max[w][c]);
    const uint32_t byte = scale_byte<FMT>(m);
    sm.inv[c] = scale_inverse(byte);
    if (col0 + c < qt.rows) store_scale(qt, col0 + c, row0 / kTile, byte);
}

template <int FMT>
__device__ __forceinline__ void cols_codes(const TileValues &v, const ulonglong2 inv, ColsSmem &sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float lo[kTileRows], hi[kTileRows];
#pragma unroll
        for (int r = 0; r < kTileRows; ++r)
            f32x2_unpack(f32x2_mul(v[r][p], p ? inv.y : inv.x), lo[r], hi[r]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float(&x)[kTileRows] = j ? hi : lo;
            const int c = 4 * lane + 2 * p + j;
            const int at = c * kTile + (((warp >> 1) ^ ((c >> 2) & 7)) << 4) +
                           (((warp & 1) ^ ((c >> 5) & 1)) << 3);
            *reinterpret_cast<uint2 *>(&sm.codes[at]) =
                make_uint2(encode4<FMT>(f32x2_pack(x[0], x[1]), f32x2_pack(x[2], x[3])),
                           encode4<FMT>(f32x2_pack(x[4], x[5]), f32x2_pack(x[6], x[7])));
        }
    }
}

__device__ __forceinline__ void cols_store(const ColsSmem &sm, const BlockView &qt, unsigned row0,
                                           unsigned col0) {
    constexpr int kRows = kTileThreads / 8;   // of qt per step
    const int c0 = threadIdx.x >> 3, k = threadIdx.x & 7;
    const unsigned r = row0 + 16 * k;
    uint8_t *p = qt.codes + row_at(col0 + c0, qt.ld) + r;
    // steps keep c >> 2 modulo 8 and bit 5 of c as they are
    static_assert(kRows % 64 == 0, "the swizzle is the same in every step");
    const uint8_t *from = &sm.codes[c0 * kTile + ((k ^ ((c0 >> 2) & 7)) << 4)];
    const bool swap = (c0 >> 5) & 1;
    const bool whole = col0 + kTile <= qt.rows && row0 + kTile <= qt.cols;
#pragma unroll
    for (int i = 0; i < kTile / kRows; ++i, p += kRows * qt.ld) {
        uint4 u = *reinterpret_cast<const uint4 *>(from + i * kRows * kTile);
        if (swap) u = make_uint4(u.z, u.w, u.x, u.y);
        const unsigned c = col0 + c0 + i * kRows;
        if (whole || (c < qt.rows && r + 16 <= qt.cols)) {
            *reinterpret_cast<uint4 *>(p) = u;
        } else if (c < qt.rows) {
            const int64_t left = qt.cols - static_cast<int64_t>(r);
            store_code_word(p, u.x, left);
            store_code_word(p + 4, u.y, left - 4);
            store_code_word(p + 8, u.z, left - 8);
            store_code_word(p + 12, u.w, left - 12);
        }
    }
}

__device__ __forceinline__ ulonglong2 cols_inv(const ColsSmem &sm) {
    return *reinterpret_cast<const ulonglong2 *>(&sm.inv[4 * (threadIdx.x & 31)]);
}

}  // namespace fp8k
