// norm_rows.cuh -- what the norms' kernels (layernorm.cu, rmsnorm.cu) share: who works on
// a row, sums over it, parameters along it, and its values kept in 8 bits.
#pragma once

#include "block.cuh"
#include "ln_plan.h"

namespace fp8k {

// Who works on a row: a warp (narrow rows; a CTA has kWarps of them at a time) or the
// whole CTA.  Thread i of the team holds columns E (i + k team) .. + E - 1 for k < VPT,
// as packed pairs.  VEC is E where rows are 16-byte aligned and a multiple of E columns
// long, and 0 where anything goes (then E = 8).  The forward takes 16: fewer lanes
// share a block's maximum.  LayerNorm's backward takes 8 like the general case, so that its
// sums are the same bits at any alignment.  (RMS norm's rows of up to 8192 columns that start
// anywhere have another order, 32 columns apart: other bits than the same values aligned.)

template <typename T, int VEC>
struct Lay {
    static constexpr int E = VEC, P = VEC / 2;
    using Raw = RawVec<T, VEC>;
    static __device__ __forceinline__ void store(T *row, int64_t c, int64_t cols, const uint64_t (&v)[P]) {
        Raw::store(row, c, cols, v);
    }
};
template <typename T>
struct Lay<T, 0> {
    static constexpr int E = 8, P = 4;
    using Raw = RawRow8<T>;
    static __device__ __forceinline__ void store(T *row, int64_t c, int64_t cols, const uint64_t (&v)[4]) {
        store_row8<T>(row, c, cols, v);
    }
};

template <bool WARP>
struct Team {
    int id, size;        // this thread's place, threads per row
    int64_t row, step;   // the first row, and from one to the next
    __device__ __forceinline__ Team() {
        if constexpr (WARP) {
            id = threadIdx.x & 31, size = 32;
            row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
            step = static_cast<int64_t>(gridDim.x) * kWarps;
        } else {
            id = threadIdx.x, size = blockDim.x;
            row = blockIdx.x, step = gridDim.x;
        }
    }
};

// Sum of a pair over the team, in a fixed order, the same in every thread.  A CTA's
// calls alternate between two buffers: a buffer is written again only after a
// barrier that follows its last read.
// The warps' sums meet in shared memory (unused places hold zeros); every thread adds up
// all of them, which is a shorter way than five more exchanges between lanes.
template <bool WARP>
__device__ __forceinline__ float2 team_sum2(float a, float b, uint64_t (&buf)[16]) {
    uint64_t v = f32x2_pack(a, b);
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f32x2_add(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(buf);
        uint64_t s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const ulonglong2 u = p[i];
            s[i] = f32x2_add(u.x, u.y);
        }
        v = f32x2_add(f32x2_add(s[0], s[1]), f32x2_add(s[2], s[3]));
        if (blockDim.x > 256) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 u = p[4 + i];
                s[i] = f32x2_add(u.x, u.y);
            }
            v = f32x2_add(v, f32x2_add(f32x2_add(s[0], s[1]), f32x2_add(s[2], s[3])));
        }
    }
    f32x2_unpack(v, a, b);
    return make_float2(a, b);
}
// One value: half the exchanges.
template <bool WARP>
__device__ __forceinline__ float team_sum(float a, uint64_t (&buf)[16]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a = __fadd_rn(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0) reinterpret_cast<float *>(buf)[threadIdx.x >> 5] = a;
        __syncthreads();
        const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(buf);
        ulonglong2 u = p[0], w = p[1];
        uint64_t v = f32x2_add(f32x2_add(u.x, u.y), f32x2_add(w.x, w.y));
        if (blockDim.x > 256) {
            u = p[2], w = p[3];
            v = f32x2_add(v, f32x2_add(f32x2_add(u.x, u.y), f32x2_add(w.x, w.y)));
        }
        float lo, hi;
        f32x2_unpack(v, lo, hi);
        a = __fadd_rn(lo, hi);
    }
    return a;
}
// Zeros in both buffers, before their first use.
__device__ __forceinline__ void clear_sums(uint64_t (&buf)[2][16]) {
    if (threadIdx.x < 32) buf[threadIdx.x >> 4][threadIdx.x & 15] = 0;
    __syncthreads();
}

__device__ __forceinline__ float sum2(uint64_t v) {
    float lo, hi;
    f32x2_unpack(v, lo, hi);
    return __fadd_rn(lo, hi);
}

// s / n given 1 / n: the product, corrected by its remainder.  An infinite sum has none
// (inf - inf): its quotient is infinite, as a division gives it.  (8192 x 4096 with both 8-bit
// outputs: 37.9 us, 37.4 without that choice, 39.8 with a division.)
__device__ __forceinline__ float quotient(float s, float n, float inv_n) {
    const float q = __fmul_rn(s, inv_n);
    const float r = __fmaf_rn(__fmaf_rn(-q, n, s), inv_n, q);
    return is_inf(fabsf(q)) ? q : r;
}

// gamma or beta at columns c .. c + 2 P - 1 (c a multiple of 8); 0 past the row.  One
// branch on the type, so that all loads are on their way together (a branch per element
// made them wait for one another: 10 us of a call).
template <typename T, int P>
__device__ __forceinline__ void load_param_as(const T *p, int64_t c, int64_t cols, uint64_t (&v)[P]) {
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && c + 2 * P <= cols) {
#pragma unroll
        for (int k = 0; k < P / 4; ++k) {
            RawVec<T, 8> raw;
            raw.load(p, c + 8 * k, cols);
            uint64_t x[4];
            raw.get(p, 0, 0, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * k + i] = x[i];
        }
    } else {
        float f[2 * P];
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) f[i] = c + i < cols ? to_f32(p[c + i]) : 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = f32x2_pack(f[2 * i], f[2 * i + 1]);
    }
}
template <int P>
__device__ __forceinline__ void load_param(const void *p, int type, int64_t c, int64_t cols,
                                           uint64_t (&v)[P]) {
    if (type == kTypeF32)
        load_param_as(static_cast<const float *>(p), c, cols, v);
    else if (type == kTypeBF16)
        load_param_as(static_cast<const __nv_bfloat16 *>(p), c, cols, v);
    else
        load_param_as(static_cast<const __half *>(p), c, cols, v);
}

// 8 codes times their scale plus a number; `left` of them belong to the row, the others
// may be anything.  (A code times a power of two is exact: one rounding either way.)
__device__ __forceinline__ void codes8(uint2 w, int fmt, float scale, uint64_t plus, int left,
                                       uint64_t (&v)[4]) {
    const uint64_t s2 = splat_f32x2(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4];
        decode4(i ? w.y : w.x, fmt, f);
        if (left < 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = 4 * i + k < left ? f[k] : 0.0f;
        }
        v[2 * i] = f32x2_fma(f32x2_pack(f[0], f[1]), s2, plus);
        v[2 * i + 1] = f32x2_fma(f32x2_pack(f[2], f[3]), s2, plus);
    }
}

// 8 codes times their scale; `left` of them belong to the row.
__device__ __forceinline__ void codes8_times(uint2 w, int fmt, float scale, int left, uint64_t (&v)[4]) {
    const uint64_t s2 = splat_f32x2(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4];
        decode4(i ? w.y : w.x, fmt, f);
        if (left < 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = 4 * i + k < left ? f[k] : 0.0f;
        }
        v[2 * i] = f32x2_mul(f32x2_pack(f[0], f[1]), s2);
        v[2 * i + 1] = f32x2_mul(f32x2_pack(f[2], f[3]), s2);
    }
}

__host__ __device__ constexpr int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

inline bool aligned_rows(const void *p, int64_t ld, int type) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (type == kTypeF32 ? 4 : 2) % 16 == 0;
}

}  // namespace fp8k
