// rmsnorm.cu -- root-mean-square norm with the residual's addition, forward and backward.
//
// Forward, per row, in fp32:
//   s = x + residual, rounded to the rows' type (s = x without a residual),
//   rstd = 1 / sqrt(sum s^2 / cols + eps),  y = (s * rstd) * gamma
// s is rounded before the norm is taken of it, so that the backward pass, which reads s
// again, has the value that the forward had.
// Backward, with xhat = s * rstd and u = dy * gamma:
//   dx = dsum + rstd * (u - xhat * sum(u * xhat) / cols)
//   dgamma = sum over rows of dy * xhat
// dsum is the gradient that reaches s on the residual's way (0 where it is not given);
// x and the residual have the same gradient, dx.
//
// Both are bound by HBM.  Forward, up to 16384 columns, and backward, up to 8192, a row stays
// in its CTA's registers between the sum and the use of the sum, and each value is read and
// written once; backward, aligned rows of up to 16384 columns wait in shared memory and are
// read from there twice.  Longer rows, and unaligned ones past 8192 columns backward, are read
// from memory twice.
// dgamma: a thread adds its CTA's rows one after the other in fp32 (54 of them at 8192 x 8192),
// and CTAs' sums are joined by a tree: known to that many and some 2^-24 of the sum of the terms'
// magnitudes.
#include <cstdint>
#include <type_traits>

#include "error_flag.h"
#include "norm_rows.cuh"
#include "once_per_device.h"

namespace fp8k {

namespace {

__device__ unsigned g_rms_error_flags = 0;

// Rows that start anywhere (their length is odd, or they are views): element by element, each
// warp instruction along 32 of them, instead of 16-byte blocks shifted into place.  A thread
// has kSpread columns 32 apart, a warp 512 in a row, four whole blocks of 128.
constexpr int kSpread = 16;
// Forward, CTAs of up to 320 threads (5120 columns) have 96 registers, so that two of them fit an
// SM, and larger ones 128: 8000 x 4099 bf16 with the sum 62.1 us, and 91.4 with 128 throughout; in
// 8 bits with the sum kept 89.1 and 134.3.  (Aligned rows, which take 118 registers: from 4097
// columns on, 8192 x 4608 in 8 bits 57.9 us, and 71.9.)
constexpr int kFwdHalf = 320;

template <typename T>
__device__ __forceinline__ uint32_t raw_of(const T *p) {
    if constexpr (sizeof(T) == 4)
        return *reinterpret_cast<const uint32_t *>(p);
    else
        return *reinterpret_cast<const uint16_t *>(p);
}
template <typename T>
__device__ __forceinline__ float value_of(uint32_t raw) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(raw);
    else return to_f32(*reinterpret_cast<const T *>(&raw));
}
// kSpread elements from p on, 32 apart; of the first `left` elements from p on (a full warp's: all)
template <typename T>
__device__ __forceinline__ void load_spread(const T *p, int left, bool full, uint32_t (&raw)[kSpread]) {
    if (full) {
#pragma unroll
        for (int j = 0; j < kSpread; ++j) raw[j] = raw_of(p + 32 * j);
    } else {
#pragma unroll
        for (int j = 0; j < kSpread; ++j) raw[j] = 32 * j < left ? raw_of(p + 32 * j) : 0u;
    }
}
template <typename T>
__device__ __forceinline__ void store_spread(T *p, int left, bool full, const float (&v)[kSpread]) {
    uint32_t raw[kSpread];
#pragma unroll
    for (int j = 0; j < kSpread; j += 2) {
        if constexpr (sizeof(T) == 4) {
            raw[j] = __float_as_uint(v[j]), raw[j + 1] = __float_as_uint(v[j + 1]);
        } else {
            raw[j] = pack2<T>(v[j], v[j + 1]);
            raw[j + 1] = raw[j] >> 16;
        }
    }
    using U = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    U *to = reinterpret_cast<U *>(p);
    if (full) {
#pragma unroll
        for (int j = 0; j < kSpread; ++j) to[32 * j] = static_cast<U>(raw[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kSpread; ++j)
            if (32 * j < left) to[32 * j] = static_cast<U>(raw[j]);
    }
}
// The warp's four blocks of a row, quantized.  Columns outside the row are 0 and not stored.
template <int FMT>
__device__ __forceinline__ void quantize_spread(const BlockView &q, int64_t row, int64_t c, int left, bool full,
                                                const float (&v)[kSpread]) {
    const int lane = threadIdx.x & 31;
    uint8_t *p = q.codes + row_at(static_cast<unsigned>(row), q.ld) + c;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        float m = absmax3(absmax3(0.0f, v[4 * b], v[4 * b + 1]), v[4 * b + 2], v[4 * b + 3]);
        if (is_inf(m)) {
            m = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!is_inf(fabsf(v[4 * b + k]))) m = absmax3(m, v[4 * b + k], v[4 * b + k]);
        }
        const uint32_t byte = scale_byte<FMT>(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m)));
        const float inv = scale_inverse(byte);
        const uint32_t w = cvt2_fp8<FMT>(__fmul_rn(v[4 * b], inv), __fmul_rn(v[4 * b + 1], inv)) |
                           cvt2_fp8<FMT>(__fmul_rn(v[4 * b + 2], inv), __fmul_rn(v[4 * b + 3], inv)) << 16;
        if (lane == 0 && 128 * b < left) store_scale(q, row, (c >> 7) + b, byte);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (full || 128 * b + 32 * k < left) p[128 * b + 32 * k] = static_cast<uint8_t>(w >> (8 * k));
    }
}
__device__ __forceinline__ void quantize_spread(const BlockView &q, int64_t row, int64_t c, int left, bool full,
                                                const float (&v)[kSpread]) {
    if (q.fmt != 0)
        quantize_spread<1>(q, row, c, left, full, v);
    else
        quantize_spread<0>(q, row, c, left, full, v);
}
// gamma at the thread's columns; 0 past the row
__device__ __forceinline__ void load_param_spread(const void *p, int type, int64_t c, int left, float (&v)[kSpread]) {
#pragma unroll
    for (int j = 0; j < kSpread; ++j) {
        v[j] = 0.0f;
        if (32 * j < left)
            v[j] = type == kTypeF32    ? static_cast<const float *>(p)[c + 32 * j]
                   : type == kTypeBF16 ? to_f32(static_cast<const __nv_bfloat16 *>(p)[c + 32 * j])
                                       : to_f32(static_cast<const __half *>(p)[c + 32 * j]);
    }
}

struct RmsFwdArgs {
    const void *x, *res;   // res null: no residual
    int64_t rows, cols, ldx, ldr;
    const void *gamma;
    int wtype;
    float eps;
    void *sum;   // null: not wanted
    int64_t lds;
    void *y;
    int64_t ldy;
    BlockView y8, x8;   // codes null: not wanted
    float *rstd;
};

// a + b as T holds it
template <typename T>
__device__ __forceinline__ uint64_t sum_as(uint64_t a, uint64_t b) {
    const uint64_t v = f32x2_add(a, b);
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        float lo, hi;
        f32x2_unpack(v, lo, hi);
        const float2 f = unpack2<T>(pack2<T>(lo, hi));
        return f32x2_pack(f.x, f.y);
    }
}

// The part that follows the statistic, for 2 P columns: `at` columns past the writers'
// first, `left` columns before the row's end.
template <typename T, int P>
__device__ __forceinline__ void rms_finish(const RmsFwdArgs &a, T *yr, const RowWriter &wy,
                                           const RowWriter &wx, int64_t c, int at, int left,
                                           uint64_t rs2, const uint64_t (&g)[P],
                                           const uint64_t (&x)[P]) {
    if (a.x8.codes != nullptr) wx.put(a.x8, x, at, left);
    if (a.y == nullptr && a.y8.codes == nullptr) return;
    uint64_t y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) y[i] = f32x2_mul(f32x2_mul(x[i], rs2), g[i]);
    if (a.y != nullptr) Lay<T, P == 8 ? 16 : 0>::store(yr, c, a.cols, y);
    if (a.y8.codes != nullptr) wy.put(a.y8, y, at, left);
}

// A team works on R rows side by side, one step apart: their sums share the exchanges and
// the barrier.  The rows after those in work are already being loaded, into registers.
// 8192 x 4096 bf16 with the sum and both in 8 bits 44.8 us = 6.0 TB/s, 0.89 of a copy's rate;
// half of the issue slots are busy, and 16 warps an SM (118 registers) do not hide the way from a
// row's sum to its codes any better.  One row of 4096 2.3 us.
// (A warp's rows in fp32 have more registers and one CTA an SM: with two they spill, 16384 x 512
// 28.3 us and 24.6; in 16 bits 12.7 with two and 15.6.  A CTA's rows spill and have two all the
// same.  fp32 with a residual, 256 threads, 336 bytes: 16384 x 2048 with sum and y 91.7 us, with
// one CTA 119.3; 8192 x 4096 91.6 and 87.6.  16 bits, 320 threads, 152 bytes and with a residual 392:
// see kFwdHalf.  Unaligned rows past 8192 columns with a residual spill 156 bytes, in fp32 384.)
template <typename T, int VPT, int THREADS, bool WARP, int VEC, bool RES>
__global__ void __launch_bounds__(THREADS, (WARP && sizeof(T) == 4) || THREADS > kFwdHalf ? 1 : 2)
    rms_fwd_kernel(const RmsFwdArgs a) {
    using L = Lay<T, VEC>;
    constexpr int E = L::E, P = L::P, R = VEC && VPT * P <= 8 ? 2 : 1;
    __shared__ __align__(16) uint64_t buf[2][16];
    const Team<WARP> team;
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols), inv_n = __fdiv_rn(1.0f, n);
    const int left0 = static_cast<int>(a.cols) - E * team.id;
    typename L::Raw raw[R][VPT], rawr[RES ? R : 1][RES ? VPT : 1];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (row + j * team.step < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    raw[j][k].load(static_cast<const T *>(a.x) + (row + j * team.step) * a.ldx,
                                   E * (team.id + k * team.size), a.cols);
                    if constexpr (RES)
                        rawr[j][k].load(static_cast<const T *>(a.res) + (row + j * team.step) * a.ldr,
                                        E * (team.id + k * team.size), a.cols);
                }
            }
    };
    if (team.row < a.rows) fetch(team.row);
    // gamma stays in registers where there is room for it
    constexpr bool kKeep = VPT * P <= 8;
    uint64_t g[kKeep ? VPT : 1][P];
    auto params = [&](int k, int slot) {
        load_param(a.gamma, a.wtype, E * (team.id + k * team.size), a.cols, g[slot]);
    };
    if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) params(k, k);
    }
    int flip = 0;
    for (int64_t row = team.row; row < a.rows; row += R * team.step, flip ^= 1) {
        uint64_t x[R][VPT][P];
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t at_row = row + j * team.step;
            uint64_t s2 = 0;
            if (at_row < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int64_t c = E * (team.id + k * team.size);
                    raw[j][k].get(static_cast<const T *>(a.x) + at_row * a.ldx, c, a.cols, x[j][k]);
                    if constexpr (RES) {
                        uint64_t r[P];
                        rawr[j][k].get(static_cast<const T *>(a.res) + at_row * a.ldr, c, a.cols, r);
#pragma unroll
                        for (int i = 0; i < P; ++i) x[j][k][i] = sum_as<T>(x[j][k][i], r[i]);
                    }
#pragma unroll
                    for (int i = 0; i < P; ++i) s2 = f32x2_fma(x[j][k][i], x[j][k][i], s2);
                }
            }
            q[j] = sum2(s2);
        }
        if (row + R * team.step < a.rows) fetch(row + R * team.step);
        if constexpr (RES) {
            if (a.sum != nullptr) {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (row + j * team.step < a.rows) {
#pragma unroll
                        for (int k = 0; k < VPT; ++k)
                            L::store(static_cast<T *>(a.sum) + (row + j * team.step) * a.lds,
                                     E * (team.id + k * team.size), a.cols, x[j][k]);
                    }
            }
        }
        float2 s;
        if constexpr (R == 2)
            s = team_sum2<WARP>(q[0], q[1], buf[flip]);
        else
            s = make_float2(team_sum<WARP>(q[0], buf[flip]), 0.0f);
        const float rs[2] = {__frsqrt_rn(__fadd_rn(quotient(s.x, n, inv_n), a.eps)),
                             __frsqrt_rn(__fadd_rn(quotient(s.y, n, inv_n), a.eps))};
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t at_row = row + j * team.step;
            if (at_row >= a.rows) break;
            if (team.id == 0) a.rstd[at_row] = rs[j];
            RowWriter wx, wy;
            wx.start(a.x8, at_row, E * team.id);
            wy.start(a.y8, at_row, E * team.id);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if constexpr (!kKeep) params(k, 0);
                const int at = E * k * team.size;
                rms_finish<T, P>(a, static_cast<T *>(a.y) + at_row * a.ldy, wy, wx, E * team.id + at, at,
                                 left0 - at, splat_f32x2(rs[j]), g[kKeep ? k : 0], x[j][k]);
            }
        }
    }
}

// Rows that start anywhere, up to 8192 columns: 3001 x 2731 fp32 with the sum 22.5 us = 5.8 TB/s
// (in 16-byte blocks shifted into place 39.2).
template <typename T, int THREADS, bool WARP, bool RES>
__global__ void __launch_bounds__(THREADS, THREADS == kFwdHalf ? 2 : 1) rms_fwd_spread_kernel(const RmsFwdArgs a) {
    __shared__ __align__(16) uint64_t buf[2][16];
    const Team<WARP> team;
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols), inv_n = __fdiv_rn(1.0f, n);
    const int64_t c = kSpread * (team.id & ~31) + (team.id & 31);
    const int left = static_cast<int>(a.cols - c);
    const bool full = left - 32 * (kSpread - 1) > 31 - (team.id & 31);   // of the whole warp
    uint32_t raw[kSpread], rawr[RES ? kSpread : 1];
    auto fetch = [&](int64_t row) {
        load_spread(static_cast<const T *>(a.x) + row * a.ldx + c, left, full, raw);
        if constexpr (RES) load_spread(static_cast<const T *>(a.res) + row * a.ldr + c, left, full, rawr);
    };
    if (team.row < a.rows) fetch(team.row);
    float g[kSpread];
    load_param_spread(a.gamma, a.wtype, c, left, g);
    int flip = 0;
    for (int64_t row = team.row; row < a.rows; row += team.step, flip ^= 1) {
        float x[kSpread], q = 0.0f;
#pragma unroll
        for (int j = 0; j < kSpread; ++j) {
            x[j] = value_of<T>(raw[j]);
            if constexpr (RES) x[j] = to_f32(from_f32<T>(__fadd_rn(x[j], value_of<T>(rawr[j]))));
            q = __fmaf_rn(x[j], x[j], q);
        }
        if (row + team.step < a.rows) fetch(row + team.step);
        if (RES && a.sum != nullptr) store_spread(static_cast<T *>(a.sum) + row * a.lds + c, left, full, x);
        const float s = team_sum<WARP>(q, buf[flip]);
        const float rs = __frsqrt_rn(__fadd_rn(quotient(s, n, inv_n), a.eps));
        if (team.id == 0) a.rstd[row] = rs;
        if (a.x8.codes != nullptr) quantize_spread(a.x8, row, c, left, full, x);
        if (a.y == nullptr && a.y8.codes == nullptr) continue;
#pragma unroll
        for (int j = 0; j < kSpread; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], rs), g[j]);
        if (a.y != nullptr) store_spread(static_cast<T *>(a.y) + row * a.ldy + c, left, full, x);
        if (a.y8.codes != nullptr) quantize_spread(a.y8, row, c, left, full, x);
    }
}

// Rows too long for a CTA's registers: s is read again for its use, from where the first
// pass put it (which may be x's or the residual's own place), else from x and the residual.
template <typename T, bool RES>
__global__ void __launch_bounds__(512) rms_fwd_wide_kernel(const RmsFwdArgs a) {
    __shared__ __align__(16) uint64_t buf[2][16];
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols);
    // whole warps stay together: the exchanges between lanes need all of them
    const int64_t warp0 = 8 * (threadIdx.x & ~31);
    RowWriter wx, wy;
    wx.start(a.x8, blockIdx.x, 8 * threadIdx.x);
    wy.start(a.y8, blockIdx.x, 8 * threadIdx.x);
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const T *xr = static_cast<const T *>(a.x) + row * a.ldx;
        const T *rr = static_cast<const T *>(a.res) + row * a.ldr;
        T *sr = static_cast<T *>(a.sum) + row * a.lds;
        auto load = [&](const T *from, bool add, int64_t c, uint64_t (&v)[4]) {
            RawRow8<T> raw, rawr;
            raw.load(from, c, a.cols);
            if (add) rawr.load(rr, c, a.cols);
            raw.get(from, c, a.cols, v);
            if (add) {
                uint64_t r[4];
                rawr.get(rr, c, a.cols, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = sum_as<T>(v[i], r[i]);
            }
        };
        uint64_t x[4], s2 = 0;
        for (int64_t w = warp0; w < a.cols; w += 8 * 512) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            load(xr, RES, c, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = f32x2_fma(x[i], x[i], s2);
            if (RES && a.sum != nullptr) {
                __syncwarp();   // in place: a lane's store may finish its neighbour's last elements
                store_row8<T>(sr, c, a.cols, x);
            }
        }
        const float ms = __fdiv_rn(team_sum<false>(sum2(s2), buf[flip]), n);   // and a barrier after the stores
        const float rs = __frsqrt_rn(__fadd_rn(ms, a.eps));
        if (threadIdx.x == 0) a.rstd[row] = rs;
        const bool stored = RES && a.sum != nullptr;
        for (int64_t w = warp0; w < a.cols; w += 8 * 512) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            uint64_t g[4];
            load_param(a.gamma, a.wtype, c, a.cols, g);
            load(stored ? sr : xr, RES && !stored, c, x);
            rms_finish<T, 4>(a, static_cast<T *>(a.y) + row * a.ldy, wy, wx, c, static_cast<int>(w - warp0),
                             static_cast<int>(a.cols - c), splat_f32x2(rs), g, x);
        }
        wx.move(a.x8, gridDim.x);
        wy.move(a.y8, gridDim.x);
    }
}

struct RmsBwdArgs {
    const void *dy, *x, *dsum;   // dsum null: none
    int64_t rows, cols, lddy, ldx, ldds, lddx;
    BlockView x8;
    const void *gamma;
    int wtype;
    const float *rstd;
    void *dx;
    float *part;       // [gridDim.x][up8(cols)]: a CTA's sums of dy * xhat
    float *row_sums;   // wide rows: [rows] sums of u * xhat
};

// Columns of x on their way, as they are or codes with their block's scale.
template <typename T, bool SAVED, int VEC>
struct RmsRawX {
    typename Lay<T, VEC>::Raw raw;
    __device__ __forceinline__ void load(const RmsBwdArgs &a, int64_t row, int64_t c) {
        raw.load(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols);
    }
    __device__ __forceinline__ void get(const RmsBwdArgs &a, int64_t row, int64_t c,
                                        uint64_t (&v)[Lay<T, VEC>::P]) const {
        raw.get(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, v);
    }
};
template <typename T, int VEC>
struct RmsRawX<T, true, VEC> {
    static constexpr int P = Lay<T, VEC>::P;
    static_assert(P == 4, "8 codes");
    uint32_t w[2], scale;
    __device__ __forceinline__ void load(const RmsBwdArgs &a, int64_t row, int64_t c) {
        w[0] = w[1] = scale = 0;
        if (c < a.cols) {
            const uint2 u = *reinterpret_cast<const uint2 *>(a.x8.codes + row * a.x8.ld + c);
            w[0] = u.x, w[1] = u.y;
            scale = fetch_scale(a.x8, row, c >> 7);
        }
    }
    __device__ __forceinline__ void get(const RmsBwdArgs &a, int64_t, int64_t c, uint64_t (&v)[P]) const {
        codes8_times(make_uint2(w[0], w[1]), a.x8.fmt, fetched_scale(a.x8, scale),
                     VEC ? 8 : static_cast<int>(a.cols - c), v);
    }
};

// xhat in place of x, and u in place of dy; their sum for the row, and the column sums
template <int P>
__device__ __forceinline__ void rms_bwd_accumulate(uint64_t rs2, const uint64_t (&g)[P], uint64_t (&dy)[P],
                                                   uint64_t (&x)[P], uint64_t (&dg)[P], uint64_t &s) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        x[i] = f32x2_mul(x[i], rs2);
        dg[i] = f32x2_fma(dy[i], x[i], dg[i]);
        dy[i] = f32x2_mul(dy[i], g[i]);
        s = f32x2_fma(dy[i], x[i], s);
    }
}

// dx in place of u: dsum + rstd (u + xhat * nm)
template <int P>
__device__ __forceinline__ void rms_bwd_finish(uint64_t rs2, uint64_t nm2, const uint64_t (&x)[P],
                                               const uint64_t (&ds)[P], uint64_t (&dy)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) dy[i] = f32x2_fma(f32x2_fma(x[i], nm2, dy[i]), rs2, ds[i]);
}

// Longer rows, and unaligned ones past 8192 columns: the row sum, in a pass of its own.
template <typename T, bool SAVED>
__global__ void __launch_bounds__(512) rms_bwd_sums_kernel(const RmsBwdArgs a) {
    __shared__ __align__(16) uint64_t buf[2][16];
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const uint64_t rs2 = splat_f32x2(a.rstd[row]);
        uint64_t s = 0;
        for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * 512) {
            const T *dyr = static_cast<const T *>(a.dy) + row * a.lddy;
            RawRow8<T> rdy;
            RmsRawX<T, SAVED, 0> rx;
            rdy.load(dyr, c, a.cols);
            rx.load(a, row, c);
            uint64_t dy[4], x[4], g[4], dg[4] = {};
            load_param(a.gamma, a.wtype, c, a.cols, g);
            rdy.get(dyr, c, a.cols, dy);
            rx.get(a, row, c, x);
            rms_bwd_accumulate(rs2, g, dy, x, dg, s);
        }
        const float sum = team_sum<false>(sum2(s), buf[flip]);
        if (threadIdx.x == 0) a.row_sums[row] = sum;
    }
}

template <int VPT, int P, typename Col>
__device__ __forceinline__ void rms_store_part(const RmsBwdArgs &a, Col col, const uint64_t (&dg)[VPT][P]) {
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * up8(a.cols);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int64_t c = col(k);
        if (c >= a.cols) continue;
#pragma unroll
        for (int i = 0; i < P / 2; ++i)
            *reinterpret_cast<ulonglong2 *>(part + c + 4 * i) = make_ulonglong2(dg[k][2 * i], dg[k][2 * i + 1]);
    }
}

// Rows of 257 .. 8192 columns, one at a time per CTA; a thread has 16 columns, and their sums
// over the CTA's rows.  The next rows of dy, x and dsum are on their way into a ring in
// shared memory by bulk copies of the 16-byte blocks that hold them, whatever their alignment;
// the barrier of a row's sum also tells that its place in the ring may be filled again (what a
// thread needs of dsum is in its registers by then).  8192 x 8192 bf16 with dsum 80.7 us = 6.66
// TB/s, 0.98 of a copy's rate; 5003 x 4111 from 8 bits with dsum 38.7 us, bound by its 36
// instructions an element (57 % of the issue slots).
constexpr int kRmsRing = 8;   // most rows in flight

struct RmsRingArgs {
    RmsBwdArgs a;
    int stages;
    uint32_t dy_span, x_span, ds_span;   // bytes of a row's place: dy, x or its codes, dsum
    uint32_t gamma_span;                 // bytes in front of the ring that hold gamma (or 0)
};

// A thread's columns of a row's copy.  ALIGNED: every row starts on a 16-byte boundary and is a
// multiple of 8 columns long; thread t has columns 8 (t + k threads) .. + 7, k < 2.  Otherwise
// columns 32 apart, as in the forward; the copy of a row starts `off` bytes after the boundary.
template <typename T, bool ALIGNED>
struct RingColumns;
template <typename T>
struct RingColumns<T, true> {
    int col[2], cols;
    RawVec<T, 8> raw[2];

    __device__ __forceinline__ explicit RingColumns(int cols_) : cols(cols_) {
        col[0] = 8 * threadIdx.x, col[1] = 8 * (threadIdx.x + blockDim.x);
    }
    __device__ __forceinline__ void load(const uint8_t *place, uint32_t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) raw[k].load(reinterpret_cast<const T *>(place), col[k], cols);
    }
    __device__ __forceinline__ void get(uint64_t (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint64_t x[4];
            raw[k].get(nullptr, 0, 0, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * k + i] = x[i];
        }
    }
    __device__ __forceinline__ void param(const void *p, int type, uint64_t (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint64_t x[4];
            load_param(p, type, col[k], cols, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * k + i] = x[i];
        }
    }
    uint32_t scale[2];
    __device__ __forceinline__ void fetch_scales(const BlockView &q, int64_t row) {
#pragma unroll
        for (int k = 0; k < 2; ++k) scale[k] = col[k] < cols ? fetch_scale(q, row, col[k] >> 7) : 0u;
    }
    float sc[2];
    __device__ __forceinline__ void take_scales(const BlockView &q) {
#pragma unroll
        for (int k = 0; k < 2; ++k) sc[k] = fetched_scale(q, scale[k]);
    }
    __device__ __forceinline__ void codes(const uint8_t *place, int fmt, uint64_t (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint2 w = make_uint2(0, 0);
            if (col[k] < cols) w = *reinterpret_cast<const uint2 *>(place + col[k]);
            uint64_t x[4];
            codes8_times(w, fmt, sc[k], 8, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * k + i] = x[i];
        }
    }
    __device__ __forceinline__ void store(T *row, const uint64_t (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint64_t x[4] = {v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
            RawVec<T, 8>::store(row, col[k], cols, x);
        }
    }
    __device__ __forceinline__ void store_sums(float *part, const uint64_t (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (col[k] >= cols) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<ulonglong2 *>(part + col[k] + 4 * i) =
                    make_ulonglong2(v[4 * k + 2 * i], v[4 * k + 2 * i + 1]);
        }
    }
};
template <typename T>
struct RingColumns<T, false> {
    int c, left;
    bool full;
    uint32_t raw[kSpread];

    __device__ __forceinline__ explicit RingColumns(int cols) {
        const int lane = threadIdx.x & 31;
        c = kSpread * (threadIdx.x & ~31) + lane;
        left = cols - c;
        full = left - 32 * (kSpread - 1) > 31 - lane;   // of the whole warp
    }
    __device__ __forceinline__ void load(const uint8_t *place, uint32_t off) {
        load_spread(reinterpret_cast<const T *>(place + off) + c, left, full, raw);
    }
    uint32_t scale;   // lane b: of the warp's block b
    __device__ __forceinline__ void fetch_scales(const BlockView &q, int64_t row) {
        const int lane = threadIdx.x & 31, block = ((c - lane) >> 7) + (lane & 3);
        scale = 128 * block < c - lane + left + lane ? fetch_scale(q, row, block) : 0u;
    }
    float sc;
    __device__ __forceinline__ void take_scales(const BlockView &q) { sc = fetched_scale(q, scale); }
    __device__ __forceinline__ void codes(const uint8_t *place, int fmt, float (&v)[kSpread]) const {
        uint32_t w[kSpread];
        if (full) {
#pragma unroll
            for (int j = 0; j < kSpread; ++j) w[j] = place[c + 32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < kSpread; ++j) w[j] = 32 * j < left ? place[c + 32 * j] : 0u;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float f[4];
            decode4(__byte_perm(__byte_perm(w[4 * b], w[4 * b + 1], 0x0040),
                                __byte_perm(w[4 * b + 2], w[4 * b + 3], 0x0040), 0x5410),
                    fmt, f);
            const float s = __shfl_sync(0xFFFFFFFFu, sc, b);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * b + k] = __fmul_rn(f[k], s);
        }
    }
};

// Two CTAs of 288 threads leave 96 registers each: gamma waits in shared memory, where the
// columns are single ones (5003 x 4111 from 8 bits 38.8 us; with gamma in registers and packed
// arithmetic 46.0, with packed arithmetic 43.3).
template <int THREADS, bool ALIGNED>
constexpr bool kGammaShared = THREADS == kRingHalf && !ALIGNED;

template <typename T, bool SAVED, int THREADS, int CTAS, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, CTAS) rms_bwd_ring_kernel(const RmsRingArgs r) {
    constexpr int kSize = static_cast<int>(sizeof(T));
    const RmsBwdArgs &a = r.a;
    extern __shared__ __align__(128) uint8_t ring_raw[];
    uint8_t *const ring = ring_raw + r.gamma_span;
    __shared__ __align__(16) uint64_t buf[2][16];
    __shared__ uint64_t bars[kRmsRing];
    __shared__ int gave_up;
    const uint32_t bar0 = smem_u32(bars), stage_bytes = r.dy_span + r.x_span + r.ds_span;
    if (threadIdx.x == 0) {
        for (int s = 0; s < r.stages; ++s) mbar_init(bar0 + 8 * s, 1);
        gave_up = 0;
        fence_mbar_init();
    }
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const uint8_t *dy0 = static_cast<const uint8_t *>(a.dy), *x0 = static_cast<const uint8_t *>(a.x);
    const uint8_t *ds0 = static_cast<const uint8_t *>(a.dsum);
    const int cols = static_cast<int>(a.cols);
    auto start_of = [](const uint8_t *p, int64_t row, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p + row * ld * kSize);
    };
    auto issue = [&](int64_t row, int s) {
        const uint32_t bar = bar0 + 8 * s, to = smem_u32(ring) + s * stage_bytes;
        const auto span = [cols](uintptr_t p, int size) {
            return (static_cast<uint32_t>(p & 15) + cols * size + 15) & ~15u;
        };
        const uintptr_t d = start_of(dy0, row, a.lddy);
        const uintptr_t x = SAVED ? reinterpret_cast<uintptr_t>(a.x8.codes + row * a.x8.ld) : start_of(x0, row, a.ldx);
        const uintptr_t e = start_of(ds0, row, a.ldds);
        const uint32_t dn = span(d, kSize), xn = span(x, SAVED ? 1 : kSize);
        const uint32_t en = ds0 != nullptr ? span(e, kSize) : 0u;
        mbar_arrive_expect_tx(bar, dn + xn + en);
        bulk_load_1d(to, reinterpret_cast<const void *>(d & ~uintptr_t(15)), dn, bar);
        bulk_load_1d(to + r.dy_span, reinterpret_cast<const void *>(x & ~uintptr_t(15)), xn, bar);
        if (en != 0)
            bulk_load_1d(to + r.dy_span + r.x_span, reinterpret_cast<const void *>(e & ~uintptr_t(15)), en, bar);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < r.stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < a.rows)
                issue(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
    const float ninv_n = -__fdiv_rn(1.0f, static_cast<float>(a.cols));
    using Columns = RingColumns<T, ALIGNED>;
    Columns own(cols);
    uint64_t dg[8] = {}, g[8];                       // packed, or
    float own_dg[kSpread] = {}, own_g[kSpread];      // one by one
    float *gamma = reinterpret_cast<float *>(ring_raw);
    if constexpr (ALIGNED) {
        own.param(a.gamma, a.wtype, g);
    } else {
        load_param_spread(a.gamma, a.wtype, own.c, own.left, own_g);
        if constexpr (kGammaShared<THREADS, ALIGNED>)
            store_spread(gamma + own.c, own.left, own.full, own_g);   // read again by its writer alone
    }
    // what does not go through the ring is fetched a row ahead
    float rs_next = 0.0f;
    auto fetch = [&](int64_t row) {
        rs_next = a.rstd[row];
        if constexpr (SAVED) own.fetch_scales(a.x8, row);
    };
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    int s = 0, flip = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const float rs = rs_next;
        const uint64_t rs2 = splat_f32x2(rs);
        if constexpr (SAVED) own.take_scales(a.x8);
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        if (!mbar_wait(bar0 + 8 * s, phase, &gave_up)) {
            // goes on with what is there, so that every thread still meets every barrier
            atomicOr(&g_rms_error_flags, kErrWaitTimeout);
            *static_cast<volatile int *>(&gave_up) = 1;
        }
        const uint8_t *stage = ring + s * stage_bytes;
        if constexpr (!ALIGNED) {
            // one by one: single columns come as single values, which packed arithmetic would have
            // to pair first
            float dy[kSpread], x[kSpread], sum = 0.0f;
            own.load(stage, static_cast<uint32_t>(start_of(dy0, row, a.lddy) & 15));
#pragma unroll
            for (int j = 0; j < kSpread; ++j) dy[j] = value_of<T>(own.raw[j]);
            if constexpr (SAVED) {
                own.codes(stage + r.dy_span, a.x8.fmt, x);
            } else {
                own.load(stage + r.dy_span, static_cast<uint32_t>(start_of(x0, row, a.ldx) & 15));
#pragma unroll
                for (int j = 0; j < kSpread; ++j) x[j] = value_of<T>(own.raw[j]);
            }
            uint32_t g_raw[kSpread];
            if constexpr (kGammaShared<THREADS, ALIGNED>) load_spread(gamma + own.c, own.left, own.full, g_raw);
#pragma unroll
            for (int j = 0; j < kSpread; ++j) {
                float gj;
                if constexpr (kGammaShared<THREADS, ALIGNED>) gj = __uint_as_float(g_raw[j]);
                else gj = own_g[j];
                x[j] = __fmul_rn(x[j], rs);
                own_dg[j] = __fmaf_rn(dy[j], x[j], own_dg[j]);
                dy[j] = __fmul_rn(dy[j], gj);
                sum = __fmaf_rn(dy[j], x[j], sum);
            }
            if (ds0 != nullptr)
                own.load(stage + r.dy_span + r.x_span, static_cast<uint32_t>(start_of(ds0, row, a.ldds) & 15));
            const float total = team_sum<false>(sum, buf[flip]);
            if (threadIdx.x == 0 && row + static_cast<int64_t>(r.stages) * gridDim.x < a.rows && !gave_up)
                issue(row + static_cast<int64_t>(r.stages) * gridDim.x, s);
            const float nm = __fmul_rn(total, ninv_n);
#pragma unroll
            for (int j = 0; j < kSpread; ++j)
                dy[j] = __fmaf_rn(__fmaf_rn(x[j], nm, dy[j]), rs, ds0 != nullptr ? value_of<T>(own.raw[j]) : 0.0f);
            store_spread(static_cast<T *>(a.dx) + row * a.lddx + own.c, own.left, own.full, dy);
        } else {
        uint64_t dy[8], x[8], sum = 0;
        own.load(stage, static_cast<uint32_t>(start_of(dy0, row, a.lddy) & 15));
        own.get(dy);
        if constexpr (SAVED) {
            own.codes(stage + r.dy_span, a.x8.fmt, x);
        } else {
            own.load(stage + r.dy_span, static_cast<uint32_t>(start_of(x0, row, a.ldx) & 15));
            own.get(x);
        }
        if (ds0 != nullptr)
            own.load(stage + r.dy_span + r.x_span, static_cast<uint32_t>(start_of(ds0, row, a.ldds) & 15));
        rms_bwd_accumulate(rs2, g, dy, x, dg, sum);
        const float total = team_sum<false>(sum2(sum), buf[flip]);
        if (threadIdx.x == 0 && row + static_cast<int64_t>(r.stages) * gridDim.x < a.rows && !gave_up)
            issue(row + static_cast<int64_t>(r.stages) * gridDim.x, s);
        uint64_t ds[8] = {};
        if (ds0 != nullptr) own.get(ds);
        rms_bwd_finish(rs2, splat_f32x2(__fmul_rn(total, ninv_n)), x, ds, dy);
        own.store(static_cast<T *>(a.dx) + row * a.lddx, dy);
        }
        if (++s == r.stages) s = 0, phase ^= 1u;
    }
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * up8(a.cols);
    if constexpr (ALIGNED)
        own.store_sums(part, dg);
    else
        store_spread(part + own.c, own.left, own.full, own_dg);
    if (gave_up && threadIdx.x == 0)   // copies still in flight land (bounded) before the CTA exits
        for (int i = 0; i < r.stages; ++i) {
            mbar_wait(bar0 + 8 * s, phase, nullptr, 100000000ull);
            if (++s == r.stages) s = 0, phase ^= 1u;
        }
}

// Aligned rows of 8193 .. 16384 columns: as above, but a thread has 32 columns, whose sums and
// gamma fill its registers, so that it takes dy and x from the ring twice, for the row's sum and
// for dx, and the row's place is free at its end alone.  (4096 x 12288
// bf16 with dsum 56.8 us, in two passes over HBM 117.2; fp32, with a place for one row alone, 137
// and 190.)
template <typename T, bool SAVED>
__global__ void __launch_bounds__(512, 1) rms_bwd_long_kernel(const RmsRingArgs r) {
    constexpr int N = 4;   // times 8 columns
    const RmsBwdArgs &a = r.a;
    extern __shared__ __align__(128) uint8_t ring_raw[];
    __shared__ __align__(16) uint64_t buf[2][16];
    __shared__ uint64_t bars[kRmsRing];
    __shared__ int gave_up;
    const uint32_t bar0 = smem_u32(bars);
    auto issue = [&](int64_t row, int s) {
        const uint32_t bar = bar0 + 8 * s, to = smem_u32(ring_raw) + s * (r.dy_span + r.x_span + r.ds_span);
        const uint32_t n = static_cast<uint32_t>(a.cols * sizeof(T));
        const uint32_t xn = SAVED ? static_cast<uint32_t>(a.cols + 15) & ~15u : n;
        mbar_arrive_expect_tx(bar, n + xn + (a.dsum != nullptr ? n : 0));
        bulk_load_1d(to, static_cast<const T *>(a.dy) + row * a.lddy, n, bar);
        if constexpr (SAVED)
            bulk_load_1d(to + r.dy_span, a.x8.codes + row * a.x8.ld, xn, bar);
        else
            bulk_load_1d(to + r.dy_span, static_cast<const T *>(a.x) + row * a.ldx, xn, bar);
        if (a.dsum != nullptr)
            bulk_load_1d(to + r.dy_span + r.x_span, static_cast<const T *>(a.dsum) + row * a.ldds, n, bar);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < r.stages; ++s) mbar_init(bar0 + 8 * s, 1);
        gave_up = 0;
        fence_mbar_init();
    }
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0)
        for (int s = 0; s < r.stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < a.rows)
                issue(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
    const float ninv_n = -__fdiv_rn(1.0f, static_cast<float>(a.cols));
    const int cols = static_cast<int>(a.cols);
    auto col = [&](int k) { return 8 * static_cast<int>(threadIdx.x + k * blockDim.x); };
    uint64_t dg[N][4] = {}, g[N][4];
#pragma unroll
    for (int k = 0; k < N; ++k) load_param(a.gamma, a.wtype, col(k), cols, g[k]);
    // what does not go through the ring is fetched a row ahead
    float rs_next = 0.0f;
    uint32_t scale[SAVED ? N : 1];
    auto fetch = [&](int64_t row) {
        rs_next = a.rstd[row];
        if constexpr (SAVED) {
#pragma unroll
            for (int k = 0; k < N; ++k) scale[k] = col(k) < cols ? fetch_scale(a.x8, row, col(k) >> 7) : 0u;
        }
    };
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    int s = 0, flip = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const uint64_t rs2 = splat_f32x2(rs_next);
        float sc[SAVED ? N : 1];
        if constexpr (SAVED) {
#pragma unroll
            for (int k = 0; k < N; ++k) sc[k] = fetched_scale(a.x8, scale[k]);
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        if (!mbar_wait(bar0 + 8 * s, phase, &gave_up)) {
            // goes on with what is there, so that every thread still meets every barrier
            atomicOr(&g_rms_error_flags, kErrWaitTimeout);
            *static_cast<volatile int *>(&gave_up) = 1;
        }
        const uint8_t *stage = ring_raw + s * (r.dy_span + r.x_span + r.ds_span);
        auto take = [&](const uint8_t *place, int k, uint64_t (&v)[4]) {
            RawVec<T, 8> raw;
            raw.load(reinterpret_cast<const T *>(place), col(k), cols);
            raw.get(nullptr, 0, 0, v);
        };
        auto take_x = [&](int k, uint64_t (&v)[4]) {
            if constexpr (SAVED) {
                uint2 w = make_uint2(0, 0);
                if (col(k) < cols) w = *reinterpret_cast<const uint2 *>(stage + r.dy_span + col(k));
                codes8_times(w, a.x8.fmt, sc[k], 8, v);
            } else {
                take(stage + r.dy_span, k, v);
            }
        };
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            uint64_t dy[4], x[4];
            take(stage, k, dy);
            take_x(k, x);
            rms_bwd_accumulate(rs2, g[k], dy, x, dg[k], sum);
        }
        const float total = team_sum<false>(sum2(sum), buf[flip]);
        const uint64_t nm2 = splat_f32x2(__fmul_rn(total, ninv_n));
#pragma unroll
        for (int k = 0; k < N; ++k) {
            uint64_t dy[4], x[4], ds[4] = {};
            take(stage, k, dy);
            take_x(k, x);
            if (a.dsum != nullptr) take(stage + r.dy_span + r.x_span, k, ds);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f32x2_mul(x[i], rs2), dy[i] = f32x2_mul(dy[i], g[k][i]);
            rms_bwd_finish(rs2, nm2, x, ds, dy);
            RawVec<T, 8>::store(static_cast<T *>(a.dx) + row * a.lddx, col(k), cols, dy);
        }
        __syncthreads();   // the place has been read
        if (threadIdx.x == 0 && row + static_cast<int64_t>(r.stages) * gridDim.x < a.rows && !gave_up)
            issue(row + static_cast<int64_t>(r.stages) * gridDim.x, s);
        if (++s == r.stages) s = 0, phase ^= 1u;
    }
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * up8(a.cols);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (col(k) < cols) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<ulonglong2 *>(part + col(k) + 4 * i) = make_ulonglong2(dg[k][2 * i], dg[k][2 * i + 1]);
        }
    if (gave_up && threadIdx.x == 0)   // copies still in flight land (bounded) before the CTA exits
        for (int i = 0; i < r.stages; ++i) {
            mbar_wait(bar0 + 8 * s, phase, nullptr, 100000000ull);
            if (++s == r.stages) s = 0, phase ^= 1u;
        }
}

// Rows of one warp: up to 256 columns, 8 per thread, which leaves registers for three CTAs an SM
// in 16 bits (65536 x 256 24.0 us; 16 columns per thread and two CTAs 45.4, the ring kernel
// 33.6).  Up to 512 columns the ring kernel, with CTAs of one warp, is ahead of 16 columns per
// thread here (65536 x 512 41.3 and 53.6 us).
constexpr int64_t kRmsNarrow = 256;
constexpr int kNarrowMost = 3;
template <typename T, int VEC>
constexpr int kNarrowCtas = sizeof(T) == 2 && VEC != 0 ? kNarrowMost : 2;   // more would spill

// Narrow rows (WARP) and wide ones.  Rows in turn; a thread keeps its columns and their sums
// over the CTA's rows.  Wide: bounded as for 512 threads, of which 256 start, so that two CTAs
// fit an SM; all but aligned 16-bit rows spill 208 to 596 bytes then (with dsum, as it is and
// bounded by 256: bf16 4000 x 20000 186.5 and 211 us, 4000 x 12001 239 and 190; fp32 4000 x 20000
// 340 and 309, 2000 x 20001 278 and 198).  WIDE: blockIdx.y, and blockIdx.z where there are more than 65535, is a
// slab of 8 VPT blockDim.x columns, and the rows' sums are already there.
template <typename T, bool SAVED, int VPT, bool WARP, int VEC>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512, WARP ? kNarrowCtas<T, VEC> : 1)
    rms_bwd_kernel(const RmsBwdArgs a) {
    using L = Lay<T, VEC>;
    constexpr int E = L::E, P = L::P;
    constexpr bool WIDE = !WARP;
    const Team<WARP> team;
    pdl_wait();
    pdl_trigger();
    const float ninv_n = -__fdiv_rn(1.0f, static_cast<float>(a.cols));
    const int64_t slab = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
    const int64_t base = WIDE ? slab * E * VPT * blockDim.x : 0;   // past the last column: nothing to do
    auto col = [&](int k) { return base + E * (team.id + k * team.size); };
    typename L::Raw rdy[VPT], rds[VPT];
    RmsRawX<T, SAVED, VEC> rx[VPT];
    float rs_next = 0.0f;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rdy[k].load(static_cast<const T *>(a.dy) + row * a.lddy, col(k), a.cols);
            rx[k].load(a, row, col(k));
            if (a.dsum != nullptr) rds[k].load(static_cast<const T *>(a.dsum) + row * a.ldds, col(k), a.cols);
        }
        rs_next = a.rstd[row];
    };
    if (team.row < a.rows) fetch(team.row);
    uint64_t dg[VPT][P] = {}, g[VPT][P];
#pragma unroll
    for (int k = 0; k < VPT; ++k) load_param(a.gamma, a.wtype, col(k), a.cols, g[k]);
    for (int64_t row = team.row; row < a.rows; row += team.step) {
        const uint64_t rs2 = splat_f32x2(rs_next);
        uint64_t dy[VPT][P], x[VPT][P], ds[VPT][P], s = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rdy[k].get(static_cast<const T *>(a.dy) + row * a.lddy, col(k), a.cols, dy[k]);
            rx[k].get(a, row, col(k), x[k]);
            if (a.dsum != nullptr) {
                rds[k].get(static_cast<const T *>(a.dsum) + row * a.ldds, col(k), a.cols, ds[k]);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) ds[k][i] = 0;
            }
        }
        if (row + team.step < a.rows) fetch(row + team.step);
#pragma unroll
        for (int k = 0; k < VPT; ++k) rms_bwd_accumulate(rs2, g[k], dy[k], x[k], dg[k], s);
        float total;
        if constexpr (WIDE) {
            total = a.row_sums[row];
        } else {
            total = sum2(s);
#pragma unroll
            for (int o = 16; o; o >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xFFFFFFFFu, total, o));
        }
        const uint64_t nm2 = splat_f32x2(__fmul_rn(total, ninv_n));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rms_bwd_finish(rs2, nm2, x[k], ds[k], dy[k]);
            L::store(static_cast<T *>(a.dx) + row * a.lddx, col(k), a.cols, dy[k]);
        }
    }
    if constexpr (WARP) {
        // the warps that had rows (the first one always) add theirs one after the other;
        // [column of the lane][lane], so that a warp's accesses meet no bank twice
        __shared__ float sums[VPT * E][32];
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w && team.row < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        float lo, hi;
                        f32x2_unpack(dg[k][i / 2], lo, hi);
                        float *p = &sums[k * E + i][lane];
                        *p = w ? __fadd_rn(*p, i & 1 ? hi : lo) : i & 1 ? hi : lo;
                    }
            }
            if (blockIdx.x * kWarps + w + 1 >= a.rows) break;   // no later warp had rows
            __syncthreads();
        }
        __syncthreads();
        float *part = a.part + static_cast<int64_t>(blockIdx.x) * up8(a.cols);
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x)
            part[c] = sums[static_cast<int>(c / (32 * E)) * E + static_cast<int>(c % E)][static_cast<int>(c / E) & 31];
    } else {
        rms_store_part(a, col, dg);
    }
}

// dgamma from the CTAs' sums [parts][padded]: 32 columns per CTA, 32 threads down the
// parts for each, then a fixed tree.
__global__ void __launch_bounds__(1024) rms_bwd_reduce_kernel(const float *__restrict__ part, int parts,
                                                              int64_t cols, float *__restrict__ dgamma) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t padded = up8(cols), c = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    float s = 0.0f;
    if (c < cols) {
        for (int p = ty; p < parts; p += 32 * 5) {   // five reads on their way together
            float v[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) v[i] = p + 32 * i < parts ? part[(p + 32 * i) * padded + c] : 0.0f;
#pragma unroll
            for (int i = 0; i < 5; ++i) s = __fadd_rn(s, v[i]);
        }
    }
    red[ty][tx] = s;
    __syncthreads();
    s = red[tx][ty];
#pragma unroll
    for (int o = 16; o; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + ty;
    if (tx == 0 && out < cols) dgamma[out] = s;
}

// --------------------------------------------------------------------- host --

// CTAs that the registers allow at once: 96 of them per thread, or 128.  (A warp's fp32 rows
// take up to 180, and their grid is two waves: 16384 x 512 24.8 us, in one 23.7.)
template <int THREADS>
int64_t fwd_ctas_per_sm(unsigned threads) {
    return (THREADS == kFwdHalf ? 2 * kFwdHalf : 512) / threads;
}

template <typename T, int VPT, int THREADS, bool WARP, int VEC, bool RES>
cudaError_t rms_fwd_rows(const RmsFwdArgs &a, int sms, cudaStream_t st) {
    const unsigned threads = WARP ? 32 * kWarps : row_threads(a.cols, VPT * Lay<T, VEC>::E);
    const int64_t resident = static_cast<int64_t>(sms) * fwd_ctas_per_sm<THREADS>(threads);
    const unsigned grid = capped(WARP ? (a.rows + kWarps - 1) / kWarps : a.rows, resident);
    return launch_pdl(rms_fwd_kernel<T, VPT, THREADS, WARP, VEC, RES>, dim3(grid), dim3(threads), 0, st, a);
}

template <typename T, int THREADS, bool WARP, bool RES>
cudaError_t rms_fwd_spread(const RmsFwdArgs &a, int sms, cudaStream_t st) {
    const unsigned threads = WARP ? 32 * kWarps : row_threads(a.cols, kSpread);
    const int64_t resident = static_cast<int64_t>(sms) * fwd_ctas_per_sm<THREADS>(threads);
    const unsigned grid = capped(WARP ? (a.rows + kWarps - 1) / kWarps : a.rows, resident);
    return launch_pdl(rms_fwd_spread_kernel<T, THREADS, WARP, RES>, dim3(grid), dim3(threads), 0, st, a);
}

template <typename T, bool RES>
cudaError_t rms_fwd_typed(const RmsFwdArgs &a, bool vec, int sms, cudaStream_t st) {
    if (vec) {
        if (a.cols <= 512) return rms_fwd_rows<T, 1, 32 * kWarps, true, 16, RES>(a, sms, st);
        if (a.cols <= 4096) return rms_fwd_rows<T, 1, 256, false, 16, RES>(a, sms, st);
        if constexpr (sizeof(T) == 2)   // fp32 spills: 8192 x 4608 124.9 us, and 109.9 in one CTA
            if (a.cols <= 16 * kFwdHalf) return rms_fwd_rows<T, 1, kFwdHalf, false, 16, RES>(a, sms, st);
        if (a.cols <= 8192) return rms_fwd_rows<T, 1, 512, false, 16, RES>(a, sms, st);
        if (a.cols <= 16384) return rms_fwd_rows<T, 2, 512, false, 16, RES>(a, sms, st);
    } else {
        if (a.cols <= 512) return rms_fwd_spread<T, 32 * kWarps, true, RES>(a, sms, st);
        if (a.cols <= kSpread * kFwdHalf) return rms_fwd_spread<T, kFwdHalf, false, RES>(a, sms, st);
        if (a.cols <= 8192) return rms_fwd_spread<T, 512, false, RES>(a, sms, st);
        if (a.cols <= 16384) return rms_fwd_rows<T, 4, 512, false, 0, RES>(a, sms, st);
    }
    return launch_pdl(rms_fwd_wide_kernel<T, RES>, dim3(capped(a.rows, 4 * sms)), dim3(512), 0, st, a);
}

constexpr int64_t kRingBytes = 200 << 10;   // of an SM's shared memory
template <typename T, bool SAVED>
RmsRingArgs ring_args(const RmsBwdArgs &a) {
    RmsRingArgs r{a, 0, 0, 0, 0, 0};
    r.dy_span = static_cast<uint32_t>((a.cols * sizeof(T) + 15 + 127) / 128 * 128 + 128);
    r.x_span = SAVED ? static_cast<uint32_t>((a.cols + 127) / 128 * 128) : r.dy_span;
    r.ds_span = a.dsum != nullptr ? r.dy_span : 0;
    return r;
}

// As many rows in flight as the CTAs of an SM have shared memory for.
template <typename T, bool SAVED, int THREADS, int CTAS, bool ALIGNED>
cudaError_t rms_bwd_ring_sized(const RmsBwdArgs &a, int grid, unsigned threads, cudaStream_t st) {
    RmsRingArgs r = ring_args<T, SAVED>(a);
    const int64_t place = r.dy_span + r.x_span + r.ds_span;
    if (kGammaShared<THREADS, ALIGNED>) r.gamma_span = static_cast<uint32_t>((a.cols * 4 + 127) / 128 * 128);
    const int64_t fit = (kRingBytes / ring_ctas_per_sm(threads) - r.gamma_span) / place;
    r.stages = static_cast<int>(fit < kRmsRing ? fit : kRmsRing);
    static SmemLimit limit;
    const cudaError_t err = limit.allow(rms_bwd_ring_kernel<T, SAVED, THREADS, CTAS, ALIGNED>, kRingBytes);
    if (err != cudaSuccess) return err;
    return launch_pdl(rms_bwd_ring_kernel<T, SAVED, THREADS, CTAS, ALIGNED>, dim3(grid), dim3(threads),
                      static_cast<size_t>(r.gamma_span + r.stages * place), st, r);
}

template <typename T, bool SAVED, bool ALIGNED>
cudaError_t rms_bwd_ring(const RmsBwdArgs &a, int grid, cudaStream_t st) {
    const unsigned threads = row_threads(a.cols, 16);
    if (threads > kRingHalf) return rms_bwd_ring_sized<T, SAVED, 512, 1, ALIGNED>(a, grid, threads, st);
    if (threads > 256) return rms_bwd_ring_sized<T, SAVED, kRingHalf, 2, ALIGNED>(a, grid, threads, st);
    return rms_bwd_ring_sized<T, SAVED, 256, 2, ALIGNED>(a, grid, threads, st);
}

constexpr int64_t kRmsLong = 16384;   // columns of 512 threads, 32 each
static_assert(3 * (kRmsLong * 4 + 15 + 127 + 128) <= kRingBytes, "a place for a row of any type");
template <typename T, bool SAVED>
cudaError_t rms_bwd_long(const RmsBwdArgs &a, int grid, cudaStream_t st) {
    RmsRingArgs r = ring_args<T, SAVED>(a);
    const int64_t fit = kRingBytes / (r.dy_span + r.x_span + r.ds_span);
    r.stages = static_cast<int>(fit < kRmsRing ? fit : kRmsRing);
    static SmemLimit limit;
    const cudaError_t err = limit.allow(rms_bwd_long_kernel<T, SAVED>, kRingBytes);
    if (err != cudaSuccess) return err;
    return launch_pdl(rms_bwd_long_kernel<T, SAVED>, dim3(grid), dim3(row_threads(a.cols, 32)),
                      static_cast<size_t>(r.stages * (r.dy_span + r.x_span + r.ds_span)), st, r);
}

template <typename T, bool SAVED, int VEC>
cudaError_t rms_bwd_typed(RmsBwdArgs a, float *dgamma, void *ws, int sms, cudaStream_t st) {
    const int g = static_cast<int>(bwd_ctas(a.rows, a.cols, sms, kRmsNarrow, kNarrowCtas<T, VEC>));
    a.part = static_cast<float *>(ws);
    cudaError_t e;
    if (a.cols <= kRmsNarrow) {
        e = launch_pdl(rms_bwd_kernel<T, SAVED, 1, true, VEC>, dim3(g), dim3(32 * kWarps), 0, st, a);
    } else if (a.cols <= kBwdWide) {
        e = rms_bwd_ring<T, SAVED, VEC != 0>(a, g, st);
    } else if (VEC != 0 && a.cols <= kRmsLong) {
        e = rms_bwd_long<T, SAVED>(a, g, st);
    } else {
        a.row_sums = a.part + static_cast<int64_t>(g) * up8(a.cols);
        e = launch_pdl(rms_bwd_sums_kernel<T, SAVED>, dim3(capped(a.rows, 4 * sms)), dim3(512), 0, st, a);
        if (e != cudaSuccess) return e;
        const unsigned slabs = static_cast<unsigned>((a.cols + kBwdSlab - 1) / kBwdSlab);
        const unsigned z = (slabs + 65534) / 65535;
        e = launch_pdl(rms_bwd_kernel<T, SAVED, 2, false, VEC>, dim3(g, (slabs + z - 1) / z, z), dim3(256),
                       0, st, a);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(rms_bwd_reduce_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32)), dim3(1024), 0,
                      st, static_cast<const float *>(a.part), g, a.cols, dgamma);
}

}  // namespace

cudaError_t launch_rms_fwd(const MatView &x, const MatView &residual, const void *gamma, int wtype,
                           float eps, const MatView &sum, const MatView &y, const BlockView &y8,
                           const BlockView &x8, float *rstd, int sm_count, cudaStream_t st) {
    if (x.rows == 0) return cudaSuccess;
    const RmsFwdArgs a{x.data, residual.data, x.rows, x.cols, x.ld, residual.ld, gamma, wtype, eps,
                       sum.data, sum.ld, y.data, y.ld, y8, x8, rstd};
    const bool vec = x.cols % 16 == 0 && aligned_rows(x.data, x.ld, x.type) &&
                     aligned_rows(residual.data, residual.ld, x.type) &&
                     aligned_rows(sum.data, sum.ld, x.type) && aligned_rows(y.data, y.ld, x.type);
#define FP8K_RMS_FWD(T)                                        \
    (residual.data != nullptr ? rms_fwd_typed<T, true>(a, vec, sm_count, st) \
                              : rms_fwd_typed<T, false>(a, vec, sm_count, st))
    if (x.type == kTypeF32) return FP8K_RMS_FWD(float);
    if (x.type == kTypeBF16) return FP8K_RMS_FWD(__nv_bfloat16);
    return FP8K_RMS_FWD(__half);
#undef FP8K_RMS_FWD
}

int64_t rms_bwd_workspace(int64_t rows, int64_t cols) {
    return bwd_ctas(rows, cols, kBwdSms, kRmsNarrow, kNarrowMost) * up8(cols) * 4 + (cols > kBwdWide ? rows * 4 : 0);
}

cudaError_t launch_rms_bwd(const MatView &dy, const MatView &x, const BlockView &x8, const void *gamma,
                           int wtype, const float *rstd, const MatView &dsum, const MatView &dx,
                           float *dgamma, void *ws, int sm_count, cudaStream_t st) {
    if (dy.rows == 0) return cudaMemsetAsync(dgamma, 0, dy.cols * 4, st);
    const RmsBwdArgs a{dy.data, x.data, dsum.data, dy.rows, dy.cols, dy.ld, x.ld, dsum.ld, dx.ld, x8,
                       gamma, wtype, rstd, dx.data, nullptr, nullptr};
    const bool saved = x8.codes != nullptr;
    const bool vec = dy.cols % 8 == 0 && aligned_rows(dy.data, dy.ld, dy.type) &&
                     aligned_rows(x.data, x.ld, dy.type) && aligned_rows(dsum.data, dsum.ld, dy.type) &&
                     aligned_rows(dx.data, dx.ld, dy.type);
#define FP8K_RMS_BWD(T)                                                              \
    (saved ? vec ? rms_bwd_typed<T, true, 8>(a, dgamma, ws, sm_count, st)              \
                 : rms_bwd_typed<T, true, 0>(a, dgamma, ws, sm_count, st)              \
     : vec ? rms_bwd_typed<T, false, 8>(a, dgamma, ws, sm_count, st)                   \
           : rms_bwd_typed<T, false, 0>(a, dgamma, ws, sm_count, st))
    if (dy.type == kTypeF32) return FP8K_RMS_BWD(float);
    if (dy.type == kTypeBF16) return FP8K_RMS_BWD(__nv_bfloat16);
    return FP8K_RMS_BWD(__half);
#undef FP8K_RMS_BWD
}

cudaError_t read_and_clear_rms_error_flag(unsigned *flags) {
    return take_error_flags(&g_rms_error_flags, flags);
}

}  // namespace fp8k
