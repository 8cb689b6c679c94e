// layernorm.cu -- LayerNorm forward and backward, with the input kept in 8 bits.
//
// Forward, per row of x [rows][cols] in fp32:
//   mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
//   y = ((x - mean) * rstd) * gamma + beta
// Backward, with xhat = (x - mean) * rstd and u = dy * gamma:
//   dx = rstd * (u - sum(u) / cols - xhat * sum(u * xhat) / cols)
//   dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
//
// Both are bound by HBM: each value is read and written once, and a row stays
// in its CTA's registers between the sums and the use of the sums.
#include <cstdint>

#include "error_flag.h"
#include "norm_rows.cuh"
#include "once_per_device.h"

namespace fp8k {

namespace {

__device__ unsigned g_ln_error_flags = 0;

struct LnFwdArgs {
    const void *x;
    int64_t rows, cols, ldx;
    const void *gamma, *beta;
    int wtype;
    float eps;
    void *y;
    int64_t ldy;
    BlockView y8, x8;   // codes null: not wanted
    float *mean, *rstd;
};

// The part of the forward that follows the statistics, for 2 P columns: `at` columns
// past the writers' first, `left` columns before the row's end.
template <typename T, int P>
__device__ __forceinline__ void ln_finish(const LnFwdArgs &a, T *yr, const RowWriter &wy,
                                          const RowWriter &wx, int64_t c, int at, int left,
                                          uint64_t nmu2, uint64_t rs2, const uint64_t (&g)[P],
                                          const uint64_t (&b)[P], const uint64_t (&x)[P]) {
    if (a.x8.codes != nullptr) wx.put(a.x8, x, at, left);
    if (a.y == nullptr && a.y8.codes == nullptr) return;
    uint64_t y[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        y[i] = f32x2_fma(f32x2_mul(f32x2_add(x[i], nmu2), rs2), g[i], b[i]);
    if (a.y != nullptr) Lay<T, P == 8 ? 16 : 0>::store(yr, c, a.cols, y);
    if (a.y8.codes != nullptr) wy.put(a.y8, y, at, left);
}

// sum of (x - mean)^2; columns past the row do not count
template <int P>
__device__ __forceinline__ uint64_t deviations(const uint64_t (&x)[P], uint64_t nmu2, int left,
                                               uint64_t s) {
    if (left >= 2 * P) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint64_t d = f32x2_add(x[i], nmu2);
            s = f32x2_fma(d, d, s);
        }
    } else if (left > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            f32x2_unpack(f32x2_add(x[i], nmu2), lo, hi);
            const uint64_t d = f32x2_pack(2 * i < left ? lo : 0.0f, 2 * i + 1 < left ? hi : 0.0f);
            s = f32x2_fma(d, d, s);
        }
    }
    return s;
}

// The rows after those in work are already being loaded, into registers.
// A team works on R rows side by side, one step apart: their sums share the exchanges and
// the barriers, and one row's arithmetic fills the other's waits (8192 x 4096, y alone:
// 27.7 us with two, 31.0 with one; y and x in 8 bits: 37.9 us, of which the blocks' maxima
// and codes are about half).  Rows that have to be shifted into place leave no
// registers for a second.
template <typename T, int VPT, bool WARP, int VEC>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512) ln_fwd_kernel(const LnFwdArgs a) {
    using L = Lay<T, VEC>;
    constexpr int E = L::E, P = L::P, R = VEC && VPT * P <= 8 ? 2 : 1;
    __shared__ __align__(16) uint64_t buf[2][16];
    const Team<WARP> team;
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols), inv_n = __fdiv_rn(1.0f, n);
    const int left0 = static_cast<int>(a.cols) - E * team.id;
    typename L::Raw raw[R][VPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (row + j * team.step < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    raw[j][k].load(static_cast<const T *>(a.x) + (row + j * team.step) * a.ldx,
                                   E * (team.id + k * team.size), a.cols);
            }
    };
    if (team.row < a.rows) fetch(team.row);
    // gamma and beta stay in registers where there is room for them
    constexpr bool kKeep = VPT * P <= 8;
    constexpr int kKept = kKeep ? VPT : 1;
    uint64_t g[kKept][P], b[kKept][P];
    auto params = [&](int k, int slot) {
        load_param(a.gamma, a.wtype, E * (team.id + k * team.size), a.cols, g[slot]);
        load_param(a.beta, a.wtype, E * (team.id + k * team.size), a.cols, b[slot]);
    };
    if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) params(k, k);
    }
    for (int64_t row = team.row; row < a.rows; row += R * team.step) {
        uint64_t x[R][VPT][P];
        float s[2] = {0.0f, 0.0f}, mu[2], rs[2];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            uint64_t s2 = 0;
            if (row + j * team.step < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    raw[j][k].get(static_cast<const T *>(a.x) + (row + j * team.step) * a.ldx,
                                  E * (team.id + k * team.size), a.cols, x[j][k]);
#pragma unroll
                    for (int i = 0; i < P; ++i) s2 = f32x2_add(s2, x[j][k][i]);
                }
            }
            s[j] = sum2(s2);
        }
        if (row + R * team.step < a.rows) fetch(row + R * team.step);
        const float2 sums = team_sum2<WARP>(s[0], s[1], buf[0]);
        mu[0] = quotient(sums.x, n, inv_n), mu[1] = quotient(sums.y, n, inv_n);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            uint64_t s2 = 0;
            if (row + j * team.step < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    s2 = deviations(x[j][k], splat_f32x2(-mu[j]), left0 - E * k * team.size, s2);
            }
            s[j] = sum2(s2);
        }
        const float2 squares = team_sum2<WARP>(s[0], s[1], buf[1]);
        rs[0] = __frsqrt_rn(__fadd_rn(quotient(squares.x, n, inv_n), a.eps));
        rs[1] = __frsqrt_rn(__fadd_rn(quotient(squares.y, n, inv_n), a.eps));
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t at_row = row + j * team.step;
            if (at_row >= a.rows) break;
            if (team.id == 0) {
                a.mean[at_row] = mu[j];
                a.rstd[at_row] = rs[j];
            }
            RowWriter wx, wy;
            wx.start(a.x8, at_row, E * team.id);
            wy.start(a.y8, at_row, E * team.id);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if constexpr (!kKeep) params(k, 0);
                const int at = E * k * team.size;
                ln_finish<T, P>(a, static_cast<T *>(a.y) + at_row * a.ldy, wy, wx, E * team.id + at, at,
                                left0 - at, splat_f32x2(-mu[j]), splat_f32x2(rs[j]), g[k % kKept],
                                b[k % kKept], x[j][k]);
            }
        }
    }
}

// Rows too long for a CTA's registers: x is read again for each use.
template <typename T>
__global__ void __launch_bounds__(512) ln_fwd_wide_kernel(const LnFwdArgs a) {
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
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *xr = static_cast<const T *>(a.x) + row * a.ldx;
        RawRow8<T> raw;
        uint64_t x[4], s2 = 0;
        for (int64_t w = warp0; w < a.cols; w += 8 * 512) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            raw.load(xr, c, a.cols);
            raw.get(xr, c, a.cols, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = f32x2_add(s2, x[i]);
        }
        const float mu = __fdiv_rn(team_sum<false>(sum2(s2), buf[0]), n);
        const uint64_t nmu2 = splat_f32x2(-mu);
        s2 = 0;
        for (int64_t w = warp0; w < a.cols; w += 8 * 512) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            raw.load(xr, c, a.cols);
            raw.get(xr, c, a.cols, x);
            s2 = deviations(x, nmu2, static_cast<int>(a.cols - c), s2);
        }
        const float var = __fdiv_rn(team_sum<false>(sum2(s2), buf[1]), n);
        const float rs = __frsqrt_rn(__fadd_rn(var, a.eps));
        if (threadIdx.x == 0) {
            a.mean[row] = mu;
            a.rstd[row] = rs;
        }
        for (int64_t w = warp0; w < a.cols; w += 8 * 512) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            uint64_t g[4], b[4];
            load_param(a.gamma, a.wtype, c, a.cols, g);
            load_param(a.beta, a.wtype, c, a.cols, b);
            raw.load(xr, c, a.cols);
            raw.get(xr, c, a.cols, x);
            ln_finish<T, 4>(a, static_cast<T *>(a.y) + row * a.ldy, wy, wx, c, static_cast<int>(w - warp0),
                         static_cast<int>(a.cols - c), nmu2, splat_f32x2(rs), g, b, x);
        }
        wx.move(a.x8, gridDim.x);
        wy.move(a.y8, gridDim.x);
    }
}

struct LnBwdArgs {
    const void *dy, *x;
    int64_t rows, cols, lddy, ldx, lddx;
    BlockView x8;
    const void *gamma;
    int wtype;
    const float *mean, *rstd;
    void *dx;
    float *part;       // [gridDim.x][2][up8(cols)]: a CTA's sums of dy * xhat and dy
    float2 *row_sums;  // wide rows: [rows] sums of u and u * xhat
};

// v + plus
template <int P>
__device__ __forceinline__ void add_all(uint64_t plus, uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = f32x2_add(v[i], plus);
}

// Columns of x on their way, as they are or codes with their block's scale; get: x - mean.
template <typename T, bool SAVED, int VEC>
struct RawX {
    typename Lay<T, VEC>::Raw raw;
    __device__ __forceinline__ void load(const LnBwdArgs &a, int64_t row, int64_t c) {
        raw.load(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols);
    }
    __device__ __forceinline__ void get(const LnBwdArgs &a, int64_t row, int64_t c, uint64_t nmu2,
                                        uint64_t (&v)[Lay<T, VEC>::P]) const {
        raw.get(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, v);
        add_all(nmu2, v);
    }
};
template <typename T, int VEC>
struct RawX<T, true, VEC> {
    static constexpr int P = Lay<T, VEC>::P;
    static_assert(P == 4, "8 codes");
    uint32_t w[P / 2], scale;
    __device__ __forceinline__ void load(const LnBwdArgs &a, int64_t row, int64_t c) {
        const uint8_t *p = a.x8.codes + row * a.x8.ld + c;
        if (c < a.cols) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
            scale = fetch_scale(a.x8, row, c >> 7);
        } else {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) w[i] = 0;
            scale = 0;
        }
    }
    __device__ __forceinline__ void get(const LnBwdArgs &a, int64_t, int64_t c, uint64_t nmu2,
                                        uint64_t (&v)[P]) const {
        codes8(make_uint2(w[0], w[1]), a.x8.fmt, fetched_scale(a.x8, scale), nmu2,
               VEC ? 8 : static_cast<int>(a.cols - c), v);
    }
};

// xhat in place of x - mean, and u in place of dy; their sums for the row, and the column
// sums
template <int P>
__device__ __forceinline__ void ln_bwd_accumulate(uint64_t rs2, const uint64_t (&g)[P],
                                                  uint64_t (&dy)[P], uint64_t (&x)[P],
                                                  uint64_t (&dg)[P], uint64_t (&db)[P], uint64_t &s1,
                                                  uint64_t &s2) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        x[i] = f32x2_mul(x[i], rs2);
        dg[i] = f32x2_fma(dy[i], x[i], dg[i]);
        db[i] = f32x2_add(db[i], dy[i]);
        dy[i] = f32x2_mul(dy[i], g[i]);
        s1 = f32x2_add(s1, dy[i]);
        s2 = f32x2_fma(dy[i], x[i], s2);
    }
}

// Wide rows: the two row sums, in a pass of their own.
template <typename T, bool SAVED>
__global__ void __launch_bounds__(512) ln_bwd_sums_kernel(const LnBwdArgs a) {
    __shared__ __align__(16) uint64_t buf[2][16];
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const uint64_t nmu2 = splat_f32x2(-a.mean[row]), rs2 = splat_f32x2(a.rstd[row]);
        uint64_t s1 = 0, s2 = 0;
        for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * 512) {
            const T *dyr = static_cast<const T *>(a.dy) + row * a.lddy;
            RawRow8<T> rdy;
            RawX<T, SAVED, 0> rx;
            rdy.load(dyr, c, a.cols);
            rx.load(a, row, c);
            uint64_t dy[4], x[4], g[4], dg[4] = {}, db[4] = {};
            load_param(a.gamma, a.wtype, c, a.cols, g);
            rdy.get(dyr, c, a.cols, dy);
            rx.get(a, row, c, nmu2, x);
            ln_bwd_accumulate(rs2, g, dy, x, dg, db, s1, s2);
        }
        const float2 s = team_sum2<false>(sum2(s1), sum2(s2), buf[flip]);
        if (threadIdx.x == 0) a.row_sums[row] = s;
    }
}

// A CTA's sums over its rows, to its part of the workspace: [2][cols up to a multiple of 8].
template <int VPT, int P, typename Col>
__device__ __forceinline__ void store_part(const LnBwdArgs &a, Col col, const uint64_t (&dg)[VPT][P],
                                           const uint64_t (&db)[VPT][P]) {
    const int64_t padded = up8(a.cols);
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * padded;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int64_t c = col(k);
        if (c >= a.cols) continue;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
            *reinterpret_cast<ulonglong2 *>(part + c + 4 * i) = make_ulonglong2(dg[k][2 * i], dg[k][2 * i + 1]);
            *reinterpret_cast<ulonglong2 *>(part + padded + c + 4 * i) =
                make_ulonglong2(db[k][2 * i], db[k][2 * i + 1]);
        }
    }
}

// Rows of 513 .. 8192 columns, one at a time per CTA: thread t has columns
// 8 (t + k threads) .. + 7, k < 2, and their sums over the CTA's rows.  The next rows of
// dy and x are on their way into a ring in shared memory by bulk copies of the 16-byte
// blocks that hold them, whatever their alignment; the barrier of a row's sums
// also tells that its place in the ring may be filled again.  (With the next row in
// registers instead, one row's loads were in flight per CTA: 91 us at 8192 x 8192 for 84, and
// 5003 x 4111 from 8 bits 104 for 70.  8192 x 8192 is at 73 now, 0.82 of a copy's rate.  Issue
// slots (44 %) and the row's barrier bind; rows that start anywhere cost 640 instructions per
// warp for 350: 5003 x 4111 from 8 bits 56 us.)
constexpr int kRing = 8;   // most rows in flight

struct RingArgs {
    LnBwdArgs a;
    int stages;
    uint32_t dy_span, x_span;   // bytes of a row's place: dy, then x or its codes
};

// ALIGNED: every row starts on a 16-byte boundary and is a multiple of 8 columns long.
template <typename T, bool SAVED, int THREADS, int CTAS, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, CTAS) ln_bwd_ring_kernel(const RingArgs r) {
    constexpr int VPT = 2, kSize = static_cast<int>(sizeof(T));
    const LnBwdArgs &a = r.a;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) uint64_t buf[2][16];
    __shared__ uint64_t bars[kRing];
    __shared__ int gave_up;
    const uint32_t bar0 = smem_u32(bars), stage_bytes = r.dy_span + r.x_span;
    if (threadIdx.x == 0) {
        for (int s = 0; s < r.stages; ++s) mbar_init(bar0 + 8 * s, 1);
        gave_up = 0;
        fence_mbar_init();
    }
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const uint8_t *dy0 = static_cast<const uint8_t *>(a.dy), *x0 = static_cast<const uint8_t *>(a.x);
    const int cols = static_cast<int>(a.cols);
    auto issue = [&](int64_t row, int s) {
        const uintptr_t d = reinterpret_cast<uintptr_t>(dy0 + row * a.lddy * kSize);
        const uintptr_t x = SAVED ? reinterpret_cast<uintptr_t>(a.x8.codes + row * a.x8.ld)
                                  : reinterpret_cast<uintptr_t>(x0 + row * a.ldx * kSize);
        const uint32_t dn = (static_cast<uint32_t>(d & 15) + cols * kSize + 15) & ~15u;
        const uint32_t xn = (static_cast<uint32_t>(x & 15) + cols * (SAVED ? 1 : kSize) + 15) & ~15u;
        const uint32_t to = smem_u32(ring) + s * stage_bytes;
        mbar_arrive_expect_tx(bar0 + 8 * s, dn + xn);
        bulk_load_1d(to, reinterpret_cast<const void *>(d & ~uintptr_t(15)), dn, bar0 + 8 * s);
        bulk_load_1d(to + r.dy_span, reinterpret_cast<const void *>(x & ~uintptr_t(15)), xn, bar0 + 8 * s);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < r.stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < a.rows)
                issue(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
    const float ninv_n = -__fdiv_rn(1.0f, static_cast<float>(a.cols));
    auto col = [&](int k) { return static_cast<int>(8 * (threadIdx.x + k * blockDim.x)); };
    uint64_t dg[VPT][4] = {}, db[VPT][4] = {}, g[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) load_param(a.gamma, a.wtype, col(k), a.cols, g[k]);
    // what does not go through the ring is fetched a row ahead
    float mu_next = 0.0f, rs_next = 0.0f;
    uint32_t sc_next[VPT] = {};
    auto fetch = [&](int64_t row) {
        mu_next = a.mean[row], rs_next = a.rstd[row];
        if constexpr (SAVED) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (col(k) < cols) sc_next[k] = fetch_scale(a.x8, row, col(k) >> 7);
        }
    };
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    int s = 0, flip = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const uint64_t nmu2 = splat_f32x2(-mu_next), rs2 = splat_f32x2(rs_next);
        float sc[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) sc[k] = SAVED ? fetched_scale(a.x8, sc_next[k]) : 0.0f;
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        if (!mbar_wait(bar0 + 8 * s, phase, &gave_up)) {
            // goes on with what is there, so that every thread still meets every barrier
            atomicOr(&g_ln_error_flags, kErrWaitTimeout);
            *static_cast<volatile int *>(&gave_up) = 1;
        }
        const uint8_t *stage = ring + s * stage_bytes;
        const uint32_t doff = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dy0 + row * a.lddy * kSize) & 15);
        const uint32_t xoff =
            SAVED ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x0 + row * a.ldx * kSize) & 15);
        uint64_t dy[VPT][4], x[VPT][4], s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int left = cols - col(k);
            if (left > 0) {
                if constexpr (ALIGNED) {
                    RawVec<T, 8> raw;
                    raw.load(reinterpret_cast<const T *>(stage), col(k), cols);
                    raw.get(nullptr, 0, 0, dy[k]);
                    if constexpr (!SAVED) {
                        raw.load(reinterpret_cast<const T *>(stage + r.dy_span), col(k), cols);
                        raw.get(nullptr, 0, 0, x[k]);
                        add_all(nmu2, x[k]);
                    }
                } else {
                    RawRow8<T> raw;
                    raw.load_shared(stage + col(k) * kSize, doff != 0);
                    raw.get(doff, left, dy[k]);
                    if constexpr (!SAVED) {
                        raw.load_shared(stage + r.dy_span + col(k) * kSize, xoff != 0);
                        raw.get(xoff, left, x[k]);
                        add_all(nmu2, x[k]);
                    }
                }
                if constexpr (SAVED) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(stage + r.dy_span + col(k));
                    codes8(w, a.x8.fmt, sc[k], nmu2, ALIGNED ? 8 : left, x[k]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) dy[k][i] = x[k][i] = 0;
            }
            ln_bwd_accumulate(rs2, g[k], dy[k], x[k], dg[k], db[k], s1, s2);
        }
        const float2 sum = team_sum2<false>(sum2(s1), sum2(s2), buf[flip]);
        if (threadIdx.x == 0 && row + static_cast<int64_t>(r.stages) * gridDim.x < a.rows && !gave_up)
            issue(row + static_cast<int64_t>(r.stages) * gridDim.x, s);
        const uint64_t nm1 = splat_f32x2(__fmul_rn(sum.x, ninv_n)), nm2 = splat_f32x2(__fmul_rn(sum.y, ninv_n));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dy[k][i] = f32x2_mul(f32x2_fma(x[k][i], nm2, f32x2_add(dy[k][i], nm1)), rs2);
            if constexpr (ALIGNED)
                RawVec<T, 8>::store(static_cast<T *>(a.dx) + row * a.lddx, col(k), a.cols, dy[k]);
            else
                store_row8<T>(static_cast<T *>(a.dx) + row * a.lddx, col(k), a.cols, dy[k]);
        }
        if (++s == r.stages) s = 0, phase ^= 1u;
    }
    store_part(a, col, dg, db);
    if (gave_up && threadIdx.x == 0)   // copies still in flight land (bounded) before the CTA exits
        for (int i = 0; i < r.stages; ++i) {
            mbar_wait(bar0 + 8 * s, phase, nullptr, 100000000ull);
            if (++s == r.stages) s = 0, phase ^= 1u;
        }
}

// Narrow rows (WARP) and wide ones.  Rows in turn; a thread keeps its columns (as in the forward) and their sums over
// the CTA's rows.  WIDE: blockIdx.y, and blockIdx.z where there are more than 65535, is a
// slab of 8 VPT blockDim.x columns, and the rows' sums are already there.
template <typename T, bool SAVED, int VPT, bool WARP, bool WIDE, int VEC>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512) ln_bwd_kernel(const LnBwdArgs a) {
    using L = Lay<T, VEC>;
    constexpr int E = L::E, P = L::P;
    __shared__ __align__(16) uint64_t buf[2][16];
    const Team<WARP> team;
    clear_sums(buf);
    pdl_wait();
    pdl_trigger();
    const float ninv_n = -__fdiv_rn(1.0f, static_cast<float>(a.cols));
    const int64_t slab = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
    const int64_t base = WIDE ? slab * E * VPT * blockDim.x : 0;   // past the last column: nothing to do
    auto col = [&](int k) { return base + E * (team.id + k * team.size); };
    typename L::Raw rdy[VPT];
    RawX<T, SAVED, VEC> rx[VPT];
    float mu_next = 0.0f, rs_next = 0.0f;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rdy[k].load(static_cast<const T *>(a.dy) + row * a.lddy, col(k), a.cols);
            rx[k].load(a, row, col(k));
        }
        mu_next = a.mean[row], rs_next = a.rstd[row];
    };
    if (team.row < a.rows) fetch(team.row);
    uint64_t dg[VPT][P] = {}, db[VPT][P] = {}, g[VPT][P];
#pragma unroll
    for (int k = 0; k < VPT; ++k) load_param(a.gamma, a.wtype, col(k), a.cols, g[k]);
    int flip = 0;
    for (int64_t row = team.row; row < a.rows; row += team.step, flip ^= 1) {
        const uint64_t nmu2 = splat_f32x2(-mu_next), rs2 = splat_f32x2(rs_next);
        uint64_t dy[VPT][P], x[VPT][P], s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rdy[k].get(static_cast<const T *>(a.dy) + row * a.lddy, col(k), a.cols, dy[k]);
            rx[k].get(a, row, col(k), nmu2, x[k]);
        }
        if (row + team.step < a.rows) fetch(row + team.step);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            ln_bwd_accumulate(rs2, g[k], dy[k], x[k], dg[k], db[k], s1, s2);
        float2 s;
        if constexpr (WIDE)
            s = a.row_sums[row];
        else
            s = team_sum2<WARP>(sum2(s1), sum2(s2), buf[flip]);
        const uint64_t nm1 = splat_f32x2(__fmul_rn(s.x, ninv_n)), nm2 = splat_f32x2(__fmul_rn(s.y, ninv_n));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                dy[k][i] = f32x2_mul(f32x2_fma(x[k][i], nm2, f32x2_add(dy[k][i], nm1)), rs2);
            L::store(static_cast<T *>(a.dx) + row * a.lddx, col(k), a.cols, dy[k]);
        }
    }
    if constexpr (WARP) {
        // the warps that had rows (the first one always) add theirs one after the other;
        // [column of the lane][lane], so that a warp's accesses meet no bank twice
        __shared__ float sums[2][VPT * E][32];
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w && team.row < a.rows) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        float lo, hi, lo2, hi2;
                        f32x2_unpack(dg[k][i / 2], lo, hi);
                        f32x2_unpack(db[k][i / 2], lo2, hi2);
                        float *p = &sums[0][k * E + i][lane], *q = &sums[1][k * E + i][lane];
                        *p = w ? __fadd_rn(*p, i & 1 ? hi : lo) : i & 1 ? hi : lo;
                        *q = w ? __fadd_rn(*q, i & 1 ? hi2 : lo2) : i & 1 ? hi2 : lo2;
                    }
            }
            if (blockIdx.x * kWarps + w + 1 >= a.rows) break;   // no later warp had rows
            __syncthreads();
        }
        __syncthreads();
        const int64_t padded = up8(a.cols);
        float *part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * padded;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const int slot = static_cast<int>(c / (32 * E)) * E + static_cast<int>(c % E);
            const int of = static_cast<int>(c / E) & 31;
            part[c] = sums[0][slot][of];
            part[padded + c] = sums[1][slot][of];
        }
    } else {
        store_part(a, col, dg, db);
    }
}

// dgamma and dbeta from the CTAs' sums [parts][2][padded]: 32 columns per CTA, 32
// threads down the parts for each, then a fixed tree.
__global__ void __launch_bounds__(1024) ln_bwd_reduce_kernel(const float *__restrict__ part,
                                                             int parts, int64_t cols,
                                                             float *__restrict__ dgamma,
                                                             float *__restrict__ dbeta) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t padded = up8(cols), c = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    float s = 0.0f;
    if (c < 2 * padded) {
        for (int p = ty; p < parts; p += 32 * 5) {   // five reads on their way together
            float v[5];
#pragma unroll
            for (int i = 0; i < 5; ++i)
                v[i] = p + 32 * i < parts ? part[(p + 32 * i) * 2 * padded + c] : 0.0f;
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
    if (tx == 0) {
        if (out < cols)
            dgamma[out] = s;
        else if (out >= padded && out < padded + cols)
            dbeta[out - padded] = s;
    }
}

template <typename T, int VPT, bool WARP, int VEC>
cudaError_t ln_fwd_rows(const LnFwdArgs &a, int sms, cudaStream_t st) {
    const unsigned threads = WARP ? 32 * kWarps : row_threads(a.cols, VPT * Lay<T, VEC>::E);
    // CTAs that the registers allow at once
    const int64_t resident = static_cast<int64_t>(sms) * (threads < 640 ? 640 / threads : 1);
    const unsigned grid = capped(WARP ? (a.rows + kWarps - 1) / kWarps : a.rows, resident);
    return launch_pdl(ln_fwd_kernel<T, VPT, WARP, VEC>, dim3(grid), dim3(threads), 0, st, a);
}

template <typename T>
cudaError_t ln_fwd_typed(const LnFwdArgs &a, bool vec, int sms, cudaStream_t st) {
    if (vec) {
        if (a.cols <= 512) return ln_fwd_rows<T, 1, true, 16>(a, sms, st);
        if (a.cols <= 8192) return ln_fwd_rows<T, 1, false, 16>(a, sms, st);
        if (a.cols <= 16384) return ln_fwd_rows<T, 2, false, 16>(a, sms, st);
    } else {
        if (a.cols <= 512) return ln_fwd_rows<T, 2, true, 0>(a, sms, st);
        if (a.cols <= 8192) return ln_fwd_rows<T, 2, false, 0>(a, sms, st);
        if (a.cols <= 16384) return ln_fwd_rows<T, 4, false, 0>(a, sms, st);
    }
    return launch_pdl(ln_fwd_wide_kernel<T>, dim3(capped(a.rows, 4 * sms)), dim3(512), 0, st, a);
}

// As many rows in flight as the CTAs of an SM have shared memory for.
template <typename T, bool SAVED, int THREADS, int CTAS, bool ALIGNED>
cudaError_t ln_bwd_ring_sized(const LnBwdArgs &a, int grid, unsigned threads, cudaStream_t st) {
    constexpr int64_t kSize = sizeof(T), kBytes = 200 << 10;
    RingArgs r{a, 0, 0, 0};
    r.dy_span = static_cast<uint32_t>((a.cols * kSize + 15 + 127) / 128 * 128 + 128);
    r.x_span = SAVED ? static_cast<uint32_t>((a.cols + 127) / 128 * 128) : r.dy_span;
    const int64_t fit = kBytes / ring_ctas_per_sm(threads) / (r.dy_span + r.x_span);
    r.stages = static_cast<int>(fit < kRing ? fit : kRing);
    static SmemLimit limit;
    const cudaError_t err = limit.allow(ln_bwd_ring_kernel<T, SAVED, THREADS, CTAS, ALIGNED>, kBytes);
    if (err != cudaSuccess) return err;
    return launch_pdl(ln_bwd_ring_kernel<T, SAVED, THREADS, CTAS, ALIGNED>, dim3(grid), dim3(threads),
                      static_cast<size_t>(r.stages) * (r.dy_span + r.x_span), st, r);
}

template <typename T, bool SAVED, bool ALIGNED>
cudaError_t ln_bwd_ring(const LnBwdArgs &a, int grid, cudaStream_t st) {
    const unsigned threads = row_threads(a.cols, 16);
    if (threads > kRingHalf) return ln_bwd_ring_sized<T, SAVED, 512, 1, ALIGNED>(a, grid, threads, st);
    if (threads > 256) return ln_bwd_ring_sized<T, SAVED, kRingHalf, 2, ALIGNED>(a, grid, threads, st);
    return ln_bwd_ring_sized<T, SAVED, 256, 2, ALIGNED>(a, grid, threads, st);
}

template <typename T, bool SAVED, int VEC>
cudaError_t ln_bwd_typed(LnBwdArgs a, float *dgamma, float *dbeta, void *ws, int sms, cudaStream_t st) {
    constexpr int VPT = 2;   // 16 columns per thread
    const int g = static_cast<int>(bwd_ctas(a.rows, a.cols, sms));
    a.part = static_cast<float *>(ws);
    const dim3 grid(g);
    cudaError_t e;
    if (a.cols <= kBwdNarrow) {
        e = launch_pdl(ln_bwd_kernel<T, SAVED, VPT, true, false, VEC>, grid, dim3(32 * kWarps), 0, st, a);
    } else if (a.cols <= kBwdWide) {
        e = ln_bwd_ring<T, SAVED, VEC != 0>(a, g, st);
    } else {
        a.row_sums = reinterpret_cast<float2 *>(a.part + static_cast<int64_t>(g) * 2 * up8(a.cols));
        e = launch_pdl(ln_bwd_sums_kernel<T, SAVED>, dim3(capped(a.rows, 4 * sms)), dim3(512), 0, st, a);
        if (e != cudaSuccess) return e;
        const unsigned slabs = static_cast<unsigned>((a.cols + kBwdSlab - 1) / kBwdSlab);
        const unsigned z = (slabs + 65534) / 65535;
        e = launch_pdl(ln_bwd_kernel<T, SAVED, VPT, false, true, VEC>, dim3(g, (slabs + z - 1) / z, z),
                       dim3(256), 0, st, a);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(ln_bwd_reduce_kernel, dim3(static_cast<unsigned>((2 * up8(a.cols) + 31) / 32)),
                      dim3(1024), 0, st, static_cast<const float *>(a.part), g, a.cols, dgamma,
                      dbeta);
}

}  // namespace

cudaError_t launch_ln_fwd(const MatView &x, const void *gamma, const void *beta, int wtype,
                          float eps, const MatView &y, const BlockView &y8, const BlockView &x8,
                          float *mean, float *rstd, int sm_count, cudaStream_t st) {
    if (x.rows == 0) return cudaSuccess;
    const LnFwdArgs a{x.data, x.rows, x.cols, x.ld, gamma, beta, wtype, eps, y.data, y.ld, y8, x8,
                      mean,   rstd};
    const bool vec = x.cols % 16 == 0 && aligned_rows(x.data, x.ld, x.type) &&
                     aligned_rows(y.data, y.ld, x.type);
    if (x.type == kTypeF32) return ln_fwd_typed<float>(a, vec, sm_count, st);
    if (x.type == kTypeBF16) return ln_fwd_typed<__nv_bfloat16>(a, vec, sm_count, st);
    return ln_fwd_typed<__half>(a, vec, sm_count, st);
}

int64_t ln_bwd_workspace(int64_t rows, int64_t cols) {
    return bwd_ctas_most(rows, cols) * 2 * up8(cols) * 4 + (cols > kBwdWide ? rows * 8 : 0);
}

cudaError_t launch_ln_bwd(const MatView &dy, const MatView &x, const BlockView &x8,
                          const void *gamma, int wtype, const float *mean, const float *rstd,
                          const MatView &dx, float *dgamma, float *dbeta, void *ws, int sm_count,
                          cudaStream_t st) {
    if (dy.rows == 0) {
        cudaError_t e = cudaMemsetAsync(dgamma, 0, dy.cols * 4, st);
        if (e != cudaSuccess) return e;
        return cudaMemsetAsync(dbeta, 0, dy.cols * 4, st);
    }
    const LnBwdArgs a{dy.data, x.data, dy.rows, dy.cols, dy.ld, x.ld, dx.ld, x8,
                      gamma,   wtype,  mean,    rstd,    dx.data, nullptr, nullptr};
    const bool saved = x8.codes != nullptr;
    const bool vec = dy.cols % 8 == 0 && aligned_rows(dy.data, dy.ld, dy.type) &&
                     aligned_rows(x.data, x.ld, dy.type) && aligned_rows(dx.data, dx.ld, dy.type);
#define FP8K_LN_BWD(T)                                                            \
    (saved ? vec ? ln_bwd_typed<T, true, 8>(a, dgamma, dbeta, ws, sm_count, st)          \
                 : ln_bwd_typed<T, true, 0>(a, dgamma, dbeta, ws, sm_count, st)         \
     : vec ? ln_bwd_typed<T, false, 8>(a, dgamma, dbeta, ws, sm_count, st)               \
           : ln_bwd_typed<T, false, 0>(a, dgamma, dbeta, ws, sm_count, st))
    if (dy.type == kTypeF32) return FP8K_LN_BWD(float);
    if (dy.type == kTypeBF16) return FP8K_LN_BWD(__nv_bfloat16);
    return FP8K_LN_BWD(__half);
#undef FP8K_LN_BWD
}

cudaError_t read_and_clear_ln_error_flag(unsigned *flags) {
    return take_error_flags(&g_ln_error_flags, flags);
}

}  // namespace fp8k
