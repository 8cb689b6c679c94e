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

#include "block.cuh"

namespace fp8k {

namespace {

// Who works on a row: a warp (rows of up to 32 x 8 x VPT columns; a CTA has kWarps rows
// at a time) or the whole CTA.  Thread i of the team holds columns 8 (i + k team) .. + 7
// for k < VPT, as packed pairs.  The row after the one in work is already being
// loaded, into registers.
constexpr int kWarps = 8;

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
template <bool WARP>
__device__ __forceinline__ float2 team_sum2(float a, float b, float2 (&buf)[32]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a = __fadd_rn(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        b = __fadd_rn(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
    }
    if constexpr (WARP) return make_float2(a, b);
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 s = lane < static_cast<int>(blockDim.x >> 5) ? buf[lane] : make_float2(0.0f, 0.0f);
    a = s.x, b = s.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a = __fadd_rn(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        b = __fadd_rn(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
    }
    return make_float2(a, b);
}

__device__ __forceinline__ float sum2(uint64_t v) {
    float lo, hi;
    f32x2_unpack(v, lo, hi);
    return __fadd_rn(lo, hi);
}

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

// The part of the forward that follows the statistics, for 8 columns: `at` columns past
// the writers' first, `left` columns before the row's end.
template <typename T>
__device__ __forceinline__ void ln_finish(const LnFwdArgs &a, T *yr, const RowWriter &wy,
                                          const RowWriter &wx, int64_t c, int at, int left,
                                          uint64_t nmu2, uint64_t rs2, const uint64_t (&g)[4],
                                          const uint64_t (&b)[4], const uint64_t (&x)[4]) {
    if (a.x8.codes != nullptr) wx.put(x, at, left);
    if (a.y == nullptr && a.y8.codes == nullptr) return;
    uint64_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = f32x2_fma(f32x2_mul(f32x2_add(x[i], nmu2), rs2), g[i], b[i]);
    if (a.y != nullptr) store_row8<T>(yr, c, a.cols, y);
    if (a.y8.codes != nullptr) wy.put(y, at, left);
}

__device__ __forceinline__ void load_param8(const void *p, int type, int64_t c, int64_t cols,
                                            uint64_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = f32x2_pack(c + 2 * i < cols ? load_any(p, type, c + 2 * i) : 0.0f,
                          c + 2 * i + 1 < cols ? load_any(p, type, c + 2 * i + 1) : 0.0f);
}

// sum of (x - mean)^2 over 8 columns; those past the row do not count
__device__ __forceinline__ uint64_t deviations(const uint64_t (&x)[4], uint64_t nmu2, int64_t c,
                                               int64_t cols, uint64_t s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t d = f32x2_add(x[i], nmu2);
        if (c + 8 > cols) {
            float lo, hi;
            f32x2_unpack(d, lo, hi);
            d = f32x2_pack(c + 2 * i < cols ? lo : 0.0f, c + 2 * i + 1 < cols ? hi : 0.0f);
        }
        s = f32x2_fma(d, d, s);
    }
    return s;
}

template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512) ln_fwd_kernel(const LnFwdArgs a) {
    __shared__ float2 buf[2][32];
    const Team<WARP> team;
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols);
    const int left0 = static_cast<int>(a.cols) - 8 * team.id;
    RowWriter wx, wy;
    wx.start(a.x8, team.row, team.step, 8 * team.id);
    wy.start(a.y8, team.row, team.step, 8 * team.id);
    RawRow8<T> raw[VPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            raw[k].load(static_cast<const T *>(a.x) + row * a.ldx, 8 * (team.id + k * team.size), a.cols);
    };
    if (team.row < a.rows) fetch(team.row);
    // gamma and beta stay in registers where there is room for them
    constexpr int kKept = VPT <= 2 ? VPT : 1;
    uint64_t g[kKept][4], b[kKept][4];
    auto params = [&](int k, int slot) {
        load_param8(a.gamma, a.wtype, 8 * (team.id + k * team.size), a.cols, g[slot]);
        load_param8(a.beta, a.wtype, 8 * (team.id + k * team.size), a.cols, b[slot]);
    };
    if constexpr (VPT <= 2) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) params(k, k);
    }
    for (int64_t row = team.row; row < a.rows; row += team.step) {
        uint64_t x[VPT][4], s2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            raw[k].get(static_cast<const T *>(a.x) + row * a.ldx, 8 * (team.id + k * team.size), a.cols,
                       x[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = f32x2_add(s2, x[k][i]);
        }
        if (row + team.step < a.rows) fetch(row + team.step);
        const float mu = __fdiv_rn(team_sum2<WARP>(sum2(s2), 0.0f, buf[0]).x, n);
        const uint64_t nmu2 = splat_f32x2(-mu);
        s2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            s2 = deviations(x[k], nmu2, 8 * (team.id + k * team.size), a.cols, s2);
        const float var = __fdiv_rn(team_sum2<WARP>(sum2(s2), 0.0f, buf[1]).x, n);
        const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
        if (team.id == 0) {
            a.mean[row] = mu;
            a.rstd[row] = rs;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if constexpr (VPT > 2) params(k, 0);
            const int at = 8 * k * team.size;
            ln_finish<T>(a, static_cast<T *>(a.y) + row * a.ldy, wy, wx, 8 * team.id + at, at, left0 - at,
                         nmu2, splat_f32x2(rs), g[k % kKept], b[k % kKept], x[k]);
        }
        wx.next_row();
        wy.next_row();
    }
}

// Rows too long for a CTA's registers: x is read again for each use.
template <typename T>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(const LnFwdArgs a) {
    __shared__ float2 buf[2][32];
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols);
    // whole warps stay together: the exchanges between lanes need all of them
    const int64_t warp0 = 8 * (threadIdx.x & ~31);
    RowWriter wx, wy;
    wx.start(a.x8, blockIdx.x, gridDim.x, 8 * threadIdx.x);
    wy.start(a.y8, blockIdx.x, gridDim.x, 8 * threadIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *xr = static_cast<const T *>(a.x) + row * a.ldx;
        RawRow8<T> raw;
        uint64_t x[4], s2 = 0;
        for (int64_t w = warp0; w < a.cols; w += 8 * 1024) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            raw.load(xr, c, a.cols);
            raw.get(xr, c, a.cols, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = f32x2_add(s2, x[i]);
        }
        const float mu = __fdiv_rn(team_sum2<false>(sum2(s2), 0.0f, buf[0]).x, n);
        const uint64_t nmu2 = splat_f32x2(-mu);
        s2 = 0;
        for (int64_t w = warp0; w < a.cols; w += 8 * 1024) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            raw.load(xr, c, a.cols);
            raw.get(xr, c, a.cols, x);
            s2 = deviations(x, nmu2, c, a.cols, s2);
        }
        const float var = __fdiv_rn(team_sum2<false>(sum2(s2), 0.0f, buf[1]).x, n);
        const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
        if (threadIdx.x == 0) {
            a.mean[row] = mu;
            a.rstd[row] = rs;
        }
        for (int64_t w = warp0; w < a.cols; w += 8 * 1024) {
            const int64_t c = w + 8 * (threadIdx.x & 31);
            uint64_t g[4], b[4];
            load_param8(a.gamma, a.wtype, c, a.cols, g);
            load_param8(a.beta, a.wtype, c, a.cols, b);
            raw.load(xr, c, a.cols);
            raw.get(xr, c, a.cols, x);
            ln_finish<T>(a, static_cast<T *>(a.y) + row * a.ldy, wy, wx, c, static_cast<int>(w - warp0),
                         static_cast<int>(a.cols - c), nmu2, splat_f32x2(rs), g, b, x);
        }
        wx.next_row();
        wy.next_row();
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
    float *part;       // [gridDim.x][2][cols]: a CTA's sums of dy * xhat and dy
    float2 *row_sums;  // wide rows: [rows] sums of u and u * xhat
};

// 8 columns of x on their way: as they are, or codes with their block's scale.
template <typename T, bool SAVED>
struct RawX8;
template <typename T>
struct RawX8<T, false> {
    RawRow8<T> raw;
    __device__ __forceinline__ void load(const LnBwdArgs &a, int64_t row, int64_t c) {
        raw.load(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols);
    }
    __device__ __forceinline__ void get(const LnBwdArgs &a, int64_t row, int64_t c, uint64_t (&v)[4]) const {
        raw.get(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, v);
    }
};
template <typename T>
struct RawX8<T, true> {
    uint2 codes;
    float scale;
    __device__ __forceinline__ void load(const LnBwdArgs &a, int64_t row, int64_t c) {
        const bool in = c < a.cols;
        codes = in ? *reinterpret_cast<const uint2 *>(a.x8.codes + row * a.x8.ld + c) : make_uint2(0, 0);
        scale = in ? load_scale(a.x8, row, c >> 7) : 0.0f;
    }
    __device__ __forceinline__ void get(const LnBwdArgs &a, int64_t, int64_t c, uint64_t (&v)[4]) const {
        float f[8];
        decode4(codes.x, a.x8.fmt, *reinterpret_cast<float(*)[4]>(f));
        decode4(codes.y, a.x8.fmt, *reinterpret_cast<float(*)[4]>(f + 4));
        const uint64_t s2 = splat_f32x2(scale);
#pragma unroll
        for (int i = 0; i < 4; ++i)   // codes past the row may be anything
            v[i] = f32x2_mul(f32x2_pack(c + 2 * i < a.cols ? f[2 * i] : 0.0f,
                                        c + 2 * i + 1 < a.cols ? f[2 * i + 1] : 0.0f),
                             s2);
    }
};

// xhat in place of x, and u in place of dy; their sums for the row, and the column sums
__device__ __forceinline__ void ln_bwd_accumulate(uint64_t nmu2, uint64_t rs2, const uint64_t (&g)[4],
                                                  uint64_t (&dy)[4], uint64_t (&x)[4],
                                                  uint64_t (&dg)[4], uint64_t (&db)[4], uint64_t &s1,
                                                  uint64_t &s2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = f32x2_mul(f32x2_add(x[i], nmu2), rs2);
        dg[i] = f32x2_fma(dy[i], x[i], dg[i]);
        db[i] = f32x2_add(db[i], dy[i]);
        dy[i] = f32x2_mul(dy[i], g[i]);
        s1 = f32x2_add(s1, dy[i]);
        s2 = f32x2_fma(dy[i], x[i], s2);
    }
}

// Wide rows: the two row sums, in a pass of their own.
template <typename T, bool SAVED>
__global__ void __launch_bounds__(1024) ln_bwd_sums_kernel(const LnBwdArgs a) {
    __shared__ float2 buf[2][32];
    pdl_wait();
    pdl_trigger();
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const uint64_t nmu2 = splat_f32x2(-a.mean[row]), rs2 = splat_f32x2(a.rstd[row]);
        uint64_t s1 = 0, s2 = 0;
        for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * 1024) {
            const T *dyr = static_cast<const T *>(a.dy) + row * a.lddy;
            RawRow8<T> rdy;
            RawX8<T, SAVED> rx;
            rdy.load(dyr, c, a.cols);
            rx.load(a, row, c);
            uint64_t dy[4], x[4], g[4], dg[4] = {}, db[4] = {};
            load_param8(a.gamma, a.wtype, c, a.cols, g);
            rdy.get(dyr, c, a.cols, dy);
            rx.get(a, row, c, x);
            ln_bwd_accumulate(nmu2, rs2, g, dy, x, dg, db, s1, s2);
        }
        const float2 s = team_sum2<false>(sum2(s1), sum2(s2), buf[flip]);
        if (threadIdx.x == 0) a.row_sums[row] = s;
    }
}

// Rows in turn; a thread keeps its columns (as in the forward) and their sums over
// the CTA's rows.  WIDE: blockIdx.y is a slab of 8 VPT blockDim.x columns and the rows'
// sums are already there.
template <typename T, bool SAVED, int VPT, bool WARP, bool WIDE>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512) ln_bwd_kernel(const LnBwdArgs a) {
    __shared__ float2 buf[2][32];
    const Team<WARP> team;
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols);
    const int64_t base = WIDE ? static_cast<int64_t>(blockIdx.y) * 8 * VPT * blockDim.x : 0;
    auto col = [&](int k) { return base + 8 * (team.id + k * team.size); };
    RawRow8<T> rdy[VPT];
    RawX8<T, SAVED> rx[VPT];
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
    uint64_t dg[VPT][4] = {}, db[VPT][4] = {}, g[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) load_param8(a.gamma, a.wtype, col(k), a.cols, g[k]);
    int flip = 0;
    for (int64_t row = team.row; row < a.rows; row += team.step, flip ^= 1) {
        const uint64_t nmu2 = splat_f32x2(-mu_next), rs2 = splat_f32x2(rs_next);
        uint64_t dy[VPT][4], x[VPT][4], s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rdy[k].get(static_cast<const T *>(a.dy) + row * a.lddy, col(k), a.cols, dy[k]);
            rx[k].get(a, row, col(k), x[k]);
        }
        if (row + team.step < a.rows) fetch(row + team.step);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            ln_bwd_accumulate(nmu2, rs2, g[k], dy[k], x[k], dg[k], db[k], s1, s2);
        float2 s;
        if constexpr (WIDE)
            s = a.row_sums[row];
        else
            s = team_sum2<WARP>(sum2(s1), sum2(s2), buf[flip]);
        const uint64_t nm1 = splat_f32x2(-__fdiv_rn(s.x, n)), nm2 = splat_f32x2(-__fdiv_rn(s.y, n));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dy[k][i] = f32x2_mul(f32x2_fma(x[k][i], nm2, f32x2_add(dy[k][i], nm1)), rs2);
            store_row8<T>(static_cast<T *>(a.dx) + row * a.lddx, col(k), a.cols, dy[k]);
        }
    }
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if constexpr (WARP) {
        // the warps add theirs one after the other
        extern __shared__ float sums[];   // [2][cols]
        for (int w = 0; w < kWarps; ++w) {
            if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t c = col(k) + i;
                        if (c >= a.cols) continue;
                        float lo, hi, lo2, hi2;
                        f32x2_unpack(dg[k][i / 2], lo, hi);
                        f32x2_unpack(db[k][i / 2], lo2, hi2);
                        const float p = i & 1 ? hi : lo, q = i & 1 ? hi2 : lo2;
                        sums[c] = w ? __fadd_rn(sums[c], p) : p;
                        sums[a.cols + c] = w ? __fadd_rn(sums[a.cols + c], q) : q;
                    }
            }
            __syncthreads();
        }
        for (int64_t c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) part[c] = sums[c];
    } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int64_t c = col(k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                f32x2_unpack(dg[k][i], lo, hi);
                if (c + 2 * i < a.cols) part[c + 2 * i] = lo;
                if (c + 2 * i + 1 < a.cols) part[c + 2 * i + 1] = hi;
                f32x2_unpack(db[k][i], lo, hi);
                if (c + 2 * i < a.cols) part[a.cols + c + 2 * i] = lo;
                if (c + 2 * i + 1 < a.cols) part[a.cols + c + 2 * i + 1] = hi;
            }
        }
    }
}

// dgamma and dbeta from the CTAs' sums [parts][2 cols]: 32 columns per CTA, 32
// threads down the parts for each, then a fixed tree.
__global__ void __launch_bounds__(1024) ln_bwd_reduce_kernel(const float *__restrict__ part,
                                                             int parts, int64_t cols,
                                                             float *__restrict__ dgamma,
                                                             float *__restrict__ dbeta) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    float s = 0.0f;
    if (c < 2 * cols)
        for (int p = ty; p < parts; p += 32) s = __fadd_rn(s, part[p * 2 * cols + c]);
    red[ty][tx] = s;
    __syncthreads();
    s = red[tx][ty];
#pragma unroll
    for (int o = 16; o; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + ty;
    if (tx == 0 && out < 2 * cols) {
        if (out < cols)
            dgamma[out] = s;
        else
            dbeta[out - cols] = s;
    }
}

// Threads of a CTA that shares a row: whole warps, 8 VPT columns each.
unsigned row_threads(int64_t cols, int vpt) {
    return static_cast<unsigned>((cols + 256 * vpt - 1) / (256 * vpt) * 32);
}

unsigned capped(int64_t n, int64_t cap) { return static_cast<unsigned>(n < cap ? n : cap); }

template <typename T, int VPT, bool WARP>
cudaError_t ln_fwd_rows(const LnFwdArgs &a, int sms, cudaStream_t st) {
    const unsigned threads = WARP ? 32 * kWarps : row_threads(a.cols, VPT);
    // CTAs that the registers allow at once
    const int64_t resident = static_cast<int64_t>(sms) * (threads < 640 ? 640 / threads : 1);
    const unsigned grid = capped(WARP ? (a.rows + kWarps - 1) / kWarps : a.rows, resident);
    return launch_pdl(ln_fwd_kernel<T, VPT, WARP>, dim3(grid), dim3(threads), 0, st, a);
}

template <typename T>
cudaError_t ln_fwd_typed(const LnFwdArgs &a, int sms, cudaStream_t st) {
    if (a.cols <= 256) return ln_fwd_rows<T, 1, true>(a, sms, st);
    if (a.cols <= 512) return ln_fwd_rows<T, 2, true>(a, sms, st);
    if (a.cols <= 8192) return ln_fwd_rows<T, 2, false>(a, sms, st);
    if (a.cols <= 16384) return ln_fwd_rows<T, 4, false>(a, sms, st);
    return launch_pdl(ln_fwd_wide_kernel<T>, dim3(capped(a.rows, 2 * sms)), dim3(1024), 0, st, a);
}

constexpr int64_t kBwdNarrow = 512;   // rows up to this belong to one warp
constexpr int64_t kBwdWide = 8192;    // rows up to this are held in a CTA's registers
constexpr int kBwdVpt = 2;
constexpr int64_t kBwdSlab = 8 * kBwdVpt * 256;   // columns of a wide row's slab

// CTAs that keep column sums of their own, at most: as many as the registers (128 per
// thread) allow at once on 152 SMs; one per SM and slab of a wide row.
int64_t bwd_ctas(int64_t rows, int64_t cols) {
    constexpr int64_t sms = 152;
    if (cols <= kBwdNarrow) return capped((rows + kWarps - 1) / kWarps, 2 * sms);
    if (cols > kBwdWide) return capped(rows, sms);
    const unsigned threads = row_threads(cols, kBwdVpt);
    return capped(rows, sms * (threads < 512 ? 512 / threads : 1));
}

template <typename T, bool SAVED>
cudaError_t ln_bwd_typed(LnBwdArgs a, float *dgamma, float *dbeta, void *ws, cudaStream_t st) {
    const int g = static_cast<int>(bwd_ctas(a.rows, a.cols));
    a.part = static_cast<float *>(ws);
    const dim3 grid(g);
    const size_t sums = static_cast<size_t>(2 * a.cols * 4);
    cudaError_t e;
    if (a.cols <= 256) {
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 1, true, false>, grid, dim3(32 * kWarps), sums, st, a);
    } else if (a.cols <= kBwdNarrow) {
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 2, true, false>, grid, dim3(32 * kWarps), sums, st, a);
    } else if (a.cols <= kBwdWide) {
        e = launch_pdl(ln_bwd_kernel<T, SAVED, kBwdVpt, false, false>, grid,
                       dim3(row_threads(a.cols, kBwdVpt)), 0, st, a);
    } else {
        a.row_sums = reinterpret_cast<float2 *>(a.part + static_cast<int64_t>(g) * 2 * a.cols);
        e = launch_pdl(ln_bwd_sums_kernel<T, SAVED>, dim3(capped(a.rows, 2 * 152)), dim3(1024), 0, st, a);
        if (e != cudaSuccess) return e;
        const dim3 slabs(g, static_cast<unsigned>((a.cols + kBwdSlab - 1) / kBwdSlab));
        e = launch_pdl(ln_bwd_kernel<T, SAVED, kBwdVpt, false, true>, slabs, dim3(256), 0, st, a);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(ln_bwd_reduce_kernel, dim3(static_cast<unsigned>((2 * a.cols + 31) / 32)),
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
    if (x.type == kTypeF32) return ln_fwd_typed<float>(a, sm_count, st);
    if (x.type == kTypeBF16) return ln_fwd_typed<__nv_bfloat16>(a, sm_count, st);
    return ln_fwd_typed<__half>(a, sm_count, st);
}

int64_t ln_bwd_workspace(int64_t rows, int64_t cols) {
    return bwd_ctas(rows, cols) * 2 * cols * 4 + (cols > kBwdWide ? rows * 8 : 0);
}

cudaError_t launch_ln_bwd(const MatView &dy, const MatView &x, const BlockView &x8,
                          const void *gamma, int wtype, const float *mean, const float *rstd,
                          const MatView &dx, float *dgamma, float *dbeta, void *ws,
                          cudaStream_t st) {
    if (dy.rows == 0) {
        cudaError_t e = cudaMemsetAsync(dgamma, 0, dy.cols * 4, st);
        if (e != cudaSuccess) return e;
        return cudaMemsetAsync(dbeta, 0, dy.cols * 4, st);
    }
    const LnBwdArgs a{dy.data, x.data, dy.rows, dy.cols, dy.ld, x.ld, dx.ld, x8,
                      gamma,   wtype,  mean,    rstd,    dx.data, nullptr, nullptr};
    const bool saved = x8.codes != nullptr;
#define FP8K_LN_BWD(T)                                                            \
    (saved ? ln_bwd_typed<T, true>(a, dgamma, dbeta, ws, st)                      \
           : ln_bwd_typed<T, false>(a, dgamma, dbeta, ws, st))
    if (dy.type == kTypeF32) return FP8K_LN_BWD(float);
    if (dy.type == kTypeBF16) return FP8K_LN_BWD(__nv_bfloat16);
    return FP8K_LN_BWD(__half);
#undef FP8K_LN_BWD
}

}  // namespace fp8k
