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

// Sum of a pair over the CTA, in a fixed order, the same in every thread.  The
// caller alternates between two buffers: a buffer is written again only after
// a barrier that follows its last read.
template <int NT>
__device__ __forceinline__ float2 cta_sum2(float a, float b, float2 (&buf)[NT / 32]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a = __fadd_rn(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        b = __fadd_rn(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
    }
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = buf[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) {
        s.x = __fadd_rn(s.x, buf[w].x);
        s.y = __fadd_rn(s.y, buf[w].y);
    }
    return s;
}

// Quantizes 8 consecutive columns per lane: 16 lanes hold a block of 128.  All
// lanes of the warp take part; lanes past the row hold zeros.
__device__ __forceinline__ void emit_block8(const float (&v)[8], const BlockView &q, int64_t row,
                                            int64_t c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_abs_bits(v[i]));
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const uint32_t byte = q.fmt == 0 ? scale_byte<0>(m) : scale_byte<1>(m);
    const float inv = scale_inverse(byte);
    if (c >= q.cols) return;
    if ((threadIdx.x & 15) == 0) store_scale(q, row, c >> 7, byte);
    uint2 w;
    if (q.fmt == 0)
        w = make_uint2(encode4<0>(v[0], v[1], v[2], v[3], inv), encode4<0>(v[4], v[5], v[6], v[7], inv));
    else
        w = make_uint2(encode4<1>(v[0], v[1], v[2], v[3], inv), encode4<1>(v[4], v[5], v[6], v[7], inv));
    uint8_t *p = q.codes + row * q.ld + c;
    if (c + 8 <= q.cols) {
        *reinterpret_cast<uint2 *>(p) = w;
    } else {
        store_code_word(p, w.x, q.cols - c);
        store_code_word(p + 4, w.y, q.cols - c - 4);
    }
}

struct LnFwdArgs {
    const void *x;
    int64_t rows, cols, ldx;
    bool vecx, vecy;
    const void *gamma, *beta;
    int wtype;
    float eps;
    void *y;
    int64_t ldy;
    BlockView y8, x8;   // codes null: not wanted
    float *mean, *rstd;
};

// One row at a time per CTA; thread t holds columns 8 (t + NT k) .. + 7, k < VPT
// (WIDE: k without a bound, x read again for each use).
template <typename T, int NT, int VPT, bool WIDE>
__global__ void __launch_bounds__(NT) ln_fwd_kernel(const LnFwdArgs a) {
    __shared__ float2 buf[2][NT / 32];
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols);
    const int64_t nk = WIDE ? (a.cols + 8 * NT - 1) / (8 * NT) : VPT;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *xr = static_cast<const T *>(a.x) + row * a.ldx;
        float v[VPT][8];
        float s = 0.0f;
        for (int64_t kk = 0; kk < nk; kk += VPT) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                load_row<T, 8>(xr, 8 * (threadIdx.x + NT * (kk + k)), a.cols, a.vecx, v[k]);
                float p = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) p = __fadd_rn(p, v[k][i]);
                s = __fadd_rn(s, p);
            }
        }
        const float mu = __fdiv_rn(cta_sum2<NT>(s, 0.0f, buf[0]).x, n);
        float d2 = 0.0f;
        for (int64_t kk = 0; kk < nk; kk += VPT) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int64_t c = 8 * (threadIdx.x + NT * (kk + k));
                if (WIDE) load_row<T, 8>(xr, c, a.cols, a.vecx, v[k]);
                float p = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = c + i < a.cols ? __fsub_rn(v[k][i], mu) : 0.0f;
                    p = __fmaf_rn(d, d, p);
                }
                d2 = __fadd_rn(d2, p);
            }
        }
        const float var = __fdiv_rn(cta_sum2<NT>(d2, 0.0f, buf[1]).x, n);
        const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
        if (threadIdx.x == 0) {
            a.mean[row] = mu;
            a.rstd[row] = rs;
        }
        for (int64_t kk = 0; kk < nk; kk += VPT) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int64_t c = 8 * (threadIdx.x + NT * (kk + k));
                if (WIDE) load_row<T, 8>(xr, c, a.cols, a.vecx, v[k]);
                if (a.x8.codes != nullptr) emit_block8(v[k], a.x8, row, c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < a.cols)
                        v[k][i] = __fadd_rn(__fmul_rn(__fmul_rn(__fsub_rn(v[k][i], mu), rs),
                                                      load_any(a.gamma, a.wtype, c + i)),
                                            load_any(a.beta, a.wtype, c + i));
                if (a.y != nullptr)
                    store_row<T, 8>(static_cast<T *>(a.y) + row * a.ldy, c, a.cols, a.vecy, v[k]);
                if (a.y8.codes != nullptr) emit_block8(v[k], a.y8, row, c);
            }
        }
    }
}

struct LnBwdArgs {
    const void *dy, *x;
    int64_t rows, cols, lddy, ldx, lddx;
    bool vecdy, vecx, vecdx;
    BlockView x8;
    const void *gamma;
    int wtype;
    const float *mean, *rstd;
    void *dx;
    float *part;       // [gridDim.x][2][cols]: a CTA's sums of dy * xhat and dy
    float2 *row_sums;  // WIDE: [rows] sums of u and u * xhat
};

template <typename T, bool SAVED>
__device__ __forceinline__ void load_pair(const LnBwdArgs &a, int64_t row, int64_t c, float mu,
                                          float rs, float (&dy)[8], float (&xh)[8]) {
    load_row<T, 8>(static_cast<const T *>(a.dy) + row * a.lddy, c, a.cols, a.vecdy, dy);
    if constexpr (SAVED) {
        const float s = c < a.cols ? load_scale(a.x8, row, c >> 7) : 0.0f;
        load_codes<8>(a.x8.codes + row * a.x8.ld, c, a.cols, a.x8.fmt, s, xh);
    } else {
        load_row<T, 8>(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, a.vecx, xh);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        xh[i] = c + i < a.cols ? __fmul_rn(__fsub_rn(xh[i], mu), rs) : 0.0f;
}

// WIDE rows: the two row sums, in a pass of their own.
template <typename T, bool SAVED, int NT>
__global__ void __launch_bounds__(NT) ln_bwd_sums_kernel(const LnBwdArgs a) {
    __shared__ float2 buf[2][NT / 32];
    pdl_wait();
    pdl_trigger();
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const float mu = a.mean[row], rs = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * NT) {
            float dy[8], xh[8];
            load_pair<T, SAVED>(a, row, c, mu, rs, dy, xh);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u =
                    c + i < a.cols ? __fmul_rn(dy[i], load_any(a.gamma, a.wtype, c + i)) : 0.0f;
                s1 = __fadd_rn(s1, u);
                s2 = __fmaf_rn(u, xh[i], s2);
            }
        }
        const float2 s = cta_sum2<NT>(s1, s2, buf[flip]);
        if (threadIdx.x == 0) a.row_sums[row] = s;
    }
}

// Rows in turn; a thread keeps its columns (as in the forward) and their sums
// over the CTA's rows.  WIDE: blockIdx.y is a slab of 8 NT VPT columns and the
// rows' sums are already there.
template <typename T, bool SAVED, int NT, int VPT, bool WIDE>
__global__ void __launch_bounds__(NT) ln_bwd_kernel(const LnBwdArgs a) {
    __shared__ float2 buf[2][NT / 32];
    pdl_wait();
    pdl_trigger();
    const float n = static_cast<float>(a.cols);
    const int64_t base = WIDE ? static_cast<int64_t>(blockIdx.y) * 8 * NT * VPT : 0;
    float dg[VPT][8] = {}, db[VPT][8] = {}, g[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int64_t c = base + 8 * (threadIdx.x + NT * k);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            g[k][i] = c + i < a.cols ? load_any(a.gamma, a.wtype, c + i) : 0.0f;
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const float mu = a.mean[row], rs = a.rstd[row];
        float dy[VPT][8], xh[VPT][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            load_pair<T, SAVED>(a, row, base + 8 * (threadIdx.x + NT * k), mu, rs, dy[k], xh[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[k][i] = __fmaf_rn(dy[k][i], xh[k][i], dg[k][i]);
                db[k][i] = __fadd_rn(db[k][i], dy[k][i]);
                const float u = __fmul_rn(dy[k][i], g[k][i]);
                s1 = __fadd_rn(s1, u);
                s2 = __fmaf_rn(u, xh[k][i], s2);
            }
        }
        float2 s;
        if constexpr (WIDE)
            s = a.row_sums[row];
        else
            s = cta_sum2<NT>(s1, s2, buf[flip]);
        const float m1 = __fdiv_rn(s.x, n), m2 = __fdiv_rn(s.y, n);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dy[k][i] = __fmul_rn(rs, __fsub_rn(__fsub_rn(__fmul_rn(dy[k][i], g[k][i]), m1),
                                                   __fmul_rn(xh[k][i], m2)));
            store_row<T, 8>(static_cast<T *>(a.dx) + row * a.lddx,
                            base + 8 * (threadIdx.x + NT * k), a.cols, a.vecdx, dy[k]);
        }
    }
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int64_t c = base + 8 * (threadIdx.x + NT * k);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i < a.cols) {
                part[c + i] = dg[k][i];
                part[a.cols + c + i] = db[k][i];
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

bool rows_vec8(const void *p, int64_t ld, int type) {
    const int64_t size = type == kTypeF32 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
}

template <typename T>
cudaError_t ln_fwd_typed(const LnFwdArgs &a, int sms, cudaStream_t st) {
    const int64_t cap = static_cast<int64_t>(sms) * 16;
    const dim3 grid(static_cast<unsigned>(a.rows < cap ? a.rows : cap));
    if (a.cols <= 1024) return launch_pdl(ln_fwd_kernel<T, 128, 1, false>, grid, dim3(128), 0, st, a);
    if (a.cols <= 4096) return launch_pdl(ln_fwd_kernel<T, 256, 2, false>, grid, dim3(256), 0, st, a);
    if (a.cols <= 8192) return launch_pdl(ln_fwd_kernel<T, 512, 2, false>, grid, dim3(512), 0, st, a);
    if (a.cols <= 16384) return launch_pdl(ln_fwd_kernel<T, 512, 4, false>, grid, dim3(512), 0, st, a);
    return launch_pdl(ln_fwd_kernel<T, 1024, 2, true>, grid, dim3(1024), 0, st, a);
}

constexpr int kBwdCtas = 304;       // most CTAs that keep sums of their own
constexpr int64_t kBwdWide = 16384; // rows up to this are held in registers

template <typename T, bool SAVED>
cudaError_t ln_bwd_typed(LnBwdArgs a, float *dgamma, float *dbeta, void *ws, cudaStream_t st) {
    const int g = static_cast<int>(a.rows < kBwdCtas ? a.rows : kBwdCtas);
    a.part = static_cast<float *>(ws);
    const dim3 grid(g);
    cudaError_t e;
    if (a.cols <= 1024)
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 128, 1, false>, grid, dim3(128), 0, st, a);
    else if (a.cols <= 4096)
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 256, 2, false>, grid, dim3(256), 0, st, a);
    else if (a.cols <= 8192)
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 512, 2, false>, grid, dim3(512), 0, st, a);
    else if (a.cols <= kBwdWide)
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 1024, 2, false>, grid, dim3(1024), 0, st, a);
    else {
        a.row_sums = reinterpret_cast<float2 *>(a.part + static_cast<int64_t>(g) * 2 * a.cols);
        e = launch_pdl(ln_bwd_sums_kernel<T, SAVED, 1024>, dim3(static_cast<unsigned>(a.rows < 2048 ? a.rows : 2048)), dim3(1024), 0, st, a);
        if (e != cudaSuccess) return e;
        const dim3 slabs(g, static_cast<unsigned>((a.cols + 4095) / 4096));
        e = launch_pdl(ln_bwd_kernel<T, SAVED, 256, 2, true>, slabs, dim3(256), 0, st, a);
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
    const LnFwdArgs a{x.data, x.rows, x.cols, x.ld, rows_vec8(x.data, x.ld, x.type),
                      rows_vec8(y.data, y.ld, x.type), gamma, beta, wtype, eps, y.data, y.ld, y8,
                      x8, mean, rstd};
    if (x.type == kTypeF32) return ln_fwd_typed<float>(a, sm_count, st);
    if (x.type == kTypeBF16) return ln_fwd_typed<__nv_bfloat16>(a, sm_count, st);
    return ln_fwd_typed<__half>(a, sm_count, st);
}

int64_t ln_bwd_workspace(int64_t rows, int64_t cols) {
    const int64_t g = rows < kBwdCtas ? rows : kBwdCtas;
    return g * 2 * cols * 4 + (cols > kBwdWide ? rows * 8 : 0);
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
    const LnBwdArgs a{dy.data, x.data, dy.rows, dy.cols, dy.ld, x.ld, dx.ld,
                      rows_vec8(dy.data, dy.ld, dy.type), rows_vec8(x.data, x.ld, dy.type),
                      rows_vec8(dx.data, dx.ld, dy.type), x8, gamma, wtype, mean, rstd, dx.data,
                      nullptr, nullptr};
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
