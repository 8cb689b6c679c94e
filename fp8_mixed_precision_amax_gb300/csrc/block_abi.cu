// block_abi.cu -- the exported C entry points of the block-scaled operators
// (the second half of include/fp8amax.h): argument checks on the host, then
// one to three launches in stream order (a product of few rows one for every
// 8,388,480 columns).  No device memory is allocated and
// the stream is never synchronized.
#include "abi_checks.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;   // as the TMA coordinates allow

fp8_status check_type(const char *fn, int32_t type, const char *name) {
    if (type != FP8_DTYPE_F32 && type != FP8_DTYPE_BF16 && type != FP8_DTYPE_F16)
        return fail(FP8_ERR_ARG, "%s: %s: bad type %d", fn, name, type);
    return FP8_OK;
}

// A matrix, or an empty view when it is NULL and may be.
fp8_status view(const char *fn, const fp8_matrix *m, const char *name, bool optional,
                fp8k::MatView *out) {
    *out = fp8k::MatView{};
    if (m == nullptr) {
        if (optional) return FP8_OK;
        return fail(FP8_ERR_ARG, "%s: %s is NULL", fn, name);
    }
    FP8_TRY(check_type(fn, m->dtype, name));
    if (m->rows < 0 || m->cols < 0 || m->rows >= kMaxDim || m->cols >= kMaxDim)
        return fail(FP8_ERR_ARG, "%s: %s: bad size %lld x %lld", fn, name,
                    static_cast<long long>(m->rows), static_cast<long long>(m->cols));
    if (m->ld < m->cols || m->ld >= kMaxDim)
        return fail(FP8_ERR_ARG, "%s: %s: row stride %lld for %lld columns", fn, name,
                    static_cast<long long>(m->ld), static_cast<long long>(m->cols));
    const uintptr_t size = m->dtype == FP8_DTYPE_F32 ? 4 : 2;
    if (m->data == nullptr && m->rows > 0 && m->cols > 0)
        return fail(FP8_ERR_ARG, "%s: %s has no data", fn, name);
    if (reinterpret_cast<uintptr_t>(m->data) % size)
        return fail(FP8_ERR_ALIGN, "%s: %s is not aligned to its elements", fn, name);
    *out = fp8k::MatView{m->data, m->rows, m->cols, m->ld, m->dtype};
    return FP8_OK;
}

fp8_status view(const char *fn, const fp8_block_tensor *q, const char *name, bool optional,
                fp8k::BlockView *out) {
    *out = fp8k::BlockView{};
    if (q == nullptr) {
        if (optional) return FP8_OK;
        return fail(FP8_ERR_ARG, "%s: %s is NULL", fn, name);
    }
    if (q->fmt != FP8_E4M3 && q->fmt != FP8_E5M2)
        return fail(FP8_ERR_ARG, "%s: %s: bad format %d", fn, name, q->fmt);
    if (q->block_rows != 1 && q->block_rows != 128)
        return fail(FP8_ERR_ARG, "%s: %s: block_rows %d is neither 1 nor 128", fn, name,
                    q->block_rows);
    if (q->scale_type != FP8_SCALE_E8M0 && q->scale_type != FP8_SCALE_F32)
        return fail(FP8_ERR_ARG, "%s: %s: bad scale type %d", fn, name, q->scale_type);
    if (q->rows < 0 || q->cols < 0 || q->rows >= kMaxDim || q->cols >= kMaxDim)
        return fail(FP8_ERR_ARG, "%s: %s: bad size %lld x %lld", fn, name,
                    static_cast<long long>(q->rows), static_cast<long long>(q->cols));
    if (q->ld < q->cols || q->ld >= kMaxDim)
        return fail(FP8_ERR_ARG, "%s: %s: row stride %lld for %lld columns", fn, name,
                    static_cast<long long>(q->ld), static_cast<long long>(q->cols));
    if (q->ld_scales < (q->cols + 127) / 128 || q->ld_scales >= kMaxDim)
        return fail(FP8_ERR_ARG, "%s: %s: %lld scales per row for %lld columns", fn, name,
                    static_cast<long long>(q->ld_scales), static_cast<long long>(q->cols));
    const bool empty = q->rows == 0 || q->cols == 0;
    if (!empty && (q->codes == nullptr || q->scales == nullptr))
        return fail(FP8_ERR_ARG, "%s: %s has no codes or no scales", fn, name);
    if (!aligned16(q->codes) || q->ld % 16)
        return fail(FP8_ERR_ALIGN, "%s: %s: rows of codes must be 16-byte aligned", fn, name);
    if (reinterpret_cast<uintptr_t>(q->scales) % 4 ||
        (q->scale_type == FP8_SCALE_E8M0 && q->ld_scales % 4))
        return fail(FP8_ERR_ALIGN, "%s: %s: rows of scales must be 4-byte aligned", fn, name);
    *out = fp8k::BlockView{q->codes, q->rows, q->cols, q->ld, q->scales, q->ld_scales, q->fmt,
                           q->block_rows, q->scale_type};
    return FP8_OK;
}

template <typename V>
fp8_status check_shape(const char *fn, const V &v, const char *name, int64_t rows, int64_t cols) {
    if (v.rows != rows || v.cols != cols)
        return fail(FP8_ERR_ARG, "%s: %s is %lld x %lld, expected %lld x %lld", fn, name,
                    static_cast<long long>(v.rows), static_cast<long long>(v.cols),
                    static_cast<long long>(rows), static_cast<long long>(cols));
    return FP8_OK;
}

// an optional output of the given shape with one scale per row and block
fp8_status check_rows_out(const char *fn, const fp8_block_tensor *q, const fp8k::BlockView &v,
                          const char *name, int64_t rows, int64_t cols) {
    if (q == nullptr) return FP8_OK;
    FP8_TRY(check_shape(fn, v, name, rows, cols));
    if (v.block_rows != 1) return fail(FP8_ERR_ARG, "%s: %s: block_rows must be 1", fn, name);
    return FP8_OK;
}

fp8_status check_tiles(const char *fn, int64_t rows, int64_t cols) {
    if (((rows + 127) / 128) * ((cols + 127) / 128) >= kMaxDim)
        return fail(FP8_ERR_ARG, "%s: more than 2^31 tiles", fn);
    return FP8_OK;
}

fp8_status check_param(const char *fn, const void *p, int32_t type, const char *name) {
    if (p == nullptr) return fail(FP8_ERR_ARG, "%s: %s is NULL", fn, name);
    if (reinterpret_cast<uintptr_t>(p) % (type == FP8_DTYPE_F32 ? 4 : 2))
        return fail(FP8_ERR_ALIGN, "%s: %s is not aligned to its elements", fn, name);
    return FP8_OK;
}

}  // namespace

extern "C" {

fp8_status fp8_block_quantize(const fp8_matrix *x, const fp8_block_tensor *q,
                              const fp8_block_tensor *qt, void *stream) {
    const char *fn = "fp8_block_quantize";
    const fp8k::CallRange range(fn);
    fp8k::MatView vx;
    fp8k::BlockView vq, vqt;
    FP8_TRY(view(fn, x, "x", false, &vx));
    FP8_TRY(view(fn, q, "q", true, &vq));
    FP8_TRY(view(fn, qt, "qt", true, &vqt));
    if (q == nullptr && qt == nullptr) return fail(FP8_ERR_ARG, "%s: q and qt are both NULL", fn);
    if (q != nullptr) FP8_TRY(check_shape(fn, vq, "q", vx.rows, vx.cols));
    if (qt != nullptr) FP8_TRY(check_shape(fn, vqt, "qt", vx.cols, vx.rows));
    if (q != nullptr && qt != nullptr &&
        (vq.fmt != vqt.fmt || vq.block_rows != vqt.block_rows || vq.scale_f32 != vqt.scale_f32))
        return fail(FP8_ERR_ARG, "%s: q and qt differ in format, block_rows or scale type", fn);
    FP8_TRY(check_tiles(fn, vx.rows, vx.cols));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_block_quantize(vx, vq, vqt, sms, static_cast<cudaStream_t>(stream)), fn);
    return FP8_OK;
}

fp8_status fp8_block_dequantize(const fp8_block_tensor *q, const fp8_matrix *out, void *stream) {
    const char *fn = "fp8_block_dequantize";
    const fp8k::CallRange range(fn);
    fp8k::BlockView vq;
    fp8k::MatView vo;
    FP8_TRY(view(fn, q, "q", false, &vq));
    FP8_TRY(view(fn, out, "out", false, &vo));
    FP8_TRY(check_shape(fn, vo, "out", vq.rows, vq.cols));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_block_dequantize(vq, vo, sms, static_cast<cudaStream_t>(stream)), fn);
    return FP8_OK;
}

fp8_status fp8_block_gemm_tn(const fp8_block_tensor *A, const fp8_block_tensor *B,
                             const fp8_matrix *D, void *stream) {
    const char *fn = "fp8_block_gemm_tn";
    const fp8k::CallRange range(fn);
    fp8k::BlockView a, b;
    fp8k::MatView d;
    FP8_TRY(view(fn, A, "A", false, &a));
    FP8_TRY(view(fn, B, "B", false, &b));
    FP8_TRY(view(fn, D, "D", false, &d));
    if (a.cols != b.cols)
        return fail(FP8_ERR_ARG, "%s: A has %lld columns, B %lld", fn,
                    static_cast<long long>(a.cols), static_cast<long long>(b.cols));
    if (a.scale_f32 != b.scale_f32)
        return fail(FP8_ERR_ARG, "%s: A and B have scales of different types", fn);
    FP8_TRY(check_shape(fn, d, "D", a.rows, b.rows));
    if (d.type != FP8_DTYPE_BF16) return fail(FP8_ERR_ARG, "%s: D must be BF16", fn);
    FP8_TRY(check_tiles(fn, a.rows, b.rows));
    int sms;
    FP8_TRY(current_device(&sms));
    const char *what = nullptr;
    const cudaError_t e =
        fp8k::launch_block_gemm(a, b, d, sms, static_cast<cudaStream_t>(stream), &what);
    if (e != cudaSuccess) return what ? fail(FP8_ERR_CUDA, "%s: %s", fn, what) : cuda_fail(e, fn);
    return FP8_OK;
}

fp8_status fp8_layernorm_fwd(const fp8_matrix *x, const void *gamma, const void *beta,
                             int32_t wtype, float eps, const fp8_matrix *y,
                             const fp8_block_tensor *y8, const fp8_block_tensor *x8, float *mean,
                             float *rstd, void *stream) {
    const char *fn = "fp8_layernorm_fwd";
    const fp8k::CallRange range(fn);
    fp8k::MatView vx, vy;
    fp8k::BlockView vy8, vx8;
    FP8_TRY(view(fn, x, "x", false, &vx));
    FP8_TRY(view(fn, y, "y", true, &vy));
    FP8_TRY(view(fn, y8, "y8", true, &vy8));
    FP8_TRY(view(fn, x8, "x8", true, &vx8));
    if (vx.cols < 1) return fail(FP8_ERR_ARG, "%s: x has no columns", fn);
    if (!(eps >= 0.0f)) return fail(FP8_ERR_ARG, "%s: eps must be >= 0", fn);
    FP8_TRY(check_type(fn, wtype, "gamma"));
    FP8_TRY(check_param(fn, gamma, wtype, "gamma"));
    FP8_TRY(check_param(fn, beta, wtype, "beta"));
    if (y != nullptr) {
        FP8_TRY(check_shape(fn, vy, "y", vx.rows, vx.cols));
        if (vy.type != vx.type) return fail(FP8_ERR_ARG, "%s: y must have x's type", fn);
    }
    FP8_TRY(check_rows_out(fn, y8, vy8, "y8", vx.rows, vx.cols));
    FP8_TRY(check_rows_out(fn, x8, vx8, "x8", vx.rows, vx.cols));
    const bool empty = vx.rows == 0;
    FP8_TRY(check_scalar(fn, mean, "mean", empty));
    FP8_TRY(check_scalar(fn, rstd, "rstd", empty));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_ln_fwd(vx, gamma, beta, wtype, eps, vy, vy8, vx8, mean, rstd, sms,
                                 static_cast<cudaStream_t>(stream)),
             fn);
    return FP8_OK;
}

int64_t fp8_layernorm_bwd_workspace(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 ? 0 : fp8k::ln_bwd_workspace(rows, cols);
}

fp8_status fp8_layernorm_bwd(const fp8_matrix *dy, const fp8_matrix *x,
                             const fp8_block_tensor *x8, const void *gamma, int32_t wtype,
                             const float *mean, const float *rstd, const fp8_matrix *dx,
                             float *dgamma, float *dbeta, void *workspace, int64_t workspace_bytes,
                             void *stream) {
    const char *fn = "fp8_layernorm_bwd";
    const fp8k::CallRange range(fn);
    fp8k::MatView vdy, vx, vdx;
    fp8k::BlockView vx8;
    FP8_TRY(view(fn, dy, "dy", false, &vdy));
    FP8_TRY(view(fn, x, "x", true, &vx));
    FP8_TRY(view(fn, x8, "x8", true, &vx8));
    FP8_TRY(view(fn, dx, "dx", false, &vdx));
    if ((x != nullptr) == (x8 != nullptr))
        return fail(FP8_ERR_ARG, "%s: exactly one of x and x8 is given", fn);
    if (vdy.cols < 1) return fail(FP8_ERR_ARG, "%s: dy has no columns", fn);
    if (x != nullptr) {
        FP8_TRY(check_shape(fn, vx, "x", vdy.rows, vdy.cols));
        if (vx.type != vdy.type) return fail(FP8_ERR_ARG, "%s: x must have dy's type", fn);
    }
    FP8_TRY(check_rows_out(fn, x8, vx8, "x8", vdy.rows, vdy.cols));
    FP8_TRY(check_shape(fn, vdx, "dx", vdy.rows, vdy.cols));
    if (vdx.type != vdy.type) return fail(FP8_ERR_ARG, "%s: dx must have dy's type", fn);
    FP8_TRY(check_type(fn, wtype, "gamma"));
    FP8_TRY(check_param(fn, gamma, wtype, "gamma"));
    const bool empty = vdy.rows == 0;
    FP8_TRY(check_scalar(fn, mean, "mean", empty));
    FP8_TRY(check_scalar(fn, rstd, "rstd", empty));
    FP8_TRY(check_scalar(fn, dgamma, "dgamma", false));
    FP8_TRY(check_scalar(fn, dbeta, "dbeta", false));
    FP8_TRY(check_ptr(fn, workspace, "workspace", empty));
    const int64_t need = fp8_layernorm_bwd_workspace(vdy.rows, vdy.cols);
    if (workspace_bytes < need)
        return fail(FP8_ERR_ARG, "%s: workspace of %lld bytes, %lld are needed", fn,
                    static_cast<long long>(workspace_bytes), static_cast<long long>(need));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_ln_bwd(vdy, vx, vx8, gamma, wtype, mean, rstd, vdx, dgamma, dbeta,
                                 workspace, sms, static_cast<cudaStream_t>(stream)),
             fn);
    return FP8_OK;
}

fp8_status fp8_layernorm_recompute(const fp8_block_tensor *x8, const void *gamma,
                                   const void *beta, int32_t wtype, const float *mean,
                                   const float *rstd, const fp8_block_tensor *yt, void *stream) {
    const char *fn = "fp8_layernorm_recompute";
    const fp8k::CallRange range(fn);
    fp8k::BlockView vx8, vyt;
    FP8_TRY(view(fn, x8, "x8", false, &vx8));
    FP8_TRY(view(fn, yt, "yt", false, &vyt));
    FP8_TRY(check_rows_out(fn, x8, vx8, "x8", vx8.rows, vx8.cols));
    FP8_TRY(check_rows_out(fn, yt, vyt, "yt", vx8.cols, vx8.rows));
    FP8_TRY(check_type(fn, wtype, "gamma"));
    FP8_TRY(check_param(fn, gamma, wtype, "gamma"));
    FP8_TRY(check_param(fn, beta, wtype, "beta"));
    const bool empty = vx8.rows == 0 || vx8.cols == 0;
    FP8_TRY(check_scalar(fn, mean, "mean", empty));
    FP8_TRY(check_scalar(fn, rstd, "rstd", empty));
    FP8_TRY(check_tiles(fn, vx8.rows, vx8.cols));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_ln_recompute(vx8, gamma, beta, wtype, mean, rstd, vyt, sms,
                                       static_cast<cudaStream_t>(stream)),
             fn);
    return FP8_OK;
}

fp8_status fp8_swiglu_fwd(const fp8_matrix *h, const fp8_block_tensor *a8,
                          const fp8_block_tensor *h8, void *stream) {
    const char *fn = "fp8_swiglu_fwd";
    const fp8k::CallRange range(fn);
    fp8k::MatView vh;
    fp8k::BlockView va8, vh8;
    FP8_TRY(view(fn, h, "h", false, &vh));
    FP8_TRY(view(fn, a8, "a8", false, &va8));
    FP8_TRY(view(fn, h8, "h8", true, &vh8));
    if (vh.cols % 256)
        return fail(FP8_ERR_ALIGN, "%s: h has %lld columns: half of them must be a multiple of 128",
                    fn, static_cast<long long>(vh.cols));
    FP8_TRY(check_rows_out(fn, a8, va8, "a8", vh.rows, vh.cols / 2));
    FP8_TRY(check_rows_out(fn, h8, vh8, "h8", vh.rows, vh.cols));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_swiglu_fwd(vh, va8, vh8, sms, static_cast<cudaStream_t>(stream)), fn);
    return FP8_OK;
}

fp8_status fp8_swiglu_bwd(const fp8_matrix *da, const fp8_block_tensor *h8,
                          const fp8_block_tensor *dh8, const fp8_block_tensor *dh8t,
                          const fp8_block_tensor *a8t, void *stream) {
    const char *fn = "fp8_swiglu_bwd";
    const fp8k::CallRange range(fn);
    fp8k::MatView vda;
    fp8k::BlockView vh8, vdh8, vdh8t, va8t;
    FP8_TRY(view(fn, da, "da", false, &vda));
    FP8_TRY(view(fn, h8, "h8", false, &vh8));
    FP8_TRY(view(fn, dh8, "dh8", true, &vdh8));
    FP8_TRY(view(fn, dh8t, "dh8t", true, &vdh8t));
    FP8_TRY(view(fn, a8t, "a8t", true, &va8t));
    const int64_t M = vda.rows, F = vda.cols;
    if (F % 128)
        return fail(FP8_ERR_ALIGN, "%s: da has %lld columns: they must be a multiple of 128", fn,
                    static_cast<long long>(F));
    if (dh8 == nullptr && dh8t == nullptr && a8t == nullptr)
        return fail(FP8_ERR_ARG, "%s: dh8, dh8t and a8t are all NULL", fn);
    FP8_TRY(check_rows_out(fn, h8, vh8, "h8", M, 2 * F));
    FP8_TRY(check_rows_out(fn, dh8, vdh8, "dh8", M, 2 * F));
    FP8_TRY(check_rows_out(fn, dh8t, vdh8t, "dh8t", 2 * F, M));
    FP8_TRY(check_rows_out(fn, a8t, va8t, "a8t", F, M));
    if (dh8 != nullptr && dh8t != nullptr && vdh8.fmt != vdh8t.fmt)
        return fail(FP8_ERR_ARG, "%s: dh8 and dh8t differ in format", fn);
    FP8_TRY(check_tiles(fn, M, F));
    int sms;
    FP8_TRY(current_device(&sms));
    FP8_CUDA(fp8k::launch_swiglu_bwd(vda, vh8, vdh8, vdh8t, va8t, sms,
                                     static_cast<cudaStream_t>(stream)),
             fn);
    return FP8_OK;
}

}  // extern "C"
