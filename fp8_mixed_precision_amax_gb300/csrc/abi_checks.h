// abi_checks.h -- argument checks and error reporting shared by the files that
// export C entry points (abi.cu, block_abi.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "../../include/fp8amax.h"
#include "kernels.h"

namespace {

inline fp8_status fail(fp8_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    fp8k::set_last_error(buf);
    return s;
}

inline fp8_status cuda_fail(cudaError_t e, const char *where) {
    return fail(FP8_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    int sm_count = 0;
    bool supported = false;
};
DeviceInfo g_dev[kMaxDevices];
std::once_flag g_dev_once[kMaxDevices];

// SM count of the current device; FP8_ERR_UNSUPPORTED unless it is an sm_103 GPU.
inline fp8_status current_device(int *sm_count) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(FP8_ERR_UNSUPPORTED, "device index %d", dev);
    std::call_once(g_dev_once[dev], [dev] {
        int major = 0, minor = 0, sms = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        g_dev[dev].sm_count = sms;
        g_dev[dev].supported = (major == 10 && minor == 3);
    });
    if (!g_dev[dev].supported)
        return fail(FP8_ERR_UNSUPPORTED, "device %d is not an sm_103 GPU", dev);
    *sm_count = g_dev[dev].sm_count;
    return FP8_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline fp8_status check_dims16(const char *fn, int64_t a, const char *na, int64_t b, const char *nb) {
    if (a < 0 || b < 0) return fail(FP8_ERR_ARG, "%s: negative size (%s=%lld, %s=%lld)", fn, na,
                                    (long long)a, nb, (long long)b);
    if (a % 16 || b % 16)
        return fail(FP8_ERR_ALIGN, "%s: %s=%lld and %s=%lld must be multiples of 16", fn, na,
                    (long long)a, nb, (long long)b);
    if (a > (int64_t(1) << 31) || b > (int64_t(1) << 31))
        return fail(FP8_ERR_ARG, "%s: dimension above 2^31", fn);
    return FP8_OK;
}

inline fp8_status check_ptr(const char *fn, const void *p, const char *name, bool may_be_null) {
    if (p == nullptr) {
        if (may_be_null) return FP8_OK;
        return fail(FP8_ERR_ARG, "%s: %s is NULL", fn, name);
    }
    if (!aligned16(p)) return fail(FP8_ERR_ALIGN, "%s: %s is not 16-byte aligned", fn, name);
    return FP8_OK;
}

// A pointer to one fp32 scalar (scale, scale_inv, amax) needs 4-byte alignment.
inline fp8_status check_scalar(const char *fn, const void *p, const char *name, bool may_be_null) {
    if (p == nullptr) {
        if (may_be_null) return FP8_OK;
        return fail(FP8_ERR_ARG, "%s: %s is NULL", fn, name);
    }
    if (reinterpret_cast<uintptr_t>(p) & 3u)
        return fail(FP8_ERR_ALIGN, "%s: %s is not 4-byte aligned", fn, name);
    return FP8_OK;
}

#define FP8_TRY(expr)                       \
    do {                                    \
        fp8_status s_ = (expr);             \
        if (s_ != FP8_OK) return s_;        \
    } while (0)

#define FP8_CUDA(expr, where)                          \
    do {                                               \
        cudaError_t e_ = (expr);                       \
        if (e_ != cudaSuccess) return cuda_fail(e_, where); \
    } while (0)

}  // namespace
