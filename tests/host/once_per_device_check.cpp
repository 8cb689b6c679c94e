// once_per_device.h with a CUDA runtime of two functions that count: set-up runs once on
// each device, again after a failure, and never for another device's sake.
#include <cstdio>
#include <initializer_list>

#include "once_per_device.h"

static int g_device = 0, g_set[64] = {}, g_fail = 0;
static const void *g_last = nullptr;
static int g_last_bytes = 0;

extern "C" cudaError_t cudaGetDevice(int *device) {
    *device = g_device;
    return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void *func, cudaFuncAttribute, int value) {
    if (g_fail > 0) {
        --g_fail;
        return cudaErrorMemoryAllocation;
    }
    if (g_device < 64) ++g_set[g_device];
    g_last = func;
    g_last_bytes = value;
    return cudaSuccess;
}

static void kernel_a(int) {}
static void kernel_b(int) {}

#define CHECK(x)                                             \
    do {                                                     \
        if (!(x)) {                                          \
            std::printf("line %d: %s\n", __LINE__, #x);      \
            return 1;                                        \
        }                                                    \
    } while (0)

int main() {
    static fp8k::SmemLimit a, b;
    for (int i = 0; i < 3; ++i) CHECK(a.allow(kernel_a, 100000) == cudaSuccess);
    CHECK(g_set[0] == 1 && g_last == reinterpret_cast<const void *>(kernel_a) && g_last_bytes == 100000);
    CHECK(b.allow(kernel_b, 5) == cudaSuccess && g_set[0] == 2);   // another kernel's own
    g_device = 1;
    for (int i = 0; i < 3; ++i) CHECK(a.allow(kernel_a, 100000) == cudaSuccess);
    CHECK(g_set[1] == 1 && g_set[0] == 2);
    g_device = 63, g_fail = 2;   // two failures, which are nobody else's and not for good
    CHECK(a.allow(kernel_a, 100000) == cudaErrorMemoryAllocation);
    g_device = 1;
    CHECK(a.allow(kernel_a, 100000) == cudaSuccess && g_set[1] == 1);
    g_device = 63;
    CHECK(a.allow(kernel_a, 100000) == cudaErrorMemoryAllocation);
    CHECK(a.allow(kernel_a, 100000) == cudaSuccess && g_set[63] == 1);
    CHECK(a.allow(kernel_a, 100000) == cudaSuccess && g_set[63] == 1);
    g_device = 64;
    CHECK(a.allow(kernel_a, 100000) == cudaErrorInvalidDevice);
    static fp8k::OncePerDevice once;
    int runs = 0, device = -1;
    for (int d : {3, 2, 3, 2}) {
        g_device = d;
        CHECK(once.run([&](int dev) { runs += dev == d; return cudaSuccess; }, &device) == cudaSuccess);
        CHECK(device == d);
    }
    CHECK(runs == 2);
    return 0;
}
