// error_flag.h with a CUDA runtime of two functions that count: a flag that is not set costs
// one copy, and nothing is written that a kernel could have set meanwhile.
#include <cstdio>
#include <cstring>

#include "error_flag.h"

static int g_reads = 0, g_writes = 0;
static unsigned g_late = 0;   // what a kernel sets right after the read
static cudaError_t g_read_error = cudaSuccess, g_write_error = cudaSuccess;

extern "C" cudaError_t cudaMemcpyFromSymbol(void *to, const void *symbol, size_t bytes, size_t at, cudaMemcpyKind) {
    ++g_reads;
    if (g_read_error != cudaSuccess) return g_read_error;
    std::memcpy(to, static_cast<const char *>(symbol) + at, bytes);
    *static_cast<unsigned *>(const_cast<void *>(symbol)) |= g_late;
    return cudaSuccess;
}
extern "C" cudaError_t cudaMemcpyToSymbol(const void *symbol, const void *from, size_t bytes, size_t at, cudaMemcpyKind) {
    ++g_writes;
    if (g_write_error != cudaSuccess) return g_write_error;
    std::memcpy(static_cast<char *>(const_cast<void *>(symbol)) + at, from, bytes);
    return cudaSuccess;
}

#define CHECK(x)                                             \
    do {                                                     \
        if (!(x)) {                                          \
            std::printf("line %d: %s\n", __LINE__, #x);      \
            return 1;                                        \
        }                                                    \
    } while (0)

int main() {
    static unsigned symbol = 0;
    unsigned got = 7;
    CHECK(fp8k::take_error_flags(&symbol, &got) == cudaSuccess && got == 0);
    CHECK(g_reads == 1 && g_writes == 0);
    symbol = 5;
    CHECK(fp8k::take_error_flags(&symbol, &got) == cudaSuccess && got == 5 && symbol == 0);
    CHECK(g_reads == 2 && g_writes == 1);
    g_late = 1;   // set between the read and what follows it: told by the next call
    CHECK(fp8k::take_error_flags(&symbol, &got) == cudaSuccess && got == 0 && symbol == 1);
    g_late = 0;
    CHECK(fp8k::take_error_flags(&symbol, &got) == cudaSuccess && got == 1 && symbol == 0);
    got = 9;
    g_read_error = cudaErrorInvalidValue;
    CHECK(fp8k::take_error_flags(&symbol, &got) == cudaErrorInvalidValue && got == 0);
    g_read_error = cudaSuccess, g_write_error = cudaErrorInvalidValue, symbol = 3;
    CHECK(fp8k::take_error_flags(&symbol, &got) == cudaErrorInvalidValue && got == 3);
    return 0;
}
