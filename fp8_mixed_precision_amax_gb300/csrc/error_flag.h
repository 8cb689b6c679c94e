// error_flag.h -- a file's device error flags, which its kernels set when a bounded wait
// gives up: read on the host, and cleared.
#pragma once

#include <cuda_runtime_api.h>

namespace fp8k {

// symbol: an unsigned in device memory.  It is written only where it was set: fp8_sync_status
// asks for seven of them (66 us, and 92 with a copy back for each), and a flag that another
// stream's kernel sets after it was read stays for the next call.
inline cudaError_t take_error_flags(const void *symbol, unsigned *flags) {
    *flags = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(flags, symbol, sizeof *flags, 0, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess || *flags == 0) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(symbol, &zero, sizeof zero, 0, cudaMemcpyHostToDevice);
}

}  // namespace fp8k
