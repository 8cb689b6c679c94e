// ln_plan.h -- how LayerNorm's launches are cut: host arithmetic without CUDA.
#pragma once

#include <cstdint>

namespace fp8k {

constexpr int kWarps = 8;   // warps of a CTA whose warps have a row each

inline unsigned capped(int64_t n, int64_t cap) { return static_cast<unsigned>(n < cap ? n : cap); }

// Threads of a CTA that shares a row: whole warps, `each` columns per thread.
inline unsigned row_threads(int64_t cols, int each) {
    return static_cast<unsigned>((cols + 32 * each - 1) / (32 * each) * 32);
}

constexpr int64_t kBwdNarrow = 512;   // rows up to this belong to one warp
constexpr int64_t kBwdWide = 8192;    // rows up to this are held in a CTA's registers
constexpr int64_t kBwdSlab = 4096;    // columns of a wide row's slab, 16 for each of 256 threads

// CTAs per SM of the ring kernel: of up to 288 threads (4608 columns) two fit beside
// each other, smaller ones by threads.  Two of 256 threads have 128 registers each, two of
// 288 only 96, since their 18 warps put five on one of the SM's four schedulers (8192 x
// 4096: 41.0 us, and 50.8 with the 96 of the larger one).  8192 x 4608 with two CTAs and with
// one: from x 55.7 and 56.0 us, from 8 bits 59.3 and 66.8.  Past that, x decides for one: 8192 x
// 5120 (320 threads) with two and with one: from x 59.2 and 57.9, from 8 bits 63.8 and 68.5.
constexpr unsigned kRingHalf = 288;
inline int64_t ring_ctas_per_sm(unsigned threads) {
    return threads > kRingHalf ? 1 : threads > 128 ? 2 : 512 / threads;
}

// CTAs that keep column sums of their own: as many as are resident on `sms` SMs at most; one
// per SM and slab of a wide row.  It only grows with sms, up to those of kBwdSms SMs, for
// which the workspace is sized without asking a device.
constexpr int64_t kBwdSms = 152;
inline int64_t bwd_ctas(int64_t rows, int64_t cols, int64_t sms, int64_t narrow = kBwdNarrow,
                        int narrow_ctas = 2) {
    if (sms > kBwdSms) sms = kBwdSms;
    if (cols <= narrow) return capped((rows + kWarps - 1) / kWarps, narrow_ctas * sms);
    if (cols > kBwdWide) return capped(rows, sms);
    // eight rows each once there is a CTA per SM: every CTA's sums are written, read and
    // added (2048 x 1024: 18.7 us with 1216 CTAs)
    const int64_t some = rows / 8 > sms ? rows / 8 : sms;
    const int64_t most = sms * ring_ctas_per_sm(row_threads(cols, 16));
    return capped(rows, some < most ? some : most);
}
inline int64_t bwd_ctas_most(int64_t rows, int64_t cols) { return bwd_ctas(rows, cols, kBwdSms); }

}  // namespace fp8k
