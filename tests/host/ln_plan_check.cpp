// ln_plan.h: LayerNorm's backward never starts more CTAs than are resident, and never more
// than its workspace, which is sized without a device, has parts for.
#include <cstdio>
#include <initializer_list>

#include "ln_plan.h"

#define CHECK(x)                                                                               \
    do {                                                                                       \
        if (!(x)) {                                                                            \
            std::printf("line %d: %s (rows %lld, cols %lld, sms %lld)\n", __LINE__, #x, rows, cols, sms); \
            return 1;                                                                          \
        }                                                                                      \
    } while (0)

int main() {
    using namespace fp8k;
    for (long long cols : {1, 511, 512, 513, 1024, 2048, 2049, 4096, 4608, 4609, 8192, 8193, 40000})
        for (long long rows : {1, 2, 7, 8, 9, 100, 152, 153, 1000, 1216, 1217, 2432, 5003, 8192, 1000000}) {
            long long before = 0;
            for (long long sms : {1, 2, 64, 75, 76, 132, 148, 151, 152, 153, 160, 1000}) {
                const long long n = bwd_ctas(rows, cols, sms);
                const long long per_sm = cols <= kBwdNarrow ? 2
                                         : cols > kBwdWide  ? 1
                                                            : ring_ctas_per_sm(row_threads(cols, 16));
                CHECK(n >= 1 && n <= rows);
                CHECK(n <= per_sm * sms);               // all resident
                CHECK(n <= bwd_ctas_most(rows, cols));  // all have a part of the workspace
                CHECK(n >= before);
                before = n;
            }
            const long long sms = 152;
            CHECK(bwd_ctas(rows, cols, sms) == bwd_ctas_most(rows, cols));
        }
    return 0;
}
