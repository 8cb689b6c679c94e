// overlap.h against a table of bytes: random areas of few rows, with equal and different
// pitches, side by side, between each other's rows and across each other.
#include <cstdio>
#include <random>
#include <vector>

#include "overlap.h"

static bool by_bytes(const fp8k::Area &a, const fp8k::Area &b) {
    std::vector<char> taken(4096);
    for (int64_t r = 0; r < a.rows; ++r)
        for (int64_t c = 0; c < a.width; ++c) taken[a.at - 1000 + r * a.pitch + c] = 1;
    for (int64_t r = 0; r < b.rows; ++r)
        for (int64_t c = 0; c < b.width; ++c)
            if (taken[b.at - 1000 + r * b.pitch + c]) return true;
    return false;
}

int main() {
    std::mt19937 g(1);
    const auto to = [&g](int n) { return static_cast<int64_t>(g() % n); };
    int met = 0, between = 0;
    for (int i = 0; i < 1000000; ++i) {
        const int64_t p = 1 + to(40), q = to(2) ? p : 1 + to(40);
        const auto at = [](int64_t n) { return reinterpret_cast<const void *>(1000 + n); };
        const fp8k::Area a = fp8k::area("a", at(to(120)), to(9), to(p + 1), p, false);
        const fp8k::Area b = fp8k::area("b", at(to(120)), to(9), to(q + 1), q, false);
        const bool want = by_bytes(a, b);
        if (fp8k::meet(a, b) != want || fp8k::meet(b, a) != want) {
            std::printf("%lld: %lld x %lld pitch %lld, %lld: %lld x %lld pitch %lld: %d\n", (long long)a.at, (long long)a.rows,
                        (long long)a.width, (long long)a.pitch, (long long)b.at, (long long)b.rows, (long long)b.width,
                        (long long)b.pitch, want);
            return 1;
        }
        met += want;
        between += !want && a.rows > 0 && b.rows > 0 && a.at < b.at && a.at + (a.rows - 1) * a.pitch > b.at;
    }
    if (met < 100000 || between < 10000) {
        std::printf("%d met, %d between each other's rows\n", met, between);
        return 1;
    }
    return 0;
}
