// overlap.h -- whether arguments of a call share memory: host arithmetic without CUDA.
#pragma once

#include <cstdint>

namespace fp8k {

// Memory of an argument: rows of `width` bytes, `pitch` bytes apart.  None: no rows.
struct Area {
    const char *name;
    uintptr_t at;
    int64_t rows, width, pitch;
    bool replace;   // an output that may take the very place of an input which says so too
};
inline Area area(const char *name, const void *p, int64_t rows, int64_t width, int64_t pitch, bool replace) {
    if (p == nullptr || width <= 0 || rows <= 0) return {name, 0, 0, 0, 1, false};
    return {name, reinterpret_cast<uintptr_t>(p), rows, width, rows == 1 ? width : pitch, replace};
}
inline Area area(const char *name, const void *p, int64_t bytes) { return area(name, p, 1, bytes, bytes, false); }

// Whether two areas have a byte in common; rows may lie between each other's.
inline bool meet(const Area &a, const Area &b) {
    if (a.rows == 0 || b.rows == 0) return false;
    const uintptr_t end_a = a.at + (a.rows - 1) * a.pitch + a.width, end_b = b.at + (b.rows - 1) * b.pitch + b.width;
    if (end_a <= b.at || end_b <= a.at) return false;
    const int64_t d = static_cast<int64_t>(b.at - a.at);
    if (a.pitch == b.pitch) {
        // row i of a and j of b, k = i - j: d - a.width < k pitch < d + b.width
        const int64_t n = d - a.width, p = a.pitch;
        int64_t k = (n >= 0 ? n / p : -((-n + p - 1) / p)) + 1;   // the first k past the lower bound
        if (k < -(b.rows - 1)) k = -(b.rows - 1);
        return k <= a.rows - 1 && k * p < d + b.width;
    }
    const Area &few = a.rows <= b.rows ? a : b, &many = a.rows <= b.rows ? b : a;
    for (int64_t i = 0; i < few.rows; ++i) {
        // the last row of `many` that begins before this one's end
        const int64_t last = static_cast<int64_t>(few.at - many.at) + i * few.pitch + few.width - 1;
        if (last < 0) continue;
        const int64_t j = last / many.pitch < many.rows ? last / many.pitch : many.rows - 1;
        if (j * many.pitch + many.width > last - few.width + 1) return true;
    }
    return false;
}
inline bool same_place(const Area &a, const Area &b) {
    return a.replace && b.replace && a.at == b.at && a.rows == b.rows && a.width == b.width && a.pitch == b.pitch;
}

}  // namespace fp8k
