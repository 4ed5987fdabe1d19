// api_checks.cuh -- what the C entry points of the sequence-layer operators check alike, and how they lay workspaces out.
#pragma once

#include <cstddef>
#include <cstdint>

#include "solver.cuh"

namespace pararnn {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Extent {  // bytes [p, p + n) that a call touches
    const void *p;
    size_t n;
};
inline bool overlaps(const Extent &a, const Extent &b) {
    const auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return a.n && b.n && a.p && b.p && pa < pb + b.n && pb < pa + a.n;
}
// no output overlaps another output or an input
inline bool disjoint(const Extent *out, int n_out, const Extent *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return false;
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i], in[j])) return false;
    }
    return true;
}

// What the size queries answer where a call needs no workspace: it then takes NULL.
constexpr size_t kNone = 1;
inline bool workspace_ok(size_t need, const void *p, size_t bytes) {
    return need == kNone || (need != 0 && p != nullptr && aligned(p, 256) && bytes >= need);
}

inline size_t esize(int dtype) { return dtype == PARARNN_F32 ? 4 : 2; }
inline bool dtype_ok(int d) { return d == PARARNN_F32 || d == PARARNN_BF16; }

// An operand [B, T, heads, width]: aligned to its elements, strides that address forward.
inline bool rows_ok(const pararnn_rows *r, int dtype) {
    return r != nullptr && r->ptr != nullptr && aligned(r->ptr, esize(dtype)) && r->stride_b >= 0 && r->stride_t >= 0 &&
           r->stride_h >= 0;
}
inline Extent extent(const pararnn_rows &r, long long B, long long T, long long heads, long long width, int dtype) {
    const size_t last = (B - 1) * r.stride_b + (T - 1) * r.stride_t + (heads - 1) * r.stride_h + width;
    return {r.ptr, last * esize(dtype)};
}

// Lays a call's workspace out; with no base it only counts.
struct Carve {
    char *base;
    size_t used;
    char *take(size_t n) {
        char *p = base + used;
        used += align256(n);
        return p;
    }
};

}  // namespace pararnn
