// rows.cuh -- vectors of elements from and to rows of fp32 or bf16, and sums over rows of partial results.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace pararnn {
namespace rows {

// V consecutive elements as fp32 (V = 4: aligned to four of them)
template <int V>
__device__ __forceinline__ void load(const float *p, float (&v)[V]) {
    if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        v[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[V]) {
    if constexpr (V == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void store(float *p, const float (&v)[V]) {
    if constexpr (V == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *p = v[0];
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[V]) {
    if constexpr (V == 4) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
    } else {
        *p = __float2bfloat16(v[0]);
    }
}
// the same where the type is known at run time only (uniform over the grid)
template <int V>
__device__ __forceinline__ void load(const void *p, long long at, bool f32, float (&v)[V]) {
    if (f32) load<V>(static_cast<const float *>(p) + at, v);
    else load<V>(static_cast<const __nv_bfloat16 *>(p) + at, v);
}
template <int V>
__device__ __forceinline__ void store(void *p, long long at, bool f32, const float (&v)[V]) {
    if (f32) store<V>(static_cast<float *>(p) + at, v);
    else store<V>(static_cast<__nv_bfloat16 *>(p) + at, v);
}

__device__ __forceinline__ int count(const int *lengths, int b, int T) {
    if (lengths == nullptr) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace rows

// Sums over the rows of part [rows, width], in a fixed order: the columns go one output after the other to out[i] [n[i]]
// (the n add up to width); nothing where an output is null.
struct RowsSum {
    const float *part;
    long long rows, width;
    float *out[3];
    long long n[3];
};
cudaError_t launch_rows_sum(const RowsSum &a, cudaStream_t s);

}  // namespace pararnn
