// rows.cu -- sums over rows of partial results, in a fixed order.
#include "rows.cuh"

namespace pararnn {
namespace {

// A CTA takes 32 columns; its 32 warps take every 32nd row, four at a time, and meet in order.  Few columns leave few CTAs, so
// the rows of one column go over many warps (592 rows of 4096 columns: 18 us a launch with eight warps to a CTA).
__global__ void __launch_bounds__(1024) rows_sum_kernel(const RowsSum a) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x % 32, k = threadIdx.x / 32;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
    float sum = 0.f;
    if (c < a.width) {
        const float *p = a.part + c;
        long long r = k;
        while (r + 96 < a.rows) {  // pieces of 64 rows: one long chain would lose digits
            float piece = 0.f;
            for (int j = 0; j < 16 && r + 96 < a.rows; ++j, r += 128) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = p[(r + 32 * i) * a.width];
                piece += (v[0] + v[1]) + (v[2] + v[3]);
            }
            sum += piece;
        }
        for (; r < a.rows; r += 32) sum += p[r * a.width];
    }
    s[k][lane] = sum;
    __syncthreads();
    // column k, part `lane`
    sum = s[lane][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    long long to = static_cast<long long>(blockIdx.x) * 32 + k;
    if (lane != 0 || to >= a.width) return;
    int i = 0;
    while (i < 2 && to >= a.n[i]) to -= a.n[i++];
    if (a.out[i] != nullptr) a.out[i][to] = sum;
}

}  // namespace

cudaError_t launch_rows_sum(const RowsSum &a, cudaStream_t s) {
    if (a.out[0] == nullptr && a.out[1] == nullptr && a.out[2] == nullptr) return cudaSuccess;
    rows_sum_kernel<<<static_cast<unsigned>((a.width + 31) / 32), 1024, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace pararnn
