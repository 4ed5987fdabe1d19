// rows.cu -- sums over rows of partial results, in a fixed order.
#include "rows.cuh"

namespace pararnn {
namespace {

// A CTA takes 32 columns; its eight warps take every eighth row, and meet in row order.
__global__ void __launch_bounds__(256) rows_sum_kernel(const float *part, float *out, long long rows, long long width,
                                                       long long stride) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x % 32, k = threadIdx.x / 32;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
    float sum = 0.f;
    if (c < width)
        for (long long r = k; r < rows; r += 8) sum += part[r * stride + c];
    s[k][lane] = sum;
    __syncthreads();
    if (k == 0 && c < width) {
        for (int i = 1; i < 8; ++i) sum += s[i][lane];
        out[c] = sum;
    }
}

}  // namespace

cudaError_t launch_rows_sum(const float *part, float *out, long long rows, long long width, long long stride, cudaStream_t s) {
    if (out == nullptr) return cudaSuccess;
    rows_sum_kernel<<<static_cast<unsigned>((width + 31) / 32), 256, 0, s>>>(part, out, rows, width, stride);
    return cudaGetLastError();
}

}  // namespace pararnn
