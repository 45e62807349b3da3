// Sums the rows of a matrix of partial results.  Memory bound: each partial is read once.
// A CTA takes 16 columns; its 64 half-warps take every 64th row each, eight loads in flight, and
// join through shared memory, so the order of the additions depends on P alone.
#include "layer_common.cuh"

namespace qd {
namespace {

constexpr int kRows = 64, kCols = 16;

__global__ void __launch_bounds__(kCols * kRows) sum_rows_kernel(const float *part, int P, int64_t M, float *out1,
                                                              int64_t M1, float *out2, int64_t M2, float *out3) {
    __shared__ float s[kRows][kCols + 1];
    const int lane = threadIdx.x % kCols, row = threadIdx.x / kCols;
    const int64_t m = (int64_t)blockIdx.x * kCols + lane;
    float acc = 0.f;
    if (m < M) {
#pragma unroll 8
        for (int p = row; p < P; p += kRows) acc += part[p * M + m];
    }
    s[row][lane] = acc;
    __syncthreads();
#pragma unroll
    for (int half = kRows / 2; half >= 4; half /= 2) {
        if (row < half) s[row][lane] += s[row + half][lane];
        __syncthreads();
    }
    if (row == 0 && m < M) {
        const float t = (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]);
        if (m < M1) {
            if (out1) out1[m] = t;
        } else if (m < M1 + M2) {
            if (out2) out2[m - M1] = t;
        } else if (out3) {
            out3[m - M1 - M2] = t;
        }
    }
}

}  // namespace

cudaError_t launch_sum_rows(const float *part, int P, int64_t M, float *out1, int64_t M1, float *out2, int64_t M2,
                            float *out3, cudaStream_t s, int *nlaunch) {
    if (M == 0) return cudaSuccess;
    sum_rows_kernel<<<(unsigned)((M + kCols - 1) / kCols), kCols * kRows, 0, s>>>(part, P, M, out1, M1, out2, M2, out3);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace qd
