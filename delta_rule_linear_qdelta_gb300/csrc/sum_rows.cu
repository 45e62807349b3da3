// Sums the rows of a matrix of partial results.  Memory bound: each partial is read once.
// A CTA takes 32 columns; its `rows` warps take every rows-th row each, eight loads in flight, and
// join through shared memory, so the order of the additions depends on P alone.  Eight warps
// where that leaves a thread at most two rounds of loads (3 MB in 64 rows: 4.7 us, 5.0 with 32),
// else 32 (7 MB in 456 rows: 8 us).
#include "layer_common.cuh"

namespace qd {
namespace {

constexpr int kMostRows = 32;

__global__ void __launch_bounds__(32 * kMostRows) sum_rows_kernel(const float *part, int P, int64_t M, float *out1,
                                                                  int64_t M1, float *out2, int64_t M2, float *out3) {
    __shared__ float s[kMostRows][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, rows = blockDim.x >> 5;
    const int64_t m = (int64_t)blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (m < M) {
#pragma unroll 8
        for (int p = row; p < P; p += rows) acc += part[p * M + m];
    }
    s[row][lane] = acc;
    __syncthreads();
    if (row == 0 && m < M) {
        float t = 0.f;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) t += s[r][lane];
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
    const int rows = P <= 128 ? 8 : kMostRows;
    sum_rows_kernel<<<(unsigned)((M + 31) / 32), 32 * rows, 0, s>>>(part, P, M, out1, M1, out2, M2, out3);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace qd
