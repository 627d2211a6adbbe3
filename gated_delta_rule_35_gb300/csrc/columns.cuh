// Sums over the rows of fp32 partial results: the second half of a gradient of what all
// tokens share, whose blocks leave a row each in the workspace.
#pragma once

#include "mixer.cuh"
#include "sm100_ptx.cuh"

namespace gdn {

constexpr int kColumnLanes = 32, kColumnRows = 32;

// part [rows, cols] -> first[0 .. split), second[0 .. cols - split); either may be NULL. A
// thread adds every kColumnRows-th row of one column, then those sums are added in order.
static __global__ void __launch_bounds__(kColumnLanes * kColumnRows)
    gdn_column_sums_kernel(const float *part, int rows, int64_t cols, int64_t split, float *first, float *second) {
    __shared__ float sums[kColumnRows][kColumnLanes];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kColumnLanes + threadIdx.x;
    float s = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int r = threadIdx.y; r < rows; r += kColumnRows) s += part[r * cols + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || c >= cols) return;
#pragma unroll
    for (int r = 1; r < kColumnRows; ++r) s += sums[r][threadIdx.x];
    if (c < split) {
        if (first) first[c] = s;
    } else if (second) {
        second[c - split] = s;
    }
}

static inline cudaError_t column_sums(const float *part, int rows, int64_t cols, int64_t split, float *first,
                                      float *second, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>((cols + kColumnLanes - 1) / kColumnLanes);
    gdn_column_sums_kernel<<<blocks, dim3(kColumnLanes, kColumnRows), 0, s>>>(part, rows, cols, split, first,
                                                                              second);
    return cudaGetLastError();
}

}  // namespace gdn
