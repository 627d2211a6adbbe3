// Sums over the rows of fp32 partial results: the second half of a gradient of what all
// tokens share, whose blocks leave a row each in the workspace.
#pragma once

#include "mixer.cuh"
#include "sm100_ptx.cuh"

namespace gdn {

constexpr int kColumnLanes = 32, kColumnRows = 32;

// part [rows, cols] -> first[0 .. split), second[0 .. cols - split); either may be NULL. A
// thread adds every blockDim.y-th row of one column, then a part of a warp adds a column's sums.
// Launched while the kernel before it still runs, whose end it waits for.
static __global__ void __launch_bounds__(kColumnLanes * kColumnRows)
    gdn_column_sums_kernel(const float *part, int rows, int64_t cols, int64_t split, float *first, float *second) {
    __shared__ float sums[kColumnRows][kColumnLanes + 1];
    const int64_t first_column = static_cast<int64_t>(blockIdx.x) * kColumnLanes, mine = first_column + threadIdx.x;
    ptx::griddep_wait();
    float s = 0.f;
    if (mine < cols)
#pragma unroll 8
        for (int r = threadIdx.y; r < rows; r += blockDim.y) s += part[r * cols + mine];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    // blockDim.y (a power of two) lanes to a column, as many columns as a warp has such parts
    const int y = blockDim.y, shift = __ffs(y) - 1;
    const int of = threadIdx.y * (kColumnLanes >> shift) + (threadIdx.x >> shift);
    s = sums[threadIdx.x & (y - 1)][of];
    for (int o = y / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t c = first_column + of;
    if ((threadIdx.x & (y - 1)) != 0 || c >= cols) return;
    if (c < split) {
        if (first) first[c] = s;
    } else if (second) {
        second[c - split] = s;
    }
}

// About eight rows to a thread: 64 rows of 40960 columns 12.0 us with two.
static inline cudaError_t column_sums(const float *part, int rows, int64_t cols, int64_t split, float *first,
                                      float *second, cudaStream_t s) {
    unsigned y = 1;
    while (y < kColumnRows && y * 8 < static_cast<unsigned>(rows)) y *= 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((cols + kColumnLanes - 1) / kColumnLanes));
    cfg.blockDim = dim3(kColumnLanes, y);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_column_sums_kernel, part, rows, cols, split, first, second);
}

}  // namespace gdn
