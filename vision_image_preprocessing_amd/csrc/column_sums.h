// column_sums.h -- the last step of a sum over rows: every workgroup of a
// kernel over rows leaves its partial sum of each column, and these are added
// up in a fixed order, so that no atomics are needed.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace mimo {
namespace {

constexpr int kSumColumns = 32, kSumParts = 32;  // of the workgroup

// out[c] = the sum over g of part[g * stride + c], for `columns` columns.
__global__ __launch_bounds__(kSumColumns *kSumParts) void column_sums_kernel(const float *part, int32_t groups, int64_t stride,
                                                                             int64_t columns, float *out) {
    __shared__ float lds[kSumParts][kSumColumns + 1];
    const int column = threadIdx.x % kSumColumns, first = threadIdx.x / kSumColumns;
    const int64_t c = int64_t(blockIdx.x) * kSumColumns + column;
    float v = 0.0f;
    if (c < columns) {
#pragma unroll 8
        for (int g = first; g < groups; g += kSumParts) v += part[int64_t(g) * stride + c];
    }
    lds[first][column] = v;
    __syncthreads();
#pragma unroll
    for (int n = kSumParts / 2; n > 0; n >>= 1) {
        if (first < n) lds[first][column] += lds[first + n][column];
        __syncthreads();
    }
    if (first == 0 && c < columns) out[c] = lds[0][column];
}

inline void launch_column_sums(const float *part, int32_t groups, int64_t stride, int64_t columns, float *out, hipStream_t stream) {
    hipLaunchKernelGGL(column_sums_kernel, dim3(unsigned((columns + kSumColumns - 1) / kSumColumns), 1, 1),
                       dim3(kSumColumns * kSumParts, 1, 1), 0, stream, part, groups, stride, columns, out);
}

}  // namespace
}  // namespace mimo
