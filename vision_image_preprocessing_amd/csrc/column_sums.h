// column_sums.h -- the last step of sums over rows: every workgroup of a
// kernel over rows leaves its partial sum of each column, and these are added
// up in a fixed order, so that no atomics are needed, and in float64, which
// takes 0.1 us at most: where a workgroup has few rows, this is where most of a
// float32 sum's error would come from (4099 rows over 1024 workgroups: 1.1e-7
// of the sums, 0.44e-7 with float64 here; 131072 over 1536, whose own float32
// sums are 85 rows long: 1.9e-7 and 1.6e-7).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

namespace mimo {
namespace {

constexpr int kSumColumns = 32, kSumParts = 32;  // of the workgroup
constexpr int kMaxSums = 3;                      // of a launch

// out[c] = the sum over g of part[g * stride + c], for `columns` columns.
struct ColumnSum {
    const float *part;
    float *out;
    int64_t stride, columns;
    int32_t groups;
    int32_t first;  // of its workgroups
};
struct ColumnSums {
    ColumnSum of[kMaxSums];
    int32_t count, workgroups;
    ColumnSums() { std::memset(this, 0, sizeof(*this)); }
    void add(const float *part, int32_t groups, int64_t stride, int64_t columns, float *out) {
        of[count++] = ColumnSum{part, out, stride, columns, groups, workgroups};
        workgroups += int32_t((columns + kSumColumns - 1) / kSumColumns);
    }
};

// 1536 sums of 1280 columns, 8 MB: 5.4 to 7.0 us; 256 of two times 5120 and 128 of
// 1280 6.3 to 7.0 (16 columns a workgroup 6.4 to 7.0 and 9.5, 8 columns 8 and 12.5).
__global__ __launch_bounds__(kSumColumns *kSumParts) void column_sums_kernel(ColumnSums a) {
    __shared__ double lds[kSumParts][kSumColumns + 1];
    int n = 0;
    while (n + 1 < a.count && int(blockIdx.x) >= a.of[n + 1].first) ++n;
    const ColumnSum s = a.of[n];
    const int column = threadIdx.x % kSumColumns, first = threadIdx.x / kSumColumns;
    const int64_t c = int64_t(int(blockIdx.x) - s.first) * kSumColumns + column;
    double v = 0.0;
    if (c < s.columns) {
#pragma unroll 8
        for (int g = first; g < s.groups; g += kSumParts) v += double(s.part[int64_t(g) * s.stride + c]);
    }
    lds[first][column] = v;
    __syncthreads();
#pragma unroll
    for (int n = kSumParts / 2; n > 0; n >>= 1) {
        if (first < n) lds[first][column] += lds[first + n][column];
        __syncthreads();
    }
    if (first == 0 && c < s.columns) s.out[c] = float(lds[0][column]);
}

// The launches made.
inline int launch_column_sums(const ColumnSums &sums, hipStream_t stream) {
    if (!sums.count) return 0;
    hipLaunchKernelGGL(column_sums_kernel, dim3(unsigned(sums.workgroups), 1, 1), dim3(kSumColumns * kSumParts, 1, 1), 0, stream, sums);
    return 1;
}

}  // namespace
}  // namespace mimo
