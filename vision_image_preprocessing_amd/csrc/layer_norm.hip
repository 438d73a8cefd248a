// layer_norm.hip -- layer norm of rows of embeddings and its backward pass
// with the reduction of the weight's and bias's gradients, for AMD Instinct
// MI355X (gfx950).
//
// What is computed, for a row x of n values (the norm of the stock Qwen2-VL
// tower, over embeddings or over whole merge units of four rows):
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   xh = (x - mean) rstd,  out = xh w + b
// and for dout, with g = dout w:
//   dx = rstd (g - sum g / n - xh sum(g xh) / n)
//   dw = sum over rows of dout xh,  db = sum over rows of dout
//
// Everything is float32 inside; inputs and outputs are float32 or bf16, each
// rounded once.  The variance is the sum of squared distances from the mean,
// formed after it from the row in registers, so that a large mean costs no
// precision.
//
// Both kernels are one pass over memory, which bounds them.  A row is held in
// registers by a wave or a workgroup (up to 16384 values); wider rows are
// read again from cache for each sum.  In the backward kernel a wave keeps
// its columns from row to row, so the parameter gradients accumulate in
// registers, over a fixed set of rows; a second kernel adds the workgroups'
// partial sums in a fixed order, and no atomics are needed.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <string>

#include "device_util.h"
#include "internal.h"
#include "row_ops.h"
#include "runtime.h"

namespace mimo {
namespace {

using namespace rows;

constexpr int kMaxWidth = 65536;
constexpr int kSumColumns = 32, kSumParts = 32;  // of the reduction kernel's workgroup

struct NormArgs {
    const void *x, *dout;
    const float *weight, *bias;  // or null
    float *mean, *rstd;          // forward: outputs or null
    void *out;                   // out, or dx
    float *part;                 // [groups][2][width]: dw, db (backward), or null
    int64_t rows;
    int32_t width;
    float eps;
};

// Chunks of eight values: chunk i of a thread is i * kThreads + its number.
// 131072 x 1280 bf16: 133 to 144 us, 0.67 GB at 4.7 to 5.0 TB/s, which is what a
// copy reaches; 4099 x 1283 float32, whose rows start at any value: 11 to 14 us.
template <typename TX, typename TO, bool kRagged, int kThreads, int kChunks>
__global__ __launch_bounds__(kRowWgThreads) void layer_norm_kernel(NormArgs a) {
    __shared__ float lds[2][4];
    const int tid = threadIdx.x % kThreads;
    const int64_t row = row_group() * (kRowWgThreads / kThreads) + threadIdx.x / kThreads;
    if (row >= a.rows) return;  // all of the threads that hold a row
    const TX *x = static_cast<const TX *>(a.x) + row * a.width;
    auto column = [&](int i) { return (i * kThreads + tid) * 8; };
    float v[kChunks][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        if (column(i) < a.width) {
            load_values<kRagged>(x + column(i), a.width - column(i), v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[i][j];
        }
    const float mean = row_sum<kThreads>(sum, lds[0]) / float(a.width);
    float squares = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        if (column(i) < a.width) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = !kRagged || column(i) + j < a.width ? v[i][j] - mean : 0.0f;
                squares = fmaf(v[i][j], v[i][j], squares);
            }
        }
    const float rstd = 1.0f / sqrtf(row_sum<kThreads>(squares, lds[1]) / float(a.width) + a.eps);
    TO *out = static_cast<TO *>(a.out) + row * a.width;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        if (column(i) < a.width) {
            const int left = a.width - column(i);
            float w[8], b[8];
            if (a.weight) load_values<kRagged>(a.weight + column(i), left, w);
            if (a.bias) load_values<kRagged>(a.bias + column(i), left, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= rstd;
                if (a.weight) v[i][j] *= w[j];
                if (a.bias) v[i][j] += b[j];
            }
            store_values<kRagged>(out + column(i), left, v[i]);
        }
    if (tid == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// Rows of any width, one workgroup each, read once for each sum.
template <typename TX, typename TO>
__global__ __launch_bounds__(kRowWgThreads) void layer_norm_wide_kernel(NormArgs a) {
    __shared__ float lds[2][4];
    const int64_t row = row_group();
    if (row >= a.rows) return;
    const TX *x = static_cast<const TX *>(a.x) + row * a.width;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) sum += float(x[c]);
    const float mean = row_sum<256>(sum, lds[0]) / float(a.width);
    float squares = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) {
        const float d = float(x[c]) - mean;
        squares = fmaf(d, d, squares);
    }
    const float rstd = 1.0f / sqrtf(row_sum<256>(squares, lds[1]) / float(a.width) + a.eps);
    TO *out = static_cast<TO *>(a.out) + row * a.width;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) {
        float v = (float(x[c]) - mean) * rstd;
        if (a.weight) v *= a.weight[c];
        if (a.bias) v += a.bias[c];
        out[c] = TO(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// dx of rows first, first + step, ...; partial dw and db of those rows.
// 131072 x 1280 bf16: 220 to 253 us, 1.0 GB at 4.0 to 4.6 TB/s; 4099 x 1283
// float32: 14 to 18 us.
template <typename TX, typename TG, bool kRagged, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads > kRowWgThreads ? kThreads : kRowWgThreads) void layer_norm_backward_kernel(NormArgs a) {
    constexpr int kRows = kThreads < kRowWgThreads ? kRowWgThreads / kThreads : 1;  // rows of the workgroup at a time
    __shared__ float lds[4][kThreads > kRowWgThreads ? kThreads / 64 : 4];
    const int tid = threadIdx.x % kThreads;
    const float inv_n = 1.0f / float(a.width);
    auto column = [&](int i) { return (i * kThreads + tid) * 8; };
    float w[kChunks][8], dw[kChunks][8], db[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = db[i][j] = 0.0f;
            w[i][j] = 1.0f;
        }
        if (a.weight && column(i) < a.width) load_values<kRagged>(a.weight + column(i), a.width - column(i), w[i]);
    }
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kThreads; row < a.rows; row += int64_t(gridDim.x) * kRows, turn ^= 1) {
        const TX *x = static_cast<const TX *>(a.x) + row * a.width;
        const TG *dout = static_cast<const TG *>(a.dout) + row * a.width;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float h[kChunks][8], g[kChunks][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
                load_values<kRagged>(x + column(i), a.width - column(i), h[i]);
                load_values<kRagged>(dout + column(i), a.width - column(i), g[i]);
            }
        // past a ragged row's end dout is zero, and with it every sum
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[i][j] = (h[i][j] - mean) * rstd;
                    dw[i][j] = fmaf(g[i][j], h[i][j], dw[i][j]);
                    db[i][j] += g[i][j];
                    g[i][j] *= w[i][j];
                    s1 += g[i][j];
                    s2 = fmaf(g[i][j], h[i][j], s2);
                }
            }
        // a turn's reductions use other words than the turn before, which a
        // slower wave may still read
        s1 = row_sum<kThreads>(s1, lds[2 * turn]) * inv_n;
        s2 = row_sum<kThreads>(s2, lds[2 * turn + 1]) * inv_n;
        TX *dx = static_cast<TX *>(a.out) + row * a.width;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = rstd * (g[i][j] - fmaf(h[i][j], s2, s1));
                store_values<kRagged>(dx + column(i), a.width - column(i), h[i]);
            }
    }
    if (!a.part) return;
    float *part = a.part + int64_t(blockIdx.x) * 2 * a.width;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
                store_values<kRagged>(part + column(i), a.width - column(i), dw[i]);
                store_values<kRagged>(part + a.width + column(i), a.width - column(i), db[i]);
            }
    } else {
        // the waves hold the same columns: added up in LDS, chunk by chunk
        __shared__ float sum[kRows][kThreads * 8];
        const int wave = threadIdx.x / kThreads;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[wave][j * kThreads + tid] = k ? db[i][j] : dw[i][j];
                __syncthreads();
                for (int e = threadIdx.x; e < kThreads * 8; e += kRowWgThreads) {
                    const int col = (i * kThreads + e % kThreads) * 8 + e / kThreads;
                    if (col < a.width) part[k * a.width + col] = (sum[0][e] + sum[1][e]) + (sum[2][e] + sum[3][e]);
                }
            }
    }
}

// dx of one row of any width.
template <typename TX, typename TG>
__global__ __launch_bounds__(kRowWgThreads) void layer_norm_backward_wide_kernel(NormArgs a) {
    __shared__ float lds[2][4];
    const int64_t row = row_group();
    if (row >= a.rows) return;
    const TX *x = static_cast<const TX *>(a.x) + row * a.width;
    const TG *dout = static_cast<const TG *>(a.dout) + row * a.width;
    const float mean = a.mean[row], rstd = a.rstd[row], inv_n = 1.0f / float(a.width);
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) {
        const float g = float(dout[c]) * (a.weight ? a.weight[c] : 1.0f);
        s1 += g;
        s2 = fmaf(g, (float(x[c]) - mean) * rstd, s2);
    }
    s1 = row_sum<256>(s1, lds[0]) * inv_n;
    s2 = row_sum<256>(s2, lds[1]) * inv_n;
    TX *dx = static_cast<TX *>(a.out) + row * a.width;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) {
        const float g = float(dout[c]) * (a.weight ? a.weight[c] : 1.0f);
        dx[c] = TX(rstd * (g - fmaf((float(x[c]) - mean) * rstd, s2, s1)));
    }
}

// Partial dw and db of 256 columns over every gridDim.y-th row.
template <typename TX, typename TG>
__global__ __launch_bounds__(kRowWgThreads) void layer_norm_columns_kernel(NormArgs a) {
    const int c = blockIdx.x * kRowWgThreads + threadIdx.x;
    if (c >= a.width) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float g = float(static_cast<const TG *>(a.dout)[row * a.width + c]);
        const float h = (float(static_cast<const TX *>(a.x)[row * a.width + c]) - a.mean[row]) * a.rstd[row];
        dw = fmaf(g, h, dw);
        db += g;
    }
    float *part = a.part + int64_t(blockIdx.y) * 2 * a.width;
    part[c] = dw;
    part[a.width + c] = db;
}

// dweight and dbias: the partial sums of each column, added in a fixed order.
// 1024 sums of 1280 columns, 10 MB from L2: 5 us, a launch's length.
__global__ __launch_bounds__(kSumColumns *kSumParts) void layer_norm_sum_kernel(const float *part, int32_t groups, int32_t width,
                                                                               float *dweight, float *dbias) {
    __shared__ float lds[kSumParts][kSumColumns + 1];
    const int column = threadIdx.x % kSumColumns, first = threadIdx.x / kSumColumns;
    const int64_t c = int64_t(blockIdx.x) * kSumColumns + column;  // of 2 width
    float v = 0.0f;
    if (c < 2 * int64_t(width)) {
#pragma unroll 8
        for (int g = first; g < groups; g += kSumParts) v += part[int64_t(g) * 2 * width + c];
    }
    lds[first][column] = v;
    __syncthreads();
#pragma unroll
    for (int n = kSumParts / 2; n > 0; n >>= 1) {
        if (first < n) lds[first][column] += lds[first + n][column];
        __syncthreads();
    }
    if (first == 0 && c < 2 * int64_t(width)) {
        if (c < width) {
            if (dweight) dweight[c] = lds[0][column];
        } else if (dbias) {
            dbias[c - width] = lds[0][column];
        }
    }
}

// How a width is laid over threads: whether rows are ragged, threads a row,
// chunks a thread; threads = 0: the row is read again for each sum.  As few
// chunks as hold the row, for the registers they take.
struct Shape {
    bool ragged;
    int threads, chunks;
};
// Forward: a wave holds a row as long as that is three chunks, since it then
// needs no barrier (131072 x 1280 bf16: 149 us, 4.5 TB/s, against 226 with
// the workgroup).
Shape forward_shape(int32_t width, bool aligned) {
    const bool ragged = !aligned || width % 8;
    if (width <= 64 * 8) return {ragged, 64, 1};
    if (width <= 64 * 8 * 3) return {ragged, 64, 3};
    if (width <= 256 * 8 * 3) return {ragged, 256, 3};
    if (width <= 256 * 8 * 8) return {ragged, 256, 8};
    return {ragged, 0, 0};
}
// Backward: a thread's columns cost five registers a value, so the workgroup
// holds a row from one chunk of a wave on (131072 x 1280 bf16: 222 us against
// 273; 4099 x 1283 float32: 21 against 26), and rows of more than three chunks
// go over 1024 threads (16384 x 12288 bf16: 246 us, 1.2 GB at 4.9 TB/s, against
// 553 with eight chunks in 256 threads, one wave a SIMD).
Shape backward_shape(int32_t width, bool aligned) {
    const bool ragged = !aligned || width % 8;
    if (width <= 64 * 8) return {ragged, 64, 1};
    if (width <= 256 * 8) return {ragged, 256, 1};
    if (width <= 256 * 8 * 3) return {ragged, 256, 3};
    if (width <= 1024 * 8 * 2) return {ragged, 1024, 2};
    return {ragged, 0, 0};
}

// Workgroups of the backward kernel, each of which adds up every so many
// rows, and partial sums of each column: as many as the card holds at once by
// their registers (four a CU with one chunk, three with three, one of 1024
// threads).
// Fewer leave memory waiting, more run in a second round and write more sums.
// us, sums included, for 256, 512, 768, 1024 and 2048 of them: 131072 x 1280
// bf16 663, 366, 270, 230, 249; 32768 x 5120 bf16 456, 302, 235, 313, 283;
// 16384 x 12288 bf16 246 and 257 for 256 and 512; with rows in a wave, which end
// in LDS, 262144 x 512 bf16 280, 168, 145, 154, 171.
int32_t backward_groups(int64_t rows, int32_t width) {
    const int64_t per = width <= 64 * 8 ? 4 : 1;
    const int64_t groups = (rows + per - 1) / per;
    const int64_t most = width <= 64 * 8 ? 768 : width <= 256 * 8 ? 1024 : width <= 256 * 8 * 3 ? 768 : 256;
    return int32_t(groups < most ? groups : most);
}

bool is_dtype(int32_t d) { return d == MIMO_F32 || d == MIMO_BF16; }

template <typename TX, typename TO>
void launch_forward(const Shape &s, const NormArgs &a, hipStream_t stream) {
    const dim3 block{unsigned(kRowWgThreads), 1, 1};
    const dim3 grid = row_grid(s.threads == 64 ? (a.rows + 3) / 4 : a.rows);
#define MIMO_NORM(R, T, C)  \
    if (s.ragged == R && s.threads == T && s.chunks == C) {  \
        hipLaunchKernelGGL((layer_norm_kernel<TX, TO, R, T, C>), grid, block, 0, stream, a);    \
        return;                                                                                 \
    }
    MIMO_NORM(false, 64, 1)
    MIMO_NORM(false, 64, 3)
    MIMO_NORM(false, 256, 3)
    MIMO_NORM(false, 256, 8)
    MIMO_NORM(true, 64, 1)
    MIMO_NORM(true, 64, 3)
    MIMO_NORM(true, 256, 3)
    MIMO_NORM(true, 256, 8)
#undef MIMO_NORM
    hipLaunchKernelGGL((layer_norm_wide_kernel<TX, TO>), grid, block, 0, stream, a);
}

template <typename TX, typename TG>
void launch_backward(const Shape &s, const NormArgs &a, int32_t groups, hipStream_t stream) {
    const dim3 block{unsigned(kRowWgThreads), 1, 1}, grid{unsigned(groups), 1, 1};
    const dim3 row_block{unsigned(s.threads > kRowWgThreads ? s.threads : kRowWgThreads), 1, 1};
#define MIMO_NORM(R, T, C)  \
    if (s.ragged == R && s.threads == T && s.chunks == C) {  \
        hipLaunchKernelGGL((layer_norm_backward_kernel<TX, TG, R, T, C>), grid, row_block, 0, stream, a);    \
        return;                                                                                              \
    }
    MIMO_NORM(false, 64, 1)
    MIMO_NORM(false, 256, 1)
    MIMO_NORM(false, 256, 3)
    MIMO_NORM(false, 1024, 2)
    MIMO_NORM(true, 64, 1)
    MIMO_NORM(true, 256, 1)
    MIMO_NORM(true, 256, 3)
    MIMO_NORM(true, 1024, 2)
#undef MIMO_NORM
    hipLaunchKernelGGL((layer_norm_backward_wide_kernel<TX, TG>), row_grid(a.rows), block, 0, stream, a);
    if (a.part)
        hipLaunchKernelGGL((layer_norm_columns_kernel<TX, TG>),
                           dim3(unsigned((a.width + kRowWgThreads - 1) / kRowWgThreads), unsigned(groups), 1), block, 0, stream, a);
}

int check_norm(const char *who, int64_t rows, int32_t width) {
    const std::string w(who);
    if (rows < 0 || width < 1) return set_error(MIMO_E_INVALID, w + ": rows must be >= 0 and width >= 1");
    if (width > kMaxWidth || rows > 0x7FFFFFFFll)
        return set_error(MIMO_E_TOO_LARGE, w + ": width above 65536 or more than 2^31 - 1 rows");
    return MIMO_OK;
}

}  // namespace
}  // namespace mimo

using namespace mimo;

extern "C" {

int mimo_layer_norm(int64_t rows, int32_t width, const void *x, int32_t x_dtype, const float *weight, const float *bias,
                    float eps, int32_t out_dtype, void *out, float *mean, float *rstd, void *stream) {
    clear_error();
    int st = check_norm("layer_norm", rows, width);
    if (st != MIMO_OK) return st;
    if (!is_dtype(x_dtype) || !is_dtype(out_dtype))
        return set_error(MIMO_E_INVALID, "layer_norm: dtypes must be MIMO_F32 or MIMO_BF16");
    if (!(eps >= 0.0f) || std::isinf(eps)) return set_error(MIMO_E_INVALID, "layer_norm: eps must be finite and >= 0");
    if (rows == 0) return MIMO_OK;
    if (!x || !out || !check_ptr_align(x, x_dtype == MIMO_F32 ? 4 : 2) || !check_ptr_align(out, out_dtype == MIMO_F32 ? 4 : 2) ||
        !check_ptr_align(weight, 4) || !check_ptr_align(bias, 4) || !check_ptr_align(mean, 4) || !check_ptr_align(rstd, 4))
        return set_error(MIMO_E_INVALID, "layer_norm: null or misaligned pointer (each aligned to its values)");
    if (mean && mean == rstd) return set_error(MIMO_E_INVALID, "layer_norm: mean and rstd must not be one array");
    if (out == x && x_dtype != out_dtype)
        return set_error(MIMO_E_INVALID, "layer_norm: out may be x only in x's dtype");
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.out = out;
    a.rows = rows;
    a.width = width;
    a.eps = eps;
    const bool aligned = check_ptr_align(x, 16) && check_ptr_align(out, 16) && check_ptr_align(weight, 16) && check_ptr_align(bias, 16);
    const Shape shape = forward_shape(width, aligned);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = timed_launch(s, [&] {
        if (x_dtype == MIMO_F32 && out_dtype == MIMO_F32)
            launch_forward<float, float>(shape, a, s);
        else if (x_dtype == MIMO_F32)
            launch_forward<float, __bf16>(shape, a, s);
        else if (out_dtype == MIMO_F32)
            launch_forward<__bf16, float>(shape, a, s);
        else
            launch_forward<__bf16, __bf16>(shape, a, s);
    });
    if (e != hipSuccess) return hip_error(e, "layer_norm: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

size_t mimo_layer_norm_workspace_bytes(int64_t rows, int32_t width) {
    if (rows < 0 || rows > 0x7FFFFFFFll || width < 1 || width > kMaxWidth) return 0;
    return size_t(backward_groups(rows, width)) * 2 * size_t(width) * sizeof(float);
}

int mimo_layer_norm_backward(int64_t rows, int32_t width, const void *x, int32_t x_dtype, const void *dout, int32_t dout_dtype,
                             const float *weight, const float *mean, const float *rstd, void *dx, float *dweight,
                             float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    const char *who = "layer_norm_backward";
    int st = check_norm(who, rows, width);
    if (st != MIMO_OK) return st;
    if (!is_dtype(x_dtype) || !is_dtype(dout_dtype))
        return set_error(MIMO_E_INVALID, "layer_norm_backward: dtypes must be MIMO_F32 or MIMO_BF16");
    const bool sums = dweight || dbias;
    if (rows == 0 && !sums) return MIMO_OK;
    if (!check_ptr_align(dweight, 4) || !check_ptr_align(dbias, 4))
        return set_error(MIMO_E_INVALID, "layer_norm_backward: dweight and dbias must be 4-byte aligned");
    if (dweight && dweight == dbias) return set_error(MIMO_E_INVALID, "layer_norm_backward: dweight and dbias must not be one array");
    if (rows > 0) {
        if (!x || !dout || !mean || !rstd || !dx || !check_ptr_align(x, x_dtype == MIMO_F32 ? 4 : 2) ||
            !check_ptr_align(dx, x_dtype == MIMO_F32 ? 4 : 2) || !check_ptr_align(dout, dout_dtype == MIMO_F32 ? 4 : 2) ||
            !check_ptr_align(weight, 4) || !check_ptr_align(mean, 4) || !check_ptr_align(rstd, 4))
            return set_error(MIMO_E_INVALID, "layer_norm_backward: null or misaligned pointer (each aligned to its values)");
        if (sums && (!workspace || !check_ptr_align(workspace, 16)))
            return set_error(MIMO_E_INVALID, "layer_norm_backward: workspace must be non-null and 16-byte aligned");
        if (sums && workspace_bytes < mimo_layer_norm_workspace_bytes(rows, width))
            return set_error(MIMO_E_CAPACITY, "layer_norm_backward: workspace smaller than mimo_layer_norm_workspace_bytes");
        if (dx == x || dx == dout) return set_error(MIMO_E_INVALID, "layer_norm_backward: dx must not be an input");
    }
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.dout = dout;
    a.weight = weight;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.out = dx;
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    a.rows = rows;
    a.width = width;
    const int32_t groups = backward_groups(rows, width);
    const bool aligned = check_ptr_align(x, 16) && check_ptr_align(dout, 16) && check_ptr_align(weight, 16) && check_ptr_align(dx, 16);
    const Shape shape = backward_shape(width, aligned);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = timed_launch(s, [&] {
        if (rows > 0) {
            if (x_dtype == MIMO_F32 && dout_dtype == MIMO_F32)
                launch_backward<float, float>(shape, a, groups, s);
            else if (x_dtype == MIMO_F32)
                launch_backward<float, __bf16>(shape, a, groups, s);
            else if (dout_dtype == MIMO_F32)
                launch_backward<__bf16, float>(shape, a, groups, s);
            else
                launch_backward<__bf16, __bf16>(shape, a, groups, s);
        }
        if (sums)
            hipLaunchKernelGGL(layer_norm_sum_kernel, dim3(unsigned((2 * int64_t(width) + kSumColumns - 1) / kSumColumns), 1, 1),
                               dim3(kSumColumns * kSumParts, 1, 1), 0, s, a.part, groups, width, dweight, dbias);
    });
    if (e != hipSuccess) return hip_error(e, "layer_norm_backward: kernel launch");
    g_dispatches.fetch_add((rows > 0 ? 1 : 0) + (rows > 0 && sums && shape.threads == 0 ? 1 : 0) + (sums ? 1 : 0));
    return MIMO_OK;
}

}  // extern "C"
