// rms_norm.hip -- the root-mean-square norm of rows of embeddings with the
// residual's addition, to float32, bf16 or 8-bit rows, and its backward pass,
// for AMD Instinct MI355X (gfx950).
//
// What is computed (NeMo Automodel "mimo_v2_flash.vision", MiMoVisionBlock: a
// norm before the attention and one before the feed-forward block, each over
// the residual stream that the branch before it was added to), for a row of n
// values:
//   h = x + residual, rounded to the residual's type    (h = x without one)
//   rstd = 1 / sqrt(sum h^2 / n + eps),  out = h rstd w
// and for dout, with g = dout w and the gradient dr that reaches h from
// elsewhere:
//   dh = dr + rstd (g - h rstd (sum g h rstd) / n)
//   dw = sum over rows of dout h rstd
// h is rounded before the norm, not after: the backward pass and the next
// addition have h in its type, so the norm is that of what they have.
//
// Everything is float32 inside, each output rounded once; rows whose squares
// float32 does not hold are summed in float64.  To 8 bits:
//   y = (h rstd) w in float32, scale = max |y| / 127, q = rint(y / scale)
// where the sum of squares is float64 and rstd its float32: which integer a
// quotient near the middle of two goes to hangs on rstd's last bit, and a
// float32 sum's depends on its order.  So integers and scales are those of the
// formula, bit for bit, whatever the kernel's shape (but for rows whose rstd
// lies within 2^-50 or so of the middle of two floats).
//
// The kernels are one pass over memory, which bounds them: a row stays in the
// registers of a wave or a workgroup (up to 16384 values); wider rows are read
// again from cache.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <string>
#include <type_traits>

#include "column_sums.h"
#include "device_util.h"
#include "internal.h"
#include "row_ops.h"
#include "runtime.h"

namespace mimo {
namespace {

using namespace rows;

constexpr int kMaxWidth = 65536;
constexpr int kPad = 128;  // 8-bit rows are multiples of this

struct RmsArgs {
    const void *x, *residual;    // residual or null
    const void *dout, *dres;     // backward; dres or null
    const float *weight;         // or null
    void *h;                     // the sum (with a residual)
    void *out;                   // out, the 8-bit rows, or dx
    float *rstd;                 // forward: or null; backward: input
    float *scale;                // of 8-bit rows
    float *part;                 // [groups][width]: partial dw, or null
    double eps;
    int64_t rows;
    int32_t width, padded;       // padded: of 8-bit rows
};

template <typename T>
__device__ __forceinline__ float rounded_to(float v) {
    return float(T(v));
}

// x of eight values and, with a residual, the sum rounded to its type and
// stored.
template <typename TX, typename TR, bool kRagged>
struct Rows {
    const TX *x;
    const TR *residual;
    TR *h;
    __device__ __forceinline__ Rows(const RmsArgs &a, int64_t row)
        : x(static_cast<const TX *>(a.x) + row * a.width),
          residual(a.residual ? static_cast<const TR *>(a.residual) + row * a.width : nullptr),
          h(static_cast<TR *>(a.h) + row * a.width) {}
    __device__ __forceinline__ void add(int col, int left, float (&v)[8], const float (&r)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = rounded_to<TR>(v[j] + r[j]);
        store_values<kRagged>(h + col, left, v);
    }
};

// What a row's sum of squares is made in, and rstd.
template <bool kExact>
using Square = typename std::conditional<kExact, double, float>::type;
__device__ __forceinline__ float rstd_of(float squares, int n, double eps) { return 1.0f / sqrtf(squares / float(n) + float(eps)); }
__device__ __forceinline__ float rstd_of(double squares, int n, double eps) { return float(1.0 / sqrt(squares / double(n) + eps)); }
// Whether the mean of a float32 sum's squares, with eps, is right: squares
// below 2^-126 lose bits (at most 2^-150 each, and so does their mean), and a sum
// may pass float32's range.  Where it is not, the row's sum is made again in
// float64, which holds the squares of all its values; every thread of a row has
// the same sum, so they all do or none.  NaN is made again too, and stays.
// The test costs nothing that shows: 131072 x 1280 bf16 with the residual 223 to
// 231 us without it and 224 to 231 with it.
__device__ __forceinline__ bool holds(float squares, int n, double eps) {
    const float mean = squares / float(n) + float(eps);
    return mean >= 0x1p-100f && mean < __builtin_inff();
}
__device__ __forceinline__ float add_square(float v, float s) { return fmaf(v, v, s); }
__device__ __forceinline__ double add_square(float v, double s) { return fma(double(v), double(v), s); }

// Scale of a row whose largest magnitude (as magnitude() has it) is top.
struct RowScale {
    float scale, inv;
    bool none;  // zeros: a row of them, or one that is not finite, whose scale is NaN
    __device__ __forceinline__ explicit RowScale(uint32_t top) {
        const bool finite = top < 0x7F800000u;
        scale = finite ? __builtin_bit_cast(float, top) / 127.0f : __builtin_nanf("");
        none = !finite || scale == 0.0f;
        inv = 1.0f / scale;
    }
};

// One row by a wave (kThreads = 64) or the workgroup; chunk i of a thread is i
// * kThreads + its number.  TO: float, bf16, or int8_t (8-bit rows).  Memory
// bounds it, and for 8-bit rows of few columns the VALU too: 131072 x 1280 bf16
// with the residual 222 to 230 us, 1.34 GB at 5.8 to 6.0 TB/s; to 8 bits 220 to
// 243 us, 1.17 GB at 4.8 to 5.3 TB/s; 4099 x 1283 float32 16 us.
template <typename TX, typename TR, typename TO, bool kRagged, int kThreads, int kChunks>
__global__ __launch_bounds__(kRowWgThreads) void rms_norm_kernel(RmsArgs a) {
    constexpr bool kBytes = std::is_same<TO, int8_t>::value;
    typedef Square<kBytes> Sum;
    __shared__ Sum lds[4];
    __shared__ double lds_again[4];
    __shared__ uint32_t lds_top[4];
    const int tid = threadIdx.x % kThreads;
    const int64_t row = row_group() * (kRowWgThreads / kThreads) + threadIdx.x / kThreads;
    if (row >= a.rows) return;  // all of the threads that hold a row
    const Rows<TX, TR, kRagged> in(a, row);
    auto column = [&](int i) { return (i * kThreads + tid) * 8; };
    float v[kChunks][8];
    if (in.residual) {
        float r[kChunks][8];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
                load_values<kRagged>(in.x + column(i), a.width - column(i), v[i]);
                load_values<kRagged>(in.residual + column(i), a.width - column(i), r[i]);
            }
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) in.add(column(i), a.width - column(i), v[i], r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) load_values<kRagged>(in.x + column(i), a.width - column(i), v[i]);
    }
    auto add_squares = [&](auto sum) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = add_square(v[i][j], sum);
            }
        return sum;
    };
    const Sum squares = row_sum<kThreads>(add_squares(Sum(0)), lds);
    float rstd = rstd_of(squares, a.width, a.eps);
    if constexpr (!kBytes)
        if (!holds(squares, a.width, a.eps)) rstd = rstd_of(row_sum<kThreads>(add_squares(0.0), lds_again), a.width, a.eps);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        if (column(i) < a.width) {
            const int left = a.width - column(i);
            float w[8];
            if (a.weight) load_values<kRagged>(a.weight + column(i), left, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= rstd;
                if (a.weight) v[i][j] *= w[j];
                if constexpr (kBytes) top = max(top, magnitude(v[i][j]));
            }
            if constexpr (!kBytes) store_values<kRagged>(static_cast<TO *>(a.out) + row * a.width + column(i), left, v[i]);
        }
    if constexpr (kBytes) {
        const RowScale s(row_max<kThreads>(top, lds_top));
        int8_t *q = static_cast<int8_t *>(a.out) + row * a.padded;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.padded) {
                u32x2 p = {0, 0};
                if (column(i) < a.width && !s.none) p = quantize(v[i], s.scale, s.inv);
                *reinterpret_cast<u32x2 *>(q + column(i)) = p;
            }
        if (tid == 0) a.scale[row] = s.scale;
    }
    if (tid == 0 && a.rstd) a.rstd[row] = rstd;
}

// Rows of any width, one workgroup each; x and the residual are read once, the
// sum again for each pass (a thread reads what it wrote).
template <typename TX, typename TR, typename TO>
__global__ __launch_bounds__(kRowWgThreads) void rms_norm_wide_kernel(RmsArgs a) {
    constexpr bool kBytes = std::is_same<TO, int8_t>::value;
    typedef Square<kBytes> Sum;
    __shared__ Sum lds[4];
    __shared__ double lds_again[4];
    __shared__ uint32_t lds_top[4];
    const int64_t row = row_group();
    if (row >= a.rows) return;
    const Rows<TX, TR, true> in(a, row);
    Sum squares = 0;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) {
        float v = float(in.x[c]);
        if (in.residual) {
            v = rounded_to<TR>(v + float(in.residual[c]));
            in.h[c] = TR(v);
        }
        squares = add_square(v, squares);
    }
    squares = row_sum<256>(squares, lds);
    float rstd = rstd_of(squares, a.width, a.eps);
    auto normed = [&](int c) { return in.residual ? float(in.h[c]) : float(in.x[c]); };
    if constexpr (!kBytes)
        if (!holds(squares, a.width, a.eps)) {
            double again = 0.0;
            for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) again = add_square(normed(c), again);
            rstd = rstd_of(row_sum<256>(again, lds_again), a.width, a.eps);
        }
    auto value = [&](int c) {
        const float v = normed(c) * rstd;
        return a.weight ? v * a.weight[c] : v;
    };
    if constexpr (kBytes) {
        uint32_t top = 0;
        for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) top = max(top, magnitude(value(c)));
        const RowScale s(row_max<256>(top, lds_top));
        int8_t *q = static_cast<int8_t *>(a.out) + row * a.padded;
        for (int c = threadIdx.x; c < a.padded; c += kRowWgThreads) {
            float v = 0.0f;
            if (c < a.width && !s.none) v = fminf(fmaxf(__builtin_rintf(value(c) / s.scale), -127.0f), 127.0f);
            q[c] = int8_t(int(v));
        }
        if (threadIdx.x == 0) a.scale[row] = s.scale;
    } else {
        TO *out = static_cast<TO *>(a.out) + row * a.width;
        for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) out[c] = TO(value(c));
    }
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
}

// dh of rows first, first + step, ...; partial dw of those rows.  A thread
// keeps its columns from row to row, so dw accumulates in registers: in float32,
// since float64 sums would take twice as many and twice the workspace (85 rows
// of 131072 x 1280 a workgroup); the workgroups' sums are added up in float64
// (column_sums.h).  131072 x
// 1280 bf16 with dresidual 240 to 258 us, 1.34 GB at 5.2 to 5.6 TB/s; 4099 x 1283
// float32 15 to 17 us.
template <typename TX, typename TG, bool kRagged, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads > kRowWgThreads ? kThreads : kRowWgThreads) void rms_norm_backward_kernel(RmsArgs a) {
    constexpr int kRows = kThreads < kRowWgThreads ? kRowWgThreads / kThreads : 1;  // rows of the workgroup at a time
    __shared__ float lds[2][kThreads > kRowWgThreads ? kThreads / 64 : 4];
    const int tid = threadIdx.x % kThreads;
    const float inv_n = 1.0f / float(a.width);
    auto column = [&](int i) { return (i * kThreads + tid) * 8; };
    float w[kChunks][8], dw[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = 0.0f;
            w[i][j] = 1.0f;
        }
        if (a.weight && column(i) < a.width) load_values<kRagged>(a.weight + column(i), a.width - column(i), w[i]);
    }
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kThreads; row < a.rows; row += int64_t(gridDim.x) * kRows, turn ^= 1) {
        const TX *x = static_cast<const TX *>(a.x) + row * a.width;
        const TG *dout = static_cast<const TG *>(a.dout) + row * a.width;
        const TX *dres = a.dres ? static_cast<const TX *>(a.dres) + row * a.width : nullptr;
        const float rstd = a.rstd[row];
        float h[kChunks][8], g[kChunks][8], d[kChunks][8];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
                load_values<kRagged>(x + column(i), a.width - column(i), h[i]);
                load_values<kRagged>(dout + column(i), a.width - column(i), g[i]);
            }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] = 0.0f;
            if (dres && column(i) < a.width) load_values<kRagged>(dres + column(i), a.width - column(i), d[i]);
        }
        // past a ragged row's end dout is zero, and with it every sum
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[i][j] *= rstd;
                    dw[i][j] = fmaf(g[i][j], h[i][j], dw[i][j]);
                    g[i][j] *= w[i][j];
                    s = fmaf(g[i][j], h[i][j], s);
                }
            }
        // a turn's reduction uses other words than the turn before, which a
        // slower wave may still read
        s = row_sum<kThreads>(s, lds[turn]) * inv_n;
        TX *dx = static_cast<TX *>(a.out) + row * a.width;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = fmaf(rstd, fmaf(-h[i][j], s, g[i][j]), d[i][j]);
                store_values<kRagged>(dx + column(i), a.width - column(i), h[i]);
            }
    }
    if (!a.part) return;
    float *part = a.part + int64_t(blockIdx.x) * a.width;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (column(i) < a.width) store_values<kRagged>(part + column(i), a.width - column(i), dw[i]);
    } else {
        // the waves hold the same columns: added up in LDS, chunk by chunk
        __shared__ float sum[kRows][kThreads * 8];
        const int wave = threadIdx.x / kThreads;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[wave][j * kThreads + tid] = dw[i][j];
            __syncthreads();
            for (int e = threadIdx.x; e < kThreads * 8; e += kRowWgThreads) {
                const int col = (i * kThreads + e % kThreads) * 8 + e / kThreads;
                if (col < a.width) part[col] = (sum[0][e] + sum[1][e]) + (sum[2][e] + sum[3][e]);
            }
        }
    }
}

// dh of one row of any width.
template <typename TX, typename TG>
__global__ __launch_bounds__(kRowWgThreads) void rms_norm_backward_wide_kernel(RmsArgs a) {
    __shared__ float lds[4];
    const int64_t row = row_group();
    if (row >= a.rows) return;
    const TX *x = static_cast<const TX *>(a.x) + row * a.width;
    const TG *dout = static_cast<const TG *>(a.dout) + row * a.width;
    const TX *dres = a.dres ? static_cast<const TX *>(a.dres) + row * a.width : nullptr;
    const float rstd = a.rstd[row];
    auto weighted = [&](int c) { return float(dout[c]) * (a.weight ? a.weight[c] : 1.0f); };
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads) s = fmaf(weighted(c), float(x[c]) * rstd, s);
    s = row_sum<256>(s, lds) * (1.0f / float(a.width));
    TX *dx = static_cast<TX *>(a.out) + row * a.width;
    for (int c = threadIdx.x; c < a.width; c += kRowWgThreads)
        dx[c] = TX(fmaf(rstd, fmaf(-float(x[c]) * rstd, s, weighted(c)), dres ? float(dres[c]) : 0.0f));
}

// Partial dw of 256 columns over every gridDim.y-th row.
template <typename TX, typename TG>
__global__ __launch_bounds__(kRowWgThreads) void rms_norm_columns_kernel(RmsArgs a) {
    const int c = blockIdx.x * kRowWgThreads + threadIdx.x;
    if (c >= a.width) return;
    float dw = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
        dw = fmaf(float(static_cast<const TG *>(a.dout)[row * a.width + c]),
                  float(static_cast<const TX *>(a.x)[row * a.width + c]) * a.rstd[row], dw);
    a.part[int64_t(blockIdx.y) * a.width + c] = dw;
}

// How a width is laid over threads: whether rows are ragged, threads a row,
// chunks a thread; threads = 0: the row is read again for each pass.
struct Shape {
    bool ragged;
    int threads, chunks;
};
Shape forward_shape(int32_t width, bool aligned) {
    const bool ragged = !aligned || width % 8;
    if (width <= 64 * 8) return {ragged, 64, 1};
    if (width <= 64 * 8 * 3) return {ragged, 64, 3};
    if (width <= 256 * 8 * 3) return {ragged, 256, 3};
    if (width <= 256 * 8 * 8) return {ragged, 256, 8};
    return {ragged, 0, 0};
}
// A wave holds a row only up to 512 values here: of 131072 x 1280 bf16 in waves
// 300 us and more, whatever their number, against 258.
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
// the registers of each shape.  us with dresidual and the sums, bf16: 131072 x
// 1280, 1024, 1536, 2048 of them: 306, 246, 345; 32768 x 5120, 512, 768, 1024:
// 354, 280, 370; 16384 x 12288, 256, 384, 512: 310, 377, 323; 262144 x 512, whose
// waves take a row each, 768, 1024, 1536, 2048: 200, 197, 205, 231.
// Where rows are few, four for each workgroup as long as every CU has one: the
// partial sums weigh more than the rows otherwise.  us with 1, 2, 4 and 6 rows
// each, bf16: 1024 x 1280, 9.7, 7.9, 7.9, 7.9; 2500 x 1280, 13.1, 13.5, 10.7, 11.6;
// 1960 x 512, 8.3, 6.4, 6.4, 6.4; 1960 x 5120, 19.8, 19.9, 20.9, 22.5.
int32_t backward_groups(int64_t rows, int32_t width) {
    const int64_t per = width <= 64 * 8 ? 4 : 1;
    const int64_t groups = (rows + per - 1) / per;
    const int64_t most = width <= 64 * 8 ? 1024 : width <= 256 * 8 ? 1536 : width <= 256 * 8 * 3 ? 768 : 256;
    const int64_t few = groups < 256 ? groups : groups / 4 > 256 ? groups / 4 : 256;
    return int32_t(few < most ? few : most);
}

bool is_dtype(int32_t d) { return d == MIMO_F32 || d == MIMO_BF16; }
int size_of(int32_t dtype) { return dtype == MIMO_F32 ? 4 : 2; }

template <typename TX, typename TR, typename TO>
void launch_forward(const Shape &s, const RmsArgs &a, hipStream_t stream) {
    const dim3 block{unsigned(kRowWgThreads), 1, 1};
    const dim3 grid = row_grid(s.threads == 64 ? (a.rows + 3) / 4 : a.rows);
#define MIMO_NORM(R, T, C)  \
    if (s.ragged == R && s.threads == T && s.chunks == C) {  \
        hipLaunchKernelGGL((rms_norm_kernel<TX, TR, TO, R, T, C>), grid, block, 0, stream, a);  \
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
    hipLaunchKernelGGL((rms_norm_wide_kernel<TX, TR, TO>), grid, block, 0, stream, a);
}

// x's and the residual's type (the residual's is x's, or float32).
template <typename TO>
void launch_forward(int32_t x_dtype, int32_t res_dtype, const Shape &s, const RmsArgs &a, hipStream_t stream) {
    if (x_dtype == MIMO_F32)
        launch_forward<float, float, TO>(s, a, stream);
    else if (res_dtype == MIMO_F32)
        launch_forward<__bf16, float, TO>(s, a, stream);
    else
        launch_forward<__bf16, __bf16, TO>(s, a, stream);
}

template <typename TX, typename TG>
void launch_backward(const Shape &s, const RmsArgs &a, int32_t groups, hipStream_t stream) {
    const dim3 block{unsigned(kRowWgThreads), 1, 1}, grid{unsigned(groups), 1, 1};
    const dim3 row_block{unsigned(s.threads > kRowWgThreads ? s.threads : kRowWgThreads), 1, 1};
#define MIMO_NORM(R, T, C)  \
    if (s.ragged == R && s.threads == T && s.chunks == C) {  \
        hipLaunchKernelGGL((rms_norm_backward_kernel<TX, TG, R, T, C>), grid, row_block, 0, stream, a);  \
        return;                                                                                          \
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
    hipLaunchKernelGGL((rms_norm_backward_wide_kernel<TX, TG>), row_grid(a.rows), block, 0, stream, a);
    if (a.part)
        hipLaunchKernelGGL((rms_norm_columns_kernel<TX, TG>),
                           dim3(unsigned((a.width + kRowWgThreads - 1) / kRowWgThreads), unsigned(groups), 1), block, 0, stream, a);
}

// What both forward entry points check alike.
int check_forward(const char *who, int64_t rows, int32_t width, const void *x, int32_t x_dtype, const void *residual,
                  int32_t residual_dtype, const float *weight, double eps, const void *residual_out, const void *out,
                  uintptr_t out_align) {
    const std::string w(who);
    if (rows < 0 || width < 1) return set_error(MIMO_E_INVALID, w + ": rows must be >= 0 and width >= 1");
    if (width > kMaxWidth || rows > 0x7FFFFFFFll)
        return set_error(MIMO_E_TOO_LARGE, w + ": width above 65536 or more than 2^31 - 1 rows");
    if (!is_dtype(x_dtype) || (residual && residual_dtype != x_dtype && residual_dtype != MIMO_F32))
        return set_error(MIMO_E_INVALID, w + ": x must be MIMO_F32 or MIMO_BF16, and the residual of x's type or MIMO_F32");
    if (!(eps >= 0.0) || std::isinf(eps)) return set_error(MIMO_E_INVALID, w + ": eps must be finite and >= 0");
    if (rows == 0) return MIMO_OK;
    if (!x || !out || !check_ptr_align(x, size_of(x_dtype)) || !check_ptr_align(out, out_align) || !check_ptr_align(weight, 4))
        return set_error(MIMO_E_INVALID, w + ": null or misaligned pointer (8-bit rows 16 bytes, the others to their values)");
    if (residual) {
        if (!residual_out || !check_ptr_align(residual, size_of(residual_dtype)) || !check_ptr_align(residual_out, size_of(residual_dtype)))
            return set_error(MIMO_E_INVALID, w + ": residual_out must be given with residual, both aligned to their values");
        if (residual_out == x && residual_dtype != x_dtype)
            return set_error(MIMO_E_INVALID, w + ": residual_out may be x only in x's dtype");
        if (residual_out == out) return set_error(MIMO_E_INVALID, w + ": out and residual_out must not be one array");
    }
    return MIMO_OK;
}

// Whether `p`, which is written a value a row while other rows are still read,
// is one of these.
bool is_one_of(const void *p, const void *x, const void *residual, const void *residual_out, const void *out) {
    return p && (p == x || p == residual || p == residual_out || p == out);
}

RmsArgs forward_args(int64_t rows, int32_t width, const void *x, const void *residual, const float *weight, double eps,
                     void *residual_out, void *out) {
    RmsArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.h = residual ? residual_out : nullptr;
    a.out = out;
    a.eps = eps;
    a.rows = rows;
    a.width = width;
    a.padded = (width + kPad - 1) / kPad * kPad;
    return a;
}

bool all_aligned(const RmsArgs &a) {
    return check_ptr_align(a.x, 16) && check_ptr_align(a.residual, 16) && check_ptr_align(a.h, 16) && check_ptr_align(a.out, 16) &&
           check_ptr_align(a.weight, 16) && check_ptr_align(a.dout, 16) && check_ptr_align(a.dres, 16);
}

}  // namespace
}  // namespace mimo

using namespace mimo;

extern "C" {

int mimo_rms_norm(int64_t rows, int32_t width, const void *x, int32_t x_dtype, const void *residual, int32_t residual_dtype,
                  const float *weight, double eps, void *residual_out, int32_t out_dtype, void *out, float *rstd, void *stream) {
    clear_error();
    if (!is_dtype(out_dtype)) return set_error(MIMO_E_INVALID, "rms_norm: out_dtype must be MIMO_F32 or MIMO_BF16");
    int st = check_forward("rms_norm", rows, width, x, x_dtype, residual, residual_dtype, weight, eps, residual_out, out, size_of(out_dtype));
    if (st != MIMO_OK || rows == 0) return st;
    if (!check_ptr_align(rstd, 4)) return set_error(MIMO_E_INVALID, "rms_norm: rstd must be 4-byte aligned");
    // workgroups that still read the weight run next to the ones that write
    if (weight && (rstd == weight || out == weight || residual_out == weight))
        return set_error(MIMO_E_INVALID, "rms_norm: no output may be the weight");
    if (is_one_of(rstd, x, residual, residual ? residual_out : nullptr, out))
        return set_error(MIMO_E_INVALID, "rms_norm: rstd must not be an input or another output");
    if ((out == x && out_dtype != x_dtype) || (residual && out == residual && out_dtype != residual_dtype))
        return set_error(MIMO_E_INVALID, "rms_norm: out may be x or the residual only in its dtype");
    const int64_t values = rows * width;
    const int res_size = residual ? size_of(residual_dtype) : 0;
    if (overlap_in_part({{out, values * size_of(out_dtype)}, {residual ? residual_out : nullptr, values * res_size}, {rstd, rows * 4}},
                        {{x, values * size_of(x_dtype)}, {residual, values * res_size}, {weight, width * 4}}))
        return set_error(MIMO_E_INVALID, "rms_norm: an output must not overlap an input or another output in part");
    RmsArgs a = forward_args(rows, width, x, residual, weight, eps, residual_out, out);
    a.rstd = rstd;
    const Shape shape = forward_shape(width, all_aligned(a));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int32_t res_dtype = residual ? residual_dtype : x_dtype;
    const hipError_t e = timed_launch(s, [&] {
        if (out_dtype == MIMO_F32)
            launch_forward<float>(x_dtype, res_dtype, shape, a, s);
        else
            launch_forward<__bf16>(x_dtype, res_dtype, shape, a, s);
    });
    if (e != hipSuccess) return hip_error(e, "rms_norm: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

int mimo_rms_norm_quantized(int64_t rows, int32_t width, const void *x, int32_t x_dtype, const void *residual,
                            int32_t residual_dtype, const float *weight, double eps, void *residual_out, void *q, float *scale,
                            void *stream) {
    clear_error();
    int st = check_forward("rms_norm_quantized", rows, width, x, x_dtype, residual, residual_dtype, weight, eps, residual_out, q, 16);
    if (st != MIMO_OK || rows == 0) return st;
    if (!scale || !check_ptr_align(scale, 4))
        return set_error(MIMO_E_INVALID, "rms_norm_quantized: scale must be non-null and 4-byte aligned");
    if (q == x || (residual && q == residual)) return set_error(MIMO_E_INVALID, "rms_norm_quantized: q must not be an input");
    if (weight && (scale == weight || q == weight || residual_out == weight))
        return set_error(MIMO_E_INVALID, "rms_norm_quantized: no output may be the weight");
    if (is_one_of(scale, x, residual, residual ? residual_out : nullptr, q))
        return set_error(MIMO_E_INVALID, "rms_norm_quantized: scale must not be an input or another output");
    const int64_t values = rows * width;
    const int res_size = residual ? size_of(residual_dtype) : 0;
    if (overlap_in_part({{q, rows * ((width + kPad - 1) / kPad * kPad)}, {residual ? residual_out : nullptr, values * res_size}, {scale, rows * 4}},
                        {{x, values * size_of(x_dtype)}, {residual, values * res_size}, {weight, width * 4}}))
        return set_error(MIMO_E_INVALID, "rms_norm_quantized: an output must not overlap an input or another output in part");
    RmsArgs a = forward_args(rows, width, x, residual, weight, eps, residual_out, q);
    a.scale = scale;
    const Shape shape = forward_shape(width, all_aligned(a));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = timed_launch(s, [&] { launch_forward<int8_t>(x_dtype, residual ? residual_dtype : x_dtype, shape, a, s); });
    if (e != hipSuccess) return hip_error(e, "rms_norm_quantized: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

size_t mimo_rms_norm_workspace_bytes(int64_t rows, int32_t width) {
    if (rows < 0 || rows > 0x7FFFFFFFll || width < 1 || width > kMaxWidth) return 0;
    return size_t(backward_groups(rows, width)) * size_t(width) * sizeof(float);
}

int mimo_rms_norm_backward(int64_t rows, int32_t width, const void *h, int32_t h_dtype, const void *dout, int32_t dout_dtype,
                           const float *weight, const float *rstd, const void *dresidual, void *dx, float *dweight,
                           void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    if (rows < 0 || width < 1) return set_error(MIMO_E_INVALID, "rms_norm_backward: rows must be >= 0 and width >= 1");
    if (width > kMaxWidth || rows > 0x7FFFFFFFll)
        return set_error(MIMO_E_TOO_LARGE, "rms_norm_backward: width above 65536 or more than 2^31 - 1 rows");
    if (!is_dtype(h_dtype) || !is_dtype(dout_dtype))
        return set_error(MIMO_E_INVALID, "rms_norm_backward: dtypes must be MIMO_F32 or MIMO_BF16");
    if (rows == 0 && !dweight) return MIMO_OK;
    if (!check_ptr_align(dweight, 4)) return set_error(MIMO_E_INVALID, "rms_norm_backward: dweight must be 4-byte aligned");
    if (rows > 0) {
        if (!h || !dout || !rstd || !dx || !check_ptr_align(h, size_of(h_dtype)) || !check_ptr_align(dx, size_of(h_dtype)) ||
            !check_ptr_align(dresidual, size_of(h_dtype)) || !check_ptr_align(dout, size_of(dout_dtype)) || !check_ptr_align(weight, 4) ||
            !check_ptr_align(rstd, 4))
            return set_error(MIMO_E_INVALID, "rms_norm_backward: null or misaligned pointer (each aligned to its values)");
        if (dweight && (!workspace || !check_ptr_align(workspace, 16)))
            return set_error(MIMO_E_INVALID, "rms_norm_backward: workspace must be non-null and 16-byte aligned");
        if (dweight && workspace_bytes < mimo_rms_norm_workspace_bytes(rows, width))
            return set_error(MIMO_E_CAPACITY, "rms_norm_backward: workspace smaller than mimo_rms_norm_workspace_bytes");
        if (dx == h || dx == dout) return set_error(MIMO_E_INVALID, "rms_norm_backward: dx must not be h or dout");
        if (dweight && (dweight == weight || dweight == rstd || is_one_of(dweight, h, dout, dresidual, dx)))
            return set_error(MIMO_E_INVALID, "rms_norm_backward: dweight must not be an input, nor dx");
        if (dx == weight || dx == rstd) return set_error(MIMO_E_INVALID, "rms_norm_backward: dx must not be the weight or rstd");
        const int64_t h_bytes = rows * width * size_of(h_dtype);
        const Span made_x{dx, h_bytes}, made_w{dweight, width * 4}, in_h{h, h_bytes}, in_g{dout, rows * width * size_of(dout_dtype)},
            in_w{weight, width * 4}, in_rstd{rstd, rows * 4}, in_res{dresidual, h_bytes};
        if (overlap_in_part({made_x, made_w}, {in_h, in_g, in_w, in_rstd, in_res}))
            return set_error(MIMO_E_INVALID, "rms_norm_backward: a gradient must not overlap an input or the other one in part");
        if (dweight && overlaps_any({workspace, int64_t(mimo_rms_norm_workspace_bytes(rows, width))}, {made_x, made_w, in_h, in_g, in_w, in_rstd, in_res}))
            return set_error(MIMO_E_INVALID, "rms_norm_backward: workspace must not overlap another argument");
    }
    RmsArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = h;
    a.dout = dout;
    a.dres = dresidual;
    a.weight = weight;
    a.rstd = const_cast<float *>(rstd);
    a.out = dx;
    a.part = dweight ? static_cast<float *>(workspace) : nullptr;
    a.rows = rows;
    a.width = width;
    const int32_t groups = backward_groups(rows, width);
    const Shape shape = backward_shape(width, all_aligned(a));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = timed_launch(s, [&] {
        if (rows > 0) {
            if (h_dtype == MIMO_F32 && dout_dtype == MIMO_F32)
                launch_backward<float, float>(shape, a, groups, s);
            else if (h_dtype == MIMO_F32)
                launch_backward<float, __bf16>(shape, a, groups, s);
            else if (dout_dtype == MIMO_F32)
                launch_backward<__bf16, float>(shape, a, groups, s);
            else
                launch_backward<__bf16, __bf16>(shape, a, groups, s);
        }
        if (dweight) {
            ColumnSums sums;
            sums.add(a.part, groups, width, width, dweight);
            launch_column_sums(sums, s);
        }
    });
    if (e != hipSuccess) return hip_error(e, "rms_norm_backward: kernel launch");
    g_dispatches.fetch_add((rows > 0 ? 1 : 0) + (rows > 0 && dweight && shape.threads == 0 ? 1 : 0) + (dweight ? 1 : 0));
    return MIMO_OK;
}

}  // extern "C"
