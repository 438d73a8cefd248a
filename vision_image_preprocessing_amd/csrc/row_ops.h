// row_ops.h -- what the kernels over rows of embeddings share: eight values
// of a row in registers, sums and maxima over the threads that hold one row,
// and its values as 8-bit integers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_util.h"

namespace mimo {
namespace rows {

constexpr int kRowWgThreads = 256;

// Workgroups of a launch over rows, and the number of one: in two dimensions,
// since a dimension of a launch has fewer than 2^32 threads.
inline dim3 row_grid(int64_t groups) {
    constexpr int64_t kWide = int64_t(1) << 20;
    return groups <= kWide ? dim3(unsigned(groups), 1, 1) : dim3(unsigned(kWide), unsigned((groups + kWide - 1) / kWide), 1);
}
__device__ __forceinline__ int64_t row_group() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }

// Eight values of a row as float32, from one or two 16-byte accesses.
// kRagged: rows of any width at any address of the type (the accesses are
// then aligned to the values only, which the hardware takes), with n of the
// eight inside the row; values past it read as zeros and are not written.
template <bool kRagged>
__device__ __forceinline__ void load_values(const float *p, int n, float (&v)[8]) {
    typedef f32x4 any_f32x4 __attribute__((aligned(4)));
    if (!kRagged || n >= 8) {
        f32x4 a, b;
        if constexpr (kRagged) {
            a = *reinterpret_cast<const any_f32x4 *>(p);
            b = *reinterpret_cast<const any_f32x4 *>(p + 4);
        } else {
            a = *reinterpret_cast<const f32x4 *>(p);
            b = *reinterpret_cast<const f32x4 *>(p + 4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.0f;
    }
}
template <bool kRagged>
__device__ __forceinline__ void load_values(const __bf16 *p, int n, float (&v)[8]) {
    typedef u32x4 any_u32x4 __attribute__((aligned(2)));
    if (!kRagged || n >= 8) {
        u32x4 w;
        if constexpr (kRagged)
            w = *reinterpret_cast<const any_u32x4 *>(p);
        else
            w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? float(p[j]) : 0.0f;
    }
}

// The same values out, rounded once (to nearest even) where the type is bf16.
template <bool kRagged>
__device__ __forceinline__ void store_values(float *p, int n, const float (&v)[8]) {
    typedef f32x4 any_f32x4 __attribute__((aligned(4)));
    if (!kRagged || n >= 8) {
        const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        if constexpr (kRagged) {
            *reinterpret_cast<any_f32x4 *>(p) = a;
            *reinterpret_cast<any_f32x4 *>(p + 4) = b;
        } else {
            *reinterpret_cast<f32x4 *>(p) = a;
            *reinterpret_cast<f32x4 *>(p + 4) = b;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = v[j];
    }
}
template <bool kRagged>
__device__ __forceinline__ void store_values(__bf16 *p, int n, const float (&v)[8]) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    typedef bf16x8 any_bf16x8 __attribute__((aligned(2)));
    bf16x8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __bf16(v[j]);
    if (!kRagged || n >= 8) {
        if constexpr (kRagged)
            *reinterpret_cast<any_bf16x8 *>(p) = h;
        else
            *reinterpret_cast<bf16x8 *>(p) = h;
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = h[j];
    }
}

// Sum over the kThreads (64: a wave, more: the workgroup) threads of a row,
// in a fixed order; every one of them gets it.  `lds`: kThreads / 64 values
// that no other reduction in flight uses.
template <int kThreads, typename T>
__device__ __forceinline__ T row_sum(T v, T *lds) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    if constexpr (kThreads > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
#pragma unroll
        for (int i = 4; i < kThreads / 64; i += 4) v += (lds[i] + lds[i + 1]) + (lds[i + 2] + lds[i + 3]);
    }
    return v;
}

// |v| as an unsigned integer: the order of the magnitudes, NaN above all.
__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

template <int kThreadsRow>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *lds) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = max(v, uint32_t(__shfl_xor(int(v), m)));
    if constexpr (kThreadsRow == 256) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = max(max(lds[0], lds[1]), max(lds[2], lds[3]));
    }
    return v;
}

// Eight quotients as bytes.  The definition divides in float32 (rounded
// correctly) and takes the nearest integer, ties to even.  A product with the
// reciprocal is within 2^-15 of the quotient (|quotient| <= 128, two
// roundings of 2^-24 and the quotient's own), so where it is further than
// kNear from the middle of two integers it rounds to the same one; only where
// one of the eight is not are they divided, which costs three times as much
// (131072 x 1536 bf16: 137 us, 116% of the VALU's cycles, with divisions
// throughout).  Scales below kSmall hold few bits or have no reciprocal: they
// are divided too, and their quotients may pass 127.
constexpr float kNear = 1e-3f, kSmall = 1e-30f;
__device__ __forceinline__ u32x2 quantize(const float (&v)[8], float scale, float inv) {
    float r[8];
    float off = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float y = v[j] * inv;
        r[j] = __builtin_rintf(y);
        off = fmaxf(off, fabsf(y - r[j]));
    }
    if (off > 0.5f - kNear || scale < kSmall) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = fminf(fmaxf(__builtin_rintf(v[j] / scale), -127.0f), 127.0f);
    }
    u32x2 p = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j / 4] |= (uint32_t(int(r[j])) & 0xFFu) << (8 * (j % 4));
    return p;
}

}  // namespace rows
}  // namespace mimo
