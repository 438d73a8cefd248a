// row_ops.h -- what the kernels over rows of embeddings share: eight values
// of a row in registers, and sums over the threads that hold one row.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_util.h"

namespace mimo {
namespace rows {

constexpr int kRowWgThreads = 256;

// kVec values of a row as float32: kVec = 8 reads 16 or 32 aligned bytes,
// kVec = 1 one value (widths or addresses that are not aligned).
template <int kVec>
__device__ __forceinline__ void load_values(const float *p, float (&v)[kVec]) {
    if constexpr (kVec == 8) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
        v[0] = *p;
    }
}
template <int kVec>
__device__ __forceinline__ void load_values(const __bf16 *p, float (&v)[kVec]) {
    if constexpr (kVec == 8) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
        }
    } else {
        v[0] = float(*p);
    }
}

// The same values out, rounded once (to nearest even) where the type is bf16.
template <int kVec>
__device__ __forceinline__ void store_values(float *p, const float (&v)[kVec]) {
    if constexpr (kVec == 8) {
        *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *p = v[0];
    }
}
template <int kVec>
__device__ __forceinline__ void store_values(__bf16 *p, const float (&v)[kVec]) {
    if constexpr (kVec == 8) {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        bf16x8 h;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = __bf16(v[j]);
        *reinterpret_cast<bf16x8 *>(p) = h;
    } else {
        *p = __bf16(v[0]);
    }
}

// Sum over the kThreads (64: a wave, 256: the workgroup) threads of a row,
// in a fixed order; every one of them gets it.  `lds`: 4 floats that no
// other reduction in flight uses.
template <int kThreads>
__device__ __forceinline__ float row_sum(float v, float *lds) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    if constexpr (kThreads == 256) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    }
    return v;
}

}  // namespace rows
}  // namespace mimo
