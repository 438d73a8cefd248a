// rotate_heads.hip -- the rotation of query and key heads by the rotary
// tables, and its inverse for their gradients, for AMD Instinct MI355X
// (gfx950).
//
// What is computed (NeMo Automodel "mimo_v2_flash.vision",
// _apply_rotary_pos_emb and _rotate_half), for every head of row r, with
// half = head_dim / 2 and the tables' row of half cosines and sines:
//   out_i        = x_i        c_i - x_{i + half} s_i       i < half
//   out_{i+half} = x_{i+half} c_i + x_i        s_i
// The inverse takes -s: it is the transposed matrix, so the gradient of x is
// the inverse rotation of out's.  Products and sums are float32, rounded once.
//
// Memory bounds it: 112640 rows of 40 heads of 64 in 229 to 234 us, 0.61 GB read,
// 0.58 written, 5.0 to 5.1 TB/s, what a copy of 1 GiB reaches, but not the most: the
// norm of rms_norm.hip moves 5.8 to 6.0.  A wave takes one row; a lane's piece is
// eight values of a head's first half and the eight that belong to them in the
// second, so that neighbouring lanes read neighbouring 16 bytes, four of them (at
// head_dim 64) each half of a line.
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

struct RotateArgs {
    const uint16_t *x;
    uint16_t *out;
    int64_t x_row, x_head, out_row, out_head;  // strides, in values
    const float *cos, *sin;                    // [rows][half]
    int64_t rows;
    int32_t heads, half;
    float sign;                                // of the sines
};

// kN of the values from p on (8: 16 bytes, 4: 8 bytes) as float32.
template <int kN>
__device__ __forceinline__ void load_piece(const uint16_t *p, float (&v)[kN]) {
    typedef uint32_t words __attribute__((ext_vector_type(kN / 2)));
    const words w = *reinterpret_cast<const words *>(p);
#pragma unroll
    for (int j = 0; j < kN / 2; ++j) {
        v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
        v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
    }
}
template <int kN>
__device__ __forceinline__ void store_piece(uint16_t *p, const float (&v)[kN]) {
    typedef __bf16 halves __attribute__((ext_vector_type(kN)));
    halves h;
#pragma unroll
    for (int j = 0; j < kN; ++j) h[j] = __bf16(v[j]);
    *reinterpret_cast<halves *>(p) = h;
}
template <int kN>
__device__ __forceinline__ void load_table(const float *p, float (&v)[kN]) {
#pragma unroll
    for (int j = 0; j < kN; j += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(p + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j + i] = w[i];
    }
}

template <int kN>
__global__ __launch_bounds__(kRowWgThreads) void rotate_heads_kernel(RotateArgs a) {
    const int64_t row = row_group() * (kRowWgThreads / 64) + (threadIdx.x >> 6);
    if (row >= a.rows) return;
    const int pieces = a.half / kN, items = a.heads * pieces;
    for (int item = threadIdx.x & 63; item < items; item += 64) {
        const int head = item / pieces, at = (item - head * pieces) * kN;
        float c[kN], s[kN], u[kN], v[kN];
        const uint16_t *x = a.x + row * a.x_row + head * a.x_head + at;
        load_piece<kN>(x, u);
        load_piece<kN>(x + a.half, v);
        load_table<kN>(a.cos + row * a.half + at, c);
        load_table<kN>(a.sin + row * a.half + at, s);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const float sj = s[j] * a.sign, first = u[j] * c[j] - v[j] * sj;
            v[j] = v[j] * c[j] + u[j] * sj;
            u[j] = first;
        }
        uint16_t *out = a.out + row * a.out_row + head * a.out_head + at;
        store_piece<kN>(out, u);
        store_piece<kN>(out + a.half, v);
    }
}

// The strides that mimo_chunk_attention takes, and a tensor that is written
// must not overlap itself.
bool heads_ok(const mimo_heads *t, int64_t rows, int32_t heads, int32_t head_dim, bool written) {
    if (!t->data || !check_ptr_align(t->data, 16) || t->row_stride % 8 || t->head_stride % 8) return false;
    if (t->row_stride < head_dim || t->row_stride > (int64_t(1) << 22) || t->head_stride < 0 || t->head_stride > (int64_t(1) << 40))
        return false;
    return !written || heads == 1 ||
           (t->head_stride >= head_dim && t->row_stride >= (heads - 1) * t->head_stride + head_dim) ||
           t->head_stride >= (rows - 1) * t->row_stride + head_dim;
}

// Whether two rows of heads, the second `offset` values behind the first, share
// a value: both by ascending addresses, going on from whichever head is behind.
bool rows_meet(int64_t offset, int64_t x_head, int64_t out_head, int32_t heads, int32_t head_dim) {
    for (int32_t i = 0, j = 0; i < heads && j < heads;) {
        const int64_t apart = offset + j * out_head - i * x_head;
        if (apart > -head_dim && apart < head_dim) return true;
        if (apart > 0)
            ++i;
        else
            ++j;
    }
    return false;
}

// Whether a value of out lies where one of x does: waves would write heads that
// others, or their own next pass, still read.  Tensors that are apart, and those
// of one row stride that go through one array side by side (heads of one
// projection's output), are told apart; others that go through the same
// addresses are taken to meet.
bool heads_meet(const mimo_heads &x, const mimo_heads &out, int64_t rows, int32_t heads, int32_t head_dim) {
    const int64_t delta = (reinterpret_cast<intptr_t>(out.data) - reinterpret_cast<intptr_t>(x.data)) / 2;
    const int64_t x_span = (heads - 1) * x.head_stride + head_dim, out_span = (heads - 1) * out.head_stride + head_dim;  // of a row
    if (delta >= (rows - 1) * x.row_stride + x_span || -delta >= (rows - 1) * out.row_stride + out_span) return false;
    if (rows == 1) return rows_meet(delta, x.head_stride, out.head_stride, heads, head_dim);
    const int64_t stride = x.row_stride;
    if (out.row_stride != stride) return true;
    // rows of out from here on lie `behind` behind a row of x, `shift` rows on
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    if (x_span <= stride && out_span <= stride) {
        const int64_t shift = floor_div(delta, stride), behind = delta - shift * stride;
        auto exists = [&](int64_t s) { return s > -rows && s < rows; };
        return (exists(shift) && rows_meet(behind, x.head_stride, out.head_stride, heads, head_dim)) ||
               (exists(shift + 1) && rows_meet(behind - stride, x.head_stride, out.head_stride, heads, head_dim));
    }
    if (heads > 1 && out.head_stride != x.head_stride) return true;
    // heads as far from each other in both: any two of them, by how many heads apart, with the nearest rows
    for (int64_t apart = 1 - heads; apart < heads; ++apart) {
        const int64_t at = delta + apart * x.head_stride, near = floor_div(at, stride);
        for (int64_t s = near; s <= near + 1; ++s) {
            const int64_t k = s < 1 - rows ? 1 - rows : s > rows - 1 ? rows - 1 : s, left = at - k * stride;
            if (left > -head_dim && left < head_dim) return true;
        }
    }
    return false;
}

}  // namespace
}  // namespace mimo

using namespace mimo;

extern "C" {

int mimo_rotate_heads(int64_t rows, int32_t heads, int32_t head_dim, const mimo_heads *x, const float *cos, const float *sin,
                      int32_t inverse, const mimo_heads *out, void *stream) {
    clear_error();
    if (rows < 0 || heads < 1 || heads > 65536 || head_dim < 8 || head_dim % 8 || head_dim > 2 * MIMO_ROPE_DIM_MAX)
        return set_error(MIMO_E_INVALID, "rotate_heads: rows must be >= 0, heads in [1, 65536], head_dim a multiple of 8 in [8, 512]");
    if (rows > (int64_t(1) << 29)) return set_error(MIMO_E_TOO_LARGE, "rotate_heads: more than 2^29 rows");
    if (!x || !out) return set_error(MIMO_E_INVALID, "rotate_heads: x and out must be given");
    if (rows == 0) return MIMO_OK;
    if (!heads_ok(x, rows, heads, head_dim, false) || !heads_ok(out, rows, heads, head_dim, true))
        return set_error(MIMO_E_INVALID, "rotate_heads: x and out must be non-null and 16-byte aligned, their strides multiples of 8 "
                                         "(row_stride in [head_dim, 2^22], head_stride >= 0), out's rows and heads apart");
    if (out->data == x->data && ((rows > 1 && out->row_stride != x->row_stride) || (heads > 1 && out->head_stride != x->head_stride)))
        return set_error(MIMO_E_INVALID, "rotate_heads: out may be x only with x's strides");
    if (out->data != x->data && heads_meet(*x, *out, rows, heads, head_dim))
        return set_error(MIMO_E_INVALID, "rotate_heads: out must not overlap x, unless it is x");
    if (!cos || !sin || !check_ptr_align(cos, 16) || !check_ptr_align(sin, 16))
        return set_error(MIMO_E_INVALID, "rotate_heads: cos and sin must be non-null and 16-byte aligned");
    const int64_t out_bytes = ((rows - 1) * out->row_stride + (heads - 1) * out->head_stride + head_dim) * 2, table_bytes = rows * head_dim * 2;
    if (arrays_meet(cos, table_bytes, out->data, out_bytes) || arrays_meet(sin, table_bytes, out->data, out_bytes))
        return set_error(MIMO_E_INVALID, "rotate_heads: cos and sin must not lie among out's rows");
    RotateArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = static_cast<const uint16_t *>(x->data);
    a.out = static_cast<uint16_t *>(out->data);
    a.x_row = x->row_stride;
    a.x_head = x->head_stride;
    a.out_row = out->row_stride;
    a.out_head = out->head_stride;
    a.cos = cos;
    a.sin = sin;
    a.rows = rows;
    a.heads = heads;
    a.half = head_dim / 2;
    a.sign = inverse ? -1.0f : 1.0f;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid = row_grid((rows + 3) / 4), block{unsigned(kRowWgThreads), 1, 1};
    const hipError_t e = timed_launch(s, [&] {
        if (a.half % 8 == 0)
            hipLaunchKernelGGL(rotate_heads_kernel<8>, grid, block, 0, s, a);
        else
            hipLaunchKernelGGL(rotate_heads_kernel<4>, grid, block, 0, s, a);
    });
    if (e != hipSuccess) return hip_error(e, "rotate_heads: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

}  // extern "C"
