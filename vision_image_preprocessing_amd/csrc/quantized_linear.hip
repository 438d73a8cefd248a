// quantized_linear.hip -- rows quantised to 8-bit integers and the matrix
// product of two such matrices, for AMD Instinct MI355X (gfx950, CDNA4).
//
// What is computed.  quantize_rows: scale = max |x| / 127 of each row, q =
// x / scale rounded to the nearest integer (ties to even), so that x is near
// scale * q; the same for the rows of a weight, whose rows are its output
// channels.  quantized_linear: with rows' scales s_r and channels' scales t_e,
//   out[r][e] = (sum_k xq[r][k] wq[e][k]) s_r t_e + bias[e]
// The sum is exact: products of 8-bit integers on v_mfma_i32_32x32x32_i8 into
// 32-bit integers, which 2^17 of them cannot overflow.  It is rounded to
// float32, multiplied by s_r, and then by t_e with the bias added in one
// operation, in every kernel here: a row's result does not depend on how many
// rows it comes with.  (The product of the two scales alone could leave
// float32's range where the result does not.  So could the sum times s_r, of
// rows with a scale of 2^97 or more: from kFarScale on, 2^32 is moved from s_r
// to t_e, which changes no rounding.)
//
// Quantised rows are padded with zeros to a multiple of 128 bytes: rows of
// whole 128-byte K steps, so the product needs no tail in K.
#include <hip/hip_runtime.h>

#include <cstring>
#include <string>
#include <type_traits>

#include "device_util.h"
#include "internal.h"
#include "row_ops.h"
#include "runtime.h"

namespace mimo {
namespace {

using namespace rows;

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kPadK = 128;          // quantised rows are multiples of this
constexpr int kMaxK = 130944;       // 2^14 kMaxK < 2^31: no overflow, values of -128 included
constexpr int kThreads = kRowWgThreads;
constexpr int kFewThreads = 512;

struct QuantizeArgs {
    const void *x;
    int8_t *q;      // [rows][padded]
    float *scale;   // [rows]
    int64_t rows;
    int32_t width, padded;
};

// One row by a wave (kThreadsRow = 64) or the workgroup, held in registers
// (kChunks chunks of eight values a thread), or read twice (kChunks = 0).
// 131072 x 1536 bf16: 107 to 119 us, 0.60 GB at 5.1 to 5.6 TB/s, with the VALU
// about as busy as memory; 4096 x 1283 float32: 9 us.
template <typename T, bool kRagged, int kThreadsRow, int kChunks>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QuantizeArgs a) {
    __shared__ uint32_t lds[4];
    const int tid = threadIdx.x % kThreadsRow;
    const int64_t row = row_group() * (kThreads / kThreadsRow) + threadIdx.x / kThreadsRow;
    if (row >= a.rows) return;
    const T *x = static_cast<const T *>(a.x) + row * a.width;
    int8_t *q = a.q + row * a.padded;
    const int count = (a.padded / 8 + kThreadsRow - 1) / kThreadsRow;
    float v[kChunks ? kChunks : 1][8];
    uint32_t top = 0;
    auto column = [&](int i) { return (i * kThreadsRow + tid) * 8; };
    // past the row's end a chunk reads zeros, which is what padding holds
    auto load = [&](int i, float (&w)[8]) {
        if (column(i) < a.width) {
            load_values<kRagged>(x + column(i), a.width - column(i), w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.0f;
        }
    };
    auto look = [&](int i, float (&w)[8]) {
        load(i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, magnitude(w[j]));
    };
    if constexpr (kChunks > 0) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) look(i, v[i]);
    } else {
        for (int i = 0; i < count; ++i) look(i, v[0]);
    }
    top = row_max<kThreadsRow>(top, lds);
    // a row that is not finite has the scale NaN and zeros, which make its
    // outputs NaN; a row of zeros (or too small for a scale) has the scale 0
    const bool finite = top < 0x7F800000u;
    const float scale = finite ? __builtin_bit_cast(float, top) / 127.0f : __builtin_nanf("");
    const bool none = !finite || scale == 0.0f;
    const float inv = 1.0f / scale;
    auto write = [&](int i, const float (&w)[8]) {
        const u32x2 p = none ? u32x2{0, 0} : quantize(w, scale, inv);
        if (column(i) < a.padded) *reinterpret_cast<u32x2 *>(q + column(i)) = p;
    };
    if constexpr (kChunks > 0) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) write(i, v[i]);
    } else {
        for (int i = 0; i < count; ++i) {
            load(i, v[0]);
            write(i, v[0]);
        }
    }
    if (tid == 0) a.scale[row] = scale;
}

struct LinearArgs {
    const int8_t *x, *w;          // [n_rows][k], [e][k]
    const float *x_scale, *w_scale, *bias;  // bias or null
    void *out;                    // OutT [n_rows][e]
    int64_t n_rows;
    int32_t e, k;                 // k: a multiple of 128
    int32_t n_tiles;              // tiles along e
};

// A row's scale from kFarScale on is taken 2^-32 times, so that its product
// with a sum (of up to 2^31) stays below 2^128, and the channel's 2^32 times.
// All of that is exact, but for a channel's scale that would become infinite:
// as the largest float it makes the same results, zero where the sum is zero
// and else infinite (2^64 times 2^96).
constexpr float kFarScale = 0x1p64f;
__device__ __forceinline__ bool is_far(float row_scale) { return fabsf(row_scale) >= kFarScale; }
__device__ __forceinline__ float near_row_scale(float s) { return is_far(s) ? s * 0x1p-32f : s; }
__device__ __forceinline__ float far_channel_scale(float t) {
    const float u = t * 0x1p32f;
    return fabsf(u) == INFINITY && fabsf(t) != INFINITY ? copysignf(0x1.fffffep127f, t) : u;
}

__device__ __forceinline__ i32x16 mfma(const i32x4 &a, const i32x4 &b, const i32x16 &c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// LDS position (in bytes) of 16-byte chunk v of row r: 128-byte rows whose
// chunks are XOR-swizzled by the row.
__device__ __forceinline__ int lds_at(int r, int v) { return r * 128 + ((v ^ ((r ^ (r >> 3)) & 7)) << 4); }

// 16 bytes of a row, non-temporal; rows of any width start at any address of
// the type, which the hardware takes.
__device__ __forceinline__ void store_piece(float *p, const float (&v)[4]) {
    typedef f32x4 any_f32x4 __attribute__((aligned(4)));
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<any_f32x4 *>(p));
}
__device__ __forceinline__ void store_piece(__bf16 *p, const float (&v)[8]) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    typedef u32x4 any_u32x4 __attribute__((aligned(2)));
    bf16x8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __bf16(v[j]);
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), reinterpret_cast<any_u32x4 *>(p));
}

// A kTile x kTile tile by four waves, a quarter each: 256 x 256 (256
// accumulators a lane, one workgroup a CU), whose LDS bytes per product are
// low enough that the matrix cores set the pace, or 128 x 128 (two workgroups
// a CU) where larger tiles would leave CUs idle.  K advances 128 bytes a
// stage; operands go from memory straight into LDS (buffer_load ... lds), x
// two stages ahead of the products (three buffers), the weight one (two
// buffers).  The five buffers are arrays of their own, so that the compiler
// sees that the loads into one never meet the reads of another; the stage
// loop is unrolled six times, after which both rings are back where they
// were.  Stages past the end are loaded through an empty resource: zeros,
// without memory traffic.
//
// 131072 x 1280 bf16 of K 5120: 785 us, 2.19 POP/s, next to 2.48 that a square
// library product of 8192 reaches; of K 1536: 329 to 375 us, 1.4 to 1.6 POP/s,
// where a tile's first loads and its store (0.34 GB in all) take about a third
// of its time, by the rate at K 5120, and nothing else runs on the CU meanwhile.
// A workgroup that stays and loads its next tile's first stages under the store
// took 3 to 5% longer (374 us against 360; 65536 x 5120: 595 against 555), 256
// x 128 tiles of 64-byte stages 322 us against 303.  128 x 128 tiles: 4096 x
// 1290 float32 of K 1408, 16 to 18 us.
typedef __attribute__((address_space(3))) void *lds_void_ptr;
constexpr int kWord3 = 0x00020000;            // raw buffer resource word 3
constexpr int kRecords = 0x7FFFFFF0;          // its size; tile offsets are below 2^25
// s_waitcnt immediates (gfx9 layout: vmcnt in bits 3:0 and 15:14, expcnt in
// 6:4, lgkmcnt in 11:8; a field at its maximum does not wait).
constexpr int kWaitAll = 0;

template <typename OutT, int kTile>
__global__ __launch_bounds__(kThreads) void linear_tile_kernel(LinearArgs a) {
    constexpr int kWave = kTile / 2, kBlocks = kWave / 32;  // a wave's quarter, in blocks of 32
    constexpr int kGroups = kTile / 8 / 4;    // groups of eight rows a wave loads of each operand
    constexpr int kSteps = 4;                 // products of 32 bytes of K in a stage
    constexpr int kWaitVmemButX = 0x0F70 | kGroups;     // vmcnt: one stage of x may stay in flight
    constexpr int kWaitLdsVmemButX = 0x0070 | kGroups;  // the same, and lgkmcnt(0)
    // two loads go out after each row of products, the weight's first: all of
    // them before the stage's wait, which counts on x's being the newest
    static_assert(kGroups <= 15 && kGroups <= (kSteps - 1) * kBlocks, "every load is issued before the last step");
    __shared__ uint8_t sx0[kTile * 128], sx1[kTile * 128], sx2[kTile * 128];
    __shared__ uint8_t sw0[kTile * 128], sw1[kTile * 128];
    const int64_t tile = xcd_contiguous_tile(blockIdx.x, gridDim.x);
    const int64_t mt = tile / a.n_tiles;
    const int64_t m0 = mt * kTile;
    const int n0 = int(tile - mt * a.n_tiles) * kTile;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int stages = a.k / 128;

    // Lane l of a wave's load lands at row l / 8, chunk l % 8 of a group of
    // eight rows, so it fetches the chunk that the swizzle puts there.  Rows
    // past the last one read the last one; they are not stored.
    auto rsrc = [&](const int8_t *p, int s) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(p), 0, s < stages ? kRecords : 0, kWord3);
    };
    auto x_rsrc = [&](int s) { return rsrc(a.x + m0 * a.k, s); };
    auto w_rsrc = [&](int s) { return rsrc(a.w + int64_t(n0) * a.k, s); };
    uint32_t x_off[kGroups], w_off[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int r = (wave * kGroups + i) * 8 + (lane >> 3);
        const int v = (lane & 7) ^ ((r ^ (r >> 3)) & 7);
        x_off[i] = uint32_t(int(min(m0 + r, a.n_rows - 1) - m0) * a.k + v * 16);
        w_off[i] = uint32_t((min(n0 + r, a.e - 1) - n0) * a.k + v * 16);
    }
    auto load = [&](const __amdgpu_buffer_rsrc_t &r, uint32_t off, int i, int s, uint8_t *d) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)(d + (wave * kGroups + i) * 1024), 16, off, s < stages ? s * 128 : 0, 0, 0);
    };
    auto load_x = [&](int i, int s, uint8_t *d) { load(x_rsrc(s), x_off[i], i, s, d); };
    auto load_w = [&](int i, int s, uint8_t *d) { load(w_rsrc(s), w_off[i], i, s, d); };
    // between stages: each wave has waited for its own loads and reads
    auto barrier = [] {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    i32x16 acc[kBlocks][kBlocks];  // [rows][channels]
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) acc[i][j] = i32x16{};
    i32x4 fx[2][kBlocks], fw[2][kBlocks];
    auto read = [&](const uint8_t *tx, const uint8_t *tw, int s, i32x4 (&x)[kBlocks], i32x4 (&w)[kBlocks]) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) x[i] = *reinterpret_cast<const i32x4 *>(tx + lds_at(wm * kWave + i * 32 + (lane & 31), 2 * s + (lane >> 5)));
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) w[i] = *reinterpret_cast<const i32x4 *>(tw + lds_at(wn * kWave + i * 32 + (lane & 31), 2 * s + (lane >> 5)));
    };
#pragma unroll
    for (int i = 0; i < kGroups; ++i) load_x(i, 0, sx0);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) load_w(i, 0, sw0);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) load_x(i, 1, sx1);
    __builtin_amdgcn_s_waitcnt(kWaitVmemButX);
    barrier();
    read(sx0, sw0, 0, fx[0], fw[0]);
    // One stage: the next step's operands are read while this one's products
    // run; the loads go out in its first half, two after each row of four
    // products; before the last step's products, whose operands are in
    // registers, the waves meet and read the next stage's first operands.
    auto stage = [&](int s, const uint8_t *tx, const uint8_t *tw, uint8_t *nw, uint8_t *nx2, const uint8_t *nx,
                     const uint8_t *nwr) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
            if (ks + 1 < kSteps) {
                read(tx, tw, ks + 1, fx[(ks + 1) & 1], fw[(ks + 1) & 1]);
            } else {
                __builtin_amdgcn_s_waitcnt(kWaitLdsVmemButX);
                barrier();
                read(nx, nwr, 0, fx[0], fw[0]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) acc[i][j] = mfma(fw[ks & 1][j], fx[ks & 1][i], acc[i][j]);
                const int slot = ks * kBlocks + i;
#pragma unroll
                for (int n = 2 * slot; n < 2 * slot + 2; ++n) {
                    if (n < kGroups)
                        load_w(n, s + 1, nw);
                    else if (n < 2 * kGroups)
                        load_x(n - kGroups, s + 2, nx2);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // stage u of a group of six
    auto ring = [&](int s, auto number) __attribute__((always_inline)) {
        constexpr int u = decltype(number)::value;
        uint8_t *const x = u % 3 == 0 ? sx0 : u % 3 == 1 ? sx1 : sx2, *const x1 = u % 3 == 0 ? sx1 : u % 3 == 1 ? sx2 : sx0;
        uint8_t *const x2 = u % 3 == 0 ? sx2 : u % 3 == 1 ? sx0 : sx1;
        uint8_t *const w = u % 2 ? sw1 : sw0, *const w1 = u % 2 ? sw0 : sw1;
        stage(s, x, w, w1, x2, x1, w1);
    };
    typedef std::integral_constant<int, 0> U0;
    typedef std::integral_constant<int, 1> U1;
    typedef std::integral_constant<int, 2> U2;
    typedef std::integral_constant<int, 3> U3;
    typedef std::integral_constant<int, 4> U4;
    typedef std::integral_constant<int, 5> U5;
    int s = 0;
    for (; s + 6 <= stages; s += 6) {
        ring(s, U0());
        ring(s + 1, U1());
        ring(s + 2, U2());
        ring(s + 3, U3());
        ring(s + 4, U4());
        ring(s + 5, U5());
    }
    // the rest, nested: where two paths met, the compiler could not tell which
    // loads are in flight and would wait for all of them before the next read
    const int rest = stages - s;
    if (rest > 0) {
        ring(s, U0());
        if (rest > 1) {
            ring(s + 1, U1());
            if (rest > 2) {
                ring(s + 2, U2());
                if (rest > 3) {
                    ring(s + 3, U3());
                    if (rest > 4) ring(s + 4, U4());
                }
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    barrier();

    // Each wave turns its block in LDS, 32 rows at a time (float32, 16-byte
    // chunks XOR-swizzled by the row): a lane then holds whole pieces of
    // rows, whose channels are the same for every row.
    constexpr int kRowBytes = kWave * 4, kChunks = kRowBytes / 16;
    uint8_t *region = (wave < 2 ? sx0 : sx1) + (wave & 1) * (32 * kRowBytes);
    static_assert(2 * 32 * kRowBytes <= kTile * 128, "two waves share a buffer");
    constexpr int kOut = 16 / int(sizeof(OutT)), kLanes = kWave / kOut, kPass = 64 / kLanes;
    const int piece = lane % kLanes;
    const int col = n0 + wn * kWave + piece * kOut;
    float t[kOut], b[kOut];
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
        const int e = min(col + j, a.e - 1);
        t[j] = a.w_scale[e];
        b[j] = a.bias ? a.bias[e] : 0.0f;
    }
    const bool whole = col + kOut <= a.e;  // at any address of the type: see store_piece
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int r = lane & 31;
        const float row_scale = a.x_scale[min(m0 + wm * kWave + i * 32 + r, a.n_rows - 1)];
        const float xs = near_row_scale(row_scale);
        const uint32_t far = uint32_t(__ballot(is_far(row_scale)));  // of rows 0 .. 31; the half-waves agree
#pragma unroll
        for (int j = 0; j < kBlocks; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = j * 8 + 2 * g + (lane >> 5);
                const f32x4 v = {float(acc[i][j][4 * g]) * xs, float(acc[i][j][4 * g + 1]) * xs, float(acc[i][j][4 * g + 2]) * xs,
                                 float(acc[i][j][4 * g + 3]) * xs};
                *reinterpret_cast<f32x4 *>(region + r * kRowBytes + ((c ^ r) % kChunks) * 16) = v;
            }
        // twice, since a branch in each pass would keep the passes apart
        // (131072 x 1280 of K 1536: 425 us with quantising, against 413)
        auto store = [&](auto some_far) __attribute__((always_inline)) {
#pragma unroll
            for (int p = 0; p < 32 / kPass; ++p) {
                const int rr = p * kPass + lane / kLanes;
                float v[kOut];
#pragma unroll
                for (int k = 0; k < kOut / 4; ++k) {
                    const f32x4 w = *reinterpret_cast<const f32x4 *>(region + rr * kRowBytes + (((piece * (kOut / 4) + k) ^ rr) % kChunks) * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float scale = t[4 * k + j];
                        v[4 * k + j] = fmaf(w[j], decltype(some_far)::value && (far >> rr & 1) ? far_channel_scale(scale) : scale, b[4 * k + j]);
                    }
                }
                const int64_t row = m0 + wm * kWave + i * 32 + rr;
                if (row >= a.n_rows) continue;
                OutT *out = static_cast<OutT *>(a.out) + row * a.e + col;
                if (whole) {
                    store_piece(out, v);
                } else {
#pragma unroll
                    for (int j = 0; j < kOut; ++j)
                        if (col + j < a.e) out[j] = OutT(v[j]);
                }
            }
        };
        if (far)
            store(std::true_type());
        else
            store(std::false_type());
    }
}

// Few rows: a workgroup takes 32 rows and 32 channels, its eight waves share
// K, and each has the operands of eight products (2 KB of K over the
// workgroup) on the way from memory at once, which is what such a call waits
// for; the waves' sums meet in LDS.  4 x 1280 of K 1280: 4 us, a launch's length.
template <typename OutT>
__global__ __launch_bounds__(kFewThreads) void linear_few_kernel(LinearArgs a) {
    constexpr int kWaves = kFewThreads / 64, kDeep = 8;
    __shared__ int32_t part[kWaves][16][64];
    const int64_t mt = blockIdx.x / a.n_tiles;
    const int64_t m0 = mt * 32;
    const int n0 = int(blockIdx.x - mt * a.n_tiles) * 32;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int8_t *x = a.x + min(m0 + (lane & 31), a.n_rows - 1) * a.k + 16 * (lane >> 5);
    const int8_t *w = a.w + int64_t(min(n0 + (lane & 31), a.e - 1)) * a.k + 16 * (lane >> 5);
    i32x16 acc{};
    for (int k0 = 32 * wave; k0 < a.k; k0 += 32 * kWaves * kDeep) {
        i32x4 fx[kDeep], fw[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int k = k0 + 32 * kWaves * i;
            if (k < a.k) {
                fw[i] = *reinterpret_cast<const i32x4 *>(w + k);
                fx[i] = *reinterpret_cast<const i32x4 *>(x + k);
            } else {
                fw[i] = fx[i] = i32x4{};
            }
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) acc = mfma(fw[i], fx[i], acc);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) part[wave][r][lane] = acc[r];
    __syncthreads();
    // two channels of a row each: value r of lane l is channel 8 (r / 4) +
    // 4 (l / 32) + r % 4 of row l % 32
    const int64_t row = m0 + threadIdx.x / 16;
    if (row >= a.n_rows) return;
    const float s = a.x_scale[row], near = near_row_scale(s);
    OutT *out = static_cast<OutT *>(a.out) + row * a.e;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 2 * (threadIdx.x % 16) + j, e = n0 + c;
        if (e >= a.e) return;
        const int r = 4 * (c / 8) + c % 4, l = int(threadIdx.x / 16) + 32 * ((c >> 2) & 1);
        int32_t sum = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) sum += part[i][r][l];
        const float t = a.w_scale[e];
        out[e] = OutT(fmaf(float(sum) * near, is_far(s) ? far_channel_scale(t) : t, a.bias ? a.bias[e] : 0.0f));
    }
}

}  // namespace
}  // namespace mimo

using namespace mimo;

extern "C" {

int mimo_quantize_rows(int64_t rows, int32_t width, const void *x, int32_t x_dtype, void *q, float *scale, void *stream) {
    clear_error();
    if (rows < 0 || width < 1) return set_error(MIMO_E_INVALID, "quantize_rows: rows must be >= 0 and width >= 1");
    if (width > kMaxK || rows > 0x7FFFFFFFll)
        return set_error(MIMO_E_TOO_LARGE, "quantize_rows: width above 130944 or more than 2^31 - 1 rows");
    if (x_dtype != MIMO_F32 && x_dtype != MIMO_BF16)
        return set_error(MIMO_E_INVALID, "quantize_rows: x_dtype must be MIMO_F32 or MIMO_BF16");
    if (rows == 0) return MIMO_OK;
    if (!x || !q || !scale || !check_ptr_align(x, x_dtype == MIMO_F32 ? 4 : 2) || !check_ptr_align(q, 16) || !check_ptr_align(scale, 4))
        return set_error(MIMO_E_INVALID, "quantize_rows: null or misaligned pointer (x to its values, q 16 bytes, scale 4)");
    if (q == x) return set_error(MIMO_E_INVALID, "quantize_rows: q must not be x");
    QuantizeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.q = static_cast<int8_t *>(q);
    a.scale = scale;
    a.rows = rows;
    a.width = width;
    a.padded = (width + kPadK - 1) / kPadK * kPadK;
    const bool ragged = width % 8 || !check_ptr_align(x, 16);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 block{unsigned(kThreads), 1, 1};
    // the padding is written by the threads that hold the row, so the widths
    // are those that the padded row fits
    auto launch = [&](auto type, auto ragged) {
        typedef decltype(type) T;
        constexpr bool R = decltype(ragged)::value;
        const dim3 waves = row_grid((rows + 3) / 4), groups = row_grid(rows);
        if (a.padded <= 64 * 8)
            hipLaunchKernelGGL((quantize_rows_kernel<T, R, 64, 1>), waves, block, 0, s, a);
        else if (a.padded <= 64 * 8 * 3)
            hipLaunchKernelGGL((quantize_rows_kernel<T, R, 64, 3>), waves, block, 0, s, a);
        else if (a.padded <= 256 * 8 * 3)
            hipLaunchKernelGGL((quantize_rows_kernel<T, R, 256, 3>), groups, block, 0, s, a);
        else
            hipLaunchKernelGGL((quantize_rows_kernel<T, R, 256, 0>), groups, block, 0, s, a);
    };
    const hipError_t e = timed_launch(s, [&] {
        if (x_dtype == MIMO_F32 && ragged)
            launch(float(), std::true_type());
        else if (x_dtype == MIMO_F32)
            launch(float(), std::false_type());
        else if (ragged)
            launch(__bf16(), std::true_type());
        else
            launch(__bf16(), std::false_type());
    });
    if (e != hipSuccess) return hip_error(e, "quantize_rows: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

int mimo_quantized_linear(int64_t n_rows, int32_t k, const void *xq, const float *x_scale, int32_t embed_dim, const void *wq,
                          const float *w_scale, const float *bias, int32_t out_dtype, void *out, void *stream) {
    clear_error();
    if (n_rows < 0 || embed_dim < 1 || k < kPadK || k % kPadK)
        return set_error(MIMO_E_INVALID, "quantized_linear: n_rows must be >= 0, embed_dim >= 1, k a multiple of 128");
    if (k > kMaxK || embed_dim > (1 << 24) || n_rows > 0x7FFFFFFFll)
        return set_error(MIMO_E_TOO_LARGE, "quantized_linear: k above 130944, embed_dim above 2^24 or more than 2^31 - 1 rows");
    if (out_dtype != MIMO_F32 && out_dtype != MIMO_BF16)
        return set_error(MIMO_E_INVALID, "quantized_linear: out_dtype must be MIMO_F32 or MIMO_BF16");
    if (n_rows == 0) return MIMO_OK;
    if (!xq || !x_scale || !wq || !w_scale || !out || !check_ptr_align(xq, 16) || !check_ptr_align(wq, 16) || !check_ptr_align(out, 16) ||
        !check_ptr_align(x_scale, 4) || !check_ptr_align(w_scale, 4) || !check_ptr_align(bias, 4))
        return set_error(MIMO_E_INVALID, "quantized_linear: null or misaligned pointer (xq, wq, out: 16 bytes; scales and bias: 4)");
    if (out == xq || out == wq) return set_error(MIMO_E_INVALID, "quantized_linear: out must not be an input");
    LinearArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = static_cast<const int8_t *>(xq);
    a.w = static_cast<const int8_t *>(wq);
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.bias = bias;
    a.out = out;
    a.n_rows = n_rows;
    a.e = embed_dim;
    a.k = k;
    // Which kernel, by size alone (us, 128 x 128 tiles against the other, K
    // 1280 or 1536 unless said).  Blocks of 32 x 32, while at most one falls
    // to each CU or one row of them reads the weight once: 4 rows x 1280: 7.8
    // against 6.5; 128 x 1280: 8.8 against 6.8; 32 x 5120, K 5120: 17.0
    // against 12.9; past that, 256 x 1280: 8.9 against 9.8.  256 x 256 tiles,
    // from four rounds of the card's 256 CUs on: 65536 x 1280: 148 against
    // 144; 65536 x 5120: 620 against 530; 131072 x 1280, K 5120: 947 against
    // 755; before that, 32768 x 1280: 77 against 83.
    const int64_t m32 = (n_rows + 31) / 32, n32 = (int64_t(embed_dim) + 31) / 32;
    const int64_t m128 = (n_rows + 127) / 128, n128 = (int64_t(embed_dim) + 127) / 128;
    const int64_t m256 = (n_rows + 255) / 256, n256 = (int64_t(embed_dim) + 255) / 256;
    const bool few = m32 == 1 || m32 * n32 <= 256, big = !few && m256 * n256 >= 1024;
    const int64_t tiles = few ? m32 * n32 : big ? m256 * n256 : m128 * n128;
    a.n_tiles = int32_t(few ? n32 : big ? n256 : n128);
    if (tiles > (int64_t(1) << 24) - 1) return set_error(MIMO_E_TOO_LARGE, "quantized_linear: more than 2^24 - 1 tiles");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid{unsigned(tiles), 1, 1}, block{unsigned(few ? kFewThreads : kThreads), 1, 1};
    const hipError_t e = timed_launch(s, [&] {
        if (few && out_dtype == MIMO_F32)
            hipLaunchKernelGGL(linear_few_kernel<float>, grid, block, 0, s, a);
        else if (few)
            hipLaunchKernelGGL(linear_few_kernel<__bf16>, grid, block, 0, s, a);
        else if (big && out_dtype == MIMO_F32)
            hipLaunchKernelGGL((linear_tile_kernel<float, 256>), grid, block, 0, s, a);
        else if (big)
            hipLaunchKernelGGL((linear_tile_kernel<__bf16, 256>), grid, block, 0, s, a);
        else if (out_dtype == MIMO_F32)
            hipLaunchKernelGGL((linear_tile_kernel<float, 128>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((linear_tile_kernel<__bf16, 128>), grid, block, 0, s, a);
    });
    if (e != hipSuccess) return hip_error(e, "quantized_linear: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

}  // extern "C"
