// gated_mlp.hip -- the gated feed-forward block and its backward pass on the
// bf16 matrix cores of AMD Instinct MI355X (gfx950, CDNA4).
//
// What is computed (NeMo Automodel "mimo_v2_flash.vision": the SwiGLU MLP of
// MiMoVisionBlock), for rows x of D values and H hidden ones:
//   g = x Wg' + bg,  u = x Wu' + bu,  h = silu(g) u,  out = h Wd' + bd
// with silu(g) = g s, s = 1 / (1 + exp -g); and for dout:
//   dh = dout Wd,  dg = dh u s (1 + g (1 - s)),  du = dh g s
//   dx = dg Wg + du Wu,  dWg = dg' x,  dWu = du' x,  dWd = dout' h
//   dbg = sum over rows of dg, and so on
//
// Launches.  Forward: both projections, the activation and the product are one
// kernel, whose tiles hold gate and up of the same channels, so h is formed
// from the accumulators and g, u need not be written; then the projection back.
// Backward: dh's product, whose epilogue forms dg and du; dx over both halves
// of its K; the three weights' gradients in one launch.
//
// Roundings: sums are float32 on the matrix cores; h, dg and du are rounded to
// bf16, once, as operands of the next product, as x, dout and the weights come
// in; outputs are rounded once.  For the backward pass g and u are kept in
// float32: in bf16 their rounding would add half as much again to the error of
// dx and the weights' gradients as the operands' own (relative to them 1.85
// roundings instead of 1.41), and to the biases' gradients, which are sums of
// unrounded dg and du, all of theirs: float32 over a tile's rows (db_down: over
// every 1024th row), and float64 over the tiles' sums.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <string>

#include "column_sums.h"
#include "device_util.h"
#include "gemm_tile.h"
#include "internal.h"
#include "row_ops.h"
#include "runtime.h"

namespace mimo {
namespace {

using namespace gemm;
using rows::row_grid;
using rows::row_group;

constexpr int kMaxWidth = 65536;
constexpr int kMaxTiles = (1 << 23) - 1;  // of up to 512 threads: a launch has fewer than 2^32
constexpr int kPad = 64;  // rows of hidden values, and copied operands, are multiples of this

struct MlpArgs {
    Product p[3];
    uint16_t *out[3];            // bf16 [m][ldo]
    int64_t ldo[3];
    int32_t products;
    Units units;
    const float *bias0, *bias1;  // or null
    float *gate_up;              // [2][rows][ldh], or null
    uint16_t *hidden;            // [rows][ldh]
    uint16_t *dgate, *dup;       // [rows][ldh]
    float *part;                 // partial sums: [slot][tile][tile] of tiles in parts, or of dg and du over rows; or null
    int64_t ldh;
    int32_t channels;            // mlp_few_kernel: of a workgroup
    int32_t all_channels;        // and those that are written, n or the padded n
};

// Eight channels to bf16, at any address of the type; `left` of them inside.
__device__ __forceinline__ void store_bf16(uint16_t *p, const float (&v)[8], int left) {
    typedef u32x4 any_u32x4 __attribute__((aligned(2)));
    bf16x8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __bf16(v[j]);
    if (left >= 8) {
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), reinterpret_cast<any_u32x4 *>(p));
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < left) reinterpret_cast<__bf16 *>(p)[j] = h[j];
    }
}
// Biases of n channels from c on, of `count`.
template <int kN>
__device__ __forceinline__ void load_bias(const float *bias, int c, int count, float (&v)[kN]) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = bias ? bias[min(c + j, count - 1)] : 0.0f;
}

// The tile's rows of a matrix of padded rows ([rows][ldh]), which the
// epilogues read and write four channels a lane, so that every access of a
// wave is whole lines.  What is past the rows or the columns reads as zeros and
// is not written; no branch keeps one access apart from the next.
template <typename T>
struct Panel {
    __amdgpu_buffer_rsrc_t r;
    uint32_t off, step;  // the lane's channels in its first row; from one of its rows to the next
    __device__ __forceinline__ Panel(const T *p, int64_t m0, int64_t m, int tile, int64_t ldh, int row, int rows_apart, int col) {
        const int rows = int(min(m - m0, int64_t(tile))), stride = int(ldh) * int(sizeof(T));
        r = __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(p + m0 * ldh), 0, rows * stride, kWord3);
        const bool in = col < int(ldh);
        off = in ? uint32_t(row * stride + col * int(sizeof(T))) : kOutside;
        step = in ? uint32_t(rows_apart * stride) : 0;
    }
    // One row's after the other.  Past the rows, or from kOutside, an offset is
    // outside the resource.
    __device__ __forceinline__ uint32_t next() {
        const uint32_t at = off;
        off += step;
        return at;
    }
};
constexpr int kStream = 2;  // non-temporal: what is not read again soon
__device__ __forceinline__ void load4(Panel<float> &p, float (&v)[4]) {
    const f32x4 w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(p.r, p.next(), 0, kStream));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = w[j];
}
__device__ __forceinline__ void store4(Panel<float> &p, const float (&v)[4]) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), p.r, p.next(), 0, kStream);
}
__device__ __forceinline__ void store4(Panel<uint16_t> &p, const float (&v)[4]) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const bf16x4 h = {__bf16(v[0]), __bf16(v[1]), __bf16(v[2]), __bf16(v[3])};
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, h), p.r, p.next(), 0, 0);
}

// Eight bf16 values from any address of the type, `left` of them inside (any
// number, none among them); zeros behind.
__device__ __forceinline__ u32x4 load_ragged(const uint16_t *p, int left) {
    typedef u32x4 any_u32x4 __attribute__((aligned(2)));
    typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
    if (left >= 8) return *reinterpret_cast<const any_u32x4 *>(p);
    u16x8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = j < left ? p[j] : uint16_t(0);
    return __builtin_bit_cast(u32x4, h);
}

// s = 1 / (1 + exp -g) by the hardware's exponential and reciprocal.  The
// exponential is one of 2 of a float32 product, so its error grows with the
// gate: at most (2 |g| + 2) 2^-24 relative, tens of units in the last place at g =
// -80, where s is next to 0; it moves silu by 2 2^-24 at most, since g^2 s (1 - s) < 1.
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// Which product of a launch a tile is of.
__device__ __forceinline__ int product_of(const MlpArgs &a, int tile) {
    return a.products > 2 && tile >= a.p[2].first ? 2 : a.products > 1 && tile >= a.p[1].first ? 1 : 0;
}

// h = silu(x Wg' + bg) (x Wu' + bu).
//
// Width 1280, hidden 5120: 131072 rows in 2.83 to 3.00 ms, 1.15 to 1.21 PFLOP/s; K
// is 20 stages, 30 us of a tile's 36, and for its first loads and the epilogue the
// matrix cores wait.  32768 rows with g and u saved 842 to 888 us: 0.86 TFLOP, 1.26
// GB read and 1.68 written, 3.4 TB/s, in tiles of 256 x 256 (of 128 x 128 952 to
// 1047, of 64 x 64 1574).  216 rows 15 to 16 us, in tiles of 64 x 64 that take
// 210 MB in from L2 and wait for that.  hidden is read again by the next product, so its
// stores stay in the caches (non-temporal ones made the kernel 5% slower).
template <int kTile, bool kSaved>
__global__ __launch_bounds__(Tile<kTile>::kThreads) void mlp_gate_kernel(MlpArgs a) {
    const Buffers<kTile> lds = tile_buffers<kTile>();
    typedef Tile<kTile> T;
    constexpr int kHalf = T::kWaveN / 2;
    const Product &p = a.p[0];
    const Place at(p, int(xcd_contiguous_tile(blockIdx.x, gridDim.x)));
    const int64_t m0 = at.mt * kTile;
    const int n0 = at.nt * (kTile / 2);
    Sums<kTile> acc;
    multiply<kTile, false, false, kGateUp>(p, m0, n0, 0, p.stages, lds, acc);
    const Turned<kTile> turned(lds);
    constexpr int kLanes = kHalf / 4, kPass = 64 / kLanes;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int piece = (lane % kLanes) * 4, col = n0 + (wave % T::kWavesN) * kHalf + piece;
    float bg[4], bu[4];
    load_bias(a.bias0, col, p.n, bg);
    load_bias(a.bias1, col, p.n, bu);
    const int row = (wave / T::kWavesN) * T::kWaveM + lane / kLanes;
    Panel<uint16_t> hidden(a.hidden, m0, p.m, kTile, a.ldh, row, kPass, col);
    Panel<float> gate(a.gate_up, m0, p.m, kTile, a.ldh, row, kPass, col), up(a.gate_up + p.m * a.ldh, m0, p.m, kTile, a.ldh, row, kPass, col);
    const bool edge = n0 + kTile / 2 > p.n;  // some of the channels are padding, and zeros
    constexpr int kPasses = 32 / kPass;
#pragma unroll
    for (int i = 0; i < T::kBlocksM; ++i) {
        turned.put(acc[i]);
        float g[kPasses][4], u[kPasses][4];
#pragma unroll
        for (int t = 0; t < kPasses; ++t) {
            turned.get(t * kPass + lane / kLanes, piece, g[t]);
            turned.get(t * kPass + lane / kLanes, kHalf + piece, u[t]);
        }
#pragma unroll
        for (int t = 0; t < kPasses; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[t][j] += bg[j];
                u[t][j] += bu[j];
            }
        }
        if (edge) {
#pragma unroll
            for (int t = 0; t < kPasses; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g[t][j] = col + j < p.n ? g[t][j] : 0.0f;
                    u[t][j] = col + j < p.n ? u[t][j] : 0.0f;
                }
        }
#pragma unroll
        for (int t = 0; t < kPasses; ++t) {
            float h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = g[t][j] * sigmoid(g[t][j]) * u[t][j];
            store4(hidden, h);
            if constexpr (kSaved) {
                store4(gate, g[t]);
                store4(up, u[t]);
            }
        }
    }
}

// dg and du from dh = dout Wd and the saved g, u; partial sums of both over
// the rows of each half of the tile.
//
// 32768 x 1280, hidden 5120: 566 to 619 us, 2.10 GB read, 1.34 of them g and u, and
// 0.68 written, 4.5 to 4.9 TB/s: memory bounds it (tiles of 128 x 128, two
// workgroups a CU, 652 to 665, of 64 x 64 901 to 928).  g and u stay on their way from one block of
// rows to the next.
template <int kTile>
__global__ __launch_bounds__(Tile<kTile>::kThreads) void mlp_dhidden_kernel(MlpArgs a) {
    const Buffers<kTile> lds = tile_buffers<kTile>();
    typedef Tile<kTile> T;
    const Product &p = a.p[0];
    const Place at(p, int(xcd_contiguous_tile(blockIdx.x, gridDim.x)));
    const int64_t m0 = at.mt * kTile;
    const int n0 = at.nt * kTile;
    Sums<kTile> acc;
    multiply<kTile, false, true, kOnce>(p, m0, n0, 0, p.stages, lds, acc);
    const Turned<kTile> turned(lds);
    constexpr int kLanes = T::kWaveN / 4, kPass = 64 / kLanes;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int piece = (lane % kLanes) * 4, col = n0 + (wave % T::kWavesN) * T::kWaveN + piece;
    const int row = (wave / T::kWavesN) * T::kWaveM + lane / kLanes;
    const int rows = int(min(p.m - m0, int64_t(kTile)));
    Panel<float> gate(a.gate_up, m0, p.m, kTile, a.ldh, row, kPass, col), up(a.gate_up + p.m * a.ldh, m0, p.m, kTile, a.ldh, row, kPass, col);
    Panel<uint16_t> dgate(a.dgate, m0, p.m, kTile, a.ldh, row, kPass, col), dup(a.dup, m0, p.m, kTile, a.ldh, row, kPass, col);
    float sg[4] = {}, su[4] = {};
    constexpr int kPasses = 32 / kPass, kAll = T::kBlocksM * kPasses;
    constexpr int kAhead = 8;  // passes whose g and u are on the way (2: 614 us, 4: 612, 8: 608, 12: 614)
    float g[kAll][4], u[kAll][4];
    auto load = [&](int t) __attribute__((always_inline)) {
        if (t >= kAll) return;
        load4(gate, g[t]);
        load4(up, u[t]);
    };
#pragma unroll
    for (int t = 0; t < kAhead; ++t) load(t);
#pragma unroll
    for (int t = 0; t < kAll; ++t) {
        if (t % kPasses == 0) turned.put(acc[t / kPasses]);
        load(t + kAhead);
        float dh[4];
        turned.get(t % kPasses * kPass + lane / kLanes, piece, dh);
        // past the columns dh is any value, and has to be zero for the
        // padding; past the rows g and u are zeros, but dh is zeros times the
        // weights, NaN where one is infinite, and has to be zero for the sums
        const int columns = row + t * kPass < rows ? p.n : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float s = sigmoid(g[t][j]), d = col + j < columns ? dh[j] : 0.0f;
            dh[j] = d * u[t][j] * (s * (1.0f + g[t][j] * (1.0f - s)));
            u[t][j] = d * (g[t][j] * s);
            sg[j] += dh[j];
            su[j] += u[t][j];
        }
        store4(dgate, dh);
        store4(dup, u[t]);
        // added here and now: the compiler would put it off to where the sums
        // are written, keep every value until then and spill (662 us, not 608)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(sg[j]), "+v"(su[j]));
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = kLanes; m < 64; m <<= 1) {
            sg[j] += __shfl_xor(sg[j], m);
            su[j] += __shfl_xor(su[j], m);
        }
    if (lane < kLanes && col < a.ldh) {
        float *part = a.part + (2 * at.mt + wave / T::kWavesN) * 2 * a.ldh + col;
        *reinterpret_cast<f32x4 *>(part) = f32x4{sg[0], sg[1], sg[2], sg[3]};
        *reinterpret_cast<f32x4 *>(part + a.ldh) = f32x4{su[0], su[1], su[2], su[3]};
    }
}

// Products whose sums are the output: out = h Wd' + bd (kWAcross false), dx
// (kWAcross), the weights' gradients (both across), or a split's partial sums.
//
// 32768 x 1280, hidden 5120, with the join: out 341 + 14 us, 1.21 PFLOP/s; dx 664 + 14,
// 1.27; the weights' gradients 979 + 11, 1.30.  The matrix cores are busy 70 to 76%
// of their cycles at the clock that the card's power leaves; 1960 rows, in tiles
// of 128 x 128, which wait for what a CU takes in, 31 + 7, 58 + 7 and 84 us, 0.67 to
// 0.92 PFLOP/s.
template <int kTile, bool kXAcross, bool kWAcross>
__global__ __launch_bounds__(Tile<kTile>::kThreads) void mlp_product_kernel(MlpArgs a) {
    const Buffers<kTile> lds = tile_buffers<kTile>();
    typedef Tile<kTile> T;
    const Unit unit(a.units);
    const int n = kXAcross ? product_of(a, unit.tile) : 0;
    const Product &p = a.p[n];
    const Place at(p, unit.tile - p.first);
    const int64_t m0 = at.mt * kTile;
    const int n0 = at.nt * kTile;
    const bool part = unit.split >= 0;
    const int begin = part ? int(int64_t(p.stages) * unit.split / a.units.splits) : 0;
    const int end = part ? int(int64_t(p.stages) * (unit.split + 1) / a.units.splits) : p.stages;
    Sums<kTile> acc;
    multiply<kTile, kXAcross, kWAcross, kWAcross && !kXAcross ? kTwice : kOnce>(p, m0, n0, begin, end, lds, acc);
    const Turned<kTile> turned(lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave_row = (wave / T::kWavesN) * T::kWaveM, wave_col = (wave % T::kWavesN) * T::kWaveN;
    if (part) {
        // the whole of the part's tile, four channels a lane
        constexpr int kLanes = T::kWaveN / 4, kPass = 64 / kLanes;
        const int piece = (lane % kLanes) * 4;
        float *sums = a.part + int64_t(unit.slot) * (kTile * kTile) + wave_col + piece;
#pragma unroll
        for (int i = 0; i < T::kBlocksM; ++i) {
            turned.put(acc[i]);
#pragma unroll
            for (int t = 0; t < 32 / kPass; ++t) {
                const int r = t * kPass + lane / kLanes;
                float v[4];
                turned.get(r, piece, v);
                *reinterpret_cast<f32x4 *>(sums + (wave_row + i * 32 + r) * kTile) = f32x4{v[0], v[1], v[2], v[3]};
            }
        }
        return;
    }
    constexpr int kLanes = T::kWaveN / 8, kPass = 64 / kLanes;
    const int piece = (lane % kLanes) * 8, col = n0 + wave_col + piece, left = p.n - col;
    float bias[8];
    load_bias(a.bias0, col, p.n, bias);
#pragma unroll
    for (int i = 0; i < T::kBlocksM; ++i) {
        turned.put(acc[i]);
#pragma unroll
        for (int t = 0; t < 32 / kPass; ++t) {
            const int r = t * kPass + lane / kLanes;
            float v[8];
            turned.get(r, piece, v);
            const int64_t row = m0 + wave_row + i * 32 + r;
            if (row >= p.m || left <= 0) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += bias[j];
            store_bf16(a.out[n] + row * a.ldo[n] + col, v, left);
        }
    }
}

// The tiles in parts: their sums in the parts' order, + bias.  32 (8 of 128 x
// 128, 2 of 64 x 64) workgroups a tile, eight channels a thread.  The sums come
// from caches: 128 tiles of 256 x 256 in two parts 14 us, 20 of 128 x 128 in twelve 4,
// a launch's length.
template <int kTile>
__global__ __launch_bounds__(256) void mlp_join_kernel(MlpArgs a) {
    constexpr int kPieces = kTile / 8, kWgs = kTile * kPieces / 256;
    const int t = int(blockIdx.x) / kWgs, tile = a.units.full + t;
    const int n = product_of(a, tile);
    const Product &p = a.p[n];
    const Place at(p, tile - p.first);
    const int id = (int(blockIdx.x) - t * kWgs) * 256 + int(threadIdx.x), r = id / kPieces, c = id % kPieces * 8;
    const int64_t row = at.mt * kTile + r;
    const int col = at.nt * kTile + c, left = p.n - col;
    if (row >= p.m || left <= 0) return;
    const float *part = a.part + int64_t(t) * (kTile * kTile) + r * kTile + c;
    float v[8];
    auto load = [&](const float *q, float (&w)[8]) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(q), y = *reinterpret_cast<const f32x4 *>(q + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = x[j];
            w[4 + j] = y[j];
        }
    };
    load(part, v);
#pragma unroll 4
    for (int s = 1; s < a.units.splits; ++s) {
        float w[8];
        load(part + int64_t(s) * a.units.tail * (kTile * kTile), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += w[j];
    }
    float b[8];
    load_bias(a.bias0, col, p.n, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
    store_bf16(a.out[n] + row * a.ldo[n] + col, v, left);
}

// Rows of any width to rows of a multiple of kPad values, zeros behind: the
// products read 16 bytes at a time.  A wave takes a row; all of a call's
// operands are one launch.  4099 x 1283 and the weights of 3421 hidden values,
// forward: 16 to 19 us, 37 MB read and 38 written, 4.0 to 4.6 TB/s.
struct PadArgs {
    const uint16_t *from[5];
    uint16_t *to[5];
    int32_t width[5], padded[5];
    int64_t first[6];  // of each operand's rows
    int32_t count;
};
__global__ __launch_bounds__(256) void mlp_pad_kernel(PadArgs a) {
    int64_t row = row_group() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= a.first[a.count]) return;
    int n = 0;
    while (n + 1 < a.count && row >= a.first[n + 1]) ++n;
    row -= a.first[n];
    const uint16_t *from = a.from[n] + row * a.width[n];
    uint16_t *to = a.to[n] + row * a.padded[n];
    for (int col = int(threadIdx.x & 63) * 8; col < a.padded[n]; col += 64 * 8)
        *reinterpret_cast<u32x4 *>(to + col) = load_ragged(from + col, a.width[n] - col);
}

// Partial sums over every gridDim.y-th group of eight rows of 256 columns.
// 32768 x 1280: 19 us, 84 MB at 4.4 TB/s.
__global__ __launch_bounds__(256) void mlp_columns_kernel(const uint16_t *x, int64_t rows, int64_t stride, int32_t columns, float *part) {
    __shared__ float lds[8][256 + 8];
    const int lane = threadIdx.x % 32, first = threadIdx.x / 32;
    const int col = blockIdx.x * 256 + lane * 8;
    float v[8] = {};
    if (col < columns) {
#pragma unroll 4
        for (int64_t row = int64_t(blockIdx.y) * 8 + first; row < rows; row += int64_t(gridDim.y) * 8) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(x + row * stride + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] += __builtin_bit_cast(float, w[j] << 16);
                v[2 * j + 1] += __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[first][lane * 8 + j] = v[j];
    __syncthreads();
    float sum = lds[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += lds[i][threadIdx.x];
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < columns) part[int64_t(blockIdx.y) * columns + c] = sum;
}

// Few rows: the weights are read once, and that is what such a call waits
// for.  A workgroup takes up to 16 channels (with kGate of both projections);
// its waves share K, 32 values a product, and each has the operands of kDeep
// products on the way from memory at once; their sums meet in LDS.  Operands
// come straight from memory, at any address of the type where kRagged, so
// nothing is copied first.
//
// A CU takes in about 25 GB/s of them, whatever waves and loads it has (80
// workgroups of 16 channels: 4.2, 5.6, 9.0, 15.6 us for K 1280, 2560, 5120,
// 10240), so what counts is that all CUs have as many channels.  4 rows of 1280,
// hidden 5120: medians of 7.7 to 8.9 us for gate and up (shortest 7.5), 26 MB at 2.9 to
// 3.4 TB/s, 7.0 for down (6.1), 13 MB; a launch that does nothing is 2 to 3 of each.
//
// v_mfma_f32_16x16x32_bf16, weights first: lane l holds row l % 16 and k = 8 (l /
// 16) .. + 7 of an operand, and channels 4 (l / 16) + r of x's row l % 16 of the
// result; kRows blocks of 16 rows.
template <bool kGate, bool kRagged, int kRows, int kWaves, int kDeep>
__global__ __launch_bounds__(kWaves * 64) void mlp_few_kernel(MlpArgs a) {
    constexpr int kParts = kGate ? 2 : 1;
    __shared__ f32x4 sums[kWaves][kParts][kRows][64];
    const Product &p = a.p[0];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = int(blockIdx.x) * a.channels, l16 = lane & 15, at = 8 * (lane >> 4);
    const uint16_t *w[kParts], *x[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) x[j] = p.x[0].p + min(int64_t(16 * j + l16), p.m - 1) * p.x[0].stride + at;
#pragma unroll
    for (int i = 0; i < kParts; ++i) w[i] = p.w[i].p + int64_t(min(n0 + l16, p.n - 1)) * p.w[i].stride + at;
    // lanes of other channels and of no row ask for nothing
    const int k_w = l16 < a.channels ? p.k - at : 0;
    int k_x[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) k_x[j] = 16 * j + l16 < p.m ? p.k - at : 0;
    auto load = [&](const uint16_t *q, int k, int end) -> bf16x8 {
        if constexpr (kRagged) return __builtin_bit_cast(bf16x8, load_ragged(q + k, end - k));
        return k < end ? *reinterpret_cast<const bf16x8 *>(q + k) : bf16x8{};
    };
    f32x4 acc[kParts][kRows] = {};
    for (int k0 = 32 * wave; k0 < p.k; k0 += 32 * kWaves * kDeep) {
        bf16x8 fw[kDeep][kParts], fx[kDeep][kRows];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int k = k0 + 32 * kWaves * d;
#pragma unroll
            for (int i = 0; i < kParts; ++i) fw[d][i] = load(w[i], k, k_w);
#pragma unroll
            for (int j = 0; j < kRows; ++j) fx[d][j] = load(x[j], k, k_x[j]);
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int j = 0; j < kRows; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[d][i], fx[d][j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
        for (int j = 0; j < kRows; ++j) sums[wave][i][j][lane] = acc[i][j];
    __syncthreads();
    // one value a thread: a channel of a row
    static_assert(kWaves * 64 >= kRows * 256, "a thread for each value");
    const int c = threadIdx.x % 16, r = threadIdx.x / 16, col = n0 + c;
    if (r >= p.m || c >= a.channels || col >= a.all_channels) return;  // m <= 16 kRows
    float v[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        v[i] = 0.0f;
#pragma unroll
        for (int s = 0; s < kWaves; ++s) v[i] += sums[s][i][r / 16][(c / 4) * 16 + r % 16][c % 4];
    }
    if constexpr (kGate) {
        const bool in = col < p.n;
        const float g = in ? v[0] + (a.bias0 ? a.bias0[col] : 0.0f) : 0.0f, u = in ? v[1] + (a.bias1 ? a.bias1[col] : 0.0f) : 0.0f;
        const int64_t to = r * a.ldh + col;
        reinterpret_cast<__bf16 *>(a.hidden)[to] = __bf16(g * sigmoid(g) * u);
        if (a.gate_up) {
            a.gate_up[to] = g;
            a.gate_up[p.m * a.ldh + to] = u;
        }
    } else if (col < p.n) {
        reinterpret_cast<__bf16 *>(a.out[0])[r * a.ldo[0] + col] = __bf16(v[0] + (a.bias0 ? a.bias0[col] : 0.0f));
    }
}

int64_t pad_to(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// How a launch's products are cut into tiles and these into parts of K.
struct Cut {
    int tile;
    Units units;
    int64_t tiles;
    int64_t part_values() const { return units.splits > 1 ? int64_t(units.tail) * units.splits * tile * tile : 0; }
};
constexpr int kCus = 256;
constexpr int kMinStages = 6;  // of a part

// What a round of the card's tiles takes, in microseconds, fitted to 17 to 32768
// rows of widths 264 to 2048 and 520 to 5120 hidden values: a stage of the
// tiles that the CUs have at once (one of 256 x 256, two of 128 x 128, three of 64
// x 64), by how many there are; a tile's first loads and its store (more where g
// and u are read or written); and what parts cost, which are written in
// float32 and joined.
double stage_us(int tile, int64_t units) {
    if (tile == 256) return 1.5;
    if (tile == 128) return units <= kCus ? 0.6 : 1.07;
    return units <= kCus ? 0.25 : units <= 2 * kCus ? 0.42 : 0.58;
}
double ends_us(int tile, bool wide) { return tile == 256 ? (wide ? 20.0 : 11.0) : tile == 128 ? (wide ? 6.0 : 4.0) : (wide ? 4.0 : 3.0); }
double parts_us(int tile) { return tile == 256 ? 19.0 : 6.0; }

// Tiles of one size.  What is left over after whole rounds would keep some CUs
// busy for all of K and leave the others idle; its K is cut into parts where
// that is quicker.
Cut cut_tiles(int tile, int64_t tiles, int64_t stages, bool splittable, bool wide, double *cost) {
    Cut c{tile, {int32_t(tiles), 0, 1}, tiles};
    const int64_t slots = int64_t(kCus) * (tile == 256 ? 1 : tile == 128 ? 2 : 3), full = tiles / slots * slots, tail = tiles - full;
    const double ends = ends_us(tile, wide);
    double rest = tail ? double(stages) * stage_us(tile, tail) + ends : 0.0;
    if (splittable && tail) {
        const int64_t most = stages / kMinStages < slots / tail ? stages / kMinStages : slots / tail;
        for (int64_t splits = 2; splits <= most; ++splits) {
            const double parts = double(ceil_div(stages, splits)) * stage_us(tile, tail * splits) + ends + parts_us(tile);
            if (parts < rest) {
                c.units = {int32_t(full), int32_t(tail), int32_t(splits)};
                rest = parts;
            }
        }
    }
    *cost = double(full / slots) * (double(stages) * stage_us(tile, slots) + ends) + rest;
    return c;
}

// One or more products [m][n] of as many stages each.
struct Extent {
    int64_t m, n;
};
int64_t tiles_of(const Extent *e, int count, int tile, int columns) {
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i) tiles += ceil_div(e[i].m, tile) * ceil_div(e[i].n, columns);
    return tiles;
}
// The quickest of the three sizes by that.  us of the forward and the backward
// pass on 64, 128 and 256, width 1280, hidden 5120: 64 rows 19, 27, 46 and 45, 48,
// 76; 512 rows 42, 42, 51 and 90, 76, 110; 1960 rows 132, 93, 102 and 275, 191, 195;
// 4096 rows 250, 167, 166 and 543, 371, 346; width 640, hidden 1000: 1024 rows 12,
// 20, 40 and 33, 43, 75; 4096 rows 33, 29, 44 and 70, 70, 100.
// gate: both projections of a channel lie in one tile, which then has half as
// many.
Cut cut(const Extent *e, int count, int64_t stages, bool splittable, bool wide, bool gate) {
    Cut best{};
    double least = 0.0;
    for (int tile = 256; tile >= 64; tile /= 2) {
        const int64_t tiles = tiles_of(e, count, tile, gate ? tile / 2 : tile);
        if (tile < 256 && tiles > kMaxTiles) break;  // a launch of fewer, larger ones
        double cost;
        const Cut c = cut_tiles(tile, tiles, stages, splittable, wide, &cost);
        if (tile == 256 || cost < least) {
            best = c;
            least = cost;
        }
    }
    return best;
}
Cut cut(int64_t m, int64_t n, int64_t stages, bool splittable, bool wide, bool gate = false) {
    const Extent e{m, n};
    return cut(&e, 1, stages, splittable, wide, gate);
}

struct Sizes {
    int64_t rows, d, h;
    bool pad_d, pad_h;   // rows of d (h) values are copied to padded ones
    int64_t dp, hp;      // strides of such copies; hp of hidden values too
    Sizes(int64_t rows, int64_t d, int64_t h)
        : rows(rows), d(d), h(h), pad_d(d % 8 != 0), pad_h(h % 8 != 0), dp(pad_to(d, kPad)), hp(pad_to(h, kPad)) {}
    // The forward pass's kernels for few rows.  us of them and of 64 x 64 tiles:
    // width 1280, hidden 5120: 1 row 12.4, 17.6; 16 rows 17.4, 17.8; 32 rows 24.6,
    // 18.1, each CU then taking in all of x twice; width 2048, hidden 2048: 17 rows
    // 13.0, 14.8, 32 rows 15.7, 15.3; width 264, hidden 520: 32 rows 7.2, 8.8; width 64,
    // hidden 6000: 4 rows 9.3, 10.8, 16 rows 12.5, 10.6.  So the rule, of rows and hidden
    // values alone, gives up to 2 us away where the second product has few channels
    // (64: as many workgroups, each with all of K) and rows pass a handful, and half
    // a microsecond at its upper corner.
    bool few() const { return rows <= 16 || (rows <= 32 && hp <= 8 * kCus); }
    int64_t ld() const { return pad_d ? dp : d; }   // of x, dout, the gate's and the up projection's weights
    int64_t lh() const { return pad_h ? hp : h; }   // of the down projection's weight
    Cut gate(bool saved) const { return few() ? Cut{} : cut(rows, hp, ceil_div(d, kStageK), false, saved, true); }  // the padding is written too
    Cut down() const { return few() ? Cut{} : cut(rows, d, ceil_div(h, kStageK), true, false); }
    Cut dhidden() const { return cut(rows, h, ceil_div(d, kStageK), false, true); }
    Cut dx() const { return cut(rows, d, 2 * ceil_div(h, kStageK), true, false); }
    // of the weights' gradients that are made
    Cut dweights(bool gate, bool up, bool down) const {
        Extent e[3];
        int n = 0;
        if (gate) e[n++] = {h, d};
        if (up) e[n++] = {h, d};
        if (down) e[n++] = {d, h};
        return cut(e, n, ceil_div(rows, kStageK), true, false, false);
    }
};

// Takes aligned parts of a workspace, or measures them.
struct Carver {
    uint8_t *base;
    size_t used = 0;
    template <typename T>
    T *take(int64_t values) {
        T *p = reinterpret_cast<T *>(base + used);
        used += align256(size_t(values) * sizeof(T));
        return p;
    }
};

struct ForwardSpace {
    uint16_t *hidden, *x, *wg, *wu, *wd;
    float *part;
    size_t bytes;
    ForwardSpace(const Sizes &s, const Cut &down, void *base) {
        Carver c{static_cast<uint8_t *>(base)};
        const bool copy_d = s.pad_d && !s.few(), copy_h = s.pad_h && !s.few();
        hidden = c.take<uint16_t>(s.rows * s.hp);
        x = c.take<uint16_t>(copy_d ? s.rows * s.dp : 0);
        wg = c.take<uint16_t>(copy_d ? s.h * s.dp : 0);
        wu = c.take<uint16_t>(copy_d ? s.h * s.dp : 0);
        wd = c.take<uint16_t>(copy_h ? s.d * s.hp : 0);
        part = c.take<float>(s.few() ? 0 : down.part_values());
        bytes = c.used;
    }
};

constexpr int kColumnGroups = 128;  // workgroups along the rows of mlp_columns_kernel
struct BackwardSpace {
    uint16_t *dgate, *dup, *x, *dout, *wg, *wu, *wd;
    float *part, *sums, *columns;
    size_t bytes;
    BackwardSpace(const Sizes &s, const Cut &dhidden, const Cut &dx, void *base) {
        Carver c{static_cast<uint8_t *>(base)};
        dgate = c.take<uint16_t>(s.rows * s.hp);
        dup = c.take<uint16_t>(s.rows * s.hp);
        x = c.take<uint16_t>(s.pad_d ? s.rows * s.dp : 0);
        dout = c.take<uint16_t>(s.pad_d ? s.rows * s.dp : 0);
        wg = c.take<uint16_t>(s.pad_d ? s.h * s.dp : 0);
        wu = c.take<uint16_t>(s.pad_d ? s.h * s.dp : 0);
        wd = c.take<uint16_t>(s.pad_h ? s.d * s.hp : 0);
        int64_t values = dx.part_values();
        // whichever of the weights' gradients are made (gate's and up's alone are
        // alike); few rows are not cut into parts
        for (int made = 1; made < 8 && s.rows >= 2 * kMinStages * kStageK - kStageK; ++made) {
            const int64_t w = made == 2 || made == 6 ? 0 : s.dweights(made & 1, made & 2, made & 4).part_values();
            if (w > values) values = w;
        }
        part = c.take<float>(values);
        sums = c.take<float>(2 * ceil_div(s.rows, dhidden.tile) * 2 * s.hp);
        columns = c.take<float>(kColumnGroups * s.d);
        bytes = c.used;
    }
};

Matrix matrix(const void *p, int64_t stride) { return Matrix{static_cast<const uint16_t *>(p), stride}; }

Product product(const Matrix &x, const Matrix &w, int64_t m, int64_t n, int64_t k, int tile, int columns) {
    Product p;
    std::memset(&p, 0, sizeof(p));
    p.x[0] = p.x[1] = x;
    p.w[0] = p.w[1] = w;
    p.m = m;
    p.n = int32_t(n);
    p.k = int32_t(k);
    p.stages = int32_t(ceil_div(k, kStageK));
    p.m_tiles = int32_t(ceil_div(m, tile));
    p.n_tiles = int32_t(ceil_div(n, columns));
    return p;
}

// Operands to copy, and their launch; the launches made.
struct Padding {
    PadArgs a;
    Padding() { std::memset(&a, 0, sizeof(a)); }
    // `p` becomes the copy.
    void add(const void *&p, int64_t rows, int64_t width, uint16_t *to, int64_t padded) {
        const int n = a.count++;
        a.from[n] = static_cast<const uint16_t *>(p);
        a.to[n] = to;
        a.width[n] = int32_t(width);
        a.padded[n] = int32_t(padded);
        a.first[n + 1] = a.first[n] + rows;
        p = to;
    }
    int launch(hipStream_t s) const {
        if (!a.count) return 0;
        hipLaunchKernelGGL(mlp_pad_kernel, row_grid(ceil_div(a.first[a.count], 4)), dim3(256, 1, 1), 0, s, a);
        return 1;
    }
};

template <int kTile>
void launch_gate(const MlpArgs &a, const dim3 &grid, hipStream_t s) {
    const dim3 block(Tile<kTile>::kThreads, 1, 1);
    if (a.gate_up)
        hipLaunchKernelGGL((mlp_gate_kernel<kTile, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((mlp_gate_kernel<kTile, false>), grid, block, 0, s, a);
}

// A launch of mlp_product_kernel, and its join; the launches made.
template <bool kXAcross, bool kWAcross>
int launch_products(MlpArgs &a, const Cut &c, float *part, hipStream_t s) {
    a.units = c.units;
    a.part = part;
    const dim3 grid(unsigned(c.units.count()), 1, 1);
    const bool joined = c.units.splits > 1;
    if (c.tile == 256) {
        hipLaunchKernelGGL((mlp_product_kernel<256, kXAcross, kWAcross>), grid, dim3(Tile<256>::kThreads, 1, 1), 0, s, a);
        if (joined) hipLaunchKernelGGL(mlp_join_kernel<256>, dim3(unsigned(c.units.tail) * 32, 1, 1), dim3(256, 1, 1), 0, s, a);
    } else if (c.tile == 128) {
        hipLaunchKernelGGL((mlp_product_kernel<128, kXAcross, kWAcross>), grid, dim3(Tile<128>::kThreads, 1, 1), 0, s, a);
        if (joined) hipLaunchKernelGGL(mlp_join_kernel<128>, dim3(unsigned(c.units.tail) * 8, 1, 1), dim3(256, 1, 1), 0, s, a);
    } else {
        hipLaunchKernelGGL((mlp_product_kernel<64, kXAcross, kWAcross>), grid, dim3(Tile<64>::kThreads, 1, 1), 0, s, a);
        if (joined) hipLaunchKernelGGL(mlp_join_kernel<64>, dim3(unsigned(c.units.tail) * 2, 1, 1), dim3(256, 1, 1), 0, s, a);
    }
    return joined ? 2 : 1;
}

// As many workgroups as CUs, or a multiple of that, of as many channels each.
template <bool kGate, int kRows, int kWaves, int kDeep>
void launch_few_kernel(MlpArgs &a, int64_t channels, bool ragged, hipStream_t s) {
    const int64_t groups = kCus * ceil_div(channels, kCus * 16);
    a.channels = int32_t(ceil_div(channels, groups));
    a.all_channels = int32_t(channels);
    const dim3 grid(unsigned(ceil_div(channels, a.channels)), 1, 1), block(kWaves * 64, 1, 1);
    if (ragged)
        hipLaunchKernelGGL((mlp_few_kernel<kGate, true, kRows, kWaves, kDeep>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((mlp_few_kernel<kGate, false, kRows, kWaves, kDeep>), grid, block, 0, s, a);
}

// The forward pass of few rows, operands as they are.
void launch_few(const Sizes &z, const mimo_mlp &args, uint16_t *hidden, uint16_t *out, hipStream_t s) {
    MlpArgs a;
    std::memset(&a, 0, sizeof(a));
    a.p[0] = product(matrix(args.x, z.d), matrix(args.w_gate, z.d), z.rows, z.h, z.d, 128, 128);
    a.p[0].w[1] = matrix(args.w_up, z.d);
    a.bias0 = args.b_gate;
    a.bias1 = args.b_up;
    a.gate_up = args.gate_up;
    a.hidden = hidden;
    a.ldh = z.hp;
    if (z.rows <= 16)
        launch_few_kernel<true, 1, 8, 5>(a, z.hp, z.pad_d, s);
    else
        launch_few_kernel<true, 2, 8, 5>(a, z.hp, z.pad_d, s);
    a.p[0] = product(matrix(hidden, z.hp), matrix(args.w_down, z.h), z.rows, z.d, z.h, 128, 128);
    a.bias0 = args.b_down;
    a.out[0] = out;
    a.ldo[0] = z.d;
    if (z.rows <= 16)
        launch_few_kernel<false, 1, 16, 10>(a, z.d, z.pad_h, s);
    else
        launch_few_kernel<false, 2, 16, 5>(a, z.d, z.pad_h, s);
}

int check_mlp(const mimo_mlp *p, const char *who) {
    const std::string w(who);
    if (!p) return set_error(MIMO_E_INVALID, w + ": null arguments");
    if (p->rows < 0 || p->width < 1 || p->hidden_width < 1)
        return set_error(MIMO_E_INVALID, w + ": rows must be >= 0, width and hidden_width >= 1");
    if (p->rows > 0x7FFFFFFFll || p->width > kMaxWidth || p->hidden_width > kMaxWidth)
        return set_error(MIMO_E_TOO_LARGE, w + ": more than 2^31 - 1 rows, or a width above 65536");
    // of 256 x 256; cut() takes no smaller ones where there would be more
    const int64_t m = ceil_div(p->rows, 256), n = ceil_div(p->hidden_width, 128) + ceil_div(p->width, 256);
    if (m * n > kMaxTiles) return set_error(MIMO_E_TOO_LARGE, w + ": more than 2^23 - 1 tiles");
    return MIMO_OK;
}

bool is_aligned(const void *p) { return p && check_ptr_align(p, 16); }

}  // namespace
}  // namespace mimo

using namespace mimo;

extern "C" {

size_t mimo_gated_mlp_workspace_bytes(int64_t rows, int32_t width, int32_t hidden_width) {
    const mimo_mlp p{rows, width, hidden_width, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    if (check_mlp(&p, "gated_mlp") != MIMO_OK) {
        clear_error();
        return 0;
    }
    const Sizes s(rows, width, hidden_width);
    return ForwardSpace(s, s.down(), nullptr).bytes;
}

int mimo_gated_mlp(const mimo_mlp *args, void *out, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    const char *who = "gated_mlp";
    int st = check_mlp(args, who);
    if (st != MIMO_OK) return st;
    if (args->rows == 0) return MIMO_OK;
    if (!is_aligned(args->x) || !is_aligned(args->w_gate) || !is_aligned(args->w_up) || !is_aligned(args->w_down) || !is_aligned(out))
        return set_error(MIMO_E_INVALID, "gated_mlp: x, the weights and out must be non-null and 16-byte aligned");
    if (!check_ptr_align(args->b_gate, 4) || !check_ptr_align(args->b_up, 4) || !check_ptr_align(args->b_down, 4))
        return set_error(MIMO_E_INVALID, "gated_mlp: biases must be 4-byte aligned");
    if ((args->gate_up != nullptr) != (args->hidden != nullptr) || !check_ptr_align(args->gate_up, 16) || !check_ptr_align(args->hidden, 16))
        return set_error(MIMO_E_INVALID, "gated_mlp: gate_up and hidden are given together, 16-byte aligned, or neither is");
    const void *const inputs[] = {args->x, args->w_gate, args->w_up, args->w_down, args->b_gate, args->b_up, args->b_down};
    const void *const written[] = {out, args->gate_up, args->hidden};
    for (const void *w : written)
        for (const void *i : inputs)
            if (w && w == i) return set_error(MIMO_E_INVALID, "gated_mlp: out, gate_up and hidden must not be inputs");
    if (out == args->gate_up || out == args->hidden || (args->hidden && args->hidden == args->gate_up))
        return set_error(MIMO_E_INVALID, "gated_mlp: out, gate_up and hidden must not be one array");
    if (!is_aligned(workspace)) return set_error(MIMO_E_INVALID, "gated_mlp: workspace must be non-null and 16-byte aligned");
    const Sizes z(args->rows, args->width, args->hidden_width);
    const Cut gate = z.gate(args->gate_up != nullptr), down = z.down();
    const ForwardSpace space(z, down, workspace);
    if (workspace_bytes < space.bytes)
        return set_error(MIMO_E_CAPACITY, "gated_mlp: workspace smaller than mimo_gated_mlp_workspace_bytes");
    const int64_t x_bytes = z.rows * z.d * 2, w_bytes = z.h * z.d * 2, h_bytes = z.rows * z.hp * 2;
    const Span made_out{out, x_bytes}, made_gu{args->gate_up, 4 * h_bytes}, made_h{args->hidden, h_bytes}, in_x{args->x, x_bytes},
        in_wg{args->w_gate, w_bytes}, in_wu{args->w_up, w_bytes}, in_wd{args->w_down, w_bytes}, in_bg{args->b_gate, z.h * 4},
        in_bu{args->b_up, z.h * 4}, in_bd{args->b_down, z.d * 4};
    if (overlap_in_part({made_out, made_gu, made_h}, {in_x, in_wg, in_wu, in_wd, in_bg, in_bu, in_bd}))
        return set_error(MIMO_E_INVALID, "gated_mlp: out, gate_up and hidden must not overlap inputs or each other in part");
    if (overlaps_any({workspace, int64_t(space.bytes)}, {made_out, made_gu, made_h, in_x, in_wg, in_wu, in_wd, in_bg, in_bu, in_bd}))
        return set_error(MIMO_E_INVALID, "gated_mlp: workspace must not overlap another argument");
    hipStream_t s = static_cast<hipStream_t>(stream);
    int launches = 0;
    const void *x = args->x, *wg = args->w_gate, *wu = args->w_up, *wd = args->w_down;
    uint16_t *hidden = args->hidden ? static_cast<uint16_t *>(args->hidden) : space.hidden;
    const hipError_t e = timed_launch(s, [&] {
        if (z.few()) {
            launches = 2;
            launch_few(z, *args, hidden, static_cast<uint16_t *>(out), s);
            return;
        }
        Padding padding;
        if (z.pad_d) {
            padding.add(x, z.rows, z.d, space.x, z.dp);
            padding.add(wg, z.h, z.d, space.wg, z.dp);
            padding.add(wu, z.h, z.d, space.wu, z.dp);
        }
        if (z.pad_h) padding.add(wd, z.d, z.h, space.wd, z.hp);
        launches += padding.launch(s);
        MlpArgs a;
        std::memset(&a, 0, sizeof(a));
        a.p[0] = product(matrix(x, z.ld()), matrix(wg, z.ld()), z.rows, z.h, z.d, gate.tile, gate.tile / 2);
        a.p[0].w[1] = matrix(wu, z.ld());
        a.p[0].n_tiles = int32_t(ceil_div(z.hp, gate.tile / 2));
        a.products = 1;
        a.bias0 = args->b_gate;
        a.bias1 = args->b_up;
        a.gate_up = args->gate_up;
        a.hidden = hidden;
        a.ldh = z.hp;
        const dim3 grid(unsigned(gate.tiles), 1, 1);
        if (gate.tile == 256)
            launch_gate<256>(a, grid, s);
        else if (gate.tile == 128)
            launch_gate<128>(a, grid, s);
        else
            launch_gate<64>(a, grid, s);
        a.p[0] = product(matrix(hidden, z.hp), matrix(wd, z.lh()), z.rows, z.d, z.h, down.tile, down.tile);
        a.out[0] = static_cast<uint16_t *>(out);
        a.ldo[0] = z.d;
        a.bias0 = args->b_down;
        launches += 1 + launch_products<false, false>(a, down, space.part, s);
    });
    if (e != hipSuccess) return hip_error(e, "gated_mlp: kernel launch");
    g_dispatches.fetch_add(launches);
    return MIMO_OK;
}

size_t mimo_gated_mlp_backward_workspace_bytes(int64_t rows, int32_t width, int32_t hidden_width) {
    const mimo_mlp p{rows, width, hidden_width, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    if (check_mlp(&p, "gated_mlp_backward") != MIMO_OK) {
        clear_error();
        return 0;
    }
    const Sizes s(rows, width, hidden_width);
    return BackwardSpace(s, s.dhidden(), s.dx(), nullptr).bytes;
}

int mimo_gated_mlp_backward(const mimo_mlp *args, const mimo_mlp_grads *grads, void *workspace, size_t workspace_bytes,
                            void *stream) {
    clear_error();
    const char *who = "gated_mlp_backward";
    int st = check_mlp(args, who);
    if (st != MIMO_OK) return st;
    if (!grads) return set_error(MIMO_E_INVALID, "gated_mlp_backward: null gradients");
    void *const made[] = {grads->dx, grads->dw_gate, grads->dw_up, grads->dw_down, grads->db_gate, grads->db_up, grads->db_down};
    const bool any_weight = grads->dw_gate || grads->dw_up || grads->dw_down;
    const bool any_bias = grads->db_gate || grads->db_up || grads->db_down;
    if (!check_ptr_align(grads->dx, 16) || !check_ptr_align(grads->dw_gate, 16) || !check_ptr_align(grads->dw_up, 16) ||
        !check_ptr_align(grads->dw_down, 16) || !check_ptr_align(grads->db_gate, 4) || !check_ptr_align(grads->db_up, 4) ||
        !check_ptr_align(grads->db_down, 4))
        return set_error(MIMO_E_INVALID, "gated_mlp_backward: dx and the weights' gradients must be 16-byte aligned, the biases' 4-byte");
    if (args->rows == 0 && !any_weight && !any_bias) return MIMO_OK;
    if (args->rows > 0) {
        if (!is_aligned(args->x) || !is_aligned(args->w_gate) || !is_aligned(args->w_up) || !is_aligned(args->w_down) ||
            !is_aligned(grads->dout) || !is_aligned(args->gate_up) || !is_aligned(args->hidden))
            return set_error(MIMO_E_INVALID, "gated_mlp_backward: x, the weights, dout, gate_up and hidden must be non-null and 16-byte aligned");
        const void *const inputs[] = {args->x, args->w_gate, args->w_up, args->w_down, grads->dout, args->gate_up, args->hidden};
        for (const void *m : made)
            for (const void *i : inputs)
                if (m && m == i) return set_error(MIMO_E_INVALID, "gated_mlp_backward: a gradient must not be an input");
    }
    for (int i = 0; i < 7; ++i)
        for (int j = 0; j < i; ++j)
            if (made[i] && made[i] == made[j]) return set_error(MIMO_E_INVALID, "gated_mlp_backward: gradients must not be one array");
    if (!is_aligned(workspace)) return set_error(MIMO_E_INVALID, "gated_mlp_backward: workspace must be non-null and 16-byte aligned");
    const Sizes z(args->rows, args->width, args->hidden_width);
    const Cut dhidden = z.dhidden(), dx = z.dx();
    const BackwardSpace space(z, dhidden, dx, workspace);
    if (workspace_bytes < space.bytes)
        return set_error(MIMO_E_CAPACITY, "gated_mlp_backward: workspace smaller than mimo_gated_mlp_backward_workspace_bytes");
    const int64_t x_bytes = z.rows * z.d * 2, w_bytes = z.h * z.d * 2, h_bytes = z.rows * z.hp * 2;
    const Span dx_made{grads->dx, x_bytes}, dwg_made{grads->dw_gate, w_bytes}, dwu_made{grads->dw_up, w_bytes}, dwd_made{grads->dw_down, w_bytes},
        dbg_made{grads->db_gate, z.h * 4}, dbu_made{grads->db_up, z.h * 4}, dbd_made{grads->db_down, z.d * 4};
    const int64_t some = z.rows > 0;  // without rows nothing is read
    const Span in_x{args->x, some * x_bytes}, in_wg{args->w_gate, some * w_bytes}, in_wu{args->w_up, some * w_bytes}, in_wd{args->w_down, some * w_bytes},
        in_g{grads->dout, some * x_bytes}, in_gu{args->gate_up, some * 4 * h_bytes}, in_h{args->hidden, some * h_bytes};
    if (overlap_in_part({dx_made, dwg_made, dwu_made, dwd_made, dbg_made, dbu_made, dbd_made}, {in_x, in_wg, in_wu, in_wd, in_g, in_gu, in_h}))
        return set_error(MIMO_E_INVALID, "gated_mlp_backward: a gradient must not overlap an input or another one in part");
    if (overlaps_any({workspace, int64_t(space.bytes)}, {dx_made, dwg_made, dwu_made, dwd_made, dbg_made, dbu_made, dbd_made, in_x, in_wg, in_wu, in_wd,
                                                         in_g, in_gu, in_h}))
        return set_error(MIMO_E_INVALID, "gated_mlp_backward: workspace must not overlap another argument");
    hipStream_t s = static_cast<hipStream_t>(stream);
    int launches = 0;
    const void *x = args->x, *dout = grads->dout, *wg = args->w_gate, *wu = args->w_up, *wd = args->w_down;
    const hipError_t e = timed_launch(s, [&] {
        Padding padding;
        if (z.rows > 0 && z.pad_d) {
            padding.add(x, z.rows, z.d, space.x, z.dp);
            padding.add(dout, z.rows, z.d, space.dout, z.dp);
            padding.add(wg, z.h, z.d, space.wg, z.dp);
            padding.add(wu, z.h, z.d, space.wu, z.dp);
        }
        if (z.rows > 0 && z.pad_h) padding.add(wd, z.d, z.h, space.wd, z.hp);
        launches += padding.launch(s);
        MlpArgs a;
        std::memset(&a, 0, sizeof(a));
        a.gate_up = args->gate_up;
        a.ldh = z.hp;
        if (z.rows > 0) {
            a.p[0] = product(matrix(dout, z.ld()), matrix(wd, z.lh()), z.rows, z.h, z.d, dhidden.tile, dhidden.tile);
            a.products = 1;
            a.dgate = space.dgate;
            a.dup = space.dup;
            a.part = grads->db_gate || grads->db_up ? space.sums : nullptr;
            const dim3 grid(unsigned(dhidden.tiles), 1, 1);
            if (dhidden.tile == 256)
                hipLaunchKernelGGL(mlp_dhidden_kernel<256>, grid, dim3(Tile<256>::kThreads, 1, 1), 0, s, a);
            else if (dhidden.tile == 128)
                hipLaunchKernelGGL(mlp_dhidden_kernel<128>, grid, dim3(Tile<128>::kThreads, 1, 1), 0, s, a);
            else
                hipLaunchKernelGGL(mlp_dhidden_kernel<64>, grid, dim3(Tile<64>::kThreads, 1, 1), 0, s, a);
            ++launches;
        }
        const int32_t halves = int32_t(2 * ceil_div(z.rows, dhidden.tile));
        ColumnSums sums;
        if (grads->db_gate) sums.add(space.sums, halves, 2 * z.hp, z.h, grads->db_gate);
        if (grads->db_up) sums.add(space.sums + z.hp, halves, 2 * z.hp, z.h, grads->db_up);
        if (grads->db_down) {
            const int64_t groups = ceil_div(z.rows, 8) < kColumnGroups ? ceil_div(z.rows, 8) : kColumnGroups;
            if (groups) {
                hipLaunchKernelGGL(mlp_columns_kernel, dim3(unsigned(ceil_div(z.d, 256)), unsigned(groups), 1), dim3(256, 1, 1), 0, s,
                                   static_cast<const uint16_t *>(dout), z.rows, z.ld(), int32_t(z.d), space.columns);
                ++launches;
            }
            sums.add(space.columns, int32_t(groups), z.d, z.d, grads->db_down);
        }
        launches += launch_column_sums(sums, s);
        if (z.rows > 0 && grads->dx) {
            a.p[0] = product(matrix(space.dgate, z.hp), matrix(wg, z.ld()), z.rows, z.d, z.h, dx.tile, dx.tile);
            a.p[0].x[1] = matrix(space.dup, z.hp);
            a.p[0].w[1] = matrix(wu, z.ld());
            a.p[0].stages *= 2;
            a.products = 1;
            a.out[0] = static_cast<uint16_t *>(grads->dx);
            a.ldo[0] = z.d;
            launches += launch_products<false, true>(a, dx, space.part, s);
        }
        if (any_weight) {
            const Cut c = z.dweights(grads->dw_gate, grads->dw_up, grads->dw_down);
            int n = 0, tiles = 0;
            auto add = [&](void *out, const Matrix &left, const Matrix &right, int64_t m, int64_t columns) {
                if (!out) return;
                a.p[n] = product(left, right, m, columns, z.rows, c.tile, c.tile);
                a.p[n].first = tiles;
                a.out[n] = static_cast<uint16_t *>(out);
                a.ldo[n] = columns;
                tiles += a.p[n].m_tiles * a.p[n].n_tiles;
                ++n;
            };
            add(grads->dw_gate, matrix(space.dgate, z.hp), matrix(x, z.ld()), z.h, z.d);
            add(grads->dw_up, matrix(space.dup, z.hp), matrix(x, z.ld()), z.h, z.d);
            add(grads->dw_down, matrix(dout, z.ld()), matrix(args->hidden, z.hp), z.d, z.h);
            a.products = n;
            launches += launch_products<true, true>(a, c, space.part, s);
        }
    });
    if (e != hipSuccess) return hip_error(e, "gated_mlp_backward: kernel launch");
    g_dispatches.fetch_add(launches);
    return MIMO_OK;
}

}  // extern "C"
