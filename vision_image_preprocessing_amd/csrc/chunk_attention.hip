// chunk_attention.hip -- attention over the plan's chunks (one chunk per
// temporal slice of an item), forward and backward, on the bf16 matrix cores
// of AMD Instinct MI355X (gfx950, CDNA4).
//
// What is computed (NeMo Automodel "mimo_v2_flash.vision", MiMoVisionAttention;
// docs.rs "cortiq_engine::mimo_vision" module conventions: frames are
// independent chunks, grouped heads, band |i - j| <= window over chunk-local
// indices, sinks added to key 0's logit).  For row i of a chunk, query head h
// and its key head g = h / (q_heads / kv_heads):
//   s_ij  = scale * q_i . k_j + [j = 0] sink_h      for |i - j| <= window
//   lse_i = log sum_j exp s_ij,  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
// and with delta_i = do_i . o_i and ds_ij = p_ij (do_i . v_j - delta_i):
//   dq_i = scale sum_j ds_ij k_j      dk_j = scale sum_{h of g, i} ds_ij q_i
//   dv_j = sum_{h of g, i} p_ij do_i  dsink_h = sum_i ds_i0
// A row that sees nothing (sink_h = -inf and key 0 alone in its band) has
// o = 0, lse = -inf and no gradient.
//
// Matrix products.  All use v_mfma_f32_32x32x16_bf16.  Its result holds one
// column per lane (lane % 32) and rows 8 (r / 4) + 4 (lane / 32) + r % 4 in
// value r.  Products are arranged so that the softmax axis that is summed
// next is the row axis of that result: a lane then owns one query row
// (forward, dq) or one key (dk, dv), and the probabilities it holds are, in
// place and only packed to bf16, the second operand of the next product,
// whose reduction runs over them in the order 8 (e / 4) + 4 (lane / 32) +
// e % 4 of each 16.  The first operand takes the same order from LDS with
// ds_read_b64_tr_b16, which hands a lane four rows of one column.
//
// Roundings: logits, softmax statistics, delta and every accumulator are
// float32; p and ds are rounded to bf16 (nearest even) as matrix-core
// operands, as q, k, v and do come in; outputs are rounded once.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <string>

#include "device_util.h"
#include "internal.h"
#include "runtime.h"

namespace mimo {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4_ptr;

constexpr int kThreads = 256;
constexpr int kWaveRows = 32;                 // rows (or keys) one wave owns
constexpr int kTileRows = 4 * kWaveRows;      // of one workgroup
constexpr int kStep = 64;                     // keys (or rows) staged in LDS at a time
constexpr int kPanel = 64;                    // head columns of one LDS panel: rows of 128 bytes
constexpr int kWord3 = 0x00020000;            // raw buffer resource word 3
constexpr uint32_t kOutside = 0x7FFFFFF8u;    // a byte offset past every resource: reads zeros
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
// The running maximum is raised only when a row outgrows it by this many
// powers of two: probabilities stay below 2^8 meanwhile, which float32 sums
// and bf16 operands hold at full relative precision.
constexpr float kRaise = 8.0f;

// One [rows][heads][head_dim] bf16 tensor; strides in values.
struct Heads {
    uint16_t *p;
    int64_t row, head;
};

struct AttentionArgs {
    Heads q, k, v, out, dout, dq, dk, dv;
    const int32_t *cu;   // [chunks + 1]
    const float *sink;   // [q_heads] or null
    float *lse;          // [q_heads][rows], or null (forward)
    float *delta;        // [q_heads][rows] (backward)
    float *dsink_part;   // [q_heads][tiles], or null
    int64_t rows;
    int32_t q_heads, kv_heads, head_dim, chunks;
    int32_t window;      // < 0: none
    int32_t tiles;       // rows / kTileRows + chunks
    float scale;
};

// A workgroup's tile: rows [first, first + kTileRows) of the chunk of len
// rows that starts at row begin; len = 0 for a tile that holds nothing.
struct Tile {
    int64_t begin;
    int32_t len, first;
};

// Tile t of the batch: chunk c's tiles are numbered from cu[c] / kTileRows + c,
// which leaves each chunk as many numbers as it needs or one more, so that
// the grid is known from the row and chunk counts alone.  A boundary outside
// [0, rows] or a descending pair gives an empty tile: nothing is read or
// written through it.
__device__ __forceinline__ Tile find_tile(const int32_t *cu, int chunks, int64_t rows, int64_t t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = chunks;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int idx = lo + lane * step;
        const bool le = idx < hi && int64_t(cu[idx]) / kTileRows + idx <= t;
        const int k = max(__popcll(__ballot(le)) - 1, 0);
        lo += k * step;
        hi = min(lo + step, hi);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int64_t b = cu[lo], e = cu[lo + 1];
    Tile r{0, 0, 0};
    const int64_t first = (t - (b / kTileRows + lo)) * kTileRows;
    if (b < 0 || e > rows || first < 0 || first >= e - b) return r;
    r.begin = b;
    r.len = __builtin_amdgcn_readfirstlane(int(e - b));
    r.first = __builtin_amdgcn_readfirstlane(int(first));
    return r;
}

// LDS position (in values) of 16-byte chunk v of panel row r: chunks are
// XOR-swizzled by the row, so that the same chunk of eight rows (operand
// reads) and half rows of eight rows (transposed reads) cover every bank.
__device__ __forceinline__ int lds_at(int r, int v) { return r * kPanel + ((v ^ ((r ^ (r >> 3)) & 7)) << 3); }

// A resource over one head's rows from `row` on, `left` of them: reads past
// them (rows behind the chunk, columns behind head_dim) give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t head_rsrc(const Heads &t, int64_t row, int head, int left, int head_dim) {
    const int64_t bytes = (int64_t(left - 1) * t.row + head_dim) * 2;
    return __builtin_amdgcn_make_buffer_rsrc(t.p + row * t.row + head * t.head, 0, left < 1 ? 0 : int(min(bytes, int64_t(0x7FFFFFF0))),
                                             kWord3);
}

__device__ __forceinline__ uint32_t head_offset(const Heads &t, int r, int col, int head_dim) {
    return col < head_dim ? uint32_t(r * int(t.row) + col) * 2 : kOutside;
}

// The operand rows of a wave straight from memory: lane l holds row l % 32,
// columns 16 s + 8 (l / 32) .. + 7 of step s.
template <int kD>
__device__ __forceinline__ void load_operand(const Heads &t, int64_t row, int head, int left, int head_dim, bf16x8 (&f)[kD / 16]) {
    const int lane = threadIdx.x & 63;
    const __amdgpu_buffer_rsrc_t rsrc = head_rsrc(t, row, head, left, head_dim);
#pragma unroll
    for (int s = 0; s < kD / 16; ++s)
        f[s] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                                              rsrc, head_offset(t, lane & 31, 16 * s + 8 * (lane >> 5), head_dim), 0, 0));
}

// kStep rows of one head between memory and LDS, through registers: panels
// of 64 columns, rows of eight 16-byte chunks, two chunks a thread and panel.
template <int kD>
struct Staged {
    static constexpr int kN = kStep * kD / 8 / kThreads;
    u32x4 v[kN];
    __device__ __forceinline__ void load(const Heads &t, int64_t row, int head, int left, int head_dim) {
        const __amdgpu_buffer_rsrc_t rsrc = head_rsrc(t, row, head, left, head_dim);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int id = (i % 2) * kThreads + threadIdx.x;
            v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 rsrc, head_offset(t, id >> 3, (i / 2) * kPanel + (id & 7) * 8, head_dim), 0, 0));
        }
    }
    __device__ __forceinline__ void store(uint16_t *lds) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int id = (i % 2) * kThreads + threadIdx.x;
            *reinterpret_cast<u32x4 *>(lds + (i / 2) * kStep * kPanel + lds_at(id >> 3, id & 7)) = v[i];
        }
    }
};

// First operand, rows of 32-row block b, 16-wide column step s.
__device__ __forceinline__ bf16x8 read_rows(const uint16_t *lds, int b, int s) {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const bf16x8 *>(lds + (s / 4) * kStep * kPanel +
                                             lds_at(b * 32 + (lane & 31), 2 * (s % 4) + (lane >> 5)));
}

// First operand, transposed: 32-column block d as its rows, over the 16
// staged rows from 16 s in the order the header gives.
__device__ __forceinline__ bf16x8 read_columns(const uint16_t *lds, int d, int s) {
    const int lane = threadIdx.x & 63;
    const int col = (d % 2) * 32 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    const int row = 16 * s + 4 * (lane >> 5) + ((lane & 15) >> 2);
    const uint16_t *p = lds + (d / 2) * kStep * kPanel;
    union {
        s16x4 h[2];
        bf16x8 f;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + lds_at(row, col >> 3) + (col & 7)));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + lds_at(row + 8, col >> 3) + (col & 7)));
    return u.f;
}

// Values 8 s .. 8 s + 7 as a bf16 operand.
__device__ __forceinline__ bf16x8 pack(const f32x16 &v, int s) {
    bf16x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = __bf16(v[8 * s + e]);
    return r;
}

// Both half-waves' values of the same column, summed, and the larger one.
__device__ __forceinline__ float sum_halves(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return __builtin_bit_cast(float, uint32_t(p[0])) + __builtin_bit_cast(float, uint32_t(p[1]));
}
__device__ __forceinline__ float max_halves(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return fmaxf(__builtin_bit_cast(float, uint32_t(p[0])), __builtin_bit_cast(float, uint32_t(p[1])));
}

__device__ __forceinline__ f32x16 mfma(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A wave's [32 columns d][32 rows] blocks, times mul, to rows of a head: the
// halves exchange groups of four so that each lane stores eight columns.
template <int kD>
__device__ __forceinline__ void store_rows(const Heads &t, int64_t row, int head, int left, int head_dim, const f32x16 (&o)[kD / 32],
                                           float mul) {
    const int lane = threadIdx.x & 63;
    uint16_t *p = t.p + (row + (lane & 31)) * t.row + head * t.head;
#pragma unroll
    for (int d = 0; d < kD / 32; ++d)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            union {
                __bf16 h[8];
                uint32_t w[4];
            } a;
#pragma unroll
            for (int e = 0; e < 8; ++e) a.h[e] = __bf16(o[d][8 * g + e] * mul);
            // words 0, 1: group 2 g; words 2, 3: group 2 g + 1; the low half
            // takes both parts of the first, the high half of the second
            const auto x = __builtin_amdgcn_permlane32_swap(a.w[0], a.w[2], false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(a.w[1], a.w[3], false, false);
            const u32x4 v = {x[0], y[0], x[1], y[1]};
            const int col = d * 32 + 16 * g + 8 * (lane >> 5);
            if ((lane & 31) < left && col < head_dim) *reinterpret_cast<u32x4 *>(p + col) = v;
        }
}

// Key range [lo, hi) that rows [first, first + count) of a chunk see.
__device__ __forceinline__ void band(int first, int count, int len, int window, int &lo, int &hi) {
    lo = 0;
    hi = len;
    if (window >= 0) {
        lo = max(0, first - window);
        hi = min(len, first + count + window);
    }
}

// Whether rows [r, r + 31] and keys [k, k + n) of a chunk meet in the band
// at all, and whether they all do.
__device__ __forceinline__ bool any_visible(int r, int k, int n, int window) {
    return window < 0 || (k <= r + 31 + window && k + n - 1 >= r - window);
}
__device__ __forceinline__ bool all_visible(int r, int k, int n, int len, int window) {
    return k + n <= len && (window < 0 || (k + n - 1 - r <= window && r + 31 - k <= window));
}

// Row of value r of a result block, without its 32-row block and the four
// rows that the upper half-wave is further down.
__device__ __forceinline__ constexpr int row_of(int r) { return 8 * (r >> 2) + (r & 3); }

// The keys a row sees (or rows that see a key), as first + [0, count): one
// subtraction and one unsigned comparison tell whether another is in it.
struct Seen {
    int first;
    uint32_t count;
};
__device__ __forceinline__ Seen seen_by(int row, int len, int window) {
    const int first = window < 0 ? 0 : max(0, row - window);
    const int end = window < 0 ? len : min(len, row + window + 1);
    return Seen{first, uint32_t(max(end - first, 0))};
}

template <int kD>
__global__ __launch_bounds__(kThreads) void attention_forward_kernel(AttentionArgs a) {
    constexpr int kSteps = kD / 16, kBlocks = kD / 32;
    __shared__ uint16_t sk[2][kStep * kD], sv[2][kStep * kD];
    const int64_t id = xcd_contiguous_tile(blockIdx.x, gridDim.x);
    const int head = int(id / a.tiles);
    const Tile tile = find_tile(a.cu, a.chunks, a.rows, id - int64_t(head) * a.tiles);
    if (tile.len == 0) return;
    const int kv = head / (a.q_heads / a.kv_heads);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int len = tile.len, window = min(a.window, len);
    const int r0 = tile.first + wave * kWaveRows;
    const int row = r0 + (lane & 31);
    const Seen seen = seen_by(row, len, window);

    bf16x8 q[kSteps];
    load_operand<kD>(a.q, tile.begin + r0, head, len - r0, a.head_dim, q);
    int lo, hi;
    band(tile.first, kTileRows, len, window, lo, hi);
    const float c2 = a.scale * kLog2e;
    const float sink = a.sink ? a.sink[head] / a.scale : 0.0f;  // in the unscaled logits' units
    f32x16 o[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) o[d] = f32x16{};
    float top = -INFINITY;  // the raised maximum, in powers of two
    float sum = 0.0f;       // of this half-wave's keys

    Staged<kD> gk, gv;
    gk.load(a.k, tile.begin + lo, kv, len - lo, a.head_dim);
    gv.load(a.v, tile.begin + lo, kv, len - lo, a.head_dim);
    gk.store(sk[0]);
    gv.store(sv[0]);
    int buf = 0;
    for (int k0 = lo; k0 < hi; k0 += kStep, buf ^= 1) {
        const bool more = k0 + kStep < hi;
        if (more) {
            gk.load(a.k, tile.begin + k0 + kStep, kv, len - k0 - kStep, a.head_dim);
            gv.load(a.v, tile.begin + k0 + kStep, kv, len - k0 - kStep, a.head_dim);
        }
        __syncthreads();  // this step's tiles are written, the other buffers read
        if (r0 < len && any_visible(r0, k0, kStep, window)) {
            const uint16_t *tk = sk[buf], *tv = sv[buf];
            f32x16 s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f32x16{};
#pragma unroll
                for (int i = 0; i < kSteps; ++i) s[b] = mfma(read_rows(tk, b, i), q[i], s[b]);
            }
            if (k0 == 0 && a.sink) s[0][0] += lane < 32 ? sink : 0.0f;
            if (!all_visible(r0, k0, kStep, len, window)) {
                const int at = k0 + 4 * (lane >> 5) - seen.first;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[b][r] = uint32_t(at + 32 * b + row_of(r)) < seen.count ? s[b][r] : -INFINITY;
            }
            float m = s[0][0];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) m = fmaxf(m, s[b][r]);
            m = max_halves(m) * c2;
            if (__any(m > top + kRaise)) {
                // a row that has seen nothing yet keeps -inf and zero sums
                const float next = fmaxf(top, m);
                const float alpha = top == next ? 1.0f : __builtin_amdgcn_exp2f(top - next);
                top = next;
                sum *= alpha;
#pragma unroll
                for (int d = 0; d < kBlocks; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
            }
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], c2, -base));
                    sum += s[b][r];
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x8 p = pack(s[i >> 1], i & 1);
#pragma unroll
                for (int d = 0; d < kBlocks; ++d) o[d] = mfma(read_columns(tv, d, i), p, o[d]);
            }
        }
        if (more) {
            gk.store(sk[buf ^ 1]);
            gv.store(sv[buf ^ 1]);
        }
    }
    sum = sum_halves(sum);
    if (r0 >= len) return;
    store_rows<kD>(a.out, tile.begin + r0, head, len - r0, a.head_dim, o, sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f);
    if (a.lse && lane < 32 && row < len)
        a.lse[int64_t(head) * a.rows + tile.begin + row] = sum == 0.0f ? -INFINITY : (top + __builtin_log2f(sum)) * kLn2;
}

// dq, delta and the sink's partial sums: the forward kernel's shape, with the
// probabilities from lse.  The partial sums use sum_j p_ij dp_ij in place of
// delta: the same number without out's rounding, which dsink (float32, a sum
// over every row) would show.
template <int kD>
__global__ __launch_bounds__(kThreads) void attention_dq_kernel(AttentionArgs a) {
    constexpr int kSteps = kD / 16, kBlocks = kD / 32;
    __shared__ uint16_t sk[2][kStep * kD], sv[2][kStep * kD];
    __shared__ float part[4];
    const int64_t id = xcd_contiguous_tile(blockIdx.x, gridDim.x);
    const int head = int(id / a.tiles);
    const int64_t t = id - int64_t(head) * a.tiles;
    const Tile tile = find_tile(a.cu, a.chunks, a.rows, t);
    float *dsink = a.dsink_part ? a.dsink_part + int64_t(head) * a.tiles + t : nullptr;
    if (tile.len == 0) {
        if (dsink && threadIdx.x == 0) *dsink = 0.0f;
        return;
    }
    const int kv = head / (a.q_heads / a.kv_heads);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int len = tile.len, window = min(a.window, len);
    const int r0 = tile.first + wave * kWaveRows;
    const int row = r0 + (lane & 31);
    const Seen seen = seen_by(row, len, window);
    const int64_t at = int64_t(head) * a.rows + tile.begin + row;

    bf16x8 q[kSteps], g[kSteps];
    load_operand<kD>(a.q, tile.begin + r0, head, len - r0, a.head_dim, q);
    load_operand<kD>(a.dout, tile.begin + r0, head, len - r0, a.head_dim, g);
    float delta = 0.0f, lse2 = 0.0f;
    {
        bf16x8 o[kSteps];
        load_operand<kD>(a.out, tile.begin + r0, head, len - r0, a.head_dim, o);
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = fmaf(float(o[i][e]), float(g[i][e]), delta);
        delta = sum_halves(delta);
        if (row < len) {
            lse2 = a.lse[at] * kLog2e;
            if (lane < 32) a.delta[at] = delta;
        }
    }
    // a row that saw nothing: every probability is zero
    if (lse2 == -INFINITY) lse2 = INFINITY;
    int lo, hi;
    band(tile.first, kTileRows, len, window, lo, hi);
    const float c2 = a.scale * kLog2e;
    const float sink = a.sink ? a.sink[head] / a.scale : 0.0f;
    f32x16 dq[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) dq[d] = f32x16{};
    float p0 = 0.0f, p0dp0 = 0.0f, pdp = 0.0f;

    Staged<kD> gk, gv;
    gk.load(a.k, tile.begin + lo, kv, len - lo, a.head_dim);
    gv.load(a.v, tile.begin + lo, kv, len - lo, a.head_dim);
    gk.store(sk[0]);
    gv.store(sv[0]);
    int buf = 0;
    for (int k0 = lo; k0 < hi; k0 += kStep, buf ^= 1) {
        const bool more = k0 + kStep < hi;
        if (more) {
            gk.load(a.k, tile.begin + k0 + kStep, kv, len - k0 - kStep, a.head_dim);
            gv.load(a.v, tile.begin + k0 + kStep, kv, len - k0 - kStep, a.head_dim);
        }
        __syncthreads();
        if (r0 < len && any_visible(r0, k0, kStep, window)) {
            const uint16_t *tk = sk[buf], *tv = sv[buf];
            const bool all = all_visible(r0, k0, kStep, len, window);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                f32x16 s{}, dp{};
#pragma unroll
                for (int i = 0; i < kSteps; ++i) s = mfma(read_rows(tk, b, i), q[i], s);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) dp = mfma(read_rows(tv, b, i), g[i], dp);
                if (b == 0 && k0 == 0 && a.sink) s[0] += lane < 32 ? sink : 0.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c2, -lse2));
                if (!all) {
                    const int at = k0 + 32 * b + 4 * (lane >> 5) - seen.first;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = uint32_t(at + row_of(r)) < seen.count ? s[r] : 0.0f;
                }
                if (a.sink) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) pdp = fmaf(s[r], dp[r], pdp);
                    if (b == 0 && k0 == 0) {
                        p0 = s[0];
                        p0dp0 = s[0] * dp[0];
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 ds = pack(s, i);
#pragma unroll
                    for (int d = 0; d < kBlocks; ++d) dq[d] = mfma(read_columns(tk, d, 2 * b + i), ds, dq[d]);
                }
            }
        }
        if (more) {
            gk.store(sk[buf ^ 1]);
            gv.store(sv[buf ^ 1]);
        }
    }
    if (r0 < len) store_rows<kD>(a.dq, tile.begin + r0, head, len - r0, a.head_dim, dq, a.scale);
    if (dsink) {
        pdp = sum_halves(pdp);
        float v = lane < 32 && row < len ? p0dp0 - p0 * pdp : 0.0f;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
        if (lane == 0) part[wave] = v;
        __syncthreads();
        if (threadIdx.x == 0) *dsink = (part[0] + part[1]) + (part[2] + part[3]);
    }
}

// dk and dv of one tile of keys of one key head: every query head of the
// group and every row in the band, in a fixed order, into registers.  The
// products' accumulators start from -lse / scale and -delta of their row, so
// that the exponent and dp - delta need no further operation.
template <int kD>
__global__ __launch_bounds__(kThreads) void attention_dkdv_kernel(AttentionArgs a) {
    constexpr int kSteps = kD / 16, kBlocks = kD / 32;
    __shared__ uint16_t sq[2][kStep * kD], sg[2][kStep * kD];
    __shared__ float sl[2][kStep], sd[2][kStep];
    const int64_t id = xcd_contiguous_tile(blockIdx.x, gridDim.x);
    const int kv = int(id / a.tiles);
    const Tile tile = find_tile(a.cu, a.chunks, a.rows, id - int64_t(kv) * a.tiles);
    if (tile.len == 0) return;
    const int group = a.q_heads / a.kv_heads;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int len = tile.len, window = min(a.window, len);
    const int c0 = tile.first + wave * kWaveRows;  // this wave's keys
    const int key = c0 + (lane & 31);
    const Seen seen = seen_by(key, len, window);

    bf16x8 k[kSteps], v[kSteps];
    load_operand<kD>(a.k, tile.begin + c0, kv, len - c0, a.head_dim, k);
    load_operand<kD>(a.v, tile.begin + c0, kv, len - c0, a.head_dim, v);
    int lo, hi;
    band(tile.first, kTileRows, len, window, lo, hi);
    const int per_head = (hi - lo + kStep - 1) / kStep;
    const int total = per_head * group;
    const float c2 = a.scale * kLog2e, inv_scale = 1.0f / a.scale;
    f32x16 dk[kBlocks], dv[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) dk[d] = dv[d] = f32x16{};

    Staged<kD> gq, gg;
    float gl = 0.0f;
    // thread 0 .. 63: lse of a row; 64 .. 127: delta of a row
    auto load = [&](int h, int q0) {
        const int head = kv * group + h;
        gq.load(a.q, tile.begin + q0, head, len - q0, a.head_dim);
        gg.load(a.dout, tile.begin + q0, head, len - q0, a.head_dim);
        const int r = q0 + (threadIdx.x & 63);
        if (threadIdx.x < 128) {
            const bool delta = threadIdx.x >= 64;
            gl = 0.0f;
            if (r < len) gl = (delta ? a.delta : a.lse)[int64_t(head) * a.rows + tile.begin + r];
            // rows behind the chunk and rows that saw nothing: probability zero
            gl = delta ? -gl : r < len && gl != -INFINITY ? -gl * inv_scale : -INFINITY;
        }
    };
    auto store = [&](int buf) {
        gq.store(sq[buf]);
        gg.store(sg[buf]);
        if (threadIdx.x < 64)
            sl[buf][threadIdx.x] = gl;
        else if (threadIdx.x < 128)
            sd[buf][threadIdx.x - 64] = gl;
    };
    load(0, lo);
    store(0);
    int h = 0, q0 = lo;
    for (int n = 0; n < total; ++n) {
        const int buf = n & 1;
        int h1 = h, q1 = q0 + kStep;
        if (q1 >= hi) {
            ++h1;
            q1 = lo;
        }
        const bool more = n + 1 < total;
        if (more) load(h1, q1);
        __syncthreads();
        if (c0 < len) {
            const float kb = a.sink && key == 0 ? a.sink[kv * group + h] * kLog2e : 0.0f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int rb = q0 + 32 * b;
                if (rb >= len || !any_visible(c0, rb, 32, window)) continue;
                f32x16 s, dp;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int off = 32 * b + 8 * g + 4 * (lane >> 5);
                    const f32x4 l = *reinterpret_cast<const f32x4 *>(&sl[buf][off]);
                    const f32x4 d = *reinterpret_cast<const f32x4 *>(&sd[buf][off]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[4 * g + e] = l[e];
                        dp[4 * g + e] = d[e];
                    }
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) s = mfma(read_rows(sq[buf], b, i), k[i], s);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) dp = mfma(read_rows(sg[buf], b, i), v[i], dp);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c2, kb));
                if (!all_visible(c0, rb, 32, len, window)) {
                    const int at = rb + 4 * (lane >> 5) - seen.first;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = uint32_t(at + row_of(r)) < seen.count ? s[r] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 p = pack(s, i);
#pragma unroll
                    for (int d = 0; d < kBlocks; ++d) dv[d] = mfma(read_columns(sg[buf], d, 2 * b + i), p, dv[d]);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] *= dp[r];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 ds = pack(s, i);
#pragma unroll
                    for (int d = 0; d < kBlocks; ++d) dk[d] = mfma(read_columns(sq[buf], d, 2 * b + i), ds, dk[d]);
                }
            }
        }
        if (more) store(buf ^ 1);
        h = h1;
        q0 = q1;
    }
    if (c0 >= len) return;
    store_rows<kD>(a.dk, tile.begin + c0, kv, len - c0, a.head_dim, dk, a.scale);
    store_rows<kD>(a.dv, tile.begin + c0, kv, len - c0, a.head_dim, dv, 1.0f);
}

// dsink[h]: the tiles' partial sums, in float64 and a fixed order.
__global__ __launch_bounds__(kThreads) void attention_dsink_kernel(const float *part, int32_t tiles, float *dsink) {
    __shared__ double lds[kThreads];
    const float *p = part + int64_t(blockIdx.x) * tiles;
    double v = 0.0;
    for (int i = threadIdx.x; i < tiles; i += kThreads) v += double(p[i]);
    lds[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int n = kThreads / 2; n > 0; n >>= 1) {
        if (int(threadIdx.x) < n) lds[threadIdx.x] += lds[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) dsink[blockIdx.x] = float(lds[0]);
}

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxRowStride = int64_t(1) << 22;  // a 64-row tile's byte offsets stay below 2^31

int check_heads(const mimo_heads &t, const char *who, const char *name, int64_t rows, int32_t heads, int32_t head_dim, bool written) {
    const std::string at = std::string(who) + ": " + name;
    if (!t.data || !check_ptr_align(t.data, 16))
        return set_error(MIMO_E_INVALID, at + " must be non-null and 16-byte aligned");
    if (t.row_stride % 8 || t.head_stride % 8 || t.row_stride < head_dim || t.head_stride < 0 ||
        t.row_stride > kMaxRowStride || t.head_stride > (int64_t(1) << 40))
        return set_error(MIMO_E_INVALID, at + "'s strides must be multiples of 8 values, row_stride in [head_dim, 2^22], head_stride >= 0");
    if (!written) return MIMO_OK;
    const bool head_inside = heads == 1 || (t.head_stride >= head_dim && t.row_stride >= (heads - 1) * t.head_stride + head_dim);
    const bool row_inside = t.head_stride >= (rows - 1) * t.row_stride + head_dim;
    if (!head_inside && !row_inside) return set_error(MIMO_E_INVALID, at + " is written, so its rows and heads must not overlap");
    return MIMO_OK;
}

// What forward and backward check alike; fills the kernels' arguments.
int check_attention(const mimo_attention *p, const char *who, AttentionArgs &a) {
    const std::string w(who);
    if (!p) return set_error(MIMO_E_INVALID, w + ": null arguments");
    if (p->rows < 0 || p->chunks < 0 || p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads || p->q_heads > 65536)
        return set_error(MIMO_E_INVALID, w + ": rows and chunks must be >= 0, q_heads a multiple of kv_heads >= 1, at most 65536");
    if (p->head_dim < 8 || p->head_dim > MIMO_HEAD_DIM_MAX || p->head_dim % 8)
        return set_error(MIMO_E_INVALID, w + ": head_dim must be a multiple of 8 in [8, 128]");
    if (!(p->scale >= 1e-18f && p->scale <= 1e18f)) return set_error(MIMO_E_INVALID, w + ": scale must be in [1e-18, 1e18]");
    if (p->rows > kMaxRows || p->chunks > kMaxRows)
        return set_error(MIMO_E_TOO_LARGE, w + ": more than 2^30 rows or chunks");
    std::memset(&a, 0, sizeof(a));
    a.rows = p->rows;
    a.q_heads = p->q_heads;
    a.kv_heads = p->kv_heads;
    a.head_dim = p->head_dim;
    a.chunks = p->chunks;
    a.window = p->window < 0 ? -1 : p->window;
    a.scale = p->scale;
    a.tiles = int32_t(p->rows / kTileRows + p->chunks);
    if (p->rows == 0 || p->chunks == 0) return MIMO_OK;
    if (int64_t(a.tiles) * p->q_heads > 0x7FFFFFFFll)
        return set_error(MIMO_E_TOO_LARGE, w + ": more than 2^31 - 1 tiles");
    if (!p->cu_seqlens || !check_ptr_align(p->cu_seqlens, 4) || !check_ptr_align(p->sink, 4))
        return set_error(MIMO_E_INVALID, w + ": cu_seqlens must be non-null; it and sink 4-byte aligned");
    int st;
    if ((st = check_heads(p->q, who, "q", p->rows, p->q_heads, p->head_dim, false)) != MIMO_OK) return st;
    if ((st = check_heads(p->k, who, "k", p->rows, p->kv_heads, p->head_dim, false)) != MIMO_OK) return st;
    if ((st = check_heads(p->v, who, "v", p->rows, p->kv_heads, p->head_dim, false)) != MIMO_OK) return st;
    auto heads = [](const mimo_heads &t) { return Heads{static_cast<uint16_t *>(t.data), t.row_stride, t.head_stride}; };
    a.q = heads(p->q);
    a.k = heads(p->k);
    a.v = heads(p->v);
    a.out = heads(p->out);
    a.cu = p->cu_seqlens;
    a.sink = p->sink;
    a.lse = p->lse;
    return MIMO_OK;
}

size_t delta_bytes(int64_t rows, int32_t q_heads) { return align256(size_t(rows) * size_t(q_heads) * sizeof(float)); }

}  // namespace
}  // namespace mimo

using namespace mimo;

extern "C" {

int mimo_chunk_attention(const mimo_attention *p, void *stream) {
    clear_error();
    AttentionArgs a;
    int st = check_attention(p, "chunk_attention", a);
    if (st != MIMO_OK) return st;
    if (a.rows == 0 || a.chunks == 0) return MIMO_OK;
    if ((st = check_heads(p->out, "chunk_attention", "out", p->rows, p->q_heads, p->head_dim, true)) != MIMO_OK) return st;
    if (!check_ptr_align(p->lse, 4)) return set_error(MIMO_E_INVALID, "chunk_attention: lse must be 4-byte aligned");
    if (p->out.data == p->q.data || p->out.data == p->k.data || p->out.data == p->v.data)
        return set_error(MIMO_E_INVALID, "chunk_attention: out must not be an input");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid{unsigned(a.tiles) * unsigned(a.q_heads), 1, 1}, block{unsigned(kThreads), 1, 1};
    const hipError_t e = timed_launch(s, [&] {
        if (a.head_dim <= 64)
            hipLaunchKernelGGL(attention_forward_kernel<64>, grid, block, 0, s, a);
        else
            hipLaunchKernelGGL(attention_forward_kernel<128>, grid, block, 0, s, a);
    });
    if (e != hipSuccess) return hip_error(e, "chunk_attention: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

size_t mimo_chunk_attention_workspace_bytes(int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t chunks) {
    if (rows < 0 || rows > kMaxRows || chunks < 0 || chunks > kMaxRows || kv_heads < 1 || q_heads < kv_heads ||
        q_heads % kv_heads || q_heads > 65536 || head_dim < 8 || head_dim > MIMO_HEAD_DIM_MAX || head_dim % 8)
        return 0;
    return delta_bytes(rows, q_heads) + align256(size_t(rows / kTileRows + chunks) * size_t(q_heads) * sizeof(float));
}

int mimo_chunk_attention_backward(const mimo_attention *p, const mimo_attention_grads *g, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    clear_error();
    AttentionArgs a;
    const char *who = "chunk_attention_backward";
    int st = check_attention(p, who, a);
    if (st != MIMO_OK) return st;
    if (!g) return set_error(MIMO_E_INVALID, std::string(who) + ": null gradients");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (g->dsink && (!p->sink && a.rows && a.chunks))
        return set_error(MIMO_E_INVALID, std::string(who) + ": dsink is given without sink");
    if (a.rows && a.chunks) {
        if ((st = check_heads(p->out, who, "out", p->rows, p->q_heads, p->head_dim, false)) != MIMO_OK) return st;
        if ((st = check_heads(g->dout, who, "dout", p->rows, p->q_heads, p->head_dim, false)) != MIMO_OK) return st;
        if ((st = check_heads(g->dq, who, "dq", p->rows, p->q_heads, p->head_dim, true)) != MIMO_OK) return st;
        if ((st = check_heads(g->dk, who, "dk", p->rows, p->kv_heads, p->head_dim, true)) != MIMO_OK) return st;
        if ((st = check_heads(g->dv, who, "dv", p->rows, p->kv_heads, p->head_dim, true)) != MIMO_OK) return st;
        if (!p->lse || !check_ptr_align(p->lse, 4) || !check_ptr_align(g->dsink, 4))
            return set_error(MIMO_E_INVALID, std::string(who) + ": lse must be non-null; it and dsink 4-byte aligned");
        const void *ins[] = {p->q.data, p->k.data, p->v.data, p->out.data, g->dout.data};
        const void *outs[] = {g->dq.data, g->dk.data, g->dv.data};
        for (int i = 0; i < 3; ++i) {
            for (const void *in : ins)
                if (outs[i] == in) return set_error(MIMO_E_INVALID, std::string(who) + ": a gradient must not be an input");
            for (int j = 0; j < i; ++j)
                if (outs[i] == outs[j]) return set_error(MIMO_E_INVALID, std::string(who) + ": two gradients are the same tensor");
        }
        if (!workspace || !check_ptr_align(workspace, 16))
            return set_error(MIMO_E_INVALID, std::string(who) + ": workspace must be non-null and 16-byte aligned");
        if (workspace_bytes < mimo_chunk_attention_workspace_bytes(a.rows, a.q_heads, a.kv_heads, a.head_dim, a.chunks))
            return set_error(MIMO_E_CAPACITY,
                             std::string(who) + ": workspace smaller than mimo_chunk_attention_workspace_bytes");
    } else if (!g->dsink) {
        return MIMO_OK;
    }
    auto heads = [](const mimo_heads &t) { return Heads{static_cast<uint16_t *>(t.data), t.row_stride, t.head_stride}; };
    a.dout = heads(g->dout);
    a.dq = heads(g->dq);
    a.dk = heads(g->dk);
    a.dv = heads(g->dv);
    a.delta = static_cast<float *>(workspace);
    if (g->dsink)
        a.dsink_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + delta_bytes(a.rows, a.q_heads));
    const int32_t tiles = a.rows && a.chunks ? a.tiles : 0;
    const dim3 dq_grid{unsigned(tiles) * unsigned(a.q_heads), 1, 1}, dkdv_grid{unsigned(tiles) * unsigned(a.kv_heads), 1, 1};
    const dim3 block{unsigned(kThreads), 1, 1}, sink_grid{unsigned(a.q_heads), 1, 1};
    const hipError_t e = timed_launch(s, [&] {
        if (tiles && a.head_dim <= 64) {
            hipLaunchKernelGGL(attention_dq_kernel<64>, dq_grid, block, 0, s, a);
            hipLaunchKernelGGL(attention_dkdv_kernel<64>, dkdv_grid, block, 0, s, a);
        } else if (tiles) {
            hipLaunchKernelGGL(attention_dq_kernel<128>, dq_grid, block, 0, s, a);
            hipLaunchKernelGGL(attention_dkdv_kernel<128>, dkdv_grid, block, 0, s, a);
        }
        if (g->dsink) hipLaunchKernelGGL(attention_dsink_kernel, sink_grid, block, 0, s, a.dsink_part, tiles, g->dsink);
    });
    if (e != hipSuccess) return hip_error(e, "chunk_attention_backward: kernel launch");
    g_dispatches.fetch_add((tiles ? 2 : 0) + (g->dsink ? 1 : 0));
    return MIMO_OK;
}

}  // extern "C"
