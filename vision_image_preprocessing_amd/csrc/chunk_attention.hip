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

#include <algorithm>
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
typedef __attribute__((address_space(3))) void *lds_void_ptr;

constexpr int kThreads = 256;
constexpr int kWaveRows = 32;                 // rows (or keys) one wave owns
constexpr int kTileRows = 4 * kWaveRows;      // of one workgroup
constexpr int kStep = 64;                     // keys (or rows) staged in LDS at a time
constexpr int kPanelBytes = kStep * 128;      // kStep rows of 64 head columns
constexpr int kWord3 = 0x00020000;            // raw buffer resource word 3
constexpr uint32_t kOutside = 0x7FFFFFF8u;    // a byte offset past every resource: reads zeros
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
// The running maximum is raised only when a row outgrows it by this many
// powers of two: probabilities stay below 2^8 meanwhile, which float32 sums
// and bf16 operands hold at full relative precision.
constexpr float kRaise = 8.0f;
// Sinks beyond this count as this.  lse is float32, and p = exp(s - lse) of
// the backward pass is off by 2^-23 |s| or so: a sink of -1e9 on a key that a
// row sees alone gave p0 = 2^30, and sinks above 3.4e38 scale became
// infinite.  At the limit (and any further out) key 0 has all of a row's
// weight or none, logits being less than some 8000 apart, and p keeps 10 bits.
constexpr float kMaxSink = MIMO_SINK_MAX;

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
    float *neg_lse;      // [q_heads][rows]: -lse / scale (backward)
    float *neg_delta;    // [q_heads][rows]: -delta (backward)
    float *dsink_part;   // [q_heads][row_tiles], or null
    float *dsink;        // [q_heads], or null
    float *part;         // [slices][2][kv_heads][rows][head_dim]: dk, dv of each slice, or null
    int64_t rows;
    int32_t q_heads, kv_heads, head_dim, chunks;
    int32_t group;       // q_heads / kv_heads
    int32_t window;      // < 0: none
    int32_t tiles;       // of the launch: rows / its tile rows + chunks
    int32_t row_tiles;   // of the dq kernel
    int32_t slices;      // parts that dk's and dv's sums are split into
    float scale;
};

// A workgroup's tile: its first row within the chunk of len rows that starts
// at row begin; len = 0 for a tile that holds nothing.
struct Tile {
    int64_t begin;
    int32_t len, first;
};

// xcd_contiguous_tile in 32 bits (a launch has fewer than 2^31 workgroups).
__device__ __forceinline__ uint32_t tile_of_xcd(uint32_t b, uint32_t grid) {
    const uint32_t per = grid / kXcds;
    return b < per * kXcds ? (b % kXcds) * per + b / kXcds : b;
}

// Tile t of the batch, kRows rows each: chunk c's tiles are numbered from
// cu[c] / kRows + c, which leaves each chunk as many numbers as it needs or
// one more, so that the grid is known from the row and chunk counts alone.
// The search relies on ascending boundaries.  Where they do not ascend it may
// take any chunk, so the chunk's own two are checked: one that is not inside
// [0, rows], or that the tile is not a part of, gives an empty tile, through
// which nothing is read or written.
template <int kRows>
__device__ __forceinline__ Tile find_tile(const int32_t *cu, int chunks, int64_t rows, int t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = chunks;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int idx = lo + lane * step;
        const bool le = idx < hi && int64_t(cu[idx] / kRows) + idx <= t;
        // in int: the count is unsigned, and less than one of it is not -1
        // (none is at most t where rows lie in front of the first boundary)
        const int k = max(int(__popcll(__ballot(le))) - 1, 0);
        lo += k * step;
        hi = min(lo + step, hi);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int64_t b = cu[lo], e = cu[lo + 1];
    Tile r{0, 0, 0};
    const int64_t first = (t - (cu[lo] / kRows + int64_t(lo))) * kRows;
    if (b < 0 || e > rows || first < 0 || first >= e - b) return r;
    r.begin = b;
    r.len = __builtin_amdgcn_readfirstlane(int(e - b));
    r.first = __builtin_amdgcn_readfirstlane(int(first));
    return r;
}

// Staged tiles.  Panel rows are 128 bytes, eight 16-byte chunks; chunk v of
// row r lies at position v ^ row_key(r % 8) ^ block_key(r / 8).  A cycle of
// LDS serves 256 bytes, two panel rows' worth of banks: 16 lanes of an operand
// read, whose rows then differ by row and block, and 32 lanes of a transposed
// read, half rows of four rows, whose keys then have to differ in their
// highest bit between rows two apart (hence the exchange of bits 1 and 2; a
// plain r ^ r / 8 measured two conflict cycles a transposed read).  All is an
// exclusive or, so a lane needs few distinct addresses, formed once;
// everything else is a constant offset.
__device__ __forceinline__ constexpr int row_key(int r) { return (r & 1) | ((r & 2) << 1) | ((r & 4) >> 1); }
__device__ __forceinline__ constexpr int block_key(int g) { return g ^ ((g & 3) >> 1); }
struct LdsAddress {
    int row[4];  // operand reads: chunk 2 s + l / 32 of row l % 32, by s ^ 2 (block)
    int col[8];  // transposed reads, by chunk ^ block_key
};
__device__ __forceinline__ LdsAddress lds_address() {
    const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5;
    LdsAddress a;
#pragma unroll
    for (int j = 0; j < 4; ++j) a.row[j] = l * 128 + ((h ^ row_key(l & 7) ^ block_key(l >> 3) ^ (2 * j)) << 4);
    const int x = 4 * h + ((lane & 15) >> 2), c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
    for (int j = 0; j < 8; ++j) a.col[j] = x * 128 + ((c ^ row_key(x) ^ j) << 4) + (lane & 1) * 8;
    return a;
}

// First operand, rows of 32-row block b, 16-wide column step s.
__device__ __forceinline__ bf16x8 read_rows(const uint8_t *lds, const LdsAddress &a, int b, int s) {
    return *reinterpret_cast<const bf16x8 *>(lds + a.row[(s & 3) ^ (2 * b)] + (s / 4) * kPanelBytes + b * 32 * 128);
}

// First operand, transposed: 32-column block d as its rows, over the 16
// staged rows from 16 s in the order the header gives.
__device__ __forceinline__ bf16x8 read_columns(const uint8_t *lds, const LdsAddress &a, int d, int s) {
    const int c = (4 * (d & 1)) ^ block_key(2 * s), c8 = (4 * (d & 1)) ^ block_key(2 * s + 1);
    const uint8_t *p = lds + (d / 2) * kPanelBytes + s * 16 * 128;
    union {
        s16x4 h[2];
        bf16x8 f;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + a.col[c]));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + a.col[c8] + 8 * 128));
    return u.f;
}

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

// 16 bytes a lane straight into LDS, one after the other.  The host's pass
// over this file does not know the size (and would drop every kernel that
// contains it), so it does not see the call.
__device__ __forceinline__ void load_to_lds(const __amdgpu_buffer_rsrc_t &rsrc, uint8_t *lds, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_ptr)lds, 16, off, 0, 0, 0);
#endif
}

// kStep rows of one head straight into LDS by the workgroup's four waves, 1 KB
// (eight rows of a panel) a load.
template <int kPanels>
struct Loader {
    static constexpr int kN = kPanels * 8 / 4;
    uint32_t off[kN];
    __device__ __forceinline__ Loader(const Heads &t, int wave, int head_dim) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int n = i * 4 + wave, g = n % 8;
            const int v = (lane & 7) ^ row_key(lane >> 3) ^ block_key(g);
            off[i] = head_offset(t, g * 8 + (lane >> 3), (n / 8) * 64 + v * 8, head_dim);
        }
    }
    __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t &rsrc, int wave, uint8_t *lds) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            load_to_lds(rsrc, lds + (i * 4 + wave) * 1024, off[i]);
        }
    }
};

// The loads into LDS that the workgroup's waves made have landed, and every
// wave has read what it wanted of the tiles before.  (__syncthreads would do,
// with a fence that the loads issued next need not wait for.)
__device__ __forceinline__ void tiles_ready() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
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

// The lane's number, counted: behind a long loop that is cheaper than keeping
// threadIdx.x through it, which has spilled a register.
__device__ __forceinline__ int lane_again() { return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)); }

// [32 columns][32 rows] blocks, times mul, to rows of a head: the halves
// exchange groups of four values so that each lane stores eight columns.
// Stores past the chunk's rows or head_dim go past the resource, which drops
// them.
template <int kBlocks>
__device__ __forceinline__ void store_rows(const Heads &t, int64_t row, int head, int left, int head_dim, const f32x16 (&o)[kBlocks],
                                           float mul) {
    const int lane = lane_again();
    const __amdgpu_buffer_rsrc_t rsrc = head_rsrc(t, row, head, left, head_dim);
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            bf16x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __bf16(o[d][8 * g + e] * mul);
            const u32x4 a = __builtin_bit_cast(u32x4, v);
            // words 0, 1: columns 8 (2 g) + 4 (lane / 32) on; words 2, 3:
            // eight further; the low half takes both parts of the first, the
            // high half of the second
            const auto x = __builtin_amdgcn_permlane32_swap(a[0], a[2], false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(a[1], a[3], false, false);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{x[0], y[0], x[1], y[1]}, rsrc,
                                                   head_offset(t, lane & 31, d * 32 + 16 * g + 8 * (lane >> 5), head_dim), 0, 0);
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

// A head's sink as it counts: within kMaxSink, -inf (no key 0) and NaN as they are.
__device__ __forceinline__ float head_sink(const float *sink, int head) {
    const float v = sink[head];
    return v > kMaxSink ? kMaxSink : v < -kMaxSink && v != -INFINITY ? -kMaxSink : v;
}

// Row of value r of a result block, without its 32-row block and the four
// rows that the upper half-wave is further down.
__device__ __forceinline__ constexpr int row_of(int r) { return 8 * (r >> 2) + (r & 3); }

// The keys a row sees (or rows that see a key): [first, end).
struct Seen {
    int first, end;
};
__device__ __forceinline__ Seen seen_by(int row, int len, int window) {
    const int first = window < 0 ? 0 : max(0, row - window);
    const int end = window < 0 ? len : min(len, row + window + 1);
    return Seen{first, max(first, end)};
}

// Which of a block's 32 keys from k on those are: bit row_of(r) for value r of
// the lane.  A value is then masked by two operations without a condition
// register: its bit, spread over a word, selects (three with one, and a wait
// between them).
__device__ __forceinline__ uint32_t seen_bits(const Seen &seen, int k) {
    auto below = [](int n) { return uint32_t(1ull << max(0, min(32, n))); };  // 2^n, modulo 2^32
    return (below(seen.end - k) - below(seen.first - k)) >> (4 * ((threadIdx.x & 63) >> 5));
}
__device__ __forceinline__ float seen_or_none(uint32_t bits, int r, float v) {
    const uint32_t all = uint32_t(__builtin_amdgcn_sbfe(int(bits), row_of(r), 1));
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, v) & all) | (__builtin_bit_cast(uint32_t, -INFINITY) & ~all));
}

// A block's logits of keys that are not seen become -inf: the band's.
__device__ __forceinline__ void mask_band(const Seen &seen, int k, f32x16 &s) {
    const uint32_t bits = seen_bits(seen, k);
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = seen_or_none(bits, r, s[r]);
}
// Values of keys behind the chunk become `other`: all there is to mask without
// a band, and only at the chunk's end, where fewer registers count for more.
__device__ __forceinline__ void mask_end(int len, int k, float other, f32x16 &s) {
    const int left = len - k - 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = row_of(r) < left ? s[r] : other;
}

// How the kernels over query rows are laid out, four waves of 32 rows that
// share each staged tile of keys and values.
//   kRowsOfOne: 128 rows of one head.
//   kHeadsOfFour: 32 rows of four heads that share a key head: the waves see
//     the same keys, so a band costs them 32 + 2 window keys, not 128 + 2
//     window (band of 64 over 32 x 3520 rows: 382 us against 471).
// Sharing out a row's keys among waves, to be joined at the end, was measured
// for calls that leave CUs idle, and gained nothing that a call shows (four
// waves of a workgroup: 12 heads of 2000 rows 33 us against 31; eight waves and
// three buffers: the same 28.2 against 29.5, 32 heads of 216 rows 7.8 against 7.4).
enum Layout { kRowsOfOne, kHeadsOfFour };
template <int kD, Layout kLayout>
struct RowsShape {
    static constexpr int kSteps = kD / 16, kBlocks = kD / 32, kPanels = (kD + 63) / 64;
    static constexpr int kRows = kLayout == kRowsOfOne ? kTileRows : kWaveRows;
    static constexpr int kTileBytes = kPanels * kPanelBytes;
};
// Where a workgroup's part of the launch is: with kHeadsOfFour, `head` of the
// launch counts groups of four heads.
template <Layout kLayout>
struct Place {
    int head, kv, tile;
    __device__ __forceinline__ Place(const AttentionArgs &a, int wave) {
        const uint32_t id = tile_of_xcd(blockIdx.x, gridDim.x), n = id / uint32_t(a.tiles);
        tile = int(id - n * uint32_t(a.tiles));
        head = int(kLayout == kHeadsOfFour ? 4 * n + wave : n);
        kv = int((kLayout == kHeadsOfFour ? 4 * n : n) / uint32_t(a.group));
    }
};

// Calls step(k0, buffer number) for every kStep keys from lo to hi, the next
// tiles' loads under way meanwhile.
template <typename Load, typename Step>
__device__ __forceinline__ void over_keys(int lo, int hi, Load load, Step step) {
    if (lo >= hi) return;
    load(lo, 0);
    for (int k0 = lo;; k0 += 2 * kStep) {
        const bool more = k0 + kStep < hi;
        tiles_ready();
        if (more) load(k0 + kStep, 1);
        step(k0, 0);
        if (!more) break;
        const bool again = k0 + 2 * kStep < hi;
        tiles_ready();
        if (again) load(k0 + 2 * kStep, 0);
        step(k0 + kStep, 1);
        if (!again) break;
    }
}

// out and lse: one pass over the keys with a running maximum and sum; the row's
// query, sums and output stay in registers, keys and values go through LDS.
//
// Without a band the VALU bounds it (83% of its cycles, matrix cores 53%; of
// a wave's 32 x 64 logits each costs an exponential, its scaling, the sum, the
// maximum and half a packing): 32 heads of 64 over 8 of 4096 rows 1.15 ms, over
// 32120 rows 8.76 ms, 0.96 PFLOP/s.  With a band, memory and VALU together: 32
// x 3520 rows, band of 64, 1.15 GB in 305 us, 3.8 TB/s (window 0: 238 us), and
// 380 us where calls follow each other without a pause, since the card then
// lowers its clock.  Tiles loaded two steps ahead of their use instead of one,
// for a workgroup less on the CU, gained nothing (428 us against 384; without
// a band 1.14 ms against 1.11), nor did an order of tiles that gives an XCD all
// heads of its rows instead of one head of all (386 against 381; 16 heads over
// 2 of 4096 rows 179 against 153).
template <int kD, Layout kLayout, bool kBand>
__global__ __launch_bounds__(kThreads, kD == 64 ? 4 : 1) void attention_forward_kernel(AttentionArgs a) {
    typedef RowsShape<kD, kLayout> S;
    constexpr int kSteps = S::kSteps, kBlocks = S::kBlocks;
    // arrays of their own, so that the compiler sees that loads into one
    // never meet reads of another
    __shared__ __attribute__((aligned(16))) uint8_t sk0[S::kTileBytes], sk1[S::kTileBytes];
    __shared__ __attribute__((aligned(16))) uint8_t sv0[S::kTileBytes], sv1[S::kTileBytes];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place<kLayout> place(a, wave);
    const int head = place.head, kv = place.kv;
    const Tile tile = find_tile<S::kRows>(a.cu, a.chunks, a.rows, place.tile);
    if (tile.len == 0) return;
    const int len = tile.len, window = kBand ? min(a.window, len) : -1;
    const int r0 = tile.first + (kLayout == kRowsOfOne ? wave * kWaveRows : 0);
    const int row = r0 + (lane & 31);
    const Seen seen = seen_by(row, len, window);
    const LdsAddress at = lds_address();

    bf16x8 q[kSteps];
    load_operand<kD>(a.q, tile.begin + r0, head, len - r0, a.head_dim, q);
    int lo, hi;
    band(tile.first, S::kRows, len, window, lo, hi);
    const float c2 = a.scale * kLog2e;
    const float sink = a.sink ? head_sink(a.sink, head) / a.scale : 0.0f;  // in the unscaled logits' units
    f32x16 o[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) o[d] = f32x16{};
    float top = -INFINITY;  // the raised maximum, in powers of two
    float sum = 0.0f;       // of this half-wave's keys

    const Loader<S::kPanels> lk(a.k, wave, a.head_dim), lv(a.v, wave, a.head_dim);
    auto load = [&](int k0, int n) __attribute__((always_inline)) {
        lk.load(head_rsrc(a.k, tile.begin + k0, kv, len - k0, a.head_dim), wave, n ? sk1 : sk0);
        lv.load(head_rsrc(a.v, tile.begin + k0, kv, len - k0, a.head_dim), wave, n ? sv1 : sv0);
    };
    auto step = [&](int k0, int n) __attribute__((always_inline)) {
        const uint8_t *tk = n ? sk1 : sk0, *tv = n ? sv1 : sv0;
        if (r0 >= len || !any_visible(r0, k0, kStep, window)) return;
        // with a band, 32 keys that no row sees are left out; without one
        // the two blocks are always taken together
        bool take[2] = {true, true};
        if constexpr (kBand) {
            take[0] = any_visible(r0, k0, 32, window);
            take[1] = k0 + 32 < len && any_visible(r0, k0 + 32, 32, window);
        }
        f32x16 s[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (kBand && !take[b]) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[b][r] = -INFINITY;
                continue;
            }
            s[b] = f32x16{};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s[b] = mfma(read_rows(tk, at, b, i), q[i], s[b]);
            // before the mask: rows that do not see key 0 have none of its sink
            if (b == 0 && k0 == 0 && a.sink) s[0][0] += lane < 32 ? sink : 0.0f;
            if (kBand && !all_visible(r0, k0 + 32 * b, 32, len, window)) mask_band(seen, k0 + 32 * b, s[b]);
        }
        if (!kBand && k0 + kStep > len) {
#pragma unroll
            for (int b = 0; b < 2; ++b) mask_end(len, k0 + 32 * b, -INFINITY, s[b]);
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
        for (int b = 0; b < 2; ++b) {
            if (kBand && !take[b]) continue;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], c2, -base));
                sum += s[b][r];
            }
#pragma unroll
            for (int i = 2 * b; i < 2 * b + 2; ++i) {
                const bf16x8 p = pack(s[b], i & 1);
#pragma unroll
                for (int d = 0; d < kBlocks; ++d) o[d] = mfma(read_columns(tv, at, d, i), p, o[d]);
            }
        }
    };
    over_keys(lo, hi, load, step);

    sum = sum_halves(sum);
    if (r0 >= len) return;
    store_rows<kBlocks>(a.out, tile.begin + r0, head, len - r0, a.head_dim, o, sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f);
    if (a.lse && lane_again() < min(32, len - r0))
        (a.lse + int64_t(head) * a.rows + tile.begin + r0)[lane_again()] = sum == 0.0f ? -INFINITY : (top + __builtin_log2f(sum)) * kLn2;
}

// dq, delta and the sink's partial sums: the forward kernel's shape, with the
// probabilities from lse.
//
// delta is do . out, which has out's rounding; the rounding of one row's
// delta moves all of its ds alike, and where few keys share the probability
// it is as large as the roundings of ds itself.  So where no row sees more
// than kFewKeys keys (the chunk is as short, or the band as narrow: a window
// of 31 or less), delta = sum_j p_ij dp_ij, the same number, from a pass over
// the keys of its own (two products more on a few keys).  Rows at a chunk's
// ends see as few keys with a window of up to 63; they take do . out like the
// others of their launch.  dsink, which is float32, always takes the sum, at
// the end of the one pass.
//
// Three products a pair of row and key: 32 heads of 64 over 8 of 4096 rows
// 1.53 ms, 1.08 PFLOP/s (VALU 67% of its cycles, matrix cores 60%).  With a
// band memory bounds it: 16 x 3520 rows, band of 64, 1.04 GB in 256 us, 4.1
// TB/s.
constexpr int kFewKeys = 64;

template <int kD, Layout kLayout, bool kBand>
__global__ __launch_bounds__(kThreads, kD == 64 ? 3 : 1) void attention_dq_kernel(AttentionArgs a) {
    typedef RowsShape<kD, kLayout> S;
    constexpr int kSteps = S::kSteps, kBlocks = S::kBlocks;
    __shared__ __attribute__((aligned(16))) uint8_t sk0[S::kTileBytes], sk1[S::kTileBytes];
    __shared__ __attribute__((aligned(16))) uint8_t sv0[S::kTileBytes], sv1[S::kTileBytes];
    __shared__ float whole[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place<kLayout> place(a, wave);
    const int head = place.head, kv = place.kv;
    const Tile tile = find_tile<S::kRows>(a.cu, a.chunks, a.rows, place.tile);
    // one partial sum for each head and tile
    float *dsink = a.dsink_part ? a.dsink_part + int64_t(head) * a.tiles + place.tile : nullptr;
    if (tile.len == 0) {
        if (dsink && (kLayout == kHeadsOfFour ? lane == 0 : threadIdx.x == 0)) *dsink = 0.0f;
        return;
    }
    const int len = tile.len, window = kBand ? min(a.window, len) : -1;
    const int r0 = tile.first + (kLayout == kRowsOfOne ? wave * kWaveRows : 0);
    const int row = r0 + (lane & 31);
    const int64_t stat = int64_t(head) * a.rows + tile.begin + row;
    const Seen seen = seen_by(row, len, window);
    const LdsAddress at = lds_address();

    bf16x8 q[kSteps], g[kSteps];
    load_operand<kD>(a.q, tile.begin + r0, head, len - r0, a.head_dim, q);
    load_operand<kD>(a.dout, tile.begin + r0, head, len - r0, a.head_dim, g);
    int lo, hi;
    band(tile.first, S::kRows, len, window, lo, hi);
    const float c2 = a.scale * kLog2e;
    const float sink = a.sink ? head_sink(a.sink, head) / a.scale : 0.0f;
    float lse2 = row < len ? a.lse[stat] * kLog2e : 0.0f;
    if (lse2 == -INFINITY) lse2 = INFINITY;  // a row that saw nothing: every probability is zero
    f32x16 dq[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) dq[d] = f32x16{};
    float delta = 0.0f, pdp = 0.0f, p0 = 0.0f, p0dp0 = 0.0f;

    const Loader<S::kPanels> lk(a.k, wave, a.head_dim), lv(a.v, wave, a.head_dim);
    auto load = [&](int k0, int n) __attribute__((always_inline)) {
        lk.load(head_rsrc(a.k, tile.begin + k0, kv, len - k0, a.head_dim), wave, n ? sk1 : sk0);
        lv.load(head_rsrc(a.v, tile.begin + k0, kv, len - k0, a.head_dim), wave, n ? sv1 : sv0);
    };
    // probabilities and dp of 32 keys
    auto block = [&](int k0, int b, const uint8_t *tk, const uint8_t *tv, bool all, f32x16 &s, f32x16 &dp) __attribute__((always_inline)) {
        s = f32x16{};
        dp = f32x16{};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) s = mfma(read_rows(tk, at, b, i), q[i], s);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) dp = mfma(read_rows(tv, at, b, i), g[i], dp);
        if (b == 0 && k0 == 0 && a.sink) s[0] += lane < 32 ? sink : 0.0f;
        const bool masked = !all && !all_visible(r0, k0 + 32 * b, 32, len, window);
        if (kBand && masked) mask_band(seen, k0 + 32 * b, s);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c2, -lse2));
        if (!kBand && masked) mask_end(len, k0 + 32 * b, 0.0f, s);
    };
    if (len <= kFewKeys || (window >= 0 && window <= (kFewKeys - 1) / 2)) {
        auto sums = [&](int k0, int n) __attribute__((always_inline)) {
            if (r0 >= len || !any_visible(r0, k0, kStep, window)) return;
            const bool all = all_visible(r0, k0, kStep, len, window);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (kBand && !all && (k0 + 32 * b >= len || !any_visible(r0, k0 + 32 * b, 32, window))) continue;
                f32x16 s, dp;
                block(k0, b, n ? sk1 : sk0, n ? sv1 : sv0, all, s, dp);
#pragma unroll
                for (int r = 0; r < 16; ++r) delta = fmaf(s[r], dp[r], delta);
            }
        };
        over_keys(lo, hi, load, sums);
        delta = sum_halves(delta);
        __syncthreads();  // the tiles are read before the next pass loads them
    } else {
        bf16x8 o[kSteps];
        load_operand<kD>(a.out, tile.begin + r0, head, len - r0, a.head_dim, o);
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = fmaf(float(o[i][e]), float(g[i][e]), delta);
        delta = sum_halves(delta);
    }
    if (row < len && lane < 32) {
        a.neg_lse[stat] = lse2 == INFINITY ? -INFINITY : -a.lse[stat] / a.scale;
        a.neg_delta[stat] = -delta;
    }
    auto step = [&](int k0, int n) __attribute__((always_inline)) {
        const uint8_t *tk = n ? sk1 : sk0, *tv = n ? sv1 : sv0;
        if (r0 >= len || !any_visible(r0, k0, kStep, window)) return;
        const bool all = all_visible(r0, k0, kStep, len, window);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (kBand && !all && (k0 + 32 * b >= len || !any_visible(r0, k0 + 32 * b, 32, window))) continue;
            f32x16 s, dp;
            block(k0, b, tk, tv, all, s, dp);
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
                for (int d = 0; d < kBlocks; ++d) dq[d] = mfma(read_columns(tk, at, d, 2 * b + i), ds, dq[d]);
            }
        }
    };
    over_keys(lo, hi, load, step);

    if (r0 < len) store_rows<kBlocks>(a.dq, tile.begin + r0, head, len - r0, a.head_dim, dq, a.scale);
    if (!dsink) return;
    pdp = sum_halves(pdp);
    float v = lane < 32 && row < len ? p0dp0 - p0 * pdp : 0.0f;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    if constexpr (kLayout == kRowsOfOne) {
        if (lane == 0) whole[wave] = v;
        __syncthreads();
        v = (whole[0] + whole[1]) + (whole[2] + whole[3]);
        if (wave > 0) return;
    }
    if (lane == 0) *dsink = v;
}

// dsink of a head: the partial sums of the dq kernel's tiles, in float64 and a
// fixed order; by workgroups of their own behind the dk, dv kernel's.
__device__ __forceinline__ void sum_dsink(const AttentionArgs &a, int head, double *lds) {
    const float *p = a.dsink_part + int64_t(head) * a.row_tiles;
    double v = 0.0;
    for (int i = threadIdx.x; i < a.row_tiles; i += kThreads) v += double(p[i]);
    lds[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int n = kThreads / 2; n > 0; n >>= 1) {
        if (int(threadIdx.x) < n) lds[threadIdx.x] += lds[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) a.dsink[head] = float(lds[0]);
}

// dk and dv of one tile of keys of one key head: the query heads of the group
// and the rows in the band, in a fixed order, into registers; or a slice of
// them, as float32 partial sums, where there are too few tiles for the CUs.
// The products' accumulators start from -lse / scale and -delta of their
// row, so that the exponent and dp - delta need no further operation.  Rows
// behind the chunk read as zeros, and a block that holds any is masked, so
// that their p is zero too, however large a sink makes it.
//
// Four products a pair: 32 heads of 64 over 8 of 4096 rows 1.98 ms, 1.11
// PFLOP/s.  No unit is full there (matrix cores 57% of the cycles, VALU 45%,
// LDS 43%): a wave's products, exponentials, packing and next products follow
// from each other, and three waves a SIMD do not cover that.  16 heads of 128
// over 2 of 4096 rows, both passes: 0.94 to 0.97 ms, 0.99 PFLOP/s, one wave a
// SIMD.  With a band of 64, 16 x 3520 rows: 221 us,
// 0.69 GB at 3.1 TB/s; its waves' keys see 160 of the 256 rows that the
// workgroup's do (32 keys a workgroup, which read the rows 2.5 times as often,
// gained nothing).
template <int kD, bool kBand>
__global__ __launch_bounds__(kThreads, kD == 128 ? 1 : kD == 64 ? 3 : 2) void attention_dkdv_kernel(AttentionArgs a) {
    constexpr int kSteps = kD / 16, kBlocks = kD / 32, kPanels = (kD + 63) / 64;
    // The chunk's end is masked in the logits, or, where the registers are
    // full anyway, in the probabilities, as the compiler allots them better
    // (8 of 4096 rows, 32 heads of 64: 2.00 ms against 2.04 with spills; both
    // passes over 2 of 4096, 16 heads of 128: 0.94 ms against 1.01).
    constexpr bool kMaskLast = kD == 128;
    __shared__ __attribute__((aligned(16))) uint8_t sq0[kPanels * kPanelBytes], sq1[kPanels * kPanelBytes];
    __shared__ __attribute__((aligned(16))) uint8_t sg0[kPanels * kPanelBytes], sg1[kPanels * kPanelBytes];
    __shared__ __attribute__((aligned(16))) float sl0[2][kStep], sl1[2][kStep];  // -lse / scale, -delta
    const uint32_t tiles = uint32_t(a.tiles) * uint32_t(a.kv_heads) * uint32_t(a.slices);
    if (blockIdx.x >= tiles) {
        sum_dsink(a, int(blockIdx.x - tiles), reinterpret_cast<double *>(sq0));
        return;
    }
    const uint32_t id = tile_of_xcd(blockIdx.x, tiles), pair = id / uint32_t(a.slices);
    const int slice = int(id - pair * uint32_t(a.slices)), kv = int(pair / uint32_t(a.tiles));
    const Tile tile = find_tile<kTileRows>(a.cu, a.chunks, a.rows, int(pair - uint32_t(kv) * uint32_t(a.tiles)));
    if (tile.len == 0) return;
    const int group = a.group;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int len = tile.len, window = kBand ? min(a.window, len) : -1;
    const int c0 = tile.first + wave * kWaveRows;  // this wave's keys
    const int key = c0 + (lane & 31);
    const Seen seen = seen_by(key, len, window);
    const LdsAddress at = lds_address();

    bf16x8 k[kSteps], v[kSteps];
    load_operand<kD>(a.k, tile.begin + c0, kv, len - c0, a.head_dim, k);
    load_operand<kD>(a.v, tile.begin + c0, kv, len - c0, a.head_dim, v);
    int lo, hi;
    band(tile.first, kTileRows, len, window, lo, hi);
    // steps of this slice, out of the group's heads' one after the other
    const int per_head = (hi - lo + kStep - 1) / kStep;
    const int64_t all_steps = int64_t(per_head) * group;
    const int64_t from = all_steps * slice / a.slices, end = all_steps * (slice + 1) / a.slices;
    const float c2 = a.scale * kLog2e;
    f32x16 dk[kBlocks], dv[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) dk[d] = dv[d] = f32x16{};

    const Loader<kPanels> lq(a.q, wave, a.head_dim), lg(a.dout, wave, a.head_dim);
    auto load = [&](int head, int q0, int n) __attribute__((always_inline)) {
        lq.load(head_rsrc(a.q, tile.begin + q0, head, len - q0, a.head_dim), wave, n ? sq1 : sq0);
        lg.load(head_rsrc(a.dout, tile.begin + q0, head, len - q0, a.head_dim), wave, n ? sg1 : sg0);
        if (wave < 2) {
            float *p = (wave ? a.neg_delta : a.neg_lse) + int64_t(head) * a.rows + tile.begin + q0;
            const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(p, 0, min(len - q0, kStep) * 4, kWord3);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_ptr)((n ? sl1 : sl0)[wave]), 4, lane * 4, 0, 0, 0);
        }
    };
    auto step = [&](int head, int q0, int n) __attribute__((always_inline)) {
        const uint8_t *tq = n ? sq1 : sq0, *tg = n ? sg1 : sg0;
        const float *tl = n ? sl1[0] : sl0[0], *td = n ? sl1[1] : sl0[1];
        if (c0 >= len) return;
        const float kb = a.sink && key == 0 ? head_sink(a.sink, head) * kLog2e : 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int rb = q0 + 32 * b;
            if (kBand && (rb >= len || !any_visible(c0, rb, 32, window))) continue;
            f32x16 s, dp;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int off = 32 * b + 8 * g + 4 * (lane >> 5);
                const f32x4 l = *reinterpret_cast<const f32x4 *>(tl + off);
                const f32x4 d = *reinterpret_cast<const f32x4 *>(td + off);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[4 * g + e] = l[e];
                    dp[4 * g + e] = d[e];
                }
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s = mfma(read_rows(tq, at, b, i), k[i], s);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) dp = mfma(read_rows(tg, at, b, i), v[i], dp);
            const bool masked = !all_visible(c0, rb, 32, len, window);
            if (kBand && masked) mask_band(seen, rb, s);
            if (!kBand && !kMaskLast && masked) mask_end(len, rb, -INFINITY, s);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c2, kb));
            if (!kBand && kMaskLast && masked) mask_end(len, rb, 0.0f, s);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bf16x8 p = pack(s, i);
#pragma unroll
                for (int d = 0; d < kBlocks; ++d) dv[d] = mfma(read_columns(tg, at, d, 2 * b + i), p, dv[d]);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] *= dp[r];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bf16x8 ds = pack(s, i);
#pragma unroll
                for (int d = 0; d < kBlocks; ++d) dk[d] = mfma(read_columns(tq, at, d, 2 * b + i), ds, dk[d]);
            }
        }
    };
    if (from < end) {
        int h = int(from / per_head), q0 = lo + int(from - int64_t(h) * per_head) * kStep;
        h += kv * group;
        int64_t left = end - from;
        auto next = [&](int &h, int &q0) __attribute__((always_inline)) {
            q0 += kStep;
            if (q0 >= hi) {
                q0 = lo;
                ++h;
            }
        };
        load(h, q0, 0);
        for (;;) {
            int h1 = h, q1 = q0;
            next(h1, q1);
            tiles_ready();
            if (left > 1) load(h1, q1, 1);
            step(h, q0, 0);
            if (left <= 1) break;
            h = h1;
            q0 = q1;
            next(h, q0);
            tiles_ready();
            if (left > 2) load(h, q0, 0);
            step(h1, q1, 1);
            left -= 2;
            if (left <= 0) break;
        }
    }
    if (c0 >= len) return;
    if (a.slices == 1) {
        store_rows<kBlocks>(a.dk, tile.begin + c0, kv, len - c0, a.head_dim, dk, a.scale);
        store_rows<kBlocks>(a.dv, tile.begin + c0, kv, len - c0, a.head_dim, dv, 1.0f);
        return;
    }
    const int last_lane = lane_again(), r = last_lane & 31;
    if (r >= len - c0) return;
    const int64_t plane = int64_t(a.kv_heads) * a.rows * a.head_dim;
    float *p = a.part + 2 * slice * plane + (int64_t(kv) * a.rows + tile.begin + c0) * a.head_dim + r * a.head_dim;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int col = d * 32 + 8 * g + 4 * (last_lane >> 5);
            if (col >= a.head_dim) continue;
            *reinterpret_cast<f32x4 *>(p + col) = f32x4{dk[d][4 * g], dk[d][4 * g + 1], dk[d][4 * g + 2], dk[d][4 * g + 3]};
            *reinterpret_cast<f32x4 *>(p + plane + col) = f32x4{dv[d][4 * g], dv[d][4 * g + 1], dv[d][4 * g + 2], dv[d][4 * g + 3]};
        }
}

// dk and dv from the slices' partial sums, added in order; four values a
// thread.  Rows of no chunk have no partial sums and are left as they are.
// The sums come from L2, and the launch is most of it: 8 slices of 1964 rows,
// 2 heads of 80: 6 us.
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttentionArgs a) {
    const int per_row = a.head_dim / 4;
    const int64_t n = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t line = n / per_row;  // of [kv_heads][rows]
    const int col = int(n - line * per_row) * 4;
    const int kv = int(line / a.rows);
    const int64_t row = line - int64_t(kv) * a.rows;
    if (kv >= a.kv_heads) return;
    // the row's chunk: the last one that starts at or before it (checked, as find_tile's is)
    int lo = 0, hi = a.chunks;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    if (row < a.cu[lo] || row >= a.cu[lo + 1] || a.cu[lo] < 0 || a.cu[lo + 1] > a.rows) return;
    const int64_t plane = int64_t(a.kv_heads) * a.rows * a.head_dim;
    const float *p = a.part + line * a.head_dim + col;
    f32x4 dk = {}, dv = {};
    for (int s = 0; s < a.slices; ++s, p += 2 * plane) {
        dk += *reinterpret_cast<const f32x4 *>(p);
        dv += *reinterpret_cast<const f32x4 *>(p + plane);
    }
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf16x4 *>(a.dk.p + row * a.dk.row + kv * a.dk.head + col) =
        bf16x4{__bf16(dk[0] * a.scale), __bf16(dk[1] * a.scale), __bf16(dk[2] * a.scale), __bf16(dk[3] * a.scale)};
    *reinterpret_cast<bf16x4 *>(a.dv.p + row * a.dv.row + kv * a.dv.head + col) =
        bf16x4{__bf16(dv[0]), __bf16(dv[1]), __bf16(dv[2]), __bf16(dv[3])};
}

// dsink without rows: zeros.
__global__ __launch_bounds__(kThreads) void attention_no_rows_kernel(AttentionArgs a) {
    if (threadIdx.x == 0) a.dsink[blockIdx.x] = 0.0f;
}

// Launch shapes, from sizes alone.
struct LaunchShape {
    Layout layout;    // of the kernels over query rows
    int32_t tiles, heads;  // their tiles, and heads (or groups of four) of the launch
    int32_t key_tiles, slices;  // of the dk, dv kernel
};
LaunchShape launch_shape(int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t chunks) {
    LaunchShape r;
    const int32_t group = q_heads / kv_heads;
    r.key_tiles = int32_t(rows / kTileRows + chunks);
    r.layout = group % 4 == 0 ? kHeadsOfFour : kRowsOfOne;
    r.tiles = r.layout == kRowsOfOne ? r.key_tiles : int32_t(std::min<int64_t>(rows / kWaveRows + chunks, 0x7FFFFFFF));
    r.heads = r.layout == kRowsOfOne ? q_heads : q_heads / 4;
    // dk's and dv's sums are split where there are fewer than two tiles a CU,
    // into at most eight slices of at least four steps of the longest chunk
    // there can be (16 heads on 8 of 4000 rows: two slices 268 us, one 298;
    // 32 heads of 216 rows: eight slices 30 us, four 24)
    const int64_t groups = std::max<int64_t>(int64_t(r.key_tiles) * kv_heads, 1);
    const int64_t steps = int64_t(group) * ((rows + kStep - 1) / kStep);
    r.slices = int32_t(std::max<int64_t>(1, std::min<int64_t>({8, (512 + groups - 1) / groups, steps / 4})));
    return r;
}

constexpr int64_t kMaxRows = int64_t(1) << 29;  // a row plus twice the window fits an int
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;
// A launch has fewer than 2^32 threads (groups of four heads take at most as
// many workgroups as 128 rows do; dsink takes one a head).
bool too_many_groups(int64_t rows, int32_t chunks, int32_t q_heads) {
    return (rows / kTileRows + chunks) * q_heads + q_heads > kMaxGroups;
}
constexpr int64_t kMaxRowStride = int64_t(1) << 22;  // a 64-row tile's byte offsets stay below 2^31

int check_heads(const mimo_heads &t, const char *who, const char *name, int64_t rows, int32_t heads, int32_t head_dim, bool written) {
    const auto at = [&] { return std::string(who) + ": " + name; };
    if (!t.data || !check_ptr_align(t.data, 16))
        return set_error(MIMO_E_INVALID, at() + " must be non-null and 16-byte aligned");
    if (t.row_stride % 8 || t.head_stride % 8 || t.row_stride < head_dim || t.head_stride < 0 ||
        t.row_stride > kMaxRowStride || t.head_stride > (int64_t(1) << 40))
        return set_error(MIMO_E_INVALID, at() + "'s strides must be multiples of 8 values, row_stride in [head_dim, 2^22], head_stride >= 0");
    if (!written) return MIMO_OK;
    const bool head_inside = heads == 1 || (t.head_stride >= head_dim && t.row_stride >= (heads - 1) * t.head_stride + head_dim);
    const bool row_inside = t.head_stride >= (rows - 1) * t.row_stride + head_dim;
    if (!head_inside && !row_inside) return set_error(MIMO_E_INVALID, at() + " is written, so its rows and heads must not overlap");
    return MIMO_OK;
}

// What forward and backward check alike; fills the kernels' arguments.
int check_attention(const mimo_attention *p, const char *who, AttentionArgs &a) {
    const auto w = [&] { return std::string(who); };
    if (!p) return set_error(MIMO_E_INVALID, w() + ": null arguments");
    if (p->rows < 0 || p->chunks < 0 || p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads || p->q_heads > 65536)
        return set_error(MIMO_E_INVALID, w() + ": rows and chunks must be >= 0, q_heads a multiple of kv_heads >= 1, at most 65536");
    if (p->head_dim < 8 || p->head_dim > MIMO_HEAD_DIM_MAX || p->head_dim % 8)
        return set_error(MIMO_E_INVALID, w() + ": head_dim must be a multiple of 8 in [8, 128]");
    if (!(p->scale >= 1e-18f && p->scale <= 1e18f)) return set_error(MIMO_E_INVALID, w() + ": scale must be in [1e-18, 1e18]");
    if (p->rows > kMaxRows || p->chunks > kMaxRows)
        return set_error(MIMO_E_TOO_LARGE, w() + ": more than 2^29 rows or chunks");
    std::memset(&a, 0, sizeof(a));
    a.rows = p->rows;
    a.q_heads = p->q_heads;
    a.kv_heads = p->kv_heads;
    a.group = p->q_heads / p->kv_heads;
    a.head_dim = p->head_dim;
    a.chunks = p->chunks;
    a.window = p->window < 0 ? -1 : p->window;
    a.scale = p->scale;
    if (p->rows == 0 || p->chunks == 0) return MIMO_OK;
    if (too_many_groups(p->rows, p->chunks, p->q_heads))
        return set_error(MIMO_E_TOO_LARGE, w() + ": (rows / 128 + chunks + 1) * q_heads is above 2^24 - 1");
    if (!p->cu_seqlens || !check_ptr_align(p->cu_seqlens, 4) || !check_ptr_align(p->sink, 4))
        return set_error(MIMO_E_INVALID, w() + ": cu_seqlens must be non-null; it and sink 4-byte aligned");
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

// The backward pass's workspace: -lse / scale and -delta of every row and
// head, the sink's partial sums of every tile, the slices' dk and dv.
struct Workspace {
    size_t stats, sums, part, total;
};
Workspace workspace_layout(const LaunchShape &l, int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    Workspace w;
    w.stats = align256(size_t(rows) * size_t(q_heads) * sizeof(float));
    w.sums = align256(size_t(l.tiles) * size_t(q_heads) * sizeof(float));
    w.part = l.slices == 1 ? 0 : align256(size_t(l.slices) * 2 * size_t(kv_heads) * size_t(rows) * size_t(head_dim) * sizeof(float));
    w.total = 2 * w.stats + w.sums + w.part;
    return w;
}

// The narrowest instance that holds head_dim: 64, 96 or 128 columns.  What it
// has beyond head_dim is multiplied as zeros: 32 heads on 8 over 8 of 4096 rows,
// forward, 32 columns 1.02 ms and 64 1.14; 72, 80 and 96 columns 1.6 to 1.7; 128
// 2.0 (backward 3.1 and 3.5; 4.8 to 5.1; 7.2).
template <int kD, bool kBand>
void launch_forward_as(const LaunchShape &l, const AttentionArgs &a, hipStream_t s) {
    const dim3 grid{unsigned(l.tiles) * unsigned(l.heads), 1, 1}, block{unsigned(kThreads), 1, 1};
    if (l.layout == kRowsOfOne)
        hipLaunchKernelGGL((attention_forward_kernel<kD, kRowsOfOne, kBand>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((attention_forward_kernel<kD, kHeadsOfFour, kBand>), grid, block, 0, s, a);
}

template <int kD>
void launch_forward(const LaunchShape &l, const AttentionArgs &a, hipStream_t s) {
    if (a.window < 0)
        launch_forward_as<kD, false>(l, a, s);
    else
        launch_forward_as<kD, true>(l, a, s);
}

template <int kD, bool kBand>
void launch_backward_as(const LaunchShape &l, const AttentionArgs &a, const AttentionArgs &b, hipStream_t s) {
    const dim3 grid{unsigned(l.tiles) * unsigned(l.heads), 1, 1}, block{unsigned(kThreads), 1, 1};
    const dim3 keys{unsigned(b.tiles) * unsigned(b.kv_heads) * unsigned(b.slices) + unsigned(b.dsink ? b.q_heads : 0), 1, 1};
    if (l.layout == kRowsOfOne)
        hipLaunchKernelGGL((attention_dq_kernel<kD, kRowsOfOne, kBand>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((attention_dq_kernel<kD, kHeadsOfFour, kBand>), grid, block, 0, s, a);
    hipLaunchKernelGGL((attention_dkdv_kernel<kD, kBand>), keys, block, 0, s, b);
}

template <int kD>
void launch_backward(const LaunchShape &l, const AttentionArgs &a, const AttentionArgs &b, hipStream_t s) {
    if (a.window < 0)
        launch_backward_as<kD, false>(l, a, b, s);
    else
        launch_backward_as<kD, true>(l, a, b, s);
}

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
    const LaunchShape l = launch_shape(a.rows, a.q_heads, a.kv_heads, a.chunks);
    a.tiles = l.tiles;
    const hipError_t e = timed_launch(s, [&] {
        if (a.head_dim <= 64)
            launch_forward<64>(l, a, s);
        else if (a.head_dim <= 96)
            launch_forward<96>(l, a, s);
        else
            launch_forward<128>(l, a, s);
    });
    if (e != hipSuccess) return hip_error(e, "chunk_attention: kernel launch");
    g_dispatches.fetch_add(1);
    return MIMO_OK;
}

size_t mimo_chunk_attention_workspace_bytes(int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t chunks) {
    if (rows < 0 || rows > kMaxRows || chunks < 0 || chunks > kMaxRows || kv_heads < 1 || q_heads < kv_heads ||
        q_heads % kv_heads || q_heads > 65536 || head_dim < 8 || head_dim > MIMO_HEAD_DIM_MAX || head_dim % 8)
        return 0;
    if (rows == 0 || chunks == 0 || too_many_groups(rows, chunks, q_heads)) return 0;
    return workspace_layout(launch_shape(rows, q_heads, kv_heads, chunks), rows, q_heads, kv_heads, head_dim).total;
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
    if (g->dsink && g->dsink == p->sink) return set_error(MIMO_E_INVALID, std::string(who) + ": dsink must not be sink");
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
    const bool work = a.rows && a.chunks;
    LaunchShape l = launch_shape(a.rows, a.q_heads, a.kv_heads, a.chunks);
    if (!work) l.tiles = l.key_tiles = 0;
    const Workspace w = workspace_layout(l, a.rows, a.q_heads, a.kv_heads, a.head_dim);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (work) {
        a.neg_lse = reinterpret_cast<float *>(ws);
        a.neg_delta = reinterpret_cast<float *>(ws + w.stats);
        if (g->dsink) a.dsink_part = reinterpret_cast<float *>(ws + 2 * w.stats);
        if (l.slices > 1) a.part = reinterpret_cast<float *>(ws + 2 * w.stats + w.sums);
    }
    a.dsink = g->dsink;
    a.row_tiles = l.tiles;
    a.slices = l.slices;
    a.tiles = l.tiles;
    AttentionArgs b = a;  // of the dk, dv kernel
    b.tiles = l.key_tiles;
    const int64_t join = (int64_t(a.kv_heads) * a.rows * (a.head_dim / 4) + kThreads - 1) / kThreads;
    const dim3 block{unsigned(kThreads), 1, 1}, sink_grid{unsigned(a.q_heads), 1, 1}, join_grid{unsigned(join), 1, 1};
    const hipError_t e = timed_launch(s, [&] {
        if (work && a.head_dim <= 64)
            launch_backward<64>(l, a, b, s);
        else if (work && a.head_dim <= 96)
            launch_backward<96>(l, a, b, s);
        else if (work)
            launch_backward<128>(l, a, b, s);
        if (work && l.slices > 1) hipLaunchKernelGGL(attention_join_kernel, join_grid, block, 0, s, b);
        if (!work) hipLaunchKernelGGL(attention_no_rows_kernel, sink_grid, block, 0, s, a);
    });
    if (e != hipSuccess) return hip_error(e, "chunk_attention_backward: kernel launch");
    g_dispatches.fetch_add(work ? (l.slices > 1 ? 3 : 2) : 1);
    return MIMO_OK;
}

}  // extern "C"
