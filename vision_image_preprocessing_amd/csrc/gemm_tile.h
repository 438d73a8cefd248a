// gemm_tile.h -- one tile of a bf16 matrix product on the matrix cores of AMD
// Instinct MI355X (gfx950, CDNA4), for operands in either order in memory:
//   sum over k of X[m][k] W[n][k]
// where a matrix is stored along k ([rows][k], the summed axis innermost) or
// across it ([k][rows]).  Forward products are along, along; a gradient of the
// input is along, across; a gradient of a weight, whose summed axis is the
// rows of both operands, is across, across.
//
// A workgroup makes a kTile x kTile tile: 256 x 256 (eight waves of 128 x 64, 128
// accumulators a lane, one workgroup a CU), 128 x 128 (four of 64 x 64, two
// workgroups a CU) or 64 x 64 (four of 32 x 32, three workgroups a CU).  K
// advances 64 values a stage.  Operands go from memory straight into LDS
// (buffer_load ... lds), two stages ahead of the products; x has three buffers,
// w two, which are filled again as soon as they are read.  In a tile of 64 x 64,
// whose stages are short, w has three, too, and its loads another stage's time
// (33 rows of 1280, hidden 5120, 21.8 to 18.2 us; 216 rows of 2048, hidden 2048, 26.6
// to 21.5; the fourth workgroup that a CU then has no room for gave less).  The
// buffers are arrays of their own, so that the compiler sees that loads into
// one never meet reads of another, and the stage loop is unrolled six times,
// after which both rings are back where they were.  Stages past the end are loaded through an
// empty resource: zeros, without memory traffic.
//
// 256 x 256, K 5120: 131072 x 1280 in 1.25 to 1.31 ms, 1.31 to 1.37 PFLOP/s, next
// to 1.43 of a large library product; a stage takes 1.5 us, a tile's first
// loads and its store about 8.  The card's power bounds that (the clock falls
// to 1.6 to 1.7 GHz; on zeros 1.2 ms), and at smaller sizes what a CU takes in,
// some 60 GB/s.  Four waves of 128 x 128 took 2 to 7% longer, all of a stage's
// loads in its first half 4%, all of a step's reads at once 2%, and tiles in
// runs of eight rows up to 6%; raised wave priority, tiles turned in two
// regions and workgroups that start staggered made no difference.
//
// In LDS a matrix stored along k lies as kTile rows of 64 values, read 16
// bytes a lane; one stored across as panels of 64 columns, 64 rows of k each,
// read by ds_read_b64_tr_b16, which hands a lane four rows of one column.
// Either way lane l of an operand holds row l % 32, k = 8 (l / 32) .. + 7 of
// the 16 that a product takes.  16-byte chunks are XOR-swizzled by the row so
// that neither kind of read meets a bank twice.
//
// Products are v_mfma_f32_32x32x16_bf16 with w as the first operand: a lane of
// the result holds one row of x (lane % 32) and channels 8 (r / 4) + 4 (lane /
// 32) + r % 4, so that it can stage and store neighbouring channels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "device_util.h"

namespace mimo {
namespace gemm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4_ptr;
typedef __attribute__((address_space(3))) bf16x8 *lds_bf16x8_ptr;
typedef __attribute__((address_space(3))) f32x4 *lds_f32x4_ptr;
typedef __attribute__((address_space(3))) uint8_t *lds_ptr;

constexpr int kStageK = 64;
constexpr int kWord3 = 0x00020000;          // raw buffer resource word 3
constexpr int kRecords = 0x7FFFFFF0;        // the largest size of a resource
constexpr uint32_t kOutside = 0x7FFFFFF8u;  // a byte offset past every resource: reads zeros
constexpr int kWaitAll = 0;                 // s_waitcnt: every counter at zero
constexpr int kGroupM = 4;                  // tiles of rows that share a run of channel tiles

// One bf16 matrix; stride in values, a multiple of 8, as is the innermost
// axis; 16-byte aligned.
struct Matrix {
    const uint16_t *p;
    int64_t stride;
};

// One product of a launch; k is that of one pair of matrices.
struct Product {
    Matrix x[2], w[2];
    int64_t m;
    int32_t n, k;
    int32_t stages;       // of all of K
    int32_t m_tiles, n_tiles;
    int32_t first;        // of its tiles in the launch
};

// How a launch's tiles are worked on: the first `full` by a workgroup each, the
// `tail` behind them by `splits` each, over as many parts of K.  Each of the
// two ranges goes to the XCDs in contiguous runs.
struct Units {
    int32_t full, tail, splits;
    __host__ __device__ int32_t count() const { return full + tail * splits; }
};
struct Unit {
    int tile, split, slot;  // split < 0: all of K; else the part's place in the workspace
    __device__ __forceinline__ explicit Unit(const Units &u) {
        const int b = int(blockIdx.x);
        if (b < u.full) {
            tile = int(xcd_contiguous_tile(b, u.full));
            split = slot = -1;
        } else {
            slot = int(xcd_contiguous_tile(b - u.full, u.tail * u.splits));
            split = slot / u.tail;
            tile = u.full + slot - split * u.tail;
        }
    }
};

// How a tile is cut among its waves: two along the rows, the others along the
// channels, each kWaveM x kWaveN in blocks of 32 x 32.
template <int kTile_>
struct Tile {
    static constexpr int kTile = kTile_;
    static constexpr int kWaves = kTile == 256 ? 8 : 4;
    static constexpr int kThreads = kWaves * 64, kWavesN = kWaves / 2;
    static constexpr int kWaveM = kTile / 2, kWaveN = kTile / kWavesN;
    static constexpr int kBlocksM = kWaveM / 32, kBlocksN = kWaveN / 32;
    static constexpr int kGroups = kTile / 8 / kWaves;  // 1 KB loads a wave makes of each operand a stage
    static constexpr int kWBuffers = kTile == 64 ? 3 : 2;
};
template <int kTile>
using Sums = f32x16[Tile<kTile>::kBlocksM][Tile<kTile>::kBlocksN];

__device__ __forceinline__ int row_key(int r) { return (r & 1) | ((r & 2) << 1) | ((r & 4) >> 1); }
__device__ __forceinline__ int block_key(int g) { return g ^ ((g & 3) >> 1); }

__device__ __forceinline__ f32x16 mfma(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Where a tile is.  Runs of kGroupM tiles of rows
// go by channels together, so that the tiles an XCD works on at one time share
// rows and channels in its L2 (a run of one row of tiles reads every channel).
struct Place {
    int64_t mt;
    int nt;
    __device__ __forceinline__ Place(const Product &p, int t) {
        const int group = t / (kGroupM * p.n_tiles), first = group * kGroupM;
        const int rows = min(p.m_tiles - first, kGroupM);
        t -= first * p.n_tiles;
        nt = t / rows;
        mt = first + t - nt * rows;
    }
};

// The tile's buffers.  Every address in them is one of these plus a lane's
// offset and a constant: through longer chains the compiler no longer sees
// which array a read is of, and waits for all loads in flight.  160 KB with
// 256, one workgroup a CU; 80 KB with 128, two; 48 KB with 64, three.
template <int kTile>
struct Buffers {
    lds_ptr x[3], w[Tile<kTile>::kWBuffers];
};
template <int kTile>
__device__ __forceinline__ Buffers<kTile> tile_buffers() {
    __shared__ __attribute__((aligned(16))) uint8_t x0[kTile * 128], x1[kTile * 128], x2[kTile * 128], w0[kTile * 128], w1[kTile * 128];
    Buffers<kTile> b{{(lds_ptr)x0, (lds_ptr)x1, (lds_ptr)x2}, {(lds_ptr)w0, (lds_ptr)w1}};
    if constexpr (Tile<kTile>::kWBuffers == 3) {
        __shared__ __attribute__((aligned(16))) uint8_t w2[kTile * 128];
        b.w[2] = (lds_ptr)w2;
    }
    return b;
}

// One operand's loads by a wave, kGroups of 1 KB a stage, and its operands.
// kAcross: stored across k.  kTile rows (columns, if across) from `first` on, of
// `count`.
template <int kTile, bool kAcross>
struct Operand {
    static constexpr int kGroups = Tile<kTile>::kGroups;
    uint32_t off[kGroups];
    int chunk;  // along: the first group's chunk of the lane's row; group i's is chunk ^ i
    int base;   // the lane's part of an operand read's address
    int wave;

    // Group i of wave w is number n = w * kGroups + i: along, rows 8 n .. + 7;
    // across, rows 8 (n % 8) .. + 7 of k in panel n / 8.  Lane l lands at row l /
    // 8, chunk l % 8 of it, so it fetches the chunk that the swizzle puts there.
    // `rows_from`: what row of the matrix the wave's first row of the tile is
    // (along); rows past the last one read as zeros (of the last one's values,
    // an infinity would be multiplied by zeros of what is saved of no row).
    // `at`: the first row (column) of the tile that the wave's operands are of.
    __device__ __forceinline__ Operand(int64_t stride, int64_t first, int64_t count, int64_t rows_from, int at) {
        const int lane = threadIdx.x & 63, l8 = lane >> 3;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if constexpr (kAcross) {
            chunk = 0;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int n = wave * kGroups + i, g = n % 8;
                const int col = (n / 8) * 64 + (((lane & 7) ^ row_key(l8) ^ block_key(g)) << 3);
                off[i] = first + col < count ? uint32_t((8 * g + l8) * int(stride) + col) * 2 : kOutside;
            }
            const int x = 8 * (lane >> 5) + ((lane & 15) >> 2), c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
            // row x of the 16 of a step, whose block of eight is 2 s + lane / 32:
            // block_key of it is (lane / 32) ^ the step's own part
            base = at / 64 * (kStageK * 128) + x * 128 + ((c ^ (4 * (at / 32 & 1)) ^ row_key(x & 7) ^ (lane >> 5)) << 4) + (lane & 1) * 8;
        } else {
            const int r = lane & 31;
            base = (at + r) * 128 + (((lane >> 5) ^ ((r ^ ((at + r) >> 3)) & 7)) << 4);
            chunk = ((lane & 7) ^ l8 ^ (wave * kGroups)) & 7;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int64_t row = rows_from + i * 8 + l8;
                off[i] = row < count ? uint32_t(int(row - first) * int(stride) + ((chunk ^ i) & 7) * 8) * 2 : kOutside;
            }
        }
    }

    // Group i of stage ks of a segment of k values, from the tile's base (row
    // `first`, or column `first`, of the matrix).
    __device__ __forceinline__ void load(const Matrix &t, int64_t first, int64_t count, int i, int ks, int k, bool live, lds_ptr d) const {
        const lds_ptr to = d + (wave * kGroups + i) * 1024;
        const int left = k - ks * kStageK;  // values of k from the stage on
        if constexpr (kAcross) {
            // its rows of the stage to the end of the last one's last chunk (a
            // size that cuts a word would cut the value in its lower half too);
            // 32 bits hold them, and no branch is needed
            const int bytes = ((min(left, kStageK) - 1) * int(t.stride) + int(((count + 7) & ~int64_t(7)) - first)) * 2;
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint16_t *>(t.p) + int64_t(ks) * kStageK * t.stride + first, 0, live && left > 0 ? bytes : 0, kWord3);
            send(r, to, off[i], 0);
        } else {
            const __amdgpu_buffer_rsrc_t r =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(t.p) + first * t.stride, 0, live ? kRecords : 0, kWord3);
            send(r, to, ((chunk ^ i) & 7) * 8 < left ? off[i] : kOutside, live ? ks * (kStageK * 2) : 0);
        }
    }
    // The host's pass over this file does not know the size (and would drop
    // every kernel that contains it), so it does not see the call.
    static __device__ __forceinline__ void send(const __amdgpu_buffer_rsrc_t &r, lds_ptr to, uint32_t off, int at) {
#if defined(__HIP_DEVICE_COMPILE__)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, off, at, 0, 0);
#endif
    }

    // Rows (columns) 32 i .. + 31 of the wave's, step s of the stage.
    __device__ __forceinline__ bf16x8 read(lds_ptr t, int i, int s) const {
        if constexpr (kAcross) {
            const int flip = ((4 * (i & 1)) ^ (2 * s) ^ (s & 1)) << 4, at = (i / 2) * (kStageK * 128) + s * 16 * 128;
            union {
                s16x4 h[2];
                bf16x8 f;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(t + ((base ^ flip) + at)));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(t + ((base ^ flip ^ (2 << 4)) + (at + 4 * 128))));
            return u.f;
        } else {
            return *(lds_bf16x8_ptr)(t + ((base ^ (((2 * s) ^ (4 * (i & 1))) << 4)) + i * 32 * 128));
        }
    }
};

// The sums of stages [begin, end) of a tile into acc ([blocks of rows][blocks
// of channels]); every load has landed and every wave has read its operands
// when it returns.
//
// kOver: what K runs over.  kOnce: the first pair of matrices; kTwice: both
// pairs, one after the other; kGateUp: the first x, with w the gate's rows and
// the up projection's.
enum Over { kOnce, kTwice, kGateUp };
template <int kTile, bool kXAcross, bool kWAcross, Over kOver>
__device__ __forceinline__ void multiply(const Product &p, int64_t m0, int n0, int begin, int end, const Buffers<kTile> &lds,
                                         Sums<kTile> &acc) {
    constexpr bool kGate = kOver == kGateUp;
    static_assert(!(kGate && kWAcross), "gate and up are stored along k");
    typedef Operand<kTile, kXAcross> X;
    typedef Operand<kTile, kWAcross> W;
    typedef Tile<kTile> T;
    constexpr int kM = T::kBlocksM, kN = T::kBlocksN, kGroups = T::kGroups, kSteps = 4;
    // Loads go out one after each row of products: first w's of two stages on,
    // from the last step on, when their buffer is free, then x's.  kEarly of
    // w's are sent before the next stage begins.  With three buffers of each
    // (kDeep) x's, of three stages on, are the first, then w's.
    constexpr int kEarly = kGroups < kM ? kGroups : kM;
    constexpr bool kDeep = T::kWBuffers == 3;
    static_assert(kGroups <= 15 && 2 * kGroups <= kSteps * kM, "a stage's loads fit its rows of products");
    // vmcnt (bits 3:0 and 15:14) and lgkmcnt: one stage of x (kDeep: of both) and
    // the early loads may stay in flight; that without these, and lgkmcnt(0)
    constexpr int kStageFlight = kDeep ? 2 * kGroups : kGroups, kFlight = kStageFlight + kEarly;
    constexpr int kWaitFirst = 0x0F70 | (kFlight & 15) | (kFlight >> 4 << 14);
    constexpr int kWaitStage = 0x0070 | kStageFlight;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::kWavesN, wn = wave % T::kWavesN;
    const int seg = (p.k + kStageK - 1) / kStageK;  // stages of a segment
    const X x(p.x[0].stride, m0, p.m, m0 + wave * (kGroups * 8), wm * T::kWaveM);
    // of a wave's channels the first half is gate's and the second up's, of the
    // same rows of the two weights; so the rows that a wave loads are of one of
    // them, gate's in even ones
    static_assert(!kGate || kGroups * 8 == T::kWaveN / 2, "a wave loads rows of one of the two");
    // (a tile may lie in the padding, past every row)
    const int w_first = kGate ? min(n0, p.n - 1) : n0;
    const W w(p.w[0].stride, w_first, p.n, kGate ? n0 + (wave >> 1) * (kGroups * 8) : n0 + wave * (kGroups * 8), wn * T::kWaveN);
    // in registers from here on: a scalar load in the loop would make every
    // wait for LDS a wait for all of it
    const Matrix x0 = p.x[0], w0 = kGate ? p.w[wave & 1] : p.w[0];
    const Matrix x1 = kOver == kTwice ? p.x[1] : x0, w1 = kOver == kTwice ? p.w[1] : w0;
    const int64_t rows = p.m;
    const int channels = p.n, k = p.k;
    auto load_x = [&](int i, int s, lds_ptr d) {
        const bool second = kOver == kTwice && s >= seg;
        x.load(second ? x1 : x0, m0, rows, i, second ? s - seg : s, k, s < end, d);
    };
    auto load_w = [&](int i, int s, lds_ptr d) {
        const bool second = kOver == kTwice && s >= seg;
        w.load(second ? w1 : w0, w_first, channels, i, second ? s - seg : s, k, s < end, d);
    };
    // between stages: each wave has waited for its own loads and reads
    auto barrier = [] {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) acc[i][j] = f32x16{};
    bf16x8 fx[2][kM], fw[2][kN];
    // operand n of a step, w's first
    auto read = [&](lds_ptr tx, lds_ptr tw, int s, int n, bf16x8 (&a)[kM], bf16x8 (&b)[kN]) __attribute__((always_inline)) {
        if (n < kN)
            b[n] = w.read(tw, n, s);
        else if (n < kN + kM)
            a[n - kN] = x.read(tx, n - kN, s);
    };
#pragma unroll
    for (int i = 0; i < kGroups; ++i) load_x(i, begin, lds.x[0]);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) load_w(i, begin, lds.w[0]);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) load_x(i, begin + 1, lds.x[1]);
#pragma unroll
    for (int i = 0; i < (kDeep ? kGroups : kEarly); ++i) load_w(i, begin + 1, lds.w[1]);
    if constexpr (kDeep) {
#pragma unroll
        for (int i = 0; i < kEarly; ++i) load_x(i, begin + 2, lds.x[2]);
    }
    __builtin_amdgcn_s_waitcnt(kWaitFirst);
    barrier();
#pragma unroll
    for (int n = 0; n < kM + kN; ++n) read(lds.x[0], lds.w[0], 0, n, fx[0], fw[0]);
    __builtin_amdgcn_sched_barrier(0);
    // One stage.  The next step's operands are read between this one's rows of
    // products, three at a time (all at once, by every wave, keep LDS busy for
    // half a step and hold the products at issue).  Before the last step's
    // products, whose operands are in registers, the waves meet, and read the
    // next stage's first operands between them.
    auto stage = [&](int s, lds_ptr tx, lds_ptr tw, lds_ptr nw, lds_ptr nx2, lds_ptr nx, lds_ptr nw2) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
            if (ks + 1 == kSteps) {
                __builtin_amdgcn_s_waitcnt(kWaitStage);
                barrier();
            }
#pragma unroll
            for (int i = 0; i < kM; ++i) {
#pragma unroll
                for (int n = 3 * i; n < 3 * i + 3; ++n) {
                    if (ks + 1 < kSteps)
                        read(tx, tw, ks + 1, n, fx[(ks + 1) & 1], fw[(ks + 1) & 1]);
                    else
                        read(nx, nw, 0, n, fx[0], fw[0]);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < kN; ++j) acc[i][j] = mfma(fw[ks & 1][j], fx[ks & 1][i], acc[i][j]);
                const int q = (ks + 1) % kSteps * kM + i;
                if constexpr (kDeep) {
                    if (q < kGroups)
                        load_x(q, ks + 1 == kSteps ? s + 3 : s + 2, ks + 1 == kSteps ? tx : nx2);
                    else if (q < 2 * kGroups)
                        load_w(q - kGroups, s + 2, nw2);
                } else {
                    if (q < kGroups)
                        load_w(q, ks + 1 == kSteps ? s + 2 : s + 1, ks + 1 == kSteps ? tw : nw);
                    else if (q < 2 * kGroups)
                        load_x(q - kGroups, s + 2, nx2);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // stage u of a group of six
    auto ring = [&](int s, auto number) __attribute__((always_inline)) {
        constexpr int u = decltype(number)::value, kW = T::kWBuffers;
        stage(s, lds.x[u % 3], lds.w[u % kW], lds.w[(u + 1) % kW], lds.x[(u + 2) % 3], lds.x[(u + 1) % 3], lds.w[(u + 2) % kW]);
    };
    typedef std::integral_constant<int, 0> U0;
    typedef std::integral_constant<int, 1> U1;
    typedef std::integral_constant<int, 2> U2;
    typedef std::integral_constant<int, 3> U3;
    typedef std::integral_constant<int, 4> U4;
    typedef std::integral_constant<int, 5> U5;
    int s = begin;
    for (; s + 6 <= end; s += 6) {
        ring(s, U0());
        ring(s + 1, U1());
        ring(s + 2, U2());
        ring(s + 3, U3());
        ring(s + 4, U4());
        ring(s + 5, U5());
    }
    // the rest, nested: where two paths met, the compiler could not tell which
    // loads are in flight and would wait for all of them before the next read
    const int rest = end - s;
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
}

// A wave's block of 32 rows and its channels, turned in LDS (float32, 16-byte
// chunks XOR-swizzled by the row): a lane then reads whole pieces of rows.
template <int kTile>
struct Turned {
    typedef Tile<kTile> T;
    static constexpr int kRowBytes = T::kWaveN * 4, kChunks = kRowBytes / 16;
    lds_ptr region;
    __device__ __forceinline__ explicit Turned(const Buffers<kTile> &lds) {
        constexpr int kHalf = T::kWaves / 2;
        static_assert(kHalf * 32 * kRowBytes <= kTile * 128, "half the waves share a buffer");
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        region = (wave < kHalf ? lds.x[0] : lds.x[1]) + (wave % kHalf) * (32 * kRowBytes);
    }
    __device__ __forceinline__ void put(const f32x16 (&acc)[T::kBlocksN]) const {
        const int lane = threadIdx.x & 63, r = lane & 31;
#pragma unroll
        for (int j = 0; j < T::kBlocksN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = j * 8 + 2 * g + (lane >> 5);
                const f32x4 v = {acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
                *(lds_f32x4_ptr)(region + r * kRowBytes + ((c ^ r) % kChunks) * 16) = v;
            }
    }
    // kN channels from c0 on (multiples of 4) of row r.
    template <int kN>
    __device__ __forceinline__ void get(int r, int c0, float (&v)[kN]) const {
#pragma unroll
        for (int k = 0; k < kN / 4; ++k) {
            const f32x4 w = *(lds_f32x4_ptr)(region + r * kRowBytes + (((c0 / 4 + k) ^ r) % kChunks) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * k + j] = w[j];
        }
    }
};

}  // namespace gemm
}  // namespace mimo
