// gemm_core.cuh -- what the grouped products on the tensor cores are built from: stages and
// tiles, the loops of the loading and the multiplying warp, what the draining warps do with
// finished tiles, and the host's tensor maps and launches.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "gsa.h"
#include "moe/status.cuh"
#include "tc.cuh"

namespace {

constexpr int kMaxE = 256;
constexpr int kRowsT = 128;          // rows of a tile: the lanes of tensor memory
constexpr int kStageK = 128;         // bytes of k per stage: one 128-byte swizzled row
constexpr int kScaleTile = 512;      // bytes of one 128 x 4 scale tile
constexpr int kThreads = 384;        // warp 0 loads, warp 1 multiplies, warps 4-11 drain
constexpr int kMaxThreads = 576;     // of the kernels that share the split's scan
constexpr int kEpiWarps = 8, kDrain = 4;   // the draining warps, the first of them
constexpr int kBoxA = 32;            // rows of A that single blocks load at a time
constexpr int kOutBuf = 32 * 128;    // a draining warp's piece of results: 32 rows x 128 bytes
constexpr int kStatic = 4096;        // what the blocks' static shared memory stays below

using gemm_status::ERR_SPLIT;
using gemm_status::ERR_TIMEOUT;

struct GemmParams {
    CUtensorMap tm_a, tm_b, tm_sa, tm_sb;
    const int64_t *split;
    const float *amax_a, *amax_b;
    void *out;
    int64_t M;             // rows of A and out
    int64_t N;
    int kt;                // stages of k per tile
    int k_bytes;           // bytes of k per row
    int E;
    int n_tiles;           // column tiles
    int b_scale_rows;      // scale tiles along N per expert
    int scale_cols;        // scale tiles along k
    int64_t a_scale_tiles; // row tiles that A's scale buffer holds
};

template <bool NV> struct Fmt;
template <> struct Fmt<false> { static constexpr int kScaleTiles = 1; };   // scale tiles per stage and 128 rows
template <> struct Fmt<true> { static constexpr int kScaleTiles = 4; };

// A block's tile is 128 rows (its lanes of tensor memory) x BN columns.  kPair: two
// blocks of a cluster share a tile of 256 rows; each brings its own rows and half
// of the columns' operand, and the pair's products read both halves.
// kOut: bytes of the draining warps' buffers.
template <bool NV, int BN, bool kPair, int kOut = kEpiWarps * kOutBuf> struct Cfg {
    static constexpr int kSc = Fmt<NV>::kScaleTiles;
    static constexpr int kRowsB = kPair ? BN / 2 : BN;
    static constexpr int kBytesA = kRowsT * kStageK, kBytesB = kRowsB * kStageK;
    static constexpr int kGroupsB = BN / 128;
    static constexpr int kBytesSA = kSc * kScaleTile, kBytesSB = kGroupsB * kSc * kScaleTile;
    static constexpr int kStageBytes = kBytesA + kBytesB + kBytesSA + kBytesSB;
    static constexpr int kStride = (kStageBytes + 1023) / 1024 * 1024;   // stages start on the swizzle's period
    static constexpr int kAcc = BN == 256 ? 1 : 2;       // accumulators in tensor memory
    static constexpr int kScCols = 4 * kSc * (1 + kGroupsB);   // scale columns of a stage
    static constexpr int kCols = 512;
    static constexpr int kBySmem = (227 * 1024 - kStatic - 1024 - kOut) / kStride, kByCols = (kCols - kAcc * BN) / kScCols;
    static constexpr int kFit = kBySmem < kByCols ? kBySmem : kByCols;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kSmem = kStages * kStride + kOut + 1024;
};

struct Barriers {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2];
    uint32_t tmem, dead;
};

struct GemmShared : Barriers {
    int row0[kMaxE + 2];        // first row of each group; group E: rows that no expert has
    int tile0[kMaxE + 2];       // first row tile of each group
    int scale0[kMaxE + 1];      // first 128-row scale tile of each expert
    int64_t scan[kMaxThreads / 32][3];
    uint32_t bad;
};

// A value that is the same in all lanes, as the compiler cannot tell.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Group bounds from the device split: rows, scale tiles and row tiles of kRows before each group.  Every thread
// of the block.  A negative size, a sum above M or more scale tiles than A's buffer holds sets sh.bad.  kTimes: rows of A for
// each that the split counts.  Without a split the one group has all rows.
template <int kRows, int kTimes = 1> __device__ void scan_split(const GemmParams &P, GemmShared &sh) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? (P.split ? P.split[t] : P.M / kTimes) : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
    m *= kTimes;
    int64_t rows = m, scales = (m + 127) / 128, tiles = (m + kRows - 1) / kRows;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, d), q = __shfl_up_sync(0xFFFFFFFFu, scales, d),
                      u = __shfl_up_sync(0xFFFFFFFFu, tiles, d);
        if (lane >= d) rows += r, scales += q, tiles += u;
    }
    if (lane == 31) sh.scan[w][0] = rows, sh.scan[w][1] = scales, sh.scan[w][2] = tiles;
    const bool any_neg = __syncthreads_or(neg);
    for (int k = 0; k < w; ++k) rows += sh.scan[k][0], scales += sh.scan[k][1], tiles += sh.scan[k][2];
    if (t < P.E) {
        sh.row0[t + 1] = static_cast<int>(rows);
        sh.scale0[t + 1] = static_cast<int>(scales);
        sh.tile0[t + 1] = static_cast<int>(tiles);
    }
    if (t == 0) sh.row0[0] = 0, sh.scale0[0] = 0, sh.tile0[0] = 0;
    if (t == P.E - 1) {
        sh.bad = any_neg || rows > P.M || scales > P.a_scale_tiles;
        sh.row0[P.E + 1] = static_cast<int>(P.M);
        sh.tile0[P.E + 1] = static_cast<int>(tiles + (P.M - (rows > P.M ? P.M : rows) + kRows - 1) / kRows);
    }
    __syncthreads();
}

// Encode scale of the quantizer: 2688 / amax (1 for amax 0), capped at FLT_MAX.
__device__ __forceinline__ float tensor_scale(float amax) {
    if (amax == 0.0f) return 1.0f;
    const float s = __fdiv_rn(2688.0f, amax);
    return s <= 3.402823466e38f ? s : 3.402823466e38f;
}

struct Tile {
    int g;          // group
    int row;        // first row
    int rows;       // rows of the tile that belong to the group
    int mt;         // row tile within the group
    int nt;         // column tile
};

// Tile number i of kRows rows, searching from group g on (tile numbers only grow).
template <int kRows> __device__ __forceinline__ Tile tile_at(const GemmParams &P, const GemmShared &sh, int64_t i, int g) {
    const int q = static_cast<int>(i / P.n_tiles);
    for (int end = P.E + 1; end - g > 1;) {   // the last group that starts at or before q: most may be empty
        const int mid = (g + end) >> 1;
        if (sh.tile0[mid] <= q) g = mid;
        else end = mid;
    }
    Tile t;
    t.g = g;
    t.nt = static_cast<int>(i - static_cast<int64_t>(q) * P.n_tiles);
    t.mt = q - sh.tile0[g];
    t.row = sh.row0[g] + t.mt * kRows;
    t.rows = min(kRows, sh.row0[g + 1] - t.row);
    return t;
}

// The same value of all lanes as one that the compiler knows to be the same: it then lives in a uniform register, of which
// the draining warps have plenty, while their accumulators leave them few others.
__device__ __forceinline__ int known_uniform(int v) { return __reduce_min_sync(0xFFFFFFFFu, v); }

// The tiles of a unit, without divisions: q counts row tiles over all groups (n_tiles column tiles each, one after another).
struct Walk {
    int q, nt, g, dq, dn;
    __device__ __forceinline__ Walk(const GemmParams &P, int unit, int units)
        : q(unit / P.n_tiles), nt(unit % P.n_tiles), g(0), dq(units / P.n_tiles), dn(units % P.n_tiles) {}
    __device__ __forceinline__ void next(const GemmParams &P) {
        q += dq, nt += dn;
        if (nt >= P.n_tiles) nt -= P.n_tiles, ++q;
    }
    // Its tile, by a whole warp; the group that q is in is this one or a later one.
    template <int kRows> __device__ __forceinline__ Tile tile(const GemmParams &P, const GemmShared &sh) {
        if (known_uniform(sh.tile0[g + 1]) <= q) {
            ++g;
            for (int end = P.E + 1; end - g > 1;) {   // the last group that starts at or before q: most may be empty
                const int mid = (g + end) >> 1;
                if (known_uniform(sh.tile0[mid]) <= q) g = mid;
                else end = mid;
            }
        }
        Tile t;
        t.g = g, t.nt = nt;
        t.mt = q - known_uniform(sh.tile0[g]);
        t.row = known_uniform(sh.row0[g]) + t.mt * kRows;
        t.rows = min(kRows, known_uniform(sh.row0[g + 1]) - t.row);
        return t;
    }
};

// Where a stage's parts lie in shared memory.
template <bool NV, int BN, bool kPair> struct Stages {
    using C = Cfg<NV, BN, kPair>;
    uint32_t base;   // a multiple of 1024: the swizzle pattern repeats every 1024 bytes
    __device__ explicit Stages(const void *dyn) : base((tc::smem_u32(dyn) + 1023u) & ~1023u) {}
    __device__ uint32_t a(int s) const { return base + s * C::kStride; }
    __device__ uint32_t b(int s) const { return a(s) + C::kBytesA; }
    __device__ uint32_t sa(int s) const { return b(s) + C::kBytesB; }
    __device__ uint32_t sb(int s) const { return sa(s) + C::kBytesSA; }
    __device__ uint32_t out(int warp) const { return a(C::kStages) + warp * kOutBuf; }
};

// The products of one stage (one elected lane): scales to their columns of
// tensor memory, then `steps` steps of 32 bytes of k.  The scale columns are the
// stage's own, so the barrier that frees the stage frees them too.
template <bool NV, int BN, bool kPair>
__device__ __forceinline__ void multiply_stage(const Stages<NV, BN, kPair> &st, int s, uint32_t d, int steps, uint32_t add) {
    using C = Cfg<NV, BN, kPair>;
    constexpr uint32_t idesc = tc::idesc_block_scaled(NV, kPair ? 2 * kRowsT : kRowsT, BN);
    constexpr int kSc = C::kSc;
    const uint32_t sfa = C::kAcc * BN + s * C::kScCols, sfb = sfa + 4 * kSc;   // the block holds all columns: they start at 0
    const uint32_t a = tc::desc_lo(st.a(0)) + s * (C::kStride / 16), b = a + C::kBytesA / 16, sa = b + C::kBytesB / 16,
                   sb = sa + C::kBytesSA / 16;
#pragma unroll
    for (int j = 0; j < kSc; ++j) {
        tc::copy_scales<kPair>(sfa + 4 * j, sa + j * (kScaleTile / 16));
#pragma unroll
        for (int g = 0; g < C::kGroupsB; ++g)
            tc::copy_scales<kPair>(sfb + 4 * (j * C::kGroupsB + g), sb + (g * kSc + j) * (kScaleTile / 16));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j > 0 && j >= steps) break;
        if (NV) tc::mma_nvf4<kPair>(d, a + 2 * j, b + 2 * j, idesc, sfa + 4 * j, sfb + 4 * C::kGroupsB * j, j ? 1 : add);
        else tc::mma_mxf8<kPair>(d, a + 2 * j, b + 2 * j, idesc | tc::idesc_scale_id(j), sfa, sfb, j ? 1 : add);
    }
}

// Waits (bounded) for the last stages' barriers, so that no copy, product or arrival
// is in flight when the block leaves.
template <int kStages> __device__ __forceinline__ void settle(uint64_t *bars, int it) {
    uint32_t none = 0;
    for (int j = it < kStages ? 0 : it - kStages; j < it; ++j)
        tc::bar_wait(tc::smem_u32(&bars[j % kStages]), (j / kStages) & 1, &none);
}

// Barriers, tensor memory, and the block's (the pair's) start and end.
template <int kStages, bool kPair, int kWarps = kEpiWarps>
__device__ __forceinline__ void open_block(Barriers &sh, int warp, uint32_t full_count, uint32_t cols) {
    if (threadIdx.x == 0) {
        sh.dead = 0;
        for (int s = 0; s < kStages; ++s) {
            tc::bar_init(tc::smem_u32(&sh.full[s]), full_count);
            tc::bar_init(tc::smem_u32(&sh.empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::bar_init(tc::smem_u32(&sh.acc_full[a]), 1);
            tc::bar_init(tc::smem_u32(&sh.acc_empty[a]), kPair ? 2 * kWarps : kWarps);
        }
        tc::bar_init_fence();
    }
    if (warp == 1) tc::tmem_alloc<kPair>(tc::smem_u32(&sh.tmem), cols);
    tc::fence_before();
    if (kPair) tc::cluster_sync();
    else __syncthreads();
    tc::fence_after();
}

// status: the device's word for reports (ERR_*).
template <bool kPair> __device__ __forceinline__ void close_block(Barriers &sh, int warp, uint32_t cols, uint32_t *status) {
    __syncwarp();
    tc::fence_before();
    if (kPair) tc::cluster_sync();   // neither block leaves while the other may read its memory or signal it
    else __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free<kPair>(0, cols);
    }
    if (threadIdx.x == 0 && sh.dead) atomicOr(status, ERR_TIMEOUT);
}

// Where the results of a warp go: its first row (o; 32 rows of `pitch` elements, `rows` of them its own), from the
// tile's column on (`cols` of them are left).  add: onto what is there.  wide: rows start on 16 bytes.
template <typename T> struct OutAt {
    T *o;
    int64_t pitch, cols;
    int rows;
    bool add, wide;
};

// 16 bytes of results: accumulators times ua and ub (kScale), rounded to T.
template <bool kScale> __device__ __forceinline__ float scaled(uint32_t v, float ua, float ub) {
    const float f = __uint_as_float(v);
    return kScale ? f * ua * ub : f;
}
template <bool kScale> __device__ __forceinline__ void finish(const uint32_t *v, float ua, float ub, uint32_t (&w)[4], float) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(scaled<kScale>(v[i], ua, ub));
}
template <bool kScale>
__device__ __forceinline__ void finish(const uint32_t *v, float ua, float ub, uint32_t (&w)[4], __nv_bfloat16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(scaled<kScale>(v[2 * i], ua, ub), scaled<kScale>(v[2 * i + 1], ua, ub));
        memcpy(&w[i], &h, 4);
    }
}

// Results of a warp, a row of kHalf columns in each lane, to memory by way of shared
// memory: 32 rows x 128 bytes at a time, each lane writing its row's 16-byte chunk c to
// c ^ (row mod 8) and reading back so that eight lanes hold 128 consecutive bytes of one
// row: no bank conflicts either way, whole lines to memory.
//   Rows straight from the lanes cost 32 passes of the load/store pipe an instruction,
// 4.5K (BF16) and 9.2K (FP32) cycles for a tile of 128 x 256.  TMA stores take 129 cycles
// for 4 KB and the operands' copies wait behind them in the same unit (a stage of 32 KB
// 331 -> 1191 cycles).
template <int kHalf, bool kScale, typename T>
__device__ __forceinline__ void store_warp(const uint32_t *v, float ua, float ub, uint32_t buf, const OutAt<T> &w, int lane) {
    constexpr int kPer = 16 / sizeof(T), kPiece = 8 * kPer;
#pragma unroll
    for (int j = 0; j < kHalf; j += kPiece) {
        if (j >= w.cols) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t x[4];
            finish<kScale>(v + j + c * kPer, ua, ub, x, T());
            tc::st_shared(buf + lane * 128 + ((c ^ (lane & 7)) << 4), x);
        }
        __syncwarp();
        const int q = lane & 7, col = j + q * kPer;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 4) {
            const int r = r0 + (lane >> 3);
            const uint4 x = tc::ld_shared(buf + r * 128 + ((q ^ (r & 7)) << 4));
            if (r < w.rows && col < w.cols) *reinterpret_cast<uint4 *>(w.o + r * w.pitch + col) = x;
        }
        __syncwarp();
    }
}

// The same for rows that do not start on 16 bytes and for results onto what is there (added in FP32, rounded once):
// 32 rows x 32 columns at a time in FP32, a column a lane.
template <int kHalf, bool kScale, typename T>
__device__ __forceinline__ void store_warp_any(const uint32_t *v, float ua, float ub, uint32_t buf, const OutAt<T> &w, int lane) {
#pragma unroll
    for (int j = 0; j < kHalf; j += 32) {
        if (j >= w.cols) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t x[4];
            finish<kScale>(v + j + c * 4, ua, ub, x, float());
            tc::st_shared(buf + lane * 128 + ((c ^ (lane & 7)) << 4), x);
        }
        __syncwarp();
        if (j + lane < w.cols) {
            T *o = w.o + j + lane;
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
                if (r >= w.rows) break;
                float f = tc::ld_shared1(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3));
                if (w.add) f += static_cast<float>(o[r * w.pitch]);
                o[r * w.pitch] = static_cast<T>(f);
            }
        }
        __syncwarp();
    }
}

// A tile without products.
template <int kHalf, typename T> __device__ __forceinline__ void zero_tile(const OutAt<T> &w, int lane) {
    constexpr int kPer = 16 / sizeof(T);
    for (int r = 0; r < 32 && r < w.rows; ++r) {
        T *o = w.o + r * w.pitch;
        if (w.wide)
            for (int c = lane * kPer; c < kHalf && c < w.cols; c += 32 * kPer) *reinterpret_cast<uint4 *>(o + c) = make_uint4(0, 0, 0, 0);
        else
            for (int c = lane; c < kHalf && c < w.cols; c += 32) o[c] = static_cast<T>(0.0f);
    }
}

// A role's place in the ring of stages: the stage, the parity of the round, and how many were issued (for settle).
template <int kStages> struct Ring {
    int s = 0;
    uint32_t round = 0;
    int issued = 0;
    __device__ __forceinline__ void next() {
        if (++s == kStages) s = 0, round ^= 1;
    }
};

// The loops of the issuing warps do not leave when a wait runs out (then every further wait returns at once and nothing
// more is issued): without such exits their counters are uniform, and so are the addresses and descriptors.

// The tensor core cuts off what its FP32 sum does not hold at every step of 32 bytes of
// k, toward zero: an error of 1 to 2e-8 of the sum a step that grows with the length
// (MXFP8, one expert of 4096 / 65536 rows: 1e-6 / 2.5e-5 of the weight gradient, sums of one
// sign twice that).  So a sum longer than this many stages is taken in pieces, which the
// draining warps add in FP32, rounding to nearest: 5e-7 at any length.  A piece costs a
// tile's end: MXFP8 weight gradients of 8192 rows an expert 72.8 -> 79.2 us, NVFP4 63.6 ->
// 65.9, products of 4096 MXFP8 columns 97.5 -> 101.  BF16 results, whose own rounding is
// 2e-3, have longer pieces (2e-5).
template <typename T> constexpr int kPiece = sizeof(T) == 4 ? 16 : 256;

// The products of one output tile, `len` bytes of k in pieces of kLen stages, by the (converged) issuing warp.  n: pieces
// so far of this unit.
template <int kLen, bool NV, int BN, bool kPair, typename R>
__device__ __forceinline__ void multiply_tile(Barriers &sh, const Stages<NV, BN, kPair> &st, int &n, R &ring, int len, bool &ok) {
    using C = Cfg<NV, BN, kPair>;
    volatile uint32_t *dead = &sh.dead;
    const int kt = (len + kStageK - 1) / kStageK;
    for (int k0 = 0; k0 < kt; k0 += kLen, ++n) {
        const int a = n % C::kAcc, k1 = min(kt, k0 + kLen);
        ok = ok && (n < C::kAcc || tc::bar_wait(tc::smem_u32(&sh.acc_empty[a]), (n / C::kAcc - 1) & 1, dead));
        __syncwarp();
        tc::fence_after();
        for (int k = k0; k < k1; ++k, ring.next()) {
            ok = ok && tc::bar_wait(tc::smem_u32(&sh.full[ring.s]), ring.round, dead);
            __syncwarp();
            tc::fence_after();
            if (tc::elect() && ok) {
                // the last stage holds only what is left of k
                multiply_stage(st, ring.s, a * BN, (len - k * kStageK + 31) / 32, k > k0);
                tc::commit<kPair>(tc::smem_u32(&sh.empty[ring.s]));
                if (k == k1 - 1) tc::commit<kPair>(tc::smem_u32(&sh.acc_full[a]));
            }
            __syncwarp();
            ring.issued += ok;
        }
    }
}

// One stage's copies by the (converged) loading warp: 128 rows of A's codes, the
// block's rows of B's (128 at a time), and the scale tiles, at (x, row) and (0, tile)
// of their maps.
struct StageAt {
    const CUtensorMap *a, *b, *sa, *sb;
    int x, a_row, b_row, a_tile, b_tile, b_tile_step;   // step: between the 128-row groups of B's scales
    int b_row_step;                                     // between B's 128-row boxes, where a block has two
    int a_boxes;                                        // single blocks: boxes of 32 rows of A that the tile has
};
// kParts: both operands' (3), or for single blocks A's (1) or B's (2) alone, of which B's come first.
template <bool NV, int BN, bool kPair, int kParts = 3, typename R>
__device__ __forceinline__ void load_stage(Barriers &sh, const Stages<NV, BN, kPair> &st, int half, R &ring, const StageAt &w,
                                           bool &ok) {
    using C = Cfg<NV, BN, kPair>;
    const int s = ring.s;
    static_assert(kParts == 3 || !kPair, "");
    if (kParts & 2) ok = ok && tc::bar_wait(tc::smem_u32(&sh.empty[s]), ring.round ^ 1, &sh.dead);   // the first round passes
    __syncwarp();
    const uint32_t own = tc::smem_u32(&sh.full[s]), bar = kPair ? tc::map_to(own, 0) : own;
    auto load = [&](uint32_t dst, const CUtensorMap *tm, int x, int y) {
        if (kPair) tc::load_2d_pair(dst, tm, x, y, bar);
        else tc::load_2d(dst, tm, x, y, bar);
    };
    if (tc::elect() && ok) {
        if (kPair) {
            if (half == 0) tc::bar_expect(own, 2 * C::kStageBytes);
            load(st.a(s), w.a, w.x, w.a_row);
        } else {   // the rows of a short tile only: the others' products go nowhere
            if (kParts & 2) tc::bar_expect(own, C::kStageBytes - (kRowsT / kBoxA - w.a_boxes) * kBoxA * kStageK);
            if (kParts & 1)
                for (int b = 0; b < w.a_boxes; ++b) load(st.a(s) + b * kBoxA * kStageK, w.a, w.x, w.a_row + b * kBoxA);
        }
        if (kParts & 2) {
#pragma unroll
            for (int b = 0; b < C::kRowsB / 128; ++b) load(st.b(s) + b * 128 * kStageK, w.b, w.x, w.b_row + b * w.b_row_step);
        }
        if (kParts & 1) load(st.sa(s), w.sa, 0, w.a_tile);
        if (kParts & 2) {
#pragma unroll
            for (int b = 0; b < C::kGroupsB; ++b) load(st.sb(s) + b * C::kSc * kScaleTile, w.sb, 0, w.b_tile + b * w.b_tile_step);
        }
    }
    __syncwarp();
    ring.issued += ok;
    ring.next();
}

// The rows' part of a later tile's stage into L2 (pairs): units that run side by side
// share it, so one of them asks memory for it and all find it there a tile later (65536 x
// 2048 x 2048 NVFP4 over 32 experts: 117.4 -> 112.7 us).  The columns' operand is left
// alone: asking for it twice costs more than the wait wherever it is read only a few times
// (128 rows an expert, 2048 x 4096 MXFP8: 226 us without, 327 with; single blocks at 16
// rows an expert 171 and 302).
__device__ __forceinline__ void prefetch_rows(const StageAt &w) {
    if (tc::elect()) {
        tc::prefetch_2d(w.a, w.x, w.a_row);
        tc::prefetch_2d(w.sa, 0, w.a_tile);
    }
    __syncwarp();
}

// The loading warp's end: the block stays until the products' arrivals on its last stages' barriers are in (they go to
// both blocks of a pair; a later one would change the shared memory of whatever block comes next).  After a wait that ran
// out: until its copies are.
template <int kStages> __device__ __forceinline__ void end_loads(Barriers &sh, int half, int it, bool ok) {
    if (ok) settle<kStages>(sh.empty, it);
    else if (half == 0) settle<kStages>(sh.full, it);
    else tc::pause(1000000);   // these copies count on the other block's barriers: time for them to land
}

// 1 / S of both sides, for a sum of NVFP4 products.
__device__ __forceinline__ void units_of(float amax_a, float amax_b, float &ua, float &ub) {
    ua = __fdiv_rn(1.0f, tensor_scale(amax_a));
    ub = __fdiv_rn(1.0f, tensor_scale(amax_b));
    // A sum (2^-20 to 2^53 units) times ua, then ub: their product may leave FP32's range where the result does not.
    // So may the first step, but only with ua far out and ub leading back, and then the product is in range.
    if ((ua > 0x1p64f && ub < 1.0f) || (ua < 0x1p-64f && ub > 4.0f)) ua *= ub, ub = 1.0f;
}

// The accumulators of a finished tile of `kt` stages, in pieces of kLen, into the registers of one draining warp: kN
// columns, one run of them at c0 or (kRuns 2) half of them at c0 and half at c1; n: pieces so far of this unit.  An
// accumulator is handed back as soon as it is in registers: scaling, rounding and stores run while the next tile is
// multiplied.  False: a wait ran out.
template <int BN, int kAcc, bool kPair, int kLen, int kRuns, int kN>
__device__ __forceinline__ bool take_tile(Barriers &sh, int &n, int kt, int q, int lane, uint32_t c0, uint32_t c1, uint32_t (&v)[kN]) {
    constexpr int kRun = kN / kRuns;
    const uint32_t row = static_cast<uint32_t>(32 * q) << 16;
    auto wait = [&] {
        const bool ok = tc::bar_wait_warp(tc::smem_u32(&sh.acc_full[n % kAcc]), (n / kAcc) & 1, &sh.dead);
        tc::fence_after();
        return ok;
    };
    auto hand_back = [&] {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
            const uint32_t bar = tc::smem_u32(&sh.acc_empty[n % kAcc]);
            if (kPair) tc::bar_arrive_cluster(tc::map_to(bar, 0));
            else tc::bar_arrive(bar);
        }
        ++n;
    };
    if (!wait()) return false;
    {
        const uint32_t at = row + (n % kAcc) * BN;
        uint32_t(&run0)[kRun] = *reinterpret_cast<uint32_t(*)[kRun]>(v);
        tc::tmem_ld(at + c0, run0);
        if constexpr (kRuns == 2) {
            uint32_t(&run1)[kRun] = *reinterpret_cast<uint32_t(*)[kRun]>(v + kRun);
            tc::tmem_ld(at + c1, run1);
        }
    }
    hand_back();
    for (int k = kLen; k < kt; k += kLen) {
        if (!wait()) return false;
        const uint32_t at = row + (n % kAcc) * BN;
#pragma unroll
        for (int j = 0; j < kN; j += 8) {   // (16 at a time spills)
            uint32_t x[8];
            tc::tmem_ld(at + (j < kRun ? c0 + j : c1 + j - kRun), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j + i] = __float_as_uint(__uint_as_float(v[j + i]) + __uint_as_float(x[i]));
        }
        hand_back();
    }
    return true;
}

// A finished tile to memory by one draining warp.  ahead(): what the next tile needs from memory, asked for before the
// stores.
template <bool NV, int BN, bool kPair, typename T, typename F>
__device__ __forceinline__ bool drain_tile(Barriers &sh, int &n, int kt, int warp, int lane, float amax_a, float amax_b, const OutAt<T> &w,
                                           uint32_t buf, F &&ahead) {
    using C = Cfg<NV, BN, kPair>;
    const int q = warp & 3, h = (warp - kDrain) >> 2;
    float ua = 1.0f, ub = 1.0f;
    if (NV) units_of(amax_a, amax_b, ua, ub);
    uint32_t v[BN / 2];
    if (!take_tile<BN, C::kAcc, kPair, kPiece<T>, 1>(sh, n, kt, q, lane, h * (BN / 2), 0, v)) return false;
    const OutAt<T> here = w;
    ahead();
    if (here.wide && !here.add) store_warp<BN / 2, NV, T>(v, ua, ub, buf, here, lane);
    else store_warp_any<BN / 2, NV, T>(v, ua, ub, buf, here, lane);
    return true;
}

// -------------------------------------------------------------------- host

// A CUDA call failed: the next call must not take its error, which the runtime keeps, for one of its own.
gsa_status cuda_error() {
    cudaGetLastError();
    return GSA_ERR_CUDA;
}

// A function of the driver (nullptr: a CUDA error).
template <typename F> F driver_fn(const char *name, std::atomic<F> &known) {
    F fn = known.load(std::memory_order_relaxed);
    if (fn) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
        known.store(fn = reinterpret_cast<F>(p), std::memory_order_relaxed);
    return fn;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    return driver_fn("cuTensorMapEncodeTiled", known);
}

// The current context's number, which no other context of the process has had (0: none is current yet).
uint64_t context_id() {
    static std::atomic<PFN_cuCtxGetId_v12000> known{nullptr};
    auto fn = driver_fn("cuCtxGetId", known);
    unsigned long long id = 0;
    return fn && fn(nullptr, &id) == CUDA_SUCCESS ? id : 0;
}

// Codes [rows, bytes]: boxes of 128 bytes x `box` rows in the 128-byte swizzle, zeros outside.
bool map_codes(CUtensorMap *tm, const void *p, int64_t rows, int64_t bytes, int box) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(bytes), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(bytes)};
    cuuint32_t b[2] = {kStageK, static_cast<cuuint32_t>(box)}, es[2] = {1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles of 512 bytes, `box` at a time, zeros past the last.
bool map_scales(CUtensorMap *tm, const void *p, int64_t tiles, int box) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {kScaleTile / 4, static_cast<cuuint64_t>(tiles)};
    cuuint64_t strides[1] = {kScaleTile};
    cuuint32_t b[2] = {kScaleTile / 4, static_cast<cuuint32_t>(box)}, es[2] = {1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<void *>(p), dims, strides, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What is asked once per device: only answers are kept, a failed query is made again.  What is set up (once()) is so in a
// context: in another one, or after the device's has been reset, it is set up again (asking which one is current takes 0.01 us,
// the shared memory of a kernel 0.2).
struct PerDevice {
    std::mutex mu;
    int n[64] = {};
    uint64_t did[64] = {};   // the context that it was last done in
    template <typename F> bool once(F &&act) {   // false: a CUDA error
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
        const uint64_t here = context_id();
        std::lock_guard<std::mutex> lock(mu);
        if (here && did[dev] == here) return true;
        if (act() != cudaSuccess) return false;
        did[dev] = here;
        return true;
    }
    template <typename F> int get(F &&ask) {   // 0: a CUDA error
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
        std::lock_guard<std::mutex> lock(mu);
        if (!n[dev]) {
            int v = 0;
            if (ask(dev, v) == cudaSuccess && v > 0) n[dev] = v;
        }
        return n[dev];
    }
};

// Number of SMs of the current device (0: a CUDA error).
int sm_count() {
    static PerDevice known;
    return known.get([](int dev, int &v) { return cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev); });
}

// A persistent launch of at most `want` blocks (kPair: pairs of blocks), as many as run at once.
template <bool kPair, typename P>
gsa_status launch(void (*kernel)(P), const P &params, int threads, size_t smem, int64_t want, cudaStream_t s, PerDevice &pairs) {
    const int sms = sm_count();
    if (!sms || !pairs.once([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)); }))
        return cuda_error();
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see wait_for_previous
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = kPair ? 2 : 1;
    int64_t units = sms;
    if (kPair) {   // the machine's clusters may not fill every SM
        units = pairs.get([&](int, int &v) {
            cfg.gridDim = dim3(2 * (sms / 2));
            return cudaOccupancyMaxActiveClusters(&v, kernel, &cfg);
        });
        if (!units) return cuda_error();
    }
    const int64_t n = want < units ? want : units;
    cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * n : n));
    return cudaLaunchKernelEx(&cfg, kernel, params) == cudaSuccess ? GSA_OK : cuda_error();
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
