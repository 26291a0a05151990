// grouped_gemm.cu -- grouped products of block-scaled (MXFP8 / NVFP4) operands on
// the 5th-generation tensor cores (sm_103a), with their C entry points.
//
//   out[r, n] = u_e sum_k A[r, k] B_e[n, k],   rows r of expert e,
// A and B_e given as codes with one scale per 32 (E8M0) or 16 (E4M3) elements of
// k, and for NVFP4 u_e = 1 / (S_A,e S_B,e) from the experts' amax (S = 2688 / amax,
// what the quantizer multiplied by).  The tensor core multiplies codes and block
// scales and sums in FP32 (tcgen05.mma with block_scale; long sums in pieces, see
// kPiece); u_e and the rounding to the output type are the epilogue.
//
// Persistent blocks walk the tiles of all experts (column tiles of a row tile one
// after another so that its rows stay in L2).  With many rows an expert, pairs of
// blocks share tiles of 256 x 256 (a block then reads 32 KB of codes for 128 x 256 x 256
// products instead of 48); with few, blocks take 128 x 128.  Warp 0 loads stages of 128
// bytes of k (A, B and their scale tiles, by TMA), warp 1 copies the scales to tensor
// memory and issues the products, and 8 warps drain the accumulators.
//   What bounds it: an NVFP4 stage of a pair is 512 cycles of products and about 200 of
// scale copies in the same queue, an MXFP8 one 512 and 50; a tile's end costs about 1000
// more.  65536 x 2048 x 2048 NVFP4 over 32 experts: 112 to 122 us on different machines (4.5
// to 4.9 PFLOP/s); 262144 x 4096 x 2048 MXFP8 over 128 experts: 1500 to 1560 us (2.9 PFLOP/s)
// at the clock that the power limit leaves, 1345 us for a launch by itself; 512 rows over 128
// experts, 2048 x 4096 NVFP4: 70 to 74 us, the weights at 6.2 TB/s.  Launched as a
// programmatic dependent, a block sets up while the kernel before it ends: 32 rows over 128
// experts 20.3 -> 18.0 us on one machine (17 to 21 over all).
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
constexpr int kEpiWarps = 8, kDrain = 4;   // the draining warps, the first of them
constexpr int kBoxA = 32;            // rows of A that single blocks load at a time
constexpr int kOutBuf = 32 * 128;    // a draining warp's piece of results: 32 rows x 128 bytes
constexpr int kStatic = 4096;        // what the blocks' static shared memory stays below

using gemm_status::ERR_SPLIT;
using gemm_status::ERR_TIMEOUT;

// What went wrong in grouped products on this device and was not yet asked for, and what the query under way took.
__device__ uint32_t g_status, g_taken;

// The kernel of a query: reports only ever set bits and queries run one at a time, so a bit seen is the bit cleared.
__global__ void take_status() {
    g_taken = gemm_status::next_report(atomicOr(&g_status, 0u));
    atomicAnd(&g_status, ~g_taken);
}

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
template <bool NV, int BN, bool kPair> struct Cfg {
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
    static constexpr int kOut = kEpiWarps * kOutBuf;   // results on their way out
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
    int64_t scan[kThreads / 32][3];
    uint32_t bad;
};

// A value that is the same in all lanes, as the compiler cannot tell.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Group bounds from the device split: rows, scale tiles and row tiles of kRows before each group.  Every thread
// of the block.  A negative size, a sum above M or more scale tiles than A's buffer holds sets sh.bad.
template <int kRows> __device__ void scan_split(const GemmParams &P, GemmShared &sh) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? P.split[t] : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
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
template <int kStages, bool kPair>
__device__ __forceinline__ void open_block(Barriers &sh, int warp, uint32_t full_count, uint32_t cols) {
    if (threadIdx.x == 0) {
        sh.dead = 0;
        for (int s = 0; s < kStages; ++s) {
            tc::bar_init(tc::smem_u32(&sh.full[s]), full_count);
            tc::bar_init(tc::smem_u32(&sh.empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::bar_init(tc::smem_u32(&sh.acc_full[a]), 1);
            tc::bar_init(tc::smem_u32(&sh.acc_empty[a]), kPair ? 2 * kEpiWarps : kEpiWarps);
        }
        tc::bar_init_fence();
    }
    if (warp == 1) tc::tmem_alloc<kPair>(tc::smem_u32(&sh.tmem), cols);
    tc::fence_before();
    if (kPair) tc::cluster_sync();
    else __syncthreads();
    tc::fence_after();
}

template <bool kPair> __device__ __forceinline__ void close_block(Barriers &sh, int warp, uint32_t cols) {
    __syncwarp();
    tc::fence_before();
    if (kPair) tc::cluster_sync();   // neither block leaves while the other may read its memory or signal it
    else __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free<kPair>(0, cols);
    }
    if (threadIdx.x == 0 && sh.dead) atomicOr(&g_status, ERR_TIMEOUT);
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

// The products of one output tile, `len` bytes of k, by the (converged) issuing warp.  n: pieces so far of this unit.
template <typename T, bool NV, int BN, bool kPair, typename R>
__device__ __forceinline__ void multiply_tile(Barriers &sh, const Stages<NV, BN, kPair> &st, int &n, R &ring, int len, bool &ok) {
    using C = Cfg<NV, BN, kPair>;
    volatile uint32_t *dead = &sh.dead;
    const int kt = (len + kStageK - 1) / kStageK;
    for (int k0 = 0; k0 < kt; k0 += kPiece<T>, ++n) {
        const int a = n % C::kAcc, k1 = min(kt, k0 + kPiece<T>);
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
// block's rows of B's, and the scale tiles, at (x, row) and (0, tile) of their
// maps.
struct StageAt {
    const CUtensorMap *a, *b, *sa, *sb;
    int x, a_row, b_row, a_tile, b_tile, b_tile_step;   // step: between the 128-row groups of B's scales
    int a_boxes;                                        // single blocks: boxes of 32 rows of A that the tile has
};
template <bool NV, int BN, bool kPair, typename R>
__device__ __forceinline__ void load_stage(Barriers &sh, const Stages<NV, BN, kPair> &st, int half, R &ring, const StageAt &w,
                                           bool &ok) {
    using C = Cfg<NV, BN, kPair>;
    const int s = ring.s;
    ok = ok && tc::bar_wait(tc::smem_u32(&sh.empty[s]), ring.round ^ 1, &sh.dead);   // the first round passes
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
            tc::bar_expect(own, C::kStageBytes - (kRowsT / kBoxA - w.a_boxes) * kBoxA * kStageK);
            for (int b = 0; b < w.a_boxes; ++b) load(st.a(s) + b * kBoxA * kStageK, w.a, w.x, w.a_row + b * kBoxA);
        }
        load(st.b(s), w.b, w.x, w.b_row);
        load(st.sa(s), w.sa, 0, w.a_tile);
#pragma unroll
        for (int b = 0; b < C::kGroupsB; ++b) load(st.sb(s) + b * C::kSc * kScaleTile, w.sb, 0, w.b_tile + b * w.b_tile_step);
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

// A finished tile of `kt` stages to memory by one draining warp; n: pieces so far of this
// unit.  An accumulator is handed back as soon as it is in registers: scaling, rounding
// and stores run while the next tile is multiplied.  ahead(): what the next tile needs from memory,
// asked for before the stores.  False: a wait ran out.
template <bool NV, int BN, bool kPair, typename T, typename F>
__device__ __forceinline__ bool drain_tile(Barriers &sh, int &n, int kt, int warp, int lane, float amax_a, float amax_b, const OutAt<T> &w,
                                           uint32_t buf, F &&ahead) {
    using C = Cfg<NV, BN, kPair>;
    const int q = warp & 3, h = (warp - kDrain) >> 2;
    float ua = 1.0f, ub = 1.0f;
    if (NV) {
        ua = __fdiv_rn(1.0f, tensor_scale(amax_a));
        ub = __fdiv_rn(1.0f, tensor_scale(amax_b));
        // A sum (2^-20 to 2^53 units) times ua, then ub: their product may leave FP32's range where the result does not.
        // So may the first step, but only with ua far out and ub leading back, and then the product is in range.
        if ((ua > 0x1p64f && ub < 1.0f) || (ua < 0x1p-64f && ub > 4.0f)) ua *= ub, ub = 1.0f;
    }
    const uint32_t at = h * (BN / 2) + (static_cast<uint32_t>(32 * q) << 16);
    auto wait = [&] {
        const bool ok = tc::bar_wait_warp(tc::smem_u32(&sh.acc_full[n % C::kAcc]), (n / C::kAcc) & 1, &sh.dead);
        tc::fence_after();
        return ok;
    };
    auto hand_back = [&] {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
            const uint32_t bar = tc::smem_u32(&sh.acc_empty[n % C::kAcc]);
            if (kPair) tc::bar_arrive_cluster(tc::map_to(bar, 0));
            else tc::bar_arrive(bar);
        }
        ++n;
    };
    if (!wait()) return false;
    uint32_t v[BN / 2];
    tc::tmem_ld(at + (n % C::kAcc) * BN, v);
    hand_back();
    for (int k = kPiece<T>; k < kt; k += kPiece<T>) {
        if (!wait()) return false;
#pragma unroll
        for (int j = 0; j < BN / 2; j += 8) {   // (16 at a time spills)
            uint32_t x[8];
            tc::tmem_ld(at + (n % C::kAcc) * BN + j, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j + i] = __float_as_uint(__uint_as_float(v[j + i]) + __uint_as_float(x[i]));
        }
        hand_back();
    }
    const OutAt<T> here = w;
    ahead();
    if (here.wide && !here.add) store_warp<BN / 2, NV, T>(v, ua, ub, buf, here, lane);
    else store_warp_any<BN / 2, NV, T>(v, ua, ub, buf, here, lane);
    return true;
}

template <bool NV, int BN, bool kPair, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_gemm(const __grid_constant__ GemmParams P) {
    using C = Cfg<NV, BN, kPair>;
    extern __shared__ uint8_t dyn[];
    __shared__ GemmShared sh;
    static_assert(sizeof(GemmShared) <= kStatic, "shared memory");
    constexpr int kRows = kPair ? 2 * kRowsT : kRowsT;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
    const int half = kPair ? blockIdx.x & 1 : 0;   // the block's 128 rows of the tile (and its rank in the cluster)
    const Stages<NV, BN, kPair> st(dyn);
    open_block<C::kStages, kPair>(sh, warp, 1, C::kCols);   // nothing in global memory: runs beside the end of the kernel before
    tc::allow_next();
    tc::wait_for_previous();
    scan_split<kRows>(P, sh);
    if (sh.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, ERR_SPLIT);
    const int64_t total = sh.bad ? 0 : static_cast<int64_t>(sh.tile0[P.E + 1]) * P.n_tiles;
    const int64_t used = sh.bad ? 0 : static_cast<int64_t>(sh.tile0[P.E]) * P.n_tiles;   // the rest is zeros

    if (warp == 0) {
        if (tc::elect()) {
            tc::prefetch_map(&P.tm_a);
            tc::prefetch_map(&P.tm_b);
        }
        Ring<C::kStages> ring;
        int g = 0;
        bool ok = true, first = false;   // first: the next tile is its rows' first
        auto at = [&](int64_t i) {
            const Tile t = tile_at<kRows>(P, sh, i, g);
            g = t.g;
            StageAt w{&P.tm_a, &P.tm_b, &P.tm_sa, &P.tm_sb};
            w.x = 0;
            w.a_row = uniform(t.row) + half * kRowsT;
            w.a_boxes = uniform((t.rows + kBoxA - 1) / kBoxA);
            w.a_tile = uniform((sh.scale0[g] + t.mt * (kRows / 128) + half) * P.scale_cols);
            w.b_row = uniform(static_cast<int>(g * P.N + static_cast<int64_t>(t.nt) * BN)) + half * C::kRowsB;
            w.b_tile = uniform((g * P.b_scale_rows + t.nt * C::kGroupsB) * P.scale_cols);
            w.b_tile_step = P.scale_cols;
            first = uniform(t.nt) == 0;
            return w;
        };
        StageAt w, next;
        if (unit < used) next = at(unit);
        for (int64_t i = unit; i < used; i += units) {
            w = next;
            const bool more = i + units < used;
            if (more) next = at(i + units);
            StageAt ahead = next;
            for (int k = 0; k < P.kt; ++k) {
                load_stage(sh, st, half, ring, w, ok);
                if (kPair && more && first) prefetch_rows(ahead);
                w.x += kStageK, w.a_tile += C::kSc, w.b_tile += C::kSc;
                ahead.x += kStageK, ahead.a_tile += C::kSc;
            }
        }
        end_loads<C::kStages>(sh, half, ring.issued, ok);
    } else if (warp == 1 && half == 0) {
        const int mine = unit < used ? uniform(static_cast<int>((used - unit + units - 1) / units)) : 0;
        Ring<C::kStages> ring;
        int n = 0;
        bool ok = true;
        for (int i = 0; i < mine; ++i) multiply_tile<T>(sh, st, n, ring, P.k_bytes, ok);
        if (!ok || *static_cast<volatile uint32_t *>(&sh.dead)) settle<C::kStages>(sh.empty, ring.issued);
    } else if (warp >= kDrain) {
        const int q = warp & 3, h = (warp - kDrain) >> 2;   // lanes 32 q .., column half h
        constexpr int kHalf = BN / 2;
        T *out = static_cast<T *>(P.out);
        const int r0 = half * kRowsT + 32 * q;   // the warp's first row of the tile
        const uint32_t buf = st.out(warp - kDrain);
        OutAt<T> w;
        w.pitch = P.N;
        w.wide = P.N * sizeof(T) % 16 == 0;
        w.add = false;
        int g = 0, n = 0;
        float amax_a = 0.0f, amax_b = 0.0f;
        auto find = [&](int64_t i) {
            if (i >= total) return;
            const Tile t = tile_at<kRows>(P, sh, i, g);
            g = t.g;
            const int64_t c0 = static_cast<int64_t>(t.nt) * BN + h * kHalf;
            w.o = out + static_cast<int64_t>(t.row + r0) * P.N + c0;
            w.cols = P.N - c0;
            w.rows = t.rows - r0;
            if (NV && g < P.E) amax_a = P.amax_a[g], amax_b = P.amax_b[g];
        };
        find(unit);
        for (int64_t i = unit; i < total; i += units) {
            if (g == P.E) {
                zero_tile<kHalf>(w, lane);
                find(i + units);
            } else if (!drain_tile<NV, BN, kPair>(sh, n, P.kt, warp, lane, amax_a, amax_b, w, buf, [&] { find(i + units); })) {
                break;
            }
        }
    }
    close_block<kPair>(sh, warp, C::kCols);
}

// ---------------------------------------------------------- weight gradient
//
//   dw_e[n, k] = u_e sum_r A[r, n] B[r, k] over the rows r of expert e,
// from columnwise copies: per expert [N, Mp_e] and [K, Mp_e], Mp_e the rows padded
// to whole scale blocks, so that the sum runs along the contiguous axis again and
// the tiles are those of the grouped product with N and K as the free sides.
//
// Every expert's matrices have an origin and a pitch of their own that only the
// device knows, so a kernel before the products writes each expert's tensor maps.
// TMA takes pitches of multiples of 16 bytes; an NVFP4 expert has Mp_e / 2, a
// multiple of 8, so that kernel also copies the experts with an odd number of
// 8-byte groups to rows 8 bytes longer.  (Bringing such rows in with loads instead
// ran at 20 to 26 bytes a cycle and SM from L2, any width and number of warps,
// against 65 to 76 by TMA: 577 us for 65536 x 2048 x 2048 over 32 experts, against 184 to 199:
// 24 for that kernel, 160 for the products, whose FP32 results of 128 KB a block and tile
// one SM stores in 5900 cycles.)  Last, scales past Mp_e are padding that nobody wrote, and a zero code
// times a NaN scale is NaN: where a product step of 64 rows is cut short, the
// scale tiles of that last stage are copied with zeros there.

struct WgradParams {
    CUtensorMap tm_sa, tm_sb, tm_ta, tm_tb;   // scale tiles; the tail copies of the last stages'
    const uint8_t *a, *b, *sa, *sb;
    const int64_t *split;
    const float *amax_a, *amax_b;
    void *out;
    CUtensorMap *maps;                 // [2][E]: A's and B's codes of each expert
    uint8_t *tail_a, *tail_b;          // [E][row tiles][4] scale tiles
    uint8_t *pack_a, *pack_b;          // copies of the experts with odd pitches
    int64_t M;
    int N, K, E;
    int n_tiles, k_tiles;              // tiles along N and K
    int64_t a_bytes, b_bytes, sa_bytes, sb_bytes;
    int accumulate;
};

struct Pads {
    int pad0[kMaxE + 1];        // padded rows before each expert
    int wide0[kMaxE + 1];       // scale tiles along the rows before each expert
    int rows[kMaxE];
    int64_t scan[kMaxE / 32][3];
    uint32_t bad;
};
struct WgradShared : Barriers {
    Pads pads;
    uint16_t order[kMaxE];      // experts by descending size
};

// Padded rows and scale tiles before each expert.  Every thread of a block of at least 256.  A negative size, a sum
// above M or more than the buffers hold sets bad.
template <int kBlock, bool NV> __device__ void scan_pads(const WgradParams &P, Pads &d) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? P.split[t] : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
    if (t < P.E) d.rows[t] = static_cast<int>(m);
    int64_t rows = m, pad = (m + kBlock - 1) / kBlock * kBlock, wide = (m + 4 * kBlock - 1) / (4 * kBlock);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, s), q = __shfl_up_sync(0xFFFFFFFFu, pad, s),
                      u = __shfl_up_sync(0xFFFFFFFFu, wide, s);
        if (lane >= s) rows += r, pad += q, wide += u;
    }
    if (w < kMaxE / 32 && lane == 31) d.scan[w][0] = rows, d.scan[w][1] = pad, d.scan[w][2] = wide;
    const bool any_neg = __syncthreads_or(neg);
    for (int k = 0; k < w && k < kMaxE / 32; ++k) rows += d.scan[k][0], pad += d.scan[k][1], wide += d.scan[k][2];
    if (t < P.E) {
        d.pad0[t + 1] = static_cast<int>(pad);
        d.wide0[t + 1] = static_cast<int>(wide);
    }
    if (t == 0) d.pad0[0] = 0, d.wide0[0] = 0;
    if (t == P.E - 1) {
        const int64_t codes = NV ? pad / 2 : pad, tiles = wide * kScaleTile;
        d.bad = any_neg || rows > P.M || codes * P.N > P.a_bytes || codes * P.K > P.b_bytes ||
                tiles * ((P.N + 127) / 128) > P.sa_bytes || tiles * ((P.K + 127) / 128) > P.sb_bytes;
    }
    __syncthreads();
}

// Where an expert's odd-pitch copy starts, in units of rows of the matrix: 8 bytes more than its codes.
__device__ __forceinline__ int64_t pack_at(const Pads &d, int e) { return d.pad0[e] / 2 + 8 * e; }

constexpr int kPrepThreads = 256;

template <bool NV>
__global__ void __launch_bounds__(kPrepThreads) wgrad_prepare(const __grid_constant__ WgradParams P,
                                                              const __grid_constant__ CUtensorMap plain_a,
                                                              const __grid_constant__ CUtensorMap plain_b) {
    __shared__ Pads d;
    __shared__ __align__(128) CUtensorMap map;
    constexpr int kBlock = NV ? 16 : 32;
    tc::allow_next();
    scan_pads<kBlock, NV>(P, d);
    if (d.bad) return;   // the products report it
    for (int i = blockIdx.x; i < 2 * P.E; i += gridDim.x) {
        const int e = i < P.E ? i : i - P.E;
        const int64_t mp = d.pad0[e + 1] - d.pad0[e], pitch = NV ? mp / 2 : mp, first = NV ? d.pad0[e] / 2 : d.pad0[e];
        const int rows = i < P.E ? P.N : P.K;
        if (threadIdx.x < 32 && mp > 0) {
            if (threadIdx.x == 0) {
                const bool odd = pitch % 16 != 0;
                const uint8_t *at = odd ? (i < P.E ? P.pack_a : P.pack_b) + pack_at(d, e) * rows
                                        : (i < P.E ? P.a : P.b) + first * rows;
                map = i < P.E ? plain_a : plain_b;
                tc::edit_map(&map, at, static_cast<uint32_t>(pitch), static_cast<uint32_t>(rows), odd ? pitch + 8 : pitch);
            }
            __syncwarp();
            tc::publish_map(P.maps + i, &map);
        }
        __syncthreads();
    }
    if (!NV) return;
    const int warp = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kPrepThreads / 32);
    const int lane = threadIdx.x & 31;
    // rows of odd pitch, four at a time a warp: 8-byte halves (a row starts on 8 bytes), 16-byte stores
    constexpr int kBatch = 4;
    const int na = (P.N + kBatch - 1) / kBatch, batches = na + (P.K + kBatch - 1) / kBatch;
    for (int64_t i = warp; i < static_cast<int64_t>(P.E) * batches; i += warps) {
        const int e = static_cast<int>(i / batches), j = static_cast<int>(i - static_cast<int64_t>(e) * batches);
        const int64_t pitch = (d.pad0[e + 1] - d.pad0[e]) / 2;
        if (pitch % 16 == 0) continue;
        const bool is_a = j < na;
        const int r = (is_a ? j : j - na) * kBatch, rows = is_a ? P.N : P.K;
        const uint8_t *src = (is_a ? P.a : P.b) + static_cast<int64_t>(d.pad0[e] / 2) * rows + r * pitch;
        uint8_t *dst = (is_a ? P.pack_a : P.pack_b) + pack_at(d, e) * rows + r * (pitch + 8);
        for (int64_t c = 16 * lane; c < pitch; c += 512) {
            uint2 x[kBatch], y[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const bool in = r + b < rows;
                x[b] = in ? __ldcs(reinterpret_cast<const uint2 *>(src + b * pitch + c)) : make_uint2(0, 0);
                y[b] = in && c + 8 < pitch ? __ldcs(reinterpret_cast<const uint2 *>(src + b * pitch + c + 8)) : make_uint2(0, 0);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (r + b < rows) *reinterpret_cast<uint4 *>(dst + b * (pitch + 8) + c) = make_uint4(x[b].x, x[b].y, y[b].x, y[b].y);
        }
    }
    // the last stages' scale tiles, zeros past the expert's scales
    const int n128 = (P.N + 127) / 128, groups = n128 + (P.K + 127) / 128;
    for (int64_t i = warp; i < static_cast<int64_t>(P.E) * groups * 4; i += warps) {
        const int j = static_cast<int>(i & 3), x = static_cast<int>(i >> 2), e = x / groups, g = x - e * groups;
        const int64_t mp = d.pad0[e + 1] - d.pad0[e];
        const int cols = static_cast<int>(mp / 16);
        if (cols % 4 == 0) continue;
        const int wide = d.wide0[e + 1] - d.wide0[e], tile = (cols - 1) / 16 * 4 + j;
        const bool is_a = g < n128;
        const int row = is_a ? g : g - n128, tiles = is_a ? n128 : groups - n128;
        uint8_t *dst = (is_a ? P.tail_a : P.tail_b) + ((static_cast<int64_t>(e) * tiles + row) * 4 + j) * kScaleTile + 16 * lane;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (tile < wide) {
            v = *reinterpret_cast<const uint4 *>((is_a ? P.sa : P.sb) + (static_cast<int64_t>(d.wide0[e]) * tiles +
                                                 static_cast<int64_t>(row) * wide + tile) * kScaleTile + 16 * lane);
            const int left = cols - 4 * tile;
            const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
            v.x &= keep, v.y &= keep, v.z &= keep, v.w &= keep;
        }
        *reinterpret_cast<uint4 *>(dst) = v;
    }
}

// A tile of the weight gradients.  A unit's r-th tile goes back and forth over the
// units (u, then units - 1 - u, ..) in the order of descending experts, so that
// long and short sums even out.
struct WTile {
    int e, nt, kt;
    int rows;   // padded rows of the expert
};
// The unit's next tile from round r on: false when there is none.
__device__ __forceinline__ bool next_wtile(const WgradParams &P, const WgradShared &sh, uint32_t &r, uint32_t unit, uint32_t units,
                                           uint32_t total, WTile &t) {
    for (;; ++r) {
        if (r * units >= total) return false;
        const uint32_t i = r * units + ((r & 1) ? units - 1 - unit : unit);
        if (i >= total) continue;
        ++r;
        const uint32_t per = P.n_tiles * P.k_tiles, x = i / per, j = i - x * per;
        t.e = sh.order[x];
        t.nt = j / P.k_tiles;
        t.kt = j - t.nt * P.k_tiles;
        t.rows = sh.pads.pad0[t.e + 1] - sh.pads.pad0[t.e];
        return true;
    }
}

template <bool NV, int BN, bool kPair, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_wgrad(const __grid_constant__ WgradParams P) {
    using C = Cfg<NV, BN, kPair>;
    extern __shared__ uint8_t dyn[];
    __shared__ WgradShared sh;
    static_assert(sizeof(WgradShared) <= kStatic, "shared memory");
    constexpr int kBlock = NV ? 16 : 32, kRows = kPair ? 2 * kRowsT : kRowsT;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
    const int half = kPair ? blockIdx.x & 1 : 0;
    const Stages<NV, BN, kPair> st(dyn);
    open_block<C::kStages, kPair>(sh, warp, 1, C::kCols);
    tc::allow_next();
    tc::wait_for_previous();
    scan_pads<kBlock, NV>(P, sh.pads);
    if (sh.pads.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, ERR_SPLIT);
    if (static_cast<int>(threadIdx.x) < P.E) {
        const int m = sh.pads.rows[threadIdx.x];
        int rank = 0;
        for (int k = 0; k < P.E; ++k) rank += sh.pads.rows[k] > m || (sh.pads.rows[k] == m && k < static_cast<int>(threadIdx.x));
        sh.order[rank] = static_cast<uint16_t>(threadIdx.x);
    }
    __syncthreads();
    const uint32_t total = sh.pads.bad ? 0 : static_cast<uint32_t>(P.E) * P.n_tiles * P.k_tiles;
    WTile t;
    uint32_t r = 0;

    if (warp == 0) {
        const int n128 = (P.N + 127) / 128, k128 = (P.K + 127) / 128;
        Ring<C::kStages> ring;
        int last = -1;
        bool ok = true;
        while (next_wtile(P, sh, r, unit, units, total, t)) {
            const int e = uniform(t.e), nt = uniform(t.nt), kt = uniform(t.kt);
            const int len = uniform(NV ? t.rows / 2 : t.rows), cols = uniform(t.rows / kBlock);
            const int wide0 = uniform(sh.pads.wide0[e]), wide = uniform(sh.pads.wide0[e + 1]) - wide0;
            if (len == 0) continue;
            StageAt w{P.maps + e, P.maps + P.E + e, &P.tm_sa, &P.tm_sb};
            w.x = 0;
            if (e != last) {   // maps written by the kernel before
                tc::acquire_map(w.a);
                tc::acquire_map(w.b);
                last = e;
            }
            const int a_group = nt * (kRows / 128) + half, b_group = kt * C::kGroupsB;
            w.a_row = nt * kRows + half * kRowsT;
            w.a_boxes = (min(kRowsT, P.N - w.a_row) + kBoxA - 1) / kBoxA;
            w.b_row = kt * BN + half * C::kRowsB;
            w.a_tile = wide0 * n128 + a_group * wide;
            w.b_tile = wide0 * k128 + b_group * wide;
            w.b_tile_step = wide;
            const int stages = (len + kStageK - 1) / kStageK;
            for (int k = 0; k < stages; ++k) {
                if (NV && k == stages - 1 && cols % 4 != 0) {
                    w.sa = &P.tm_ta, w.sb = &P.tm_tb;
                    w.a_tile = (e * n128 + a_group) * 4;
                    w.b_tile = (e * k128 + b_group) * 4;
                    w.b_tile_step = 4;
                }
                load_stage(sh, st, half, ring, w, ok);
                w.x += kStageK, w.a_tile += C::kSc, w.b_tile += C::kSc;
            }
        }
        end_loads<C::kStages>(sh, half, ring.issued, ok);
    } else if (warp == 1 && half == 0) {
        Ring<C::kStages> ring;
        int n = 0;
        bool ok = true;
        while (next_wtile(P, sh, r, unit, units, total, t)) {
            const int len = uniform(NV ? t.rows / 2 : t.rows);
            if (len > 0) multiply_tile<T>(sh, st, n, ring, len, ok);
        }
        if (!ok || *static_cast<volatile uint32_t *>(&sh.dead)) settle<C::kStages>(sh.empty, ring.issued);
    } else if (warp >= kDrain) {
        const int q = warp & 3, h = (warp - kDrain) >> 2;
        constexpr int kHalf = BN / 2;
        T *out = static_cast<T *>(P.out);
        const uint32_t buf = st.out(warp - kDrain);
        OutAt<T> w;
        w.pitch = P.K;
        w.wide = P.K * sizeof(T) % 16 == 0;
        w.add = P.accumulate != 0;
        int n = 0;
        float amax_a = 0.0f, amax_b = 0.0f;
        bool more = true;
        auto find = [&] {
            more = next_wtile(P, sh, r, unit, units, total, t);
            if (!more) return;
            const int row = t.nt * kRows + half * kRowsT + 32 * q, c0 = t.kt * BN + h * kHalf;
            w.o = out + (static_cast<int64_t>(t.e) * P.N + row) * P.K + c0;
            w.cols = static_cast<int64_t>(P.K) - c0;
            w.rows = P.N - row;
            if (NV) amax_a = P.amax_a[t.e], amax_b = P.amax_b[t.e];
        };
        find();
        while (more) {
            if (t.rows == 0) {   // no rows: a zero gradient
                if (!w.add) zero_tile<kHalf>(w, lane);
                find();
            } else {
                const int stages = ((NV ? t.rows / 2 : t.rows) + kStageK - 1) / kStageK;
                if (!drain_tile<NV, BN, kPair>(sh, n, stages, warp, lane, amax_a, amax_b, w, buf, find)) break;
            }
        }
    }
    close_block<kPair>(sh, warp, C::kCols);
}

// -------------------------------------------------------------------- host

// A CUDA call failed: the next call must not take its error, which the runtime keeps, for one of its own.
gsa_status cuda_error() {
    cudaGetLastError();
    return GSA_ERR_CUDA;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_relaxed);
    if (fn) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        known.store(fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p), std::memory_order_relaxed);
    return fn;
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

// What is asked once per device: only answers are kept, a failed query is made again.
struct PerDevice {
    std::mutex mu;
    int n[64] = {};
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
    if (!sms) return cuda_error();
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return cuda_error();
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kPair ? 2 : 1;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see wait_for_previous
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
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

template <bool NV, int BN, bool kPair, typename T>
gsa_status launch_gemm(const GemmParams &P, int64_t tiles, cudaStream_t s) {
    static PerDevice pairs;
    return launch<kPair, GemmParams>(grouped_gemm<NV, BN, kPair, T>, P, kThreads, Cfg<NV, BN, kPair>::kSmem, tiles * P.n_tiles,
                                     s, pairs);
}

template <bool NV, int BN, bool kPair, typename T> gsa_status launch_wgrad(const WgradParams &P, cudaStream_t s) {
    static PerDevice pairs;
    return launch<kPair, WgradParams>(grouped_wgrad<NV, BN, kPair, T>, P, kThreads, Cfg<NV, BN, kPair>::kSmem,
                                      static_cast<int64_t>(P.E) * P.n_tiles * P.k_tiles, s, pairs);
}

// Workspace of the weight gradient (byte offsets; the maps come first).
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256 * 64, kMaxSide = int64_t(1) << 30;
struct WgradSpace {
    size_t tail_a = 0, tail_b = 0, pack_a = 0, pack_b = 0, bytes = 0;
    WgradSpace(int64_t E, int64_t M, int64_t N, int64_t K, bool nv) {
        auto take = [&](int64_t n) {
            const size_t at = bytes;
            bytes += (static_cast<size_t>(n) + 255) / 256 * 256;
            return at;
        };
        take(2 * E * static_cast<int64_t>(sizeof(CUtensorMap)));
        if (!nv) return;
        tail_a = take(E * ((N + 127) / 128) * 4 * kScaleTile);
        tail_b = take(E * ((K + 127) / 128) * 4 * kScaleTile);
        const int64_t used = E < M ? E : M, cols = (M + 15 * used) / 2 + 8 * E;   // bytes of all padded rows, and 8 an expert
        pack_a = take(cols * N);
        pack_b = take(cols * K);
    }
};

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" {

gsa_status gsa_grouped_gemm(const gsa_qin *a, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M,
                            int64_t N, int64_t K, int32_t recipe_kind, void *out, int32_t out_dtype,
                            gsa_stream_t stream) {
    if (!a || !b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (out_dtype != GSA_BF16 && out_dtype != GSA_FP32) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    if (E > kMaxE || K % 64 != 0 || K > (int64_t(1) << 30) || M >= (int64_t(1) << 31) - 256 ||
        N >= (int64_t(1) << 31) / E - 256)
        return GSA_ERR_UNSUPPORTED;
    if (M == 0) return GSA_OK;
    if (!a->data || !a->scale || !b->data || !b->scale || !split_sizes_dev || !out) return GSA_ERR_INVALID_ARG;
    if (nv && (!a->amax || !b->amax)) return GSA_ERR_INVALID_ARG;
    if (!aligned(a->data, 16) || !aligned(a->scale, 16) || !aligned(b->data, 16) || !aligned(b->scale, 16) ||
        !aligned(out, 16) || !aligned(split_sizes_dev, 8) || !aligned(a->amax, 4) || !aligned(b->amax, 4))
        return GSA_ERR_ALIGNMENT;
    const int64_t k_bytes = nv ? K / 2 : K;
    const int64_t cols = (K / (nv ? 16 : 32) + 3) / 4, n128 = (N + 127) / 128;
    const int64_t a_rows = a->scale_bytes / (kScaleTile * cols);   // row tiles that the buffer holds
    if (a->data_bytes < M * k_bytes || b->data_bytes < E * N * k_bytes || a_rows < (M > 0) ||
        b->scale_bytes < E * n128 * cols * kScaleTile)
        return GSA_ERR_INVALID_ARG;
    if (a_rows * cols >= (int64_t(1) << 31) || E * n128 * cols >= (int64_t(1) << 31)) return GSA_ERR_UNSUPPORTED;

    GemmParams P;
    std::memset(&P, 0, sizeof(P));
    // Pairs (256 x 256) from 128 rows an expert on, single blocks (128 x 128) below, where tiles are mostly cut
    // short and the weights are what there is to read.  Pairs / singles, us, 128 experts, 2048 x 4096: 64 rows an
    // expert 125 / 109 (NVFP4), 323 / 193 (MXFP8; both pairs' figures with B prefetched), 128 rows 125 / 132 and
    // 226 / 230, 256 rows 159 / 185 and 293 / 320; 16 experts, 4096 x 4096, 256 rows 49.5 / 52.1 and 85.0 / 85.6.
    // All of these have tiles for every unit; the rule does not look at how many there are, and few tiles (few experts,
    // small N) leave units without one in either shape.
    const bool pair = M >= 128 * E;
    const int BN = pair ? 256 : 128;
    const int sc = nv ? 4 : 1;
    if (!map_codes(&P.tm_a, a->data, M, k_bytes, pair ? kRowsT : kBoxA) || !map_codes(&P.tm_b, b->data, E * N, k_bytes, 128) ||
        !map_scales(&P.tm_sa, a->scale, a_rows * cols, sc) || !map_scales(&P.tm_sb, b->scale, E * n128 * cols, sc))
        return cuda_error();
    P.split = split_sizes_dev;
    P.amax_a = a->amax;
    P.amax_b = b->amax;
    P.out = out;
    P.M = M;
    P.N = N;
    P.kt = static_cast<int>((k_bytes + kStageK - 1) / kStageK);
    P.k_bytes = static_cast<int>(k_bytes);
    P.E = static_cast<int>(E);
    P.n_tiles = static_cast<int>((N + BN - 1) / BN);
    P.b_scale_rows = static_cast<int>(n128);
    P.scale_cols = static_cast<int>(cols);
    P.a_scale_tiles = a_rows;
    // row tiles: at most one partial tile per expert that has rows, and the tail's
    const int64_t tiles = (M + kRowsT - 1) / kRowsT + (E < M ? E : M);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    gsa_status st;
    auto typed = [&](auto fmt, auto type) {
        return pair ? launch_gemm<decltype(fmt)::value, 256, true, decltype(type)>(P, tiles, s)
                    : launch_gemm<decltype(fmt)::value, 128, false, decltype(type)>(P, tiles, s);
    };
    auto sized = [&](auto fmt) { return out_dtype == GSA_BF16 ? typed(fmt, __nv_bfloat16()) : typed(fmt, float()); };
    st = nv ? sized(std::true_type()) : sized(std::false_type());
    return st;
}

size_t gsa_grouped_gemm_wgrad_workspace_size(int64_t E, int64_t M, int64_t N, int64_t K, int32_t recipe_kind) {
    if (E <= 0 || E > kMaxE || M < 0 || N <= 0 || K <= 0 || M >= kMaxRows || N >= kMaxSide || K >= kMaxSide ||
        (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4))
        return 0;
    return WgradSpace(E, M, N, K, recipe_kind == GSA_NVFP4).bytes;
}

gsa_status gsa_grouped_gemm_wgrad(const gsa_qin *a, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E,
                                  int64_t M, int64_t N, int64_t K, int32_t recipe_kind, void *dw, int32_t out_dtype,
                                  int32_t accumulate, void *workspace, size_t workspace_bytes, gsa_stream_t stream) {
    if (!a || !b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (out_dtype != GSA_BF16 && out_dtype != GSA_FP32) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    if (E > kMaxE || M >= kMaxRows || N >= kMaxSide || K >= kMaxSide) return GSA_ERR_UNSUPPORTED;
    // TMA: an expert's NVFP4 codes start on 16 bytes (8 bytes of codes a block times the width)
    if (nv && (N % 2 != 0 || K % 2 != 0)) return GSA_ERR_UNSUPPORTED;
    if (!a->data || !a->scale || !b->data || !b->scale || !split_sizes_dev || !dw) return GSA_ERR_INVALID_ARG;
    if (nv && (!a->amax || !b->amax)) return GSA_ERR_INVALID_ARG;
    if (!aligned(a->data, 16) || !aligned(a->scale, 16) || !aligned(b->data, 16) || !aligned(b->scale, 16) ||
        !aligned(dw, 16) || !aligned(split_sizes_dev, 8) || !aligned(a->amax, 4) || !aligned(b->amax, 4) ||
        !aligned(workspace, 256))
        return GSA_ERR_ALIGNMENT;
    const WgradSpace ws(E, M, N, K, nv);
    if (!workspace || workspace_bytes < ws.bytes) return GSA_ERR_WORKSPACE;

    const int64_t n128 = (N + 127) / 128, k128 = (K + 127) / 128;
    const int64_t a_tiles = a->scale_bytes / kScaleTile, b_tiles = b->scale_bytes / kScaleTile;
    if (a_tiles >= (int64_t(1) << 31) || b_tiles >= (int64_t(1) << 31) || E * n128 * 4 >= (int64_t(1) << 31) ||
        E * k128 * 4 >= (int64_t(1) << 31))
        return GSA_ERR_UNSUPPORTED;
    // Pairs wherever a side has more than one tile of 128 (not measured against single blocks where tiles are few).
    const bool pair = N > 128 && K > 128;
    const int64_t tile = pair ? 256 : 128, n_tiles = (N + tile - 1) / tile, k_tiles = (K + tile - 1) / tile;
    if (E * n_tiles * k_tiles >= (int64_t(1) << 31) - 4096) return GSA_ERR_UNSUPPORTED;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    WgradParams P;
    std::memset(&P, 0, sizeof(P));
    const int sc = nv ? 4 : 1;
    // The experts' maps but for origin, extents and pitch.  Encoded for the smallest matrix: from a large one something
    // stays in the map that editing does not change, and copies then touch memory up to 128 KB behind an expert's origin,
    // past the operand's end (encoded 4096 x 4096, 128 x 4096 or 65536 x 128: seen; 128 x 128 and below: none).
    CUtensorMap plain_a, plain_b;
    if (!map_codes(&plain_a, w, 1, 16, pair ? kRowsT : kBoxA) || !map_codes(&plain_b, w, 1, 16, 128) ||
        // (without rows the scale buffers may be empty: nothing is loaded then)
        !map_scales(&P.tm_sa, a_tiles ? a->scale : w, a_tiles ? a_tiles : 1, sc) ||
        !map_scales(&P.tm_sb, b_tiles ? b->scale : w, b_tiles ? b_tiles : 1, sc) ||
        (nv && (!map_scales(&P.tm_ta, w + ws.tail_a, E * n128 * 4, 4) || !map_scales(&P.tm_tb, w + ws.tail_b, E * k128 * 4, 4))))
        return cuda_error();
    P.a = static_cast<const uint8_t *>(a->data);
    P.b = static_cast<const uint8_t *>(b->data);
    P.sa = static_cast<const uint8_t *>(a->scale);
    P.sb = static_cast<const uint8_t *>(b->scale);
    P.split = split_sizes_dev;
    P.amax_a = a->amax;
    P.amax_b = b->amax;
    P.out = dw;
    P.maps = reinterpret_cast<CUtensorMap *>(w);
    P.tail_a = w + ws.tail_a;
    P.tail_b = w + ws.tail_b;
    P.pack_a = w + ws.pack_a;
    P.pack_b = w + ws.pack_b;
    P.M = M;
    P.N = static_cast<int>(N);
    P.K = static_cast<int>(K);
    P.E = static_cast<int>(E);
    P.n_tiles = static_cast<int>(n_tiles);
    P.k_tiles = static_cast<int>(k_tiles);
    P.a_bytes = a->data_bytes;
    P.b_bytes = b->data_bytes;
    P.sa_bytes = a->scale_bytes;
    P.sb_bytes = b->scale_bytes;
    P.accumulate = accumulate != 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (!sms) return cuda_error();
    // An ordinary launch: as a programmatic dependent too, a pass of 65536 rows, 32 experts took 208 us instead of 191.
    if (nv) wgrad_prepare<true><<<4 * sms, kPrepThreads, 0, s>>>(P, plain_a, plain_b);
    else wgrad_prepare<false><<<static_cast<unsigned>(2 * E < sms ? 2 * E : sms), kPrepThreads, 0, s>>>(P, plain_a, plain_b);
    if (cudaGetLastError() != cudaSuccess) return GSA_ERR_CUDA;
    gsa_status st;
    auto typed = [&](auto fmt, auto type) {
        return pair ? launch_wgrad<decltype(fmt)::value, 256, true, decltype(type)>(P, s)
                    : launch_wgrad<decltype(fmt)::value, 128, false, decltype(type)>(P, s);
    };
    auto sized = [&](auto fmt) { return out_dtype == GSA_BF16 ? typed(fmt, __nv_bfloat16()) : typed(fmt, float()); };
    st = nv ? sized(std::true_type()) : sized(std::false_type());
    return st;
}

gsa_status gsa_grouped_gemm_status(gsa_stream_t stream) {
    static std::mutex one;   // g_taken is one query's at a time
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &capturing) != cudaSuccess || capturing != cudaStreamCaptureStatusNone) return cuda_error();
    std::lock_guard<std::mutex> lock(one);
    // nothing here touches a capture that another thread may have under way
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return cuda_error();
    uint32_t report = 0;
    take_status<<<1, 1, 0, s>>>();
    const bool ok = cudaGetLastError() == cudaSuccess &&
                    cudaMemcpyFromSymbolAsync(&report, g_taken, sizeof(report), 0, cudaMemcpyDeviceToHost, s) == cudaSuccess &&
                    cudaStreamSynchronize(s) == cudaSuccess;
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (!ok) return cuda_error();
    return gemm_status::status_of(report);
}

}  // extern "C"
