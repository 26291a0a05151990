// grouped_gemm.cu -- grouped products of block-scaled (MXFP8 / NVFP4) operands on
// the 5th-generation tensor cores (sm_103a), with their C entry points.
//
//   out[r, n] = u_e sum_k A[r, k] B_e[n, k],   rows r of expert e,
// A and B_e given as codes with one scale per 32 (E8M0) or 16 (E4M3) elements of
// k, and for NVFP4 u_e = 1 / (S_A,e S_B,e) from the experts' amax (S = 2688 / amax,
// what the quantizer multiplied by).  The tensor core multiplies codes and block
// scales and sums in FP32 (tcgen05.mma with block_scale); u_e and the rounding to
// the output type are the epilogue.
//
// Persistent blocks walk the tiles of all experts (128 rows x BN columns, column
// tiles of a row tile one after another so that its rows stay in L2).  Warp 0
// loads stages of 128 bytes of k (A, B and their scale tiles, by TMA), warp 1
// copies the scales to tensor memory and issues the products, and 8 warps drain
// the accumulators.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cstring>
#include <mutex>
#include <type_traits>

#include "gsa.h"
#include "launches.h"
#include "tc.cuh"

namespace {

constexpr int kMaxE = 256;
constexpr int kRowsT = 128;          // rows of a tile: the lanes of tensor memory
constexpr int kStageK = 128;         // bytes of k per stage: one 128-byte swizzled row
constexpr int kScaleTile = 512;      // bytes of one 128 x 4 scale tile
constexpr int kThreads = 384;        // warp 0 loads, warp 1 multiplies, warps 4-11 drain
constexpr int kEpiWarps = 8;

enum { ERR_SPLIT = 1, ERR_TIMEOUT = 2 };

// What went wrong in grouped products on this device since the last query.
__device__ uint32_t g_status;

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
    static constexpr int kBySmem = (227 * 1024 - 8192 - 1024) / kStride, kByCols = (kCols - kAcc * BN) / kScCols;
    static constexpr int kFit = kBySmem < kByCols ? kBySmem : kByCols;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kSmem = kStages * kStride + 1024;
};

struct Shared {
    int64_t row0[kMaxE + 2];    // first row of each group; group E: rows that no expert has
    int tile0[kMaxE + 2];       // first row tile of each group
    int scale0[kMaxE + 1];      // first 128-row scale tile of each expert
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2];
    uint32_t tmem;
    uint32_t dead, bad;
    int64_t scan[kThreads / 32][3];
};

// A value that is the same in all lanes, as the compiler cannot tell.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Group bounds from the device split: rows, scale tiles and row tiles of kRows before each group.  Every thread
// of the block.  A negative size, a sum above M or more scale tiles than A's buffer holds sets sh.bad.
template <int kRows> __device__ void scan_split(const GemmParams &P, Shared &sh) {
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
        sh.row0[t + 1] = rows;
        sh.scale0[t + 1] = static_cast<int>(scales);
        sh.tile0[t + 1] = static_cast<int>(tiles);
    }
    if (t == 0) sh.row0[0] = 0, sh.scale0[0] = 0, sh.tile0[0] = 0;
    __syncthreads();
    if (t == 0) {
        const int64_t sum = sh.row0[P.E];
        sh.bad = any_neg || sum > P.M || sh.scale0[P.E] > P.a_scale_tiles;
        sh.row0[P.E + 1] = P.M;
        sh.tile0[P.E + 1] = sh.tile0[P.E] + static_cast<int>((P.M - (sum > P.M ? P.M : sum) + kRows - 1) / kRows);
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
    int64_t row;    // first row
    int rows;       // rows of the tile that belong to the group
    int mt;         // row tile within the group
    int nt;         // column tile
};

// Tile number i of kRows rows, searching from group g on (tile numbers only grow).
template <int kRows> __device__ __forceinline__ Tile tile_at(const GemmParams &P, const Shared &sh, int64_t i, int g) {
    const int q = static_cast<int>(i / P.n_tiles);
    while (q >= sh.tile0[g + 1]) ++g;
    Tile t;
    t.g = g;
    t.nt = static_cast<int>(i - static_cast<int64_t>(q) * P.n_tiles);
    t.mt = q - sh.tile0[g];
    t.row = sh.row0[g] + static_cast<int64_t>(t.mt) * kRows;
    const int64_t left = sh.row0[g + 1] - t.row;
    t.rows = left < kRows ? static_cast<int>(left) : kRows;
    return t;
}

// 32 bytes of results at o.  align: the bytes that o is aligned to (32, 16 or less); n: how many of the results
// there are (at most 32 bytes of them).
__device__ __forceinline__ void store_raw(uint8_t *o, const uint32_t *w, int align) {
    if (align == 32)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(o + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ void store_some(__nv_bfloat16 *o, const uint32_t *w, int n, int align) {
    if (n >= 16 && align >= 16) {
        store_raw(reinterpret_cast<uint8_t *>(o), w, align);
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) reinterpret_cast<uint16_t *>(o)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
}

__device__ __forceinline__ void store_some(float *o, const uint32_t *w, int n, int align) {
    if (n >= 8 && align >= 16) {
        store_raw(reinterpret_cast<uint8_t *>(o), w, align);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) o[i] = __uint_as_float(w[i]);
}

// Largest of 32, 16 and 1 that every row start of out [.., n] is aligned to.
template <typename T> __device__ __forceinline__ int row_align(const T *out, int64_t n) {
    const uint64_t x = reinterpret_cast<uint64_t>(out) | static_cast<uint64_t>(n * static_cast<int64_t>(sizeof(T)));
    return x % 32 == 0 ? 32 : x % 16 == 0 ? 16 : 1;
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
};

// The products of one stage (one elected lane): scales to their columns of
// tensor memory, then `steps` steps of 32 bytes of k.  The scale columns are the
// stage's own, so the barrier that frees the stage frees them too.
template <bool NV, int BN, bool kPair>
__device__ __forceinline__ void multiply_stage(const Stages<NV, BN, kPair> &st, int s, uint32_t tmem, uint32_t d, int steps,
                                               bool first) {
    using C = Cfg<NV, BN, kPair>;
    constexpr uint32_t idesc = tc::idesc_block_scaled(NV, kPair ? 2 * kRowsT : kRowsT, BN);
    constexpr int kSc = C::kSc;
    const uint32_t sfa = tmem + C::kAcc * BN + s * C::kScCols, sfb = sfa + 4 * kSc;
#pragma unroll
    for (int j = 0; j < kSc; ++j) {
        tc::copy_scales<kPair>(sfa + 4 * j, tc::desc_scales(st.sa(s) + j * kScaleTile));
#pragma unroll
        for (int b = 0; b < C::kGroupsB; ++b)
            tc::copy_scales<kPair>(sfb + 4 * (j * C::kGroupsB + b), tc::desc_scales(st.sb(s) + (b * kSc + j) * kScaleTile));
    }
    for (int j = 0; j < steps; ++j) {
        const uint64_t da = tc::desc_sw128(st.a(s) + 32 * j), db = tc::desc_sw128(st.b(s) + 32 * j);
        const bool add = !first || j > 0;
        if (NV) tc::mma_nvf4<kPair>(d, da, db, idesc, sfa + 4 * j, sfb + 4 * C::kGroupsB * j, add);
        else tc::mma_mxf8<kPair>(d, da, db, idesc | tc::idesc_scale_id(j), sfa, sfb, add);
    }
}

// After a wait that ran out: waits (bounded) for the last stages' barriers, so
// that no copy or product is in flight when the block leaves.
template <int kStages> __device__ __forceinline__ void settle(uint64_t *bars, int it) {
    uint32_t none = 0;
    for (int j = it < kStages ? 0 : it - kStages; j < it; ++j)
        tc::bar_wait(tc::smem_u32(&bars[j % kStages]), (j / kStages) & 1, &none);
}

// Barriers, tensor memory, and the block's (the pair's) start and end.
template <int kStages, bool kPair>
__device__ __forceinline__ void open_block(Shared &sh, int warp, uint32_t full_count, uint32_t cols) {
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

template <bool kPair> __device__ __forceinline__ void close_block(Shared &sh, int warp, uint32_t cols) {
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

// 32 bytes of results: accumulators times ua and ub (kScale), rounded to T.
template <bool kScale> __device__ __forceinline__ void finish(const uint32_t *v, float ua, float ub, uint32_t (&w)[8], float) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = kScale ? __float_as_uint(__uint_as_float(v[i]) * ua * ub) : v[i];
}
template <bool kScale>
__device__ __forceinline__ void finish(const uint32_t *v, float ua, float ub, uint32_t (&w)[8], __nv_bfloat16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(v[2 * i]), y = __uint_as_float(v[2 * i + 1]);
        const __nv_bfloat162 h = kScale ? __floats2bfloat162_rn(x * ua * ub, y * ua * ub) : __floats2bfloat162_rn(x, y);
        memcpy(&w[i], &h, 4);
    }
}

// The same onto the n values at o.
__device__ __forceinline__ void finish_add(const float *o, const uint32_t *v, float ua, float ub, int n, uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint((i < n ? o[i] : 0.0f) + __uint_as_float(v[i]) * ua * ub);
}
__device__ __forceinline__ void finish_add(const __nv_bfloat16 *o, const uint32_t *v, float ua, float ub, int n,
                                           uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = 2 * i < n ? __bfloat162float(o[2 * i]) : 0.0f, y = 2 * i + 1 < n ? __bfloat162float(o[2 * i + 1]) : 0.0f;
        const __nv_bfloat162 h = __floats2bfloat162_rn(x + __uint_as_float(v[2 * i]) * ua * ub,
                                                       y + __uint_as_float(v[2 * i + 1]) * ua * ub);
        memcpy(&w[i], &h, 4);
    }
}

// One accumulator to memory: this thread's lane and kHalf columns from tensor
// memory, times ua and ub (kScale), to o[0 .. cols), or onto what is there (add).
// on: the lane holds a row of the result.  The accumulator is handed back
// (`release`) as soon as it is in registers: scaling, rounding and stores run while
// the next tile is multiplied.
template <int kHalf, bool kScale, typename T, typename F>
__device__ __forceinline__ void drain(uint32_t src, float ua, float ub, T *o, int64_t cols, bool on, int align, bool add,
                                      F &&release) {
    constexpr int kPer = 32 / sizeof(T);
    uint32_t v[kHalf];
    tc::tmem_ld(src, v);
    release();
    if (!on) return;
#pragma unroll
    for (int j = 0; j < kHalf; j += kPer) {
        if (j >= cols) break;
        const int n = cols - j < kPer ? static_cast<int>(cols - j) : kPer;
        uint32_t w[8];
        if (add) finish_add(o + j, v + j, ua, ub, n, w);
        else finish<kScale>(v + j, ua, ub, w, T());
        store_some(o + j, w, n, align);
    }
}

template <typename T> __device__ __forceinline__ void zeros(T *o, int half, int64_t cols, int align) {
    constexpr int kPer = 32 / sizeof(T);
    const uint32_t zero[8] = {};
    for (int c = 0; c < half && c < cols; c += kPer)
        store_some(o + c, zero, cols - c < kPer ? static_cast<int>(cols - c) : kPer, align);
}

template <bool NV, int BN, bool kPair, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_gemm(const __grid_constant__ GemmParams P) {
    using C = Cfg<NV, BN, kPair>;
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    constexpr int kRows = kPair ? 2 * kRowsT : kRowsT, kSc = C::kSc;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    scan_split<kRows>(P, sh);
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
    const int half = kPair ? blockIdx.x & 1 : 0;   // the block's 128 rows of the tile (and its rank in the cluster)
    if (sh.bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, ERR_SPLIT);
        return;
    }
    const int64_t total = static_cast<int64_t>(sh.tile0[P.E + 1]) * P.n_tiles;
    const int64_t used = static_cast<int64_t>(sh.tile0[P.E]) * P.n_tiles;   // the rest is zeros
    if (unit >= total) return;
    const Stages<NV, BN, kPair> st(dyn);
    open_block<C::kStages, kPair>(sh, warp, 1, C::kCols);
    constexpr uint32_t tmem = 0;   // the block holds all columns
    volatile uint32_t *dead = &sh.dead;

    if (warp == 0) {
        if (tc::elect()) {
            tc::prefetch_map(&P.tm_a);
            tc::prefetch_map(&P.tm_b);
        }
        int g = 0, it = 0;
        bool ok = true;
        for (int64_t i = unit; i < used && ok; i += units) {
            const Tile t = tile_at<kRows>(P, sh, i, g);
            g = t.g;
            const int row = uniform(static_cast<int>(t.row)) + half * kRowsT;
            const int a_tile = uniform((sh.scale0[g] + t.mt * (kRows / 128) + half) * P.scale_cols);
            const int b_row = uniform(static_cast<int>(g * P.N + static_cast<int64_t>(t.nt) * BN)) + half * C::kRowsB;
            const int b_tile = uniform((g * P.b_scale_rows + t.nt * C::kGroupsB) * P.scale_cols);
            for (int k = 0; k < P.kt; ++k, ++it) {
                const int s = it % C::kStages;
                if (it >= C::kStages && !tc::bar_wait_warp(tc::smem_u32(&sh.empty[s]), (it / C::kStages - 1) & 1, dead)) {
                    ok = false;
                    break;
                }
                const uint32_t own = tc::smem_u32(&sh.full[s]), bar = kPair ? tc::map_to(own, 0) : own;
                auto load = [&](uint32_t dst, const CUtensorMap *tm, int x, int y) {
                    if (kPair) tc::load_2d_pair(dst, tm, x, y, bar);
                    else tc::load_2d(dst, tm, x, y, bar);
                };
                if (tc::elect()) {
                    if (half == 0) tc::bar_expect(own, kPair ? 2 * C::kStageBytes : C::kStageBytes);
                    load(st.a(s), &P.tm_a, k * kStageK, row);
                    load(st.b(s), &P.tm_b, k * kStageK, b_row);
                    load(st.sa(s), &P.tm_sa, 0, a_tile + k * kSc);
#pragma unroll
                    for (int b = 0; b < C::kGroupsB; ++b)
                        load(st.sb(s) + b * kSc * kScaleTile, &P.tm_sb, 0, b_tile + b * P.scale_cols + k * kSc);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (half == 0) settle<C::kStages>(sh.full, it);
            else tc::pause(1000000);   // its copies count on the other block's barriers: time for them to land
        }
    } else if (warp == 1 && half == 0) {
        const int mine = unit < used ? uniform(static_cast<int>((used - unit + units - 1) / units)) : 0;
        int it = 0;
        bool ok = true;
        for (int n = 0; n < mine && ok; ++n) {
            const int a = n % C::kAcc;
            if (n >= C::kAcc && !tc::bar_wait_warp(tc::smem_u32(&sh.acc_empty[a]), (n / C::kAcc - 1) & 1, dead)) break;
            tc::fence_after();
            for (int k = 0; k < P.kt; ++k, ++it) {
                const int s = it % C::kStages;
                if (!tc::bar_wait_warp(tc::smem_u32(&sh.full[s]), (it / C::kStages) & 1, dead)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                if (tc::elect()) {
                    // the last stage holds only what is left of k
                    multiply_stage(st, s, tmem, tmem + a * BN, min(4, (P.k_bytes - k * kStageK) / 32), k == 0);
                    tc::commit<kPair>(tc::smem_u32(&sh.empty[s]));
                    if (k == P.kt - 1) tc::commit<kPair>(tc::smem_u32(&sh.acc_full[a]));
                }
                __syncwarp();
            }
        }
        if (!ok || *dead) settle<C::kStages>(sh.empty, it);
    } else if (warp >= 4) {
        const int q = warp & 3, h = (warp - 4) >> 2;   // lanes 32 q .., column half h
        constexpr int kHalf = BN / 2;
        T *out = static_cast<T *>(P.out);
        const int align = row_align(out, P.N);
        int g = 0, n = 0;
        for (int64_t i = unit; i < total; i += units) {
            const Tile t = tile_at<kRows>(P, sh, i, g);
            g = t.g;
            const int r = half * kRowsT + 32 * q + lane;
            const int64_t c0 = static_cast<int64_t>(t.nt) * BN + h * kHalf;
            T *o = out + (t.row + r) * P.N + c0;
            const int64_t cols = P.N - c0;   // columns from c0 on
            if (g == P.E) {
                if (r < t.rows) zeros(o, kHalf, cols, align);
                continue;
            }
            const int a = n % C::kAcc;
            float ua = 1.0f, ub = 1.0f;
            if (NV) {
                ua = __fdiv_rn(1.0f, tensor_scale(P.amax_a[g]));
                ub = __fdiv_rn(1.0f, tensor_scale(P.amax_b[g]));
            }
            if (!tc::bar_wait_warp(tc::smem_u32(&sh.acc_full[a]), (n / C::kAcc) & 1, dead)) break;
            ++n;
            tc::fence_after();
            drain<kHalf, NV>(tmem + a * BN + h * kHalf + (static_cast<uint32_t>(32 * q) << 16), ua, ub, o, cols, r < t.rows,
                             align, false, [&] {
                                 tc::fence_before();
                                 __syncwarp();
                                 if (lane == 0) {
                                     const uint32_t bar = tc::smem_u32(&sh.acc_empty[a]);
                                     if (kPair) tc::bar_arrive_cluster(tc::map_to(bar, 0));
                                     else tc::bar_arrive(bar);
                                 }
                             });
        }
    }
    close_block<kPair>(sh, warp, C::kCols);
}

// ---------------------------------------------------------- weight gradient
//
//   dw_e[n, k] = u_e sum_r A[r, n] B[r, k] over the rows r of expert e,
// from columnwise copies: per expert [N, Mp_e] and [K, Mp_e], Mp_e the rows padded
// to whole scale blocks, so that the sum runs along the contiguous axis again.
// An expert's pitch is Mp_e codes: a multiple of 8 bytes only (NVFP4), which TMA
// does not take, so three warps bring the stages in with 16- or 8-byte
// asynchronous copies, zeros past the matrices.  Scales past Mp_e are padding that
// nobody wrote: they are masked to zero, since a zero code times a NaN scale would
// still be NaN.

struct WgradParams {
    const uint8_t *a, *b, *sa, *sb;
    const int64_t *split;
    const float *amax_a, *amax_b;
    void *out;
    int64_t M;
    int N, K, E;
    int n_tiles, k_tiles;              // tiles along N (128) and K (BN)
    int64_t a_bytes, b_bytes, sa_bytes, sb_bytes;
    int accumulate;
};

constexpr int kLoadWarps = 3;        // warps 0, 2 and 3; warp 1 multiplies, warps 4-11 drain
constexpr int kLoaders = 32 * kLoadWarps;

struct WgradShared : Shared {
    int64_t pad0[kMaxE + 1];    // padded rows before each expert
    int wide0[kMaxE + 1];       // scale tiles along the rows before each expert
    int order[kMaxE];           // experts by descending size
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Writes to shared memory so far become visible to the tensor core's reads.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// 128 rows of a matrix [n, pitch bytes] from row r0 on, as one loader thread sees
// them.  A warp's copy takes 4 rows in chunks of 16 bytes, or 2 in chunks of 8
// where the pitch is no multiple of 16; the warps take every kLoadWarps-th such
// group.  Chunk c of row r lies at c ^ (r mod 8) of the swizzled stage.
struct CodeLoad {
    const uint8_t *p;   // the thread's chunk of its first row, at k = 0
    int64_t step;       // bytes from a row of the thread to its next
    int row, rows;      // its first row within the 128, and how many rows the matrix has from r0 on
    int c;              // its chunk
    bool wide;          // chunks of 16 bytes
    __device__ CodeLoad(const uint8_t *m, int64_t pitch, int n, int r0, int warp, int lane) {
        wide = pitch % 16 == 0;
        c = wide ? lane & 7 : lane & 15;
        row = wide ? 4 * warp + (lane >> 3) : 2 * warp + (lane >> 4);
        rows = n - r0;
        step = (wide ? 4 : 2) * kLoadWarps * pitch;
        p = m + static_cast<int64_t>(r0 + row) * pitch + c * (wide ? 16 : 8);
    }
    // 128 bytes of k from k0 on (pitch: the matrix' bytes of k), zeros past the matrix.
    __device__ __forceinline__ void operator()(uint32_t stage, int64_t k0, int64_t pitch) const {
        const uint8_t *src = p + k0;
        if (wide) {
            const int left = k0 + 16 * c < pitch ? rows : 0;
#pragma unroll
            for (int j = 0; j < (32 + kLoadWarps - 1) / kLoadWarps; ++j) {
                const int r = row + 4 * kLoadWarps * j;
                if (r < kRowsT) cp_async16(stage + r * 128 + ((c ^ (r & 7)) << 4), r < left ? src : p, r < left ? 16 : 0);
                src += step;
            }
        } else {
            const int left = k0 + 8 * c < pitch ? rows : 0;
#pragma unroll
            for (int j = 0; j < (64 + kLoadWarps - 1) / kLoadWarps; ++j) {
                const int r = row + 2 * kLoadWarps * j;
                if (r < kRowsT)
                    cp_async8(stage + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + 8 * (c & 1), r < left ? src : p, r < left ? 8 : 0);
                src += step;
            }
        }
    }
};

// The scale tiles of a stage for 128-row groups g0 .. of a matrix: tiles
// [c0, c0 + kSc) of each row of tiles, entries from `cols` on as zero.
template <int kSc, int kGroups>
__device__ __forceinline__ void load_scales(uint32_t dst, uint8_t *dst_p, const uint8_t *m, int groups, int g0, int wide,
                                            int c0, int cols, int thread) {
    constexpr int kChunks = kSc * (kScaleTile / 16);   // of a group: contiguous in memory and in the stage
#pragma unroll
    for (int i = thread; i < kGroups * kChunks; i += kLoaders) {
        const int g = i / kChunks, j = (i % kChunks) >> 5;
        const bool in = g0 + g < groups && c0 + j < wide;
        const uint8_t *src = in ? m + (static_cast<int64_t>(g0 + g) * wide + c0) * kScaleTile + (i % kChunks) * 16 : m;
        const int left = cols - 4 * (c0 + j);
        if (!in || left >= 4) {
            cp_async16(dst + i * 16, src, in ? 16 : 0);
        } else {
            const uint32_t keep = left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            uint4 v = *reinterpret_cast<const uint4 *>(src);
            v.x &= keep, v.y &= keep, v.z &= keep, v.w &= keep;
            *reinterpret_cast<uint4 *>(dst_p + i * 16) = v;
        }
    }
}

// Padded rows and scale tiles before each expert, and the experts by descending size.  Every thread of the block.
template <int kBlock> __device__ void scan_wgrad(const WgradParams &P, WgradShared &sh, bool nv) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? P.split[t] : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
    if (t < P.E) sh.row0[t] = m;   // sizes, until sorted
    int64_t rows = m, pad = (m + kBlock - 1) / kBlock * kBlock, wide = (m + 4 * kBlock - 1) / (4 * kBlock);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, d), q = __shfl_up_sync(0xFFFFFFFFu, pad, d),
                      u = __shfl_up_sync(0xFFFFFFFFu, wide, d);
        if (lane >= d) rows += r, pad += q, wide += u;
    }
    if (w < kThreads / 32 && lane == 31) sh.scan[w][0] = rows, sh.scan[w][1] = pad, sh.scan[w][2] = wide;
    const bool any_neg = __syncthreads_or(neg);
    for (int k = 0; k < w && k < kThreads / 32; ++k) rows += sh.scan[k][0], pad += sh.scan[k][1], wide += sh.scan[k][2];
    if (t < P.E) {
        sh.pad0[t + 1] = pad;
        sh.wide0[t + 1] = static_cast<int>(wide);
        int rank = 0;
        for (int k = 0; k < P.E; ++k) rank += sh.row0[k] > m || (sh.row0[k] == m && k < t);
        sh.order[rank] = t;
    }
    if (t == 0) sh.pad0[0] = 0, sh.wide0[0] = 0;
    if (t == P.E - 1) {
        const int64_t codes = nv ? pad / 2 : pad, tiles = wide * kScaleTile;
        sh.bad = any_neg || rows > P.M || codes * P.N > P.a_bytes || codes * P.K > P.b_bytes ||
                 tiles * ((P.N + 127) / 128) > P.sa_bytes || tiles * ((P.K + 127) / 128) > P.sb_bytes;
    }
    __syncthreads();
}

// A tile of the weight gradients.  A unit's r-th tile goes back and forth over the
// units (u, then units - 1 - u, ..) in the order of descending experts, so that
// long and short sums even out.
struct WTile {
    int e, nt, kt;
    int64_t pad0, rows;   // padded rows before the expert, and its own
};
__device__ __forceinline__ int64_t wgrad_tile(int64_t r, int unit, int units) {
    return r * units + ((r & 1) ? units - 1 - unit : unit);
}
__device__ __forceinline__ WTile wtile_at(const WgradParams &P, const WgradShared &sh, int64_t i) {
    const int per = P.n_tiles * P.k_tiles;
    WTile t;
    const int x = static_cast<int>(i / per), j = static_cast<int>(i - static_cast<int64_t>(x) * per);
    t.e = sh.order[x];
    t.nt = j / P.k_tiles;
    t.kt = j - t.nt * P.k_tiles;
    t.pad0 = sh.pad0[t.e];
    t.rows = sh.pad0[t.e + 1] - t.pad0;
    return t;
}

template <bool NV, int BN, bool kPair, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_wgrad(const __grid_constant__ WgradParams P) {
    using C = Cfg<NV, BN, kPair>;
    extern __shared__ uint8_t dyn[];
    __shared__ WgradShared sh;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kBlock = NV ? 16 : 32, kSc = C::kSc, kDepth = C::kStages - 2;
    constexpr int kRows = kPair ? 2 * kRowsT : kRowsT;
    scan_wgrad<kBlock>(P, sh, NV);
    if (sh.bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, ERR_SPLIT);
        return;
    }
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
    const int half = kPair ? blockIdx.x & 1 : 0;
    const int64_t total = static_cast<int64_t>(P.E) * P.n_tiles * P.k_tiles;
    const Stages<NV, BN, kPair> st(dyn);
    open_block<C::kStages, kPair>(sh, warp, (kPair ? 2 : 1) * kLoadWarps, C::kCols);
    constexpr uint32_t tmem = 0;   // the block holds all columns
    volatile uint32_t *dead = &sh.dead;

    if (warp == 1) {
        if (half == 0) {
            int it = 0, n = 0;
            bool ok = true;
            for (int64_t r = 0;; ++r) {
                const int64_t i = wgrad_tile(r, unit, units);
                if (i >= total) {
                    if (r * units >= total) break;
                    continue;
                }
                const WTile t = wtile_at(P, sh, i);
                const int len = uniform(static_cast<int>(NV ? t.rows / 2 : t.rows));
                if (len == 0) continue;
                const int a = n % C::kAcc, kt = (len + kStageK - 1) / kStageK;
                if (n >= C::kAcc && !tc::bar_wait_warp(tc::smem_u32(&sh.acc_empty[a]), (n / C::kAcc - 1) & 1, dead)) break;
                ++n;
                tc::fence_after();
                for (int k = 0; k < kt; ++k, ++it) {
                    const int s = it % C::kStages;
                    if (!tc::bar_wait_warp(tc::smem_u32(&sh.full[s]), (it / C::kStages) & 1, dead)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    if (tc::elect()) {
                        multiply_stage(st, s, tmem, tmem + a * BN, min(4, (len - k * kStageK + 31) / 32), k == 0);
                        tc::commit<kPair>(tc::smem_u32(&sh.empty[s]));
                        if (k == kt - 1) tc::commit<kPair>(tc::smem_u32(&sh.acc_full[a]));
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            if (!ok || *dead) settle<C::kStages>(sh.empty, it);
        }
    } else if (warp < 4) {
        const int loader = warp == 0 ? 0 : warp - 1, thread = 32 * loader + lane;
        const int n128 = (P.N + 127) / 128, k128 = (P.K + 127) / 128;
        auto arrive = [&](int j) {   // stage j's copies of this warp have landed
            fence_async();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = tc::smem_u32(&sh.full[j % C::kStages]);
                if (kPair) tc::bar_arrive_cluster(tc::map_to(bar, 0));
                else tc::bar_arrive(bar);
            }
        };
        int it = 0;
        bool ok = true;
        for (int64_t r = 0; ok; ++r) {
            const int64_t i = wgrad_tile(r, unit, units);
            if (i >= total) {
                if (r * units >= total) break;
                continue;
            }
            const WTile t = wtile_at(P, sh, i);
            const int64_t pitch = NV ? t.rows / 2 : t.rows, first = NV ? t.pad0 / 2 : t.pad0;
            const int wide = sh.wide0[t.e + 1] - sh.wide0[t.e], cols = static_cast<int>(t.rows / kBlock);
            const uint8_t *sa = P.sa + static_cast<int64_t>(sh.wide0[t.e]) * n128 * kScaleTile;
            const uint8_t *sb = P.sb + static_cast<int64_t>(sh.wide0[t.e]) * k128 * kScaleTile;
            const CodeLoad load_a(P.a + first * P.N, pitch, P.N, t.nt * kRows + half * kRowsT, loader, lane);
            const CodeLoad load_b(P.b + first * P.K, pitch, P.K, t.kt * BN + half * C::kRowsB, loader, lane);
            for (int64_t k = 0; k < pitch; k += kStageK, ++it) {
                const int s = it % C::kStages;
                if (it >= C::kStages && !tc::bar_wait_warp(tc::smem_u32(&sh.empty[s]), (it / C::kStages - 1) & 1, dead)) {
                    ok = false;
                    break;
                }
                load_a(st.a(s), k, pitch);
                load_b(st.b(s), k, pitch);
                const int c0 = static_cast<int>(k / kStageK) * kSc;
                uint8_t *p = dyn + (st.sa(s) - tc::smem_u32(dyn));
                load_scales<kSc, 1>(st.sa(s), p, sa, n128, t.nt * (kRows / 128) + half, wide, c0, cols, thread);
                load_scales<kSc, C::kGroupsB>(st.sb(s), p + C::kBytesSA, sb, k128, t.kt * C::kGroupsB, wide, c0, cols, thread);
                cp_commit();
                if (it >= kDepth) {   // the stage kDepth before this one has arrived
                    cp_wait<kDepth>();
                    arrive(it - kDepth);
                }
            }
        }
        cp_wait<0>();
        if (ok)
            for (int j = it < kDepth ? 0 : it - kDepth; j < it; ++j) arrive(j);
    } else {
        const int q = warp & 3, h = (warp - 4) >> 2;
        constexpr int kHalf = BN / 2;
        T *out = static_cast<T *>(P.out);
        const int align = row_align(out, P.K);
        const bool add = P.accumulate != 0;
        int n = 0;
        for (int64_t r = 0;; ++r) {
            const int64_t i = wgrad_tile(r, unit, units);
            if (i >= total) {
                if (r * units >= total) break;
                continue;
            }
            const WTile t = wtile_at(P, sh, i);
            const int row = t.nt * kRows + half * kRowsT + 32 * q + lane, c0 = t.kt * BN + h * kHalf;
            T *o = out + (static_cast<int64_t>(t.e) * P.N + row) * P.K + c0;
            const int64_t left = static_cast<int64_t>(P.K) - c0;
            if (t.rows == 0) {   // no rows: a zero gradient
                if (row < P.N && !add) zeros(o, kHalf, left, align);
                continue;
            }
            const int a = n % C::kAcc;
            float ua = 1.0f, ub = 1.0f;
            if (NV) {
                ua = __fdiv_rn(1.0f, tensor_scale(P.amax_a[t.e]));
                ub = __fdiv_rn(1.0f, tensor_scale(P.amax_b[t.e]));
            }
            if (!tc::bar_wait_warp(tc::smem_u32(&sh.acc_full[a]), (n / C::kAcc) & 1, dead)) break;
            ++n;
            tc::fence_after();
            drain<kHalf, NV>(tmem + a * BN + h * kHalf + (static_cast<uint32_t>(32 * q) << 16), ua, ub, o, left, row < P.N,
                             align, add, [&] {
                                 tc::fence_before();
                                 __syncwarp();
                                 if (lane == 0) {
                                     const uint32_t bar = tc::smem_u32(&sh.acc_empty[a]);
                                     if (kPair) tc::bar_arrive_cluster(tc::map_to(bar, 0));
                                     else tc::bar_arrive(bar);
                                 }
                             });
        }
    }
    close_block<kPair>(sh, warp, C::kCols);
}

// -------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
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

// Number of SMs of the current device (0: a CUDA error), asked once per device.
int sm_count() {
    static std::mutex mu;
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!n[dev] && cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n[dev];
}

// A persistent launch of at most `want` blocks (kPair: pairs of blocks), as many as run at once.
template <bool kPair, typename P>
gsa_status launch(void (*kernel)(P), const P &params, int threads, size_t smem, int64_t want, cudaStream_t s, int &pairs,
                  std::once_flag &once) {
    const int sms = sm_count();
    if (!sms) return GSA_ERR_CUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return GSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kPair ? 2 : 1;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (kPair)   // the machine's clusters may not fill every SM
        std::call_once(once, [&] {
            cfg.gridDim = dim3(2 * (sms / 2));
            if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess) pairs = 0;
        });
    if (kPair && pairs <= 0) return GSA_ERR_CUDA;
    const int64_t units = kPair ? pairs : sms, n = want < units ? want : units;
    cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * n : n));
    return cudaLaunchKernelEx(&cfg, kernel, params) == cudaSuccess ? GSA_OK : GSA_ERR_CUDA;
}

template <bool NV, int BN, bool kPair, typename T>
gsa_status launch_gemm(const GemmParams &P, int64_t tiles, cudaStream_t s) {
    static std::once_flag once;
    static int pairs = 0;
    return launch<kPair, GemmParams>(grouped_gemm<NV, BN, kPair, T>, P, kThreads, Cfg<NV, BN, kPair>::kSmem, tiles * P.n_tiles,
                                     s, pairs, once);
}

template <bool NV, int BN, bool kPair, typename T> gsa_status launch_wgrad(const WgradParams &P, cudaStream_t s) {
    static std::once_flag once;
    static int pairs = 0;
    return launch<kPair, WgradParams>(grouped_wgrad<NV, BN, kPair, T>, P, kThreads, Cfg<NV, BN, kPair>::kSmem,
                                      static_cast<int64_t>(P.E) * P.n_tiles * P.k_tiles, s, pairs, once);
}

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
    if (M == 0) {
        gsa::set_last_launches(0);
        return GSA_OK;
    }
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
    const int BN = 256;
    const bool pair = M >= 64 * E;
    const int sc = nv ? 4 : 1;
    if (!map_codes(&P.tm_a, a->data, M, k_bytes, kRowsT) || !map_codes(&P.tm_b, b->data, E * N, k_bytes, pair ? BN / 2 : BN) ||
        !map_scales(&P.tm_sa, a->scale, a_rows * cols, sc) || !map_scales(&P.tm_sb, b->scale, E * n128 * cols, sc))
        return GSA_ERR_CUDA;
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
    auto go = [&](auto fmt, auto two, auto type) {
        return launch_gemm<decltype(fmt)::value, BN, decltype(two)::value, decltype(type)>(P, tiles, s);
    };
    auto typed = [&](auto fmt, auto two) { return out_dtype == GSA_BF16 ? go(fmt, two, __nv_bfloat16()) : go(fmt, two, float()); };
    auto sized = [&](auto fmt) { return pair ? typed(fmt, std::true_type()) : typed(fmt, std::false_type()); };
    st = nv ? sized(std::true_type()) : sized(std::false_type());
    if (st == GSA_OK) gsa::set_last_launches(1);
    return st;
}

gsa_status gsa_grouped_gemm_wgrad(const gsa_qin *a, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E,
                                  int64_t M, int64_t N, int64_t K, int32_t recipe_kind, void *out, int32_t out_dtype,
                                  int32_t accumulate, gsa_stream_t stream) {
    if (!a || !b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (out_dtype != GSA_BF16 && out_dtype != GSA_FP32) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    if (E > kMaxE || M >= (int64_t(1) << 31) - 256 * 64 || N >= (int64_t(1) << 30) || K >= (int64_t(1) << 30))
        return GSA_ERR_UNSUPPORTED;
    if (!a->data || !a->scale || !b->data || !b->scale || !split_sizes_dev || !out) return GSA_ERR_INVALID_ARG;
    if (nv && (!a->amax || !b->amax)) return GSA_ERR_INVALID_ARG;
    if (!aligned(a->data, 16) || !aligned(a->scale, 16) || !aligned(b->data, 16) || !aligned(b->scale, 16) ||
        !aligned(out, 16) || !aligned(split_sizes_dev, 8) || !aligned(a->amax, 4) || !aligned(b->amax, 4))
        return GSA_ERR_ALIGNMENT;
    // an expert's codes start on 16 bytes: its padded rows (a multiple of the block) times the width
    if ((nv ? N * 8 : N * 32) % 16 != 0 || (nv ? K * 8 : K * 32) % 16 != 0) return GSA_ERR_UNSUPPORTED;

    WgradParams P;
    std::memset(&P, 0, sizeof(P));
    P.a = static_cast<const uint8_t *>(a->data);
    P.b = static_cast<const uint8_t *>(b->data);
    P.sa = static_cast<const uint8_t *>(a->scale);
    P.sb = static_cast<const uint8_t *>(b->scale);
    P.split = split_sizes_dev;
    P.amax_a = a->amax;
    P.amax_b = b->amax;
    P.out = out;
    P.M = M;
    P.N = static_cast<int>(N);
    P.K = static_cast<int>(K);
    P.E = static_cast<int>(E);
    const bool pair = N > 128 && K > 128;
    const int tile = pair ? 256 : 128;
    P.n_tiles = static_cast<int>((N + tile - 1) / tile);
    P.k_tiles = static_cast<int>((K + tile - 1) / tile);
    P.a_bytes = a->data_bytes;
    P.b_bytes = b->data_bytes;
    P.sa_bytes = a->scale_bytes;
    P.sb_bytes = b->scale_bytes;
    P.accumulate = accumulate != 0;
    if (static_cast<int64_t>(P.n_tiles) * P.k_tiles >= (int64_t(1) << 31)) return GSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    gsa_status st;
    auto typed = [&](auto fmt, auto type) {
        return pair ? launch_wgrad<decltype(fmt)::value, 256, true, decltype(type)>(P, s)
                    : launch_wgrad<decltype(fmt)::value, 128, false, decltype(type)>(P, s);
    };
    auto sized = [&](auto fmt) { return out_dtype == GSA_BF16 ? typed(fmt, __nv_bfloat16()) : typed(fmt, float()); };
    st = nv ? sized(std::true_type()) : sized(std::false_type());
    if (st == GSA_OK) gsa::set_last_launches(1);
    return st;
}

gsa_status gsa_grouped_gemm_status(gsa_stream_t stream) {
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return GSA_ERR_CUDA;
    uint32_t err = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&err, g_status, 4) != cudaSuccess) return GSA_ERR_CUDA;
    if (err && cudaMemcpyToSymbol(g_status, &zero, 4) != cudaSuccess) return GSA_ERR_CUDA;
    if (err & ERR_SPLIT) return GSA_ERR_INVALID_ARG;
    return err ? GSA_ERR_DEVICE_TIMEOUT : GSA_OK;
}

}  // extern "C"
