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

template <bool NV, int BN> struct Cfg {
    static constexpr int kSc = Fmt<NV>::kScaleTiles;
    static constexpr int kBytesA = kRowsT * kStageK, kBytesB = BN * kStageK;
    static constexpr int kGroupsB = BN / 128;
    static constexpr int kBytesSA = kSc * kScaleTile, kBytesSB = kGroupsB * kSc * kScaleTile;
    static constexpr int kStageBytes = kBytesA + kBytesB + kBytesSA + kBytesSB;
    static constexpr int kStride = (kStageBytes + 1023) / 1024 * 1024;   // stages start on the swizzle's period
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kAcc = BN == 256 ? 1 : 2;       // accumulators in tensor memory
    static constexpr int kScCols = 4 * kSc * (1 + kGroupsB);   // scale columns of a stage
    static constexpr int kCols = 512;
    static_assert(kAcc * BN + kStages * kScCols <= kCols, "tensor memory");
    static constexpr int kSmem = kStages * kStride + 1024;
};

struct Shared {
    int64_t row0[kMaxE + 2];    // first row of each group; group E: rows that no expert has
    int tile0[kMaxE + 2];       // first row tile of each group (in tiles of all column tiles: times n_tiles)
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2];
    uint32_t tmem;
    uint32_t dead, bad;
    int64_t scan[kThreads / 32][2];
};

// Group bounds from the device split: rows and row tiles before each group.  Every thread of the block.
// A negative size, a sum above M or more scale tiles than A's buffer holds sets sh.bad.
__device__ void scan_split(const GemmParams &P, Shared &sh) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? P.split[t] : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
    int64_t rows = m, tiles = (m + kRowsT - 1) / kRowsT;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, d), q = __shfl_up_sync(0xFFFFFFFFu, tiles, d);
        if (lane >= d) rows += r, tiles += q;
    }
    if (lane == 31) sh.scan[w][0] = rows, sh.scan[w][1] = tiles;
    const bool any_neg = __syncthreads_or(neg);
    int64_t r0 = 0, q0 = 0;
    for (int k = 0; k < w; ++k) r0 += sh.scan[k][0], q0 += sh.scan[k][1];
    rows += r0, tiles += q0;
    if (t < P.E) sh.row0[t + 1] = rows, sh.tile0[t + 1] = static_cast<int>(tiles);
    if (t == 0) sh.row0[0] = 0, sh.tile0[0] = 0;
    __syncthreads();
    if (t == 0) {
        const int64_t sum = sh.row0[P.E];
        sh.bad = any_neg || sum > P.M || sh.tile0[P.E] > P.a_scale_tiles;
        sh.row0[P.E + 1] = P.M;
        sh.tile0[P.E + 1] = sh.tile0[P.E] + static_cast<int>((P.M - (sum > P.M ? P.M : sum) + kRowsT - 1) / kRowsT);
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

// Tile number i, searching from group g on (tile numbers only grow).
__device__ __forceinline__ Tile tile_at(const GemmParams &P, const Shared &sh, int64_t i, int g) {
    const int q = static_cast<int>(i / P.n_tiles);
    while (q >= sh.tile0[g + 1]) ++g;
    Tile t;
    t.g = g;
    t.nt = static_cast<int>(i - static_cast<int64_t>(q) * P.n_tiles);
    t.mt = q - sh.tile0[g];
    t.row = sh.row0[g] + static_cast<int64_t>(t.mt) * kRowsT;
    const int64_t left = sh.row0[g + 1] - t.row;
    t.rows = left < kRowsT ? static_cast<int>(left) : kRowsT;
    return t;
}

__device__ __forceinline__ void store_row(__nv_bfloat16 *o, const float *v, int n, bool wide) {
    if (wide && n == 8) {
        uint4 w;
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        memcpy(&w, h, 16);
        *reinterpret_cast<uint4 *>(o) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) o[i] = __float2bfloat16_rn(v[i]);
    }
}

__device__ __forceinline__ void store_row(float *o, const float *v, int n, bool wide) {
    if (wide && n == 8) {
        *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) o[i] = v[i];
    }
}

template <bool NV, int BN, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_gemm(const __grid_constant__ GemmParams P) {
    using C = Cfg<NV, BN>;
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    scan_split(P, sh);
    if (sh.bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, ERR_SPLIT);
        return;
    }
    const int64_t total = static_cast<int64_t>(sh.tile0[P.E + 1]) * P.n_tiles;
    if (static_cast<int64_t>(blockIdx.x) >= total) return;
    const uint32_t base = (tc::smem_u32(dyn) + 1023u) & ~1023u;   // the swizzle pattern repeats every 1024 bytes
    auto sA = [&](int s) { return base + s * C::kStride; };
    auto sB = [&](int s) { return sA(s) + C::kBytesA; };
    auto sSA = [&](int s) { return sB(s) + C::kBytesB; };
    auto sSB = [&](int s) { return sSA(s) + C::kBytesSA; };
    if (threadIdx.x == 0) {
        sh.dead = 0;
        for (int s = 0; s < C::kStages; ++s) {
            tc::bar_init(tc::smem_u32(&sh.full[s]), 1);
            tc::bar_init(tc::smem_u32(&sh.empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::bar_init(tc::smem_u32(&sh.acc_full[a]), 1);
            tc::bar_init(tc::smem_u32(&sh.acc_empty[a]), kEpiWarps);
        }
        tc::bar_init_fence();
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_u32(&sh.tmem), C::kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *dead = &sh.dead;
    constexpr int kSc = C::kSc;

    if (warp == 0 && lane == 0) {
        tc::prefetch_map(&P.tm_a);
        tc::prefetch_map(&P.tm_b);
        int g = 0, it = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
            const Tile t = tile_at(P, sh, i, g);
            g = t.g;
            if (g == P.E) break;   // only zeros from here on
            const int a_tile = (sh.tile0[g] + t.mt) * P.scale_cols;
            for (int k = 0; k < P.kt; ++k, ++it) {
                const int s = it % C::kStages;
                if (it >= C::kStages && !tc::bar_wait(tc::smem_u32(&sh.empty[s]), (it / C::kStages - 1) & 1, dead)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = tc::smem_u32(&sh.full[s]);
                tc::bar_expect(bar, C::kStageBytes);
                tc::load_2d(sA(s), &P.tm_a, k * kStageK, static_cast<int>(t.row), bar);
                tc::load_2d(sB(s), &P.tm_b, k * kStageK, static_cast<int>(g * P.N + static_cast<int64_t>(t.nt) * BN), bar);
                tc::load_2d(sSA(s), &P.tm_sa, 0, a_tile + k * kSc, bar);
#pragma unroll
                for (int b = 0; b < C::kGroupsB; ++b)
                    tc::load_2d(sSB(s) + b * kSc * kScaleTile, &P.tm_sb, 0,
                                (g * P.b_scale_rows + t.nt * C::kGroupsB + b) * P.scale_cols + k * kSc, bar);
            }
        }
        // a block that gives up waits for its copies in flight before it leaves
        if (!ok) {
            uint32_t none = 0;
            const int first = it < C::kStages ? 0 : it - C::kStages;
            for (int j = first; j < it; ++j) tc::bar_wait(tc::smem_u32(&sh.full[j % C::kStages]), (j / C::kStages) & 1, &none);
        }
    } else if (warp == 1 && lane == 0) {
        constexpr uint32_t idesc = tc::idesc_block_scaled(NV, kRowsT, BN);
        int g = 0, it = 0, n = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x, ++n) {
            const Tile t = tile_at(P, sh, i, g);
            g = t.g;
            if (g == P.E) break;
            const int a = n % C::kAcc;
            if (n >= C::kAcc && !tc::bar_wait(tc::smem_u32(&sh.acc_empty[a]), (n / C::kAcc - 1) & 1, dead)) break;
            tc::fence_after();
            const uint32_t d = tmem + a * BN;
            for (int k = 0; k < P.kt; ++k, ++it) {
                const int s = it % C::kStages;
                if (!tc::bar_wait(tc::smem_u32(&sh.full[s]), (it / C::kStages) & 1, dead)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t sfa = tmem + C::kAcc * BN + s * C::kScCols, sfb = sfa + 4 * kSc;
#pragma unroll
                for (int j = 0; j < kSc; ++j) {
                    tc::copy_scales(sfa + 4 * j, tc::desc_scales(sSA(s) + j * kScaleTile));
#pragma unroll
                    for (int b = 0; b < C::kGroupsB; ++b)
                        tc::copy_scales(sfb + 4 * (j * C::kGroupsB + b), tc::desc_scales(sSB(s) + (b * kSc + j) * kScaleTile));
                }
                // steps of 32 bytes of k; the last stage holds only what is left
                const int steps = min(4, (P.k_bytes - k * kStageK) / 32);
                for (int j = 0; j < steps; ++j) {
                    const uint64_t da = tc::desc_sw128(sA(s) + 32 * j), db = tc::desc_sw128(sB(s) + 32 * j);
                    const bool add = k > 0 || j > 0;
                    if (NV) tc::mma_nvf4(d, da, db, idesc, sfa + 4 * j, sfb + 4 * C::kGroupsB * j, add);
                    else tc::mma_mxf8(d, da, db, idesc | tc::idesc_scale_id(j), sfa, sfb, add);
                }
                tc::commit(tc::smem_u32(&sh.empty[s]));
            }
            if (ok) tc::commit(tc::smem_u32(&sh.acc_full[a]));
        }
        if (!ok || *dead) {   // the products issued so far end before the memory they read goes
            uint32_t none = 0;
            const int first = it < C::kStages ? 0 : it - C::kStages;
            for (int j = first; j < it; ++j) tc::bar_wait(tc::smem_u32(&sh.empty[j % C::kStages]), (j / C::kStages) & 1, &none);
        }
    } else if (warp >= 4) {
        const int q = warp & 3, h = (warp - 4) >> 2;   // lanes 32 q .., column half h
        constexpr int kHalf = BN / 2;
        T *out = static_cast<T *>(P.out);
        const bool wide = (P.N * sizeof(T)) % 16 == 0;
        int g = 0, n = 0;
        for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
            const Tile t = tile_at(P, sh, i, g);
            g = t.g;
            const int r = 32 * q + lane;
            const int64_t c0 = static_cast<int64_t>(t.nt) * BN + h * kHalf;
            T *o = out + (t.row + r) * P.N + c0;
            const int64_t cols = P.N - c0;   // columns from c0 on
            if (g == P.E) {
                const float zero[8] = {};
                if (r < t.rows)
                    for (int c = 0; c < kHalf && c < cols; c += 8)
                        store_row(o + c, zero, static_cast<int>(cols - c < 8 ? cols - c : 8), wide);
                continue;
            }
            const int a = n % C::kAcc;
            if (!tc::bar_wait(tc::smem_u32(&sh.acc_full[a]), (n / C::kAcc) & 1, dead)) break;
            ++n;
            __syncwarp();
            tc::fence_after();
            float ua = 1.0f, ub = 1.0f;
            if (NV) {
                ua = __fdiv_rn(1.0f, tensor_scale(P.amax_a[g]));
                ub = __fdiv_rn(1.0f, tensor_scale(P.amax_b[g]));
            }
#pragma unroll
            for (int c = 0; c < kHalf; c += 64) {
                uint32_t v[64];
                tc::tmem_ld64(tmem + a * BN + h * kHalf + c + (static_cast<uint32_t>(32 * q) << 16), v);
                if (c + 64 == kHalf) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::bar_arrive(tc::smem_u32(&sh.acc_empty[a]));
                }
                if (r < t.rows) {
#pragma unroll
                    for (int j = 0; j < 64; j += 8) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[j + e]) * ua * ub;
                        const int64_t left = cols - c - j;
                        if (left > 0) store_row(o + c + j, f, static_cast<int>(left < 8 ? left : 8), wide);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free(tmem, C::kCols);
    }
    if (threadIdx.x == 0 && sh.dead) atomicOr(&g_status, ERR_TIMEOUT);
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

template <bool NV, int BN, typename T>
gsa_status launch(const GemmParams &P, int64_t tiles, cudaStream_t s) {
    const int sms = sm_count();
    if (!sms) return GSA_ERR_CUDA;
    auto k = grouped_gemm<NV, BN, T>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NV, BN>::kSmem) != cudaSuccess)
        return GSA_ERR_CUDA;
    const int64_t grid = tiles * P.n_tiles < sms ? tiles * P.n_tiles : sms;
    k<<<static_cast<unsigned>(grid), kThreads, Cfg<NV, BN>::kSmem, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? GSA_OK : GSA_ERR_CUDA;
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
    const int sc = nv ? 4 : 1;
    if (!map_codes(&P.tm_a, a->data, M, k_bytes, kRowsT) || !map_codes(&P.tm_b, b->data, E * N, k_bytes, BN) ||
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
    if (nv) st = out_dtype == GSA_BF16 ? launch<true, 256, __nv_bfloat16>(P, tiles, s) : launch<true, 256, float>(P, tiles, s);
    else st = out_dtype == GSA_BF16 ? launch<false, 256, __nv_bfloat16>(P, tiles, s) : launch<false, 256, float>(P, tiles, s);
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
