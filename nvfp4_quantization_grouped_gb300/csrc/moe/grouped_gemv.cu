// grouped_gemv.cu -- products of a few unquantized rows an expert with its block-scaled
// (MXFP8 / NVFP4) weights, plain and gated, with their C entry points.
//
//   out[r, n] = u_e sum_k x[r, k] B_e[n, k],   rows r of expert e
//   y[r, n] = p_r act(u_g sum_k x[r, k] B_e[n, k], u_l sum_k x[r, k] B_e[N + n, k])
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <cstring>
#include <type_traits>

#include "glu_act.cuh"
#include "gsa.h"
#include "moe/status.cuh"

namespace {

constexpr int kMaxE = 256, kThreads = 256, kScaleTile = 512;

struct GemvParams {
    const void *x;
    const uint8_t *codes, *scales;
    const float *amax;
    const int64_t *split;   // nullptr: one expert has all rows
    const float *probs;
    void *out;
    uint32_t *status;
    int64_t M, N, K;
    int E, x_type, out_type;
    int scale_cols, scale_rows, up_tiles;   // scale tiles along k; of an expert along its rows; from a gate row to its linear row
    int b_groups;
    glu::Act act;
};

struct Shared {
    int row0[kMaxE + 2];
    int64_t scan[kThreads / 32];
    uint32_t bad;
};

__device__ void scan_rows(const GemvParams &P, Shared &sh) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? (P.split ? P.split[t] : P.M) : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
    int64_t rows = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, d);
        if (lane >= d) rows += r;
    }
    if (lane == 31) sh.scan[w] = rows;
    const bool any_neg = __syncthreads_or(neg);
    for (int k = 0; k < w; ++k) rows += sh.scan[k];
    if (t < P.E) sh.row0[t + 1] = static_cast<int>(rows < P.M ? rows : P.M);
    if (t == 0) sh.row0[0] = 0;
    if (t == P.E - 1) sh.bad = any_neg || rows > P.M;
    __syncthreads();
}

__device__ __forceinline__ float unit_of(float amax) {
    if (amax == 0.0f) return 1.0f;
    const float s = __fdiv_rn(2688.0f, amax);
    return __fdiv_rn(1.0f, s <= 3.402823466e38f ? s : 3.402823466e38f);
}

__device__ __forceinline__ float element(const void *p, int type, int64_t i) {
    if (type == GSA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    if (type == GSA_FP16) return __half2float(static_cast<const __half *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void put(void *p, int type, int64_t i, float v) {
    if (type == GSA_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else if (type == GSA_FP16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float e4m3(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(__half(h));
}

__device__ __forceinline__ float e8m0(uint8_t c) {
    return __uint_as_float(c == 255 ? 0x7FFFFFFFu : c == 0 ? 0x00400000u : static_cast<uint32_t>(c) << 23);
}

// Weight (row of all, row of its scale tile, k), without the unit.
template <bool NV> __device__ __forceinline__ float weight(const GemvParams &P, int64_t row, int64_t tile_row, int lr, int64_t k) {
    constexpr int B = NV ? 16 : 32;
    const int64_t c = k / B;
    const uint8_t s = P.scales[(tile_row * P.scale_cols + c / 4) * kScaleTile + 16 * (lr % 32) + 4 * (lr / 32) + c % 4];
    if (!NV) return e4m3(P.codes[row * P.K + k]) * e8m0(s);
    const int code = P.codes[row * (P.K / 2) + k / 2] >> (k & 1 ? 4 : 0) & 15, m = code & 7;
    const float v = m < 2 ? 0.5f * m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return (code & 8 ? -v : v) * e4m3(s);
}

__device__ __forceinline__ float gated(const glu::Act &A, float g, float u) {
    const float2 a = make_float2(g, g), b = make_float2(u, u);
    return A.clamped ? glu::value<true>(A, a, b).x : glu::value<false>(A, a, b).x;
}

constexpr int kRowsAtOnce = 8;

template <bool NV, bool kGlu> __global__ void __launch_bounds__(kThreads) gemv(const __grid_constant__ GemvParams P) {
    __shared__ Shared sh;
    scan_rows(P, sh);
    if (sh.bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.status, gemm_status::ERR_SPLIT);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t warp = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5, warps = gridDim.x * static_cast<int64_t>(kThreads / 32);
    const int64_t sides = kGlu ? 2 : 1;
    for (int64_t i = warp; i < P.E * P.N; i += warps) {
        const int e = static_cast<int>(i / P.N);
        const int64_t n = i - e * P.N;
        for (int r0 = sh.row0[e]; r0 < sh.row0[e + 1]; r0 += kRowsAtOnce) {
            const int rows = min(kRowsAtOnce, sh.row0[e + 1] - r0);
            float acc[2][kRowsAtOnce] = {};
            for (int64_t k = lane; k < P.K; k += 32) {
                float w[2];
                for (int s = 0; s < sides; ++s)
                    w[s] = weight<NV>(P, (e * sides + s) * P.N + n, static_cast<int64_t>(e) * P.scale_rows + s * P.up_tiles + n / 128, n % 128, k);
#pragma unroll
                for (int r = 0; r < kRowsAtOnce; ++r) {
                    if (r >= rows) break;
                    const float x = element(P.x, P.x_type, (r0 + r) * P.K + k);
                    for (int s = 0; s < sides; ++s) acc[s][r] = __fmaf_rn(x, w[s], acc[s][r]);
                }
            }
            for (int r = 0; r < rows; ++r) {
                float v[2];
                for (int s = 0; s < sides; ++s) {
                    v[s] = acc[s][r];
                    for (int d = 16; d > 0; d >>= 1) v[s] += __shfl_xor_sync(0xFFFFFFFFu, v[s], d);
                    if (NV) v[s] *= unit_of(P.amax[e * P.b_groups + (s ? P.b_groups - 1 : 0)]);
                }
                const float p = P.probs ? P.probs[r0 + r] : 1.0f;
                if (lane == 0) put(P.out, P.out_type, (r0 + r) * P.N + n, kGlu ? p * gated(P.act, v[0], v[1]) : v[0]);
            }
        }
    }
    const int64_t first = sh.row0[P.E] * P.N;   // rows that no expert has
    for (int64_t i = first + blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < P.M * P.N; i += gridDim.x * static_cast<int64_t>(kThreads))
        put(P.out, P.out_type, i, 0.0f);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

gsa_status cuda_error() {
    cudaGetLastError();
    return GSA_ERR_CUDA;
}

bool known_type(int32_t t) { return t == GSA_BF16 || t == GSA_FP16 || t == GSA_FP32; }

gsa_status run_gemv(GemvParams &P, bool glu, const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split, int64_t E, int64_t M, int64_t N,
                    int64_t K, int32_t recipe_kind, int32_t b_groups, void *out, int32_t out_dtype, gsa_stream_t stream) {
    if (!b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (!known_type(x_dtype) || !known_type(out_dtype) || (b_groups != 1 && b_groups != 2)) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    const int64_t sides = glu ? 2 : 1;
    if (E > kMaxE || K % 64 != 0 || K > 65536 || M >= (int64_t(1) << 31) - 256 || N >= (int64_t(1) << 30) / E - 256) return GSA_ERR_UNSUPPORTED;
    if (glu && b_groups == 1 && N % 128 != 0) return GSA_ERR_UNSUPPORTED;
    if (M == 0) return GSA_OK;
    if (!x || !b->data || !b->scale || !out || (!split && E != 1) || (nv && !b->amax)) return GSA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(b->data, 16) || !aligned(b->scale, 16) || !aligned(out, 16) || !aligned(split, 8) || !aligned(b->amax, 4) ||
        !aligned(P.probs, 4))
        return GSA_ERR_ALIGNMENT;
    const int64_t n128 = (N + 127) / 128, cols = (K / (nv ? 16 : 32) + 3) / 4;
    if (b->data_bytes < E * sides * N * (nv ? K / 2 : K) || b->scale_bytes < E * sides * n128 * cols * kScaleTile) return GSA_ERR_INVALID_ARG;
    P.x = x;
    P.codes = static_cast<const uint8_t *>(b->data);
    P.scales = static_cast<const uint8_t *>(b->scale);
    P.amax = b->amax;
    P.split = split;
    P.out = out;
    P.M = M, P.N = N, P.K = K;
    P.E = static_cast<int>(E);
    P.x_type = x_dtype, P.out_type = out_dtype;
    P.scale_cols = static_cast<int>(cols);
    P.scale_rows = static_cast<int>(sides * n128);
    P.up_tiles = static_cast<int>(n128);
    P.b_groups = b_groups;
    P.status = gemm_status::word();
    if (!P.status) return cuda_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = 152 * 4;
    if (nv && glu) gemv<true, true><<<grid, kThreads, 0, s>>>(P);
    else if (nv) gemv<true, false><<<grid, kThreads, 0, s>>>(P);
    else if (glu) gemv<false, true><<<grid, kThreads, 0, s>>>(P);
    else gemv<false, false><<<grid, kThreads, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? GSA_OK : GSA_ERR_CUDA;
}

}  // namespace

extern "C" {

gsa_status gsa_grouped_gemv(const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M, int64_t N,
                            int64_t K, int32_t recipe_kind, void *out, int32_t out_dtype, gsa_stream_t stream) {
    GemvParams P;
    std::memset(&P, 0, sizeof(P));
    return run_gemv(P, false, x, x_dtype, b, split_sizes_dev, E, M, N, K, recipe_kind, 1, out, out_dtype, stream);
}

gsa_status gsa_grouped_glu_gemv(const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M, int64_t N,
                                int64_t K, int32_t recipe_kind, int32_t act_kind, const gsa_act_params *act_params, const float *probs,
                                int32_t b_groups, void *y, int32_t out_dtype, gsa_stream_t stream) {
    GemvParams P;
    std::memset(&P, 0, sizeof(P));
    if (!glu::act_of(act_kind, act_params, P.act)) return GSA_ERR_INVALID_ARG;
    P.probs = probs;
    return run_gemv(P, true, x, x_dtype, b, split_sizes_dev, E, M, N, K, recipe_kind, b_groups, y, out_dtype, stream);
}

}  // extern "C"
