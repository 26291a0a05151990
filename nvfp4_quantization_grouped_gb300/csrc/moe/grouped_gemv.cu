// grouped_gemv.cu -- products of a few unquantized rows an expert with its block-scaled
// (MXFP8 / NVFP4) weights, plain and gated, with their C entry points.
//
//   out[r, n] = u_e sum_k x[r, k] B_e[n, k],   rows r of expert e
//   y[r, n] = p_r act(u_g sum_k x[r, k] B_e[n, k], u_l sum_k x[r, k] B_e[N + n, k])
//
// What there is to do is to read the weights once: 0.56 (NVFP4) or 1.03 bytes each, so at the
// memory's rate an SM decodes 20 to 45 of them a cycle, and a multiply-add for each row of x and
// weight would not keep up.  So the weights go to the tensor core (mma.sync, 16 weight rows x 8
// rows of x x 16 k), as FP16: an NVFP4 code times its block scale has 6 bits and lies between
// 2^-10 and 2688, exact; an MXFP8 code is exact, and its block's scale, any power of two, is
// applied to the block's sums in FP32.  x is brought to FP16 too: scaled by a power of two to
// [2^14, 2^15), FP32 rows as the sum of two.
//   A block holds the rows of x of one expert in shared memory (up to 16, a pass) and walks
// a run of tiles of 16 weight rows, its 16 warps sharing out the steps of 128 bytes of each; their
// sums meet in shared memory.  Loads run kDepth steps ahead, over the ends of tiles, passes and
// experts.  How a sum is split goes by K alone: a row's result has the same bits whatever rows it
// comes with.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>
#include <mutex>
#include <type_traits>

#include "glu_act.cuh"
#include "gsa.h"
#include "moe/status.cuh"
#include "tc.cuh"

namespace {

constexpr int kMaxE = 256, kWarps = 16, kThreads = 32 * kWarps, kScaleTile = 512;
template <bool NV> constexpr int kStep = NV ? 256 : 128;   // k of a step: 128 bytes of a weight row
constexpr int kMaxRows = 16;                // rows of x a pass
constexpr int kSpace = (227 - 3) * 1024;    // bytes that a block has beside its static ones
constexpr int64_t kMaxK = 32768;            // a row of x beside the rest (FP32: half of it)

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
    int64_t expert_bytes, side_bytes;   // of codes: of an expert, of its gate rows
    int row_bytes;          // of a weight row's codes
    int scale_cols, scale_rows, up_tiles;   // scale tiles along k; of an expert along its rows; from a gate row to its linear row
    int b_groups;
    int steps, wk;          // steps of k; warps that share them out (a power of two)
    int tiles;              // tiles of 16 * (kWarps / wk) weight rows an expert
    int rows16;             // tiles of 16 weight rows an expert
    int pass_rows, pitch;   // rows of x a pass; bytes of a row in shared memory
    glu::Act act;
};

// A warp's sums: `n` groups of 8 rows of x, 16 weight rows each, 20 floats apart (the lanes' values of a product then meet no
// bank twice); two floats more, so that four slabs further on lie eight banks on.
constexpr int kRowSums = 20, kGroupSums = 8 * kRowSums;
__host__ __device__ constexpr int slab(int n) { return kGroupSums * n + 2; }

struct Shared {
    int row0[kMaxE + 1];     // first row of each expert
    int pass0[kMaxE + 1];    // first pass of each expert
    int64_t scan[kWarps][2];
    uint32_t bad;
    uint32_t largest[kMaxRows];   // bits of a row's largest finite value
    float unscale[kMaxRows];      // 2^-s of a row
    float probs[kMaxRows];
    float unit[2];                // of the weights: plain or gate, linear
};

// Rows and passes before each expert; every thread.
__device__ void scan_rows(const GemvParams &P, Shared &sh) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int64_t m = t < P.E ? (P.split ? P.split[t] : P.M) : 0;
    const bool neg = m < 0 || m > P.M;
    if (neg) m = 0;
    int64_t rows = m, passes = (m + P.pass_rows - 1) / P.pass_rows;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows, d), q = __shfl_up_sync(0xFFFFFFFFu, passes, d);
        if (lane >= d) rows += r, passes += q;
    }
    if (lane == 31) sh.scan[w][0] = rows, sh.scan[w][1] = passes;
    const bool any_neg = __syncthreads_or(neg);
    for (int k = 0; k < w; ++k) rows += sh.scan[k][0], passes += sh.scan[k][1];
    if (t < P.E) sh.row0[t + 1] = static_cast<int>(rows), sh.pass0[t + 1] = static_cast<int>(passes);
    if (t == 0) sh.row0[0] = 0, sh.pass0[0] = 0;
    if (t == P.E - 1) sh.bad = any_neg || rows > P.M;
    __syncthreads();
}

__device__ __forceinline__ float unit_of(float amax) {
    if (amax == 0.0f) return 1.0f;
    const float s = __fdiv_rn(2688.0f, amax);
    return __fdiv_rn(1.0f, s <= 3.402823466e38f ? s : 3.402823466e38f);
}

__device__ __forceinline__ void put(void *p, int type, int64_t i, float v) {
    if (type == GSA_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else if (type == GSA_FP16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// -------------------------------------------------------------- rows of x

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight consecutive values (i a multiple of 8).
template <int kPieces> struct Raw {   // 2: FP32
    uint4 r[kPieces];
    __device__ __forceinline__ void load(const void *x, int64_t i) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x) + i * (2 * kPieces));
#pragma unroll
        for (int k = 0; k < kPieces; ++k) r[k] = __ldg(p + k);
    }
    // Bits of the largest magnitudes so far, in halves for BF16 (`kFinite`: of finite values).
    template <bool kFinite> __device__ __forceinline__ uint32_t largest(uint32_t most) const {
        constexpr uint32_t kAbs = kPieces == 2 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a = w[j] & kAbs;
                if constexpr (kPieces == 2) {
                    if (!kFinite || a < 0x7F800000u) most = max(most, a);
                } else {
                    if (kFinite) a = ((a >> 16) < 0x7F80u ? a & 0xFFFF0000u : 0) | ((a & 0xFFFFu) < 0x7F80u ? a & 0xFFFFu : 0);
                    most = max_u16x2(most, a);
                }
            }
        }
        return most;
    }
    __device__ __forceinline__ void values(bool bf16, float (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (kPieces == 2) {
                    v[4 * k + j] = __uint_as_float(w[j]);
                } else if (bf16) {
                    v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                } else {
                    __half2 h;
                    memcpy(&h, &w[j], 4);
                    const float2 f = __half22float2(h);
                    v[2 * j] = f.x, v[2 * j + 1] = f.y;
                }
            }
        }
    }
};

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}

// Where the eight values from k on (a multiple of 8) lie in a row: in order (MXFP8: a lane's eight codes of a block of 32
// meet them in one 16-byte load), or with the 16-byte words of 128 values transposed, 4 x 4 (NVFP4: a lane has 32 codes in a
// row, and the four lanes of a weight row meet the words jj of theirs at once).
template <bool NV> __device__ __forceinline__ int place(int k) {
    const int c = k % 128 / 8;
    return k / 128 * 256 + 16 * (NV ? (c & 3) * 4 + (c >> 2) : c);
}

// Rows r0 .. r0 + rows of x to shared memory (kPieces 2: the FP16 halves of FP32 values, `rows` rows apart); every thread.
template <bool NV, int kPieces> __device__ void stage_rows(const GemvParams &P, Shared &sh, uint8_t *xs, int r0, int rows, float unit, int sides) {
    int threads = kThreads;   // a row: whole warps
    for (int r = 1; r < rows; r *= 2) threads /= 2;
    const int row = threadIdx.x / threads, t = threadIdx.x % threads, words = P.steps * (kStep<NV> / 8);
    const int64_t at = (r0 + static_cast<int64_t>(row)) * P.K;
    if (threadIdx.x < kMaxRows) sh.largest[threadIdx.x] = 0;
    __syncthreads();   // also: nobody reads the rows before any more
    if (threadIdx.x < sides) sh.unit[threadIdx.x] = unit;
    const bool bf16 = P.x_type == GSA_BF16;
    const int live = static_cast<int>(P.K) / 8;
    constexpr int kBatch = kPieces == 2 ? 4 : 8;   // words asked for at once
    if (P.x_type != GSA_FP16 && row < rows) {
        auto over = [&](auto finite) {
            uint32_t most = 0;
            for (int c0 = t; c0 < live; c0 += kBatch * threads) {
                Raw<kPieces> raw[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) raw[b].load(P.x, at + 8 * static_cast<int64_t>(min(c0 + b * threads, live - 1)));
#pragma unroll
                for (int b = 0; b < kBatch; ++b) most = raw[b].template largest<decltype(finite)::value>(most);
            }
            if (kPieces == 1) most = max(most & 0xFFFF0000u, most << 16);   // a BF16 is the high half of its FP32
            return __reduce_max_sync(0xFFFFFFFFu, most);
        };
        uint32_t most = over(std::false_type());
        if (most >= 0x7F800000u) most = over(std::true_type());   // infinities and NaN keep their place but set no scale
        if (threadIdx.x % 32 == 0) atomicMax(&sh.largest[row], most);
    }
    if (P.x_type != GSA_FP16) {
        __syncthreads();
    }
    if (row < rows) {
        float scale = 1.0f;
        if (P.x_type != GSA_FP16) {
            const uint32_t most = sh.largest[row];
            int s = 14 - (static_cast<int>(most >> 23) - 127);   // (subnormal: 141, cut off below)
            if (most == 0) s = 0;
            if (s > 126) s = 126;
            scale = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
            if (t == 0) sh.unscale[row] = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
        } else if (t == 0) {
            sh.unscale[row] = 1.0f;
        }
        if (t == 0) sh.probs[row] = P.probs ? P.probs[r0 + row] : 1.0f;
        for (int c0 = t; c0 < words; c0 += kBatch * threads) {
            Raw<kPieces> raw[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) raw[b].load(P.x, at + 8 * static_cast<int64_t>(min(c0 + b * threads, live - 1)));
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int c = c0 + b * threads;
                if (c >= words) break;
                float v[8];
                raw[b].values(bf16, v);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = c < live ? v[2 * j] * scale : 0.0f, q = c < live ? v[2 * j + 1] * scale : 0.0f;
                    hi[j] = half2_bits(p, q);
                    if (kPieces == 2) {
                        const float hp = __half2float(__float2half_rn(p)), hq = __half2float(__float2half_rn(q));
                        // an infinite value's rest would be NaN
                        lo[j] = half2_bits(fabsf(p) <= 65504.0f ? p - hp : 0.0f, fabsf(q) <= 65504.0f ? q - hq : 0.0f);
                    }
                }
                uint8_t *to = xs + row * P.pitch + place<NV>(8 * c);
                *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (kPieces == 2) *reinterpret_cast<uint4 *>(to + P.pass_rows * P.pitch) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- weights

// A lane's part of 128 k (a step, NVFP4: half of one): weight rows a (its low row of the tile) and b.
template <bool NV> struct Item;
template <> struct Item<true> {    // 32 codes of each row, and their scales (two, in the low half)
    uint4 a, b;
    uint32_t sa, sb;
};
template <> struct Item<false> {   // 8 codes of each of 4 blocks, and their scales
    uint2 a[4], b[4];
    uint32_t sa, sb;
};

// Weights on their way: each warp has kDepth steps in shared memory.  (In registers, slots of several steps share the few
// scoreboards, and any use waits for the newest load: 55 us where this took 41, 32 rows over 128 experts, 2048 x 4096 NVFP4.)
// Copies are 16 bytes, eight lanes a row.  A slot has the 16 rows' 128 bytes, with their halves (NVFP4) or their four blocks
// (MXFP8) swapped by row, so that the lanes of a load meet no bank twice, and the scales: 64 bytes a scale tile (4 rows of 4
// quarters of 4), four of them or one.
template <bool NV> constexpr int kSlot = 2048 + (NV ? 256 : 64);
template <int kG> constexpr int kDepth = kG == 1 ? 3 : 2;

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 16-byte word c of row r of a slot.
template <bool NV> __device__ __forceinline__ uint32_t word_at(int r, int c) { return r * 128 + 16 * (NV ? c ^ (4 * (r & 1)) : c ^ (2 * (r & 3))); }

// (Plain loads: as volatile statements they would keep their order among the products, each waiting for the one before.)
template <typename T> __device__ __forceinline__ T at_byte(const uint8_t *p, int at) { return *reinterpret_cast<const T *>(p + at); }

template <bool NV> __device__ __forceinline__ Item<NV> item_at(const uint8_t *slot, int half, int lane) {
    Item<NV> it;
    const int g = lane >> 2, t = lane & 3, word = 16 * (g & 3) + 4 * (g >> 2);
    if constexpr (NV) {
        const int c = word_at<NV>(g, 4 * half + t), s = 2048 + 64 * (2 * half + (t >> 1)) + word;
        it.a = at_byte<uint4>(slot, c);
        it.b = at_byte<uint4>(slot, c + 8 * 128);   // row g + 8 is swapped alike
        it.sa = at_byte<uint32_t>(slot, s) >> (16 * (t & 1));
        it.sb = at_byte<uint32_t>(slot, s + 8) >> (16 * (t & 1));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = word_at<NV>(g, 2 * j) + 8 * t;
            it.a[j] = at_byte<uint2>(slot, c);
            it.b[j] = at_byte<uint2>(slot, c + 8 * 128);
        }
        it.sa = at_byte<uint32_t>(slot, 2048 + word);
        it.sb = at_byte<uint32_t>(slot, 2048 + word + 8);
    }
    return it;
}

// Where a lane copies one side of a tile from.  The tile i of 16 weight rows holds rows 4 (i mod 8) .. + 3 of each quarter of
// scale tile i / 8 (row r of the tile: r mod 4 of quarter r / 4), whose scales are 64 bytes in a row.  A lane has 16 bytes of
// four rows, one of each quarter.  Nothing is predicated: rows past the last read the last (their results are not stored), and
// what lies past the end of k reads the row's last word again (x is zero there).
template <bool NV> struct Aim {
    const uint8_t *codes, *scales;   // of the expert
    const uint8_t *row[4], *s;
    __device__ __forceinline__ void expert(const GemvParams &P, int e, int lane) {
        codes = P.codes + e * P.expert_bytes;
        scales = P.scales + static_cast<int64_t>(e * P.scale_rows) * P.scale_cols * kScaleTile + 16 * (lane & 3);
    }
    __device__ __forceinline__ void at(const GemvParams &P, bool linear, int i, int lane) {
        const int last = static_cast<int>(P.N) - 1, inside = 128 * (i >> 3) + 4 * (i & 7) + (lane >> 3);
        const uint8_t *first = linear ? codes + P.side_bytes : codes;
#pragma unroll
        for (int k = 0; k < 4; ++k) row[k] = first + static_cast<int64_t>(min(inside + 32 * k, last)) * P.row_bytes;
        s = scales + static_cast<int64_t>((linear ? P.up_tiles : 0) + (i >> 3)) * (P.scale_cols * kScaleTile) + 64 * (i & 7);
    }
    __device__ __forceinline__ void load(const GemvParams &P, uint32_t slot, int step, int lane) const {
        const uint32_t c = min(step * 128 + 16 * (lane & 7), P.row_bytes - 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) copy_async(slot + word_at<NV>((lane >> 3) + 4 * k, lane & 7), row[k] + c);
        const int tile = NV ? 4 * step + (lane >> 2) : step;
        if (lane < (NV ? 16 : 4)) copy_async(slot + 2048 + 16 * lane, s + min(tile, P.scale_cols - 1) * kScaleTile);
    }
};

// Eight E2M1 codes, four E4M3 codes as FP16, and two E8M0 scales as FP32 (255: NaN).
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
    return h;
}
__device__ __forceinline__ void e8m0x4(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.bf16x2.ue8m0x2 %0, a;\n cvt.rn.bf16x2.ue8m0x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
    f[0] = __uint_as_float(lo << 16), f[1] = __uint_as_float(lo & 0xFFFF0000u);
    f[2] = __uint_as_float(hi << 16), f[3] = __uint_as_float(hi & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The products of 128 k with `groups` groups of 8 rows of x (xs: the lane's place there, by group 8 rows apart;
// left: k from the first on, MXFP8: a word of scales holds padding behind the last block, maybe NaN).  The
// sums of a step start from zero and are added in FP32: the tensor core cuts off what it adds to (about 2^-24 of it a step of
// 16), which would grow with the length.
template <bool NV, int kG, int kPieces>
__device__ __forceinline__ void multiply(const Item<NV> &it, float (&acc)[kG][4], const uint8_t *const (&xs)[kG], int groups, int piece_bytes, int left) {
    if constexpr (NV) {
        const uint32_t sa = e4m3x2(it.sa), sb = e4m3x2(it.sb);
        const uint32_t wa[4] = {it.a.x, it.a.y, it.a.z, it.a.w}, wb[4] = {it.b.x, it.b.y, it.b.z, it.b.w};
        uint32_t A[8][4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t fa = __byte_perm(sa, 0, w < 2 ? 0x1010 : 0x3232), fb = __byte_perm(sb, 0, w < 2 ? 0x1010 : 0x3232);
            uint32_t a[4], b[4];
            e2m1x8(wa[w], a);
            e2m1x8(wb[w], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                A[2 * w + (i >> 1)][2 * (i & 1)] = mul_half2(a[i], fa);
                A[2 * w + (i >> 1)][2 * (i & 1) + 1] = mul_half2(b[i], fb);
            }
        }
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            if (q >= groups) break;
            float d[2][4] = {};   // two chains: a product waits for the one before it in its chain
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const uint4 b = at_byte<uint4>(xs[q], p * piece_bytes + 64 * jj);
                    mma(d[0], A[2 * jj], b.x, b.y);
                    mma(d[1], A[2 * jj + 1], b.z, b.w);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][i] += d[0][i] + d[1][i];
        }
    } else {
        const uint32_t keep = left > 64 ? 0xFFFFFFFFu : 0xFFFFu;   // K is a multiple of 64
        float fa[4], fb[4];
        e8m0x4(it.sa & keep, fa);
        e8m0x4(it.sb & keep, fb);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t A0[4], A1[4];
            e4m3x4(it.a[b].x, A0[0], A0[2]);
            e4m3x4(it.b[b].x, A0[1], A0[3]);
            e4m3x4(it.a[b].y, A1[0], A1[2]);
            e4m3x4(it.b[b].y, A1[1], A1[3]);
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                if (q >= groups) break;
                float d[4] = {};
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    const uint4 x = at_byte<uint4>(xs[q], p * piece_bytes + 64 * b);
                    mma(d, A0, x.x, x.y);
                    mma(d, A1, x.z, x.w);
                }
                acc[q][0] = __fmaf_rn(fa[b], d[0], acc[q][0]);
                acc[q][1] = __fmaf_rn(fa[b], d[1], acc[q][1]);
                acc[q][2] = __fmaf_rn(fb[b], d[2], acc[q][2]);
                acc[q][3] = __fmaf_rn(fb[b], d[3], acc[q][3]);
            }
        }
    }
}

// A place in a block's run of tiles.
struct Cursor {
    int e, pass, tile;
    __device__ __forceinline__ void next(const GemvParams &P, const Shared &sh) {
        if (++tile < P.tiles) return;
        tile = 0;
        if (++pass >= sh.pass0[e + 1]) find(P, sh);   // (only asked for where there is a next tile)
    }
    __device__ __forceinline__ void find(const GemvParams &P, const Shared &sh) {   // the expert of the pass
        e = 0;
        for (int end = P.E; end - e > 1;) {   // the last that starts at or before it
            const int mid = (e + end) >> 1;
            if (sh.pass0[mid] <= pass) e = mid;
            else end = mid;
        }
    }
};

__device__ __forceinline__ float gated(const glu::Act &A, float g, float u) {
    const float2 a = make_float2(g, g), b = make_float2(u, u);
    return A.clamped ? glu::value<true>(A, a, b).x : glu::value<false>(A, a, b).x;
}

// A sum times the weights' unit and the row's 2^-s: in the order that leaves FP32's range last.
__device__ __forceinline__ float scaled(float v, float unit, float unscale) {
    if ((unit > 0x1p64f && unscale < 1.0f) || (unit < 0x1p-64f && unscale > 4.0f)) return v * (unit * unscale);
    return v * unit * unscale;
}

template <bool NV, bool kGlu, int kG, int kPieces> __global__ void __launch_bounds__(kThreads, 1) gemv(const __grid_constant__ GemvParams P) {
    constexpr int kSides = kGlu ? 2 : 1;
    constexpr int kAhead = kDepth<kG>;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ Shared sh;
    float *const sums = reinterpret_cast<float *>(dyn);   // [2][warp][kSlab]
    constexpr int kSlab = slab(kSides * kG);
    uint8_t *ring = dyn + 2 * kWarps * kSlab * sizeof(float), *xs = ring + kWarps * kAhead * kSlot<NV>;
    tc::allow_next();
    tc::wait_for_previous();
    scan_rows(P, sh);
    if (sh.bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.status, gemm_status::ERR_SPLIT);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wk = warp & (P.wk - 1), wn = warp / P.wk, wns = kWarps / P.wk;
    // the block's run of tiles: `all` in equal parts, the first `more` one longer
    const int64_t all = static_cast<int64_t>(sh.pass0[P.E]) * P.tiles;
    const bool small = all >> 32 == 0;   // divisions of 64 bits take hundreds of cycles
    const int64_t part = small ? static_cast<uint32_t>(all) / gridDim.x : all / gridDim.x, more = all - part * gridDim.x;
    const int64_t first = part * blockIdx.x + (blockIdx.x < more ? blockIdx.x : more), left = part + (blockIdx.x < more);
    if (left > 0) {
        Cursor ahead;   // of the loads
        ahead.pass = static_cast<int>(small ? static_cast<uint32_t>(first) / static_cast<uint32_t>(P.tiles) : first / P.tiles);
        ahead.tile = static_cast<int>(first - static_cast<int64_t>(ahead.pass) * P.tiles);
        ahead.find(P, sh);
        Cursor at = ahead;
        const int rounds = (P.steps + P.wk - 1) / P.wk;   // a warp's steps of a side of a tile
        int64_t to_ask = left, to_do = left;              // tiles
        Aim<NV> aim;
        int ask_side = 0, ask_round = 0;
        auto take_aim = [&] { aim.at(P, kGlu && ask_side, min(ahead.tile * wns + wn, P.rows16 - 1), lane); };
        const uint8_t *own = ring + warp * (kAhead * kSlot<NV>);
        const uint32_t slots = tc::smem_u32(own);
        auto ask = [&](int slot) {   // the next step's weights; one group of copies a call
            if (to_ask > 0) aim.load(P, slots + slot * kSlot<NV>, ask_round * P.wk + wk, lane);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (to_ask == 0) return;
            if (++ask_round < rounds) return;
            ask_round = 0;
            if (kGlu && ask_side == 0) {
                ask_side = 1;
            } else {
                ask_side = 0;
                if (--to_ask == 0) return;
                const int before = ahead.e;
                ahead.next(P, sh);
                if (ahead.e != before) aim.expert(P, ahead.e, lane);
            }
            take_aim();
        };
        aim.expert(P, ahead.e, lane);
        take_aim();
        for (int d = 0; d < kAhead; ++d) ask(d);

        float acc[kG][4] = {};
        const uint8_t *place_of[kG];
        const int piece_bytes = P.pass_rows * P.pitch;
        const int runs = min(4, P.wk), runs_log = runs >> 1, each = P.wk / runs, wns_log = 31 - __clz(wns);
        int staged = -1, rows = 0, groups = 0, r0 = 0, side = 0, round = 0, buffer = 0;
        auto stage = [&] {
            staged = at.pass;
            float unit = 1.0f;
            const int p = at.pass - sh.pass0[at.e];
            r0 = sh.row0[at.e] + p * P.pass_rows;
            rows = min(P.pass_rows, sh.row0[at.e + 1] - r0);
            groups = (rows + 7) / 8;
            if (NV && threadIdx.x < kSides) unit = unit_of(P.amax[at.e * P.b_groups + (threadIdx.x ? P.b_groups - 1 : 0)]);
            stage_rows<NV, kPieces>(P, sh, xs, r0, rows, unit, kSides);
#pragma unroll
            for (int q = 0; q < kG; ++q)   // lanes past the last row read it again: their columns are not stored
                place_of[q] = xs + min(8 * q + (lane >> 2), rows - 1) * P.pitch + 16 * (lane & 3);
        };
        // A warp's sums of a side of the tile to shared memory.
        auto hand_in = [&] {
            float *mine = sums + (buffer * kWarps + warp) * kSlab + side * kG * kGroupSums + 2 * (lane & 3) * kRowSums + (lane >> 2);
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                if (q >= groups) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mine[q * kGroupSums + (k & 1) * kRowSums + (k >> 1) * 8] = acc[q][k];
                    acc[q][k] = 0.0f;
                }
            }
        };
        // The tile's sums over the warps, and its results.  Of each result up to four runs of warps' sums, each in order, then
        // pairs of runs: by one lane, or by two or four where there are lanes enough, in the same order.
        auto finish = [&] {
            __syncthreads();
            const int results = 16 * wns * rows, lanes_log = results * 4 <= kThreads ? runs_log : results * 2 <= kThreads ? min(1, runs_log) : 0;
            const int mine = runs >> lanes_log, lanes = 1 << lanes_log, part = threadIdx.x & (lanes - 1);
            for (int base = 0; base < results << lanes_log; base += kThreads) {
                const int o = (base + static_cast<int>(threadIdx.x)) >> lanes_log;
                const int a = o & 15, b = (o >> 4) & (wns - 1), r = (o >> 4) >> wns_log;   // weight row, warp row, row of x
                const bool on = o < results;
                const float *from = sums + (buffer * kWarps + b * P.wk + part * mine * each) * kSlab + (on ? r >> 3 : 0) * kGroupSums + (r & 7) * kRowSums + a;
                float v[kSides];
#pragma unroll
                for (int s = 0; s < kSides; ++s) {
                    float run[4] = {};
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (p < mine) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < each) run[p] += from[s * kG * kGroupSums + (p * each + k) * kSlab];
                        }
                    v[s] = run[0];
                    if (mine > 1) v[s] += run[1];
                    if (mine > 2) v[s] += run[2] + run[3];
                }
#pragma unroll
                for (int d = 1; d < 4; d <<= 1)
                    if (d < lanes) {
#pragma unroll
                        for (int s = 0; s < kSides; ++s) v[s] += __shfl_xor_sync(0xFFFFFFFFu, v[s], d);
                    }
                const int i = at.tile * wns + b, n = 128 * (i >> 3) + 4 * (i & 7) + (a & 3) + 32 * (a >> 2);
                if (part != 0 || !on || i >= P.rows16 || n >= P.N) continue;
                const float unscale = sh.unscale[r];
                float y = scaled(v[0], sh.unit[0], unscale);
                if constexpr (kGlu) y = sh.probs[r] * gated(P.act, y, scaled(v[kSides - 1], sh.unit[1], unscale));
                put(P.out, P.out_type, (r0 + static_cast<int64_t>(r)) * P.N + n, y);
            }
            buffer ^= 1;
        };
        for (int slot = 0; to_do > 0; slot = slot + 1 < kAhead ? slot + 1 : 0) {
            if (staged != at.pass) stage();
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            __syncwarp();   // the other lanes' copies
            const int step = round * P.wk + wk;
            if (step < P.steps) {
#pragma unroll
                for (int half = 0; half < kStep<NV> / 128; ++half) {
                    const uint8_t *from[kG];
#pragma unroll
                    for (int q = 0; q < kG; ++q) from[q] = place_of[q] + step * (kStep<NV> * 2) + half * 256;
                    multiply<NV, kG, kPieces>(item_at<NV>(own + slot * kSlot<NV>, half, lane), acc, from, groups, piece_bytes, static_cast<int>(P.K) - step * kStep<NV>);
                }
            }
            __syncwarp();   // all lanes have what the slot held
            ask(slot);
            if (++round < rounds) continue;
            round = 0;
            hand_in();
            if (kGlu && side == 0) {
                side = 1;
                continue;
            }
            side = 0;
            finish();
            if (--to_do > 0) at.next(P, sh);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    // rows that no expert has
    const int64_t tail = sh.row0[P.E] * P.N;
    for (int64_t i = tail + blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < P.M * P.N; i += gridDim.x * static_cast<int64_t>(kThreads))
        put(P.out, P.out_type, i, 0.0f);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

gsa_status cuda_error() {
    cudaGetLastError();
    return GSA_ERR_CUDA;
}

bool known_type(int32_t t) { return t == GSA_BF16 || t == GSA_FP16 || t == GSA_FP32; }

int sm_count() {
    static std::mutex mu;
    static int known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) known[dev] = v;
    }
    return known[dev];
}

// Shared memory but for x: sums and weights under way.
template <bool NV, bool kGlu, int kG> constexpr int own_bytes() {
    return 2 * kWarps * slab((kGlu ? 2 : 1) * kG) * static_cast<int>(sizeof(float)) + kWarps * kDepth<kG> * kSlot<NV>;
}

template <bool NV, bool kGlu, int kG, int kPieces> gsa_status launch_gemv(const GemvParams &P, cudaStream_t s) {
    const int sms = sm_count();
    if (!sms) return cuda_error();
    const int smem = P.pass_rows * P.pitch * kPieces + own_bytes<NV, kGlu, kG>();
    auto kernel = gemv<NV, kGlu, kG, kPieces>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return cuda_error();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see tc::wait_for_previous
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? GSA_OK : cuda_error();
}

gsa_status run_gemv(GemvParams &P, bool glu, const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split, int64_t E, int64_t M, int64_t N,
                    int64_t K, int32_t recipe_kind, int32_t b_groups, void *out, int32_t out_dtype, gsa_stream_t stream) {
    if (!b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (!known_type(x_dtype) || !known_type(out_dtype) || (b_groups != 1 && b_groups != 2)) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    const int64_t sides = glu ? 2 : 1;
    if (E > kMaxE || K % 64 != 0 || K > (x_dtype == GSA_FP32 ? kMaxK / 2 : kMaxK) || M >= (int64_t(1) << 31) - 256 || N >= (int64_t(1) << 30) / E - 256) return GSA_ERR_UNSUPPORTED;
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
    const int step = nv ? kStep<true> : kStep<false>;
    P.steps = static_cast<int>((K + step - 1) / step);
    P.row_bytes = static_cast<int>(nv ? K / 2 : K);
    P.side_bytes = N * P.row_bytes;
    P.expert_bytes = sides * P.side_bytes;
    P.wk = 1;
    while (P.wk < kWarps && P.wk < P.steps) P.wk *= 2;
    const int64_t rest = N % 128;
    P.rows16 = static_cast<int>(8 * (N / 128) + (rest >= 32 ? 8 : (rest + 3) / 4));
    // As few warps to a sum as leave six tiles a block (of as many experts as can have rows): each tile ends with a barrier and
    // the warps' sums.
    while (P.wk > 2 && (E < M ? E : M) * P.rows16 * P.wk / (2 * kWarps) >= 6 * 152) P.wk /= 2;
    const int wns = kWarps / P.wk;
    P.tiles = (P.rows16 + wns - 1) / wns;
    P.pitch = P.steps * step * 2 + 64;   // rows on alternating halves of the banks
    const int pieces = x_dtype == GSA_FP32 ? 2 : 1;
    auto space = [&](int groups) {   // of x, with 8 rows or 16 a pass
        auto own = [&](auto fmt, auto gated) {
            constexpr bool NV = decltype(fmt)::value, kGlu = decltype(gated)::value;
            return groups == 1 ? own_bytes<NV, kGlu, 1>() : own_bytes<NV, kGlu, 2>();
        };
        return kSpace - (nv ? (glu ? own(std::true_type(), std::true_type()) : own(std::true_type(), std::false_type()))
                            : (glu ? own(std::false_type(), std::true_type()) : own(std::false_type(), std::false_type())));
    };
    int64_t rows = space(2) / (P.pitch * pieces);
    int groups = 2;
    if (M <= 8 || rows <= 8) rows = space(groups = 1) / (P.pitch * pieces);
    if (rows > 8 * groups) rows = 8 * groups;
    P.pass_rows = static_cast<int>(rows < M ? rows : M);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto fmt, auto gated, auto many) {
        constexpr bool NV = decltype(fmt)::value, kGlu = decltype(gated)::value;
        constexpr int kG = decltype(many)::value;
        return pieces == 2 ? launch_gemv<NV, kGlu, kG, 2>(P, s) : launch_gemv<NV, kGlu, kG, 1>(P, s);
    };
    auto grouped = [&](auto fmt, auto gated) {
        return groups == 1 ? go(fmt, gated, std::integral_constant<int, 1>()) : go(fmt, gated, std::integral_constant<int, 2>());
    };
    auto sided = [&](auto fmt) { return glu ? grouped(fmt, std::true_type()) : grouped(fmt, std::false_type()); };
    return nv ? sided(std::true_type()) : sided(std::false_type());
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
