// grouped_gemv.cu -- products of a few unquantized rows an expert with its block-scaled
// (MXFP8 / NVFP4) weights, plain and gated, with their C entry points.
//
//   out[r, n] = u_e sum_k x[r, k] B_e[n, k],   rows r of expert e
//   y[r, n] = p_r act(u_g sum_k x[r, k] B_e[n, k], u_l sum_k x[r, k] B_e[N + n, k])
//
// What there is to do is to read the weights once.  Decoding them costs more than that: at the
// memory's rate 20 (MXFP8) to 45 (NVFP4) a cycle and SM, for which conversions, block scales
// and mma.sync products took twice the time of the loads (32 rows over 128 experts, 2048 x 4096
// NVFP4: 29 us, against 17 to 18 for the product of quantized rows).  So it is x that is brought
// to the weights' format, without losing it: as eight digits,
//   x[r, k] = 2^t_r sum_d 2^-c_d D_d[r, k] 2^q[r, block of k],
// D_0 the code nearest to x in its block's scale, D_1 the code nearest to what that leaves, and
// so on: eight rows of one block-scaled operand, which go through the block-scaled product
// (tcgen05) with the weights as they lie in memory.  An E2M1 code leaves an eighth of its
// unit's half, an E4M3 code less: eight leave 2^-22 of the block's largest value, and nothing of
// BF16 and FP16 values down to 2^-10 of it.  That is as far as block scales reach below the row's largest
// value: E4M3's to 2^-17 of it, E8M0's to 2^-87 or further.  Blocks below 2^-16 (2^-80) have digits in that
// last unit, which leave 2^-37 of the row's largest value at most.  A lane of tensor memory holds a digit's sum, so the eight
// lanes of a row are added on the way out.
//   The rest is the grouped product's kernel with 16 rows of x to a tile of 128 x 128 (gated: 128
// of both sides), whose loads leave the absent rows out, and which starts on the weights while
// the digits are written.  GPU time in a graph: 32 rows over 128 experts, 2048 x 4096 NVFP4
// 20 to 21 us (11 of them the weights' stream at the memory's rate, 4 the start and the digits,
// 3 the end); one row, 4096 x 4096 NVFP4 10; 64 rows over 8, 4096 x 4096 MXFP8 30; gated, 8 rows
// over 128 experts, 4096 x 2048 NVFP4 17 to 18; 64 over 128, 2048 x 2048 MXFP8 48.  The host takes
// 17 to 23 a call (two launches and two allocations), which is what small calls cost outside of
// graphs.  In one launch, with every block making the digits of its rows in its own stages, the
// same calls took 46, 10, 83, 22 and 71: a row's digits are made again for each column tile.
#include "gemm_core.cuh"
#include "glu_act.cuh"

namespace {

constexpr int kDigits = 8, kDigitsLog = 3;

// -c_d: the power of two of a digit's unit.  E2M1 values to 6: a remainder up to 1 (of a value past 4) is 4 quarters; from then
// on the remainder is half a unit at most, 4 eighths.  E4M3 values to 256: a remainder up to 8 is 128 sixteenths, then 4 units
// at most, 128 times 2^-5.
template <bool NV> __device__ __forceinline__ int digit_exponent(int d) { return d == 0 ? 0 : NV ? 1 - 3 * d : 1 - 5 * d; }

struct RowInfo {
    int t;        // exponent of the row's scale
    int infinite; // infinite values (their digits are theirs alone), or 0
};

struct DigitParams {
    const void *x;
    const int64_t *split;   // nullptr: one expert has all rows
    uint8_t *codes, *scales;
    RowInfo *info;
    int64_t M, tiles;       // rows; row tiles that the scales have room for
    int E, K, x_type;
    int scale_cols;
};

// Eight values, in FP32.  (Plain loads: the kernel may have started before x was written, see tc::wait_for_previous.)
__device__ __forceinline__ void load8(const void *x, int type, int64_t i, float (&v)[8]) {
    if (type == GSA_FP32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
    const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (type == GSA_BF16) {
            v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        } else {
            __half2 h;
            memcpy(&h, &w[k], 4);
            const float2 f = __half22float2(h);
            v[2 * k] = f.x, v[2 * k + 1] = f.y;
        }
    }
}

// 2^e times f, in two factors that FP32 holds.  (Beyond their ends, 2^-252 and 2^254, every sum here is 0 or infinite.)
__device__ __forceinline__ float times_power(float f, int e) {
    e = max(-252, min(254, e));
    const int h = e / 2;
    return f * __uint_as_float(static_cast<uint32_t>(127 + h) << 23) * __uint_as_float(static_cast<uint32_t>(127 + e - h) << 23);
}

// The exponent that brings a block's largest value (> 0) to [3, 6] (E2M1) or [128, 256) (E4M3).
template <bool NV> __device__ __forceinline__ int block_exponent(float most) {
    int e;
    const float m = frexpf(most, &e);   // [1/2, 1)
    return NV ? (m <= 0.75f ? e - 3 : e - 2) : e - 8;
}

// Four E2M1 or two E4M3 codes of the nearest values, and the values.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi, float &a, float &b) {
    uint32_t c, h;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %3, %2;\n cvt.rn.f16x2.e2m1x2 %1, t;\n cvt.u32.u8 %0, t;\n}" : "=r"(c), "=r"(h) : "f"(lo), "f"(hi));
    __half2 v;
    memcpy(&v, &h, 4);
    const float2 f = __half22float2(v);
    a = f.x, b = f.y;
    return c;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi, float &a, float &b) {
    uint16_t c;
    uint32_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    __half2 v;
    memcpy(&v, &h, 4);
    const float2 f = __half22float2(v);
    a = f.x, b = f.y;
    return c;
}

constexpr int kDigitThreads = 512, kNone = -100000;

// Digits of row blockIdx.x, eight values a thread: two (NVFP4) or four lanes a block.  Infinite values get digits of their own (one each, the first eight; finite values are nothing
// beside them): products with them have the sign or, of zero weights, the NaN that the weights give.  A NaN, or more infinities,
// makes the row NaN by a NaN scale.
template <bool NV> __global__ void __launch_bounds__(kDigitThreads) split_digits(const __grid_constant__ DigitParams P) {
    constexpr int kLanes = NV ? 2 : 4;   // of a block
    __shared__ int64_t rows_of[kDigitThreads / 32];
    __shared__ int tiles_of[kDigitThreads / 32], first_row, first_tile, most_t, infinite, nan, placed;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int64_t r = blockIdx.x;
    // In this order: once the product's blocks run, everything before this kernel is done, and they read the split and the
    // weights without waiting for the digits.
    tc::wait_for_previous();
    tc::allow_next();
    if (t == 0) first_row = -1, most_t = kNone, infinite = 0, nan = 0, placed = 0;
    const int parts = P.K / 8, rounded = (parts + 31) & ~31;   // of eight values; whole warps go round
    const bool once = parts <= kDigitThreads;                  // a part a thread: read once
    float v[8] = {};
    auto load = [&](int i) {
        if (i < parts) load8(P.x, P.x_type, r * P.K + static_cast<int64_t>(i) * 8, v);
    };
    load(t);
    // the expert that has the row: its first row and scale tile
    int64_t m = t < P.E ? (P.split ? P.split[t] : P.M) : 0;
    if (m < 0 || m > P.M) m = 0;   // (a bad split: the product reports it and writes nothing)
    const int own_tiles = static_cast<int>((m * kDigits + 127) / 128);
    int64_t rows = m;
    int tiles = own_tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xFFFFFFFFu, rows, d);
        const int b = __shfl_up_sync(0xFFFFFFFFu, tiles, d);
        if (lane >= d) rows += a, tiles += b;
    }
    if (lane == 31) rows_of[w] = rows, tiles_of[w] = tiles;
    __syncthreads();
    for (int k = 0; k < w; ++k) rows += rows_of[k], tiles += tiles_of[k];
    if (r < rows && r >= rows - m) first_row = static_cast<int>(rows - m), first_tile = tiles - own_tiles;

    auto largest = [&](int i, bool &finite) {   // of the block that part i is in; its other lanes are here too
        if (!once) load(i);
        float most = 0.0f;
        finite = true;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            finite &= fabsf(v[k]) <= 3.402823466e38f;
            most = fmaxf(most, fabsf(v[k]));
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        return most;
    };
    int mine = kNone;
    for (int i = t; i < rounded; i += kDigitThreads) {
        bool finite;
        const float most = largest(i, finite);
        if (i >= parts) continue;
        if (most > 0.0f && most <= 3.402823466e38f) mine = max(mine, block_exponent<NV>(most));
        if (finite) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (v[k] != v[k]) nan = 1;
            else if (isinf(v[k])) atomicAdd(&infinite, 1);
        }
    }
    mine = __reduce_max_sync(0xFFFFFFFFu, mine);
    if (lane == 0 && mine != kNone) atomicMax(&most_t, mine);
    __syncthreads();
    const bool is_nan = nan || infinite > kDigits, special = nan || infinite;
    // Exponents of the largest block's scale and of the least.  E4M3's largest power of two; E8M0 has room for x's own size, from
    // 2^-40 to 1: a small row against large weights (up to 2^136) then has sums of its results' size, where a row scaled to the
    // top took them through infinity, and below 2^-40 no sum can get there.
    const int most = most_t == kNone ? 0 : most_t, top = NV ? 8 : max(-40, min(0, most));
    constexpr int kLow = NV ? -9 : -127;
    const int row_t = most - top;
    if (t == 0) P.info[r] = {special ? 0 : row_t, is_nan ? 0 : infinite};
    // A bad split may leave the row, or room for its scales, to no expert.
    const int at = static_cast<int>(r - first_row) * kDigits, lr = at & 127;
    const int64_t tile = static_cast<int64_t>(first_tile) + (at >> 7);
    if (first_row < 0 || tile < 0 || tile >= P.tiles) return;
    const int64_t pitch = NV ? P.K / 2 : P.K;
    uint8_t *codes = P.codes + r * kDigits * pitch, *scales = P.scales + tile * P.scale_cols * kScaleTile + 16 * (lr & 31) + 4 * (lr >> 5);
    for (int i = t; i < rounded; i += kDigitThreads) {
        bool finite;
        const float most = largest(i, finite);
        if (i >= parts) continue;
        const int b = i / kLanes;
        int q = kLow;
        if (most > 0.0f && !special) q = max(kLow, block_exponent<NV>(most) - row_t);
        uint8_t scale = NV ? (q >= -6 ? (q + 7) << 3 : 1 << (q + 9)) : q + 127;
        if (special) scale = is_nan ? (NV ? 0x7F : 0xFF) : (NV ? 7 << 3 : 127);
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = special ? 0.0f : times_power(v[k], -row_t - q);
#pragma unroll
        for (int d = 0; d < kDigits; ++d) {
            uint32_t c[NV ? 1 : 2] = {};
            const float next = NV ? (d == 0 ? 4.0f : 8.0f) : (d == 0 ? 16.0f : 32.0f);
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                float lo, hi;
                if (NV) c[0] |= e2m1x2(x[k], x[k + 1], lo, hi) << 4 * k;
                else c[k / 4] |= e4m3x2(x[k], x[k + 1], lo, hi) << 8 * (k % 4);
                x[k] = (x[k] - lo) * next, x[k + 1] = (x[k + 1] - hi) * next;
            }
            uint8_t *to = codes + d * pitch + static_cast<int64_t>(i) * (NV ? 4 : 8);
            if constexpr (NV) *reinterpret_cast<uint32_t *>(to) = c[0];
            else *reinterpret_cast<uint2 *>(to) = make_uint2(c[0], c[1]);
        }
        // the block's scale, the same for its eight digits: a few of them by each of its lanes
#pragma unroll
        for (int d = 0; d < kDigits / kLanes; ++d)
            scales[static_cast<int64_t>(b >> 2) * kScaleTile + 16 * (i % kLanes * (kDigits / kLanes) + d) + (b & 3)] = scale;
    }
    if (!special || is_nan) return;
    __syncthreads();   // the zeros are there
    for (int k = t; k < P.K; k += kDigitThreads) {
        const int64_t i = r * P.K + k;
        const float x = P.x_type == GSA_FP32   ? static_cast<const float *>(P.x)[i]
                        : P.x_type == GSA_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(P.x)[i])
                                               : __half2float(static_cast<const __half *>(P.x)[i]);
        if (!isinf(x)) continue;
        float a, z;
        uint8_t *row = codes + atomicAdd(&placed, 1) * pitch;   // whichever digit: sums of infinities have no order
        const float s = copysignf(1.0f, x);
        if (NV) row[k / 2] = static_cast<uint8_t>(k & 1 ? e2m1x2(0.0f, s, a, z) : e2m1x2(s, 0.0f, a, z));
        else row[k] = static_cast<uint8_t>(e4m3x2(s, 0.0f, a, z));
    }
}

// ----------------------------------------------------------------- products

struct FewParams : GemmParams {   // M: rows of digits; N: columns of one side
    glu::Act act;
    const RowInfo *info;
    const float *probs;
    uint32_t *status;
    int up_tiles, b_groups, out_type;
};

__device__ __forceinline__ void put(void *p, int type, int64_t i, float v) {
    if (type == GSA_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else if (type == GSA_FP16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// Eight columns of this lane's digit, weighted, summed over the eight lanes of its row: lane d of them gets column d.  (Each
// exchange halves the columns that a lane still has a part of: seven shuffles, not 24.)
__device__ __forceinline__ float sum_digits(const uint32_t *v, float weight, int lane) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]) * weight;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {
        const bool high = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, high ? x[i] : x[i + d], d);
            x[i] = (high ? x[i + d] : x[i]) + other;
        }
    }
    return x[0];
}

// A sum times a unit and 2^t: by the unit's mantissa, then its and the row's exponent together.
struct Scale {
    float mantissa;
    int exponent;
    __device__ __forceinline__ void of(float amax) {
        mantissa = 1.0f, exponent = 0;
        if (amax < 0.0f) return;   // MXFP8
        mantissa = frexpf(__fdiv_rn(1.0f, tensor_scale(amax)), &exponent);
        if (!(fabsf(mantissa) < 1.0f)) exponent = 0;   // (infinite, NaN)
    }
    __device__ __forceinline__ float operator()(float sum, int t) const { return times_power(sum * mantissa, exponent + t); }
};

constexpr int kCols = 64;   // columns of a side that a warp drains
template <bool NV, bool kGlu> using FewCfg = Cfg<NV, kGlu ? 256 : 128, false, 0>;   // results go straight from the registers

template <bool NV, bool kGlu, bool kClamp> __global__ void __launch_bounds__(kThreads, 1) grouped_few(const __grid_constant__ FewParams P) {
    constexpr int BN = kGlu ? 256 : 128, kLen = kPiece<float>;
    using C = FewCfg<NV, kGlu>;
    extern __shared__ uint8_t dyn[];
    __shared__ GemmShared sh;
    static_assert(sizeof(GemmShared) <= kStatic, "shared memory");
    const int warp = known_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Stages<NV, BN, false> st(dyn);
    open_block<C::kStages, false>(sh, warp, 1, C::kCols);
    tc::allow_next();
    scan_split<kRowsT, kDigits>(P, sh);
    if (sh.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.status, ERR_SPLIT);
    const int total = known_uniform(sh.bad ? 0 : sh.tile0[P.E + 1]), used = known_uniform(sh.bad ? 0 : sh.tile0[P.E]);   // row tiles; the rest is zeros
    Walk walk(P, blockIdx.x, gridDim.x);

    if (warp == 0) {
        if (tc::elect()) {
            tc::prefetch_map(&P.tm_a);
            tc::prefetch_map(&P.tm_b);
        }
        Ring<C::kStages> ring;
        bool ok = true;
        auto at = [&](const Tile &t) {
            StageAt w{&P.tm_a, &P.tm_b, &P.tm_sa, &P.tm_sb};
            w.x = 0;
            w.a_row = t.row;
            w.a_boxes = (t.rows + kBoxA - 1) / kBoxA;
            w.a_tile = (known_uniform(sh.scale0[t.g]) + t.mt) * P.scale_cols;
            w.b_row = static_cast<int>((kGlu ? 2 : 1) * t.g * P.N) + t.nt * 128;
            w.b_row_step = static_cast<int>(P.N);
            w.b_tile = (t.g * P.b_scale_rows + t.nt) * P.scale_cols;
            w.b_tile_step = P.up_tiles * P.scale_cols;
            return w;
        };
        // While the digits are written: the first stages' weights.  (Further ones into L2 as well gained nothing.)
        Walk ahead = walk;
        int early = 0;
        for (; ahead.q < used && early < C::kStages; ahead.next(P)) {
            StageAt w = at(ahead.tile<kRowsT>(P, sh));
            for (int k = 0; k < P.kt && early < C::kStages; ++k, ++early) {
                load_stage<NV, BN, false, 2>(sh, st, 0, ring, w, ok);
                w.x += kStageK, w.b_tile += C::kSc;
            }
        }
        tc::wait_for_previous();
        ring = Ring<C::kStages>();
        for (; walk.q < used; walk.next(P)) {
            StageAt w = at(walk.tile<kRowsT>(P, sh));
            for (int k = 0; k < P.kt; ++k) {
                if (early > 0) {
                    --early;
                    load_stage<NV, BN, false, 1>(sh, st, 0, ring, w, ok);
                } else {
                    load_stage(sh, st, 0, ring, w, ok);
                }
                w.x += kStageK, w.a_tile += C::kSc, w.b_tile += C::kSc;
            }
        }
        end_loads<C::kStages>(sh, 0, ring.issued, ok);
    } else if (warp == 1) {
        tc::wait_for_previous();   // (all of the block's warps, that it does not end before the digits' kernel)
        Ring<C::kStages> ring;
        int n = 0;
        bool ok = true;
        for (; walk.q < used; walk.next(P)) multiply_tile<kLen>(sh, st, n, ring, P.k_bytes, ok);
        if (!ok || *static_cast<volatile uint32_t *>(&sh.dead)) settle<C::kStages>(sh.empty, ring.issued);
    } else if (warp >= kDrain) {
        const int q = warp & 3, h = (warp - kDrain) >> 2, digit = lane & (kDigits - 1);   // lanes 32 q .., columns from 64 h
        int n = 0, last = -1;
        Scale gate, linear;
        tc::wait_for_previous();
        for (; walk.q < total; walk.next(P)) {
            const Tile t = walk.tile<kRowsT>(P, sh);
            const int rows = t.rows - 32 * q;   // of digits
            const int64_t row = (static_cast<int64_t>(t.row) + 32 * q + lane) >> kDigitsLog, c0 = static_cast<int64_t>(t.nt) * 128 + h * kCols;
            const bool on = lane < rows;
            if (t.g == P.E) {
                for (int c = digit; c < kCols && c0 + c < P.N; c += kDigits)
                    if (on) put(P.out, P.out_type, row * P.N + c0 + c, 0.0f);
                continue;
            }
            const RowInfo info = on ? P.info[row] : RowInfo{0, 0};
            const float p = kGlu && P.probs && on ? P.probs[row] : 1.0f;
            if (t.g != last) {
                gate.of(NV ? P.amax_b[t.g * P.b_groups] : -1.0f);
                if (kGlu) linear.of(NV ? P.amax_b[(t.g + 1) * P.b_groups - 1] : -1.0f);
                last = t.g;
            }
            uint32_t v[kGlu ? 2 * kCols : kCols];
            if (!take_tile<BN, C::kAcc, false, kLen, kGlu ? 2 : 1>(sh, n, P.kt, q, lane, h * kCols, 128 + h * kCols, v)) break;
            const float unit = __uint_as_float(static_cast<uint32_t>(127 + digit_exponent<NV>(digit)) << 23);
            const float weight = info.infinite ? (digit < info.infinite ? __uint_as_float(0x7F800000u) : 0.0f) : unit;
#pragma unroll
            for (int j = 0; j < kCols; j += 8) {
                if (c0 + j >= P.N) break;
                float y = gate(sum_digits(v + j, weight, lane), info.t);
                if constexpr (kGlu) {
                    const float u = linear(sum_digits(v + kCols + j, weight, lane), info.t);
                    y = p * glu::value<kClamp>(P.act, make_float2(y, y), make_float2(u, u)).x;
                }
                if (on && c0 + j + digit < P.N) put(P.out, P.out_type, row * P.N + c0 + j + digit, y);
            }
        }
    }
    close_block<false>(sh, warp, C::kCols, P.status);
}

// -------------------------------------------------------------------- host

template <bool NV, bool kGlu, bool kClamp> gsa_status launch_few(const FewParams &P, int64_t tiles, cudaStream_t s) {
    static PerDevice pairs;
    return launch<false, FewParams>(grouped_few<NV, kGlu, kClamp>, P, kThreads, FewCfg<NV, kGlu>::kSmem, tiles * P.n_tiles, s, pairs);
}

template <bool NV> gsa_status launch_digits(const DigitParams &P, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(P.M));
    cfg.blockDim = dim3(kDigitThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see tc::wait_for_previous
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, split_digits<NV>, P) == cudaSuccess ? GSA_OK : cuda_error();
}

// Workspace: what the rows are, their digits, and those's scales (byte offsets).
struct DigitSpace {
    size_t codes = 0, scales = 0, bytes = 0;
    int64_t tiles;   // row tiles of scales, whatever the split
    DigitSpace(int64_t E, int64_t M, int64_t K, bool nv) {
        auto take = [&](int64_t n) {
            const size_t at = bytes;
            bytes += (static_cast<size_t>(n) + 255) / 256 * 256;
            return at;
        };
        tiles = (kDigits * M + 127) / 128 + (E < M ? E : M);
        take(M * static_cast<int64_t>(sizeof(RowInfo)));
        codes = take(kDigits * M * (nv ? K / 2 : K));
        scales = take(tiles * ((K / (nv ? 16 : 32) + 3) / 4) * kScaleTile);
    }
};

bool in_range(int64_t E, int64_t M, int64_t N, int64_t K) {
    return E <= kMaxE && K % 64 == 0 && K <= (int64_t(1) << 30) && M < (int64_t(1) << 28) && N < (int64_t(1) << 30) / E - 256;
}

bool known_type(int32_t t) { return t == GSA_BF16 || t == GSA_FP16 || t == GSA_FP32; }

gsa_status run_few(FewParams &P, bool glu, const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split, int64_t E, int64_t M, int64_t N,
                   int64_t K, int32_t recipe_kind, int32_t b_groups, void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
                   gsa_stream_t stream) {
    if (!b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (!known_type(x_dtype) || !known_type(out_dtype) || (b_groups != 1 && b_groups != 2)) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    const int64_t sides = glu ? 2 : 1;
    if (!in_range(E, M, N, K)) return GSA_ERR_UNSUPPORTED;
    if (glu && b_groups == 1 && N % 128 != 0) return GSA_ERR_UNSUPPORTED;
    if (M == 0) return GSA_OK;
    if (!x || !b->data || !b->scale || !out || (!split && E != 1) || (nv && !b->amax)) return GSA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(b->data, 16) || !aligned(b->scale, 16) || !aligned(out, 16) || !aligned(split, 8) || !aligned(b->amax, 4) ||
        !aligned(P.probs, 4) || !aligned(workspace, 256))
        return GSA_ERR_ALIGNMENT;
    const int64_t n128 = (N + 127) / 128, cols = (K / (nv ? 16 : 32) + 3) / 4, k_bytes = nv ? K / 2 : K;
    if (b->data_bytes < E * sides * N * k_bytes || b->scale_bytes < E * sides * n128 * cols * kScaleTile) return GSA_ERR_INVALID_ARG;
    const DigitSpace ws(E, M, K, nv);
    if (ws.tiles * cols >= (int64_t(1) << 31) || E * sides * n128 * cols >= (int64_t(1) << 31)) return GSA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ws.bytes) return GSA_ERR_WORKSPACE;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    const int sc = nv ? 4 : 1;
    if (!map_codes(&P.tm_a, w + ws.codes, kDigits * M, k_bytes, kBoxA) || !map_codes(&P.tm_b, b->data, E * sides * N, k_bytes, 128) ||
        !map_scales(&P.tm_sa, w + ws.scales, ws.tiles * cols, sc) || !map_scales(&P.tm_sb, b->scale, E * sides * n128 * cols, sc))
        return cuda_error();
    P.status = gemm_status::word();
    if (!P.status) return cuda_error();
    P.split = split;
    P.amax_b = b->amax;
    P.out = out;
    P.M = kDigits * M;
    P.N = N;
    P.kt = static_cast<int>((k_bytes + kStageK - 1) / kStageK);
    P.k_bytes = static_cast<int>(k_bytes);
    P.E = static_cast<int>(E);
    P.n_tiles = static_cast<int>(n128);
    P.b_scale_rows = static_cast<int>(sides * n128);
    P.up_tiles = static_cast<int>(n128);
    P.b_groups = b_groups;
    P.scale_cols = static_cast<int>(cols);
    P.a_scale_tiles = ws.tiles;
    P.out_type = out_dtype;
    P.info = reinterpret_cast<const RowInfo *>(w);
    DigitParams D;
    D.x = x;
    D.split = split;
    D.codes = w + ws.codes, D.scales = w + ws.scales;
    D.info = reinterpret_cast<RowInfo *>(w);
    D.M = M;
    D.tiles = ws.tiles;
    D.E = P.E, D.K = static_cast<int>(K), D.x_type = x_dtype, D.scale_cols = P.scale_cols;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const gsa_status st = nv ? launch_digits<true>(D, s) : launch_digits<false>(D, s);
    if (st != GSA_OK) return st;
    if (!glu) return nv ? launch_few<true, false, false>(P, ws.tiles, s) : launch_few<false, false, false>(P, ws.tiles, s);
    if (P.act.clamped) return nv ? launch_few<true, true, true>(P, ws.tiles, s) : launch_few<false, true, true>(P, ws.tiles, s);
    return nv ? launch_few<true, true, false>(P, ws.tiles, s) : launch_few<false, true, false>(P, ws.tiles, s);
}

}  // namespace

extern "C" {

size_t gsa_grouped_gemv_workspace_size(int64_t E, int64_t M, int64_t K, int32_t recipe_kind) {
    if (E <= 0 || M <= 0 || K <= 0 || !in_range(E, M, 1, K) || (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4)) return 0;
    return DigitSpace(E, M, K, recipe_kind == GSA_NVFP4).bytes;
}

gsa_status gsa_grouped_gemv(const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M, int64_t N,
                            int64_t K, int32_t recipe_kind, void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
                            gsa_stream_t stream) {
    FewParams P;
    std::memset(&P, 0, sizeof(P));
    return run_few(P, false, x, x_dtype, b, split_sizes_dev, E, M, N, K, recipe_kind, 1, out, out_dtype, workspace, workspace_bytes, stream);
}

gsa_status gsa_grouped_glu_gemv(const void *x, int32_t x_dtype, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M, int64_t N,
                                int64_t K, int32_t recipe_kind, int32_t act_kind, const gsa_act_params *act_params, const float *probs,
                                int32_t b_groups, void *y, int32_t out_dtype, void *workspace, size_t workspace_bytes, gsa_stream_t stream) {
    FewParams P;
    std::memset(&P, 0, sizeof(P));
    if (!glu::act_of(act_kind, act_params, P.act)) return GSA_ERR_INVALID_ARG;
    P.probs = probs;
    return run_few(P, true, x, x_dtype, b, split_sizes_dev, E, M, N, K, recipe_kind, b_groups, y, out_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
