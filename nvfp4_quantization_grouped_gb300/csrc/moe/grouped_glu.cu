// grouped_glu.cu -- the gated first projection of the experts in one product, and its
// gradient, on block-scaled operands (MXFP8 / NVFP4), with their C entry points.
//
//   g[r, n] = sum_k A[r, k] B_e[n, k],  u[r, n] = sum_k A[r, k] B_e[N + n, k]     rows r of expert e
//   y[r, n] = p_r act(g, u)                                                       (glu_act.cuh)
//   dg = dy p d act / d g,  du = dy p d act / d u,  dp_r = sum_n dy act(g, u)
//
// A tile of the grouped product whose 256 columns are 128 of the gate and the same 128 of the
// linear side: a pair of blocks loads one each, the draining warps find g and u of an element
// in the same lane, and neither is rounded or written.  The gradient multiplies again instead
// of reading them: a training step keeps only the quantized rows, which the weight gradient
// needs anyway.  A lane holds a row's 32 columns, so dp takes no shuffles: each warp writes a
// partial sum a row, and a second kernel adds them in order.
//   65536 rows over 32 experts, N and K 2048, NVFP4: 188 to 202 us alone in a graph (5.6 PFLOP/s; 5900
// cycles a tile, of which products and scale copies take 5700), 212 to 220 among other calls;
// gradient 258 to 270, 9500 cycles a tile: the draining warps' round, of which the mathematics take
// 2400 and 64 KB of results, which leave the block at 16 to 20 bytes a cycle, 3500 to 4000, during which
// its load/store unit serves nothing else (without the stores 204 us; a pair that alone of all stores
// takes as long as all do).  The same with half or all of the results as TMA stores, behind which the
// operands' copies then wait (260 to 265), with a third buffer for them (268), with units that start
// up to a tile apart (no change), and with the rows' operand shared by two pairs of a cluster
// through multicast (269; forward 201).
// 262144 x 4096 x 2048 MXFP8 over 128 experts: 3080 to 3150 us (2.8 PFLOP/s, what the power limit
// leaves).  512 rows over 128 experts, 2048 x 2048 NVFP4: 66 to 71 us, the weights at 6.1 TB/s.
#include "gemm_core.cuh"
#include "glu_act.cuh"

namespace {

constexpr int kBN = 256, kSide = kBN / 2, kCols = 32;   // columns of a tile; of one side; of one side that a warp drains
// Sixteen warps drain (8 in the grouped product): with 64 accumulators a side a warp has too few registers left to work on
// several elements at once (gradient, 65536 x 2048 x 2048 NVFP4: 323 -> 287 us).
constexpr int kWarps = 16, kFirst = 2, kGluThreads = 32 * (kFirst + kWarps);   // (the first of them)
constexpr int kBuf = 32 * 64;   // a warp's piece of dy or results: 32 rows x 64 bytes
static_assert(kGluThreads <= kMaxThreads, "threads");

constexpr int kParts = kSide / kCols;   // of a row's sum of dp, a tile

struct GluParams : GemmParams {   // N: columns of one side; out: y, or dx
    glu::Act act;
    const float *probs;
    const __nv_bfloat16 *dy;
    float *part;          // [kParts n_tiles][M] partial sums of dp
    uint32_t *status;     // the device's word for reports
    uint32_t *bad;        // this call's: a bad split (with part)
    int up_tiles;         // scale tiles from a gate row's to its linear row's, in rows of tiles
    int b_groups;         // amax of B an expert
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes) {   // 16 bytes; zeros from `bytes` on
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Row r's 16-byte chunk c of a warp's buffer: eight lanes that hold one chunk of eight rows, or both of two rows' four, meet
// no bank twice.
__device__ __forceinline__ uint32_t chunk(uint32_t buf, int r, int c) { return buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }

// A warp's 32 x 32 piece of dy into its buffer, zeros where there is none.
__device__ __forceinline__ void load_dy(uint32_t buf, const OutAt<const __nv_bfloat16> &w, const __nv_bfloat16 *any, int lane) {
    if (w.wide) {
        const int c = lane & 3;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 8) {
            const int r = r0 + (lane >> 2);
            const bool in = r < w.rows && 8 * c < w.cols;
            copy_async(chunk(buf, r, c), in ? w.o + r * w.pitch + 8 * c : any, in ? 16 : 0);
        }
    } else if (w.pitch % 2 == 0) {   // rows start on 4 bytes: two columns a lane
        const int c = lane & 15;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 2) {
            const int r = r0 + (lane >> 4);
            const bool in = r < w.rows && 2 * c < w.cols;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(chunk(buf, r, c >> 2) + 4 * (c & 3)), "l"(in ? w.o + r * w.pitch + 2 * c : any),
                         "r"(in ? 4 : 0)
                         : "memory");
        }
    } else {   // a column a lane; all rows asked for before the first is there (gradient, 167450 x 1071 x 64 NVFP4: 650 -> 540 to 563 us)
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            uint16_t x = 0;
            if (r < w.rows && lane < w.cols) x = __ldcs(reinterpret_cast<const uint16_t *>(w.o + r * w.pitch + lane));
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(chunk(buf, r, lane >> 3) + 2 * (lane & 7)), "h"(x) : "memory");
        }
    }
}

__device__ __forceinline__ float ld_result(uint32_t at, float) { return tc::ld_shared1(at); }
__device__ __forceinline__ __nv_bfloat16 ld_result(uint32_t at, __nv_bfloat16) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
    return __ushort_as_bfloat16(x);
}

// 32 bytes of results to memory.
__device__ __forceinline__ void store_sector(void *p, const uint32_t *x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]),
                 "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// A lane's results: a row's 32 columns, rounded to T as soon as there are eight (they then take half of the registers).
constexpr int kPieceWords = 16;                                        // 64 bytes
template <typename T> constexpr int kPerPiece = 64 / sizeof(T);       // columns of them
template <typename T> struct Results {
    uint32_t w[kCols * sizeof(T) / 4];
    __device__ __forceinline__ void put(int j, const uint32_t *v) {   // columns j .. j + 7
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / kPer; ++i) finish<false>(v + i * kPer, 1.0f, 1.0f, reinterpret_cast<uint32_t(&)[4]>(w[(j + i * kPer) / kPer * 4]), T());
    }
};

// A warp's 32 x 32 results, straight from the registers: 64 bytes of an even lane's row by it and the next, then of the odd
// one's.  (A row a lane, an instruction meets 32 lines: gradient, 65536 x 2048 x 2048 NVFP4, 278 -> 268 us.)
template <typename T> __device__ __forceinline__ void store_pairs(const Results<T> &v, const OutAt<T> &w, int lane) {
    constexpr int kPer = kPerPiece<T> / 2;
    const bool odd = lane & 1;
    const int even = lane & ~1, c = odd ? kPer : 0;
    T *o = w.o + even * w.pitch + c;
#pragma unroll
    for (int j = 0; j < kCols; j += 2 * kPer) {
        const uint32_t *x = v.w + j / (2 * kPer) * kPieceWords;
        uint32_t first[8], second[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? x[i] : x[8 + i], 1);
            first[i] = odd ? got : x[i];
            second[i] = odd ? x[8 + i] : got;
        }
        if (j + c < w.cols && even < w.rows) store_sector(o + j, first);
        if (j + c < w.cols && even + 1 < w.rows) store_sector(o + w.pitch + j, second);
    }
}

// A warp's 32 x 32 results to memory.  Whole sectors from the lanes' registers wherever rows start on them: the products and
// their copies use most of shared memory's bandwidth, and results that pass through it slow them (forward, 65536 x 2048 x 2048
// NVFP4: 220 -> 216 us).  Else by way of the warp's buffer, 64 bytes of a row at a time.
template <typename T> __device__ __forceinline__ void store_rows(const Results<T> &v, uint32_t buf, const OutAt<T> &w, int lane) {
    constexpr int kPer = 16 / sizeof(T), kPiece = kPerPiece<T>;
    if (w.wide && (w.pitch | w.cols) * sizeof(T) % 32 == 0 && reinterpret_cast<uintptr_t>(w.o) % 32 == 0) {
        store_pairs(v, w, lane);
        return;
    }
#pragma unroll
    for (int j = 0; j < kCols; j += kPiece) {
        if (j >= w.cols) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::st_shared(chunk(buf, lane, c), v.w + j / kPiece * kPieceWords + 4 * c);
        __syncwarp();
        if (w.wide) {   // (16 bytes a lane straight from the registers: gradient of 4999 x 1000 x 1024 MXFP8 30 us, this way 27)
            const int c = lane & 3;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {
                const int r = r0 + (lane >> 2);
                const uint4 x = tc::ld_shared(chunk(buf, r, c));
                if (r < w.rows && j + c * kPer < w.cols) *reinterpret_cast<uint4 *>(w.o + r * w.pitch + j + c * kPer) = x;
            }
        } else if (sizeof(T) == 4 || ((w.pitch | w.cols) % 2 == 0 && reinterpret_cast<uintptr_t>(w.o) % 4 == 0)) {
            // 4 bytes a lane (100000 x 1074 x 64 NVFP4: 124 -> 101 us, gradient 325 -> 250)
            constexpr int kOne = 4 / sizeof(T);
            const int c = lane & 15;
            if (j + c * kOne < w.cols) {
#pragma unroll 16
                for (int r = lane >> 4; r < 32; r += 2) {
                    const float x = tc::ld_shared1(chunk(buf, r, c >> 2) + 4 * (c & 3));
                    if (r < w.rows) *reinterpret_cast<float *>(w.o + r * w.pitch + j + c * kOne) = x;
                }
            }
        } else {   // a column a lane
            const int c = lane & (kPiece - 1);
            if (j + c < w.cols) {
#pragma unroll 16
                for (int r = lane / kPiece; r < 32; r += 32 / kPiece) {
                    const uint32_t at = chunk(buf, r, c / kPer) + sizeof(T) * (c % kPer);
                    if (r < w.rows) w.o[r * w.pitch + j + c] = ld_result(at, T());
                }
            }
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
}

// A pair of sums times what their units leave (NVFP4).
template <bool NV> __device__ __forceinline__ float2 pair_of(const uint32_t *v, float u) {
    const float2 f = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
    return NV ? glu::mul2(f, u) : f;
}

// 1 / (S_A S_B) of a side's sums, where FP32 holds it to full precision (nearly always).  Where the product is subnormal, past
// FP32's end, infinite or NaN: minus the smaller factor, and sums are multiplied by minus the larger one (*first) before.
// Sums are 0 or 2^-20 to 2^53, so that this first step leaves FP32's range only where the result does, and what an infinite
// amax makes of its zero sums is NaN.
__device__ __forceinline__ float unit_of(float amax_a, float amax_b, float *first) {
    const float a = __fdiv_rn(1.0f, tensor_scale(amax_a)), b = __fdiv_rn(1.0f, tensor_scale(amax_b)), u = a * b;
    const bool near = u >= 0x1p-126f && u <= 3.402823466e38f;
    *first = near ? 1.0f : -fmaxf(a, b);
    return near ? u : -fminf(a, b);
}

struct GluShared : GemmShared {
    float first[kWarps][2];   // of a warp's gate and linear sums: read where it is not 1 alone (kept in registers, of which the
                              // gradient has too few: 269 -> 293 us, 65536 x 2048 x 2048)
};

// What a draining warp has in shared memory: a buffer for results, or (gradient) two for dy of this tile, whose place dx
// takes, and of the next; probs of the rows of both.
constexpr int kProbs = 32 * 4;
template <bool kBwd> constexpr int kOwn = (kBwd ? 2 : 1) * kBuf + 2 * kProbs;
template <bool NV, bool kPair, bool kBwd> using GluCfg = Cfg<NV, kBN, kPair, kWarps * kOwn<kBwd>>;

template <bool NV, bool kPair, bool kBwd, bool kClamp, typename T>
__global__ void __launch_bounds__(kGluThreads, 1) grouped_glu(const __grid_constant__ GluParams P) {
    using C = GluCfg<NV, kPair, kBwd>;
    // Sums of the gradient in short pieces: dp is an FP32 result, and adds up what the tensor core cuts off of both sides.
    constexpr int kLen = kBwd ? kPiece<float> : kPiece<T>;
    extern __shared__ uint8_t dyn[];
    __shared__ GluShared sh;
    static_assert(sizeof(GluShared) <= kStatic, "shared memory");
    constexpr int kRows = kPair ? 2 * kRowsT : kRowsT;
    const int warp = known_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
    const int half = kPair ? blockIdx.x & 1 : 0;
    const Stages<NV, kBN, kPair> st(dyn);
    open_block<C::kStages, kPair, kWarps>(sh, warp, 1, C::kCols);
    tc::allow_next();
    tc::wait_for_previous();
    scan_split<kRows>(P, sh);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (sh.bad) atomicOr(P.status, ERR_SPLIT);
        if (kBwd && P.part) *P.bad = sh.bad;
    }
    const int total = known_uniform(sh.bad ? 0 : sh.tile0[P.E + 1]), used = known_uniform(sh.bad ? 0 : sh.tile0[P.E]);   // row tiles; the rest is zeros
    Walk walk(P, unit, units);

    if (warp == 0) {
        if (tc::elect()) {
            tc::prefetch_map(&P.tm_a);
            tc::prefetch_map(&P.tm_b);
        }
        Ring<C::kStages> ring;
        bool ok = true;
        while (walk.q < used) {
            Tile t = walk.tile<kRows>(P, sh);
            StageAt w{&P.tm_a, &P.tm_b, &P.tm_sa, &P.tm_sb}, ahead = w;
            auto rows_at = [&](StageAt &s) {   // what the column tiles of a row tile share
                s.x = 0;
                s.a_row = t.row + half * kRowsT;
                s.a_tile = (known_uniform(sh.scale0[t.g]) + t.mt * (kRows / 128) + half) * P.scale_cols;
            };
            rows_at(w);
            w.a_boxes = (t.rows + kBoxA - 1) / kBoxA;
            w.b_row = static_cast<int>((2 * t.g + half) * P.N) + t.nt * kSide;   // the pair's second block has the linear side
            w.b_row_step = static_cast<int>(P.N);
            w.b_tile = (t.g * P.b_scale_rows + t.nt) * P.scale_cols;
            w.b_tile_step = P.up_tiles * P.scale_cols;
            walk.next(P);
            bool first = false;   // the next tile is its rows' first
            if (kPair && walk.q < used && walk.nt == 0) {
                first = true;
                t = walk.tile<kRows>(P, sh);
                rows_at(ahead);
            }
            for (int k = 0; k < P.kt; ++k) {
                load_stage(sh, st, half, ring, w, ok);
                if (first) prefetch_rows(ahead);
                w.x += kStageK, w.a_tile += C::kSc, w.b_tile += C::kSc;
                ahead.x += kStageK, ahead.a_tile += C::kSc;
            }
        }
        end_loads<C::kStages>(sh, half, ring.issued, ok);
    } else if (warp == 1 && half == 0) {
        Ring<C::kStages> ring;
        int n = 0;
        bool ok = true;
        for (; walk.q < used; walk.next(P)) multiply_tile<kLen>(sh, st, n, ring, P.k_bytes, ok);
        if (!ok || *static_cast<volatile uint32_t *>(&sh.dead)) settle<C::kStages>(sh.empty, ring.issued);
    } else if (warp >= kFirst) {
        const int q = warp & 3, h = (warp - kFirst) >> 2;   // lanes 32 q .., 32 columns of both sides from 32 h
        const int r0 = half * kRowsT + 32 * q, c0 = h * kCols;
        const uint32_t own = st.a(C::kStages) + (warp - kFirst) * kOwn<kBwd>;
        uint32_t turn = 0;   // 0 or 1: which dy buffer and probs are this tile's
        auto buf = [&](uint32_t i) { return own + 2 * kProbs + (kBwd ? i * kBuf : 0); };
        int n = 0, last = -1;
        float ug = 1.0f, uu = 1.0f;   // NVFP4: the units of a gate sum and of a linear sum
        auto out_at = [&](int row, int nt, int rows, int cols) {
            OutAt<T> w;
            w.pitch = kBwd ? 2 * P.N : P.N;
            w.o = static_cast<T *>(P.out) + row * w.pitch + nt * kSide + c0;
            w.cols = cols, w.rows = rows;
            w.wide = P.N * sizeof(T) % 16 == 0;
            w.add = false;
            return w;
        };
        auto ask = [&](uint32_t i) {   // what the tile that the walk has come to needs from memory
            if (walk.q >= used) return;
            const Tile t = walk.tile<kRows>(P, sh);
            const int row = t.row + r0, rows = t.rows - r0;
            if (P.probs && lane < rows)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(own + i * kProbs + 4 * lane), "l"(P.probs + row + lane) : "memory");
            if (kBwd) {
                OutAt<const __nv_bfloat16> d;
                d.o = P.dy + row * P.N + t.nt * kSide + c0;
                d.pitch = P.N;
                d.cols = P.N - t.nt * kSide - c0, d.rows = rows;
                d.wide = P.N % 8 == 0;
                load_dy(buf(i), d, P.dy, lane);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        ask(0);
        while (walk.q < total) {
            const Tile t = walk.tile<kRows>(P, sh);
            const int row = t.row + r0, rows = t.rows - r0, nt = t.nt, cols = static_cast<int>(P.N) - nt * kSide - c0;   // the warp's part
            auto partial = [&](float dp) {
                if (kBwd && P.part && lane < rows) P.part[(kParts * nt + h) * P.M + row + lane] = dp;
            };
            walk.next(P);
            if (t.g == P.E) {
                if (P.out) {
                    OutAt<T> w = out_at(row, nt, rows, cols);
                    zero_tile<kCols>(w, lane);
                    if (kBwd) {
                        w.o += P.N;
                        zero_tile<kCols>(w, lane);
                    }
                }
                partial(0.0f);
                continue;
            }
            if (NV && t.g != last) {
                const float a = P.amax_a[t.g];
                float fg, fu;
                ug = unit_of(a, P.amax_b[t.g * P.b_groups], &fg);
                uu = unit_of(a, P.amax_b[(t.g + 1) * P.b_groups - 1], &fu);
                __syncwarp();
                if (lane == 0) sh.first[warp - kFirst][0] = fg, sh.first[warp - kFirst][1] = fu;
                last = t.g;
            }
            wait_copies();
            ask(turn ^ 1);
            uint32_t v[2 * kCols];   // columns of g, and of u
            if (!take_tile<kBN, C::kAcc, kPair, kLen, 2>(sh, n, P.kt, q, lane, c0, kSide + c0, v)) break;
            if (NV && fminf(ug, uu) < 0.0f) {
                const float fg = sh.first[warp - kFirst][0], fu = sh.first[warp - kFirst][1];
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    v[j] = __float_as_uint(__uint_as_float(v[j]) * fg);
                    v[kCols + j] = __float_as_uint(__uint_as_float(v[kCols + j]) * fu);
                }
            }
            const float p = P.probs ? tc::ld_shared1(own + turn * kProbs + 4 * lane) : 1.0f;
            if (kBwd) {
                if (cols < kCols) {   // past the last column: whatever the next rows and the scales' padding give, NaN too
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        if (j >= cols) v[j] = v[kCols + j] = 0;
                }
                float2 dp = make_float2(0.0f, 0.0f);
                Results<T> of_gate, of_linear;
#pragma unroll
                for (int j = 0; j < kCols; j += 8) {
                    const uint4 x = tc::ld_shared(chunk(buf(turn), lane, j >> 3));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 dy = make_float2(__uint_as_float(xs[k >> 1] << 16), __uint_as_float(xs[k >> 1] & 0xFFFF0000u));
                        uint32_t *g = v + j + k, *u = v + kCols + j + k;
                        float2 dg, du;
                        const float2 y = glu::gradient<kClamp>(P.act, pair_of<NV>(g, ug), pair_of<NV>(u, uu), glu::mul2(dy, p), dg, du);
                        dp = glu::fma2(dy, y, dp);
                        g[0] = __float_as_uint(dg.x), g[1] = __float_as_uint(dg.y);
                        u[0] = __float_as_uint(du.x), u[1] = __float_as_uint(du.y);
                    }
                    of_gate.put(j, v + j);
                    of_linear.put(j, v + kCols + j);
                }
                __syncwarp();
                partial(dp.x + dp.y);
                if (P.out) {
                    OutAt<T> w = out_at(row, nt, rows, cols);
                    store_rows(of_gate, buf(turn), w, lane);
                    w.o += P.N;
                    store_rows(of_linear, buf(turn), w, lane);
                }
            } else {
                Results<T> of_y;
#pragma unroll
                for (int j = 0; j < kCols; j += 8) {
#pragma unroll
                    for (int k = j; k < j + 8; k += 2) {
                        const float2 y = glu::mul2(glu::value<kClamp>(P.act, pair_of<NV>(v + k, ug), pair_of<NV>(v + kCols + k, uu)), p);
                        v[k] = __float_as_uint(y.x), v[k + 1] = __float_as_uint(y.y);
                    }
                    of_y.put(j, v + j);
                }
                store_rows(of_y, buf(0), out_at(row, nt, rows, cols), lane);
            }
            turn ^= 1;
        }
        wait_copies();   // after a wait that ran out: those under way
    }
    close_block<kPair>(sh, warp, C::kCols, P.status);
}

// dp_r: a row's partial sums, in order.
__global__ void __launch_bounds__(256) sum_partials(const float *part, const uint32_t *bad, int parts, int64_t M, float *dprobs) {
    const int64_t r = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (*bad || r >= M) return;
    float s = 0.0f;
    for (int j = 0; j < parts; ++j) s += __ldcs(part + j * M + r);
    dprobs[r] = s;
}

template <bool kBwd> gsa_status launch_glu(const GluParams &P, bool nv, bool pair, int32_t out_dtype, int64_t tiles, cudaStream_t s) {
    auto go = [&](auto fmt, auto pairs, auto clamp, auto type) {
        constexpr bool NV = decltype(fmt)::value, kPair = decltype(pairs)::value;
        static PerDevice clusters;
        return launch<kPair, GluParams>(grouped_glu<NV, kPair, kBwd, decltype(clamp)::value, decltype(type)>, P, kGluThreads,
                                        GluCfg<NV, kPair, kBwd>::kSmem, tiles * P.n_tiles, s, clusters);
    };
    auto typed = [&](auto fmt, auto pairs, auto clamp) {
        return out_dtype == GSA_BF16 ? go(fmt, pairs, clamp, __nv_bfloat16()) : go(fmt, pairs, clamp, float());
    };
    auto clamped = [&](auto fmt, auto pairs) { return P.act.clamped ? typed(fmt, pairs, std::true_type()) : typed(fmt, pairs, std::false_type()); };
    auto paired = [&](auto fmt) { return pair ? clamped(fmt, std::true_type()) : clamped(fmt, std::false_type()); };
    return nv ? paired(std::true_type()) : paired(std::false_type());
}

// Checks the arguments that both directions take, fills P and says whether pairs take the tiles.
gsa_status glu_params(GluParams &P, bool &pair, int64_t &tiles, const gsa_qin *a, const gsa_qin *b, const int64_t *split, int64_t E, int64_t M,
                      int64_t N, int64_t K, int32_t recipe_kind, int32_t act_kind, const gsa_act_params *act, const float *probs,
                      int32_t b_groups, int32_t out_dtype, bool has_space) {
    std::memset(&P, 0, sizeof(P));
    if (!a || !b || E <= 0 || M < 0 || N <= 0 || K <= 0) return GSA_ERR_INVALID_ARG;
    if (recipe_kind != GSA_MXFP8 && recipe_kind != GSA_NVFP4) return GSA_ERR_INVALID_ARG;
    if (out_dtype != GSA_BF16 && out_dtype != GSA_FP32) return GSA_ERR_INVALID_ARG;
    if (b_groups != 1 && b_groups != 2) return GSA_ERR_INVALID_ARG;
    if (!glu::act_of(act_kind, act, P.act)) return GSA_ERR_INVALID_ARG;
    const bool nv = recipe_kind == GSA_NVFP4;
    if (E > kMaxE || K % 64 != 0 || K > (int64_t(1) << 30) || M >= (int64_t(1) << 31) - 256 || N >= (int64_t(1) << 30) / E - 256)
        return GSA_ERR_UNSUPPORTED;
    if (b_groups == 1 && N % 128 != 0) return GSA_ERR_UNSUPPORTED;   // the linear rows' scales start inside a tile
    if (M == 0) return GSA_OK;
    if (!a->data || !a->scale || !b->data || !b->scale || !split) return GSA_ERR_INVALID_ARG;
    if (nv && (!a->amax || !b->amax)) return GSA_ERR_INVALID_ARG;
    if (!aligned(a->data, 16) || !aligned(a->scale, 16) || !aligned(b->data, 16) || !aligned(b->scale, 16) || !aligned(split, 8) ||
        !aligned(a->amax, 4) || !aligned(b->amax, 4) || !aligned(probs, 4))
        return GSA_ERR_ALIGNMENT;
    const int64_t k_bytes = nv ? K / 2 : K, cols = (K / (nv ? 16 : 32) + 3) / 4;
    const int64_t n128 = (N + 127) / 128, a_rows = a->scale_bytes / (kScaleTile * cols);
    if (a->data_bytes < M * k_bytes || b->data_bytes < 2 * E * N * k_bytes || a_rows < 1 ||
        b->scale_bytes < 2 * E * n128 * cols * kScaleTile)
        return GSA_ERR_INVALID_ARG;
    if (a_rows * cols >= (int64_t(1) << 31) || 2 * E * n128 * cols >= (int64_t(1) << 31)) return GSA_ERR_UNSUPPORTED;
    if (!has_space) return GSA_ERR_WORKSPACE;
    // Pairs of blocks (256 rows) from 128 rows an expert on and where there is a tile of theirs for every two SMs (76 pairs on
    // 152), single blocks (128 rows) else.  By M and E: the split is on the device.
    // Pairs / singles, us, even splits of 128 experts, 2048 x 2048: 96 rows an expert 113 / 103 (NVFP4), 197 / 180 (MXFP8),
    // gradient 138 / 134 and 226 / 203; 128 rows 116 / 113, 200 / 200, 147 / 161, 233 / 224; 192 rows 120 / 133, 204 / 239,
    // 155 / 197, 244 / 267.  Few tiles, 8 experts x 256 rows, 1024 x 1024: 9.9 / 8.7, 11.5 / 10.7, 17.2 / 14.9, 18.2 / 16.4.
    const int sms = sm_count();
    if (!sms) return cuda_error();
    pair = M >= 128 * E && M / 256 * n128 >= sms / 2;
    const int sc = nv ? 4 : 1;
    if (!map_codes(&P.tm_a, a->data, M, k_bytes, pair ? kRowsT : kBoxA) || !map_codes(&P.tm_b, b->data, 2 * E * N, k_bytes, 128) ||
        !map_scales(&P.tm_sa, a->scale, a_rows * cols, sc) || !map_scales(&P.tm_sb, b->scale, 2 * E * n128 * cols, sc))
        return cuda_error();
    P.split = split;
    P.amax_a = a->amax;
    P.amax_b = b->amax;
    P.probs = probs;
    P.M = M;
    P.N = N;
    P.kt = static_cast<int>((k_bytes + kStageK - 1) / kStageK);
    P.k_bytes = static_cast<int>(k_bytes);
    P.E = static_cast<int>(E);
    P.n_tiles = static_cast<int>(n128);
    P.b_scale_rows = static_cast<int>(2 * n128);
    P.up_tiles = static_cast<int>(n128);
    P.b_groups = b_groups;
    P.scale_cols = static_cast<int>(cols);
    P.a_scale_tiles = a_rows;
    P.status = gemm_status::word();
    if (!P.status) return cuda_error();
    tiles = (M + kRowsT - 1) / kRowsT + (E < M ? E : M);
    return GSA_OK;
}

constexpr size_t kHead = 256;   // bytes before the partial sums

}  // namespace

extern "C" {

gsa_status gsa_grouped_glu(const gsa_qin *a, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M, int64_t N, int64_t K,
                           int32_t recipe_kind, int32_t act_kind, const gsa_act_params *act_params, const float *probs, int32_t b_groups,
                           void *y, int32_t out_dtype, gsa_stream_t stream) {
    GluParams P;
    bool pair = false;
    int64_t tiles = 0;
    if (a && b && M > 0 && !y) return GSA_ERR_INVALID_ARG;
    if (!aligned(y, 16)) return GSA_ERR_ALIGNMENT;
    const gsa_status st = glu_params(P, pair, tiles, a, b, split_sizes_dev, E, M, N, K, recipe_kind, act_kind, act_params, probs, b_groups, out_dtype, true);
    if (st != GSA_OK || M == 0) return st;
    P.out = y;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launch_glu<false>(P, recipe_kind == GSA_NVFP4, pair, out_dtype, tiles, s);
}

size_t gsa_grouped_glu_bwd_workspace_size(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0 || M >= (int64_t(1) << 31) || N >= (int64_t(1) << 30)) return 0;
    return kHead + (static_cast<size_t>((N + kSide - 1) / kSide) * kParts * M * 4 + 255) / 256 * 256;
}

gsa_status gsa_grouped_glu_bwd(const void *dy_bf16, const gsa_qin *a, const gsa_qin *b, const int64_t *split_sizes_dev, int64_t E, int64_t M,
                               int64_t N, int64_t K, int32_t recipe_kind, int32_t act_kind, const gsa_act_params *act_params,
                               const float *probs, int32_t b_groups, void *dx_opt, int32_t out_dtype, float *dprobs_opt, void *workspace,
                               size_t workspace_bytes, gsa_stream_t stream) {
    GluParams P;
    bool pair = false;
    int64_t tiles = 0;
    if (a && b && M > 0 && (!dy_bf16 || (!dx_opt && !dprobs_opt))) return GSA_ERR_INVALID_ARG;
    if (!aligned(dy_bf16, 16) || !aligned(dx_opt, 16) || !aligned(dprobs_opt, 4) || !aligned(workspace, 256)) return GSA_ERR_ALIGNMENT;
    gsa_status st = glu_params(P, pair, tiles, a, b, split_sizes_dev, E, M, N, K, recipe_kind, act_kind, act_params, probs, b_groups, out_dtype,
                               !dprobs_opt || (workspace && workspace_bytes >= gsa_grouped_glu_bwd_workspace_size(M, N)));
    if (st != GSA_OK || M == 0) return st;
    if (dprobs_opt) {
        P.bad = static_cast<uint32_t *>(workspace);
        P.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kHead);
    }
    P.dy = static_cast<const __nv_bfloat16 *>(dy_bf16);
    P.out = dx_opt;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = launch_glu<true>(P, recipe_kind == GSA_NVFP4, pair, out_dtype, tiles, s);
    if (st != GSA_OK || !dprobs_opt) return st;
    // (As a programmatic dependent: 4999 x 1000 x 1024 MXFP8 28.5 us, this way 26.4.)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((M + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    // the launch's own status: an error that another call left in the runtime is not this one's
    return cudaLaunchKernelEx(&cfg, sum_partials, static_cast<const float *>(P.part), static_cast<const uint32_t *>(P.bad), kParts * P.n_tiles, M,
                              dprobs_opt) == cudaSuccess
               ? GSA_OK
               : cuda_error();
}

}  // extern "C"
