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
// needs anyway.  A lane holds a row's 64 columns, so dp takes no shuffles: each warp writes a
// partial sum a row, and a second kernel adds them in order.
#include "gemm_core.cuh"
#include "glu_act.cuh"

namespace {

constexpr int kBN = 256, kSide = kBN / 2, kCols64 = 64;   // columns of a tile, of one side, of a warp

struct GluParams : GemmParams {   // N: columns of one side; out: y, or dx
    glu::Act act;
    const float *probs;
    const __nv_bfloat16 *dy;
    float *part;          // [2 n_tiles][M] partial sums of dp
    uint32_t *status;     // the device's word for reports
    uint32_t *bad;        // this call's: a bad split (with part)
    int up_tiles;         // scale tiles from a gate row's to its linear row's, in rows of tiles
    int b_groups;         // amax of B an expert
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes) {   // 16 bytes; zeros from `bytes` on
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A warp's 32 x 64 piece of dy into its buffer: row r's 16-byte chunk c at c ^ (r mod 8), zeros where there is none.
__device__ __forceinline__ void load_dy(uint32_t buf, const OutAt<const __nv_bfloat16> &w, const __nv_bfloat16 *any, int lane) {
    if (w.wide) {
        const int c = lane & 7;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 4) {
            const int r = r0 + (lane >> 3);
            const bool in = r < w.rows && 8 * c < w.cols;
            copy_async(buf + r * 128 + ((c ^ (r & 7)) << 4), in ? w.o + r * w.pitch + 8 * c : any, in ? 16 : 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    } else {   // a column a lane, twice
#pragma unroll
        for (int j = 0; j < kCols64; j += 32) {
            const int col = j + lane;
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
                uint16_t x = 0;
                if (r < w.rows && col < w.cols) x = __ldcs(reinterpret_cast<const uint16_t *>(w.o + r * w.pitch + col));
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(buf + r * 128 + (((col >> 3) ^ (r & 7)) << 4) + 2 * (col & 7)), "h"(x) : "memory");
            }
        }
    }
}

__device__ __forceinline__ void wait_dy() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
}

template <bool NV> __device__ __forceinline__ float2 pair_of(const uint32_t *v, float ua, float ub) {
    const float2 f = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
    return NV ? glu::mul2(glu::mul2(f, ua), ub) : f;
}

// The tiles of a unit, without divisions: q counts row tiles over all groups (n_tiles column tiles each, one after another).
struct Walk {
    int q, nt, g, dq, dn;
    __device__ __forceinline__ Walk(const GluParams &P, int unit, int units)
        : q(unit / P.n_tiles), nt(unit % P.n_tiles), g(0), dq(units / P.n_tiles), dn(units % P.n_tiles) {}
    __device__ __forceinline__ void next(const GluParams &P) {
        q += dq, nt += dn;
        if (nt >= P.n_tiles) nt -= P.n_tiles, ++q;
    }
    // The group that q is in: this one or a later one.
    template <int kRows> __device__ __forceinline__ Tile tile(const GluParams &P, const GemmShared &sh) {
        if (sh.tile0[g + 1] <= q) {
            ++g;
            for (int end = P.E + 1; end - g > 1;) {   // the last group that starts at or before q: most may be empty
                const int mid = (g + end) >> 1;
                if (sh.tile0[mid] <= q) g = mid;
                else end = mid;
            }
        }
        Tile t;
        t.g = g, t.nt = nt;
        t.mt = q - sh.tile0[g];
        t.row = sh.row0[g] + t.mt * kRows;
        t.rows = min(kRows, sh.row0[g + 1] - t.row);
        return t;
    }
};

template <bool NV, bool kPair, bool kBwd, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_glu(const __grid_constant__ GluParams P) {
    constexpr int kBufs = kBwd ? 2 : 1;   // the gradient: dy of this tile, whose place dx takes, and of the next
    using C = Cfg<NV, kBN, kPair, kBufs>;
    // Sums of the gradient in short pieces: dp is an FP32 result, and adds up what the tensor core cuts off of both sides.
    constexpr int kLen = kBwd ? kPiece<float> : kPiece<T>;
    extern __shared__ uint8_t dyn[];
    __shared__ GemmShared sh;
    static_assert(sizeof(GemmShared) <= kStatic, "shared memory");
    constexpr int kRows = kPair ? 2 * kRowsT : kRowsT;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x, units = kPair ? gridDim.x >> 1 : gridDim.x;
    const int half = kPair ? blockIdx.x & 1 : 0;
    const Stages<NV, kBN, kPair> st(dyn);
    open_block<C::kStages, kPair>(sh, warp, 1, C::kCols);
    tc::allow_next();
    tc::wait_for_previous();
    scan_split<kRows>(P, sh);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (sh.bad) atomicOr(P.status, ERR_SPLIT);
        if (kBwd && P.part) *P.bad = sh.bad;
    }
    const int total = sh.bad ? 0 : sh.tile0[P.E + 1], used = sh.bad ? 0 : sh.tile0[P.E];   // row tiles; the rest is zeros
    Walk walk(P, unit, units);

    if (warp == 0) {
        if (tc::elect()) {
            tc::prefetch_map(&P.tm_a);
            tc::prefetch_map(&P.tm_b);
        }
        Ring<C::kStages> ring;
        bool ok = true, first = false;
        auto at = [&] {
            const Tile t = walk.tile<kRows>(P, sh);
            const int g = uniform(t.g);
            StageAt w{&P.tm_a, &P.tm_b, &P.tm_sa, &P.tm_sb};
            w.x = 0;
            w.a_row = uniform(t.row) + half * kRowsT;
            w.a_boxes = uniform((t.rows + kBoxA - 1) / kBoxA);
            w.a_tile = uniform((sh.scale0[g] + t.mt * (kRows / 128) + half) * P.scale_cols);
            w.b_row = uniform(static_cast<int>((2 * g + half) * P.N) + t.nt * kSide);   // the pair's second block has the linear side
            w.b_row_step = static_cast<int>(P.N);
            w.b_tile = uniform((g * P.b_scale_rows + t.nt) * P.scale_cols);
            w.b_tile_step = P.up_tiles * P.scale_cols;
            first = uniform(t.nt) == 0;
            return w;
        };
        StageAt w, next;
        if (walk.q < used) next = at();
        while (uniform(walk.q) < used) {
            w = next;
            walk.next(P);
            const bool more = uniform(walk.q) < used;
            if (more) next = at();
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
        Ring<C::kStages> ring;
        int n = 0;
        bool ok = true;
        for (; uniform(walk.q) < used; walk.next(P)) multiply_tile<kLen>(sh, st, n, ring, P.k_bytes, ok);
        if (!ok || *static_cast<volatile uint32_t *>(&sh.dead)) settle<C::kStages>(sh.empty, ring.issued);
    } else if (warp >= kDrain) {
        const int q = warp & 3, h = (warp - kDrain) >> 2;   // lanes 32 q .., 64 columns of both sides from 64 h
        const int r0 = half * kRowsT + 32 * q, c0 = h * kCols64;
        const uint32_t buf0 = st.a(C::kStages) + (warp - kDrain) * kBufs * kOutBuf;
        uint32_t buf = buf0;
        int n = 0, last = -1;
        float ug = 1.0f, vg = 1.0f, uu = 1.0f, vu = 1.0f;   // NVFP4: what a gate sum (ug, then vg) and a linear sum are multiplied by
        auto out_at = [&](int row, int nt, int rows, int cols) {
            OutAt<T> w;
            w.pitch = kBwd ? 2 * P.N : P.N;
            w.o = static_cast<T *>(P.out) + row * w.pitch + nt * kSide + c0;
            w.cols = cols, w.rows = rows;
            w.wide = P.N * sizeof(T) % 16 == 0;
            w.add = false;
            return w;
        };
        auto get_dy = [&](uint32_t to) {   // of the tile that the walk has come to
            if (walk.q >= used) return;
            const Tile t = walk.tile<kRows>(P, sh);
            OutAt<const __nv_bfloat16> d;
            d.o = P.dy + (t.row + r0) * P.N + t.nt * kSide + c0;
            d.pitch = P.N;
            d.cols = P.N - t.nt * kSide - c0, d.rows = t.rows - r0;
            d.wide = P.N % 8 == 0;
            load_dy(to, d, P.dy, lane);
        };
        auto store = [&](const uint32_t *v, const OutAt<T> &at) {
            if (at.wide) store_warp<kCols64, false, T>(v, 1.0f, 1.0f, buf, at, lane);
            else store_warp_any<kCols64, false, T>(v, 1.0f, 1.0f, buf, at, lane);
        };
        if (kBwd) get_dy(buf);
        while (walk.q < total) {
            const Tile t = walk.tile<kRows>(P, sh);
            const int row = t.row + r0, rows = t.rows - r0, nt = t.nt, cols = static_cast<int>(P.N) - nt * kSide - c0;   // the warp's part
            auto partial = [&](float dp) {
                if (kBwd && P.part && lane < rows) P.part[(2 * nt + h) * P.M + row + lane] = dp;
            };
            walk.next(P);
            if (t.g == P.E) {
                if (P.out) {
                    OutAt<T> w = out_at(row, nt, rows, cols);
                    zero_tile<kCols64>(w, lane);
                    if (kBwd) {
                        w.o += P.N;
                        zero_tile<kCols64>(w, lane);
                    }
                }
                partial(0.0f);
                continue;
            }
            const float p = P.probs && lane < rows ? P.probs[row + lane] : 1.0f;
            if (NV && t.g != last) {
                const float a = P.amax_a[t.g];
                units_of(a, P.amax_b[t.g * P.b_groups], ug, vg);
                uu = ug, vu = vg;
                if (P.b_groups == 2) units_of(a, P.amax_b[2 * t.g + 1], uu, vu);
                last = t.g;
            }
            if (kBwd) {
                wait_dy();
                get_dy(2 * buf0 + kOutBuf - buf);   // a tile ahead, into the other buffer
            }
            uint32_t v[kSide];   // 64 columns of g, and of u
            if (!take_tile<kBN, C::kAcc, kPair, kLen, 2>(sh, n, P.kt, q, lane, c0, kSide + c0, v)) break;
            if (kBwd) {
                if (cols < kCols64) {   // past the last column: whatever the next rows and the scales' padding give, NaN too
#pragma unroll
                    for (int j = 0; j < kCols64; ++j)
                        if (j >= cols) v[j] = v[kCols64 + j] = 0;
                }
                float2 dp = make_float2(0.0f, 0.0f);
                auto all = [&](auto clamp) {
#pragma unroll
                    for (int j = 0; j < kCols64; j += 8) {
                        const uint4 x = tc::ld_shared(buf + lane * 128 + (((j >> 3) ^ (lane & 7)) << 4));
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            const float2 dy = make_float2(__uint_as_float(xs[k >> 1] << 16), __uint_as_float(xs[k >> 1] & 0xFFFF0000u));
                            uint32_t *g = v + j + k, *u = v + kCols64 + j + k;
                            float2 dg, du;
                            const float2 y = glu::gradient<decltype(clamp)::value>(P.act, pair_of<NV>(g, ug, vg), pair_of<NV>(u, uu, vu),
                                                                                   glu::mul2(dy, p), dg, du);
                            dp = glu::fma2(dy, y, dp);
                            g[0] = __float_as_uint(dg.x), g[1] = __float_as_uint(dg.y);
                            u[0] = __float_as_uint(du.x), u[1] = __float_as_uint(du.y);
                        }
                    }
                };
                if (P.act.clamped) all(std::true_type());
                else all(std::false_type());
                __syncwarp();
                partial(dp.x + dp.y);
                if (P.out) {
                    OutAt<T> w = out_at(row, nt, rows, cols);
                    store(v, w);
                    w.o += P.N;
                    store(v + kCols64, w);
                }
                buf = 2 * buf0 + kOutBuf - buf;
            } else {
                auto all = [&](auto clamp) {
#pragma unroll
                    for (int j = 0; j < kCols64; j += 2) {
                        const float2 y = glu::mul2(glu::value<decltype(clamp)::value>(P.act, pair_of<NV>(v + j, ug, vg), pair_of<NV>(v + kCols64 + j, uu, vu)), p);
                        v[j] = __float_as_uint(y.x), v[j + 1] = __float_as_uint(y.y);
                    }
                };
                if (P.act.clamped) all(std::true_type());
                else all(std::false_type());
                store(v, out_at(row, nt, rows, cols));
            }
        }
        if (kBwd) wait_dy();   // after a wait that ran out: the copies under way
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

template <bool NV, bool kPair, bool kBwd, typename T> gsa_status launch_glu(const GluParams &P, int64_t tiles, cudaStream_t s) {
    static PerDevice pairs;
    return launch<kPair, GluParams>(grouped_glu<NV, kPair, kBwd, T>, P, kThreads, Cfg<NV, kBN, kPair, kBwd ? 2 : 1>::kSmem, tiles * P.n_tiles, s, pairs);
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
    pair = M >= 128 * E;
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
    auto typed = [&](auto fmt, auto type) {
        return pair ? launch_glu<decltype(fmt)::value, true, false, decltype(type)>(P, tiles, s)
                    : launch_glu<decltype(fmt)::value, false, false, decltype(type)>(P, tiles, s);
    };
    auto sized = [&](auto fmt) { return out_dtype == GSA_BF16 ? typed(fmt, __nv_bfloat16()) : typed(fmt, float()); };
    return recipe_kind == GSA_NVFP4 ? sized(std::true_type()) : sized(std::false_type());
}

size_t gsa_grouped_glu_bwd_workspace_size(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0 || M >= (int64_t(1) << 31) || N >= (int64_t(1) << 30)) return 0;
    return kHead + (static_cast<size_t>((N + 127) / 128) * 2 * M * 4 + 255) / 256 * 256;
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
    auto typed = [&](auto fmt, auto type) {
        return pair ? launch_glu<decltype(fmt)::value, true, true, decltype(type)>(P, tiles, s)
                    : launch_glu<decltype(fmt)::value, false, true, decltype(type)>(P, tiles, s);
    };
    auto sized = [&](auto fmt) { return out_dtype == GSA_BF16 ? typed(fmt, __nv_bfloat16()) : typed(fmt, float()); };
    st = recipe_kind == GSA_NVFP4 ? sized(std::true_type()) : sized(std::false_type());
    if (st != GSA_OK || !dprobs_opt) return st;
    sum_partials<<<static_cast<unsigned>((M + 255) / 256), 256, 0, s>>>(P.part, P.bad, 2 * P.n_tiles, M, dprobs_opt);
    return cudaGetLastError() == cudaSuccess ? GSA_OK : GSA_ERR_CUDA;
}

}  // extern "C"
