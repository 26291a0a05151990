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

// What a draining warp knows of its tile.
struct Here {
    int64_t row, cols;   // the lane's row of the tensors; columns left from the warp's first on
    float p;
    float ug, vg, uu, vu;   // NVFP4: what a gate sum (ug, then vg) and a linear sum are multiplied by
    int nt, rows;           // column tile; the warp's rows
};

template <bool NV, bool kPair, bool kBwd, typename T>
__global__ void __launch_bounds__(kThreads, 1) grouped_glu(const __grid_constant__ GluParams P) {
    using C = Cfg<NV, kBN, kPair>;
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
    const int64_t total = sh.bad ? 0 : static_cast<int64_t>(sh.tile0[P.E + 1]) * P.n_tiles;
    const int64_t used = sh.bad ? 0 : static_cast<int64_t>(sh.tile0[P.E]) * P.n_tiles;   // the rest is zeros

    if (warp == 0) {
        if (tc::elect()) {
            tc::prefetch_map(&P.tm_a);
            tc::prefetch_map(&P.tm_b);
        }
        Ring<C::kStages> ring;
        int g = 0;
        bool ok = true, first = false;
        auto at = [&](int64_t i) {
            const Tile t = tile_at<kRows>(P, sh, i, g);
            g = t.g;
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
        for (int i = 0; i < mine; ++i) multiply_tile<kLen>(sh, st, n, ring, P.k_bytes, ok);
        if (!ok || *static_cast<volatile uint32_t *>(&sh.dead)) settle<C::kStages>(sh.empty, ring.issued);
    } else if (warp >= kDrain) {
        const int q = warp & 3, h = (warp - kDrain) >> 2;   // lanes 32 q .., 64 columns of both sides from 64 h
        const int64_t pitch = kBwd ? 2 * P.N : P.N;
        T *out = static_cast<T *>(P.out);
        const int r0 = half * kRowsT + 32 * q;
        const uint32_t buf = st.out(warp - kDrain);
        OutAt<const __nv_bfloat16> d;
        d.pitch = P.N;
        d.wide = P.N % 8 == 0;
        OutAt<T> w;
        w.pitch = pitch;
        w.wide = P.N * sizeof(T) % 16 == 0;
        w.add = false;
        Here c;
        int g = 0, n = 0, last = -1;
        auto find = [&](int64_t i) {
            if (i >= total) return;
            const Tile t = tile_at<kRows>(P, sh, i, g);
            g = t.g;
            const int64_t c0 = static_cast<int64_t>(t.nt) * kSide + h * kCols64, row = t.row + r0;
            c.nt = t.nt;
            c.row = row + lane;
            c.cols = P.N - c0;
            c.rows = t.rows - r0;
            w.o = out + row * pitch + c0;
            w.cols = c.cols;
            w.rows = c.rows;
            if (kBwd) d.o = P.dy + row * P.N + c0, d.cols = c.cols, d.rows = c.rows;
            c.p = P.probs && lane < c.rows && g < P.E ? P.probs[c.row] : 1.0f;
            if (NV && g < P.E && g != last) {
                const float a = P.amax_a[g];
                units_of(a, P.amax_b[g * P.b_groups], c.ug, c.vg);
                c.uu = c.ug, c.vu = c.vg;
                if (P.b_groups == 2) units_of(a, P.amax_b[2 * g + 1], c.uu, c.vu);
                last = g;
            }
        };
        auto partial = [&](const Here &at, float dp) {
            if (kBwd && P.part && lane < at.rows) P.part[(2 * static_cast<int64_t>(at.nt) + h) * P.M + at.row] = dp;
        };
        auto store = [&](const uint32_t *v, const OutAt<T> &at) {
            if (at.wide) store_warp<kCols64, false, T>(v, 1.0f, 1.0f, buf, at, lane);
            else store_warp_any<kCols64, false, T>(v, 1.0f, 1.0f, buf, at, lane);
        };
        find(unit);
        if (kBwd && unit < used) load_dy(buf, d, P.dy, lane);
        for (int64_t i = unit; i < total; i += units) {
            if (g == P.E) {
                if (P.out) {
                    zero_tile<kCols64>(w, lane);
                    if (kBwd) {
                        OutAt<T> up = w;
                        up.o += P.N;
                        zero_tile<kCols64>(up, lane);
                    }
                }
                partial(c, 0.0f);
                find(i + units);
                continue;
            }
            uint32_t v[kSide];   // 64 columns of g, and of u
            if (!take_tile<kBN, C::kAcc, kPair, kLen, 2>(sh, n, P.kt, q, lane, h * kCols64, kSide + h * kCols64, v)) break;
            const Here at = c;
            OutAt<T> here = w;
            if (kBwd) {
                wait_dy();
                if (at.cols < kCols64) {   // past the last column: whatever the next rows and the scales' padding give, NaN too
                    const int left = static_cast<int>(at.cols);
#pragma unroll
                    for (int j = 0; j < kCols64; ++j)
                        if (j >= left) v[j] = v[kCols64 + j] = 0;
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
                            uint32_t *vg = v + j + k, *vu = v + kCols64 + j + k;
                            float2 dg, du;
                            const float2 y = glu::gradient<decltype(clamp)::value>(P.act, pair_of<NV>(vg, at.ug, at.vg), pair_of<NV>(vu, at.uu, at.vu),
                                                                                   glu::mul2(dy, at.p), dg, du);
                            dp = glu::fma2(dy, y, dp);
                            vg[0] = __float_as_uint(dg.x), vg[1] = __float_as_uint(dg.y);
                            vu[0] = __float_as_uint(du.x), vu[1] = __float_as_uint(du.y);
                        }
                    }
                };
                if (P.act.clamped) all(std::true_type());
                else all(std::false_type());
                __syncwarp();
                partial(at, dp.x + dp.y);
                find(i + units);
                if (P.out) {
                    store(v, here);
                    here.o += P.N;
                    store(v + kCols64, here);
                }
                if (i + units < used) load_dy(buf, d, P.dy, lane);
            } else {
                auto all = [&](auto clamp) {
#pragma unroll
                    for (int j = 0; j < kCols64; j += 2) {
                        const float2 y = glu::mul2(glu::value<decltype(clamp)::value>(P.act, pair_of<NV>(v + j, at.ug, at.vg),
                                                                                      pair_of<NV>(v + kCols64 + j, at.uu, at.vu)), at.p);
                        v[j] = __float_as_uint(y.x), v[j + 1] = __float_as_uint(y.y);
                    }
                };
                if (P.act.clamped) all(std::true_type());
                else all(std::false_type());
                find(i + units);
                store(v, here);
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
    return launch<kPair, GluParams>(grouped_glu<NV, kPair, kBwd, T>, P, kThreads, Cfg<NV, kBN, kPair>::kSmem, tiles * P.n_tiles, s, pairs);
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
