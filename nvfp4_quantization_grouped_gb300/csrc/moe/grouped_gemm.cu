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
#include "gemm_core.cuh"

namespace {

// What went wrong in grouped products on this device and was not yet asked for, and what the query under way took.
__device__ uint32_t g_status, g_taken;

// The kernel of a query: reports only ever set bits and queries run one at a time, so a bit seen is the bit cleared.
__global__ void take_status() {
    g_taken = gemm_status::next_report(atomicOr(&g_status, 0u));
    atomicAnd(&g_status, ~g_taken);
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
        for (int i = 0; i < mine; ++i) multiply_tile<kPiece<T>>(sh, st, n, ring, P.k_bytes, ok);
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
    close_block<kPair>(sh, warp, C::kCols, &g_status);
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
            if (len > 0) multiply_tile<kPiece<T>>(sh, st, n, ring, len, ok);
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
    close_block<kPair>(sh, warp, C::kCols, &g_status);
}

// -------------------------------------------------------------------- host

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

}  // namespace

uint32_t *gemm_status::word() {
    static std::mutex mu;
    static struct {
        uint64_t context;   // whose address it is
        uint32_t *at;
    } known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    const uint64_t here = context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (here && known[dev].context == here) return known[dev].at;
    // a first call may be inside a capture, which this does not touch
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
    void *p = nullptr;
    const bool ok = cudaGetSymbolAddress(&p, g_status) == cudaSuccess;
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (!ok) return nullptr;
    known[dev] = {here, static_cast<uint32_t *>(p)};
    return known[dev].at;
}

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
