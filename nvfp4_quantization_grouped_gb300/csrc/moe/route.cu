// route.cu -- tokens into expert order and back, for sm_103a: the sort plan
// of the routed expert indices, the gather of the token rows (permute), the
// weighted way back (unpermute) and both gradients, with their C entry points.
//
// With slot s = (t, j) of token t, e(s) its expert and n = tokens * topk:
//   row(s)  = #{s' : e(s') < e(s)} + #{s' < s : e(s') = e(s)}    (a stable counting sort)
//   permute            xs[row(t, j)] = x[t],  ps[row(t, j)] = p[t, j]
//   its gradient       dx[t] = sum_j dxs[row(t, j)],  dp[t, j] = dps[row(t, j)]
//   unpermute          out[t] = sum_j w[t, j] ys[row(t, j)]
//   its gradient       dys[row(t, j)] = w[t, j] dout[t],  dw[t, j] = <dout[t], ys[row(t, j)]>
// A dropped slot (no expert in [0, E)) sorts behind every expert; the plan holds
// ~row for it, its rows are written as zeros and never read back.
//
// Everything after the plan moves each byte once and is bound by memory.  All
// four kernels go by token: a token's own row is read (or written) once whatever
// topk is, and only the expert side moves topk rows.  Sums run in FP32 in slot
// order, so results do not depend on the launch shape (dw: see unpermute_bwd).
//   32768 tokens x 8 x 2048 BF16, 128 experts: sort 10.5 us, permute 181 us (6.7 TB/s),
// unpermute 180 us (6.7 TB/s); gradient of unpermute on a quarter of it 94 us (6.1 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gsa.h"

namespace {

constexpr int kMaxBins = 257;        // 256 experts and the dropped slots
constexpr int kSortWarps = 32;
constexpr int kGradRows = 4, kGradBlocks = 4;   // unpermute_bwd: a token's slots at a time, blocks per SM
constexpr int kFewWarps = 16 * 152;   // unpermute_bwd: 16 warps an SM (a constant: sizes alone decide the order of sums)

// ------------------------------------------------------------------- sort

__device__ __forceinline__ int bin_of(const void *idx, int idx_bytes, int64_t s, int E) {
    const int64_t e = idx_bytes == 8 ? static_cast<const int64_t *>(idx)[s]
                                     : static_cast<int64_t>(static_cast<const int32_t *>(idx)[s]);
    return e >= 0 && e < E ? static_cast<int>(e) : E;
}

// Counts of segment blockIdx.x: counts[bin][blockIdx.x], rows of `pitch` entries.
__global__ void __launch_bounds__(1024) sort_count(const void *idx, int idx_bytes, int64_t n, int E, int64_t seg,
                                                   int pitch, int *counts) {
    __shared__ int bins[kMaxBins];
    for (int b = threadIdx.x; b <= E; b += blockDim.x) bins[b] = 0;
    __syncthreads();
    const int64_t s1 = min(n, (blockIdx.x + 1) * seg);
    for (int64_t s = blockIdx.x * seg + threadIdx.x; s < s1; s += blockDim.x) atomicAdd(&bins[bin_of(idx, idx_bytes, s, E)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= E; b += blockDim.x) counts[static_cast<int64_t>(b) * pitch + blockIdx.x] = bins[b];
}

// Rows of the slots of segment blockIdx.x.  counts: the segments' counts, or
// nullptr when one block holds every slot (at most one chunk) and counts itself.
// A warp takes 32 * kSteps consecutive slots of a chunk and ranks them among
// themselves, 32 at a time in slot order: lanes of the same expert find one another
// with match_any, so no atomics are needed and the order is the slots' own.
template <int kSteps>
__global__ void __launch_bounds__(1024) sort_rank(const void *idx, int idx_bytes, int64_t n, int E, int64_t seg, int pitch,
                                                  const int *counts, int32_t *row_of_slot, int64_t *split) {
    __shared__ int bins[kSortWarps][kMaxBins];   // a warp's slots of each expert, then the expert's next row for the warp
    __shared__ int next[kMaxBins];               // next row of each expert for this block
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5, nb = E + 1;
    const int64_t s1 = min(n, (blockIdx.x + 1) * seg), chunk = static_cast<int64_t>(nw) * 32 * kSteps;
    if (counts) {
        // rows of each expert in all segments (into bins[0]) and in those before this one
        for (int b = w; b < nb; b += nw) {
            int all = 0, first = 0;
            for (int k = lane; k < static_cast<int>(gridDim.x); k += 32) {
                const int c = counts[static_cast<int64_t>(b) * pitch + k];
                all += c;
                first += k < static_cast<int>(blockIdx.x) ? c : 0;
            }
            all = __reduce_add_sync(0xFFFFFFFFu, all);
            first = __reduce_add_sync(0xFFFFFFFFu, first);
            if (lane == 0) bins[0][b] = all, next[b] = first;
        }
        __syncthreads();
    }
    // expert b's first row, added to next[b]; the first block writes the split
    auto first_rows = [&](const int *total) {
        int carry = 0;
        for (int b = lane; b < (nb + 31) / 32 * 32; b += 32) {
            const int c = b < nb ? total[b] : 0;
            int inc = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                if (lane >= d) inc += v;
            }
            if (b < nb) {
                next[b] += carry + inc - c;
                if (blockIdx.x == 0) split[b] = c;
            }
            carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
    };
    if (counts) {
        if (w == 0) first_rows(bins[0]);
        __syncthreads();
    }
    for (int64_t c0 = blockIdx.x * seg; c0 == blockIdx.x * seg || c0 < s1; c0 += chunk) {
        for (int b = lane; b < nb; b += 32) bins[w][b] = 0;
        __syncwarp();
        int bin[kSteps], rank[kSteps];
        const int64_t w0 = c0 + static_cast<int64_t>(w) * 32 * kSteps + lane;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) bin[i] = w0 + 32 * i < s1 ? bin_of(idx, idx_bytes, w0 + 32 * i, E) : kMaxBins;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, bin[i]);
            const int before = __popc(same & ((1u << lane) - 1u)), base = bin[i] < kMaxBins ? bins[w][bin[i]] : 0;
            __syncwarp();
            if (bin[i] < kMaxBins && before == 0) bins[w][bin[i]] = base + __popc(same);
            __syncwarp();
            rank[i] = base + before;
        }
        __syncthreads();
        for (int b = threadIdx.x; b < nb; b += blockDim.x) {
            int row = counts ? next[b] : 0;
            for (int k = 0; k < nw; ++k) {
                const int c = bins[k][b];
                bins[k][b] = row;
                row += c;
            }
            next[b] = row;
        }
        __syncthreads();
        if (!counts) {   // the only chunk: its counts are the split
            __shared__ int total[kMaxBins];
            for (int b = threadIdx.x; b < nb; b += blockDim.x) total[b] = next[b], next[b] = 0;
            __syncthreads();
            if (w == 0) first_rows(total);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (bin[i] < kMaxBins) {
                const int32_t row = bins[w][bin[i]] + rank[i] + (counts ? 0 : next[bin[i]]);
                row_of_slot[w0 + 32 * i] = bin[i] == E ? ~row : row;
            }
        }
        __syncthreads();
    }
}

// One block up to kOneBlockSlots slots (a chunk of 32 warps x 4 steps), else segments
// of 2048 slots (32 warps x 2 steps) and two launches; at most 512 segments, since
// every block reads the counts of all.  One block / segments, 128 experts, us: 128 slots
// 3.0 / 7.5, 1024 4.2 / 8.4, 4096 7.8 / 9.5, 8192 11.7 / 10.1 (262144: 10.5).
constexpr int64_t kOneBlockSlots = 4096;

int64_t sort_segment(int64_t n) {
    if (n <= kOneBlockSlots) return n;
    return ((n + 511) / 512 + 2047) / 2048 * 2048;
}
int sort_pitch(int64_t n) { return static_cast<int>((n + sort_segment(n) - 1) / sort_segment(n) + 31) / 32 * 32; }

// ------------------------------------------------------- rows and vectors

template <int V> struct Raw;
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<2> { using T = uint16_t; };

// Rows are read once: past L1, whose lines nothing would hit.
template <int V> __device__ __forceinline__ typename Raw<V>::T load_once(const void *p) {
    return __ldcs(static_cast<const typename Raw<V>::T *>(p));
}

__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half &d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void put(float &d, float v) { d = v; }

template <typename T, int V> union Vec {
    typename Raw<V>::T raw;
    T e[V / sizeof(T)];
    __device__ Vec() {}
};

// Rows that start anywhere, by 16-byte words all the same: a kernel goes by the words
// of the row it writes, and reads the rows it reads at whatever offset that gives: two
// words, the second of which the next lane has just asked for, shifted together.  What
// lies before a row's first whole word and behind its last goes element by element.
// Worth it where stores of 2 (or 4) bytes are the alternative; 8192 tokens x 8 x 2047 / 2046
// / 2044 BF16 and 1111 FP32, by elements or pairs / by words, us: permute (with its sort)
// 141 / 84, 94 / 84, 76 / 82, 102 / 95; gradient of unpermute 223 / 145, 148 / 144, 121 / 140,
// 156 / 179; unpermute (one row written for 8 read) 95 / 95, 63 / 91, 47 / 80, 64 / 93.
struct Edges {
    int64_t words;      // whole words of the row
    int head, count;    // elements before the first word; elements before it and behind the last
    template <typename T> static __device__ __forceinline__ Edges of(const T *row, int64_t hidden) {
        Edges x;
        const int64_t head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T);
        x.head = static_cast<int>(head < hidden ? head : hidden);
        x.words = (hidden - x.head) * sizeof(T) / 16;
        x.count = static_cast<int>(hidden - x.words * (16 / sizeof(T)));
        return x;
    }
    // Column of the i-th edge element.
    template <typename T> __device__ __forceinline__ int64_t column(int i) const {
        return i < head ? i : words * static_cast<int64_t>(16 / sizeof(T)) + i;
    }
};

// 16 bytes at p, a multiple of sizeof(T) (both words inside [.., end) but for the bytes that are not asked for).
template <typename T> __device__ __forceinline__ uint4 load_any(const T *p, const T *end) {
    const uint32_t s = reinterpret_cast<uintptr_t>(p) & 15;
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - s);
    const uint4 a = __ldg(q);
    if (s == 0) return a;
    Vec<T, 16> b;
    b.raw = make_uint4(0, 0, 0, 0);
    if (reinterpret_cast<uintptr_t>(q + 2) <= reinterpret_cast<uintptr_t>(end)) {
        b.raw = __ldg(q + 1);
    } else {   // the tensor ends inside the second word
        const T *r = reinterpret_cast<const T *>(q + 1);
#pragma unroll
        for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i)
            if (i < static_cast<int>(s / sizeof(T))) b.e[i] = r[i];
    }
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.raw.x, b.raw.y, b.raw.z, b.raw.w};
    if (s & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (s & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = 8 * (s & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

// Row index of a plan entry, -1 where the slot is dropped (or out of range).
__device__ __forceinline__ int live_row(int32_t r, int n) {
    return static_cast<uint32_t>(r) < static_cast<uint32_t>(n) ? r : -1;
}

// The blocks are (columns, tokens): threadIdx.x walks a row's vectors, blockDim.y tokens per block.

template <int V>
__global__ void __launch_bounds__(256) permute_fwd(const uint8_t *x, const float *probs, const int32_t *row_of_slot,
                                                   int tokens, int topk, int64_t nv, uint8_t *xs, float *ps) {
    using R = typename Raw<V>::T;
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    const int n = tokens * topk;
    const int32_t *rows = row_of_slot + static_cast<int64_t>(t) * topk;
    if (ps && blockIdx.y == 0) {
        for (int j = threadIdx.x; j < topk; j += blockDim.x) {
            const int32_t r = rows[j];
            const int at = r < 0 ? ~r : r;
            if (at < n) ps[at] = r < 0 ? 0.0f : probs[static_cast<int64_t>(t) * topk + j];
        }
    }
    for (int64_t c = blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x; c < nv;
         c += static_cast<int64_t>(gridDim.y) * blockDim.x) {
        const R v = load_once<V>(x + (t * nv + c) * V);
        const R zero{};
        for (int j = 0; j < topk; ++j) {
            const int32_t r = rows[j];
            const int at = r < 0 ? ~r : r;
            if (at < n) *reinterpret_cast<R *>(xs + (at * nv + c) * V) = r < 0 ? zero : v;
        }
    }
}

// out[t] = sum_j w_j rows[row(t, j)] (w = 1 without weights): unpermute, and the
// gradient of permute (which also brings the probabilities' gradients back).  A
// thread loads kU columns of G rows before it uses the first: enough bytes in
// flight for memory, whatever topk.
template <typename T, int V, int G, int kU>
__global__ void __launch_bounds__(256, 4) combine(const uint8_t *ys, const float *weights, const int32_t *row_of_slot,
                                               int tokens, int topk, int64_t nv, uint8_t *out, const float *dps,
                                               float *dprobs) {
    constexpr int N = V / sizeof(T);
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    const int n = tokens * topk;
    const int32_t *rows = row_of_slot + static_cast<int64_t>(t) * topk;
    if (dprobs && blockIdx.y == 0) {
        for (int j = threadIdx.x; j < topk; j += blockDim.x) {
            const int r = live_row(rows[j], n);
            dprobs[static_cast<int64_t>(t) * topk + j] = r < 0 ? 0.0f : dps[r];
        }
    }
    const int64_t step = blockDim.x;
    for (int64_t c = blockIdx.y * step * kU + threadIdx.x; c < nv; c += gridDim.y * step * kU) {
        float acc[kU][N];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[u][i] = 0.0f;
        for (int j0 = 0; j0 < topk; j0 += G) {
            Vec<T, V> v[G][kU];
            uint32_t live = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int r = j0 + g < topk ? live_row(rows[j0 + g], n) : -1;
                if (r < 0) continue;
                live |= 1u << g;
                const uint8_t *p = ys + (r * nv + c) * V;
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (u == 0 || c + u * step < nv) v[g][u].raw = load_once<V>(p + u * step * V);
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (live >> g & 1) {
                    const float w = weights ? weights[static_cast<int64_t>(t) * topk + j0 + g] : 1.0f;
#pragma unroll
                    for (int u = 0; u < kU; ++u)
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[u][i] = __fmaf_rn(w, as_f32(v[g][u].e[i]), acc[u][i]);
                }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            Vec<T, V> o;
#pragma unroll
            for (int i = 0; i < N; ++i) put(o.e[i], acc[u][i]);
            if (c + u * step < nv) *reinterpret_cast<typename Raw<V>::T *>(out + (t * nv + c + u * step) * V) = o.raw;
        }
    }
}

// G partial dot products of a token's warps summed and written: over the lanes by halving distances, over the warps in
// order.  Every thread of the block; left: slots that the token still has.
template <int G>
__device__ __forceinline__ void finish_dots(float (&part)[8][G], float (&acc)[G], bool on, int wpt, int warp, int lane, int left,
                                            float *dw) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) acc[g] += __shfl_xor_sync(0xFFFFFFFFu, acc[g], s);
    }
    if (wpt > 1) {
        __syncthreads();
        if (lane == 0) {
#pragma unroll
            for (int g = 0; g < G; ++g) part[warp][g] = acc[g];
        }
        __syncthreads();
    }
    const int mine = threadIdx.x;
    if (on && mine < G && mine < left) {
        float s = 0.0f;
        if (wpt > 1) {
            for (int k = 0; k < wpt; ++k) s += part[threadIdx.y * wpt + k][mine];
        } else {
#pragma unroll
            for (int k = 0; k < G; ++k)
                if (k == mine) s = acc[k];
        }
        dw[mine] = s;
    }
}

// dys[row] = w dout[t] and dw = <dout[t], ys[row]> in one pass.  blockDim.y
// groups of wpt warps take a token each and kGradRows of its slots at a time; a
// thread keeps their partial dot products, summed over its columns in order, then
// over the lanes by halving distances and over the token's warps in order: the
// sum's order depends on wpt alone, which the launch takes from tokens and width.
// Slots at a time / blocks per SM at 1, 2, 4 and 8 warps a token, 8192 tokens x 8 x
// 2048 BF16, us: 8 / 2: 100.9, 96.6, 102.4, 119.2; 8 / 3 (spills): 115.1, 113.3, 113.6,
// 125.3; 4 / 4: 98.8, 96.2, 93.8, 100.6; 4 / 5: 113.3, 100.9, 98.4, 102.9; 2 / 6: 127.4,
// 102.3, 96.8, 103.4.  93.8 us is 6.1 TB/s of the bytes it has to move.
template <typename T, int V>
__global__ void __launch_bounds__(256, kGradBlocks) unpermute_bwd(const uint8_t *dout, const uint8_t *ys,
                                                                  const float *weights, const int32_t *row_of_slot,
                                                                  int tokens, int topk, int64_t nv, uint8_t *dys,
                                                                  float *dw) {
    constexpr int N = V / sizeof(T), G = kGradRows;
    __shared__ float part[8][G];
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    const int n = tokens * topk;
    const int lane = threadIdx.x & 31, wpt = blockDim.x >> 5, warp = threadIdx.y * wpt + (threadIdx.x >> 5);
    const bool on = t < tokens;
    const int64_t slot0 = static_cast<int64_t>(on ? t : 0) * topk;
    for (int j0 = 0; j0 < topk; j0 += G) {
        int32_t r[G];
        float acc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            r[g] = on && j0 + g < topk ? row_of_slot[slot0 + j0 + g] : n;   // n: nothing to do
            acc[g] = 0.0f;
        }
        if (on) {
            for (int64_t c = threadIdx.x; c < nv; c += blockDim.x) {
                Vec<T, V> d, y[G];
                d.raw = *reinterpret_cast<const typename Raw<V>::T *>(dout + (t * nv + c) * V);
                if (dw) {
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        if (live_row(r[g], n) >= 0) y[g].raw = load_once<V>(ys + (r[g] * nv + c) * V);
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const bool live = live_row(r[g], n) >= 0;
                    const int at = r[g] < 0 ? ~r[g] : r[g];
                    if (dw && live) {
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[g] = __fmaf_rn(as_f32(d.e[i]), as_f32(y[g].e[i]), acc[g]);
                    }
                    if (dys && at < n) {
                        const float w = weights ? weights[slot0 + j0 + g] : 1.0f;
                        Vec<T, V> o;
#pragma unroll
                        for (int i = 0; i < N; ++i) put(o.e[i], live ? w * as_f32(d.e[i]) : 0.0f);
                        *reinterpret_cast<typename Raw<V>::T *>(dys + (at * nv + c) * V) = o.raw;
                    }
                }
            }
        }
        if (dw) finish_dots<G>(part, acc, on, wpt, warp, lane, topk - j0, dw + slot0 + j0);
    }
}

// ------------------------------------------------ rows that start anywhere

template <typename T>
__global__ void __launch_bounds__(256) any_permute_fwd(const T *x, const float *probs, const int32_t *row_of_slot, int tokens,
                                                       int topk, int64_t hidden, T *xs, float *ps) {
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    const int n = tokens * topk;
    const int32_t *rows = row_of_slot + static_cast<int64_t>(t) * topk;
    if (ps && blockIdx.y == 0) {
        for (int j = threadIdx.x; j < topk; j += blockDim.x) {
            const int32_t r = rows[j];
            const int at = r < 0 ? ~r : r;
            if (at < n) ps[at] = r < 0 ? 0.0f : probs[static_cast<int64_t>(t) * topk + j];
        }
    }
    const T *src = x + t * hidden, *end = x + tokens * hidden;
#pragma unroll 2
    for (int j = 0; j < topk; ++j) {
        const int32_t r = rows[j];
        const int at = r < 0 ? ~r : r;
        if (at >= n) continue;
        T *dst = xs + at * hidden;
        const Edges e = Edges::of(dst, hidden);
        for (int64_t c = blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x; c < e.words;
             c += static_cast<int64_t>(gridDim.y) * blockDim.x) {
            const int64_t col = e.head + c * static_cast<int64_t>(16 / sizeof(T));
            *reinterpret_cast<uint4 *>(dst + col) = r < 0 ? make_uint4(0, 0, 0, 0) : load_any(src + col, end);
        }
        if (blockIdx.y == 0)
            for (int i = threadIdx.x; i < e.count; i += blockDim.x) {
                const int64_t col = e.column<T>(i);
                T v;
                put(v, 0.0f);
                dst[col] = r < 0 ? v : src[col];
            }
    }
}

// dys and ys rows lie alike, dout at an offset; a slot at a time.  (The order of a dot product's terms goes by the
// words of its row.)
template <typename T>
__global__ void __launch_bounds__(256) any_unpermute_bwd(const T *dout, const T *ys, const float *weights,
                                                         const int32_t *row_of_slot, int tokens, int topk, int64_t hidden,
                                                         T *dys, float *dw) {
    constexpr int N = 16 / sizeof(T), G = 2;
    __shared__ float part[8][G];
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    const int n = tokens * topk;
    const int lane = threadIdx.x & 31, wpt = blockDim.x >> 5, warp = threadIdx.y * wpt + (threadIdx.x >> 5);
    const bool on = t < tokens;
    const int64_t slot0 = static_cast<int64_t>(on ? t : 0) * topk;
    const T *src = dout + (on ? t : 0) * hidden, *end = dout + tokens * hidden;
    for (int j0 = 0; j0 < topk; j0 += G) {
        float acc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            acc[g] = 0.0f;
            const int32_t r = on && j0 + g < topk ? row_of_slot[slot0 + j0 + g] : n;
            const int at = r < 0 ? ~r : r;
            const bool live = live_row(r, n) >= 0;
            if (at >= n || (!live && !dys)) continue;
            const float w = live && weights ? weights[slot0 + j0 + g] : 1.0f;
            const Edges e = Edges::of((dys ? dys : ys) + at * hidden, hidden);   // both tensors start on 16 bytes
            for (int64_t c = threadIdx.x; c < e.words; c += blockDim.x) {
                const int64_t col = e.head + c * N;
                Vec<T, 16> d, y, o;
                if (dw && live) y.raw = load_once<16>(ys + at * hidden + col);
                if (live) d.raw = load_any(src + col, end);
                if (dw && live) {
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[g] = __fmaf_rn(as_f32(d.e[i]), as_f32(y.e[i]), acc[g]);
                }
                if (dys) {
#pragma unroll
                    for (int i = 0; i < N; ++i) put(o.e[i], live ? w * as_f32(d.e[i]) : 0.0f);
                    *reinterpret_cast<uint4 *>(dys + at * hidden + col) = o.raw;
                }
            }
            for (int i = threadIdx.x; i < e.count; i += blockDim.x) {
                const int64_t col = e.column<T>(i);
                const float d = live ? as_f32(src[col]) : 0.0f;
                if (dw && live) acc[g] = __fmaf_rn(d, as_f32(ys[at * hidden + col]), acc[g]);
                if (dys) put(dys[at * hidden + col], live ? w * d : 0.0f);
            }
        }
        if (dw) finish_dots<G>(part, acc, on, wpt, warp, lane, topk - j0, dw + slot0 + j0);
    }
}

// ----------------------------------------------------------------- launch

int elem_bytes(int dtype) { return dtype == GSA_FP32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Widest access that every row start allows (the tensors start on 16 bytes).
int vector_bytes(int64_t row_bytes) {
    for (int v = 16; v > 2; v /= 2)
        if (row_bytes % v == 0) return v;
    return 2;
}

struct Shape {
    dim3 grid, block;
};

// Columns x tokens of a block of at most 256 threads, `unroll` columns a thread;
// columns beyond one pass of a block go to further blocks along grid.y, all as wide as
// they need to be (1111 columns, unroll 4: 2 x 160 threads, not 256 and 22).
Shape row_shape(int64_t tokens, int64_t nv, int unroll = 1) {
    const int64_t per = (nv + unroll - 1) / unroll;   // threads that the columns take
    int64_t gy = (per + 255) / 256;
    int64_t x = 1;
    if (per < 32) while (x < per) x *= 2;
    else x = ((per + gy - 1) / gy + 31) / 32 * 32;
    const int y = static_cast<int>(256 / x);
    if (gy > 64) gy = 64;
    return {dim3(static_cast<unsigned>((tokens + y - 1) / y), static_cast<unsigned>(gy)), dim3(static_cast<unsigned>(x), y)};
}

gsa_status check_shape(int64_t tokens, int64_t topk, int64_t hidden, int32_t dtype) {
    if (tokens < 0 || topk <= 0 || hidden <= 0) return GSA_ERR_INVALID_ARG;
    if (dtype != GSA_BF16 && dtype != GSA_FP16 && dtype != GSA_FP32) return GSA_ERR_INVALID_ARG;
    if (topk >= (int64_t(1) << 31) || tokens >= (int64_t(1) << 31) || tokens * topk >= (int64_t(1) << 31) ||
        hidden >= (int64_t(1) << 31))
        return GSA_ERR_UNSUPPORTED;
    return GSA_OK;
}

gsa_status done() { return cudaGetLastError() == cudaSuccess ? GSA_OK : GSA_ERR_CUDA; }

// Calls f<T, V>() for the element type and access width.
template <typename T, typename F> void with_vector(int v, F &&f) {
    switch (v) {
    case 16: f(T(), std::integral_constant<int, 16>()); break;
    case 8: f(T(), std::integral_constant<int, 8>()); break;
    case 4: f(T(), std::integral_constant<int, 4>()); break;
    default:
        if constexpr (sizeof(T) == 2) f(T(), std::integral_constant<int, 2>());
    }
}

template <typename F> void with_type(int dtype, F &&f) {
    if (dtype == GSA_BF16) f(__nv_bfloat16());
    else if (dtype == GSA_FP16) f(__half());
    else f(float());
}
template <typename F> void with_type(int dtype, int v, F &&f) {
    with_type(dtype, [&](auto tag) { with_vector<decltype(tag)>(v, f); });
}

gsa_status run_combine(const void *ys, const float *weights, const int32_t *row_of_slot, int64_t tokens, int64_t topk,
                       int64_t hidden, int32_t dtype, void *out, const float *dps, float *dprobs,
                       gsa_stream_t stream) {
    const int v = vector_bytes(hidden * elem_bytes(dtype));
    const int64_t nv = hidden * elem_bytes(dtype) / v;
    with_type(dtype, v, [&](auto tag, auto width) {
        auto go = [&](auto group, auto unroll) {
            const Shape s = row_shape(tokens, nv, decltype(unroll)::value);
            combine<decltype(tag), decltype(width)::value, decltype(group)::value, decltype(unroll)::value>
                <<<s.grid, s.block, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
                    static_cast<const uint8_t *>(ys), weights, row_of_slot, static_cast<int>(tokens),
                    static_cast<int>(topk), nv, static_cast<uint8_t *>(out), dps, dprobs);
        };
        if (topk > 4) go(std::integral_constant<int, 8>(), std::integral_constant<int, decltype(width)::value == 16 ? 1 : 2>());
        else go(std::integral_constant<int, 4>(), std::integral_constant<int, decltype(width)::value == 16 ? 2 : 4>());
    });
    return done();
}

}  // namespace

extern "C" {

size_t gsa_moe_sort_workspace_size(int64_t tokens, int64_t topk, int64_t experts) {
    if (tokens < 0 || topk <= 0 || experts <= 0 || experts >= kMaxBins || tokens >= (int64_t(1) << 31) ||
        topk >= (int64_t(1) << 31) || tokens * topk >= (int64_t(1) << 31))
        return 0;
    const int64_t n = tokens * topk;
    return n <= kOneBlockSlots ? 0 : static_cast<size_t>(sort_pitch(n)) * (experts + 1) * 4;
}

gsa_status gsa_moe_sort(const void *expert_idx, int32_t idx_bytes, int64_t tokens, int64_t topk, int64_t experts,
                        int32_t *row_of_slot, int64_t *split_sizes, void *workspace, size_t workspace_bytes,
                        gsa_stream_t stream) {
    if (tokens < 0 || topk <= 0 || experts <= 0 || (idx_bytes != 4 && idx_bytes != 8)) return GSA_ERR_INVALID_ARG;
    if (experts >= kMaxBins || tokens >= (int64_t(1) << 31) || topk >= (int64_t(1) << 31) ||
        tokens * topk >= (int64_t(1) << 31))
        return GSA_ERR_UNSUPPORTED;
    const int64_t n = tokens * topk;
    if (!split_sizes || (n > 0 && (!expert_idx || !row_of_slot))) return GSA_ERR_INVALID_ARG;
    if (!aligned(expert_idx, idx_bytes) || !aligned(row_of_slot, 16) || !aligned(split_sizes, 8) || !aligned(workspace, 16))
        return GSA_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int E = static_cast<int>(experts);
    const int64_t seg = sort_segment(n);
    if (n <= kOneBlockSlots) {
        int threads = 128;   // also what the bins take
        while (threads < 1024 && threads < n) threads *= 2;
        if (n <= threads) sort_rank<1><<<1, threads, 0, s>>>(expert_idx, idx_bytes, n, E, seg, 0, nullptr, row_of_slot, split_sizes);
        else sort_rank<4><<<1, threads, 0, s>>>(expert_idx, idx_bytes, n, E, seg, 0, nullptr, row_of_slot, split_sizes);
        return done();
    }
    if (!workspace || workspace_bytes < gsa_moe_sort_workspace_size(tokens, topk, experts)) return GSA_ERR_WORKSPACE;
    const unsigned blocks = static_cast<unsigned>((n + seg - 1) / seg);
    int *counts = static_cast<int *>(workspace);
    sort_count<<<blocks, 1024, 0, s>>>(expert_idx, idx_bytes, n, E, seg, sort_pitch(n), counts);
    sort_rank<2><<<blocks, 1024, 0, s>>>(expert_idx, idx_bytes, n, E, seg, sort_pitch(n), counts, row_of_slot, split_sizes);
    return done();
}

gsa_status gsa_moe_permute(const void *x, const float *probs, const int32_t *row_of_slot, int64_t tokens, int64_t topk,
                           int64_t hidden, int32_t dtype, void *xs, float *ps, gsa_stream_t stream) {
    gsa_status st = check_shape(tokens, topk, hidden, dtype);
    if (st != GSA_OK) return st;
    if ((probs == nullptr) != (ps == nullptr) && tokens > 0) return GSA_ERR_INVALID_ARG;
    if (tokens > 0 && (!x || !xs || !row_of_slot)) return GSA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(row_of_slot, 4) || !aligned(probs, 4) || !aligned(ps, 4))
        return GSA_ERR_ALIGNMENT;
    if (tokens == 0) return GSA_OK;
    const int v = vector_bytes(hidden * elem_bytes(dtype));
    const int64_t bytes = hidden * elem_bytes(dtype), nv = v >= 8 ? bytes / v : (bytes + 15) / 16;
    const Shape g = row_shape(tokens, nv);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int nt = static_cast<int>(tokens), nk = static_cast<int>(topk);
    const uint8_t *from = static_cast<const uint8_t *>(x);
    uint8_t *to = static_cast<uint8_t *>(xs);
    if (v == 16) permute_fwd<16><<<g.grid, g.block, 0, s>>>(from, probs, row_of_slot, nt, nk, nv, to, ps);
    else if (v == 8) permute_fwd<8><<<g.grid, g.block, 0, s>>>(from, probs, row_of_slot, nt, nk, nv, to, ps);
    else
        with_type(dtype, [&](auto tag) {
            using T = decltype(tag);
            any_permute_fwd<T><<<g.grid, g.block, 0, s>>>(static_cast<const T *>(x), probs, row_of_slot, nt, nk, hidden,
                                                          static_cast<T *>(xs), ps);
        });
    return done();
}

gsa_status gsa_moe_permute_bwd(const void *dxs, const float *dps, const int32_t *row_of_slot, int64_t tokens,
                               int64_t topk, int64_t hidden, int32_t dtype, void *dx, float *dprobs,
                               gsa_stream_t stream) {
    gsa_status st = check_shape(tokens, topk, hidden, dtype);
    if (st != GSA_OK) return st;
    if ((dps == nullptr) != (dprobs == nullptr) && tokens > 0) return GSA_ERR_INVALID_ARG;
    if (tokens > 0 && (!dxs || !dx || !row_of_slot)) return GSA_ERR_INVALID_ARG;
    if (!aligned(dxs, 16) || !aligned(dx, 16) || !aligned(row_of_slot, 4) || !aligned(dps, 4) || !aligned(dprobs, 4))
        return GSA_ERR_ALIGNMENT;
    if (tokens == 0) return GSA_OK;
    return run_combine(dxs, nullptr, row_of_slot, tokens, topk, hidden, dtype, dx, dps, dprobs, stream);
}

gsa_status gsa_moe_unpermute(const void *ys, const float *weights, const int32_t *row_of_slot, int64_t tokens,
                             int64_t topk, int64_t hidden, int32_t dtype, void *out, gsa_stream_t stream) {
    gsa_status st = check_shape(tokens, topk, hidden, dtype);
    if (st != GSA_OK) return st;
    if (tokens > 0 && (!ys || !out || !row_of_slot)) return GSA_ERR_INVALID_ARG;
    if (!aligned(ys, 16) || !aligned(out, 16) || !aligned(row_of_slot, 4) || !aligned(weights, 4))
        return GSA_ERR_ALIGNMENT;
    if (tokens == 0) return GSA_OK;
    return run_combine(ys, weights, row_of_slot, tokens, topk, hidden, dtype, out, nullptr, nullptr, stream);
}

gsa_status gsa_moe_unpermute_bwd(const void *dout, const void *ys, const float *weights, const int32_t *row_of_slot,
                                 int64_t tokens, int64_t topk, int64_t hidden, int32_t dtype, void *dys,
                                 float *dweights, gsa_stream_t stream) {
    gsa_status st = check_shape(tokens, topk, hidden, dtype);
    if (st != GSA_OK) return st;
    if (tokens > 0 && (!dout || !row_of_slot || (!dys && !dweights) || (dweights && !ys))) return GSA_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(row_of_slot, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return GSA_ERR_ALIGNMENT;
    if (tokens == 0) return GSA_OK;
    const int v = vector_bytes(hidden * elem_bytes(dtype));
    const int64_t bytes = hidden * elem_bytes(dtype), nv = v == 2 ? (bytes + 15) / 16 : bytes / v;   // v 2: by words
    // warps per token: two vectors a thread and at most 4 (measured above), or one and
    // at most 8 where the tokens are too few to fill the machine with 4
    int wpt = 1;
    while (wpt < 4 && wpt * 128 <= nv) wpt *= 2;
    while (wpt < 8 && tokens * wpt < kFewWarps && wpt * 64 <= nv) wpt *= 2;
    const dim3 block(32 * wpt, 8 / wpt), grid(static_cast<unsigned>((tokens + block.y - 1) / block.y));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int nt = static_cast<int>(tokens), nk = static_cast<int>(topk);
    if (v == 2)
        with_type(dtype, [&](auto tag) {
            using T = decltype(tag);
            any_unpermute_bwd<T><<<grid, block, 0, s>>>(static_cast<const T *>(dout), static_cast<const T *>(ys), weights,
                                                        row_of_slot, nt, nk, hidden, static_cast<T *>(dys), dweights);
        });
    else
        with_type(dtype, v, [&](auto tag, auto width) {
            if constexpr (decltype(width)::value > 2)
                unpermute_bwd<decltype(tag), decltype(width)::value><<<grid, block, 0, s>>>(
                    static_cast<const uint8_t *>(dout), static_cast<const uint8_t *>(ys), weights, row_of_slot, nt, nk, nv,
                    static_cast<uint8_t *>(dys), dweights);
        });
    return done();
}

}  // extern "C"
