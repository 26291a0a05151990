// tc.cuh -- mbarriers, TMA and 5th-generation tensor-core (tcgen05) primitives
// of the grouped products, as inline PTX for sm_103a.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------- mbarrier

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 1000000;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

constexpr uint64_t kLimitNs = 2000000000ull;

// Bounded wait: false after about 2 s, or at once when `dead` (a word in shared
// memory) says that another wait of the block has run out.
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t *dead) {
    const uint64_t t0 = now_ns();
    for (;;) {
        if (bar_try(bar, parity)) return true;
        if (*dead) return false;
        if (now_ns() - t0 > kLimitNs) {
            *dead = 1;
            return false;
        }
    }
}

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t *dead) {
    if (bar_try(bar, parity)) return true;
    return bar_wait_slow(bar, parity, dead);
}

__device__ __forceinline__ void pause(uint64_t ns) {
    const uint64_t t0 = now_ns();
    while (now_ns() - t0 < ns) __nanosleep(1000);
}

// The same for a whole warp in uniform control flow: the result is uniform too.
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t *dead) {
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, dead));
}

// One lane of a converged warp.  The warps that issue copies and products run their
// loops as a whole and elect the lane only around the instructions, so that
// addresses and descriptors stay in uniform registers, which these instructions
// take: issued from a branch of one lane, every operand is moved there first
// (measured: 50 to 75 cycles for each copy to tensor memory).
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void st_shared(uint32_t at, const uint32_t *w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared1(uint32_t at) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(at) : "memory");
    return f;
}

// --------------------------------------------------------------------- TMA

__device__ __forceinline__ void prefetch_map(const CUtensorMap *tm) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}

__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(tm), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Brings what load_2d would copy into L2.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *tm, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tm), "r"(x), "r"(y) : "memory");
}

// Into this block's shared memory; the bytes count on a barrier of the pair's first block.
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y), "r"(cluster_bar)
        : "memory");
}

// Origin, extents (bytes of a row, rows) and pitch of a tensor map of bytes in shared memory.
__device__ __forceinline__ void edit_map(CUtensorMap *map, const void *p, uint32_t bytes, uint32_t rows, uint64_t pitch) {
    const uint32_t m = smem_u32(map);
    asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(m), "l"(p) : "memory");
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 0, %1;" ::"r"(m), "r"(bytes) : "memory");
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(m), "r"(rows) : "memory");
    asm volatile("tensormap.replace.tile.global_stride.shared::cta.b1024.b64 [%0], 0, %1;" ::"r"(m), "l"(pitch) : "memory");
}

// Whole warp: a finished map from shared to global memory, released to the proxy through which copies read maps (which
// plain stores and the end of a kernel do not order).
__device__ __forceinline__ void publish_map(CUtensorMap *to, const CUtensorMap *map) {
    asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(to),
                 "r"(smem_u32(map))
                 : "memory");
}

// Before the first copy through a map that another kernel wrote to global memory.
__device__ __forceinline__ void acquire_map(const CUtensorMap *map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}

// -------------------------------------------------------- dependent launch

// A kernel launched as a programmatic dependent may start while the kernel before it in the stream ends: this waits until
// that one is done and its results are visible (at once where the launch was an ordinary one).  The other lets the next
// such kernel start.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ----------------------------------------------------------------- cluster

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of another block's copy of a shared-memory location.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// On a barrier of any block of the cluster.  Relaxed: it says that this warp has what it read from tensor memory (the
// loads are complete, nothing is passed on in memory); with the tcgen05 fences on both sides this is the order that the
// ISA gives tcgen05 operations of different threads.  A release at cluster scope would first wait for the warp's stores of the
// tile before, 1.9K cycles in which the tensor core stands still.
__device__ __forceinline__ void bar_arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// ----------------------------------------------------------------- tcgen05

// kPair: the operation of a CTA pair (cta_group::2), issued by the pair's first block (allocation: by both).

// Whole warp: `cols` columns of tensor memory, their address into *slot.
template <bool kPair> __device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <bool kPair> __device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The barrier (a pair: that of both blocks) is arrived on once every tcgen05 operation this thread has issued is done.
template <bool kPair> __device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (kPair)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory matrix descriptors: the low word is the address in units of 16 bytes, which is all that changes
// from step to step; the rest is constant.
constexpr uint32_t kDescLo = 1u << 16;                             // (leading offset: unused)
constexpr uint32_t kDescSw128 = 64u | (1u << 14) | (2u << 29);     // rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart
constexpr uint32_t kDescScales = 8u | (1u << 14);                  // 32 rows of 16 bytes, 8-row groups 128 bytes apart: a 512-byte scale tile
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | kDescLo; }

// One scale tile (128 rows x 4 scales) into 4 columns of tensor memory, repeated for the four lane quarters.
template <bool kPair> __device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t lo) {
    if constexpr (kPair)
        asm volatile("{\n .reg .b64 a;\n mov.b64 a, {%1, %2};\n tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], a;\n}" ::"r"(tmem), "r"(lo),
                     "n"(kDescScales)
                     : "memory");
    else
        asm volatile("{\n .reg .b64 a;\n mov.b64 a, {%1, %2};\n tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], a;\n}" ::"r"(tmem), "r"(lo),
                     "n"(kDescScales)
                     : "memory");
}

// D += A B^T (add: else D =) with block scales: E4M3 with one E8M0 scale per 32 (32 elements of K) ...
template <bool kPair>
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add) {
    if constexpr (kPair)
        asm volatile(
            "{\n .reg .b64 a, b;\n .reg .pred p;\n mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], p;\n}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add), "n"(kDescSw128)
            : "memory");
    else
        asm volatile(
            "{\n .reg .b64 a, b;\n .reg .pred p;\n mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], p;\n}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add), "n"(kDescSw128)
            : "memory");
}

// ... and E2M1 with one E4M3 scale per 16 (64 elements of K).
template <bool kPair>
__device__ __forceinline__ void mma_nvf4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add) {
    if constexpr (kPair)
        asm volatile(
            "{\n .reg .b64 a, b;\n .reg .pred p;\n mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %3, [%4], [%5], p;\n}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add), "n"(kDescSw128)
            : "memory");
    else
        asm volatile(
            "{\n .reg .b64 a, b;\n .reg .pred p;\n mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %3, [%4], [%5], p;\n}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add), "n"(kDescSw128)
            : "memory");
}

// The next 8, 64 or 128 columns of this warp's 32 lanes, thread i holding lane i's.  The load and its wait are
// one statement: nothing can use the registers before they are written.
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
        "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
        "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63, %64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, "
        "%82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, %100, "
        "%101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, "
        "%117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]),
          "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]),
          "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]),
          "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]),
          "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(addr)
        : "memory");
}

// Instruction descriptor of a block-scaled product of K-major operands, M x N.
__host__ __device__ constexpr uint32_t idesc_block_scaled(bool nvfp4, int m, int n) {
    return (nvfp4 ? (1u << 7) | (1u << 10) : (1u << 23)) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// The scale of K step k within a 4-scale word (MXFP8, one scale per step).
__host__ __device__ constexpr uint32_t idesc_scale_id(uint32_t k) { return (k << 4) | (k << 29); }

}  // namespace tc
