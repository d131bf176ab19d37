// Inline-PTX wrappers of the matrix operators that ptx.cuh does not have: CTA
// pairs (cta_group::2), cluster barriers and distributed shared memory.
#pragma once
#include "ptx.cuh"

namespace mhcpb {
namespace ptx {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Address in shared::cluster of the same variable in the block of rank `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Arrival on a barrier of any block of the cluster (a shared::cluster address).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_try_wait that also orders what other blocks of the cluster did before they arrived.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

// The wrappers below whose name ends in _one are called by a whole warp with the
// same arguments in every lane, and issue their instructions in one lane (always the
// same: elect.sync is deterministic).  Under a branch on the lane number a step of 64 k took
// 840 clocks to issue, this way 500.
__device__ __forceinline__ void mbar_expect_one(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}
// 2-D tiled load into this block's shared memory, counted on `bar`: with PAIR a
// barrier of either block of the pair (a shared::cluster address).
template <bool PAIR>
__device__ __forceinline__ void tma_load_one(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xFFFFFFFF;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xFFFFFFFF;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

// TMEM of a block, or of both blocks of a pair (each block's warp calls it).
template <bool PAIR>
__device__ __forceinline__ void tmem_get(uint32_t holder, uint32_t columns) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(holder), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(holder, columns);
        tmem_relinquish();
    }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t columns) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns) : "memory");
    else
        tmem_dealloc(taddr, columns);
}

// 32 columns of this warp's 32 lanes of TMEM, and the wait for such stores.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
        "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
        "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
        "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]),
        "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[smem] B[smem] over 64 k: four MMAs of 16-bit operands with FP32
// accumulation, the descriptors a_step and b_step apart.
#define MHCM_MMA64(GROUP)                                                                      \
    asm volatile(                                                                              \
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 x, y;\n\t"                                     \
        "elect.sync _|q, 0xFFFFFFFF;\n\t"                                                     \
        "setp.ne.b32 p, %6, 0;\n\t"                                                           \
        "setp.eq.b32 t, 0, 0;\n\t"                                                            \
        "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], %1, %2, %3, p;\n\t"               \
        "add.s64 x, %1, %4;\n\tadd.s64 y, %2, %5;\n\t"                                       \
        "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], x, y, %3, t;\n\t"                 \
        "add.s64 x, x, %4;\n\tadd.s64 y, y, %5;\n\t"                                         \
        "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], x, y, %3, t;\n\t"                 \
        "add.s64 x, x, %4;\n\tadd.s64 y, y, %5;\n\t"                                         \
        "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),      \
        "l"(a), "l"(b), "r"(idesc), "l"(a_step), "l"(b_step), "r"(accumulate)                  \
        : "memory")
template <bool PAIR>
__device__ __forceinline__ void mma64_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t a_step,
                                          uint64_t b_step, uint32_t accumulate) {
    if constexpr (PAIR)
        MHCM_MMA64("2");
    else
        MHCM_MMA64("1");
}
#undef MHCM_MMA64
// One arrival, when this warp's MMAs so far are done, on the barrier at this
// offset in each block whose bit is set in `mask` (without PAIR: in this block).
template <bool PAIR>
__device__ __forceinline__ void mma_commit_one(uint32_t bar, uint16_t mask) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xFFFFFFFF;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            "\n\t}" ::"r"(bar),
            "h"(mask)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xFFFFFFFF;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
            : "memory");
}

// Two FP32 in one register pair, and the packed multiply-add.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float sum_of(uint64_t v) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return lo + hi;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

// Instruction descriptor of kind::f16 with FP32 accumulators: as idesc_bf16_f32,
// with FP16 operands (format 0) or BF16 ones (format 1).
__host__ __device__ constexpr uint32_t idesc_16bit(uint32_t M, uint32_t N, bool bf16, bool a_mn, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Bytes [p, end) towards L2: the 16-byte vectors that lie in them.
__device__ __forceinline__ void prefetch_l2(const void* p, const void* end) {
    const uint64_t from = (reinterpret_cast<uint64_t>(p) + 15) & ~15ull, to = reinterpret_cast<uint64_t>(end) & ~15ull;
    if (to > from)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(reinterpret_cast<void*>(from))),
                     "r"((uint32_t)(to - from))
                     : "memory");
}

}  // namespace ptx
}  // namespace mhcpb
