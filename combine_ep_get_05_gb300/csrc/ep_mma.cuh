// ep_mma.cuh -- tensor-core products of a pair of CTAs (tcgen05, cta_group::2): descriptors,
// the instruction, tensor memory, and the barriers between the two CTAs. Internal header.
//
// A pair multiplies M = 256 rows of A (128 from each CTA's shared memory) with N columns of B
// (N/2 from each), 16 k at a time, into tensor memory: CTA 0 holds rows 0 .. 127, CTA 1 rows
// 128 .. 255, a row a lane, a column a 32-bit column. With M = 128 each CTA has 64 rows of A, and of the
// sums lanes 0 .. 63 hold their columns 0 .. N/2 - 1, lanes 64 .. 127 the others. Operands lie in shared memory as 128-byte
// swizzled tensor copies leave them, in one of two ways:
//   along k:       rows of 64 k (128 bytes), 8 rows an atom of 1024 bytes
//   across k:      blocks of 64 rows of the operand: 64 lines of one k each, 64 values a line
#pragma once

#include "ep_tma.cuh"

namespace ep {

constexpr int kBlockK = 64;                    // k of a stage: 128 bytes of bf16
constexpr uint32_t kCrossBlock = 64 * 64 * 2;  // bytes of a block of 64 rows by 64 k, across k

// a value that all lanes hold, so that the compiler knows it, too
template <class T>
__device__ __forceinline__ T uniform(T v) {
    return __shfl_sync(0xffffffffu, v, 0);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// one lane of the (converged) warp, the same one every time
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// the cluster's barrier in two parts: what the threads wrote before arriving is seen after waiting
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the same without order for memory accesses (a release waits until all stores have reached L2)
__device__ __forceinline__ void cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// the address, in the cluster's window, of `p`'s counterpart in CTA `rank`
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
// Arrivals at a barrier of either CTA (a cluster address). The first is a release to the cluster for what
// was written to this CTA's shared memory, and for that only: one for all memory waits until the SM's
// stores have reached L2, some 2000 cycles. The second orders nothing, for tensor memory, which tcgen05's
// own fences order.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    mbar_arrive_cluster_relaxed(addr);
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// One poll of a barrier's phase; the poll itself waits a little in hardware. kCluster: the other
// CTA's threads arrive there too.
template <bool kCluster>
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    if (kCluster)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
    return done != 0;
}
// What a CTA's waits look at (shared memory): whether one of them gave up, and how many stages have been
// filled so far, since a wait may be for a tile of any number of stages.
struct Watch {
    int stop;
    uint32_t stages;
};
// Waits until the phase is over; gives up, and returns false, after about 2 s in which no stage was filled,
// or once the watch says so. Without a watch: after about 2 s.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, const volatile Watch* watch) {
    unsigned long long start = 0;
    uint32_t stages = 0;
    for (uint32_t i = 0; i < (1u << 26); ++i) {
        if (mbar_try<kCluster>(bar, parity)) return true;
        if ((i & 63u) != 63u) continue;
        if (watch != nullptr && watch->stop != 0) break;
        const unsigned long long now = globaltimer_ns();
        const uint32_t filled = watch != nullptr ? watch->stages : 0;
        if (start == 0 || filled != stages)
            start = now, stages = filled, i = 0;
        else if (now - start > 2000000000ull)
            break;
    }
    return false;
}

// the same for a whole warp
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile Watch* watch) {
    if (__all_sync(0xffffffffu, mbar_try<kCluster>(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, watch));
}

// tensor loads whose bytes are counted on a barrier of either CTA of the pair (a cluster address)
__device__ __forceinline__ void tma_load_pair_2d(uint32_t dst, const CUtensorMap& map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap_addr(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_pair_3d(uint32_t dst, const CUtensorMap& map, int x, int y, int z,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap_addr(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// tensor memory: `columns` for the pair, the address into *at (shared); one warp of each CTA
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* at, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand descriptor: address and strides in units of 16 bytes, version 1, 128-byte
// swizzle. Along k an atom of 8 rows follows another every 1024 bytes (and 16 k are 32 bytes
// further); across k, 8 lines of k are 1024 bytes and a block of 64 rows kCrossBlock (and 16 k
// are 16 lines, 2048 bytes, further). The lower half has what changes from product to product.
__device__ __forceinline__ uint32_t operand_low(uint32_t addr, bool across) {
    return (addr & 0x3ffffu) >> 4 | (across ? kCrossBlock >> 4 : 1u) << 16;
}
constexpr uint32_t kOperandHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
constexpr uint32_t kStepAlong = 32 >> 4, kStepAcross = 2048 >> 4;  // a descriptor's, per 16 k

// Instruction descriptor: bf16 operands, fp32 sums, M = m (128 or 256), N = n; bits 15 and 16: A, B across k.
__device__ __forceinline__ uint32_t product_desc(int m, int n, bool a_across, bool b_across) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_across ? 1u << 15 : 0u) | (b_across ? 1u << 16 : 0u) |
           static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}
// D (+)= A B^T over 16 k; one thread of CTA 0, for the pair
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(desc), "r"(static_cast<uint32_t>(add)), "n"(kOperandHigh)
        : "memory");
}
// arrives on this CTA's barrier when the thread's products so far are done
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// arrives on the barrier, in both CTAs, when the thread's products so far are done
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ---------------------------------------------------------------------------- 32 x 16 sums a warp
// A warp's 32 lanes of tensor memory by 16 columns, as the fragments of 8 x 8 matrices that
// stmatrix and ldmatrix move: v[8 h + 4 q + i] is lane 16 h + 8 (i / 2) + t / 4, column
// 8 q + 2 (t % 4) + i % 2, for thread t of the warp; or packed, w[4 q + b] holds two columns,
// 8 q + 2 (t % 4) and the next, of lane 8 b + t / 4.
constexpr int kChunk = 16;

__device__ __forceinline__ constexpr int fragment(int q, int b) { return 8 * (b / 2) + 4 * q + 2 * (b % 2); }

__device__ __forceinline__ void tmem_load_half(float* v, uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_load(float (&v)[16], uint32_t at) {
    tmem_load_half(v, at);
    tmem_load_half(v + 8, at + (16u << 16));
}
// until the loads are done; the values are used only after it
__device__ __forceinline__ void tmem_load_wait(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15])
                 :
                 : "memory");
}

// Between fragments and rows: a warp's patch of shared memory, 16 rows (columns of the sums) of
// 32 channels (lanes) of 16 bits, 64 bytes each. A row's four 16-byte vectors change places with
// the row, so that both the eight rows of a matrix and two whole rows fall on all banks.
constexpr uint32_t kPatchBytes = kChunk * 64;

__device__ __forceinline__ uint32_t patch_vector(uint32_t patch, int row, int vector) {
    return patch + row * 64 + ((vector ^ (row / 2 % 4)) * 16);
}
// a thread's vector of 8 rows from 8 q on: as the matrices take them, and row by row (row t / 4,
// vector t % 4: neighbours in memory)
__device__ __forceinline__ uint32_t matrix_place(uint32_t patch, int q, int lane) {
    return patch_vector(patch, lane % 8, lane / 8) + q * 512;
}
__device__ __forceinline__ uint32_t row_place(uint32_t patch, int q, int lane) {
    return patch_vector(patch, lane / 4, lane % 4) + q * 512;
}
// The same for a patch that two warps share, 16 rows of 64 channels, 128 bytes each, in the places
// of the 128-byte swizzle; `side`: which 32 channels.
__device__ __forceinline__ uint32_t wide_matrix_place(uint32_t patch, int q, int side, int lane) {
    return patch + (8 * q + lane % 8) * 128 + (((4 * side + lane / 8) ^ (lane % 8)) * 16);
}
__device__ __forceinline__ void matrices_put(uint32_t at, const uint32_t (&w)[8], int q) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[4 * q]),
                 "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
}
__device__ __forceinline__ void patch_put(uint32_t patch, const uint32_t (&w)[8], int lane) {
#pragma unroll
    for (int q = 0; q < 2; ++q) matrices_put(matrix_place(patch, q, lane), w, q);
}
__device__ __forceinline__ void patch_get(uint32_t (&w)[8], uint32_t patch, int lane) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                     : "r"(matrix_place(patch, q, lane))
                     : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

}  // namespace ep
