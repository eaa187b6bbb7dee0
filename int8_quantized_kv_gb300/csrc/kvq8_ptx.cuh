// kvq8_ptx.cuh -- thin inline-PTX wrappers used by the decode kernel:
// mbarriers (with a bounded wait), 1-D bulk async copies global->shared,
// an L2 eviction policy, the m16n8k16 fp16 tensor-core MMA, named barriers
// and programmatic-dependent-launch controls.
#pragma once

#include <stdint.h>

namespace kvq8 {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Makes mbarrier initialisation visible to the async (bulk-copy) proxy.
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same, asleep for up to about ns nanoseconds while the phase is not complete.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t global_timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits for the phase of `parity` to complete; gives up after timeout_ns and
// returns false (the caller records the error and unwinds).
__device__ __forceinline__ bool mbar_wait_bounded(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > timeout_ns) return false;
    }
    return true;
}

// Waits for a phase by up to 2^20 tries that sleep up to two microseconds each; false when they are used up.  (The
// nanosecond timer is slow to read: a chain of short waits has this one.)
__device__ __forceinline__ bool mbar_wait_tries(uint32_t bar, uint32_t parity) {
    int left = 1 << 20;
#pragma unroll 1
    while (!mbar_try_wait_for(bar, parity, 2000u))
        if (--left == 0) return false;
    return true;
}

// What was done before *at got the value that it has (by a kernel that is over) is seen by the loads behind this, whatever
// this SM's L1 holds of it.
__device__ __forceinline__ void acquire_gpu(const int32_t *at) {
    asm volatile("{\n\t.reg .s32 x;\n\tld.relaxed.gpu.global.s32 x, [%0];\n\tfence.acq_rel.gpu;\n\t}" ::"l"(at) : "memory");
}

// L2 policy for data read exactly once (the streamed KV cache).
__device__ __forceinline__ uint64_t l2_evict_first_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// 1-D bulk copy global -> shared, completing `bytes` of transaction on `bar`.
// dst, src 16-byte aligned; bytes a multiple of 16.
__device__ __forceinline__ void bulk_copy_g2s(uint32_t dst, const void *src, uint32_t bytes,
                                              uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// 16-byte asynchronous copy global -> shared (cached in L2 only); dst and
// src 16-byte aligned.  Completion through commit / wait groups.
__device__ __forceinline__ void cp_async16_cg(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}

// 8 bytes (dst, src 8-byte aligned), through L1.
__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most N of this thread's copy groups are pending.
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Hint: bring `bytes` of global memory at src into L2 (no completion to wait
// for).  src 16-byte aligned; bytes a multiple of 16.
__device__ __forceinline__ void bulk_prefetch_l2(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// 2^x by the hardware's approximate base-2 exponential (relative error about
// 2^-22, far inside the decode's output tolerance; results below 2^-126, which
// weigh nothing next to a running maximum's 1, flush to 0; -inf gives 0).
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D (16x8 fp32) += A (16x16 fp16, row) * B (16x8 fp16, col).
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void named_barrier_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Thread-block clusters: this CTA's rank, a barrier over all their threads (with
// their shared memory's writes before it visible after it), and loads of what
// lies at `p` of this CTA's shared memory in the shared memory of CTA `rank`.
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_addr(const void *p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ int load_cluster_int(const int *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ int4 load_cluster_int4(const int4 *p, int rank) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(cluster_addr(p, rank))
                 : "memory");
    return v;
}

// ------------------------------------------------ 5th-generation tensor cores --
// Tensor memory: 512 columns of 128 lanes of 32 bits per SM; an address is
// (lane << 16) | column, and warp w of a CTA reaches lanes 32 * (w % 4) .. + 31.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand of 8 x 8 (16-byte) cores without swizzle: `k_bytes`
// from one core to the next along the contraction, `n_bytes` along the other
// dimension (leading and stride offsets of the descriptor, in this order for
// both a contraction-major and an n-major operand).
__device__ __forceinline__ uint64_t core_desc(uint32_t addr, uint32_t k_bytes, uint32_t n_bytes) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((k_bytes >> 4) & 0x3fff) << 16 |
           (uint64_t)((n_bytes >> 4) & 0x3fff) << 32 | 1ull << 46;
}

// Instruction word of a 128 x n MMA of fp16 operands with fp32 accumulators; A
// is contraction-major, B too or (n_major) not.
__host__ __device__ constexpr uint32_t mma_word(int n, bool n_major) {
    return 1u << 4 | (n_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

// D (tensor memory, 128 x n) (+)= A (tensor memory, 128 x 128 halves: eight steps of 8 columns) B (shared memory, n x
// 128: steps 256 bytes apart).  The whole warp comes here and elects the lane that issues, so that the operands stay in
// uniform registers: a step takes 31 clocks to issue (17 to run, for n = 32), with a lane chosen by its number 67.
// kDown: what D held counts 2^-kDown of itself (0 .. 15).
template <int kDown = 0>
__device__ __forceinline__ void mma_k128(uint32_t d, uint32_t a, uint64_t b, uint32_t word, bool accumulate) {
#define KVQ8_MMA_STEP "add.u32 ta, ta, 8;\n\tadd.s64 tb, tb, 16;\n\t@p tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], tb, %3, r;\n\t"
    asm volatile(
        "{\n\t.reg .pred p, q, r;\n\t.reg .b32 ta;\n\t.reg .b64 tb;\n\t"
        "elect.sync _|p, 0xffffffff;\n\tsetp.ne.u32 q, %4, 0;\n\tsetp.eq.u32 r, %0, %0;\n\t"
        "mov.b32 ta, %1;\n\tmov.b64 tb, %2;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], tb, %3, q, %5;\n\t"
        KVQ8_MMA_STEP KVQ8_MMA_STEP KVQ8_MMA_STEP KVQ8_MMA_STEP KVQ8_MMA_STEP KVQ8_MMA_STEP KVQ8_MMA_STEP "}" ::"r"(d),
        "r"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate), "n"(kDown)
        : "memory");
#undef KVQ8_MMA_STEP
}

// One arrival on the mbarrier when the MMAs that this warp has issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Columns of this warp's lanes.  (A load's registers hold their values after tmem_wait_ld; the caller orders what
// uses them behind it.)
#define KVQ8_R8(r) "=f"((r)[0]), "=f"((r)[1]), "=f"((r)[2]), "=f"((r)[3]), "=f"((r)[4]), "=f"((r)[5]), "=f"((r)[6]), "=f"((r)[7])
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : KVQ8_R8(r) : "r"(addr));
}
// Sixteen lanes (from addr's lane on) x 8 * kGroups columns as MMA fragments: of column group g, r[4g], r[4g + 1] are
// lane t / 4, columns 8g + 2 (t % 4), + 1 for thread t, and r[4g + 2], r[4g + 3] the same of lane t / 4 + 8.
template <int kGroups>
__device__ __forceinline__ void tmem_ld_fragments(uint32_t addr, float *r) {
    if constexpr (kGroups == 4) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : KVQ8_R8(r), KVQ8_R8(r + 8)
            : "r"(addr));
    } else {
        static_assert(kGroups == 2, "groups");
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : KVQ8_R8(r) : "r"(addr));
    }
}
#undef KVQ8_R8

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Four 8 x 8 matrices of halves, each given as MMA fragments, to rows of 16 bytes; lane l says where row l % 8 of matrix
// l / 8 goes.
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// Shared-memory writes of this thread become visible to the async proxy (MMA operands).
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Barrier over `threads` threads that says whether any of them has `x` set.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

template <int N>
__device__ __forceinline__ void regs_shrink() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_grow() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// 1-D bulk copy global -> shared without an L2 hint.
__device__ __forceinline__ void bulk_copy_g2s_plain(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Programmatic dependent launch: let the next kernel in the stream start its
// launch, and (in that kernel) wait until this grid's results are visible.
__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace kvq8
