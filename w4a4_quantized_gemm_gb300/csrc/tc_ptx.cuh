// Inline-PTX wrappers for the sm_100-family async machinery used by the
// tcgen05 GEMM: mbarriers, 1-D bulk copies, tensor-memory allocation, the
// tcgen05 MMA / commit / load instructions and their shared-memory matrix
// descriptors.  Every wait is bounded (see wait_parity).
#pragma once
#include "common.cuh"

namespace w4a4 {
namespace tc {

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx_only(uint32_t bar, uint32_t bytes) {  // no arrival
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Same test, but a thread whose phase is not complete sleeps in the barrier
// unit until it completes or `hint_ns` elapses, instead of spinning: a
// polling warp would take issue slots that the tensor core's work needs.
__device__ __forceinline__ bool mbar_try_wait_sleep(uint32_t bar, uint32_t parity, uint32_t hint_ns) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(hint_ns)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t globaltimer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(t));
    return t;
}

// Wait until the phase with the given parity has completed, giving up after
// `limit_ns` or as soon as another role has raised *abort.  Returns false on
// give-up (the caller then unwinds).  Between tries the warp sleeps for
// `backoff_ns`: a polling warp would take issue slots from the warps doing
// the work (and from the tensor core's instruction stream).  The clock and the
// abort flag are read every 16 tries.
__device__ __forceinline__ bool wait_parity(uint32_t bar, uint32_t parity, volatile int* abort,
                                            uint64_t limit_ns, uint32_t backoff_ns = 0) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (backoff_ns) __nanosleep(backoff_ns);
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > limit_ns) return false;
        }
    }
}

// Same contract, but a warp whose phase is not complete is suspended in the
// barrier unit -- woken when the phase completes, or after `hint_ns` -- instead
// of polling: no issue slots are spent while waiting, and no sleep is added
// after the completion.  The clock and the abort flag are read after every
// suspension.
__device__ __forceinline__ bool wait_parity_suspend(uint32_t bar, uint32_t parity, volatile int* abort,
                                                    uint64_t limit_ns, uint32_t hint_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, hint_ns)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}
__device__ __forceinline__ bool warp_wait_parity_suspend(uint32_t bar, uint32_t parity, volatile int* abort,
                                                         uint64_t limit_ns, uint32_t hint_ns) {
    const bool ok = wait_parity_suspend(bar, parity, abort, limit_ns, hint_ns);
    return __all_sync(0xffffffffu, ok);
}

// Warp-wide wait: every lane polls the same barrier (no divergent branch around
// a blocking instruction) and the lanes agree on the outcome.  The phase cannot
// complete twice before this warp itself arrives somewhere, so all lanes see
// the same completion.
__device__ __forceinline__ bool warp_wait_parity(uint32_t bar, uint32_t parity, volatile int* abort,
                                                 uint64_t limit_ns, uint32_t backoff_ns = 0) {
    const bool ok = wait_parity(bar, parity, abort, limit_ns, backoff_ns);
    return __all_sync(0xffffffffu, ok);
}

// ---- thread-block clusters: distributed shared memory --------------------
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// Address of the same shared-memory location in CTA `rank` of this cluster.
__device__ __forceinline__ uint32_t mapa_shared(uint32_t saddr, uint32_t rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(d) : "r"(saddr), "r"(rank));
    return d;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}
// Asynchronous 16-byte store into another CTA's shared memory that completes
// 16 bytes of transaction count on an mbarrier of that CTA (both addresses
// from mapa_shared); no fence is needed for the receiver to see the data once
// it observes the barrier phase.
__device__ __forceinline__ void st_async_b64(uint32_t remote_addr, long long v, uint32_t remote_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];\n" ::"r"(remote_addr),
                 "l"(v), "r"(remote_bar)
                 : "memory");
}
__device__ __forceinline__ void st_async_v2(uint32_t remote_addr, float a, float b, uint32_t remote_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];\n" ::"r"(
                     remote_addr),
                 "f"(a), "f"(b), "r"(remote_bar)
                 : "memory");
}
__device__ __forceinline__ void st_async_v4(uint32_t remote_addr, float4 v, uint32_t remote_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];\n" ::"r"(
                     remote_addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(remote_bar)
                 : "memory");
}
// Named barrier over `nthreads` threads (a multiple of 32) of this CTA.
__device__ __forceinline__ void named_bar_sync(uint32_t id, uint32_t nthreads) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(nthreads) : "memory");
}
// Arrive on a named barrier without waiting (producer side of a handoff whose
// consumer calls named_bar_sync with the same id and count).
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t nthreads) {
    asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(nthreads) : "memory");
}
// Named barrier over `nthreads` threads with an OR reduction: every
// participant receives the OR of the participants' predicates, so all of them
// take the same branch after it.
__device__ __forceinline__ bool named_bar_red_or(uint32_t id, uint32_t nthreads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\n"
        "bar.red.or.pred q, %2, %3, p;\n"
        "selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(uint32_t(pred)), "r"(id), "r"(nthreads)
        : "memory");
    return r != 0;
}
// Arrive on an mbarrier of another CTA of the cluster, releasing this thread's
// earlier (distributed) shared-memory writes to whoever acquires the phase.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(remote_bar) : "memory");
}
// Cluster-scope acquire of a completed phase (pairs with mbar_arrive_remote).
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait_parity_cluster(uint32_t bar, uint32_t parity, volatile int* abort,
                                                         uint64_t limit_ns) {
    bool ok = mbar_try_wait_cluster(bar, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t n = 1;; ++n) {
            __nanosleep(64);
            if (mbar_try_wait_cluster(bar, parity)) {
                ok = true;
                break;
            }
            if ((n & 15u) == 0 && (*abort || globaltimer_ns() - t0 > limit_ns)) break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}
// The two halves of a cluster barrier, for work placed between them.
// ---- flags in global memory shared by the CTAs of one launch --------------
__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release_gpu(uint32_t* p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;\n" ::"l"(p), "r"(v) : "memory");
}
// One 32-byte store from a thread (p 32-byte aligned): a whole L2 sector, half the
// store transactions of two 16-byte stores to the same bytes.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// Release-ordered increment: this thread's earlier writes are visible to whoever
// acquires the counter's new value.
__device__ __forceinline__ void red_add_release_gpu(uint32_t* p, uint32_t v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;\n" ::"l"(p), "r"(v) : "memory");
}
// Waits, for at most limit_ns, until *p == want (acquire: the writes released
// with the flag are visible afterwards); false on time-out or abort.
__device__ __forceinline__ bool wait_flag_gpu(const uint32_t* p, uint32_t want, volatile int* abort,
                                              uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 0;; ++n) {
        if (ld_acquire_gpu(p) == want) return true;
        if ((n & 15u) == 15u && (*abort || globaltimer_ns() - t0 > limit_ns)) return false;
        __nanosleep(64);
    }
}

__device__ __forceinline__ void cluster_arrive_release() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_acquire() {
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// Every thread of every CTA of the cluster: no CTA leaves before the others are
// done with its shared memory.
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Arrive on a CTA mbarrier once every cp.async this thread issued so far has
// landed; the arrival counts toward the barrier's initial count (noinc).
__device__ __forceinline__ void cp_async_mbar_arrive_noinc(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// The same with an arrival of its own, which the phase then waits for: counted when this is
// issued, before an arrival that the barrier counts on.
__device__ __forceinline__ void cp_async_mbar_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

// Prefetch `bytes` (a multiple of 16, 16-byte aligned) of global memory into L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(src), "r"(bytes) : "memory");
}

// 16-byte cp.async global -> shared that copies src_bytes (16 or 0) and fills
// the rest of the 16 bytes with zeros.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// 1-D bulk copy global -> shared, completing `bytes` of transaction count on bar.
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// A box of a 4-D tensor map (coordinates innermost first) into shared memory.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_tensor_map(const void* map) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// ---- tensor memory --------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}

// Shared-memory matrix descriptor: K-major operand stored as planes of
// [rows][32 bytes] with the 32-byte swizzle; 8-row core groups 256 bytes apart.
// Fields: start address >> 4 (bits 0-13), leading byte offset >> 4 (16-29,
// unused for swizzled K-major), stride byte offset >> 4 (32-45), descriptor
// version 1 (46-47), base offset 0 (49-51), swizzle mode 6 = 32B (61-63).
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t saddr) {
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFFu) >> 4);
    d |= uint64_t(1) << 16;
    d |= uint64_t(256 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(6) << 61;
    return d;
}

// Instruction descriptor: fp32 accumulator (bits 4-5 = 1), A/B format code 0
// (E4M3 for kind::f8f6f4, F16 for kind::f16), both K-major, N >> 3 at bit 17,
// M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_m128(int n) {
    return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Same, with the A operand in tensor memory (lane = row, byte k % 4 of column
// k / 4 for the 32 k of one MMA) and B in shared memory.
__device__ __forceinline__ void mma_f8_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                              uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Shared-memory matrix descriptors of tiles stored as planes of [rows][128 bytes] with the
// 128-byte swizzle (a row's 16-byte pieces XORed with its number modulo 8; planes 1024-byte
// aligned).  As a K-major operand a row is a row of the matrix and the plane's 64 16-bit
// elements are a piece of its K; 8-row groups lie 1024 bytes apart.  As an MN-major operand a
// row is one k and the plane's elements are 64 of the rows (columns) of the matrix; planes
// are `plane` bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t plane = 16) {
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFFu) >> 4);
    d |= uint64_t(plane >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}
// kind::f16 with the operands' type (bits 7-9, 10-12: 1 = BF16) and an MN-major B (bit 16).
__host__ __device__ constexpr uint32_t idesc_m128_16bit(int n, bool bf16, bool b_mn) {
    return idesc_m128(n) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u);
}
// A row of kind::f16 MMAs in one block, so that their descriptors are sums of an immediate and
// the first one's low word: left to the compiler, the sums of all of them are kept (and
// spilled) between the rows, and loading them holds the tensor cores up.  `acc`: whether the
// first one adds to the accumulator; the others do.
// STEPS 16-element steps of K of two K-major operands in planes of 128 rows of 128 bytes.
template <int STEPS>
__device__ __forceinline__ void mma_f16_rows(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool acc) {
    static_assert(STEPS == 4 || STEPS == 6 || STEPS == 8, "planes of four steps");
    if constexpr (STEPS == 4)
        asm volatile(
            "{\n.reg .pred p, q;\n.reg .b64 a, b;\n.reg .b32 x, y;\nsetp.ne.b32 p, %5, 0;\nsetp.eq.b32 q, 0, 0;\n"
            "add.u32 x, %1, 0;\nadd.u32 y, %2, 0;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
            "add.u32 x, %1, 2;\nadd.u32 y, %2, 2;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 4;\nadd.u32 y, %2, 4;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 6;\nadd.u32 y, %2, 6;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "}\n" ::"r"(d_tmem), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(uint32_t(acc))
            : "memory");
    else if constexpr (STEPS == 6)
        asm volatile(
            "{\n.reg .pred p, q;\n.reg .b64 a, b;\n.reg .b32 x, y;\nsetp.ne.b32 p, %5, 0;\nsetp.eq.b32 q, 0, 0;\n"
            "add.u32 x, %1, 0;\nadd.u32 y, %2, 0;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
            "add.u32 x, %1, 2;\nadd.u32 y, %2, 2;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 4;\nadd.u32 y, %2, 4;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 6;\nadd.u32 y, %2, 6;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 1024;\nadd.u32 y, %2, 1024;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 1026;\nadd.u32 y, %2, 1026;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "}\n" ::"r"(d_tmem), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(uint32_t(acc))
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p, q;\n.reg .b64 a, b;\n.reg .b32 x, y;\nsetp.ne.b32 p, %5, 0;\nsetp.eq.b32 q, 0, 0;\n"
            "add.u32 x, %1, 0;\nadd.u32 y, %2, 0;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
            "add.u32 x, %1, 2;\nadd.u32 y, %2, 2;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 4;\nadd.u32 y, %2, 4;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 6;\nadd.u32 y, %2, 6;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 1024;\nadd.u32 y, %2, 1024;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 1026;\nadd.u32 y, %2, 1026;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 1028;\nadd.u32 y, %2, 1028;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "add.u32 x, %1, 1030;\nadd.u32 y, %2, 1030;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n"
            "}\n" ::"r"(d_tmem), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(uint32_t(acc))
            : "memory");
}
// The A operand 64 elements of K in tensor memory (lane = row, k = 2 * column + half), B an
// MN-major operand of 64 rows of 128 bytes (a plane).
__device__ __forceinline__ void mma_f16_tmem_a_rows(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t hi, uint32_t idesc,
                                                    bool acc) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 b;\n.reg .b32 x, y;\nsetp.ne.b32 p, %5, 0;\nsetp.eq.b32 q, 0, 0;\n"
        "add.u32 x, %1, 0;\nadd.u32 y, %2, 0;\nmov.b64 b, {y, %3};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, p;\n"
        "add.u32 x, %1, 8;\nadd.u32 y, %2, 128;\nmov.b64 b, {y, %3};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n"
        "add.u32 x, %1, 16;\nadd.u32 y, %2, 256;\nmov.b64 b, {y, %3};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n"
        "add.u32 x, %1, 24;\nadd.u32 y, %2, 384;\nmov.b64 b, {y, %3};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, q;\n"
        "}\n" ::"r"(d_tmem), "r"(a_tmem), "r"(b), "r"(hi), "r"(idesc), "r"(uint32_t(acc))
        : "memory");
}
// Arrive on `bar` once every tcgen05 operation issued so far by this thread completes.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
                 : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns -> 32 registers per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 16 consecutive 32-bit columns -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Same load into 32 consecutive floats of a larger register array.
__device__ __forceinline__ void tmem_ld32_at(uint32_t taddr, float* v) {
    tmem_ld32(taddr, *reinterpret_cast<float(*)[32]>(v));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }

// registers -> 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
        "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
        "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
        "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
        "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
        "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
        : "memory");
}
// registers -> 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15]))
        : "memory");
}
// 16 raw 32-bit words -> 32 lanes x 16 consecutive columns.
__device__ __forceinline__ void tmem_st16_b32(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 32 raw 32-bit words -> 32 lanes x 32 consecutive columns.
__device__ __forceinline__ void tmem_st32_b32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Per-warpgroup register re-budgeting (all four warps of a warpgroup execute
// the same instruction).  The sum over warpgroups must stay within the
// registers the block was launched with, or the increase never completes.
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Packed fp32 pairs held as 64-bit values, so that a chain of pair FMAs keeps
// its operands in register pairs (no repacking between instructions).
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
// d = a * b + c on both halves.
__device__ __forceinline__ uint64_t ffma2_b64(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// d = a + b on both halves.
__device__ __forceinline__ uint64_t fadd2_b64(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// d = a * b on both halves.
__device__ __forceinline__ uint64_t fmul2_b64(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Four 8x8 b16 matrices from shared memory (row addresses from lanes 8i..8i+7
// for matrix i); lane l receives the 32-bit word (row l / 4, column pair l % 4)
// of each.
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t saddr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}

// Packed fp32 pair FMA (sm_100 family): d = a * b + c elementwise.
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 ra, rb, rc, rd;\n"
        "mov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\nmov.b64 rc, {%6, %7};\n"
        "fma.rn.f32x2 rd, ra, rb, rc;\n"
        "mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

}  // namespace tc
}  // namespace w4a4
