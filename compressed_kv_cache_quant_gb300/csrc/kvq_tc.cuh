// What the tcgen05 kernels share: mbarriers with bounded waits, TMA, descriptors, products, TMEM, and tensor maps.
#pragma once

#include <cuda.h>

#include <atomic>

#include "kvq_internal.cuh"

constexpr uint32_t KVQ_SPIN = 1u << 16;   // bound on the polls of one mbarrier wait

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
// a page of one kv head: the map's dims are 64 values, 8 rows, 2 halves of a row, groups of 8 rows
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int group, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(0), "r"(group), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: start address, byte offsets between the 64-element
// blocks of a matrix whose rows run along K (`lead`), and between groups of eight rows (`group`).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t group) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(group >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of f16 x f16 -> f32 products; KVQ_A_MN / KVQ_B_MN: the operand's rows run along K (its
// M or N index is the contiguous one), else along M or N.
constexpr uint32_t KVQ_A_MN = 1u << 15, KVQ_B_MN = 1u << 16;
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n) { return (1u << 4) | (n / 8 << 17) | (m / 16 << 24); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

#define R8(v, o) "=r"((v)[o]), "=r"((v)[o + 1]), "=r"((v)[o + 2]), "=r"((v)[o + 3]), "=r"((v)[o + 4]), "=r"((v)[o + 5]), "=r"((v)[o + 6]), "=r"((v)[o + 7])
#define W8(v, o) "r"((v)[o]), "r"((v)[o + 1]), "r"((v)[o + 2]), "r"((v)[o + 3]), "r"((v)[o + 4]), "r"((v)[o + 5]), "r"((v)[o + 6]), "r"((v)[o + 7])
// 32 columns of this thread's lane; the wait is part of the statement, so nothing reads v before it
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24)
        : "r"(addr)
        : "memory");
}
// all 128 columns of a score tile
__device__ __forceinline__ void tm_ld128(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24), R8(v, 32), R8(v, 40), R8(v, 48), R8(v, 56), R8(v, 64), R8(v, 72), R8(v, 80),
          R8(v, 88), R8(v, 96), R8(v, 104), R8(v, 112), R8(v, 120)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        W8(v, 0), W8(v, 8), W8(v, 16), W8(v, 24)
        : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(v, 0), R8(v, 8)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        W8(v, 0), W8(v, 8)
        : "memory");
}
__device__ __forceinline__ void tm_st1(uint32_t addr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// two fp32 values per instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// CLUSTER: arrivals of other CTAs of the cluster are among those waited for (bar_arrive_in)
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}
// Waits for a phase of bar.  After `limit` polls it flags the timeout, and every wait of the CTA that is
// not over by then returns at once: the roles run through to their ends without waiting, on data that is
// not valid, so no step needs a branch for the failure; only the loads stop (a barrier must not be armed
// twice).  Most waits of the issuing warps find their phase done: one poll and nothing else.
template <bool CLUSTER = false>
__device__ __forceinline__ void bar_wait(int32_t* abort, KvqWsHeader* hdr, uint64_t* bar, uint32_t parity,
                                         uint32_t limit = KVQ_SPIN) {
    const uint32_t at = saddr(bar);
    for (uint32_t it = 0; !bar_done<CLUSTER>(at, parity); ++it) {
        if ((it & 63) != 63) continue;
        if (*(volatile int32_t*)abort) return;
        if (it > limit) {
            *(volatile int32_t*)abort = 1;
            kvq_dev_flag(hdr, KVQ_DEV_TIMEOUT, (int32_t)blockIdx.x);
            return;
        }
    }
}
__device__ __forceinline__ bool aborted(int32_t* abort) {
    return __any_sync(0xffffffffu, *(volatile int32_t*)abort != 0);
}

// The end of a CTA whose wait gave up: its own copies and products land (again with a limit) before it ends.  Every
// thread calls it; `issuer` is one thread of the warp that issued products, `drain` a barrier that nothing else uses.
__device__ __forceinline__ void drain_after_abort(bool issuer, uint64_t* drain) {
    if (issuer) {
        tc_commit(drain);
        for (uint32_t it = 0; it < KVQ_SPIN && !bar_done(saddr(drain), 0); ++it) {}
    }
    const long long began = clock64();
    while (clock64() - began < 2000000) __nanosleep(1000);  // about a millisecond: far above a copy's time
    __syncthreads();
}

// ---- pairs of CTAs (cta_group::2): rank 0 issues the products of both

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of a shared variable in the CTA of that rank
__device__ __forceinline__ uint32_t saddr_in(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr(p)), "r"(rank));
    return r;
}
// Arrives at a barrier of another CTA (an address of saddr_in), and releases to the cluster what the arriving thread has
// written or seen: the waiting thread acquires it with bar_wait<true>.  It takes some 2000 cycles under load.
__device__ __forceinline__ void bar_arrive_in(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// a copy into this CTA that signals a barrier of the pair (an address of saddr_in)
__device__ __forceinline__ void tma_page_pair(uint32_t dst, const CUtensorMap* map, int group, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %2, %2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(map), "r"(0), "r"(group), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void map_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// brings a page into L2
__device__ __forceinline__ void tma_page_prefetch(const CUtensorMap* map, int group) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %1, %1, %2}];" ::"l"(map), "r"(0), "r"(group) : "memory");
}
// arrives at the barrier in both CTAs when all products so far are done
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
__device__ __forceinline__ void mma_ss_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// A tensor map of fp16 values in boxes whose innermost extent is 64 values, 128-byte swizzle.
static inline int make_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
             const char* fn) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static std::atomic<Encode> found_encode{nullptr};   // (threads that make the first call together each look it up)
    Encode encode = found_encode.load(std::memory_order_relaxed);
    if (encode == nullptr) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || f == nullptr) {
            cudaGetLastError();
            return kvq_fail(KVQ_ERR_CUDA, "%s: the driver has no cuTensorMapEncodeTiled", fn);
        }
        encode = reinterpret_cast<Encode>(f);
        found_encode.store(encode, std::memory_order_relaxed);
    }
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const auto fill = [&] {
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void*>(base),
                      reinterpret_cast<const cuuint64_t*>(dims), reinterpret_cast<const cuuint64_t*>(strides), box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = fill();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // the thread has made no runtime call yet that makes its device's context current, as a launch would
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = fill();
    }
    if (r != CUDA_SUCCESS) return kvq_fail(KVQ_ERR_CUDA, "%s: tensor map (%d)", fn, (int)r);
    return KVQ_OK;
}
