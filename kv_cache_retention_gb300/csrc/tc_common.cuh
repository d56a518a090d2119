// PTX wrappers of the attention kernels on the 5th-generation tensor cores: mbarriers with bounded waits, TMA loads, MMAs
// with operands in shared memory and TMEM, TMEM reads and writes.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "kvsel_internal.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 128;              // rows of a tile, keys of a step
constexpr uint64_t kWaitNs = 1000000000ull;

// A block's waits: whether one has given up, and how long each goes on.
struct Stop {
    volatile int given_up;
    uint64_t limit_ns;
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(saddr(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t gtimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Bounded wait for a phase; false when this or another role gave up.
__device__ __forceinline__ bool wait_phase(uint64_t* b, uint32_t parity, Stop* stop, unsigned* err) {
    if (mbar_try(b, parity)) return true;
    const uint64_t t0 = gtimer();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try(b, parity)) return true;
        if ((i & 63) == 0) {
            if (stop->given_up) return false;
            if (gtimer() - t0 > stop->limit_ns) {
                stop->given_up = 1;
                atomicOr(err, (unsigned)KVSEL_DEV_TIMEOUT);
                return false;
            }
        }
    }
}
// The same for a whole warp, with one answer for its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* b, uint32_t parity, Stop* stop, unsigned* err) {
    return __all_sync(0xffffffffu, wait_phase(b, parity, stop, err));
}
// Bounded wait that ignores the abort flag: a role's own copies or MMAs before the block ends.
__device__ __forceinline__ void drain_phase(uint64_t* b, uint32_t parity) {
    const uint64_t t0 = gtimer();
    while (!mbar_try(b, parity) && gtimer() - t0 < kWaitNs) {
    }
}
__device__ __forceinline__ void tma_load(const CUtensorMap* map, uint64_t* bar, void* dst, int d, int h, int t) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            saddr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(saddr(bar)), "r"(d), "r"(h), "r"(t)
        : "memory");
}
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// kind::f16 instruction descriptor: fp32 sums, bf16 operands, M = 128; b_mn: B's rows run along K.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTile >> 4) << 24);
}
// Shared-memory descriptors, 128-byte swizzle: the low word holds the address and the leading offset, the high
// word the stride offset (1024 bytes), version and swizzle.  K-major: groups of 8 rows 1024 bytes apart.  MN-major:
// groups of 8 K rows 1024 bytes apart (stride offset), blocks of 64 columns one tile block apart (leading offset).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t leading) {
    return ((addr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16);
}
// v, the same in every lane, in a uniform register: MMA operands that come from ordinary registers cost a move of
// about 10 cycles each, four for an MMA of 64.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
// MMAs and commits are issued by the lane whose `lead` is set; the operands are computed by the whole warp, so
// that they stay in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 x, y;\n mov.b64 x, {%1, %6};\n mov.b64 y, {%2, %6};\n setp.ne.b32 p, %4, 0;\n"
        " setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(accum), "r"(lead), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 y;\n mov.b64 y, {%2, %6};\n setp.ne.b32 p, %4, 0;\n"
        " setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(accum), "r"(lead), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(lead)
        : "memory");
}
// The same issued by one thread that elect_one has chosen, in a branch of its own: elections and predicates of each MMA fall
// away, which halves the instructions (attention of 2048 tokens behind 32768 cached ones, two issuers in turn: 857 us, 965
// with the predicated ones).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void mma_ss_one(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(accum), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(accum), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_commit_one(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define O4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define I4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
// 32 columns of the thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%"
        "21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : O4(r, 0), O4(r, 4), O4(r, 8), O4(r, 12), O4(r, 16), O4(r, 20), O4(r, 24), O4(r, 28)
        : "r"(addr));
}
// 16 of them.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : O4(r, 0), O4(r, 4), O4(r, 8), O4(r, 12)
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
        "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::I4(r, 0),
        I4(r, 4), I4(r, 8), I4(r, 12), I4(r, 16), I4(r, 20), I4(r, 24), I4(r, 28), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::I4(r, 0),
                 I4(r, 4), I4(r, 8), I4(r, 12), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace
