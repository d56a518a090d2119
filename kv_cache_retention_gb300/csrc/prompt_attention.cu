// kvsel_prompt_attention: causal attention over packed prompts with grouped heads,
// on the 5th-generation tensor cores.
//
// Sequence s holds tokens [cu[s], cu[s+1]); row i of it sees its rows 0..i:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale log2e q_i . k_j - ref),
//   lse = ln sum_j e^(scale q_i . k_j).
//
// A block takes one query head and 256 consecutive rows of one sequence, as two tiles
// of 128 rows (TMEM lanes), and goes once over the keys from the diagonal down, 128 at
// a time:
//   S = Q K^T   tcgen05.mma, both operands from shared memory, 128 fp32 columns a tile
//   P = 2^(S sc - ref) in bf16, written over S in TMEM
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory as it lies (its rows are
//               the product's K axis: an "MN-major" operand)
// The two tiles share every K and V tile that is loaded (with one tile a block would
// ask L2 for 64 bytes a cycle and SM, about what it gives) and take turns: while one
// tile's softmax runs, the tensor cores work on the other's products.
//
// The softmax keeps per row a reference that only follows the running maximum when
// that has passed it by 8 (log2): weights are then at most 2^8, which bf16 and the fp32
// sums hold as well as 1, and O is rescaled only then.  P is rounded to bf16 since both
// operands of the product have one type and V's range is bf16's; its relative rounding
// of 2^-9 per weight is random and comes to about the output's own rounding.
//
// 384 threads: warp 0 loads (TMA), warps 1 and 2 issue the MMAs of one tile each, warp 3
// looks over the V tiles of the diagonal (below), warps 4-7 and 8-11 are the softmax of the two tiles, a
// row per thread.  TMEM: S of tile 0 and 1 at columns 0 and 128, O at 256 and 384.
//
// Masked places.  A weight of zero does not hide a NaN or an infinity in V.  Key tiles
// below the diagonal are seen by every row of a tile, so only the first two tiles of a
// block's pass hold values that some rows must not see; there warp 3 sets such values
// to zero in shared memory before the product, and if there were any, each row adds
// those it does see to its output at the end (what the sum would be: infinite or NaN).
//
// Every wait is bounded (1 s); on a timeout the block flags KVSEL_ERR_TIMEOUT in the
// device error word, drains its own copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <limits.h>

#include "kvsel_internal.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 128;              // rows of a tile, keys of a step
constexpr int kUnit = 2 * kTile;        // rows of a block
constexpr int kThreads = 384;
constexpr float kSlack = 8.f;           // how far (log2) a row's maximum may pass its reference
constexpr uint64_t kWaitNs = 1000000000ull;
// Registers per thread: at launch, then after the first warpgroup's setmaxnreg.dec and
// the softmax warpgroups' .inc.  An .inc beyond the launch's registers would wait
// forever; the launcher checks the compiled count.
constexpr int kRegsLaunch = 168, kRegsCtl = 80, kRegsSoft = 208;
static_assert(kRegsCtl + 2 * kRegsSoft <= 3 * kRegsLaunch && kRegsLaunch * kThreads <= 65536, "register split");

// All of TMEM is allocated, so its base is column 0.
constexpr uint32_t kTmem = 0;
constexpr int kColS = 0, kColO = 256, kTmemCols = 512;

struct PromptArgs {
    const __nv_bfloat16* v;
    int64_t v_stride;
    const int32_t* cu;
    int S, T, Hq, Hkv, n_virtual;
    float scale2;           // scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
};

template <int D>
struct Cfg {
    static constexpr int kBlock = kTile * 128;             // 128 rows x 64 dims, 128-byte swizzled
    static constexpr int kBytes = D / 64 * kBlock;         // one tile of Q, K or V
    static constexpr int kStages = 5;                      // K and V tiles share the ring
    struct Tail {
        uint64_t q_full, full[kStages], empty[kStages], s_full[2], p_full[2][2], o_done[2], v_ok[2], turn[2], drained;
        uint32_t tmem;
        int abort_flag, odd_v;
    };
    static constexpr size_t kSmem = (size_t)(2 + kStages) * kBytes + sizeof(Tail) + 1024;
    static_assert(kSmem <= 232448, "shared memory per block");
};

// ---- PTX wrappers ----------------------------------------------------------

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
__device__ __forceinline__ bool wait_phase(uint64_t* b, uint32_t parity, volatile int* abort_flag, unsigned* err) {
    if (mbar_try(b, parity)) return true;
    const uint64_t t0 = gtimer();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try(b, parity)) return true;
        if ((i & 63) == 0) {
            if (*abort_flag) return false;
            if (gtimer() - t0 > kWaitNs) {
                *abort_flag = 1;
                atomicOr(err, (unsigned)KVSEL_DEV_TIMEOUT);
                return false;
            }
        }
    }
}
// The same for a whole warp, with one answer for its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* b, uint32_t parity, volatile int* abort_flag, unsigned* err) {
    return __all_sync(0xffffffffu, wait_phase(b, parity, abort_flag, err));
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
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
        "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::I4(r, 0),
        I4(r, 4), I4(r, 8), I4(r, 12), I4(r, 16), I4(r, 20), I4(r, 24), I4(r, 28), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Place in the ring of step i's K and V tile: K0, K1, V0, K2, V1, ..., V(n-1).
__device__ __forceinline__ int at_k(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int at_v(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// ---- MMAs: a warp per tile -------------------------------------------------
// Two issuers on two SM sub-partitions: what one spends on barriers, between the softmax's instructions, passes
// while the other's products run.  They take turns, so that one tile's products run beside the other's softmax.
template <int D, int X>
__device__ __forceinline__ void issue_tile(typename Cfg<D>::Tail& t, const uint8_t* sq, const uint8_t* ring, int n, bool two,
                                           int lane, volatile int* abort_flag, unsigned* err) {
    using C = Cfg<D>;
    constexpr uint32_t kStages = C::kStages;
    const uint32_t lead = lane == 0;
    if (X == 0 || two) {
        const int from = X == 0 && two ? 1 : 0;   // the tile's first step
        const uint32_t q = desc_low(saddr(sq) + X * C::kBytes, 16);
        constexpr uint32_t ts = kTmem + kColS + X * kTile, to = kTmem + kColO + X * D;
        auto issue_s = [&](uint32_t k_desc, bool pass) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * C::kBlock + (k & 3) * 32) >> 4;
                // the other tile's turn: its issuer is under way while the last of these are issued
                if (k == D / 32 && pass && lead) mbar_arrive(&t.turn[1 - X]);
                mma_ss(ts, q + off, k_desc + off, idesc(kTile, false), k > 0, lead);
            }
            mma_commit(saddr(&t.s_full[X]), lead);
        };
        auto k_desc = [&](uint32_t st) { return uniform(desc_low(saddr(ring) + st * C::kBytes, 16)); };
        auto v_desc = [&](uint32_t st) { return uniform(desc_low(saddr(ring) + st * C::kBytes, C::kBlock)); };
        if (from == 1 && lead) {                  // the first K and V tile are the other tile's alone
            mbar_arrive(&t.empty[0]);
            mbar_arrive(&t.empty[at_v(0, n) % kStages]);
        }
        bool ok = wait_warp(&t.q_full, 0, abort_flag, err) && wait_warp(&t.full[at_k(from)], 0, abort_flag, err);
        if (ok) {
            tc_after();
            issue_s(k_desc(at_k(from)), false);
            mma_commit(saddr(&t.empty[at_k(from)]), lead);
        }
        // stages and phases of the tiles of step i: K(i + 1), V(i)
        uint32_t sk = at_k(from + 1) % kStages, pk = at_k(from + 1) / kStages & 1;
        uint32_t sv = at_v(from, n) % kStages, pv = at_v(from, n) / kStages & 1;
        for (int i = from; i < n && ok; ++i) {
            const bool more = i + 1 < n;
            if (!more) sv = at_v(i, n) % kStages, pv = at_v(i, n) / kStages & 1;
            const uint32_t kd = k_desc(sk), vd = v_desc(sv);
            if (more) ok = wait_phase(&t.full[sk], pk, abort_flag, err) && ok;
            ok = wait_phase(&t.full[sv], pv, abort_flag, err) && ok;
            if (i < 2) ok = wait_phase(&t.v_ok[i], 0, abort_flag, err) && ok;
            // the tiles' turns, tile 1 first
            if (two && (X == 0 || i > 0)) ok = wait_phase(&t.turn[X], (uint32_t)((i - 1) & 1), abort_flag, err) && ok;
            ok = wait_phase(&t.p_full[X][0], (uint32_t)((i - from) & 1), abort_flag, err) && ok;
            tc_after();
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
                mma_ts(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), i > from || k > 0, lead);
            ok = wait_phase(&t.p_full[X][1], (uint32_t)((i - from) & 1), abort_flag, err) && ok;
            tc_after();
#pragma unroll
            for (int k = kTile / 32; k < kTile / 16; ++k) mma_ts(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), 1, lead);
            // writes over the P that the product above reads: one thread's MMAs run in the order of issue
            if (more)
                issue_s(kd, two);  // its commit covers the product above too
            else
                mma_commit(saddr(&t.o_done[X]), lead);
            if (!more && two && lead) mbar_arrive(&t.turn[1 - X]);
            mma_commit(saddr(&t.empty[sv]), lead);
            if (more) mma_commit(saddr(&t.empty[sk]), lead);
            ok = __all_sync(0xffffffffu, ok);  // one answer for the warp's lanes
            sk += 2, sv += 2;
            if (sk >= kStages) sk -= kStages, pk ^= 1;
            if (sv >= kStages) sv -= kStages, pv ^= 1;
        }
    }
    mma_commit(saddr(&t.drained), lead);
    drain_phase(&t.drained, 0);
}

// ---- the kernel ------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const PromptArgs a) {
    using C = Cfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* const sq = smem;                     // [2][kBytes]
    uint8_t* const ring = smem + 2 * C::kBytes;   // [kStages][kBytes]
    typename C::Tail& t = *reinterpret_cast<typename C::Tail*>(smem + (2 + kStages) * C::kBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* const abort_flag = &t.abort_flag;

    // The block's rows.  Row tiles are numbered by their sequence's start: sequence s has the numbers from
    // cu[s] / 256 + s on, which leaves it at least ceil(length / 256) of them (some stay empty); long rows first.
    const int head = blockIdx.x % a.Hq, g = head / (a.Hq / a.Hkv);
    const int number = a.n_virtual - 1 - (int)(blockIdx.x / a.Hq);
    int lo = 0, hi = a.S;                         // the last sequence whose first number is not above
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) / kUnit + mid <= number) lo = mid; else hi = mid;
    }
    const int first = __ldg(a.cu + lo), len = min(__ldg(a.cu + lo + 1), a.T) - first;
    const int unit = number - (first / kUnit + lo);
    if (first < 0) {
        if (threadIdx.x == 0) atomicOr(a.err, (unsigned)KVSEL_DEV_BAD_LENGTH);
        return;
    }
    if (unit < 0 || (int64_t)unit * kUnit >= len) return;
    const int row0 = unit * kUnit;
    const bool two = row0 + kTile < len;          // the second tile has rows
    const int n = 2 * unit + (two ? 2 : 1);       // steps; step i takes key tile n - 1 - i
    const int skip0 = two ? 1 : 0;                // tile 0 starts at step skip0

    if (threadIdx.x == 0) {
        mbar_init(&t.q_full, 1);
        for (int i = 0; i < kStages; ++i) mbar_init(&t.full[i], 1), mbar_init(&t.empty[i], two ? 2 : 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t.s_full[i], 1);
            mbar_init(&t.p_full[i][0], 4);
            mbar_init(&t.p_full[i][1], 4);
            mbar_init(&t.o_done[i], 1);
            mbar_init(&t.v_ok[i], 1);
            mbar_init(&t.turn[i], 1);
        }
        mbar_init(&t.drained, 2);
        t.abort_flag = t.odd_v = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&t.tmem)), "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = t.tmem;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        if (warp == 0 && lane == 0) {
            // ---- loads ----
            mbar_expect_tx(&t.q_full, (two ? 2 : 1) * C::kBytes);
            for (int x = 0; x < (two ? 2 : 1); ++x)
                for (int b = 0; b < D / 64; ++b)
                    tma_load(&map_q, &t.q_full, sq + x * C::kBytes + b * C::kBlock, 64 * b, head, first + row0 + x * kTile);
            int done = 0;
            for (int pos = 0; pos < 2 * n; ++pos, ++done) {
                const bool is_v = pos == 2 * n - 1 || (pos > 0 && pos % 2 == 0);
                const int i = pos == 2 * n - 1 ? n - 1 : is_v ? pos / 2 - 1 : (pos + 1) / 2;
                const int st = pos % kStages;
                if (!wait_phase(&t.empty[st], (uint32_t)((pos / kStages) & 1) ^ 1u, abort_flag, a.err)) break;
                mbar_expect_tx(&t.full[st], C::kBytes);
                for (int b = 0; b < D / 64; ++b)
                    tma_load(is_v ? &map_v : &map_k, &t.full[st], ring + st * C::kBytes + b * C::kBlock, 64 * b, g,
                             first + (n - 1 - i) * kTile);
            }
            drain_phase(&t.q_full, 0);
            for (int pos = done > kStages ? done - kStages : 0; pos < done; ++pos)
                drain_phase(&t.full[pos % kStages], (uint32_t)((pos / kStages) & 1));
        } else if (warp == 1) {
            issue_tile<D, 0>(t, sq, ring, n, two, lane, abort_flag, a.err);
        } else if (warp == 2) {
            issue_tile<D, 1>(t, sq, ring, n, two, lane, abort_flag, a.err);
        } else if (warp == 3) {
            // ---- V tiles of the first two steps: NaN and infinities to zero ----
            for (int i = 0; i < 2 && i < n; ++i) {
                const int vp = at_v(i, n);
                if (!wait_phase(&t.full[vp % kStages], (uint32_t)((vp / kStages) & 1), abort_flag, a.err)) break;
                uint4* const tile = reinterpret_cast<uint4*>(ring + (vp % kStages) * C::kBytes);
                bool odd = false;
                #pragma unroll 4
                for (int e = lane; e < C::kBytes / 16; e += 32) {
                    uint4 w = tile[e];
                    uint32_t u[4] = {w.x, w.y, w.z, w.w}, hit = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) hit |= (u[k] & 0x7F807F80u) + 0x00800080u;
                    if (hit & 0x80008000u) {
                        odd = true;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((u[k] & 0x7F80u) == 0x7F80u) u[k] &= 0xFFFF0000u;
                            if ((u[k] & 0x7F800000u) == 0x7F800000u) u[k] &= 0x0000FFFFu;
                        }
                        tile[e] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
                if (odd) t.odd_v = 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.v_ok[i]);
            }
        }
        __syncwarp();
        tc_before();
        __syncthreads();
        tc_after();
        if (warp == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ---- softmax: one row per thread ----
    const int x = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = kTmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t ts = lane_base + kColS + x * kTile, to = lane_base + kColO + x * D;
    const int from = x == 0 ? skip0 : 0;
    const int steps = x == 1 && !two ? 0 : n - from;
    const float sc = a.scale2;
    float ref = 0.f;
    float2 sum = make_float2(0.f, 0.f);
    bool ok = true;
    for (int k = 0; k < steps; ++k) {
        if (!(ok = wait_warp(&t.s_full[x], (uint32_t)(k & 1), abort_flag, a.err))) break;
        tc_after();
        uint32_t s[kTile];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s + 32 * i);
        tmem_wait_ld();
        if (k == 0) {  // the diagonal: key c of the tile is seen by rows r >= c
#pragma unroll
            for (int c = 0; c < kTile; ++c)
                if (c > r) s[c] = 0xFF800000u;
        }
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = __uint_as_float(s[i]);
#pragma unroll
        for (int c = 4; c + 8 <= kTile; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = max3(m[i], __uint_as_float(s[c + i]), __uint_as_float(s[c + 4 + i]));
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], __uint_as_float(s[kTile - 4 + i]));
        const float top = fmaxf(max3(m[0], m[1], m[2]), m[3]) * sc;
        if (k == 0) {
            ref = top == -INFINITY ? 0.f : top;
        } else if (__any_sync(0xffffffffu, top > ref + kSlack)) {
            // references move up: the sums so far and O shrink with them
            const float next = fmaxf(ref, top), f = ex2(ref - next);
            ref = next;
            sum.x *= f, sum.y *= f;
            // (the commit that brought this S came after the last step's product: O is at rest)
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                uint32_t o[32];
                tmem_ld32(to + 32 * b, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(to + 32 * b, o);
            }
        }
        const float2 sc2 = make_float2(sc, sc), nr = make_float2(-ref, -ref);
        // in two halves, so that the product with V starts on the first while the second is worked out
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t p[kTile / 4];
#pragma unroll
            for (int c = 0; c < kTile / 4; ++c) {
                const int e0 = half * (kTile / 2) + 2 * c;
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[e0]), __uint_as_float(s[e0 + 1])), sc2, nr);
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                sum = __fadd2_rn(sum, e);
                p[c] = pack_bf16(e.x, e.y);
            }
            tmem_st32(ts + 32 * half, p);
            tmem_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.p_full[x][half]);
        }
    }
    // ---- output ----
    if (ok && steps > 0) ok = wait_warp(&t.o_done[x], 0, abort_flag, a.err);
    if (ok && steps > 0) {
        tc_after();
        bool odd = false;
        for (int i = 0; i < 2 && i < n && ok; ++i) ok = wait_warp(&t.v_ok[i], 0, abort_flag, a.err);
        odd = *(volatile int*)&t.odd_v != 0;
        const int row = row0 + x * kTile + r;
        const float l = sum.x + sum.y, inv = 1.f / l;
        const int64_t at = (int64_t)(first + row) * a.Hq + head;
        const int key0 = n > 1 ? (n - 2) * kTile : 0;   // first key of the tiles that were looked over
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            uint32_t o[32];
            tmem_ld32(to + 32 * b, o);
            tmem_wait_ld();
            if (row >= len) continue;
            if (odd) {
                for (int j = key0; j <= row; ++j) {
                    const __nv_bfloat16* v = a.v + (int64_t)(first + j) * a.v_stride + (int64_t)g * D + 32 * b;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float w = __bfloat162float(v[i]);
                        if (!(fabsf(w) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + w);
                    }
                }
            }
            uint4* const dst = reinterpret_cast<uint4*>(a.out + at * D + 32 * b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
                dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (a.lse && row < len) a.lse[at] = (ref + log2f(l)) * kLn2;
    }
    tc_before();
    __syncthreads();
}

// bf16 rows [T][H][D], tokens `stride` elements apart: boxes of 64 dims of one head, 128 tokens, zero fill.
bool make_map(CUtensorMap* map, const void* base, int T, int H, int D, int64_t stride) {
    auto fn = kvsel_tmap_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kTile};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptArgs& a, cudaStream_t s) {
    auto* kernel = prompt_attention_kernel<D>;
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split counts on it
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)a.n_virtual * a.Hq, kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

extern "C" int kvsel_prompt_attention(kvsel_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens, int S, int T, int Hq,
                                      int Hkv, int D, float scale, void* out, float* lse, void* stream) {
    const kvsel_trace trace_("kvsel_prompt_attention");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (S < 0 || T < 0 || Hq <= 0 || Hkv <= 0) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "prompt_attention: bad sizes");
    if (Hq % Hkv) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "prompt_attention: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
    if (D != 64 && D != 128) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "prompt_attention: D=%d unsupported", D);
    if (S > 65535 || Hq > 65535 || T > (1 << 24))
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "prompt_attention: S, T or Hq too large");
    if (!(scale > 0.f) || scale > 1e30f)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "prompt_attention: scale must be positive and finite");
    if (S == 0 || T == 0) return KVSEL_OK;
    if (!q || !k || !v || !cu_seqlens || !out) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "prompt_attention: null pointer");
    if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "prompt_attention: token stride smaller than a token's heads");
    auto off16 = [](const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15u) || (stride * 2) % 16; };
    if (off16(q, q_stride) || off16(k, k_stride) || off16(v, v_stride) || off16(out, 0))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "prompt_attention: q, k, v, out and the strides must be 16-byte aligned");
    const int n_virtual = T / kUnit + S;
    if ((int64_t)n_virtual * Hq > INT_MAX) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "prompt_attention: too many rows");
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, q, T, Hq, D, q_stride) || !make_map(&mk, k, T, Hkv, D, k_stride) || !make_map(&mv, v, T, Hkv, D, v_stride))
        return kvsel_fail(ctx, KVSEL_ERR_CUDA, "prompt_attention: tensor map encoding failed");
    const PromptArgs a{(const __nv_bfloat16*)v, v_stride, cu_seqlens, S, T, Hq, Hkv, n_virtual, scale * kLog2e,
                       (__nv_bfloat16*)out, lse, ctx->dev_err};
    const cudaError_t e = D == 64 ? launch<64>(mq, mk, mv, a, (cudaStream_t)stream) : launch<128>(mq, mk, mv, a, (cudaStream_t)stream);
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "prompt_attention launch");
}
