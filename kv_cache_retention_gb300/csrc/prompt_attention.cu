// kvsel_prompt_attention: causal attention over packed prompts with grouped heads,
// on the 5th-generation tensor cores.
//
// Sequence s holds tokens [cu[s], cu[s+1]); row i of it sees its rows 0..i:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale log2e q_i . k_j - ref),
//   lse = ln sum_j e^(scale q_i . k_j).
//
// A unit of work is one query head and 256 consecutive rows of one sequence, as two tiles
// of 128 rows (TMEM lanes; 128 rows and one tile where there are few units), and goes once over the keys from the diagonal down, 128 at
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
// operands of the product have one type and V's range is bf16's; its relative rounding,
// 2^-8 at most per weight, is random and comes to about the output's own rounding.
//
// 384 threads: warp 0 loads (TMA), warps 1 and 2 issue the MMAs of one tile each, warp 3
// hands out the units and looks over the V tiles of the diagonal (below), warps 4-7 and
// 8-11 are the softmax of the two tiles, a row per thread.  TMEM: S of tile 0 and 1 at columns 0 and 128, O at 256 and 384.
//
// Masked places.  A weight of zero does not hide a NaN or an infinity in V.  Key tiles
// below the diagonal are seen by every row of a tile, so only the first two tiles of a
// block's pass hold values that some rows must not see; there warp 3 sets such values
// to zero in shared memory before the product, and if there were any, each row adds
// those it does see to its output at the end (what the sum would be: infinite or NaN).
// Warp 3 runs up to a unit ahead of the ring, whose barriers' parities would tell it
// nothing there: the V tiles that it looks over land on barriers of their own (v_raw),
// and its arrival completes their ring stages.
//
// Blocks are as many as there are units, the last sequence's first and of a sequence the
// longest first, but one per SM runs: when its
// unit is done it claims the unit of a block that has not been launched yet (cluster
// launch control), and the next unit's loads and first products run beside the end of the
// last.  With a block per unit the 9 prompts below took 398 us, 16384 tokens 1.78 ms.
//
// What bounds it: the tensor cores within a unit (128 keys for both tiles take 1.5 us, 91%
// of the rate of a large library product; both operands of S come from shared memory, at
// its bandwidth's limit), and some 5 us a unit in which they wait: the first softmax, the
// last product, the output.  Measured for D = 128: 16384 tokens of 40 / 8 heads 1.66 to 1.74
// ms (1.6 PFLOP/s counting what the mask leaves, 85% of that rate), 4096 of 32 / 8 heads 117
// us (63%), 9 prompts of 14700 tokens together 328 us (61%).
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
    int unit;               // rows of a unit: two tiles, or one
    float scale2;           // scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
    uint64_t wait_ns;       // how long a wait goes on
    int stuck;              // tile 0's issuer waits for what never comes (test entry)
};

// A block's waits: whether one has given up, and how long each goes on.
struct Stop {
    volatile int given_up;
    uint64_t limit_ns;
};

template <int D>
struct Cfg {
    static constexpr int kBlock = kTile * 128;             // 128 rows x 64 dims, 128-byte swizzled
    static constexpr int kBytes = D / 64 * kBlock;         // one tile of Q, K or V
    static constexpr int kStages = 4;                      // K and V tiles share the ring
    static constexpr int kOut = 8 * 32 * 128;              // 32 rows of 64 dims for each softmax warp, on their way out
    // A unit of work, as warp 3 hands it out; n == 0: there are no more.
    struct Unit {
        int first, len, row0, head, n, two;  // two: it has rows in its second tile
    };
    struct Tail {
        uint4 claimed;  // the answer of a claim
        uint64_t q_full, q_empty, full[kStages], empty[kStages], s_full[2], p_full[2][2], o_done[2], o_free[2], v_raw[2],
            v_ok[2][2], turn[2], unit_full[2], unit_empty[2], claim, drained;
        Stop stop;
        uint64_t never;         // nothing completes it
        uint32_t tmem;
        int odd_v[2];
        Unit unit[2];
    };
    static constexpr size_t kSmem = (size_t)(2 + kStages) * kBytes + kOut + sizeof(Tail) + 1024;
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
// One copy of the code for both, and one of each run of MMAs: with a copy per tile the kernel's loops passed the
// instruction cache (16384 tokens: 1.92 ms, with one copy 1.73 ms).
template <int D>
__device__ __forceinline__ void issue_tiles(typename Cfg<D>::Tail& t, const uint8_t* sq, const uint8_t* ring, int tile, int lane,
                                            bool stuck, Stop* stop, unsigned* err) {
    using C = Cfg<D>;
    constexpr uint32_t kStages = C::kStages;
    const uint32_t lead = lane == 0, X = uniform(tile);
    const uint32_t q = uniform(desc_low(saddr(sq) + X * C::kBytes, 16));
    const uint32_t ts = uniform(kTmem + kColS + X * kTile), to = uniform(kTmem + kColO + X * D);
    auto desc = [&](uint32_t st, uint32_t leading) { return uniform(desc_low(saddr(ring) + st * C::kBytes, leading)); };
    uint32_t base = 0, steps = 0, turns = 0, mine = 0;  // ring places and this tile's steps, turns and units so far
    bool ok = !stuck || wait_warp(&t.never, 0, stop, err);
    for (uint32_t u = 0; ok; ++u) {
        if (!(ok = wait_warp(&t.unit_full[u & 1], (u >> 1) & 1, stop, err))) break;
        const int n = t.unit[u & 1].n;
        const bool two = t.unit[u & 1].two;
        __syncwarp();
        if (lead) mbar_arrive(&t.unit_empty[u & 1]);
        if (n == 0) break;
        if (X == 1 && !two) {
            // no rows for this tile: it sees and releases the unit's loads all the same, since a wait of the next unit
            // would take a phase two before its own for its own
            ok = wait_warp(&t.q_full, u & 1, stop, err);
            if (ok && lead) mbar_arrive(&t.q_empty);
            for (const uint32_t end = base + 2 * n; ok && base < end; ++base) {
                ok = wait_warp(&t.full[base % kStages], base / kStages & 1, stop, err);
                if (ok && lead) mbar_arrive(&t.empty[base % kStages]);
            }
            continue;
        }
        const int from = X == 0 && two ? 1 : 0;       // the tile's first step
        auto release = [&](uint64_t* b) { mma_commit(saddr(b), lead); };
        ok = wait_phase(&t.q_full, u & 1, stop, err);
        // Round i: O += P V of step i (not in the first round, i = from - 1), then S of step i + 1 (not in the last).
        // Stages and phases of its tiles, K(i + 1) and V(i):
        uint32_t at = base + at_k(from);
        uint32_t sk = at % kStages, pk = at / kStages & 1, sv = 0, pv = 0;
        for (int i = from - 1; i < n && ok; ++i) {
            const bool more = i + 1 < n, first = i < from;
            if (first || i == from || !more) {        // the places' step is 2 in between
                at = base + at_v(max(i, 0), n), sv = at % kStages, pv = at / kStages & 1;
                at = base + at_k(i + 1), sk = at % kStages, pk = at / kStages & 1;
            }
            const uint32_t kd = desc(sk, 16), vd = desc(sv, C::kBlock);
            if (more) ok = wait_phase(&t.full[sk], pk, stop, err) && ok;
            if (!first) {
                ok = wait_phase(&t.full[sv], pv, stop, err) && ok;
                if (i == from && mine) ok = wait_phase(&t.o_free[X], (mine - 1) & 1, stop, err) && ok;
                // the tiles' turns, tile 1 first
                if (two && (X == 0 || i > 0)) ok = wait_phase(&t.turn[X], turns++ & 1, stop, err) && ok;
                ok = wait_phase(&t.p_full[X][0], steps & 1, stop, err) && ok;
                tc_after();
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                    mma_ts(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), i > from || k > 0, lead);
                ok = wait_phase(&t.p_full[X][1], steps & 1, stop, err) && ok;
                tc_after();
#pragma unroll
                for (int k = kTile / 32; k < kTile / 16; ++k)
                    mma_ts(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), 1, lead);
                ++steps;
            } else {
                tc_after();
            }
            if (more) {
                const bool pass = two && !first && lead;
                // writes over the P that the product above reads: one thread's MMAs run in the order of issue
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * C::kBlock + (k & 3) * 32) >> 4;
                    // the other tile's turn: its issuer is under way while the last of these are issued
                    if (k == D / 32 && pass) mbar_arrive(&t.turn[X ^ 1]);
                    mma_ss(ts, q + off, kd + off, idesc(kTile, false), k > 0, lead);
                }
                mma_commit(saddr(&t.s_full[X]), lead);  // covers the product above too
                if (i + 2 == n) release(&t.q_empty);
                release(&t.empty[sk]);
            } else {
                if (X == 0 && two && lead) mbar_arrive(&t.turn[1]);
                mma_commit(saddr(&t.o_done[X]), lead);
            }
            if (!first) {
                release(&t.empty[sv]);
            } else if (from == 1) {                   // the first K and V tile are the other tile's alone
                for (int k = 0; k < 2; ++k) {
                    at = base + (k ? at_v(0, n) : 0);
                    const uint32_t st = at % kStages;
                    ok = wait_phase(&t.full[st], at / kStages & 1, stop, err) && ok;
                    if (lead) mbar_arrive(&t.empty[st]);
                }
            }
            ok = __all_sync(0xffffffffu, ok);  // one answer for the warp's lanes
            sk += 2, sv += 2;
            if (sk >= kStages) sk -= kStages, pk ^= 1;
            if (sv >= kStages) sv -= kStages, pv ^= 1;
        }
        base += 2 * n;
        ++mine;
    }
    mma_commit(saddr(&t.drained), lead);
    drain_phase(&t.drained, 0);
}

// ---- units of work ---------------------------------------------------------
// Block b's unit: query head b % Hq and a row tile of a.unit rows of one sequence.  Row tiles are numbered by their
// sequence's start: sequence s has the numbers from cu[s] / a.unit + s on, which leaves it at least ceil(length / a.unit)
// of them (some stay empty); the last numbers come first, a sequence's longest rows before its others.  n = 0: no rows.
template <int D>
__device__ __forceinline__ typename Cfg<D>::Unit unit_of(const PromptArgs& a, uint32_t block, int lane) {
    const int number = a.n_virtual - 1 - (int)(block / a.Hq);
    int lo = 0, size = a.S;                       // the last sequence whose first number is not above lies in [lo, lo + size)
    while (size > 1) {
        const int piece = (size + 31) / 32, i = lane * piece;
        const bool below = i < size && (lane == 0 || __ldg(a.cu + lo + i) / a.unit + lo + i <= number);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
        lo += last * piece;
        size = min(piece, size - last * piece);
    }
    typename Cfg<D>::Unit w;
    const int stop = __ldg(a.cu + lo + 1);
    w.first = __ldg(a.cu + lo);
    w.len = w.first < 0 || stop < w.first ? 0 : min(stop, a.T) - w.first;
    const int tile = number - (w.first / a.unit + lo);
    const bool rows = tile >= 0 && (int64_t)tile * a.unit < w.len;
    w.row0 = rows ? tile * a.unit : 0;
    w.head = (int)(block % a.Hq);
    w.two = a.unit > kTile && w.row0 + kTile < w.len;
    w.n = rows ? w.row0 / kTile + 1 + w.two : 0;
    return w;
}

// Asks for a block of the grid that has not been launched; the answer lands in t.claimed.
template <class Tail>
__device__ __forceinline__ void claim_start(Tail& t) {
    mbar_expect_tx(&t.claim, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     saddr(&t.claimed)),
                 "r"(saddr(&t.claim))
                 : "memory");
}
// The claim's answer: whether there was a block, and which.
template <class Tail>
__device__ __forceinline__ bool claim_next(Tail& t, uint32_t& claims, uint32_t& block, int lane, bool start,
                                           Stop* stop, unsigned* err) {
    if (start && lane == 0) claim_start(t);
    const bool ok = wait_warp(&t.claim, claims++ & 1, stop, err);
    if (!ok) drain_phase(&t.claim, (claims - 1) & 1);
    uint32_t got, id;
    asm volatile(
        "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%2];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}\n"
        : "=r"(got), "=r"(id)
        : "r"(saddr(&t.claimed))
        : "memory");
    __syncwarp();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read before the next answer is written
    block = id;
    return ok && got;
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
    typename C::Tail& t = *reinterpret_cast<typename C::Tail*>(smem + (2 + kStages) * C::kBytes + C::kOut);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Stop* const stop = &t.stop;

    if (threadIdx.x == 0) {
        mbar_init(&t.q_full, 1);
        mbar_init(&t.q_empty, 2);
        mbar_init(&t.claim, 1);
        for (int i = 0; i < kStages; ++i) mbar_init(&t.full[i], 1), mbar_init(&t.empty[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t.s_full[i], 1);
            mbar_init(&t.p_full[i][0], 4);
            mbar_init(&t.p_full[i][1], 4);
            mbar_init(&t.o_done[i], 1);
            mbar_init(&t.o_free[i], 4);
            mbar_init(&t.v_raw[i], 1);
            mbar_init(&t.v_ok[i][0], 1);
            mbar_init(&t.v_ok[i][1], 1);
            mbar_init(&t.turn[i], 1);
            mbar_init(&t.unit_full[i], 1);
            mbar_init(&t.unit_empty[i], 1 + 2 + 8);  // the loads, the issuers, the softmax warps
        }
        mbar_init(&t.drained, 2);
        mbar_init(&t.never, 1);
        t.stop.given_up = 0;
        t.stop.limit_ns = a.wait_ns;
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
            uint32_t c = 0, loaded_q = 0;  // ring places filled, Q loads
            uint32_t raw = 0, looked_any = 0, looked_phase = 0;  // stages whose last load was on v_raw; v_raw used; its next phases: a bit each
            bool ok = true;
            for (uint32_t u = 0; ok; ++u) {
                if (!(ok = wait_phase(&t.unit_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
                const typename C::Unit w = t.unit[u & 1];
                mbar_arrive(&t.unit_empty[u & 1]);
                if (w.n == 0) break;
                const int g = w.head / (a.Hq / a.Hkv), tiles = 1 + w.two;
                if (u && !(ok = wait_phase(&t.q_empty, (u - 1) & 1, stop, a.err))) break;
                mbar_expect_tx(&t.q_full, tiles * C::kBytes);
                for (int x = 0; x < tiles; ++x)
                    for (int b = 0; b < D / 64; ++b)
                        tma_load(&map_q, &t.q_full, sq + x * C::kBytes + b * C::kBlock, 64 * b, w.head, w.first + w.row0 + x * kTile);
                ++loaded_q;
                for (int pos = 0; pos < 2 * w.n; ++pos, ++c) {
                    const bool is_v = pos == 2 * w.n - 1 || (pos > 0 && pos % 2 == 0);
                    const int i = pos == 2 * w.n - 1 ? w.n - 1 : is_v ? pos / 2 - 1 : (pos + 1) / 2;
                    const uint32_t st = c % kStages;
                    if (!(ok = wait_phase(&t.empty[st], (c / kStages & 1) ^ 1u, stop, a.err))) break;
                    const bool looked = is_v && i < 2;
                    uint64_t* const bar = looked ? &t.v_raw[i] : &t.full[st];
                    mbar_expect_tx(bar, C::kBytes);
                    for (int b = 0; b < D / 64; ++b)
                        tma_load(is_v ? &map_v : &map_k, bar, ring + st * C::kBytes + b * C::kBlock, 64 * b, g,
                                 w.first + (w.n - 1 - i) * kTile);
                    raw = (raw & ~(1u << st)) | (uint32_t)looked << st;
                    if (looked) looked_any |= 1u << i, looked_phase ^= 1u << i;
                }
            }
            if (loaded_q) drain_phase(&t.q_full, (loaded_q - 1) & 1);
            for (int i = 0; i < 2; ++i)
                if (looked_any >> i & 1) drain_phase(&t.v_raw[i], (looked_phase >> i & 1) ^ 1);
            for (uint32_t pos = c > kStages ? c - kStages : 0; pos < c; ++pos)
                if (!(raw >> (pos % kStages) & 1)) drain_phase(&t.full[pos % kStages], pos / kStages & 1);
        } else if (warp == 1 || warp == 2) {
            issue_tiles<D>(t, sq, ring, warp - 1, lane, a.stuck && warp == 1, stop, a.err);
        } else if (warp == 3) {
            // ---- units of work, and the V tiles of each unit's first two steps ----
            // The block starts with its own unit and then claims those of blocks that have not been launched yet, in
            // the order of launch, until none is left.
            uint32_t block = blockIdx.x, base = 0, claims = 0, looked_phase = 0;  // looked_phase: v_raw's next phases, a bit each
            bool ok = true, any = true, look = false;
            for (uint32_t u = 0; ok; ++u) {
                typename C::Unit w;
                w.n = 0;
                while (any) {
                    look |= block == 0;
                    w = unit_of<D>(a, block, lane);
                    if (w.n) break;
                    any = claim_next(t, claims, block, lane, true, stop, a.err);
                }
                if (u >= 2 && !(ok = wait_warp(&t.unit_empty[u & 1], ((u >> 1) - 1) & 1, stop, a.err))) break;
                if (lane == 0) {
                    t.unit[u & 1] = w;
                    t.odd_v[u & 1] = 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.unit_full[u & 1]);
                if (look) {  // with the first block's unit: do the sequences lie in [0, T], one behind the other?
                    look = false;
                    for (int s = lane; s < a.S; s += 32) {
                        const int start = __ldg(a.cu + s), stop = __ldg(a.cu + s + 1);
                        if (start < 0 || stop < start || stop > a.T) atomicOr(a.err, (unsigned)KVSEL_DEV_BAD_LENGTH);
                    }
                    __syncwarp();
                }
                if (w.n == 0) break;
                if (lane == 0) claim_start(t);
                for (int i = 0; i < 2 && ok; ++i) {  // NaN and infinities to zero
                    if (i < w.n) {
                        const uint32_t at = base + at_v(i, w.n), st = at % kStages;
                        if (!(ok = wait_warp(&t.v_raw[i], looked_phase >> i & 1, stop, a.err))) break;
                        looked_phase ^= 1u << i;
                        uint4* const tile = reinterpret_cast<uint4*>(ring + st * C::kBytes);
                        bool odd = false;
#pragma unroll 4
                        for (int e = lane; e < C::kBytes / 16; e += 32) {
                            const uint4 v = tile[e];
                            uint32_t x[4] = {v.x, v.y, v.z, v.w}, hit = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) hit |= (x[k] & 0x7F807F80u) + 0x00800080u;
                            if (hit & 0x80008000u) {
                                odd = true;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if ((x[k] & 0x7F80u) == 0x7F80u) x[k] &= 0xFFFF0000u;
                                    if ((x[k] & 0x7F800000u) == 0x7F800000u) x[k] &= 0x0000FFFFu;
                                }
                                tile[e] = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                        }
                        if (odd) t.odd_v[u & 1] = 1;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&t.full[st]);
                    }
                    if (lane == 0) mbar_arrive(&t.v_ok[u & 1][i]);
                }
                any = claim_next(t, claims, block, lane, false, stop, a.err);
                base += 2 * w.n;
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
    const float sc = a.scale2;
    uint32_t done = 0, mine = 0;                      // this tile's steps and units so far
    bool ok = true;
    for (uint32_t u = 0; ok; ++u) {
    if (!(ok = wait_warp(&t.unit_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
    const typename C::Unit w = t.unit[u & 1];
    __syncwarp();
    const bool two = w.two;
    const int steps = w.n == 0 || (x == 1 && !two) ? 0 : x == 0 && two ? w.n - 1 : w.n;
    float ref = 0.f;
    float2 sum = make_float2(0.f, 0.f);
    for (int k = 0; k < steps; ++k, ++done) {
        if (!(ok = wait_warp(&t.s_full[x], done & 1, stop, a.err))) break;
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
            ref = fmaxf(top, -3e38f);  // of a row whose logits here are all -inf: low, and finite
        } else if (__any_sync(0xffffffffu, top > ref + kSlack)) {
            // references move up: the sums so far and O shrink with them
            const float next = fmaxf(ref, top), f = ex2(ref - next);
            ref = next;
            sum.x *= f, sum.y *= f;
            // (the commit that brought this S came after the last step's product: O is at rest)
#pragma unroll 1
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
    if (ok && steps > 0) ok = wait_warp(&t.o_done[x], mine++ & 1, stop, a.err);
    if (ok && steps > 0) {
        tc_after();
        for (int i = 0; i < 2 && ok; ++i) ok = wait_warp(&t.v_ok[u & 1][i], (u >> 1) & 1, stop, a.err);
        const bool odd = *(volatile int*)&t.odd_v[u & 1] != 0;
        const int row = w.row0 + x * kTile + r;
        const float l = sum.x + sum.y, inv = 1.f / l;
        const int64_t at = (int64_t)(w.first + row) * a.Hq + w.head;
        // through shared memory, so that a store covers 128 bytes of each of four rows (a row per lane took 3 us a
        // unit); 16-byte pieces are swizzled by their row against bank conflicts
        uint8_t* const stage = smem + (2 + kStages) * C::kBytes + (warp - 4) * (32 * 128);
        uint32_t all[D];                  // all at once, so that the next unit's products may start on O (4 us of 317 for 9 prompts)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) tmem_ld32(to + 32 * i, all + 32 * i);
        tmem_wait_ld();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&t.o_free[x]);
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
            const uint32_t* const o = all + 64 * b;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    e[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                *reinterpret_cast<uint4*>(stage + lane * 128 + (i ^ (lane & 7)) * 16) = make_uint4(e[0], e[1], e[2], e[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rr = 4 * i + (lane >> 3), out_row = w.row0 + x * kTile + quarter * 32 + rr;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((lane & 7) ^ (rr & 7)) * 16);
                if (out_row < w.len)
                    *reinterpret_cast<uint4*>(a.out + ((int64_t)(w.first + out_row) * a.Hq + w.head) * D + 64 * b + 8 * (lane & 7)) = v;
            }
            __syncwarp();
        }
        if (a.lse && row < w.len) a.lse[at] = (ref + log2f(l)) * kLn2;
        if (odd && row < w.len) {
            // what the row sees of the values that were set to zero: a sum of infinities and NaN
            const int key0 = w.n > 1 ? (w.n - 2) * kTile : 0;  // first key of the tiles that were looked over
            const __nv_bfloat16* v = a.v + (int64_t)(w.first + key0) * a.v_stride + (int64_t)(w.head / (a.Hq / a.Hkv)) * D;
#pragma unroll 1
            for (int d = 0; d < D; ++d) {
                float add = 0.f;
#pragma unroll 1
                for (int j = 0; j <= row - key0; ++j) {
                    const float e = __bfloat162float(v[j * a.v_stride + d]);
                    if (!(fabsf(e) < INFINITY)) add += e;
                }
                if (!(add == 0.f)) a.out[at * D + d] = __float2bfloat16_rn(__bfloat162float(a.out[at * D + d]) + add);
            }
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&t.unit_empty[u & 1]);  // only now: the unit's odd_v has been read
    if (w.n == 0) break;
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
cudaError_t launch(kvsel_ctx* ctx, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptArgs& a,
                   cudaStream_t s) {
    auto* kernel = prompt_attention_kernel<D>;
    constexpr unsigned kBit = 1u << (D / 64);
    if (!(ctx->ready & kBit)) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split counts on it
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        ctx->ready |= kBit;
    }
    kernel<<<(unsigned)a.n_virtual * a.Hq, kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

int attention_call(kvsel_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                   int64_t v_stride, const int32_t* cu_seqlens, int S, int T, int Hq, int Hkv, int D, float scale, void* out,
                   float* lse, void* stream, uint64_t wait_ns, int stuck) {
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
    // Units of one tile where the SMs would not run out of those: nothing is shared, and a step is shorter with no other
    // tile's between (4096 tokens of 4 heads, D 128: 50 us and 54 with two tiles; of 8 heads, 136 units of two tiles, 67 and
    // 54).
    const int unit = (int64_t)(T / (2 * kTile) + S) * Hq <= ctx->num_sms / 2 ? kTile : 2 * kTile;
    const int n_virtual = T / unit + S;
    if ((int64_t)n_virtual * Hq > INT_MAX) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "prompt_attention: too many rows");
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, q, T, Hq, D, q_stride) || !make_map(&mk, k, T, Hkv, D, k_stride) || !make_map(&mv, v, T, Hkv, D, v_stride))
        return kvsel_fail(ctx, KVSEL_ERR_CUDA, "prompt_attention: tensor map encoding failed");
    const PromptArgs a{(const __nv_bfloat16*)v, v_stride, cu_seqlens, S, T, Hq, Hkv, n_virtual, unit, scale * kLog2e,
                       (__nv_bfloat16*)out, lse, ctx->dev_err, wait_ns, stuck};
    const cudaError_t e = D == 64 ? launch<64>(ctx, mq, mk, mv, a, (cudaStream_t)stream) : launch<128>(ctx, mq, mk, mv, a, (cudaStream_t)stream);
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "prompt_attention launch");
}

}  // namespace

extern "C" int kvsel_prompt_attention(kvsel_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens, int S, int T, int Hq,
                                      int Hkv, int D, float scale, void* out, float* lse, void* stream) {
    const kvsel_trace trace_("kvsel_prompt_attention");
    return attention_call(ctx, q, k, v, q_stride, k_stride, v_stride, cu_seqlens, S, T, Hq, Hkv, D, scale, out, lse, stream,
                          kWaitNs, 0);
}

// Test entry (not part of the public header): kvsel_prompt_attention in which the issuer of tile 0 of every block waits on
// a barrier that nothing completes, with every wait limited to wait_ns.  It gives up while copies and the other issuer's
// MMAs are in flight; out and lse hold no meaningful values afterwards.
extern "C" int kvsel_test_prompt_attention_give_up(kvsel_ctx* ctx, const void* q, const void* k, const void* v,
                                                   int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                                   const int32_t* cu_seqlens, int S, int T, int Hq, int Hkv, int D,
                                                   float scale, void* out, float* lse, uint64_t wait_ns, void* stream) {
    const kvsel_trace trace_("kvsel_test_prompt_attention_give_up");
    if (wait_ns == 0 || wait_ns > kWaitNs)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "test_prompt_attention_give_up: wait_ns must be in (0, 1 s]");
    return attention_call(ctx, q, k, v, q_stride, k_stride, v_stride, cu_seqlens, S, T, Hq, Hkv, D, scale, out, lse, stream,
                          wait_ns, 1);
}
