// kvsel_kv4_attention: attention of a few query rows per session over the 4-bit
// paged cache.
//
// Row (s, t, h) sits at position pos = len_s - Tq + t of session s and sees the
// tokens j <= pos whose slot is live:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale log2e (q . k_j - max)),
//   lse = ln sum_j e^(scale q . k_j).
// A warp takes 32 live tokens at a time and up to 8 * NT rows of one kv head:
//   S^T [tokens][rows] = K q^T   mma.sync m16n8k16 (fp16, fp32 sums), K the A operand
//   O^T [dims][rows]  += V^T p^T  likewise, V^T the A operand, p through movmatrix
// so the small side, the rows, is the one that is padded (to 8), and both products
// read K and V as they lie in memory: which dims and tokens a lane's fragment
// positions stand for is free, so a lane takes 16 contiguous bytes of a K row (the
// query fragments are laid out to match) and D/16 contiguous bytes of each of four V
// rows.  Codes become fp16 by the hardware conversion of E2M1 pairs and one exact
// multiplication by the scale; V's pairs, which run along tokens, are first put
// together from two rows' nibbles by bit selects.  mma.sync and not tcgen05: the
// kernel is bound by memory and by the conversions, and both products find their
// operands in registers.
//
// The query rows are scaled by a power of two each to a largest value in [2^14, 2^15),
// which fp16 holds exactly but for values below 2^-31 of it (those are off by up to
// 2^-39 of it).  The softmax runs over
// the tokens once: per row a reference m within 5 (log2) of the running maximum or
// above, weights 2^(x - m + 10), so that fp16 holds weights down to 2^-24 of the
// largest with full precision.  Sums and outputs are fp32, moved when the reference
// moves.
//
// Tokens come to a warp through cp.async into a ring of two or three buffers of its own, so
// the loop has no block barrier.  Slots are read 32 at a time; live ones queue up, so
// dropped tokens (most of a pruned session's slot map) cost a slot read and no more.
// Where 32 slots are two runs of 16 rows, four pairs of bulk copies bring them instead.
//
// What bounds it: the latency of dependent instructions, before memory.  For D = 128 a
// warp executes about 850 for 32 tokens of one kv head, 4.6 KB, of which 270 are the
// conversions and the scales' multiplications and 33 the products; a scheduler has four
// warps to choose from (three with two row tiles) and issues on 61% (51%) of its active
// cycles.  Measured: 36 sessions of 32 / 8 heads pruned to a quarter, 278 MB: 80 us (3.5
// TB/s), of which the instructions would fill 43; 16 sessions of 4 query rows, 306 MB:
// 98 us (3.1 TB/s) and 46; one of 92160 tokens, 106 MB: 35 us, of which some 6 us go by
// before the first tokens arrive and 5 us with the join; one of 2048 tokens, 9.5 us.  More warps per SM (10 a block, 96 registers) took 104, 115 and 40 us for
// the first three when these took 85, 117 and 36.
//
// One wave of two blocks per SM.  The work is the chunks of 32 positions of every
// session, laid end to end with some for the start of each; it is cut into equal,
// contiguous shares, found from the lengths on the device, so that sessions of uneven length keep every SM busy to the end
// (with blocks for a fixed part of a session, 16 uneven sessions took 146 us, 92160
// tokens of one 38 us).  A share is a few pieces of sessions, and neighbouring blocks
// take it for one kv head (and row tile) each: the heads' rows of a page lie side by
// side, and reading them at about the same time is what DRAM's pages want (laid end to
// end over the heads as well, the 16 sessions took 169 us).
// The block's warps take every kWarps-th chunk of a piece and join through shared
// memory; a unit that several blocks share is joined from their partial results by a
// second, small kernel, in the order of the blocks, launched as a dependent of the first
// so that its start costs little.  (Joined by the last block to arrive instead, the join
// took 4 to 10 us at the end of that block, and its registers came out of the loop's.)
// Where the maps reach some hundred positions only, sharing is not worth
// it: blocks take whole units, and there is nothing to join.
#include <cuda_bf16.h>
#include <limits.h>

#include <type_traits>

#include "kv4_format.cuh"
#include "kvsel_internal.h"

namespace {

constexpr int kTile = 32;   // tokens per stage
constexpr unsigned kBulk = 0x80u;
constexpr int kPartialFloats = 16 * (128 + 2) + 4;           // the largest partial result
// Positions up to which units are not shared: kWhole, or kWholeMany where there are kMany sessions.  A share's further
// pieces and the join then cost more than even shares save: one session of 32 / 8 heads, D 128, and 500 tokens took 8.7 us
// whole and 10.8 shared, of 1000 tokens 11.6 and 10.5; 8 of 1000 tokens 12.1 and 13.4; 64 of 1000 tokens 29 and 34, of 50 to
// 1000 tokens 26 and 28, of 50 to 2000 tokens 39 and 36.
constexpr int kWhole = 768, kWholeMany = 1024, kMany = 8;
// Chunks that the start of another session within a share counts as: its queries, first slots and tokens, and the join of
// the warps.  With 0, 16 sessions of 301 to 32768 tokens and 4 rows took 110 us and 8 of 300 to 8000 tokens 25 us; with 8,
// 105 and 21; with 20, 98 and 20; with 32, 99 and 21.
constexpr int kStart = 20;
constexpr int kLeast = 1;                                    // chunks per warp that a share has at least
constexpr float kUnset = 3e38f;  // ref of a row that has seen nothing
constexpr float kHead = 10.f;   // log2 of the weight at the reference
constexpr float kSlack = 5.f;   // how far (log2) a logit may pass the reference: weights stay below 2^15
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A unit (session, kv head, row tile) that several shares hold a part of: their partials are joined.
struct Shared {
    int sharers, session, late;   // late: the first sharer's partial is that of its last piece; sharers 0: no such unit
};

struct AttnArgs {
    const __nv_bfloat16* q;
    int64_t q_stride;
    int Tq, Hq, Hkv;
    const uint8_t *kc, *ks, *vc, *vs;
    int P, page, page_shift;  // page_shift: log2(page), or -1
    const int32_t* lens;
    const int32_t* map;       // slot map, or block table
    int n_slots;
    int ld;                   // row length of map
    int max_len;              // tokens that a row of it reaches
    int dead;
    int row_tiles;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
    int S;
    int whole;                // units are not shared
    uint64_t wait_ns;         // how long a wait for a bulk copy goes on
    int stuck;                // each block's first warp waits for what never comes (test entry)
    float* partials;          // two for each block: of its first piece and of its last, where others share their units
    struct Shared* shared;    // for each block, its shared unit that starts in its share
};

// D dims, NT tiles of 8 rows, W warps per block, MAP: tokens found through a slot map, not a block table
template <int D, int NT, int W, bool MAP>
struct Cfg {
    // Chunks of 32 slots read at a time.  Few of a pruned session's slots may be live (36 sessions, a quarter live: 82 us
    // with four, 103 us with one); a block table's nearly all are, and one makes for less code (16 sessions of 4 query
    // rows: 111 us with one, 117 us with four).
    static constexpr int kBatch = MAP ? 4 : 1;
    static constexpr int kQueue = MAP ? 256 : 64;                // a power of two, at least 31 + kTile * kBatch
    static constexpr int kWarps = W, kThreads = 32 * W;
    static constexpr int kRows = 8 * NT;
    static constexpr int kStages = D == 64 ? 3 : 2;  // two blocks per SM (D = 256: one)
    static constexpr int kCode = D / 2, kScale = D / kKv4Group;  // bytes per row
    static constexpr int kStage = kTile * 2 * (kCode + kScale);
    static constexpr int kKC = 0, kKS = kTile * kCode, kVC = kKS + kTile * kScale, kVS = kVC + kTile * kCode;
    struct Warp {
        int2 queue[kQueue];         // live tokens waiting for a stage: slot, position
        int stage_pos[kStages][kTile];
        uint64_t landed[kStages];   // mbarriers of the stages' bulk copies
    };
    struct Part {
        int nan_tail, gave_up;
        uint64_t never;             // a barrier that nothing completes
        // pieces are worked out by one thread, the next one during the loop over tokens, and kept here
        struct Piece {
            int session, chunk0, chunk1, share0, sharers;
            bool late;              // the session starts in share0, and not with it
        } piece[2];
        int session;                // of the next piece, and where that is
        long long pos, end, before, quota, sums[kWarps];
        float m[kRows], l[kRows];   // the block's maxima and totals
        float wm[kWarps][kRows], wl[kWarps][kRows];
        uint2 q[NT == 2 ? 2 * D / 16 * 32 : 1];  // query fragments of two row tiles: they would take too many registers
    };
    static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
    static constexpr size_t kMerge = (size_t)kWarps * kRows * D * 4;  // over the ring when the loop has ended
    static constexpr size_t kBuf = kRing > kMerge ? kRing : kMerge;
    static constexpr int kElems = kRows * D / 4;
    // The warps' sums as they lie in the fragments, four values per lane: element e of kElems holds rows n, n + 1 by
    // dims d, d + 1.
    static __device__ __forceinline__ int row_at(int e) { return 8 * ((e >> 5) / (D / 16)) + 2 * (e & 3); }
    static __device__ __forceinline__ int dim_at(int e) { return ((e & 31) >> 2) * (D / 8) + 2 * ((e >> 5) % (D / 16)); }
    static constexpr int kPartial = kRows * (D + 2) + 4;  // floats: sums, maxima, totals, the NaN mark; a multiple of 4
    static constexpr size_t kSmem = kBuf + kWarps * sizeof(Warp) + sizeof(Part);
    static_assert(kSmem <= 232448, "shared memory per block");
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool real) {
    const int n = real ? BYTES : 0;  // 0: the destination is filled with zeros, nothing is read
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned), counted by bar.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Ordinary writes of this thread to shared memory (stores and cp.async that have landed) come before bulk copies to the
// same place that are issued after a barrier.
__device__ __forceinline__ void fence_bulk() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Waits for a phase of bar, limit_ns (a second) at most; one answer for the warp's lanes.
__device__ __forceinline__ bool wait_lane(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63) == 63) {
            uint64_t t;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            if (!t0)
                t0 = t;
            else if (t - t0 > limit_ns)
                return false;
        }
    }
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, wait_lane(bar, parity, limit_ns));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// fp16 scale of byte b in both halves; of bytes lo and hi in one half each.
__device__ __forceinline__ uint32_t scale2(uint32_t b) { return (b << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t scale2(uint32_t lo, uint32_t hi) { return (lo << 7) | (hi << 23); }

// Slot of token j as the map or the block table has it; negative where a page is not live.
template <bool MAP>
__device__ __forceinline__ int raw_slot(const AttnArgs& a, const int32_t* map, int j, unsigned& err) {
    if constexpr (MAP) return __ldg(map + j);
    const int b = a.page_shift >= 0 ? j >> a.page_shift : j / a.page;
    const int pg = __ldg(map + b);
    if (pg >= a.P) err |= KVSEL_DEV_BAD_PAGE;
    return pg < 0 || pg >= a.P ? -1 : pg * a.page + (j - b * a.page);
}
__device__ __forceinline__ uint32_t row_of(const AttnArgs& a, int slot, int g) {
    const int pg = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page;
    return ((uint32_t)pg * (a.Hkv - 1) + g) * a.page + slot;
}

__device__ __forceinline__ int length_of(const AttnArgs& a, int s) { return min(max(__ldg(a.lens + s), 0), a.max_len); }
__device__ __forceinline__ int chunks_of(int len) { return max(1, (len + kTile - 1) / kTile); }

// Blocks per SM.
template <int D, int W>
constexpr int C_blocks() { return D == 256 ? 1 : 16 / W; }

// Writes element e of unit y of session s; m, l: the rows' maxima and totals.
template <class C, int D, bool MAP>
__device__ __forceinline__ void finish(const AttnArgs& a, int s, int y, int e, float4 v, const float* m, const float* l,
                                       bool nan_tail, unsigned& err) {
    const int G = a.Hq / a.Hkv, R = a.Tq * G, g = y / a.row_tiles, row0 = (y - g * a.row_tiles) * C::kRows;
    const int n = C::row_at(e), d = C::dim_at(e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = row0 + n + h;
        if (row >= R) break;
        float v0 = h ? v.y : v.x, v1 = h ? v.w : v.z;
        const float top = m[n + h], sum = l[n + h];
        const int tok = row / G, head = g * G + row - tok * G;
        if (nan_tail) {  // NaN groups of tokens that not every row sees
            const int32_t* const map = a.map + (int64_t)s * a.ld;
            const int common = length_of(a, s) - a.Tq;
            for (int j = max(common + 1, 0); j <= common + tok; ++j) {
                const int slot = raw_slot<MAP>(a, map, j, err);
                if (slot >= 0 && slot != a.dead && slot < a.n_slots &&
                    __ldg(a.vs + (int64_t)row_of(a, slot, g) * C::kScale + d / kKv4Group) == kKv4NanByte)
                    v0 = v1 = __int_as_float(0x7FC00000);
            }
        }
        const int64_t at = ((int64_t)s * a.Tq + tok) * a.Hq + head;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<__nv_bfloat162*>(a.out + at * D + d) = __floats2bfloat162_rn(v0 * inv, v1 * inv);
        if (a.lse && d == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top - kHead + log2f(sum)) * kLn2;
    }
}

// Joins block blockIdx.x's shared unit that starts in its share: a quarter of its elements per block.
template <int D, int NT, bool MAP>
__global__ void __launch_bounds__(256) kv4_join_kernel(const AttnArgs a) {
    using C = Cfg<D, NT, 8, MAP>;
    constexpr int kRows = C::kRows, kPart = C::kElems / 4, kGroups = 256 / kPart;  // thread groups take every kGroups-th sharer
    extern __shared__ __align__(16) float fs[];  // [kRows][sharers] factors, then [256] sums of four
    __shared__ float m[kRows], l[kRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Shared u = a.shared[blockIdx.x];
    if (!u.sharers) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Y = a.Hkv * a.row_tiles;
    auto partial = [&](int k) { return a.partials + (size_t)(2 * ((int)blockIdx.x + k * Y) + (k == 0 && u.late)) * kPartialFloats; };
    const int group = threadIdx.x / kPart, e = blockIdx.y * kPart + threadIdx.x % kPart;
    float4 x[8];                            // on their way while the factors are worked out
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (group + k * kGroups < u.sharers) x[k] = reinterpret_cast<const float4*>(partial(group + k * kGroups))[e];
    bool mark = false;
    for (int n = warp; n < kRows; n += 8) {  // a row per warp: each sharer's maximum becomes its factor
        float top = -INFINITY, sum = 0.f;
        for (int k = lane; k < u.sharers; k += 32) {
            const float* from = partial(k) + kRows * D + n;
            const float mk = from[0], lk = from[kRows];
            mark |= from[2 * kRows - n] != 0.f;
            const float up = fmaxf(top, mk);
            if (up != -INFINITY) sum = sum * ex2(top - up) + lk * ex2(mk - up);
            top = up;
            fs[n * u.sharers + k] = mk;
        }
        float all = top;
#pragma unroll
        for (int k = 16; k; k >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, k));
        if (top != -INFINITY) sum *= ex2(top - all);
#pragma unroll
        for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        for (int k = lane; k < u.sharers; k += 32) fs[n * u.sharers + k] = all == -INFINITY ? 0.f : ex2(fs[n * u.sharers + k] - all);
        if (lane == 0) m[n] = all, l[n] = sum;
    }
    const bool nan_tail = __syncthreads_or(mark);
    const float* const f = fs + C::row_at(e) * u.sharers;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = group; k0 < u.sharers; k0 += 8 * kGroups) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k * kGroups < u.sharers) {
                const float z0 = f[k0 + k * kGroups], z1 = f[u.sharers + k0 + k * kGroups];
                v.x = fmaf(x[k].x, z0, v.x), v.y = fmaf(x[k].y, z1, v.y);
                v.z = fmaf(x[k].z, z0, v.z), v.w = fmaf(x[k].w, z1, v.w);
            }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + (k + 8) * kGroups < u.sharers) x[k] = reinterpret_cast<const float4*>(partial(k0 + (k + 8) * kGroups))[e];
    }
    float4* const sums = reinterpret_cast<float4*>(fs + (kRows * u.sharers + 3) / 4 * 4);
    sums[threadIdx.x] = v;
    __syncthreads();
    unsigned err = 0;
    if (threadIdx.x < kPart) {
#pragma unroll
        for (int k = 1; k < kGroups; ++k) {
            const float4 z = sums[k * kPart + threadIdx.x];
            v.x += z.x, v.y += z.y, v.z += z.z, v.w += z.w;
        }
        finish<C, D, MAP>(a, u.session, blockIdx.x % Y, e, v, m, l, nan_tail, err);
    }
    if (err) atomicOr(a.err, err);
}

template <int D, int NT, int W, bool MAP>
__global__ void __launch_bounds__(32 * W, C_blocks<D, W>()) kv4_attention_kernel(const AttnArgs a) {
    using C = Cfg<D, NT, W, MAP>;
    constexpr int kBatch = C::kBatch, kQueue = C::kQueue;
    constexpr int kRows = C::kRows, kStages = C::kStages, kWarps = W, kThreads = 32 * W;
    constexpr int MT = D / 16;              // 16-dim tiles of V^T
    constexpr int KK = D / 16;              // 16-dim steps of K q^T
    extern __shared__ __align__(16) uint8_t smem[];
    typename C::Warp* const warps = reinterpret_cast<typename C::Warp*>(smem + C::kBuf);
    typename C::Part& part = *reinterpret_cast<typename C::Part*>(smem + C::kBuf + kWarps * sizeof(typename C::Warp));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int G = a.Hq / a.Hkv, R = a.Tq * G, Y = a.Hkv * a.row_tiles;
    typename C::Warp& w = warps[warp];
    uint8_t* const ring = smem + (size_t)warp * kStages * C::kStage;
    unsigned err = 0;
    unsigned parity = 0;                    // next phase of each stage's barrier, a bit each
    if (lane < kStages)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\nfence.mbarrier_init.release.cluster;" ::"r"(saddr(&w.landed[lane])) : "memory");

    // ---- the block's share: `quota` chunks from `start` on ----
    // Session s takes kStart + chunks places, the first session's start lying before place 0.
    // Sums of the sessions' places up to and with each thread's session, kThreads sessions at a time.
    auto scan = [&](int s, long long& upto) {
        long long v = s < a.S ? kStart + chunks_of(length_of(a, s)) : 0;
        const long long own = v;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, v, k);
            if (lane >= k) v += x;
        }
        __syncthreads();
        if (lane == 31) part.sums[warp] = v;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) v += part.sums[k];
            all += part.sums[k];
        }
        upto = v;
        return make_longlong2(own, all);
    };
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < a.S; s += kThreads)
            if (__ldg(a.lens + s) != length_of(a, s)) err |= KVSEL_DEV_BAD_LENGTH;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Shares of sessions, and the block's: number blockIdx.x / Y, for unit y = blockIdx.x % Y of the sessions in it.
    // With more units than blocks there is one share, and blocks take every gridDim.x-th y, one after the other.
    const int shares = max(1, (int)gridDim.x / Y), share = (int)gridDim.x < Y ? 0 : blockIdx.x / Y;
    int y = (int)gridDim.x < Y ? blockIdx.x : blockIdx.x % Y;
    if (a.whole) {                                   // sessions share, share + shares, ...
        if (threadIdx.x == 0) part.pos = share, part.end = a.S, part.quota = shares;
    } else {
        long long total = -kStart, upto = 0;
        longlong2 mine = make_longlong2(0, 0);
        for (int s0 = 0; s0 < a.S; s0 += kThreads) {
            mine = scan(s0 + threadIdx.x, upto);
            total += mine.y;
        }
        long long quota = total < (1ll << 31) ? (unsigned)(total + shares - 1) / (unsigned)shares : (total + shares - 1) / shares;
        quota = max(quota, (long long)kWarps * kLeast);
        const long long start = share * quota, end = min(start + quota, total);
        for (long long s0 = 0, run = -kStart; s0 < a.S; s0 += kThreads) {
            if (a.S > kThreads) mine = scan((int)s0 + threadIdx.x, upto);
            const long long from = run + upto - mine.x;
            if (mine.x && from <= start && start < from + mine.x) part.session = (int)s0 + threadIdx.x, part.before = from;
            run += mine.y;
        }
        if (threadIdx.x == 0) part.pos = start, part.end = share < shares ? end : 0, part.quota = quota, a.shared[blockIdx.x].sharers = 0;
    }

    // Piece number k of the share, by thread 0; session -1: there are no more.
    auto next_piece = [&](int k) {
        auto& x = part.piece[k & 1];
        x.session = -1;
        if (part.pos >= part.end) return;
        if (a.whole) {
            x.session = (int)part.pos;
            x.chunk0 = 0, x.chunk1 = chunks_of(length_of(a, x.session)), x.sharers = 1;
            part.pos += part.quota;
            return;
        }
        const long long first = part.before + kStart, q = part.quota;  // first: of the session's own chunks
        const unsigned q32 = (unsigned)min(q, (long long)UINT_MAX);    // divides numbers below 2^31 alike
        const int chunks = chunks_of(length_of(a, part.session));
        if (part.end <= first) return;                 // only the place of its start is left
        int share1;
        if (first + chunks < (1ll << 31)) {
            x.share0 = (int)((unsigned)first / q32);
            share1 = (int)((unsigned)(first + chunks - 1) / q32);
        } else {
            x.share0 = (int)(first / q);
            share1 = (int)((first + chunks - 1) / q);
        }
        x.session = part.session;
        x.chunk0 = (int)max(part.pos - first, 0ll);
        x.chunk1 = (int)min((long long)chunks, part.end - first);
        x.sharers = share1 - x.share0 + 1;
        x.late = part.before > x.share0 * q;
        if (x.sharers > 1 && x.share0 == share) a.shared[blockIdx.x] = Shared{x.sharers, x.session, x.late};
        part.pos = first + x.chunk1;
        if (x.chunk1 == chunks) part.before = part.pos, ++part.session;
    };
    __syncthreads();
    if (threadIdx.x == 0) {
        part.nan_tail = part.gave_up = 0;
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&part.never)) : "memory");
        next_piece(0);
    }
    __syncthreads();

    for (int number = 0;; ++number) {
    // ---- a piece: chunks [chunk0, chunk1) of unit y of session s ----
    const auto& piece = part.piece[number & 1];
    const int s = piece.session;
    if (s < 0) {
        if ((int)gridDim.x >= Y || (y += gridDim.x) >= Y) break;
        __syncthreads();                             // the next y, over the one share's sessions again
        if (threadIdx.x == 0) {
            part.pos = 0, part.session = 0, part.before = -kStart;
            next_piece(number + 1);
        }
        __syncthreads();
        continue;
    }
    const int len = length_of(a, s);
    const int g = y / a.row_tiles, row0 = (y - g * a.row_tiles) * kRows;
    const int common = len - a.Tq;          // the last token that every query row sees

    // ---- the warp's stream of live tokens ----
    // Slots are read kBatch chunks of 32 at a time, one such batch ahead of its use.
    const int32_t* const map = a.map + (int64_t)s * a.ld;
    constexpr int step = kWarps * kTile;
    const int last = (int)min((long long)len, (long long)piece.chunk1 * kTile);
    int j0 = (piece.chunk0 + warp) * kTile;                // first chunk of the batch in `ahead`
    int ahead[kBatch], batch_j = 0;                  // slots read, not looked at yet
    uint32_t rows[kBatch];                           // rows of the current batch's chunks in `bulk`
    unsigned bulk = 0;
    unsigned head = 0, queued = 0;
    constexpr uint32_t kRowStep = C::kScale < 16 ? 16 / C::kScale : 1;  // rows at which scales are 16-byte aligned
    auto read_slots = [&](int from) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int j = from + k * step + lane;
            ahead[k] = j < last ? raw_slot<MAP>(a, map, j, err) : -1;
        }
    };
    const unsigned below = (1u << lane) - 1;
    const bool runs = a.page % 16 == 0;
    if (j0 < last) read_slots(j0);

    // query fragments: lane (n = r, c) holds row n's dims 128 m + 32 c .. + 31 (D = 64: 16 c .. + 15)
    constexpr bool kQShared = NT == 2;
    uint32_t qf[kQShared ? 1 : KK][2];
    float cf[NT][2];                        // logit (base 2) = S * cf for the lane's rows 8 t + 2 c, + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = row0 + 8 * t + r;
        const int tok = n / G, h = g * G + n - tok * G;
        const __nv_bfloat16* src = a.q + ((int64_t)s * a.Tq + tok) * a.q_stride + (int64_t)h * D;
        uint32_t raw[KK][2];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            const int d = D == 64 ? 16 * c + 4 * k : 128 * (k >> 3) + 32 * c + 4 * (k & 7);
            const uint2 v = n < R ? __ldg(reinterpret_cast<const uint2*>(src + d)) : make_uint2(0, 0);
            raw[k][0] = v.x, raw[k][1] = v.y;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(raw[k][i] << 16)), fabsf(__uint_as_float(raw[k][i] & 0xFFFF0000u))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top in [2^e, 2^(e+1)); the factor 2^(14 - e) stays a normal number
        const int e = max((int)(__float_as_uint(top) >> 23) - 127, -110);
        const float f = __uint_as_float((uint32_t)(14 - e + 127) << 23);
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                raw[k][i] = pack_half2(__uint_as_float(raw[k][i] << 16) * f, __uint_as_float(raw[k][i] & 0xFFFF0000u) * f);
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            if constexpr (kQShared) {
                if (warp == 0) part.q[(k * NT + t) * 32 + lane] = make_uint2(raw[k][0], raw[k][1]);
            } else {
                qf[k][0] = raw[k][0], qf[k][1] = raw[k][1];
            }
        }
        // not 0, so that a masked S of -inf stays -inf
        const float back = fmaxf(a.scale * kLog2e * __uint_as_float((uint32_t)(e - 14 + 127) << 23), 0x1p-126f);
        cf[t][0] = __shfl_sync(0xffffffffu, back, 8 * c);      // row 2 c's lanes start at 4 (2 c)
        cf[t][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
    }

    // ref = kHead - the row's reference, so that a weight is 2^(S cf + ref)
    float o[NT][MT][4], l[NT][2], ref[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        ref[t][0] = ref[t][1] = kUnset;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }

    // Puts 32 live tokens (fewer at the end) on their way into stage st; their number, plus kBulk where
    // they come by bulk copies.
    auto produce = [&](int st) -> unsigned {
        const uint32_t base = saddr(ring + st * C::kStage);
        while (!bulk && queued < (unsigned)kTile && j0 < last) {  // the next batch: whole runs stay in `rows`, other live tokens queue up
            int slot[kBatch];
            bool bad = false;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) slot[k] = ahead[k];
            batch_j = j0;
            j0 += kBatch * step;
            if (j0 < last) read_slots(j0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool ok = slot[k] >= 0 && slot[k] != a.dead, real = ok && (!MAP || slot[k] < a.n_slots);
                bad |= ok != real;
                const unsigned live = __ballot_sync(0xffffffffu, real);
                // two runs of 16 consecutive rows?  Pages of a multiple of 16 give them, and a map's slots may
                if (live == 0xffffffffu && (MAP || runs)) {
                    rows[k] = row_of(a, slot[k], g);
                    bool run = true;
                    if constexpr (MAP) {
                        const uint32_t first = __shfl_sync(0xffffffffu, rows[k], lane & 16);
                        run = __all_sync(0xffffffffu, rows[k] == first + (lane & 15) && first % kRowStep == 0);
                    }
                    if (run) {
                        bulk |= 1u << k;
                        continue;
                    }
                }
                if (real) {
                    w.queue[(head + queued + __popc(live & below)) % kQueue] = make_int2(slot[k], batch_j + k * step + lane);
                }
                queued += __popc(live);
            }
            if (bad) err |= KVSEL_DEV_BAD_SLOT;
        }
        if (bulk) {  // eight bulk copies: codes and scales of K and V, two runs each
            const int k = __ffs(bulk) - 1;
            bulk &= bulk - 1;
            uint32_t row = rows[0];
#pragma unroll
            for (int i = 1; i < kBatch; ++i) row = k == i ? rows[i] : row;
            w.stage_pos[st][lane] = batch_j + k * step + lane;
            const uint32_t bar = saddr(&w.landed[st]);
            if (lane == 0)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "n"(C::kStage) : "memory");
            const uint32_t half = lane & 1, from = __shfl_sync(0xffffffffu, row, half * 16);
            __syncwarp();
            if (lane < 4)
                copy_bulk(base + (lane < 2 ? C::kKC : C::kVC) + half * (16 * C::kCode),
                          (lane < 2 ? a.kc : a.vc) + (uint64_t)from * C::kCode, 16 * C::kCode, bar);
            else if (lane < 8)
                copy_bulk(base + (lane < 6 ? C::kKS : C::kVS) + half * (16 * C::kScale),
                          (lane < 6 ? a.ks : a.vs) + (uint64_t)from * C::kScale, 16 * C::kScale, bar);
            asm volatile("cp.async.commit_group;" ::: "memory");
            return kTile | kBulk;
        }
        __syncwarp();
        const int n = min(queued, (unsigned)kTile);
        if (n) {
            const int2 token = w.queue[(head + lane) % kQueue];
            w.stage_pos[st][lane] = token.y;
            const uint32_t row = lane < n ? row_of(a, token.x, g) : 0;
            constexpr int kPer = C::kCode / 16;      // 16-byte pieces of a row's codes
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = k * 32 + lane, t = i / kPer;
                const uint32_t from = __shfl_sync(0xffffffffu, row, t);
                copy_async<16>(base + C::kKC + i * 16, a.kc + (lane % kPer) * 16 + (uint64_t)from * C::kCode, t < n);
                copy_async<16>(base + C::kVC + i * 16, a.vc + (lane % kPer) * 16 + (uint64_t)from * C::kCode, t < n);
            }
            copy_async<C::kScale>(base + C::kKS + lane * C::kScale, a.ks + (uint64_t)row * C::kScale, lane < n);
            copy_async<C::kScale>(base + C::kVS + lane * C::kScale, a.vs + (uint64_t)row * C::kScale, lane < n);
            head = (head + n) % kQueue;
            queued -= n;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return n;
    };

    const int perm = (r >> 1) + 4 * (r & 1);         // token of fragment row r in a tile of 16 (row r + 8: 8 more)
    auto consume = [&](auto tailc, int st, int n) {
        constexpr bool tail = decltype(tailc)::value;  // the stage is short, or holds tokens that not every row sees
        const uint8_t* const buf = ring + st * C::kStage;
        // S^T: two tiles of 16 tokens
        float x[NT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][u][0] = x[t][u][1] = x[t][u][2] = x[t][u][3] = 0.f;
        // one row tile: both token tiles at once; two: one after the other, for the registers
        constexpr int kU = NT == 1 ? 2 : 1;
#pragma unroll
        for (int u0 = 0; u0 < 2; u0 += kU)
#pragma unroll
            for (int mm = 0; mm < (D == 64 ? 1 : D / 128); ++mm) {
                constexpr int kWords = D == 64 ? 2 : 4;          // 32-bit words of codes per row and lane
                uint32_t kw[2 * kU][kWords], sc[2 * kU];         // rows perm, perm + 8 (, perm + 16, perm + 24)
#pragma unroll
                for (int k = 0; k < 2 * kU; ++k) {
                    const int tok = 16 * u0 + perm + 8 * k;
                    if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2*>(buf + C::kKC + tok * C::kCode + 8 * c);
                        kw[k][0] = v.x, kw[k][1] = v.y;
                        sc[k] = buf[C::kKS + tok * C::kScale + c];
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(buf + C::kKC + tok * C::kCode + 64 * mm + 16 * c);
                        kw[k][0] = v.x, kw[k][1] = v.y, kw[k][2] = v.z, kw[k][3] = v.w;
                        sc[k] = *reinterpret_cast<const uint16_t*>(buf + C::kKS + tok * C::kScale + 8 * mm + 2 * c);
                    }
                }
#pragma unroll
                for (int i = 0; i < kWords; ++i) {               // a word is two steps of 4 dims per lane
                    uint32_t h[2 * kU][4];
#pragma unroll
                    for (int k = 0; k < 2 * kU; ++k) {
                        const uint32_t s2 = i < 2 ? scale2(sc[k] & 0xFFu) : scale2(sc[k] >> 8);
                        kv4_pairs(kw[k][i], h[k]);
#pragma unroll
                        for (int b = 0; b < 4; ++b) h[k][b] = mul2(h[k][b], s2);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int kk = 8 * mm + 2 * i + k;
                            uint2 q;
                            if constexpr (kQShared)
                                q = part.q[(kk * NT + t) * 32 + lane];
                            else
                                q = make_uint2(qf[kk][0], qf[kk][1]);
#pragma unroll
                            for (int u = 0; u < kU; ++u)
                                mma16816(x[t][u0 + u], h[2 * u][2 * k], h[2 * u + 1][2 * k], h[2 * u][2 * k + 1],
                                         h[2 * u + 1][2 * k + 1], q.x, q.y);
                        }
                }
            }
        // what a row does not see becomes -inf
        bool past = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (tail) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 16 * u + perm + (i >> 1) * 8;
                        const int row = row0 + 8 * t + 2 * c + (i & 1);
                        if (tok >= n || w.stage_pos[st][tok] > common + row / G) x[t][u][i] = -INFINITY;
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float top = fmaxf(fmaxf(x[t][0][e], x[t][0][2 + e]), fmaxf(x[t][1][e], x[t][1][2 + e]));
                past |= fmaf(top, cf[t][e], ref[t][e]) > kHead + kSlack;
            }
        }
        if (__any_sync(0xffffffffu, past)) {         // some reference moves up to its row's maximum
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(fmaxf(x[t][0][e], x[t][0][2 + e]), fmaxf(x[t][1][e], x[t][1][2 + e]));
#pragma unroll
                    for (int k = 4; k <= 16; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                    const float to = fminf(ref[t][e], kHead - top * cf[t][e]);
                    const float f = ex2(to - ref[t][e]);
                    ref[t][e] = to;
                    l[t][e] *= f;
#pragma unroll
                    for (int i = 0; i < MT; ++i) o[t][i][e] *= f, o[t][i][2 + e] *= f;
                }
        }
        uint32_t pf[NT][2][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float p0 = ex2(fmaf(x[t][u][0], cf[t][0], ref[t][0])), p1 = ex2(fmaf(x[t][u][1], cf[t][1], ref[t][1]));
                const float p2 = ex2(fmaf(x[t][u][2], cf[t][0], ref[t][0])), p3 = ex2(fmaf(x[t][u][3], cf[t][1], ref[t][1]));
                l[t][0] += p0 + p2;
                l[t][1] += p1 + p3;
                pf[t][u][0] = transpose8x8(pack_half2(p0, p1));
                pf[t][u][1] = transpose8x8(pack_half2(p2, p3));
            }
        }
        // O^T += V^T p^T: the lane's tokens are c, 4 + c, 8 + c, 12 + c of each tile, its dims r D/8 .. + D/8 - 1
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            constexpr int kWords = D / 64;           // 32-bit words of codes per token and lane
            uint32_t vw[4][kWords], vsc[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tok = 16 * u + 4 * k + c;
                const uint8_t* src = buf + C::kVC + tok * C::kCode + r * (4 * kWords);
                if constexpr (kWords == 1) {
                    vw[k][0] = *reinterpret_cast<const uint32_t*>(src);
                    vsc[k] = buf[C::kVS + tok * C::kScale + (r >> 1)];
                } else if constexpr (kWords == 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    vw[k][0] = v.x, vw[k][1] = v.y;
                    vsc[k] = buf[C::kVS + tok * C::kScale + r];
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    vw[k][0] = v.x, vw[k][1] = v.y, vw[k][2] = v.z, vw[k][3] = v.w;
                    vsc[k] = *reinterpret_cast<const uint16_t*>(buf + C::kVS + tok * C::kScale + 2 * r);
                }
                if (tail && tok < n && w.stage_pos[st][tok] > common) {
                    // a NaN group that some rows do not see must not reach them through weights of zero: it
                    // counts as zero here and is put back at the end for the rows that see it
                    if ((vsc[k] & 0xFFu) == kKv4NanByte) vsc[k] &= 0xFF00u, part.nan_tail = 1;
                    if ((vsc[k] >> 8) == kKv4NanByte) vsc[k] &= 0xFFu, part.nan_tail = 1;
                }
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const bool hi = kWords == 4 && i >= 2;
                const uint32_t s01 = hi ? scale2(vsc[0] >> 8, vsc[1] >> 8) : scale2(vsc[0] & 0xFFu, vsc[1] & 0xFFu);
                const uint32_t s23 = hi ? scale2(vsc[2] >> 8, vsc[3] >> 8) : scale2(vsc[2] & 0xFFu, vsc[3] & 0xFFu);
                constexpr uint32_t kLow = 0x0F0F0F0Fu;
                uint32_t e01[4], o01[4], e23[4], o23[4];         // even and odd dims, token pairs
                kv4_pairs((vw[0][i] & kLow) | ((vw[1][i] << 4) & ~kLow), e01);
                kv4_pairs(((vw[0][i] >> 4) & kLow) | (vw[1][i] & ~kLow), o01);
                kv4_pairs((vw[2][i] & kLow) | ((vw[3][i] << 4) & ~kLow), e23);
                kv4_pairs(((vw[2][i] >> 4) & kLow) | (vw[3][i] & ~kLow), o23);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t a0 = mul2(e01[b], s01), a1 = mul2(o01[b], s01), a2 = mul2(e23[b], s23), a3 = mul2(o23[b], s23);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(o[t][4 * i + b], a0, a1, a2, a3, pf[t][u][0], pf[t][u][1]);
                }
            }
        }
    };

    unsigned counts = 0;                             // produce()'s answers for the stages on their way, a byte each, oldest lowest
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) counts |= produce(st) << (8 * st);
    __syncthreads();                                 // the shared query fragments are set
    if (threadIdx.x == 0) next_piece(number + 1);
    bool ok = true;
    if (a.stuck && warp == 0) ok = wait_phase(saddr(&part.never), 0, a.wait_ns);
    int st = 0;
    while (ok && (counts & 0xFFu)) {
        counts |= produce(st == 0 ? kStages - 1 : st - 1) << (8 * (kStages - 1));
        if (counts & kBulk) {
            ok = wait_phase(saddr(&w.landed[st]), (parity >> st) & 1u, a.wait_ns);
            if (!ok) break;
            parity ^= 1u << st;
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            fence_bulk();
        }
        __syncwarp();
        const int n = counts & 0x3Fu;
        if (n < kTile || (a.Tq > 1 && __any_sync(0xffffffffu, w.stage_pos[st][lane] > common)))
            consume(std::true_type{}, st, n);
        else
            consume(std::false_type{}, st, n);
        __syncwarp();
        counts >>= 8;
        st = st == kStages - 1 ? 0 : st + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!ok) {                                       // no more is asked for; what is on its way lands before the block ends
        err |= KVSEL_DEV_TIMEOUT;
        part.gave_up = 1;
        for (; counts; counts >>= 8, st = st == kStages - 1 ? 0 : st + 1)
            if (counts & kBulk) wait_phase(saddr(&w.landed[st]), (parity >> st) & 1u, kWaitNs);
    }

    // ---- join: warps, then blocks, in fixed order ----
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int k = 4; k <= 16; k <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], k);
            if (r == 0) {
                part.wm[warp][8 * t + 2 * c + e] = ref[t][e] != kUnset ? kHead - ref[t][e]
                                                           : l[t][e] == l[t][e] ? -INFINITY : 0.f;  // only NaN logits: a NaN
                part.wl[warp][8 * t + 2 * c + e] = l[t][e];
            }
        }
    __syncthreads();                                 // also: every warp is done with its ring
    if (part.gave_up) break;                         // the block's other pieces are left out, the error word tells
    constexpr int kElems = C::kElems;
    float4* const merge = reinterpret_cast<float4*>(smem);  // [kWarps][kElems]
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = 8 * t + 2 * c + e;
            float top = part.wm[0][n];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) top = fmaxf(top, part.wm[k][n]);
            f[e] = top == -INFINITY ? 0.f : ex2(part.wm[warp][n] - top);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
            merge[warp * kElems + (t * MT + i) * 32 + lane] =
                make_float4(o[t][i][0] * f[0], o[t][i][1] * f[1], o[t][i][2] * f[0], o[t][i][3] * f[1]);
    }
    if (threadIdx.x < kRows) {
        const int n = threadIdx.x;
        float top = part.wm[0][n], sum = 0.f;
#pragma unroll
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, part.wm[k][n]);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum += top == -INFINITY ? 0.f : part.wl[k][n] * ex2(part.wm[k][n] - top);
        part.m[n] = top;
        part.l[n] = sum;
    }
    __syncthreads();
    auto block_sum = [&](int e) {
        float4 v = merge[e];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) {
            const float4 x = merge[k * kElems + e];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        return v;
    };
    if (piece.sharers > 1) {
        // the partial of the block's first piece, but for a unit that starts within its share
        float* const own = a.partials + (size_t)(2 * blockIdx.x + (piece.share0 == share && piece.late)) * kPartialFloats;
        for (int e = threadIdx.x; e < kElems; e += kThreads) reinterpret_cast<float4*>(own)[e] = block_sum(e);
        if (threadIdx.x < kRows) {
            own[kRows * D + threadIdx.x] = part.m[threadIdx.x];
            own[kRows * (D + 1) + threadIdx.x] = part.l[threadIdx.x];
        }
        if (threadIdx.x == 0) own[kRows * (D + 2)] = part.nan_tail ? 1.f : 0.f;
    } else {
        for (int e = threadIdx.x; e < kElems; e += kThreads)
            finish<C, D, MAP>(a, s, y, e, block_sum(e), part.m, part.l, part.nan_tail != 0, err);
    }
    fence_bulk();                                    // the sums lay over the ring
    __syncthreads();                                 // shared memory is free for the next piece
    if (threadIdx.x == 0) part.nan_tail = 0;         // (a sync lies between this and the piece's loop)
    }
    if (err) atomicOr(a.err, err);
}

template <int D, int NT, int W, bool MAP>
cudaError_t launch(kvsel_ctx* ctx, AttnArgs a, cudaStream_t s) {
    using C = Cfg<D, NT, W, MAP>;
    static_assert(C::kPartial <= kPartialFloats, "a partial result");
    auto* kernel = kv4_attention_kernel<D, NT, W, MAP>;
    constexpr unsigned kBit = 1u << (D / 64 * 2 + NT + (MAP ? 8 : 0));  // 3, 4; 5, 6; 9, and 8 more
    if (!(ctx->ready & kBit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        ctx->ready |= kBit;
    }
    // whole shares of Y blocks, no more than there are sessions to take whole
    const int Y = a.Hkv * a.row_tiles, most = ctx->num_sms * C_blocks<D, W>();
    a.whole = a.max_len <= (a.S >= kMany ? kWholeMany : kWhole);
    const int blocks = Y >= most ? most : Y * (a.whole && a.S < most / Y ? a.S : most / Y);
    kernel<<<blocks, C::kThreads, C::kSmem, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.whole) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, 4);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = (size_t)(C::kRows * blocks + 4) * sizeof(float) + 256 * sizeof(float4);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, MAP>, a);
}

// Two blocks of 8 warps per SM, or of 6 where two row tiles of D = 128 need the registers (16 sessions of 16 rows: 117 us;
// 136 us with 8 warps and spilled registers); D = 256: one block.
template <bool MAP>
cudaError_t launch_for(kvsel_ctx* ctx, const AttnArgs& a, int D, bool wide, cudaStream_t s) {
    if (D == 256) return launch<256, 1, 8, MAP>(ctx, a, s);
    if (D == 128) return wide ? launch<128, 2, 6, MAP>(ctx, a, s) : launch<128, 1, 8, MAP>(ctx, a, s);
    return wide ? launch<64, 2, 8, MAP>(ctx, a, s) : launch<64, 1, 8, MAP>(ctx, a, s);
}

int attention_call(kvsel_ctx* ctx, const void* q, int64_t q_stride, int S, int Tq, int Hq, int Hkv, int D,
                   const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales, int P,
                   int page, const int32_t* seq_lens, const int32_t* slot_map, const int32_t* block_table, int ld,
                   int dead_slot, float scale, void* out, float* lse, void* stream, uint64_t wait_ns, int stuck) {
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (S < 0 || Tq < 0 || Hq <= 0 || Hkv <= 0 || P < 0 || page <= 0 || ld < 0)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "kv4_attention: bad sizes");
    if (Hq % Hkv) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "kv4_attention: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
    if (D != 64 && D != 128 && D != 256)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: D=%d unsupported", D);
    if (!slot_map == !block_table)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_attention: one of slot_map and block_table is needed");
    const int64_t reach = slot_map ? ld : (int64_t)ld * page;
    if ((int64_t)P * page > INT_MAX || reach > INT_MAX - 4096)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: slots and positions must fit 31 bits");
    if ((int64_t)P * page * Hkv > UINT_MAX)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: P*page*Hkv does not fit 32 bits");
    if (S > 65535 || Tq > 1024 || Hq > 65535)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: S, Tq or Hq too large");
    if (!(scale > 0.f) || scale > 1e30f)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_attention: scale must be positive and finite");
    if (S == 0 || Tq == 0) return KVSEL_OK;
    if (!q || !seq_lens || !out || (P > 0 && (!k_codes || !k_scales || !v_codes || !v_scales)))
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_attention: null pointer");
    if (q_stride < (int64_t)Hq * D) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "kv4_attention: token stride < Hq*D");
    auto off16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; };
    if (off16(q) || (q_stride * 2) % 16 || off16(out) || off16(k_codes) || off16(k_scales) || off16(v_codes) ||
        off16(v_scales))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "kv4_attention: q, its stride, out and the caches must be 16-byte aligned");
    const int R = Tq * (Hq / Hkv);
    // Two tiles of 8 rows share the decoded K and V where there are more than 8 rows (16 sessions of 16 rows: 151 us
    // with a tile each, 109 with two); for D = 256 their sums would take all registers.
    const bool wide = R > 8 && D != 256;
    const int tiles = (R + (wide ? 16 : 8) - 1) / (wide ? 16 : 8);
    if ((int64_t)Hkv * tiles > 65535) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: too many rows");
    int shift = -1;
    if ((page & (page - 1)) == 0)
        for (shift = 0; (1 << shift) < page;) ++shift;
    const AttnArgs a{(const __nv_bfloat16*)q, q_stride, Tq, Hq, Hkv, k_codes, k_scales, v_codes, v_scales, P, page, shift,
                     seq_lens, slot_map ? slot_map : block_table, P * page, ld, (int)reach,
                     dead_slot, tiles, scale, (__nv_bfloat16*)out, lse, ctx->dev_err, S, 0, wait_ns, stuck,
                     (float*)ctx->kv4_partials, (Shared*)((float*)ctx->kv4_partials + (size_t)ctx->num_sms * 4 * kPartialFloats)};
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = slot_map ? launch_for<true>(ctx, a, D, wide, st) : launch_for<false>(ctx, a, D, wide, st);
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_attention launch");
}

}  // namespace

size_t kv4_partials_bytes(int num_sms) { return (size_t)num_sms * 2 * (2 * kPartialFloats * sizeof(float) + sizeof(Shared)); }

extern "C" int kvsel_kv4_attention(kvsel_ctx* ctx, const void* q, int64_t q_stride, int S, int Tq, int Hq, int Hkv, int D,
                                   const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                                   const uint8_t* v_scales, int P, int page, const int32_t* seq_lens,
                                   const int32_t* slot_map, const int32_t* block_table, int ld, int dead_slot,
                                   float scale, void* out, float* lse, void* stream) {
    const kvsel_trace trace_("kvsel_kv4_attention");
    return attention_call(ctx, q, q_stride, S, Tq, Hq, Hkv, D, k_codes, k_scales, v_codes, v_scales, P, page, seq_lens,
                          slot_map, block_table, ld, dead_slot, scale, out, lse, stream, kWaitNs, 0);
}

// Test entry (not part of the public header): kvsel_kv4_attention in which the first warp of every block waits on a
// barrier that nothing completes, while its first bulk copies are on their way, and every wait for copies is limited to
// wait_ns.  The blocks that have a piece give up: they flag KVSEL_ERR_TIMEOUT, wait for their own copies, and return.  out
// and lse hold no meaningful values afterwards.
extern "C" int kvsel_test_kv4_attention_give_up(kvsel_ctx* ctx, const void* q, int64_t q_stride, int S, int Tq, int Hq,
                                                int Hkv, int D, const uint8_t* k_codes, const uint8_t* k_scales,
                                                const uint8_t* v_codes, const uint8_t* v_scales, int P, int page,
                                                const int32_t* seq_lens, const int32_t* slot_map,
                                                const int32_t* block_table, int ld, int dead_slot, float scale, void* out,
                                                float* lse, uint64_t wait_ns, void* stream) {
    const kvsel_trace trace_("kvsel_test_kv4_attention_give_up");
    if (wait_ns == 0 || wait_ns > kWaitNs)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "test_kv4_attention_give_up: wait_ns must be in (0, 1 s]");
    return attention_call(ctx, q, q_stride, S, Tq, Hq, Hkv, D, k_codes, k_scales, v_codes, v_scales, P, page, seq_lens,
                          slot_map, block_table, ld, dead_slot, scale, out, lse, stream, wait_ns, 1);
}
