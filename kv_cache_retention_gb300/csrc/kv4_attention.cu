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
// which fp16 holds exactly but for values below 2^-38 of it.  The softmax runs over
// the tokens once: per row a reference m within 5 (log2) of the running maximum or
// above, weights 2^(x - m + 10), so that fp16 holds weights down to 2^-24 of the
// largest with full precision.  Sums and outputs are fp32, moved when the reference
// moves.
//
// Tokens come to a warp through cp.async into a ring of two or three buffers of its own, so
// the loop has no block barrier.  Slots are read 32 at a time; live ones queue up, so
// dropped tokens (most of a pruned session's slot map) cost a slot read and no more.
//
// The warps of a block take every kWarps-th chunk of 32 positions, the `splits` blocks
// of one (session, kv head, row tile) the same again.  A block joins its warps through
// shared memory; with splits > 1 it leaves its sums in the context's partials, and the
// last of the blocks to arrive (a counter, which it sets back to 0) joins them in the
// order of their ranks, so results do not depend on the order of arrival.  (A cluster
// of blocks joined through distributed shared memory needs no partials, but clusters of
// 16 left half of the SMs idle: 92160 tokens of 8 kv heads took 63 us.)
#include <cuda_bf16.h>
#include <limits.h>

#include <type_traits>

#include "kv4_format.cuh"
#include "kvsel_internal.h"

namespace {

constexpr int kTile = 32;   // tokens per stage
constexpr int kBatch = 4;   // chunks of 32 slots read at a time
constexpr int kQueue = 256;  // at least 31 + kTile * kBatch
constexpr unsigned kBulk = 0x80u;
constexpr int kMaxSplitBlocks = 1024;                        // blocks of a launch that splits
constexpr int kPartialFloats = 16 * (128 + 2) + 4;           // the largest share of a block
constexpr float kUnset = 3e38f;  // ref of a row that has seen nothing
constexpr float kHead = 10.f;   // log2 of the weight at the reference
constexpr float kSlack = 5.f;   // how far (log2) a logit may pass the reference: weights stay below 2^15
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnArgs {
    const __nv_bfloat16* q;
    int64_t q_stride;
    int Tq, Hq, Hkv;
    const uint8_t *kc, *ks, *vc, *vs;
    int P, page, page_shift;  // page_shift: log2(page), or -1
    const int32_t* lens;
    const int32_t* map;       // slot map, or block table (by_page)
    int by_page, n_slots;
    int ld;                   // row length of map
    int max_len;              // tokens that a row of it reaches
    int dead;
    int row_tiles;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
    float* partials;          // [blocks][kRows * (D + 2) + 2], splits > 1 only
    unsigned* arrived;        // one counter for each (session, kv head, row tile), 0 between launches
};

// D dims, NT tiles of 8 rows, W warps per block
template <int D, int NT, int W>
struct Cfg {
    static constexpr int kWarps = W, kThreads = 32 * W;
    static constexpr int kRows = 8 * NT;
    static constexpr int kStages = D == 64 ? 3 : 2;  // two blocks per SM (D = 256: one)
    static constexpr int kCode = D / 2, kScale = D / kKv4Group;  // bytes per row
    static constexpr int kStage = kTile * 2 * (kCode + kScale);
    static constexpr int kKC = 0, kKS = kTile * kCode, kVC = kKS + kTile * kScale, kVS = kVC + kTile * kCode;
    struct Warp {
        int slot[kQueue], pos[kQueue];  // live tokens waiting for a stage
        int stage_pos[kStages][kTile];
        uint64_t landed[kStages];   // mbarriers of the stages' bulk copies
    };
    struct Part {
        int nan_tail, last;
        float wm[kWarps][kRows], wl[kWarps][kRows];
        uint2 q[NT == 2 ? 2 * D / 16 * 32 : 1];  // query fragments of two row tiles: they would take too many registers
    };
    static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
    static constexpr size_t kMerge = (size_t)kWarps * kRows * D * 4;  // over the ring when the loop has ended
    static constexpr size_t kBuf = kRing > kMerge ? kRing : kMerge;
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
// Waits for a phase of bar, a second at most.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
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
            else if (t - t0 > 1000000000ull)
                return false;
        }
    }
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
__device__ __forceinline__ int raw_slot(const AttnArgs& a, const int32_t* map, int j, unsigned& err) {
    if (!a.by_page) return __ldg(map + j);
    const int b = a.page_shift >= 0 ? j >> a.page_shift : j / a.page;
    const int pg = __ldg(map + b);
    if (pg >= a.P) err |= KVSEL_DEV_BAD_PAGE;
    return pg < 0 || pg >= a.P ? -1 : pg * a.page + (j - b * a.page);
}
__device__ __forceinline__ uint32_t row_of(const AttnArgs& a, int slot, int g) {
    const int pg = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page;
    return (uint32_t)(pg * (a.Hkv - 1) + g) * a.page + slot;
}

// grid (splits, Hkv * row_tiles, S)
template <int D, int NT, int W>
__global__ void __launch_bounds__(32 * W, D == 256 ? 1 : 16 / W) kv4_attention_kernel(const AttnArgs a) {
    using C = Cfg<D, NT, W>;
    constexpr int kRows = C::kRows, kStages = C::kStages, kWarps = W, kThreads = 32 * W;
    constexpr int MT = D / 16;              // 16-dim tiles of V^T
    constexpr int KK = D / 16;              // 16-dim steps of K q^T
    extern __shared__ __align__(16) uint8_t smem[];
    typename C::Warp* const warps = reinterpret_cast<typename C::Warp*>(smem + C::kBuf);
    typename C::Part& part = *reinterpret_cast<typename C::Part*>(smem + C::kBuf + kWarps * sizeof(typename C::Warp));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int splits = gridDim.x, rank = blockIdx.x;
    const int g = blockIdx.y / a.row_tiles, row0 = (blockIdx.y - g * a.row_tiles) * kRows, s = blockIdx.z;
    const int G = a.Hq / a.Hkv, R = a.Tq * G;
    typename C::Warp& w = warps[warp];
    uint8_t* const ring = smem + (size_t)warp * kStages * C::kStage;
    unsigned err = 0;

    const int len0 = __ldg(a.lens + s);
    const int len = min(max(len0, 0), a.max_len);
    if (len != len0) err |= KVSEL_DEV_BAD_LENGTH;
    const int common = len - a.Tq;          // the last token that every query row sees
    if (threadIdx.x == 0) part.nan_tail = 0;

    // ---- the warp's stream of live tokens ----
    // Slots are read four chunks of 32 at a time, one such batch ahead of its use.
    const int32_t* const map = a.map + (int64_t)s * a.ld;
    const int step = splits * kWarps * kTile;
    int j0 = (rank * kWarps + warp) * kTile;         // first chunk of the batch in `ahead`
    int ahead[kBatch], batch_j = 0;                  // slots read, not looked at yet
    uint32_t rows[kBatch];                           // rows of the current batch's chunks in `bulk`
    unsigned bulk = 0;
    int head = 0, queued = 0;
    unsigned parity = 0;                             // next phase of each stage's barrier, a bit each
    constexpr uint32_t kRowStep = C::kScale < 16 ? 16 / C::kScale : 1;  // rows at which scales are 16-byte aligned
    auto read_slots = [&](int from) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int j = from + k * step + lane;
            ahead[k] = j < len ? raw_slot(a, map, j, err) : -1;
        }
    };
    if (j0 < len) read_slots(j0);
    if (lane < kStages)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\nfence.mbarrier_init.release.cluster;" ::"r"(saddr(&w.landed[lane])) : "memory");

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
        while (!bulk && queued < kTile && j0 < len) {  // the next batch: whole runs stay in `rows`, other live tokens queue up
            int slot[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) slot[k] = ahead[k];
            batch_j = j0;
            j0 += kBatch * step;
            if (j0 < len) read_slots(j0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool ok = slot[k] >= 0 && slot[k] != a.dead;
                const bool real = ok && slot[k] < a.n_slots;
                if (ok && !real) err |= KVSEL_DEV_BAD_SLOT;
                const unsigned live = __ballot_sync(0xffffffffu, real);
                if (live == 0xffffffffu) {
                    // two runs of 16 consecutive rows, as whole pages give them?
                    rows[k] = row_of(a, slot[k], g);
                    const uint32_t first = __shfl_sync(0xffffffffu, rows[k], lane & 16);
                    if (__all_sync(0xffffffffu, rows[k] == first + (lane & 15) && first % kRowStep == 0)) {
                        bulk |= 1u << k;
                        continue;
                    }
                }
                if (real) {
                    const int at = (head + queued + __popc(live & ((1u << lane) - 1))) % kQueue;
                    w.slot[at] = slot[k];
                    w.pos[at] = batch_j + k * step + lane;
                }
                queued += __popc(live);
            }
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
        const int n = min(queued, kTile);
        if (n) {
            const int at = (head + lane) % kQueue;
            w.stage_pos[st][lane] = w.pos[at];
            const uint32_t row = lane < n ? row_of(a, w.slot[at], g) : 0;
            constexpr int kPer = C::kCode / 16;      // 16-byte pieces of a row's codes
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = k * 32 + lane, t = i / kPer;
                const uint64_t off = (uint64_t)__shfl_sync(0xffffffffu, row, t) * C::kCode + (lane % kPer) * 16;
                copy_async<16>(base + C::kKC + i * 16, a.kc + off, t < n);
                copy_async<16>(base + C::kVC + i * 16, a.vc + off, t < n);
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
    __syncthreads();                                 // nan_tail and the shared query fragments are set
    for (int st = 0; counts & 0xFFu;) {
        counts |= produce(st == 0 ? kStages - 1 : st - 1) << (8 * (kStages - 1));
        if (counts & kBulk) {
            if (!wait_phase(saddr(&w.landed[st]), (parity >> st) & 1u)) err |= KVSEL_DEV_TIMEOUT;
            parity ^= 1u << st;
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
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
    float* const merge = reinterpret_cast<float*>(smem);  // [kWarps][kRows][D]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = 8 * t + 2 * c + e;
            float top = part.wm[0][n];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) top = fmaxf(top, part.wm[k][n]);
            const float f = top == -INFINITY ? 0.f : ex2(part.wm[warp][n] - top);
            float* dst = merge + ((size_t)warp * kRows + n) * D + r * (D / 8);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[t][i][e] * f, o[t][i][2 + e] * f);
        }
    __syncthreads();
    // the block's maximum, total and values of row i / D, four dims from i % D on
    auto block_sums = [&](int i, float& top, float& sum) {
        const int n = i / D;
        top = part.wm[0][n], sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, part.wm[k][n]);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            sum += top == -INFINITY ? 0.f : part.wl[k][n] * ex2(part.wm[k][n] - top);
            const float4 x = *reinterpret_cast<const float4*>(merge + (size_t)k * kRows * D + i);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        return v;
    };
    bool nan_tail = part.nan_tail != 0;
    const float* gathered = nullptr;                 // the blocks' partials, where this block joins them
    if (splits > 1) {
        const int unit = blockIdx.z * gridDim.y + blockIdx.y;
        float* const mine = a.partials + ((size_t)unit * splits + rank) * C::kPartial;
        for (int i = threadIdx.x * 4; i < kRows * D; i += kThreads * 4) {
            float top, sum;
            *reinterpret_cast<float4*>(mine + i) = block_sums(i, top, sum);
            if (i % D == 0) {
                mine[kRows * D + i / D] = top;
                mine[kRows * (D + 1) + i / D] = sum;
            }
        }
        if (threadIdx.x == 0) mine[kRows * (D + 2)] = nan_tail ? 1.f : 0.f;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            const bool last = atomicAdd(a.arrived + unit, 1u) == (unsigned)splits - 1u;
            part.last = last;
            if (last) a.arrived[unit] = 0;
        }
        __syncthreads();
        if (!part.last) {
            if (err) atomicOr(a.err, err);
            return;
        }
        __threadfence();
        gathered = a.partials + (size_t)unit * splits * C::kPartial;
        // each (block, row)'s maximum becomes its factor, its total what it adds to the row's
        float* const fs = reinterpret_cast<float*>(smem);            // [splits][kRows], over the merge buffer
        float* const ls = fs + splits * kRows;
        bool mark = false;
        for (int i = threadIdx.x; i < splits * kRows; i += kThreads) {
            const float* from = gathered + (size_t)(i / kRows) * C::kPartial + kRows * D;
            fs[i] = __ldcg(from + i % kRows);
            ls[i] = __ldcg(from + kRows + i % kRows);
            if (i % kRows == 0) mark |= __ldcg(from + 2 * kRows) != 0.f;
        }
        nan_tail = __syncthreads_or(mark);
        if (threadIdx.x < kRows) {
            const int n = threadIdx.x;
            float top = -INFINITY, sum = 0.f;
            for (int k = 0; k < splits; ++k) top = fmaxf(top, fs[k * kRows + n]);
            for (int k = 0; k < splits; ++k) {
                const float f = top == -INFINITY ? 0.f : ex2(fs[k * kRows + n] - top);
                fs[k * kRows + n] = f;
                sum = fmaf(ls[k * kRows + n], f, sum);
            }
            part.wm[0][n] = top;
            part.wl[0][n] = sum;
        }
        __syncthreads();
    }
    for (int i = threadIdx.x * 4; i < kRows * D; i += kThreads * 4) {
        const int n = i / D, d = i % D, row = row0 + n;
        if (row >= R) break;
        float top, sum;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!gathered) {
            v = block_sums(i, top, sum);
        } else {
            top = part.wm[0][n], sum = part.wl[0][n];
            const float* const fs = reinterpret_cast<const float*>(smem) + n;
            for (int k0 = 0; k0 < splits; k0 += 16) {  // 16 loads on their way at a time
                float4 x[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (k0 + k < splits) x[k] = __ldcg(reinterpret_cast<const float4*>(gathered + (size_t)(k0 + k) * C::kPartial + i));
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (k0 + k < splits) {
                        const float f = fs[(k0 + k) * kRows];
                        v.x = fmaf(x[k].x, f, v.x), v.y = fmaf(x[k].y, f, v.y);
                        v.z = fmaf(x[k].z, f, v.z), v.w = fmaf(x[k].w, f, v.w);
                    }
            }
        }
        const int tok = row / G, h = g * G + row - tok * G;
        if (nan_tail) {
            for (int j = max(common + 1, 0); j <= common + tok; ++j) {
                const int slot = raw_slot(a, map, j, err);
                if (slot >= 0 && slot != a.dead && slot < a.n_slots && __ldg(a.vs + (int64_t)row_of(a, slot, g) * C::kScale + d / kKv4Group) == kKv4NanByte)
                    v.x = v.y = v.z = v.w = __int_as_float(0x7FC00000);
            }
        }
        const int64_t at = ((int64_t)s * a.Tq + tok) * a.Hq + h;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv), hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(a.out + at * D + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        if (a.lse && d == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top - kHead + log2f(sum)) * kLn2;
    }
    if (err) atomicOr(a.err, err);
}

template <int D, int NT, int W>
cudaError_t launch(kvsel_ctx* ctx, const AttnArgs& a, int S, int splits, cudaStream_t s) {
    using C = Cfg<D, NT, W>;
    static_assert(C::kPartial <= kPartialFloats, "a block's share of the partials");
    auto* kernel = kv4_attention_kernel<D, NT, W>;
    constexpr unsigned kBit = 1u << (D / 64 * 2 + NT);  // 3, 4; 5, 6; 9
    if (!(ctx->ready & kBit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        ctx->ready |= kBit;
    }
    kernel<<<dim3(splits, a.Hkv * a.row_tiles, S), C::kThreads, C::kSmem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

extern "C" int kvsel_kv4_attention(kvsel_ctx* ctx, const void* q, int64_t q_stride, int S, int Tq, int Hq, int Hkv, int D,
                                   const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                                   const uint8_t* v_scales, int P, int page, const int32_t* seq_lens,
                                   const int32_t* slot_map, const int32_t* block_table, int ld, int dead_slot,
                                   float scale, void* out, float* lse, void* stream) {
    const kvsel_trace trace_("kvsel_kv4_attention");
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
    const bool wide = R > 8 && D != 256;  // two tiles of 8 rows share the decoded K and V
    const int tiles = (R + (wide ? 16 : 8) - 1) / (wide ? 16 : 8);
    if ((int64_t)Hkv * tiles > 65535) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: too many rows");
    int shift = -1;
    if ((page & (page - 1)) == 0)
        for (shift = 0; (1 << shift) < page;) ++shift;
    AttnArgs a{(const __nv_bfloat16*)q, q_stride, Tq, Hq, Hkv, k_codes, k_scales, v_codes, v_scales, P, page, shift,
                     seq_lens, slot_map ? slot_map : block_table, block_table != nullptr, P * page, ld, (int)reach, dead_slot, tiles, scale, (__nv_bfloat16*)out, lse,
                     ctx->dev_err, nullptr, nullptr};
    const int64_t work = (int64_t)S * Hkv * tiles;
    // Splits of a session's tokens: none where the units of work fill the SMs (36 sessions of 8 kv heads: 87 us, split
    // in two 98); one wave of two blocks per SM for a single session (92160 tokens: 38 us with 38 splits, 45 with 19);
    // finer for several, whose lengths differ (16 sessions: 145 us with 8 splits, 153 with 3).  At least one chunk of
    // 32 tokens per warp.
    int64_t splits = 1;
    if (work < ctx->num_sms) splits = (S == 1 ? 2 * ctx->num_sms : kMaxSplitBlocks) / work;
    if (splits > (reach + 255) / 256) splits = (reach + 255) / 256;
    if (splits < 1) splits = 1;
    const cudaStream_t st = (cudaStream_t)stream;
    if (splits > 1) {
        if (!ctx->kv4_partials) {
            const size_t bytes = (size_t)kMaxSplitBlocks * (kPartialFloats + 1) * 4;
            cudaError_t e = cudaMalloc(&ctx->kv4_partials, bytes);
            if (e == cudaSuccess) e = cudaMemset(ctx->kv4_partials, 0, bytes);
            if (e == cudaSuccess) e = cudaDeviceSynchronize();
            if (e != cudaSuccess) {
                if (ctx->kv4_partials) cudaFree(ctx->kv4_partials);
                ctx->kv4_partials = nullptr;
                return kvsel_cuda_fail(ctx, e, "kv4_attention: allocation of the partials");
            }
        }
        a.arrived = (unsigned*)ctx->kv4_partials;
        a.partials = (float*)ctx->kv4_partials + kMaxSplitBlocks;
    }
    cudaError_t e;
    if (D == 256)
        e = launch<256, 1, 8>(ctx, a, S, (int)splits, st);
    else if (D == 128)
        e = wide ? launch<128, 2, 8>(ctx, a, S, (int)splits, st) : launch<128, 1, 8>(ctx, a, S, (int)splits, st);
    else
        e = wide ? launch<64, 2, 8>(ctx, a, S, (int)splits, st) : launch<64, 1, 8>(ctx, a, S, (int)splits, st);
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_attention launch");
}
