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
// The warps of a block take every kWarps-th chunk of 32 positions, the blocks of a
// cluster the same again, and the partial results are joined through shared and
// distributed shared memory in a fixed order: one launch, no workspace, no atomics.
#include <cuda_bf16.h>
#include <limits.h>

#include "kv4_format.cuh"
#include "kvsel_internal.h"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;   // tokens per stage
constexpr int kMaxSplit = 16;
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
    const int32_t* slot_map;
    const int32_t* table;
    int ld;                   // of slot_map or table
    int max_len;              // tokens that the map or table reaches
    int dead;
    int row_tiles;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
};

template <int D, int NT>
struct Cfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStages = D == 64 ? 3 : 2;  // two blocks per SM (D = 256: one)
    static constexpr int kCode = D / 2, kScale = D / kKv4Group;  // bytes per row
    static constexpr int kStage = kTile * 2 * (kCode + kScale);
    static constexpr int kKC = 0, kKS = kTile * kCode, kVC = kKS + kTile * kScale, kVS = kVC + kTile * kCode;
    struct Warp {
        uint64_t row[64];           // queue of live tokens: row index in the cache
        int pos[64];
        int stage_pos[kStages][kTile];
    };
    // the block's partial results, read by the other blocks of the cluster
    struct Part {
        float m[kRows], l[kRows];
        int nan_tail;
        float wm[kWarps][kRows], wl[kWarps][kRows];
        float o[kRows][D];
    };
    static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
    static constexpr size_t kMerge = (size_t)kWarps * kRows * D * 4;  // over the ring when the loop has ended
    static constexpr size_t kBuf = kRing > kMerge ? kRing : kMerge;
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The four bytes of w as pairs of fp16 values.
__device__ __forceinline__ void pairs4(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// fp16 scale of byte b in both halves; of bytes lo and hi in one half each.
__device__ __forceinline__ uint32_t scale2(uint32_t b) { return (b << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t scale2(uint32_t lo, uint32_t hi) { return (lo << 7) | (hi << 23); }

// Slot of token j, -1 where it is not live; bad slots set err.
__device__ __forceinline__ int slot_of(const AttnArgs& a, int s, int j, unsigned& err) {
    int slot;
    if (a.slot_map) {
        slot = __ldg(a.slot_map + (int64_t)s * a.ld + j);
    } else {
        const int b = a.page_shift >= 0 ? j >> a.page_shift : j / a.page;
        const int pg = __ldg(a.table + (int64_t)s * a.ld + b);
        if (pg < 0) return -1;
        if (pg >= a.P) {
            err |= KVSEL_DEV_BAD_PAGE;
            return -1;
        }
        slot = pg * a.page + (j - b * a.page);
    }
    if (slot < 0 || slot == a.dead) return -1;
    if ((int64_t)slot >= (int64_t)a.P * a.page) {
        err |= KVSEL_DEV_BAD_SLOT;
        return -1;
    }
    return slot;
}
__device__ __forceinline__ int64_t row_of(const AttnArgs& a, int slot, int g) {
    const int pg = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page;
    return ((int64_t)pg * a.Hkv + g) * a.page + (slot - pg * a.page);
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of p's counterpart in the cluster's block `rank`.
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float remote_f(const float* p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)) : "memory");
    return v;
}

// grid (splits, Hkv * row_tiles, S), clusters of (splits, 1, 1)
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (D == 128 && NT == 1) || D == 64 ? 2 : 1) kv4_attention_kernel(const AttnArgs a) {
    using C = Cfg<D, NT>;
    constexpr int kRows = C::kRows, kStages = C::kStages;
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

    // query fragments: lane (n = r, c) holds row n's dims 128 m + 32 c .. + 31 (D = 64: 16 c .. + 15)
    uint32_t qf[NT][KK][2];
    float cf[NT][2];                        // x = S * cf for the lane's rows 8 t + 2 c, + 1
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
                qf[t][k][i] = pack_half2(__uint_as_float(raw[k][i] << 16) * f, __uint_as_float(raw[k][i] & 0xFFFF0000u) * f);
        const float back = a.scale * kLog2e * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
        cf[t][0] = __shfl_sync(0xffffffffu, back, 8 * c);      // row 2 c's lanes start at 4 (2 c)
        cf[t][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
    }

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }

    // ---- the warp's stream of live tokens ----
    const int step = splits * kWarps * kTile;
    int j0 = (rank * kWarps + warp) * kTile;         // the chunk whose slots are in `next`
    int next = j0 + lane < len ? slot_of(a, s, j0 + lane, err) : -1;
    int head = 0, queued = 0;                        // ring queue of 64
    // Puts the next 32 live tokens (fewer at the end) on their way into stage st; their number.
    auto produce = [&](int st) {
        while (queued < kTile && j0 < len) {
            const int slot = next, j = j0 + lane;
            j0 += step;
            next = j0 + lane < len ? slot_of(a, s, j0 + lane, err) : -1;
            const unsigned live = __ballot_sync(0xffffffffu, slot >= 0);
            if (slot >= 0) {
                const int at = (head + queued + __popc(live & ((1u << lane) - 1))) & 63;
                w.row[at] = (uint64_t)row_of(a, slot, g);
                w.pos[at] = j;
            }
            queued += __popc(live);
        }
        __syncwarp();
        const int n = min(queued, kTile);
        if (n) {
            w.stage_pos[st][lane] = w.pos[(head + lane) & 63];
            const uint32_t base = saddr(ring + st * C::kStage);
            constexpr int kPer = C::kCode / 16;      // 16-byte pieces of a row's codes
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = k * 32 + lane, t = i / kPer, piece = i % kPer;
                const int64_t row = (int64_t)w.row[(head + t) & 63];
                const int64_t off = t < n ? row * C::kCode + piece * 16 : 0;
                copy_async<16>(base + C::kKC + i * 16, a.kc + off, t < n);
                copy_async<16>(base + C::kVC + i * 16, a.vc + off, t < n);
            }
            const int64_t off = lane < n ? (int64_t)w.row[(head + lane) & 63] * C::kScale : 0;
            copy_async<C::kScale>(base + C::kKS + lane * C::kScale, a.ks + off, lane < n);
            copy_async<C::kScale>(base + C::kVS + lane * C::kScale, a.vs + off, lane < n);
            head = (head + n) & 63;
            queued -= n;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        __syncwarp();
        return n;
    };

    const int perm = (r >> 1) + 4 * (r & 1);         // token of fragment row r in a tile of 16 (row r + 8: 8 more)
    auto consume = [&](int st, int n) {
        const uint8_t* const buf = ring + st * C::kStage;
        // S^T: two tiles of 16 tokens
        float x[NT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][u][0] = x[t][u][1] = x[t][u][2] = x[t][u][3] = 0.f;
            const int t0 = 16 * u + perm, t1 = t0 + 8;
#pragma unroll
            for (int mm = 0; mm < (D == 64 ? 1 : D / 128); ++mm) {
                constexpr int kWords = D == 64 ? 2 : 4;          // 32-bit words of codes per row and lane
                uint32_t w0[kWords], w1[kWords], s0, s1;
                if constexpr (D == 64) {
                    const uint2 v0 = *reinterpret_cast<const uint2*>(buf + C::kKC + t0 * C::kCode + 8 * c);
                    const uint2 v1 = *reinterpret_cast<const uint2*>(buf + C::kKC + t1 * C::kCode + 8 * c);
                    w0[0] = v0.x, w0[1] = v0.y, w1[0] = v1.x, w1[1] = v1.y;
                    s0 = buf[C::kKS + t0 * C::kScale + c];
                    s1 = buf[C::kKS + t1 * C::kScale + c];
                } else {
                    const uint4 v0 = *reinterpret_cast<const uint4*>(buf + C::kKC + t0 * C::kCode + 64 * mm + 16 * c);
                    const uint4 v1 = *reinterpret_cast<const uint4*>(buf + C::kKC + t1 * C::kCode + 64 * mm + 16 * c);
                    w0[0] = v0.x, w0[1] = v0.y, w0[2] = v0.z, w0[3] = v0.w;
                    w1[0] = v1.x, w1[1] = v1.y, w1[2] = v1.z, w1[3] = v1.w;
                    s0 = *reinterpret_cast<const uint16_t*>(buf + C::kKS + t0 * C::kScale + 8 * mm + 2 * c);
                    s1 = *reinterpret_cast<const uint16_t*>(buf + C::kKS + t1 * C::kScale + 8 * mm + 2 * c);
                }
#pragma unroll
                for (int i = 0; i < kWords; ++i) {               // a word is two steps of 4 dims per lane
                    const uint32_t sc0 = scale2(i < 2 ? s0 & 0xFFu : s0 >> 8), sc1 = scale2(i < 2 ? s1 & 0xFFu : s1 >> 8);
                    uint32_t h0[4], h1[4];
                    pairs4(w0[i], h0);
                    pairs4(w1[i], h1);
#pragma unroll
                    for (int b = 0; b < 4; ++b) h0[b] = mul2(h0[b], sc0), h1[b] = mul2(h1[b], sc1);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int kk = 8 * mm + 2 * i + k;
                            mma16816(x[t][u], h0[2 * k], h1[2 * k], h0[2 * k + 1], h1[2 * k + 1], qf[t][kk][0], qf[t][kk][1]);
                        }
                }
            }
        }
        // logits to base 2; what a row does not see becomes -inf
        bool tail = false;                           // the stage holds tokens that not every row sees
        if (a.Tq > 1) tail = __any_sync(0xffffffffu, lane < n && w.stage_pos[st][lane] > common);
        bool past = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[t][u][i] *= cf[t][i & 1];
            if (n < kTile || tail) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 16 * u + perm + (i >> 1) * 8;
                        const int row = row0 + 8 * t + 2 * c + (i & 1);
                        if (tok >= n || (tail && w.stage_pos[st][tok] > common + row / G)) x[t][u][i] = -INFINITY;
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float top = fmaxf(fmaxf(x[t][0][e], x[t][0][2 + e]), fmaxf(x[t][1][e], x[t][1][2 + e]));
                past |= top > m[t][e] + kSlack;
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
                    const float mn = fmaxf(m[t][e], top);
                    const float f = mn == -INFINITY ? 1.f : ex2(m[t][e] - mn);
                    m[t][e] = mn;
                    l[t][e] *= f;
#pragma unroll
                    for (int i = 0; i < MT; ++i) o[t][i][e] *= f, o[t][i][2 + e] *= f;
                }
        }
        uint32_t pf[NT][2][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float b0 = m[t][0] == -INFINITY ? 0.f : kHead - m[t][0], b1 = m[t][1] == -INFINITY ? 0.f : kHead - m[t][1];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float p0 = ex2(x[t][u][0] + b0), p1 = ex2(x[t][u][1] + b1);
                const float p2 = ex2(x[t][u][2] + b0), p3 = ex2(x[t][u][3] + b1);
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
                if (tail && w.stage_pos[st][tok] > common) {
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
                pairs4((vw[0][i] & kLow) | ((vw[1][i] << 4) & ~kLow), e01);
                pairs4(((vw[0][i] >> 4) & kLow) | (vw[1][i] & ~kLow), o01);
                pairs4((vw[2][i] & kLow) | ((vw[3][i] << 4) & ~kLow), e23);
                pairs4(((vw[2][i] >> 4) & kLow) | (vw[3][i] & ~kLow), o23);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t a0 = mul2(e01[b], s01), a1 = mul2(o01[b], s01), a2 = mul2(e23[b], s23), a3 = mul2(o23[b], s23);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(o[t][4 * i + b], a0, a1, a2, a3, pf[t][u][0], pf[t][u][1]);
                }
            }
        }
    };

    unsigned counts = 0;                             // tokens in each stage on its way, a byte each, oldest lowest
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) counts |= (unsigned)produce(st) << (8 * st);
    __syncthreads();                                 // nan_tail is set to 0
    for (int it = 0; counts & 0xFFu; ++it) {
        counts |= (unsigned)produce((it + kStages - 1) % kStages) << (8 * (kStages - 1));
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        consume(it % kStages, (int)(counts & 0xFFu));
        __syncwarp();
        counts >>= 8;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join: warps, then the cluster's blocks, in fixed order ----
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int k = 4; k <= 16; k <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], k);
            if (r == 0) {
                part.wm[warp][8 * t + 2 * c + e] = m[t][e];
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
            const float f = top == -INFINITY ? 0.f : ex2(m[t][e] - top);
            float* dst = merge + ((size_t)warp * kRows + n) * D + r * (D / 8);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[t][i][e] * f, o[t][i][2 + e] * f);
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
    for (int i = threadIdx.x; i < kRows * D; i += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum += merge[(size_t)k * kRows * D + i];
        part.o[i / D][i % D] = sum;
    }
    cluster_sync();
    // block `rank` finishes every splits-th pair of dims of the tile
    bool nan_tail = false;
    if (a.Tq > 1)
        for (int k = 0; k < splits; ++k) {
            int v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote(&part.nan_tail, k)) : "memory");
            nan_tail |= v != 0;
        }
    for (int i = (rank * kThreads + threadIdx.x) * 2; i < kRows * D; i += splits * kThreads * 2) {
        const int n = i / D, d = i % D, row = row0 + n;
        if (row >= R) break;
        float top = -INFINITY;
        for (int k = 0; k < splits; ++k) top = fmaxf(top, remote_f(&part.m[n], k));
        float sum = 0.f, v0 = 0.f, v1 = 0.f;
        for (int k = 0; k < splits; ++k) {
            const float f = top == -INFINITY ? 0.f : ex2(remote_f(&part.m[n], k) - top);
            sum = fmaf(remote_f(&part.l[n], k), f, sum);
            v0 = fmaf(remote_f(&part.o[n][d], k), f, v0);
            v1 = fmaf(remote_f(&part.o[n][d + 1], k), f, v1);
        }
        const int tok = row / G, h = g * G + row - tok * G;
        if (nan_tail) {
            for (int j = max(common + 1, 0); j <= common + tok; ++j) {
                const int slot = slot_of(a, s, j, err);
                if (slot >= 0 && __ldg(a.vs + row_of(a, slot, g) * C::kScale + d / kKv4Group) == kKv4NanByte)
                    v0 = v1 = __int_as_float(0x7FC00000);
            }
        }
        const int64_t at = ((int64_t)s * a.Tq + tok) * a.Hq + h;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<__nv_bfloat162*>(a.out + at * D + d) = __floats2bfloat162_rn(v0 * inv, v1 * inv);
        if (a.lse && d == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top - kHead + log2f(sum)) * kLn2;
    }
    cluster_sync();                                  // no block leaves while others read its results
    if (err) atomicOr(a.err, err);
}

template <int D, int NT>
cudaError_t launch(const AttnArgs& a, int S, int splits, cudaStream_t s) {
    using C = Cfg<D, NT>;
    auto* kernel = kv4_attention_kernel<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, a.Hkv * a.row_tiles, S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
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
    const AttnArgs a{(const __nv_bfloat16*)q, q_stride, Tq, Hq, Hkv, k_codes, k_scales, v_codes, v_scales, P, page, shift,
                     seq_lens, slot_map, block_table, ld, (int)reach, dead_slot, tiles, scale, (__nv_bfloat16*)out, lse,
                     ctx->dev_err};
    // splits of the tokens over a cluster: enough blocks for two per SM, at least one chunk of 32 tokens per warp
    int splits = 1;
    while (splits < kMaxSplit && (int64_t)S * Hkv * tiles * splits < 2 * ctx->num_sms && (int64_t)splits * kThreads < reach)
        splits *= 2;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = D == 64    ? (wide ? launch<64, 2>(a, S, splits, st) : launch<64, 1>(a, S, splits, st))
                          : D == 128 ? (wide ? launch<128, 2>(a, S, splits, st) : launch<128, 1>(a, S, splits, st))
                                     : launch<256, 1>(a, S, splits, st);
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_attention launch");
}
