// kvsel_evict_slots: eviction of the tokens of least score from the slot maps of sessions above their budget.
//
// Session s of n = seq_lens[s] tokens holds L live ones (slot not negative, not dead_slot); those at positions in
// [n_sink, n - n_recent) may leave.  E = min(max(L - budget, 0), how many may leave, room in the list) do: the ones of
// least score, of equal scores the later position, a NaN before any number.
//
// The E-th least score is found by radix selection on the scores' bits (11, 11 and 10 of them), the keys held in
// shared memory after one pass over scores and slots.  A session is worked on by a thread-block cluster that shares its
// positions; histograms and counts are read from the other blocks' shared memory.  Warps own contiguous positions, so
// the places of the evicted in the list follow from each warp's count of smaller and of equal keys.
// Measured: a token each of 36 sessions of up to 8192 positions 14 us, a tenth kept of 92160 25 us (latency: the passes of
// a cluster), a fifth of 64 sessions of up to 92160 evicted 50 us (28 M instructions, 58% of issue slots, DRAM 10%).
#include <cooperative_groups.h>

#include <limits.h>

#include "kvsel_internal.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048;
static_assert(kBins == 4 * kThreads && kWarps <= 32, "four bins a thread, a warp for the warps' sums");
constexpr int kBatch = 8;     // positions of a lane whose loads are in flight at once
constexpr int kHeld = 32768;  // keys of a block that shared memory holds
constexpr uint32_t kStays = 0xFFFFFFFFu;  // key of a token that may not leave; no score has it

struct EvictArgs {
    const float* score;
    int64_t score_ld;
    const int32_t *lens, *budget, *map;
    int ld, dead, n_sink, n_recent;
    int32_t *out, *freed, *n_freed;
    int room;              // row length of freed
    unsigned* err;
};

// Scores in the order of eviction: NaN, then ascending; -0 and 0 alike.
__device__ __forceinline__ uint32_t key_of(float f) {
    if (f != f) return 0u;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Shared {
    alignas(16) unsigned hist[2][kBins];   // two, so that a pass clears one while others still read the last
    unsigned live, may;        // this block's counts
    unsigned less, equal;      // of its keys below the threshold, and at it
    unsigned warp_less[kWarps], warp_equal[kWarps];
    unsigned scan[kWarps];
    unsigned digit, before;    // the digit that holds the wanted rank, and the keys of lower digits
};

// HELD: the block's keys stay in shared memory; else scores and slots are read again for each pass.
template <bool HELD>
__global__ void __launch_bounds__(kThreads, 3) evict_slots_kernel(const EvictArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int c = (int)cluster.num_blocks(), r = (int)cluster.block_rank(), s = (int)(blockIdx.x / c);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int length = __ldg(a.lens + s), n = min(max(length, 0), a.ld);
    if (r == 0 && tid == 0 && n != length) atomicOr(a.err, (unsigned)KVSEL_DEV_BAD_LENGTH);
    // this block's positions [p0, p1), this warp's [w0, w1)
    const int per = (int)(((int64_t)a.ld + (int64_t)c * kWarps - 1) / ((int64_t)c * kWarps) + 31) & ~31;
    const int64_t base = (int64_t)r * kWarps * per;
    const int w0 = (int)min((int64_t)a.ld, base + (int64_t)warp * per), w1 = (int)min((int64_t)a.ld, base + (int64_t)(warp + 1) * per);
    const float* const score = a.score + s * a.score_ld;
    const int32_t* const in = a.map + (int64_t)s * a.ld;
    int32_t* const out = a.out + (int64_t)s * a.ld;

    auto key_from = [&](int p, int slot, float value) {  // of a position below n
        return slot >= 0 && slot != a.dead && p >= a.n_sink && p < n - a.n_recent ? key_of(value) : kStays;
    };
    auto key_at = [&](int p) {
        return HELD ? keys[p - (int)base] : p < n ? key_from(p, in[p], score[p]) : kStays;
    };
    for (int i = tid; i < 2 * kBins; i += kThreads) sh.hist[0][i] = 0;
    if (tid == 0) sh.live = sh.may = 0;
    __syncthreads();
    unsigned n_live = 0, n_may = 0;
    for (int q = w0 + lane; q < w1; q += 32 * kBatch) {
        int slot[kBatch];
        float value[kBatch];            // (of dead tokens too: its load does not wait for the slot's)
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int p = q + 32 * k;
            slot[k] = p < min(n, w1) ? in[p] : -1;
            value[k] = p < min(n, w1) ? score[p] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int p = q + 32 * k;
            if (p >= w1) break;
            const uint32_t key = key_from(p, slot[k], value[k]);
            if (HELD) keys[p - (int)base] = key;
            n_live += slot[k] >= 0 && slot[k] != a.dead;
            n_may += key != kStays;
            if (key != kStays) atomicAdd(&sh.hist[0][key >> 21], 1u);
        }
    }
    n_live = __reduce_add_sync(0xffffffffu, n_live);
    n_may = __reduce_add_sync(0xffffffffu, n_may);
    if (lane == 0) atomicAdd(&sh.live, n_live), atomicAdd(&sh.may, n_may);
    cluster.sync();
    unsigned live = 0, may = 0;
    for (int b = 0; b < c; ++b) {
        const Shared* const o = cluster.map_shared_rank(&sh, b);
        live += o->live;
        may += o->may;
    }
    const int64_t over = (int64_t)live - __ldg(a.budget + s);
    const unsigned leave = (unsigned)min(min(max(over, (int64_t)0), (int64_t)may), (int64_t)a.room);

    // ---- the key of rank leave - 1 ----
    uint32_t threshold = 0;
    unsigned rank = leave;        // of the keys with the digits found so far, how many leave
    if (leave) {                  // the same in every block of the cluster
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
            unsigned* const hist = sh.hist[pass & 1];
            if (pass) {
                const uint32_t above = pass == 1 ? 21 : 10;
#pragma unroll 4
                for (int p = w0 + lane; p < w1; p += 32) {
                    const uint32_t key = key_at(p);
                    if (key != kStays && key >> above == threshold >> above) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
                }
                cluster.sync();
            }
            // four bins a thread, summed over the blocks; then the digit that holds the rank
            uint4 x = make_uint4(0, 0, 0, 0);
            if (4 * tid < bins) {
#pragma unroll 4
                for (int b = 0; b < c; ++b) {
                    const uint4 v = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, b) + 4 * tid);
                    x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
                }
            }
            const unsigned all = x.x + x.y + x.z + x.w;
            unsigned upto = all;
#pragma unroll
            for (int k = 1; k < 32; k *= 2) {
                const unsigned y = __shfl_up_sync(0xffffffffu, upto, k);
                if (lane >= k) upto += y;
            }
            if (lane == 31) sh.scan[warp] = upto;
            __syncthreads();
            // (every warp adds up the warps before it)
            unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[lane] : 0u) + upto - all;
            const unsigned bin[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (before < rank && rank <= before + bin[k]) sh.digit = 4 * tid + k, sh.before = before;
                before += bin[k];
            }
            if (pass == 1)        // (the blocks have read this one: a sync of the cluster lies between)
                for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
            __syncthreads();
            threshold |= sh.digit << shift;
            rank -= sh.before;
        }
    }
    // ---- who leaves, and where it stands in the list ----
    unsigned w_less = 0, w_equal = 0;
    if (leave)
#pragma unroll 4
        for (int p = w0 + lane; p < w1; p += 32) {
            const uint32_t key = key_at(p);
            w_less += key < threshold;
            w_equal += key == threshold;
        }
    w_less = __reduce_add_sync(0xffffffffu, w_less);
    w_equal = __reduce_add_sync(0xffffffffu, w_equal);
    if (lane == 0) sh.warp_less[warp] = w_less, sh.warp_equal[warp] = w_equal;
    __syncthreads();
    unsigned less = 0, equal = 0, b_equal = 0;   // before this warp's positions; b_equal: of the whole session
    {
        const unsigned l = lane < kWarps ? sh.warp_less[lane] : 0u, e = lane < kWarps ? sh.warp_equal[lane] : 0u;
        less = __reduce_add_sync(0xffffffffu, lane < warp ? l : 0u);
        equal = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0u);
        const unsigned all_l = __reduce_add_sync(0xffffffffu, l), all_e = __reduce_add_sync(0xffffffffu, e);
        if (tid == 0) sh.less = all_l, sh.equal = all_e;
    }
    cluster.sync();
    for (int b = 0; b < c; ++b) {
        const Shared* const o = cluster.map_shared_rank(&sh, b);
        if (b < r) less += o->less, equal += o->equal;
        b_equal += o->equal;
    }
    cluster.sync();               // no block ends, and its shared memory with it, while another reads it
    const unsigned spared = leave ? b_equal - rank : 0u;  // the first `spared` of the keys at the threshold stay
    const unsigned below = (1u << lane) - 1;
    int32_t* const freed = a.freed ? a.freed + (int64_t)s * a.room : nullptr;
    for (int q = w0; q < w1; q += 32 * kBatch) {
        int slot[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) slot[k] = q + 32 * k + lane < w1 ? in[q + 32 * k + lane] : 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int p = q + 32 * k + lane;
            const uint32_t key = leave && p < w1 ? key_at(p) : kStays;
            const unsigned lm = __ballot_sync(0xffffffffu, leave && key < threshold);
            const unsigned em = __ballot_sync(0xffffffffu, leave && key == threshold && key != kStays);
            if (p < w1) {
                const unsigned eq = equal + __popc(em & below);
                const bool gone = (lm >> lane & 1) || ((em >> lane & 1) && eq >= spared);
                if (gone && freed) freed[less + __popc(lm & below) + (eq > spared ? eq - spared : 0u)] = slot[k];
                out[p] = gone ? a.dead : slot[k];
            }
            less += __popc(lm);
            equal += __popc(em);
        }
    }
    if (freed)
        for (int64_t i = (int64_t)leave + (int64_t)r * kThreads + tid; i < a.room; i += (int64_t)c * kThreads) freed[i] = -1;
    if (a.n_freed && r == 0 && tid == 0) a.n_freed[s] = (int)leave;
}

}  // namespace

extern "C" int kvsel_evict_slots(kvsel_ctx* ctx, const float* score, int64_t score_ld, const int32_t* seq_lens,
                                 const int32_t* budget, int S, const int32_t* slot_map, int ld, int32_t dead_slot, int n_sink,
                                 int n_recent, int32_t* slot_out, int32_t* freed, int ld_freed, int32_t* n_freed, void* stream) {
    const kvsel_trace trace_("kvsel_evict_slots");
    const kvsel_device_scope scope_;
    const int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (S < 0 || ld < 0 || ld_freed < 0 || n_sink < 0 || n_recent < 0)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "evict_slots: bad sizes");
    if (S > 65535 || ld > INT_MAX - (1 << 20)) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "evict_slots: S or ld too large");
    if (score_ld < ld) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "evict_slots: score rows shorter than the maps'");
    if (!freed && ld_freed) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "evict_slots: ld_freed without freed");
    if (S == 0) return KVSEL_OK;
    if (!seq_lens || !budget || (ld > 0 && (!score || !slot_map || !slot_out)))
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "evict_slots: null pointer");
    if (!(ctx->ready & KVSEL_READY_EVICT)) {
        const cudaError_t e = cudaFuncSetAttribute(evict_slots_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4);
        if (e != cudaSuccess) return kvsel_cuda_fail(ctx, e, "evict_slots set-up");
        ctx->ready |= KVSEL_READY_EVICT;
    }
    // A cluster as large as keeps all sessions' blocks on the GPU at once, three an SM, and leaves a thread four positions.  (Three
    // fit while a block holds 14000 keys or fewer; of longer rows one or two do, and many such sessions take several rounds.)
    int c = 1;
    while (c < 8 && 2 * (int64_t)S * c <= 3 * ctx->num_sms && ld > c * 4 * kThreads) c *= 2;
    const int64_t per = (((int64_t)ld + c * kWarps - 1) / (c * kWarps) + 31) & ~31;
    const bool held = per * kWarps <= kHeld;
    const EvictArgs a{score, score_ld, seq_lens, budget, slot_map, ld, dead_slot, n_sink, n_recent, slot_out, freed, n_freed,
                      freed ? ld_freed : INT_MAX, ctx->dev_err};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S * c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = held ? (size_t)per * kWarps * 4 : 0;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, held ? evict_slots_kernel<true> : evict_slots_kernel<false>, a);
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "evict_slots launch");
}
