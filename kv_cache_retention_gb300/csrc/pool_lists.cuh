// Lists of live tokens, 128 each, that one warp of a block makes from a session's map for the others, and the loads of
// their rows.
#pragma once

#include <limits.h>

#include "pool_tokens.cuh"
#include "tc_common.cuh"

namespace {

constexpr unsigned kIdleNs = 100;

// Bounded waits in few instructions, of a lane and with one answer for the warp's lanes: the kernels of these lists have some
// twenty, and all their roles' code has to fit the instruction cache (with wait_warp in their places, 1.45 ms and not 1.15 ms for
// 2048 tokens behind 32768).  The clock and the other roles' giving up are looked at once in 64 tries: looked at each time, by
// all who wait, they took a fifth of the kernel's instructions.
__device__ __forceinline__ bool gives_up(uint32_t& tries, uint32_t& t0, Stop* stop, unsigned* err) {
    if (++tries & 63) return false;
    uint32_t now;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
    now |= 1;
    if (!t0) t0 = now;
    if (stop->given_up) return true;
    if (now - t0 <= (uint32_t)stop->limit_ns) return false;
    stop->given_up = 1;
    atomicOr(err, (unsigned)KVSEL_DEV_TIMEOUT);
    return true;
}
__device__ __forceinline__ bool wait_lane(uint64_t* b, uint32_t parity, Stop* stop, unsigned* err) {
    uint32_t t0 = 0, tries = 0;
#pragma unroll 1
    while (!mbar_try(b, parity))
        if (gives_up(tries, t0, stop, err)) return false;
    return true;
}
// For those that nothing waits for at once: they ask less often, since each try takes its turn at shared memory.
__device__ __forceinline__ bool wait_idle(uint64_t* b, uint32_t parity, Stop* stop, unsigned* err) {
    uint32_t t0 = 0, tries = 0;
    bool ok = true;
#pragma unroll 1
    while (!mbar_try(b, parity)) {
        __nanosleep(kIdleNs);
        if (gives_up(tries, t0, stop, err)) {
            ok = false;
            break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_short(uint64_t* b, uint32_t parity, Stop* stop, unsigned* err) {
    return __all_sync(0xffffffffu, wait_lane(b, parity, stop, err));
}

// wait_lane for two or four phases at once, whose answers come in the time of one: next to MMAs, which take all of shared memory's
// bandwidth, an answer takes some hundred cycles.
__device__ __forceinline__ bool wait_lane2(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, Stop* stop, unsigned* err) {
    uint32_t t0 = 0, tries = 0;
#pragma unroll 1
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p, q;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4, 20000;\n"
            " and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(saddr(b0)), "r"(p0), "r"(saddr(b1)), "r"(p1)
            : "memory");
        if (done) return true;
        if (gives_up(tries, t0, stop, err)) return false;
    }
}
__device__ __forceinline__ bool wait_lane4(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t* b2, uint32_t p2, uint64_t* b3,
                                           uint32_t p3, Stop* stop, unsigned* err) {
    uint32_t t0 = 0, tries = 0;
#pragma unroll 1
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p, q, r, s;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4, 20000;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6, 20000;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 s, [%7], %8, 20000;\n"
            " and.pred p, p, q;\n and.pred r, r, s;\n and.pred p, p, r;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(saddr(b0)), "r"(p0), "r"(saddr(b1)), "r"(p1), "r"(saddr(b2)), "r"(p2), "r"(saddr(b3)), "r"(p3)
            : "memory");
        if (done) return true;
        if (gives_up(tries, t0, stop, err)) return false;
    }
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int k = 16; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
    return v;
}

constexpr int kRun = 16;            // slots that one TMA load brings where they are consecutive

struct ListMeta {
    int n;          // tokens; 0 only where a piece has none
    int causal;     // not all of them are seen by every row
    int last;       // of its piece
    int first;      // position of its first token
    unsigned runs;  // of each four tokens, whether all are there and go on a run of slots that starts with their kRun; a bit each
};

// A ring of N lists.  token: slot and position, in ascending positions; behind the n-th the slot of the first.
template <int N>
struct alignas(16) Lists {
    static constexpr int kAhead = 4;    // rounds whose entries are on their way
    int2 token[N * kTile];
    int entry[kAhead * kTile];          // the making warp's own
    ListMeta meta[N];
    uint64_t full[N], empty[N];
    volatile int progress[2];           // of the piece whose lists are made (by its number's parity): 2 * lists handed out + whether those are all
};

// Makes the lists of positions [p0, p1) of a session, at least one; pos0: where the first row that will look at them sits.
// A list is handed out when it is known whether another follows.  made: lists of the block so far.  The whole warp calls.
// MAP: a slot map, not a block table.
// A round takes 128 positions, four of each lane (with one of each lane and 32 a round, the chain of dependent instructions
// took 640 cycles for those), and is not unrolled, for the instruction cache's sake.  Entries come through cp.async, kAhead
// rounds ahead of their use.
template <bool MAP, int N>
__device__ __forceinline__ bool make_lists(Lists<N>& t, const TokenMap& m, const int32_t* row, int p0, int p1, int pos0, uint32_t& made,
                                           volatile int* progress, int lane, Stop* stop, unsigned* err_word, unsigned& err) {
    constexpr int kAhead = Lists<N>::kAhead;
    const unsigned below = (1u << lane) - 1;
    uint32_t l = made;                  // the list that tokens go to, and how many it has
    int n = 0;
    bool ok = l < N || wait_idle(&t.empty[l % N], (l / N - 1) & 1, stop, err_word);
    const bool wide = MAP && (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    auto read = [&](int p, int at) {    // (nothing is read behind p1)
        const int j = p + 4 * lane;
        const uint32_t to = saddr(&t.entry[at * kTile + 4 * lane]);
        if (wide) {
            if (j < p1)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(row + j), "r"(4 * min(4, p1 - j)) : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < p1)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * k), "l"(row + (MAP ? j + k : entry_of(m, j + k)))
                                 : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int k = 0; k < kAhead - 1; ++k) read(p0 + k * kTile, k);
    // hands out list l of n tokens
    auto hand_out = [&](int last) {
        __syncwarp();
        const int2* const list = &t.token[l % N * kTile];
        const int4 s01 = *reinterpret_cast<const int4*>(list + 4 * lane), s23 = *reinterpret_cast<const int4*>(list + 4 * lane + 2);
        const int first = list[(lane & ~(kRun / 4 - 1)) * 4].x, off = 4 * (lane % (kRun / 4));
        // (places behind the n-th token are in no run: their rows are to be zeros)
        const bool run = 4 * lane + 3 < n && s01.x == first + off && s01.z == s01.x + 1 && s23.x == s01.x + 2 && s23.z == s01.x + 3;
        const unsigned runs = __ballot_sync(0xffffffffu, run);
        if (lane == 0) {
            t.meta[l % N] = ListMeta{n, n > 0 && list[n - 1].y > pos0, last, list[0].y, runs};
            mbar_arrive(&t.full[l % N]);
            *progress = 2 * (int)(l - made + (n > 0)) + last;
        }
        ++l;
    };
    int round = 0;
#pragma unroll 1
    for (int p = p0; ok && p < p1; p += kTile) {
        read(p1 - p > (kAhead - 1) * kTile ? p + (kAhead - 1) * kTile : p1, (round + kAhead - 1) % kAhead);
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");  // (a lane reads what it has copied itself)
        const int4 entry = *reinterpret_cast<const int4*>(&t.entry[round * kTile + 4 * lane]);
        round = (round + 1) % kAhead;
        const int j = p + 4 * lane;
        int slot[4] = {entry.x, entry.y, entry.z, entry.w}, at[4];
        int before = n, more = 0, mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            slot[k] = j + k < p1 ? live_slot<MAP>(m, slot[k], j + k, err) : -1;
            const unsigned live = __ballot_sync(0xffffffffu, slot[k] >= 0);
            before += __popc(live & below);
            more += __popc(live);
            at[k] = mine;
            mine += slot[k] >= 0;
        }
        int2* const list = &t.token[l % N * kTile];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            at[k] += before;
            if (slot[k] >= 0 && at[k] < kTile) list[at[k]] = make_int2(slot[k], j + k);
        }
        n += more;
        if (n > kTile) {                // the list is full, and others follow
            const int rest = n - kTile;
            n = kTile;
            hand_out(0);
            if (l >= N) ok = wait_idle(&t.empty[l % N], (l / N - 1) & 1, stop, err_word);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (ok && slot[k] >= 0 && at[k] >= kTile) t.token[l % N * kTile + at[k] - kTile] = make_int2(slot[k], j + k);
            n = rest;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok) return false;
    __syncwarp();
    if (n > 0) {
        const int spare = t.token[l % N * kTile].x;
        __syncwarp();
        for (int e = n + lane; e < kTile; e += 32) t.token[l % N * kTile + e].x = spare;
    }
    hand_out(1);
    made = l;
    return true;
}

// Rows of a pool as TMA sees them: 64 dims of kRun consecutive slots.
inline bool make_pool_map(CUtensorMap* map, const void* base, int n_slots, int Hkv, int D, int64_t stride) {
    auto fn = kvsel_tmap_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)Hkv * D, (cuuint64_t)n_slots};
    cuuint64_t strides[1] = {(cuuint64_t)(n_slots > 1 ? stride : (int64_t)Hkv * D) * 2};
    cuuint32_t box[2] = {64, kRun};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Query rows [T][Hq][D]: 64 dims of `heads` heads of `tokens` tokens a load, zeros behind the last token.
inline bool make_query_map(CUtensorMap* map, const void* base, int T, int Hq, int D, int64_t stride, int heads, int tokens) {
    auto fn = kvsel_tmap_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)(T > 1 ? stride : (int64_t)Hq * D) * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The rows of a list's 128 slots, D dims from dim x of a slot on, to a tile of blocks of 64 dims in the layout of the 128-byte
// swizzle; by W warps, warp w of them a share, whose lanes signal `full` (a count of 32 W) when the rows have landed.  Runs of
// kRun slots come by TMA, others row by row through cp.async (TMA gathers of four slots took 45 ns each from one thread, 6 us for a list's K and V).
// Such rows are written through the generic proxy: who has seen `full` fences before MMAs on them.  Rows behind the n-th token
// are zeros.
template <int D, int W>
__device__ __forceinline__ void load_rows(const CUtensorMap* map, const __nv_bfloat16* pool, uint32_t stride_bytes, int x, const int2* tokens,
                                          int n, unsigned runs, const uint8_t* tile, uint64_t* full, int w, int lane) {
    constexpr int kChunks = D / 8, kRows = 32 / kChunks;  // 16-byte chunks of a row; rows of one instruction
    const int chunk = lane % kChunks, low = lane / kChunks;
    const char* const from = reinterpret_cast<const char*>(pool + x) + chunk * 16;
    const uint32_t to = saddr(tile) + (chunk >> 3) * (kTile * 128) + low * 128;
    const uint32_t swizzled = ((chunk & 7) ^ low) << 4;    // of row `low`; of row i + low, i a multiple of kRows: ^ (i & 7) << 4
    constexpr unsigned kAll = (1u << kRun / 4) - 1;
    // the runs, a lane each
    const bool run = lane < kTile / kRun && (runs >> (lane * (kRun / 4)) & kAll) == kAll;
    const unsigned by_tma = __ballot_sync(0xffffffffu, run);
    if (run && (W == 1 || lane / (kTile / kRun / W) == w)) {
        const int first = tokens[lane * kRun].x;
        const uint32_t dst = saddr(tile) + lane * (kRun * 128);
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(saddr(full)), "r"(kRun * D * 2) : "memory");
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                    dst + b * (kTile * 128)),
                "l"(reinterpret_cast<uint64_t>(map)), "r"(saddr(full)), "r"(x + 64 * b), "r"(first)
                : "memory");
    }
    if (by_tma != (1u << kTile / kRun) - 1) {
#pragma unroll 1
        for (int r = w * (kTile / W); r < (w + 1) * (kTile / W); r += 32) {
            const int slot = tokens[r + lane].x;
#pragma unroll
            for (int i = 0; i < 32; i += kRows) {
                const uint32_t s = __shfl_sync(0xffffffffu, slot, i + low);
                if (!(by_tma >> ((r + i) / kRun) & 1))
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (r + i) * 128 + (swizzled ^ ((i & 7) << 4))),
                                 "l"(from + (uint64_t)s * stride_bytes), "r"(r + i + low < n ? 16 : 0)
                                 : "memory");
            }
        }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(full)) : "memory");
}
// Rows that load_rows has written, and zeros written into them, come before the MMAs that follow.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace
