// Lists of live tokens, 128 each, that one warp of a block makes from a session's map for the others, and the loads of
// their rows.
#pragma once

#include "pool_tokens.cuh"
#include "tc_common.cuh"

namespace {

// A bounded wait in few instructions, with one answer for the warp's lanes: the kernels of these lists have some twenty, and
// all their roles' code has to fit the instruction cache (with wait_warp in their places, 1.45 ms and not 1.15 ms for 2048
// tokens behind 32768).
__device__ __forceinline__ bool wait_short(uint64_t* b, uint32_t parity, Stop* stop, unsigned* err) {
    uint32_t t0 = 0;
    bool ok;
#pragma unroll 1
    while (!(ok = mbar_try(b, parity))) {
        uint32_t now;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
        now |= 1;
        if (!t0) t0 = now;
        if (stop->given_up) break;
        if (now - t0 > (uint32_t)stop->limit_ns) {
            stop->given_up = 1;
            atomicOr(err, (unsigned)KVSEL_DEV_TIMEOUT);
            break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

struct ListMeta {
    int n;          // tokens; 0 only where a piece has none
    int masked;     // not all of them are seen by every row, or there are fewer than 128
    int last;       // of its piece
};

// A ring of N lists.  slot, pos: the tokens in ascending positions; behind the n-th the slot of the first.
template <int N>
struct Lists {
    static constexpr int kAhead = 8;
    int slot[N * kTile], pos[N * kTile];
    int entry[32 * kAhead];             // the making warp's own
    ListMeta meta[N];
    uint64_t full[N], empty[N];
};

// Makes the lists of positions [p0, p1) of a session, at least one; pos0: where the first row that will look at them sits.
// A list is handed out when it is known whether another follows.  made: lists of the block so far.  The whole warp calls.
// The loop takes 32 positions a round and is not unrolled (with 8 rounds unrolled the code passed the instruction cache, and a
// round took 800 cycles); entries are read kAhead rounds at a time, while the ones before are gone through, and wait for
// their round in shared memory (a queue of registers would wait for its loads whenever it moves).
template <int N>
__device__ __forceinline__ bool make_lists(Lists<N>& t, const TokenMap& m, const int32_t* row, int p0, int p1, int pos0, uint32_t& made,
                                           int lane, Stop* stop, unsigned* err_word, unsigned& err) {
    constexpr int kAhead = Lists<N>::kAhead;
    const unsigned below = (1u << lane) - 1;
    uint32_t l = made;                  // the list that tokens go to, and how many it has
    int n = 0, j = p0 + lane;
    bool ok = l < N || wait_short(&t.empty[l % N], (l / N - 1) & 1, stop, err_word);
    int next[kAhead];
    auto read = [&](int p) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) next[k] = p + 32 * k < p1 ? raw_entry(m, row, p + 32 * k) : -1;
    };
    read(j);
    // hands out list l of n tokens
    auto hand_out = [&](int last) {
        __syncwarp();
        if (lane == 0) {
            t.meta[l % N] = ListMeta{n, n < kTile || t.pos[l % N * kTile + n - 1] > pos0, last};
            mbar_arrive(&t.full[l % N]);
        }
        ++l;
    };
    int round = kAhead;
#pragma unroll 1
    for (; ok && j - lane < p1; j += 32, ++round) {
        if (round == kAhead) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) t.entry[32 * k + lane] = next[k];
            if (p1 - (j - lane) > 32 * kAhead) read(j + 32 * kAhead);
            round = 0;
        }
        const int slot = live_slot(m, t.entry[32 * round + lane], j, err);
        const unsigned live = __ballot_sync(0xffffffffu, slot >= 0);
        if (!live) continue;
        int at = n + __popc(live & below);
        if (slot >= 0 && at < kTile) t.slot[l % N * kTile + at] = slot, t.pos[l % N * kTile + at] = j;
        n += __popc(live);
        if (n > kTile) {                // the list is full, and others follow
            const int rest = n - kTile;
            n = kTile;
            hand_out(0);
            ok = l < N || wait_short(&t.empty[l % N], (l / N - 1) & 1, stop, err_word);
            at -= kTile;
            if (ok && slot >= 0 && at >= 0) t.slot[l % N * kTile + at] = slot, t.pos[l % N * kTile + at] = j;
            n = rest;
        }
    }
    if (!ok) return false;
    __syncwarp();
    if (n > 0) {
        const int spare = t.slot[l % N * kTile];
        for (int e = n + lane; e < kTile; e += 32) t.slot[l % N * kTile + e] = spare;
    }
    hand_out(1);
    made = l;
    return true;
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
// The rows of a list's 128 slots, D dims from `base` on, to a tile of blocks of 64 dims in the layout of the 128-byte swizzle;
// by W warps, warp w of them a share, whose lanes signal `full` (a count of 32 W) when the rows have landed.  cp.async and not TMA gathers of four
// slots: those took 45 ns each from one thread, 6 us for a list's K and V.  The rows are written through the generic proxy:
// who has seen `full` fences before MMAs on them.
template <int D, int W>
__device__ __forceinline__ void load_rows(const __nv_bfloat16* base, uint32_t stride_bytes, const int* slots, const uint8_t* tile,
                                          uint64_t* full, int w, int lane) {
    constexpr int kChunks = D / 8, kRows = 32 / kChunks;  // 16-byte chunks of a row; rows of one instruction
    const int chunk = lane % kChunks, low = lane / kChunks;
    constexpr int kShare = kTile / W;
    const char* const from = reinterpret_cast<const char*>(base) + chunk * 16;
    const uint32_t to = saddr(tile) + (chunk >> 3) * (kTile * 128) + (kShare * w + low) * 128;
    const uint32_t swizzled = ((chunk & 7) ^ low) << 4;    // of row `low`; of row i + low, i a multiple of kRows: ^ (i & 7) << 4
    int slot[kShare / 32];
#pragma unroll
    for (int j = 0; j < kShare / 32; ++j) slot[j] = slots[kShare * w + 32 * j + lane];
#pragma unroll
    for (int i = 0; i < kShare; i += kRows) {
        const uint32_t s = __shfl_sync(0xffffffffu, slot[i / 32], i % 32 + low);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 128 + (swizzled ^ ((i & 7) << 4))),
                     "l"(from + (uint64_t)s * stride_bytes)
                     : "memory");
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(full)) : "memory");
}
// Rows that load_rows has written, and zeros written into them, come before the MMAs that follow.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace
