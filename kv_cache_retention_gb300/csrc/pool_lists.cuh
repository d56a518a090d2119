// Lists of live tokens, 128 each, that one warp of a block makes from a session's map for the others, and the loads of
// their rows.
#pragma once

#include "pool_tokens.cuh"
#include "tc_common.cuh"

namespace {

struct ListMeta {
    int n;          // tokens; 0 only where a piece has none
    int masked;     // not all of them are seen by every row, or there are fewer than 128
    int last;       // of its piece
};

// A ring of N lists.  slot, pos: the tokens in ascending positions; behind the n-th the slot of the first.
template <int N>
struct Lists {
    static constexpr int kEntries = N * kTile;
    int slot[kEntries], pos[kEntries];
    ListMeta meta[N];
    uint64_t full[N], empty[N];
};

// Makes the lists of positions [p0, p1) of a session, at least one; pos0: where the first row that will look at them sits.
// A list is handed out when it is known whether another follows.  made: lists of the block so far.  The whole warp calls.
template <int N>
__device__ __forceinline__ bool make_lists(Lists<N>& t, const TokenMap& m, const int32_t* row, int p0, int p1, int pos0, uint32_t& made,
                                           int lane, Stop* stop, unsigned* err_word, unsigned& err) {
    constexpr int kBatch = 8;           // entries in flight per lane, read ahead of their use
    int tail = 0, out = 0, ready = 0;   // tokens, lists handed out, lists whose places are free
    bool ok = true;
    const unsigned below = (1u << lane) - 1;
    auto place = [&](int e) { return (made % N * kTile + (uint32_t)e) % (uint32_t)Lists<N>::kEntries; };
    auto reserve = [&](int lists) {
        for (; ok && ready < lists; ++ready) {
            const uint32_t l = made + ready;
            if (l >= N) ok = wait_warp(&t.empty[l % N], (l / N - 1) & 1, stop, err_word);
        }
    };
    auto hand_out = [&](int n, bool last) {
        const uint32_t l = (made + out) % N;
        __syncwarp();
        if (lane == 0) {
            t.meta[l] = ListMeta{n, n < kTile || t.pos[place(out * kTile + n - 1)] > pos0, last};
            mbar_arrive(&t.full[l]);
        }
        ++out;
    };
    int next[kBatch];
    auto read = [&](int p) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) next[k] = p + 32 * k + lane < p1 ? raw_entry(m, row, p + 32 * k + lane) : -1;
    };
    read(p0);
    for (int p = p0; ok && p < p1; p += 32 * kBatch) {
        int entry[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) entry[k] = next[k];
        if (p1 - p > 32 * kBatch) read(p + 32 * kBatch);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int j = p + 32 * k + lane, slot = live_slot(m, entry[k], j, err);
            const unsigned live = __ballot_sync(0xffffffffu, slot >= 0);
            if (!live) continue;
            const int n = __popc(live);
            if (ready * kTile < tail + n) reserve((tail + n - 1) / kTile + 1);
            if (!ok) break;
            if (slot >= 0) {
                const uint32_t at = place(tail + __popc(live & below));
                t.slot[at] = slot, t.pos[at] = j;
            }
            tail += n;
            if (tail > (out + 1) * kTile) hand_out(kTile, false);
        }
    }
    if (ok) reserve(out + 1);
    if (!ok) return false;
    const int rest = tail - out * kTile;
    if (rest > 0) {
        __syncwarp();
        const int spare = t.slot[place(out * kTile)];
        for (int e = rest + lane; e < kTile; e += 32) t.slot[place(out * kTile + e)] = spare;
        hand_out(rest, true);
    } else {
        if (lane == 0) {
            t.meta[(made + out) % N] = ListMeta{0, 1, 1};
            mbar_arrive(&t.full[(made + out) % N]);
        }
        ++out;
    }
    made += out;
    return true;
}

// Rows of a pool as TMA sees them: 64 dims of one slot; four slots a load.
inline bool make_pool_map(CUtensorMap* map, const void* base, int n_slots, int Hkv, int D, int64_t stride) {
    auto fn = kvsel_tmap_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)Hkv * D, (cuuint64_t)n_slots};
    cuuint64_t strides[1] = {(cuuint64_t)(n_slots > 1 ? stride : (int64_t)Hkv * D) * 2};
    cuuint32_t box[2] = {64, 1};
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
// Dims [x, x + 64) of four slots' rows.
__device__ __forceinline__ void tma_gather(const CUtensorMap* map, uint32_t bar, uint32_t dst, int x, int4 s) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, "
        "%7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(s.x), "r"(s.y), "r"(s.z), "r"(s.w)
        : "memory");
}
// 128 slots' rows of D dims from dim x on, as blocks of 64 dims; one thread calls, the bytes are expected by bar.
template <int D>
__device__ __forceinline__ void load_rows(const CUtensorMap* map, uint64_t* bar, const uint8_t* dst, int x, const int* slots) {
    const uint32_t b = saddr(bar), to = saddr(dst);
#pragma unroll 4
    for (int i = 0; i < kTile / 4; ++i) {
        const int4 s = *reinterpret_cast<const int4*>(slots + 4 * i);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) tma_gather(map, b, to + d * (kTile * 128) + i * 512, x + 64 * d, s);
    }
}

}  // namespace
