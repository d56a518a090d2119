// What the two kernels of kvsel_pool_attention share.
#pragma once

#include "pool_lists.cuh"

namespace {

constexpr float kSlack = 8.f;           // how far (log2) a row's maximum may pass its reference

// All of TMEM is allocated, so its base is column 0.
constexpr uint32_t kTmem = 0;
constexpr int kColS = 0, kColO = 256, kTmemCols = 512;

// What a block has of a unit that others share: O as [D/4][128 rows] of four dims, then references and sums; per tile.
constexpr int kPartTile = kTile * (128 + 2), kPart = 2 * kPartTile;

// A unit that several shares have a part of, kept with the block that has its first keys; sharers 0: none.
struct Joint {
    int sharers, row, tokens;           // row, tokens: its first token in q, and how many
};

struct PoolArgs {
    const int32_t *cu, *lens;
    int S, T, Hq, Hkv, G;
    int tile_tokens;                    // tokens of a tile
    int few;                            // sessions of up to as many new tokens are the other kernel's
    const __nv_bfloat16 *k, *v;
    uint32_t k_bytes, v_bytes;          // from a slot's rows to the next one's
    TokenMap map;
    float scale2;                       // scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
    int shares;
    float* parts;                       // [blocks][2]: of a unit that began before the share, and of one that goes on behind it
    Joint* joints;                      // [blocks]
    uint64_t wait_ns;                   // how long a wait goes on
    int stuck;                          // tile 0's issuer waits for what never comes (test entry)
};

// What a row sees of V's values that were set to zero in lists that not every row sees whole: put(d, sum) for the dims whose
// sum, of infinities and NaN, is one.  from: the first key of such a list; upto: the last key that the lane's row sees, -1
// for none.  The whole warp calls, a row a lane: its lanes read the map 32 positions at a time and look at each live token's row
// together, eight dims in a walk, since such a list may span a whole session of which little is live.
template <int D, bool MAP, class Put>
__device__ __forceinline__ void add_odd(const PoolArgs& a, int session, int head, int from, int upto, int lane, Put put) {
    unsigned err = 0;                   // (what is wrong with the map has been said)
    const int32_t* const map = a.map.map + (int64_t)session * a.map.ld;
    const __nv_bfloat16* const v = a.v + (int64_t)head * D;
    const int end = __reduce_max_sync(0xffffffffu, upto);
#pragma unroll 1
    for (int d = 0; d < D; d += 8) {
        float add[8] = {};
#pragma unroll 1
        for (int p = from; p <= end; p += 32) {
            const int j = p + lane;
            const int slot = j <= end ? live_slot<MAP>(a.map, raw_entry(a.map, map, j), j, err) : -1;
#pragma unroll 1
            for (unsigned live = __ballot_sync(0xffffffffu, slot >= 0); live; live &= live - 1) {
                const int k = __ffs(live) - 1;
                const uint32_t s = __shfl_sync(0xffffffffu, slot, k);
                const uint4 y = *reinterpret_cast<const uint4*>(v + (uint64_t)s * (a.v_bytes / 2) + d);
                const uint32_t e[4] = {y.x, y.y, y.z, y.w};
                if (p + k > upto) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = __uint_as_float(i & 1 ? e[i / 2] & 0xFFFF0000u : e[i / 2] << 16);
                    if (!(fabsf(f) < INFINITY)) add[i] += f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (add[i] != 0.f) put(d + i, add[i]);  // (a NaN is not 0)
    }
}

}  // namespace
