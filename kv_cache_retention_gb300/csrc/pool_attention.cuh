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

}  // namespace
