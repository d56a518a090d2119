// How the calls over the bf16 page pools find their tokens: sessions' rows from cu_new and seq_lens, slots from slot maps
// or block tables.
#pragma once

#include <limits.h>

#include "kvsel_internal.h"

namespace {

// Slot maps (page == 0) or block tables, int32 [S][ld].
struct TokenMap {
    const int32_t* map;
    int ld, reach;           // row length, and the positions that a row holds
    int page;
    uint32_t mul, shift;     // j / page = j mul >> shift
    int limit;               // entries lie below it: pages or slots
    int dead;
};

// A session's new tokens: rows [first, first + count) of q, the last of its len tokens.
struct Session {
    int first, count, len;
};

__device__ __forceinline__ int entry_of(const TokenMap& m, int j) {
    return (int)(((uint64_t)(uint32_t)j * m.mul) >> m.shift);
}
// What the map says of position j (below its reach): a slot, or the page that holds it.
__device__ __forceinline__ int raw_entry(const TokenMap& m, const int32_t* row, int j) { return __ldg(row + entry_of(m, j)); }
// Slot of position j, from what the map says; -1 where it is not live.  MAP: a slot map, not a block table.
template <bool MAP>
__device__ __forceinline__ int live_slot(const TokenMap& m, int entry, int j, unsigned& err) {
    if ((unsigned)entry >= (unsigned)m.limit) {
        if (entry >= 0 && (!MAP || entry != m.dead)) err |= MAP ? KVSEL_DEV_BAD_SLOT : KVSEL_DEV_BAD_PAGE;
        return -1;
    }
    const int slot = MAP ? entry : entry * m.page + (j - entry_of(m, j) * m.page);
    return slot == m.dead ? -1 : slot;
}

// Session s.  Sequences that start below 0 or end before they start have no rows; they end at T, lengths at the reach.
__device__ __forceinline__ Session session_at(const int32_t* cu, const int32_t* lens, int T, int reach, int s) {
    const int first = __ldg(cu + s), stop = __ldg(cu + s + 1);
    Session x;
    x.first = first;
    x.count = first < 0 || stop < first ? 0 : max(0, min(stop, T) - first);
    x.len = min(max(__ldg(lens + s), 0), reach);
    return x;
}
// What of session s's arguments is outside its range.
__device__ __forceinline__ unsigned session_errors(const int32_t* cu, const int32_t* lens, int T, int reach, int s) {
    const int first = __ldg(cu + s), stop = __ldg(cu + s + 1), len = __ldg(lens + s);
    return first < 0 || stop < first || stop > T || len < 0 || len > reach ? KVSEL_DEV_BAD_LENGTH : 0u;
}

// The rules that the calls over the pools share: sizes, the map, pools, strides.  Fills map.
inline int check_pool_call(kvsel_ctx* ctx, const char* who, int S, int T, int Hq, int Hkv, int D, int64_t q_stride,
                           const void* const* pools, const int64_t* strides, int n_pools, int P, int page,
                           const int32_t* slot_map, const int32_t* block_table, int ld, int dead_slot, float scale,
                           TokenMap* map) {
    if (S < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || P < 0 || page <= 0 || ld < 0)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "%s: bad sizes", who);
    if (Hq % Hkv) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "%s: Hq=%d not a multiple of Hkv=%d", who, Hq, Hkv);
    if (D != 64 && D != 128) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: D=%d unsupported", who, D);
    if (Hq / Hkv > 128) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: group size Hq/Hkv=%d > 128", who, Hq / Hkv);
    if ((slot_map && block_table) || (!slot_map && !block_table && S > 0 && ld > 0))  // (maps without elements may be NULL)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "%s: one of slot_map and block_table is needed", who);
    const int64_t reach = slot_map ? ld : (int64_t)ld * page;
    if ((int64_t)P * page > INT_MAX || reach > INT_MAX - 4096)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: slots and positions must fit 31 bits", who);
    if (S > 65535 || Hq > 65535 || T > (1 << 24)) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: S, T or Hq too large", who);
    if (!(scale > 0.f) || scale > 1e30f)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
    if (T > 1 && q_stride < (int64_t)Hq * D) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "%s: token stride < Hq*D", who);
    if ((q_stride * 2) % 16) return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "%s: q's stride must be 16-byte aligned", who);
    for (int i = 0; i < n_pools; ++i) {
        if (P > 0 && !pools[i]) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "%s: null pointer", who);
        if ((int64_t)P * page > 1 && strides[i] < (int64_t)Hkv * D)
            return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "%s: slot stride < Hkv*D", who);
        if (strides[i] > INT_MAX / 2) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: slot stride too large", who);
        if ((reinterpret_cast<uintptr_t>(pools[i]) & 15u) || (strides[i] * 2) % 16)
            return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "%s: pools and their strides must be 16-byte aligned", who);
    }
    *map = TokenMap{slot_map ? slot_map : block_table, ld, (int)reach, 0, 1, 0, P * page, dead_slot};
    if (!slot_map) {
        map->page = page, map->limit = P;
        if (page > 1) {  // with 2^(l-1) < page <= 2^l, (2^(31+l) / page + 1) j >> (31+l) is the quotient for every j < 2^31
            int l = 1;
            while (((int64_t)1 << l) < page) ++l;
            map->mul = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)page + 1);
            map->shift = 31 + l;
        }
    }
    return KVSEL_OK;
}

}  // namespace
