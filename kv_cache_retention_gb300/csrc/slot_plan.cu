// kvsel_plan_slots: block tables, slots and positions of a step's new tokens and
// slot maps of the sessions, built on the GPU from the sessions' lengths.
//
// With c_s tokens cached, n_s new ones and pages of `page` slots, session s holds
// have_s = ceil(c_s / page) pages and needs need_s = ceil((c_s + n_s) / page); its
// new pages are free_pages[before_s + i], before_s = sum over earlier sessions of
// need - have.  Token i of the session's new ones lies at position c_s + i and at
// packed place cu_s + i, cu the exclusive sums of n.  A position p of the session
// has slot  page_of(p / page) * page + p % page.
//
// One launch.  A block takes one session and one chunk of its positions; where the
// chunk holds new tokens it adds up the lengths of the earlier sessions itself (S
// loads spread over its threads, from L2), so no block waits for another and no
// workspace is needed.  The last blocks clear the packed places behind the last token.
// Small calls are bound by the chain of loads (length, table, free list), large ones by
// the slot maps' stores: four positions at a time, with one look at the table where
// they share a page.  64 sessions with slot maps of 92160 positions and up to 2048 new
// tokens each, 25 MB: 8.8 us (2.9 TB/s; one position at a time, with a second launch
// for the sums, 17 us); one new token for each of 36 sessions: 4.0 us.
#include <limits.h>

#include "kvsel_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;  // positions (or packed places) per block

struct PlanArgs {
    const int32_t* cached;
    const int32_t* new_len;
    int S;
    int page, page_shift, P;  // page_shift: log2(page), or -1
    const int32_t* free_pages;
    int n_free;
    int32_t* table;
    int max_blocks;
    int32_t* cu_new;
    int32_t* new_slots;
    int32_t* new_pos;
    int T;
    int32_t* slot_map;
    int ld;
    int32_t* counts;
    unsigned* err;
    int n_chunks;  // chunks per session
};

__device__ __forceinline__ int page_index(const PlanArgs& a, int p) {
    return a.page_shift >= 0 ? p >> a.page_shift : p / a.page;
}

// A session's lengths, brought into [0, cap]; bad: they were not there.
struct Lens {
    int c, n, have, need;
    bool bad;
};
__device__ __forceinline__ Lens lens_of(const PlanArgs& a, int s, int cap) {
    const int c0 = __ldg(a.cached + s), n0 = __ldg(a.new_len + s);
    Lens l;
    l.c = min(max(c0, 0), cap);
    l.n = min(max(n0, 0), cap - l.c);
    l.bad = l.c != c0 || l.n != n0;
    l.have = l.c > 0 ? page_index(a, l.c - 1) + 1 : 0;
    l.need = l.c + l.n > 0 ? page_index(a, l.c + l.n - 1) + 1 : 0;
    return l;
}

// Sums of x and y over the block.
__device__ __forceinline__ void block_sum(long long& x, long long& y, long long (*sh)[2]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5][0] = x, sh[threadIdx.x >> 5][1] = y;
    __syncthreads();
    x = y = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x += sh[w][0], y += sh[w][1];
}

__global__ void __launch_bounds__(kThreads) plan_slots_kernel(const PlanArgs a) {
    __shared__ long long sh[kThreads / 32][2];
    const int cap = a.max_blocks * a.page;  // the launcher keeps it below 2^31
    const int s = min((int)(blockIdx.x / a.n_chunks), a.S);
    unsigned err = 0;

    // sums over the earlier sessions (s == S: over all), where the block has a use for them
    const int chunk = blockIdx.x - s * a.n_chunks;
    Lens l = {};
    if (s < a.S) l = lens_of(a, s, cap);
    long long n_before = 0, take_before = 0;
    if (s == a.S || chunk == 0 || (l.n > 0 && (long long)chunk * kChunk < (long long)l.c + l.n && (chunk + 1ll) * kChunk > l.c)) {
        for (int i = threadIdx.x; i < s; i += kThreads) {
            const Lens e = lens_of(a, i, cap);
            n_before += e.n;
            take_before += e.need - e.have;
        }
        block_sum(n_before, take_before, sh);
    }

    if (s == a.S) {  // behind the last token
        const long long i0 = (long long)(blockIdx.x - (unsigned)a.S * a.n_chunks) * kChunk;
        const long long i1 = min(i0 + kChunk, (long long)a.T);
        for (long long i = max(i0, n_before) + threadIdx.x; i < i1; i += kThreads) {
            a.new_slots[i] = -1;
            a.new_pos[i] = -1;
        }
        if (i0 == 0 && threadIdx.x == 0) {
            a.counts[0] = (int)min(n_before, (long long)INT_MAX);
            a.counts[1] = (int)min(take_before, (long long)INT_MAX);
            a.cu_new[0] = 0;
            if (n_before > a.T) err |= KVSEL_DEV_BAD_LENGTH;
            if (take_before > a.n_free) err |= KVSEL_DEV_POOL_FULL;
            if (err) atomicOr(a.err, err);
        }
        return;
    }

    if (chunk == 0 && threadIdx.x == 0) {
        a.cu_new[s + 1] = (int)min(n_before + l.n, (long long)INT_MAX);
        if (l.bad || (a.slot_map && l.c + l.n > a.ld)) err |= KVSEL_DEV_BAD_LENGTH;
    }
    int32_t* const row = a.table + (int64_t)s * a.max_blocks;
    // page j of the session: an old one from its table, a new one from the free list; -1: none
    auto page_of = [&](int j) {
        int pg = -1;
        if (j < l.have) {
            pg = __ldg(row + j);
        } else {
            const long long f = take_before + (j - l.have);
            if (f >= a.n_free) return -1;
            pg = __ldg(a.free_pages + f);
        }
        if (pg < 0 || pg >= a.P) {
            err |= KVSEL_DEV_BAD_PAGE;
            return -1;
        }
        return pg;
    };
    const long long p0 = (long long)chunk * kChunk, p1 = p0 + kChunk;

    // new table entries whose first position lies in the chunk
    const int j0 = max((int)((p0 + a.page - 1) / a.page), l.have);
    const int j1 = (int)min((p1 + a.page - 1) / a.page, (long long)l.need);
    for (int j = j0 + threadIdx.x; j < j1; j += kThreads) row[j] = page_of(j);

    // new tokens at the chunk's positions
    const int t1 = (int)min(p1, (long long)l.c + l.n);
    for (int p = (int)max(p0, (long long)l.c) + threadIdx.x; p < t1; p += kThreads) {
        const long long i = n_before + (p - l.c);
        if (i >= a.T) break;
        const int j = page_index(a, p), pg = page_of(j);
        a.new_slots[i] = pg < 0 ? -1 : pg * a.page + (p - j * a.page);
        a.new_pos[i] = p;
    }

    // the session's slot map
    if (a.slot_map) {
        int32_t* const map = a.slot_map + (int64_t)s * a.ld;
        const int m1 = (int)min(p1, (long long)a.ld), end = l.c + l.n;
        auto slot_at = [&](int p) {
            if (p >= end) return -1;
            const int j = page_index(a, p), pg = page_of(j);
            return pg < 0 ? -1 : pg * a.page + (p - j * a.page);
        };
        // rows of a multiple of four on 16 bytes, pages of a multiple of four: four positions share a page and a store
        if (a.ld % 4 == 0 && a.page % 4 == 0 && (reinterpret_cast<uintptr_t>(a.slot_map) & 15u) == 0) {
            for (int p = (int)p0 + 4 * threadIdx.x; p < m1; p += 4 * kThreads) {
                const int first = slot_at(p);
                int4 v = make_int4(first, -1, -1, -1);
                if (first >= 0) {
                    if (p + 1 < end) v.y = first + 1;
                    if (p + 2 < end) v.z = first + 2;
                    if (p + 3 < end) v.w = first + 3;
                }
                *reinterpret_cast<int4*>(map + p) = v;
            }
        } else {
            for (int p = (int)p0 + threadIdx.x; p < m1; p += kThreads) map[p] = slot_at(p);
        }
    }
    if (err) atomicOr(a.err, err);
}

}  // namespace

extern "C" int kvsel_plan_slots(kvsel_ctx* ctx, const int32_t* cached, const int32_t* new_len, int S, int page, int P,
                                const int32_t* free_pages, int n_free, int32_t* block_table, int max_blocks,
                                int32_t* cu_new, int32_t* new_slots, int32_t* new_pos, int T, int32_t* slot_map, int ld,
                                int32_t* counts, void* stream) {
    const kvsel_trace trace_("kvsel_plan_slots");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (S < 0 || page <= 0 || P < 0 || n_free < 0 || max_blocks < 0 || T < 0 || ld < 0)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "plan_slots: bad sizes");
    if (S > 16384) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "plan_slots: S=%d > 16384 sessions", S);
    if ((int64_t)P * page > INT_MAX || (int64_t)max_blocks * page > INT_MAX - 4096 || ld > INT_MAX - 4096)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "plan_slots: slots and positions must fit 31 bits");
    if (!cu_new || !counts || (S > 0 && (!cached || !new_len)) || (S > 0 && max_blocks > 0 && !block_table) ||
        (n_free > 0 && !free_pages) || (T > 0 && (!new_slots || !new_pos)) || (S > 0 && ld > 0 && !slot_map))
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "plan_slots: null pointer");
    int64_t reach = (int64_t)max_blocks * page;
    if (slot_map && ld > reach) reach = ld;
    int64_t n_chunks = (reach + kChunk - 1) / kChunk;
    if (n_chunks < 1) n_chunks = 1;
    const int64_t tail = T > 0 ? ((int64_t)T + kChunk - 1) / kChunk : 1;
    const int64_t blocks = S * n_chunks + tail;
    if (blocks > INT_MAX) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "plan_slots: too many positions");
    int shift = -1;
    if ((page & (page - 1)) == 0)
        for (shift = 0; (1 << shift) < page;) ++shift;
    const PlanArgs a{cached, new_len, S, page, shift, P, free_pages, n_free, block_table, max_blocks, cu_new, new_slots,
                     new_pos, T, ld > 0 ? slot_map : nullptr, ld, counts, ctx->dev_err, (int)n_chunks};
    plan_slots_kernel<<<(unsigned)blocks, kThreads, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "plan_slots launch");
}
