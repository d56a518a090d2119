// kvsel_attention_mass: the softmax weight that the new tokens give to each token of their session, on the 5th-generation
// tensor cores.
//
//   score_out[s,j] = score_in[s,j] + sum_{i,h} 2^(scale log2e q_ih . k_j - log2e lse_ih)   over the rows whose token i sees j.
//
// The keys are the rows of the product, S^T = K Q^T: a thread has a key (a TMEM lane), so that its sum over query rows stays
// in a register, for one kv head after the other, and is added to its score once.
//
// Keys go through lists of 128 live tokens (dropped tokens cost an entry's read and no more).  An item is two lists; for
// each kv head its two K tiles stay in shared memory while the session's query rows pass, a tile of the G = Hq/Hkv heads of
// as many tokens as fit 128 rows at a time, which both K tiles share: per tile two products of 128 x 128 x D, then 2^x of
// each element.  Tiles whose tokens lie before the item's keys are left out.
//
// 512 threads: warp 0 plans and makes the lists, warps 1 and 3 issue the MMAs of the two lists, warp 2 loads Q tiles and reads
// the rows' lse, warps 4-7 load K tiles, warps 8-11 and 12-15 sum the two lists' weights.  TMEM: two buffers of 128 columns for each list.
//
// Shares.  All sessions' chunks of 128 positions, each counted as the row tiles it meets and some for its own loads, are cut
// into equal contiguous shares, a block each, found from the lengths on the device.  Where there are few chunks, several
// blocks take a share's kv heads in turn and a second kernel adds their parts up in order.
//
// Measured, 32/8 heads of 128: 2048 tokens over 34816 0.51 ms (1.11 PFLOP/s; tensor pipe 50%, issue slots 45%, DRAM 2%: no unit
// is full); a decode step of 36 sessions pruned to a quarter, 500 MB, 112 us (4.5 TB/s).
//
// Every wait is bounded (1 s); on a timeout the block flags KVSEL_ERR_TIMEOUT in the device error word, drains its own copies
// and MMAs, frees TMEM and returns.
#include <type_traits>

#include "pool_lists.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kLists = 8;
constexpr int kLoad = 2;                // row tiles that a chunk's own loads and its start count as (1 costs 2048 tokens 1%; 4 and 8 nothing)
constexpr uint32_t kTmem = 0;           // all of TMEM is allocated, so its base is column 0
constexpr int kTmemCols = 512;

struct MassArgs {
    const int32_t *cu, *lens;
    int S, T, Hq, Hkv, G;
    int tile_tokens, small_tokens;      // tokens of a row tile; of one small load
    const float* lse;
    const __nv_bfloat16* k;
    uint32_t k_bytes;                   // from a slot's rows to the next one's
    TokenMap map;
    float scale2;                       // scale * log2(e)
    float* score;                       // added to; or, with several blocks a share, their parts
    int64_t score_ld, part;             // part: elements between the parts, 0: none
    unsigned* err;
    int shares, split;                  // blocks that share a share's kv heads
    uint64_t wait_ns;
    int stuck;
};

template <int D>
struct MassCfg {
    static constexpr int kBlock = kTile * 128;             // 128 rows x 64 dims, 128-byte swizzled
    static constexpr int kBytes = D / 64 * kBlock;         // one tile of K or Q
    static constexpr int kK = 4, kQ = 2, kL = 4;           // tiles of K (two for each list of an item), of Q; lse rows
    struct Piece {
        int row, count, pos0, session, end;
    };
    struct Tail {
        Lists<kLists> lists;
        alignas(16) float lse[kL][kTile];  // -log2e lse; -inf where the row has no weight
        uint64_t k_full[kK], k_empty[kK], q_full[kQ], q_empty[kQ], l_full[kL], l_empty[kL], s_full[2][2], s_empty[2][2],
            piece_full[2], piece_empty[2], drained;
        Stop stop;
        uint64_t never;
        uint32_t tmem;
        Piece piece[2];
    };
    static constexpr size_t kSmem = (size_t)(kK + kQ) * kBytes + sizeof(Tail) + 1024;
    static_assert(kSmem <= 232448, "shared memory per block");
    static_assert(offsetof(Tail, lse) % 16 == 0 && alignof(Tail) == 16, "read 16 bytes at a time");
};

// The next item of a piece, as a role sees it: lists l and, with nl = 2, l + 1; n, first: tokens and first position.
struct Item {
    int nl, n0, n1, first;
    bool last;
};
// Waits for it; false at the piece's end (an empty list) or when a wait gave up.  The caller releases the lists.
template <class Tail>
__device__ __forceinline__ bool next_item(Tail& t, uint32_t l, Item& it, Stop* stop, unsigned* err, bool& ok) {
    it.n1 = 0;
    if (!(ok = wait_idle(&t.lists.full[l % kLists], l / kLists & 1, stop, err))) return false;
    const ListMeta m = t.lists.meta[l % kLists];
    it.nl = 1, it.n0 = m.n, it.first = m.first, it.last = m.last;
    if (!m.last) {
        ++l;
        if (!(ok = wait_idle(&t.lists.full[l % kLists], l / kLists & 1, stop, err))) return false;
        it.nl = 2, it.n1 = t.lists.meta[l % kLists].n, it.last = t.lists.meta[l % kLists].last;
    }
    return true;
}

template <int D, bool MAP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_mass_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_small,
                          const __grid_constant__ CUtensorMap map_k, const MassArgs a) {
    using C = MassCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    // (an offset and not a cast, so that the compiler knows it for shared memory)
    uint8_t* const smem = smem_raw + (-saddr(smem_raw) & 1023u);
    uint8_t* const sk = smem;                       // [kK][kBytes]
    uint8_t* const sq = smem + C::kK * C::kBytes;   // [kQ][kBytes]
    typename C::Tail& t = *reinterpret_cast<typename C::Tail*>(smem + (C::kK + C::kQ) * C::kBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head0 = (int)(blockIdx.x % a.split), share = (int)(blockIdx.x / a.split);
    Stop* const stop = &t.stop;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kK; ++i) mbar_init(&t.k_full[i], 64), mbar_init(&t.k_empty[i], 1);
        for (int i = 0; i < C::kQ; ++i) mbar_init(&t.q_full[i], 1), mbar_init(&t.q_empty[i], 2);
        for (int i = 0; i < C::kL; ++i) mbar_init(&t.l_full[i], 1), mbar_init(&t.l_empty[i], 8);
        for (int i = 0; i < 4; ++i) mbar_init(&t.s_full[i >> 1][i & 1], 1), mbar_init(&t.s_empty[i >> 1][i & 1], 4);
        for (int i = 0; i < 2; ++i) mbar_init(&t.piece_full[i], 1), mbar_init(&t.piece_empty[i], 3 + 4 + 8);
        for (int i = 0; i < kLists; ++i) mbar_init(&t.lists.full[i], 1), mbar_init(&t.lists.empty[i], 3 + 4 + 8);
        mbar_init(&t.drained, 2);
        mbar_init(&t.never, 1);
        t.stop.given_up = 0;
        t.stop.limit_ns = a.wait_ns;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&t.tmem)), "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (a.tile_tokens * a.G < kTile) {  // rows that no tile fills: zeros (their columns are not looked at)
        for (int i = threadIdx.x; i < C::kQ * C::kBytes / 16; i += kThreads) reinterpret_cast<uint4*>(sq)[i] = make_uint4(0, 0, 0, 0);
        fence_async();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = t.tmem;

    bool ok = true;
    uint32_t l = 0;                     // lists so far
    auto release = [&](uint32_t list) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&t.lists.empty[list % kLists]);
    };
    auto next_piece = [&](uint32_t u, typename C::Piece& w, bool keep) {
        if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, a.err))) return false;
        w = t.piece[u & 1];
        __syncwarp();
        if (lane == 0 && !keep) mbar_arrive(&t.piece_empty[u & 1]);
        return !w.end;
    };
    auto row_tiles = [&](const typename C::Piece& w) { return (w.count + a.tile_tokens - 1) / a.tile_tokens; };
    auto first_tile = [&](const typename C::Piece& w, const Item& it) { return max(0, it.first - w.pos0) / a.tile_tokens; };

    if (warp == 0) {
        // ---- the share's pieces, and their lists ----
        unsigned err = 0;
        uint32_t u = 0;
        auto publish = [&](const typename C::Piece& w) {
            if (u >= 2 && !(ok = wait_idle(&t.piece_empty[u & 1], ((u >> 1) - 1) & 1, stop, a.err))) return;
            if (lane == 0) t.piece[u & 1] = w;
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.piece_full[u & 1]);
            ++u;
        };
        // what a chunk of 128 positions of the session counts as, and how many there are
        auto weight = [&](const Session& x) { return (int64_t)kLoad + (x.count + a.tile_tokens - 1) / a.tile_tokens; };
        auto chunks = [&](const Session& x) { return x.count > 0 ? (int64_t)((x.len + (int64_t)kTile - 1) / kTile) : 0; };
        int64_t total = 0;
        for (int s = lane; s < a.S; s += 32) {
            const Session x = session_at(a.cu, a.lens, a.T, a.map.reach, s);
            total += chunks(x) * weight(x);
            if (blockIdx.x == 0) err |= session_errors(a.cu, a.lens, a.T, a.map.reach, s);
        }
        total = warp_sum(total);
        const int64_t quota = max((total + a.shares - 1) / a.shares, (int64_t)1), from = share * quota, to = from + quota;
        int64_t at = 0;                 // where session s starts
        for (int s0 = 0; ok && s0 < a.S && at < to; s0 += 32) {
            Session mine{0, 0, 0};
            if (s0 + lane < a.S) mine = session_at(a.cu, a.lens, a.T, a.map.reach, s0 + lane);
            const int64_t size = chunks(mine) * weight(mine), all = warp_sum(size);
            if (at + all <= from) {     // 32 sessions before the share
                at += all;
                continue;
            }
            for (int i = 0; ok && i < 32 && s0 + i < a.S && at < to; ++i) {
                Session x;
                x.first = __shfl_sync(0xffffffffu, mine.first, i);
                x.count = __shfl_sync(0xffffffffu, mine.count, i);
                x.len = __shfl_sync(0xffffffffu, mine.len, i);
                const int64_t n = chunks(x), w = weight(x);
                // the chunks that start in the share
                const int64_t c0 = at >= from ? 0 : min(n, (from - at + w - 1) / w), c1 = min(n, (to - at + w - 1) / w);
                at += n * w;
                if (c0 >= c1) continue;
                publish(typename C::Piece{x.first, x.count, x.len - x.count, s0 + i, 0});
                ok = ok && make_lists<MAP>(t.lists, a.map, a.map.map + (int64_t)(s0 + i) * a.map.ld, (int)c0 * kTile,
                                      (int)min((int64_t)x.len, c1 * kTile), INT_MIN, l, &t.lists.progress[0], lane, stop, a.err, err);
            }
        }
        if (ok) publish(typename C::Piece{0, 0, 0, 0, 1});
        if (err) atomicOr(a.err, err);
    } else if (warp == 1 || warp == 3) {
        // ---- MMAs: a warp for each list of an item (one warp for both took 638 us for the mass of 2048 tokens) ----
        const uint32_t x = warp >> 1;
        uint32_t ck = 0, cq = 0, cs = 0;  // K tiles, Q tiles, and this list's buffers used so far
        ok = !a.stuck || wait_short(&t.never, 0, stop, a.err);
        typename C::Piece w;
        for (uint32_t u = 0; ok && next_piece(u, w, false); ++u) {
            const int nt = row_tiles(w);
            // columns of a product: the rows of a small load, else all of a tile's
            const uint32_t id = uniform(w.count <= a.small_tokens ? idesc((w.count * a.G + 15) & ~15, false) : idesc(kTile, false));
            Item it;
            do {
                if (!next_item(t, l, it, stop, a.err, ok)) break;
                for (int y = 0; y < it.nl; ++y) release(l + y);
                l += it.nl;
                const int t0 = first_tile(w, it);
                const bool mine = (int)x < it.nl;
#pragma unroll 1
                for (int g = head0; ok && it.n0 && g < a.Hkv; g += a.split, ck += 2) {
                    const uint32_t st = (ck + x) % C::kK;
                    const uint32_t k = uniform(desc_low(saddr(sk) + st * C::kBytes, 16));
                    ok = wait_lane(&t.k_full[st], (ck + x) / C::kK & 1, stop, a.err) && ok;
                    fence_async();
#pragma unroll 1
                    for (int i = t0; ok && i < nt; ++i, ++cq) {
                        const uint32_t b = cs & 1, d = uniform(kTmem + x * 256 + b * 128), sq_at = cq % C::kQ;
                        const uint32_t q = uniform(desc_low(saddr(sq) + sq_at * C::kBytes, 16));
                        uint64_t* const qf = &t.q_full[sq_at];
                        const uint32_t qp = cq / C::kQ & 1;
                        ok = wait_lane2(qf, qp, mine ? &t.s_empty[x][b] : qf, mine ? ((cs >> 1) & 1) ^ 1 : qp, stop, a.err) && ok;
                        tc_after();
                        if (elect_one()) {
                            if (mine) {
#pragma unroll
                                for (int j = 0; j < D / 16; ++j) {
                                    const uint32_t off = ((j >> 2) * C::kBlock + (j & 3) * 32) >> 4;
                                    mma_ss_one(d, k + off, q + off, id, j > 0);
                                }
                                mma_commit_one(saddr(&t.s_full[x][b]));
                            }
                            mma_commit_one(saddr(&t.q_empty[sq_at]));
                            if (i == nt - 1) mma_commit_one(saddr(&t.k_empty[st]));
                        }
                        __syncwarp();
                        cs += mine;
                        ok = __all_sync(0xffffffffu, ok);
                    }
                }
            } while (ok && !it.last);
        }
        if (elect_one()) mma_commit_one(saddr(&t.drained));
        __syncwarp();
        drain_phase(&t.drained, 0);
    } else if (warp == 2) {
        // ---- Q tiles, and the rows' lse ----
        uint32_t c = 0, loaded = 0;
        typename C::Piece w;
        for (uint32_t u = 0; ok && next_piece(u, w, false); ++u) {
            const int nt = row_tiles(w);
            const bool small = w.count <= a.small_tokens;
            const int bytes = D / 64 * (small ? a.small_tokens : a.tile_tokens) * a.G * 128;
            Item it;
            do {
                if (!next_item(t, l, it, stop, a.err, ok)) break;
                for (int x = 0; x < it.nl; ++x) release(l + x);
                l += it.nl;
                const int t0 = first_tile(w, it);
#pragma unroll 1
                for (int g = head0; ok && it.n0 && g < a.Hkv; g += a.split)
#pragma unroll 1
                    for (int i = t0; ok && i < nt; ++i, ++c) {
                        float v[kTile / 32];
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k) {
                            const int col = lane + 32 * k, tok = i * a.tile_tokens + col / a.G;
                            const bool real = col < a.tile_tokens * a.G && tok < w.count;
                            const float x = real ? __ldg(a.lse + (int64_t)(w.row + tok) * a.Hq + g * a.G + col % a.G) : -INFINITY;
                            v[k] = x == -INFINITY ? -INFINITY : x * -kLog2e;
                        }
                        const uint32_t st = c % C::kQ;
                        if (!(ok = wait_short(&t.q_empty[st], (c / C::kQ & 1) ^ 1, stop, a.err))) break;
                        if (lane == 0) {
                            mbar_expect_tx(&t.q_full[st], bytes);
                            for (int b = 0; b < D / 64; ++b)
                                tma_load(small ? &map_small : &map_q, &t.q_full[st], sq + st * C::kBytes + b * C::kBlock, 64 * b, g * a.G,
                                         w.row + i * a.tile_tokens);
                        }
                        loaded = c + 1;
                        if (!(ok = wait_idle(&t.l_empty[c % C::kL], (c / C::kL & 1) ^ 1, stop, a.err))) break;
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k) t.lse[c % C::kL][lane + 32 * k] = v[k];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&t.l_full[c % C::kL]);
                    }
            } while (ok && !it.last);
        }
        for (uint32_t at = loaded > C::kQ ? loaded - C::kQ : 0; at < loaded; ++at) drain_phase(&t.q_full[at % C::kQ], at / C::kQ & 1);
    } else if (warp < 8) {
        // ---- K tiles: two warps for each list of an item, half a tile each ----
        static_assert(C::kK == 4, "a stage of the ring is one list's");
        const int x = (warp - 4) >> 1;
        uint32_t c = 0, loaded = 0;     // places of the ring so far; one behind the last that this warp has filled
        typename C::Piece w;
        for (uint32_t u = 0; ok && next_piece(u, w, false); ++u) {
            Item it;
            do {
                if (!next_item(t, l, it, stop, a.err, ok)) break;
                const uint32_t at = (l + (x < it.nl ? x : 0)) % kLists;
#pragma unroll 1
                for (int g = head0; ok && it.n0 && g < a.Hkv; g += a.split, c += 2) {
                    const uint32_t st = (c + x) % C::kK;
                    if (!(ok = wait_short(&t.k_empty[st], ((c + x) / C::kK & 1) ^ 1, stop, a.err))) break;
                    if (x < it.nl)
                        load_rows<D, 2>(&map_k, a.k, a.k_bytes, g * D, t.lists.token + at * kTile, t.lists.meta[at].n,
                                        t.lists.meta[at].runs,
                                        sk + st * C::kBytes, &t.k_full[st], warp & 1, lane);
                    else
                        mbar_arrive(&t.k_full[st]);  // (there is no second list)
                    loaded = c + x + 1;
                }
                for (int y = 0; ok && y < it.nl; ++y) release(l + y);
                l += it.nl;
            } while (ok && !it.last);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (uint32_t at = loaded > 2 ? loaded - 3 : loaded - 1; loaded && at < loaded; at += 2)
            drain_phase(&t.k_full[at % C::kK], at / C::kK & 1);
    } else {
        // ---- sums: a key per thread ----
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the score has been copied
        const int x = (warp - 8) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t ts = kTmem + ((uint32_t)(quarter * 32) << 16) + x * 256;
        const float2 sc2 = make_float2(a.scale2, a.scale2);
        const int full = a.tile_tokens * a.G;       // rows of a full tile: more than 64, whatever G is
        uint32_t c = 0, cs = 0;                     // row tiles, and this list's buffers used so far
        typename C::Piece w;
        for (uint32_t u = 0; ok && next_piece(u, w, true); ++u) {
            const int nt = row_tiles(w);
            Item it;
            do {
                if (!next_item(t, l, it, stop, a.err, ok)) break;
                const int t0 = first_tile(w, it), n = x == 0 ? it.n0 : it.n1;
                const int pos = t.lists.token[(l + (x < it.nl ? x : 0)) % kLists * kTile + r].y;
                const int behind = r < n ? pos - w.pos0 : 0;  // the first token that sees the key
                float2 sum = make_float2(0.f, 0.f), sum2 = sum;  // (two, which depend on themselves half as often)
#pragma unroll 1
                for (int g = head0; ok && it.n0 && g < a.Hkv; g += a.split)
#pragma unroll 1
                    for (int i = t0; ok && i < nt; ++i, ++c) {
                        const uint32_t b = cs & 1;
                        uint64_t* const lf = &t.l_full[c % C::kL];
                        const uint32_t lp = c / C::kL & 1;
                        ok = wait_lane2(lf, lp, x < it.nl ? &t.s_full[x][b] : lf, x < it.nl ? (cs >> 1) & 1 : lp, stop, a.err);
                        if (x < it.nl) {
                            ++cs;
                            tc_after();
                            // columns that count: of tokens that see the key, and of the session's tokens
                            const int lo = min(max(behind - i * a.tile_tokens, 0), a.tile_tokens) * a.G;
                            const int hi = min(a.tile_tokens, w.count - i * a.tile_tokens) * a.G;
                            const bool part = __any_sync(0xffffffffu, lo > 0) || hi < full;
                            const float* const nl = t.lse[c % C::kL];
                            uint32_t s0[32], s1[32];
                            auto taken = [&]() {    // the buffer's columns are all in registers
                                tc_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&t.s_empty[x][b]);
                            };
                            tmem_ld32(ts + b * 128, s0);
                            tmem_wait_ld();
                            // 32 columns at a time, the next ones on their way meanwhile.  Columns behind the tile's rows, from
                            // place `first` on, are no logits (rows of zeros times an infinite key, or what a narrow product
                            // has not written: NaN, which their bias of -inf would not hide), and are set to zero.  Groups of up
                            // to 12 heads leave 8 columns at most, and those of a power of two none (2048 tokens over 34816: setting
                            // 8 costs 1% with groups of 5 and 7, where all 64 cost 8 and 10%, and 9% with groups of 13).
                            auto whole = [&](auto first) {
                                auto add = [&](uint32_t* s, int h) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        if (h + k >= decltype(first)::value) s[k] = h + k < full ? s[k] : 0u;
#pragma unroll
                                    for (int k = 0; k < 8; ++k) {
                                        const float4 m = *reinterpret_cast<const float4*>(nl + h + 4 * k);
                                        const float2 y0 = __ffma2_rn(make_float2(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])),
                                                                     sc2, make_float2(m.x, m.y));
                                        const float2 y1 = __ffma2_rn(make_float2(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])),
                                                                     sc2, make_float2(m.z, m.w));
                                        sum = __fadd2_rn(sum, make_float2(ex2(y0.x), ex2(y0.y)));
                                        sum2 = __fadd2_rn(sum2, make_float2(ex2(y1.x), ex2(y1.y)));
                                    }
                                };
                                tmem_ld32(ts + b * 128 + 32, s1);
                                add(s0, 0);
                                tmem_wait_ld();
                                tmem_ld32(ts + b * 128 + 64, s0);
                                add(s1, 32);
                                tmem_wait_ld();
                                tmem_ld32(ts + b * 128 + 96, s1);
                                add(s0, 64);
                                tmem_wait_ld();
                                taken();
                                add(s1, 96);
                            };
                            if (!part && full == kTile) {
                                whole(std::integral_constant<int, kTile>());
                            } else if (!part && full >= kTile - 8) {
                                whole(std::integral_constant<int, kTile - 8>());
                            } else if (!part) {
                                whole(std::integral_constant<int, kTile / 2>());
                            } else {
                                const unsigned wide = (unsigned)max(hi - lo, 0);
#pragma unroll 1
                                for (int h = 0; h < hi; h += 32) {
                                    if (h) {
                                        tmem_ld32(ts + b * 128 + h, s0);
                                        tmem_wait_ld();
                                    }
                                    if (h + 32 >= hi) taken();
#pragma unroll
                                    for (int k = 0; k < 32; ++k) {
                                        const float e = ex2(fmaf(__uint_as_float(s0[k]), a.scale2, nl[h + k]));
                                        if ((unsigned)(h + k - lo) < wide) sum.x += e;
                                    }
                                }
                            }
                        }
                        ok = __all_sync(0xffffffffu, ok);
                        if (lane == 0) mbar_arrive(&t.l_empty[c % C::kL]);
                    }
                if (ok && r < n) {
                    float* const to = a.score + (a.part ? head0 * a.part : 0) + w.session * a.score_ld + pos;
                    const float mass = (sum.x + sum2.x) + (sum.y + sum2.y);
                    *to = a.part ? mass : *to + mass;
                }
                for (int y = 0; ok && y < it.nl; ++y) release(l + y);
                l += it.nl;
            } while (ok && !it.last);
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
        }
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// score_out = score_in, or 0: a row per blockIdx.y.
__global__ void __launch_bounds__(256) mass_copy_kernel(const float* before, float* score, int64_t ld, int n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = (int64_t)blockIdx.y * ld;
    // (64 bits: the last step may pass 2^31)
    for (int64_t j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) score[row + j] = before ? before[row + j] : 0.f;
}

// score_out = score_in + the parts of the blocks that shared the kv heads, in their order, where a token is live.
template <bool MAP>
__global__ void __launch_bounds__(256) mass_add_kernel(const MassArgs a, const float* before, float* score, int64_t ld) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.y;
    unsigned err = 0;
    const Session x = session_at(a.cu, a.lens, a.T, a.map.reach, s);
    const int32_t* const row = a.map.map + (int64_t)s * a.map.ld;
    // (the reach is far below 2^31 here: the parts fit the context's memory for them)
    for (int j = blockIdx.x * 256 + threadIdx.x; j < a.map.reach; j += gridDim.x * 256) {
        float sum = 0.f;
        if (x.count > 0 && j < x.len && live_slot<MAP>(a.map, raw_entry(a.map, row, j), j, err) >= 0)
            for (int k = 0; k < a.split; ++k) sum += a.score[k * a.part + s * a.score_ld + j];
        score[s * ld + j] = (before ? before[s * ld + j] : 0.f) + sum;
    }
}

template <int D, bool MAP>
cudaError_t launch(kvsel_ctx* ctx, const CUtensorMap& mq, const CUtensorMap& ms, const CUtensorMap& mk, const MassArgs& a,
                   const float* before, float* score, int64_t score_ld, cudaStream_t s) {
    auto* kernel = attention_mass_kernel<D, MAP>;
    constexpr uint64_t kBit = (uint64_t)KVSEL_READY_MASS << (D / 64 - 1 + 2 * MAP);
    if (!(ctx->ready & kBit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MassCfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        ctx->ready |= kBit;
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.shares * a.split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = MassCfg<D>::kSmem;
    cfg.stream = s;
    const dim3 rows((unsigned)min((a.map.reach + 1023) / 1024, 1024), a.S);
    if (!a.part && before != score) {
        mass_copy_kernel<<<rows, 256, 0, s>>>(before, score, score_ld, a.map.reach);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, mq, ms, mk, a);
    if (e != cudaSuccess || !a.part) return e;
    cfg.gridDim = rows;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mass_add_kernel<MAP>, a, before, score, score_ld);
}

int mass_call(kvsel_ctx* ctx, const void* q, int64_t q_stride, const float* lse, const int32_t* cu_new, int S, int T, int Hq, int Hkv,
              int D, const void* k_pool, int64_t k_stride, int P, int page, const int32_t* seq_lens, const int32_t* slot_map,
              const int32_t* block_table, int ld, int dead_slot, float scale, const float* score_in, float* score_out,
              int64_t score_ld, void* stream, uint64_t wait_ns, int stuck) {
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    const void* pools[1] = {k_pool};
    TokenMap map;
    rc = check_pool_call(ctx, "attention_mass", S, T, Hq, Hkv, D, q_stride, pools, &k_stride, 1, P, page, slot_map, block_table,
                         ld, dead_slot, scale, &map);
    if (rc) return rc;
    if (score_ld < map.reach) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "attention_mass: score rows shorter than the map's reach");
    if (S == 0 || map.reach == 0) return KVSEL_OK;
    if (!cu_new || !seq_lens || !score_out || (T > 0 && (!q || !lse)))
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "attention_mass: null pointer");
    if (reinterpret_cast<uintptr_t>(q) & 15u) return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "attention_mass: q must be 16-byte aligned");
    const int G = Hq / Hkv, tile_tokens = kTile / G, small_tokens = G < 16 ? 16 / G : 1;
    CUtensorMap mq, ms, mk;
    const bool work = T > 0 && P > 0;   // else nothing is live, or there are no rows: the score is copied
    if (work && (!make_query_map(&mq, q, T, Hq, D, q_stride, G, tile_tokens) ||
                 !make_query_map(&ms, q, T, Hq, D, q_stride, G, small_tokens) || !make_pool_map(&mk, k_pool, P * page, Hkv, D, k_stride)))
        return kvsel_fail(ctx, KVSEL_ERR_CUDA, "attention_mass: tensor map encoding failed");
    // Few chunks: the kv heads of a share go to up to 8 blocks, as long as their parts fit the context's memory for them.
    const int64_t chunks = (int64_t)S * ((map.reach + kTile - 1) / kTile), positions = (int64_t)S * map.reach;
    int split = 1;
    while (split < 8 && 2 * split <= Hkv && chunks * split < ctx->num_sms &&
           positions * 2 * split * (int64_t)sizeof(float) <= (int64_t)pool_parts_bytes(ctx->num_sms))
        split *= 2;
    const MassArgs a{cu_new, seq_lens, S, T, Hq, Hkv, G, tile_tokens, small_tokens, lse, (const __nv_bfloat16*)k_pool,
                     (uint32_t)(k_stride * 2), map, scale * kLog2e, split > 1 ? (float*)ctx->pool_parts : score_out,
                     split > 1 ? map.reach : score_ld, split > 1 ? positions : 0, ctx->dev_err, max(1, ctx->num_sms / split), split,
                     wait_ns, stuck};
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (!work) {
        if (score_in == score_out) return KVSEL_OK;
        mass_copy_kernel<<<dim3((unsigned)min((map.reach + 1023) / 1024, 1024), S), 256, 0, s>>>(score_in, score_out, score_ld, map.reach);
        e = cudaGetLastError();
    } else {
        auto run = [&](auto call) { return call(ctx, mq, ms, mk, a, score_in, score_out, score_ld, s); };
        e = slot_map ? D == 64 ? run(launch<64, true>) : run(launch<128, true>) : D == 64 ? run(launch<64, false>) : run(launch<128, false>);
    }
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "attention_mass launch");
}

}  // namespace

extern "C" int kvsel_attention_mass(kvsel_ctx* ctx, const void* q, int64_t q_stride, const float* lse, const int32_t* cu_new,
                                    int S, int T, int Hq, int Hkv, int D, const void* k_pool, int64_t k_stride, int P, int page,
                                    const int32_t* seq_lens, const int32_t* slot_map, const int32_t* block_table, int ld,
                                    int dead_slot, float scale, const float* score_in, float* score_out, int64_t score_ld,
                                    void* stream) {
    const kvsel_trace trace_("kvsel_attention_mass");
    return mass_call(ctx, q, q_stride, lse, cu_new, S, T, Hq, Hkv, D, k_pool, k_stride, P, page, seq_lens, slot_map, block_table, ld,
                     dead_slot, scale, score_in, score_out, score_ld, stream, kWaitNs, 0);
}

// Test entry (not part of the public header): kvsel_attention_mass in which the issuer of every block waits on a barrier that
// nothing completes, with every wait limited to wait_ns.  It gives up while copies are in flight; the score holds no
// meaningful values afterwards.
extern "C" int kvsel_test_attention_mass_give_up(kvsel_ctx* ctx, const void* q, int64_t q_stride, const float* lse,
                                                 const int32_t* cu_new, int S, int T, int Hq, int Hkv, int D, const void* k_pool,
                                                 int64_t k_stride, int P, int page, const int32_t* seq_lens, const int32_t* slot_map,
                                                 const int32_t* block_table, int ld, int dead_slot, float scale,
                                                 const float* score_in, float* score_out, int64_t score_ld, uint64_t wait_ns,
                                                 void* stream) {
    const kvsel_trace trace_("kvsel_test_attention_mass_give_up");
    if (wait_ns == 0 || wait_ns > kWaitNs)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "test_attention_mass_give_up: wait_ns must be in (0, 1 s]");
    return mass_call(ctx, q, q_stride, lse, cu_new, S, T, Hq, Hkv, D, k_pool, k_stride, P, page, seq_lens, slot_map, block_table, ld,
                     dead_slot, scale, score_in, score_out, score_ld, stream, wait_ns, 1);
}
