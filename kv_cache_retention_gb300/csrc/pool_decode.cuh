// kvsel_pool_attention for sessions of few new tokens (decode steps, drafted tokens): up to 32 rows for each kv head.
//
// The mathematics are those of pool_attention.cu.  What bounds these sessions is the way of their K and V from memory, so here
// a block takes two neighbouring kv heads of the same tokens at once, as the two tiles: they share the lists (making them
// is what took longest where few tokens of a long map are live), their rows of a slot lie side by side, and each has a ring of
// three K and V tiles of its own, so that the next list's rows are on their way during this one's softmax.  The rows of tile 0
// are TMEM lanes 0 to 31, those of tile 1 lanes 32 to 63: one warp each has the softmax, on SM sub-partitions of their own.  The
// other lanes' rows are whatever lies behind the queries in shared memory, and are not looked at.
// Measured: 36 sessions of 20000 to 32768 tokens pruned to a quarter, 32/8 heads of 128, 977 MB: 179 us with the join (5.5 TB/s,
// 82% of a copy's rate; DRAM reads are 977 MB, so each row is read once); the chunks' kernel took 263 us.  One session of 92160
// tokens, 40/8 heads: 71 us (5.3 TB/s).
//
// 384 threads: warp 0 plans and makes the lists, warps 1 and 2 issue the two tiles' MMAs, warp 3 loads the queries, warps 4, 5
// and 6, 7 the K and V tiles, warps 8 and 9 are the softmax (10 and 11 only make up their warpgroup).
#pragma once

#include "pool_attention.cuh"

namespace {
namespace decode {

constexpr int kThreads = 384;
// Registers per thread: at launch, then after setmaxnreg (an .inc beyond the launch's registers would wait forever; the launcher
// checks the compiled count).
constexpr int kRegsLaunch = 168, kRegsCtl = 120, kRegsSoft = 240;
static_assert(2 * kRegsCtl + kRegsSoft <= 3 * kRegsLaunch && kRegsLaunch * kThreads <= 65536, "register split");
constexpr int kRows = 32, kHeads = 2;
constexpr int kLists = 8;
// Lists that the start of a session counts as when shares are cut, and that a share has at least, so cut.  Measured: starts of 1
// and 4 and shares of 2 change nothing; with shares of 4 one token behind 2048 takes 16.4 us, not 13.
constexpr int kStart = 2, kLeast = 1;

// What a block has of a session that others share: O as [D/4][32 rows] of four dims, then references and sums; per head.
constexpr int kPartHead = kRows * (128 + 2), kPart = kHeads * kPartHead;

template <int D>
struct Cfg {
    static constexpr int kBlock = kTile * 128;             // 128 rows x 64 dims, 128-byte swizzled
    static constexpr int kBytes = D / 64 * kBlock;         // one tile of K or V
    static constexpr int kQBlock = kRows * 128;            // the same of the queries, 32 rows
    static constexpr int kQ = kHeads * (D / 64) * kQBlock;
    static constexpr int kStages = 3;                      // K and V tiles of each head, in turn
    static constexpr int kOut = kHeads * 32 * 64;          // 32 rows of 32 dims of each head, on their way out
    struct Piece {
        int row, tokens, pos0, session, stop, part, end;   // as in pool_attention.cu
    };
    struct Tail {
        Lists<kLists> lists;
        uint64_t q_full, q_empty, full[kHeads][kStages], empty[kHeads][kStages], s_full[2], p_full[2][2], o_done[2], o_free[2][2],
            piece_full[2], piece_empty[2], drained;
        Stop stop;
        uint64_t never;                 // nothing completes it
        uint32_t tmem;
        Piece piece[2];
    };
    static constexpr size_t kSmem = (size_t)kQ + kHeads * kStages * kBytes + kOut + sizeof(Tail) + 1024;
    static_assert(kSmem <= 232448, "shared memory per block");
};

// K of list i is tile 2 i of its head's, V tile 2 i + 1: stage and phase of the p-th.
__device__ __forceinline__ uint32_t stage_of(uint32_t p) { return p % 3; }
__device__ __forceinline__ uint32_t phase_of(uint32_t p) { return p / 3 & 1; }

template <int D>
__device__ __forceinline__ void issue_tiles(typename Cfg<D>::Tail& t, const uint8_t* sq, const uint8_t* ring, int tile, bool idle, int lane,
                                            bool stuck, Stop* stop, unsigned* err) {
    using C = Cfg<D>;
    const uint32_t X = uniform(tile);
    uint32_t base = 0, steps = 0;       // tiles and steps so far
    bool ok = !stuck || wait_short(&t.never, 0, stop, err);
    const uint32_t ts = uniform(kTmem + kColS + X * kTile), to = uniform(kTmem + kColO + X * D);
    // (rows 32 and on of tile 1 are its queries)
    const uint32_t q = uniform(desc_low(saddr(sq) + X * (D / 64 * C::kQBlock - kRows * 128), 16));
    for (uint32_t u = 0; ok; ++u) {
        if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, err))) break;
        if (t.piece[u & 1].end) break;
        int n = 0;                      // lists of the piece that are known of
        bool ended = false;
        auto there_is = [&](int i) {    // list i; looks no more often than it has to
            if (ended || n > i) return i < n;
            uint32_t t0 = 0, tries = 0;
#pragma unroll 1
            for (;;) {
                const int p = t.lists.progress[u & 1];
                n = p >> 1;
                ended = p & 1;
                if (ended || n > i) break;
                __nanosleep(50);
                if (gives_up(tries, t0, stop, err)) {
                    ok = false;
                    break;
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            n = __shfl_sync(0xffffffffu, n, 0);
            ended = __shfl_sync(0xffffffffu, ended, 0);
            return i < n;
        };
        ok = wait_short(&t.q_full, u & 1, stop, err);
        if (idle) {
            if (ok && lane == 0) mbar_arrive(&t.q_empty);
        } else {
            // Round i: O += P V of list i (not before the first), then S of list i + 1 (while there is one).
#pragma unroll 1
            for (int i = -1; ok; ++i) {
                const bool more = there_is(i + 1), product = i >= 0;
                const uint32_t pv = base + 2 * i + 1, pk = pv + 1, sv = stage_of(pv), sk = stage_of(pk);
                const uint32_t vd = uniform(desc_low(saddr(ring) + (X * C::kStages + sv) * C::kBytes, C::kBlock));
                const uint32_t kd = uniform(desc_low(saddr(ring) + (X * C::kStages + sk) * C::kBytes, 16));
                if (product) {
                    if (u && i == 0) ok = wait_lane(&t.o_free[X][(u - 1) & 1], ((u - 1) >> 1) & 1, stop, err) && ok;
                    ok = wait_lane2(&t.full[X][sv], phase_of(pv), &t.p_full[X][0], steps & 1, stop, err) && ok;
                    fence_async();
                    tc_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k)
                            mma_ts_one(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), k > 0 || i > 0);
                    }
                    __syncwarp();
                    ok = wait_lane(&t.p_full[X][1], steps & 1, stop, err) && ok;
                    tc_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = kTile / 32; k < kTile / 16; ++k)
                            mma_ts_one(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), 1);
                        // (V's stage takes the K tile after next: it is not to wait for the next one's arrival)
                        mma_commit_one(saddr(&t.empty[X][sv]));
                    }
                    __syncwarp();
                    ++steps;
                }
                if (more) {             // S writes over the P read above: one thread's MMAs run in the order of issue
                    ok = wait_lane(&t.full[X][sk], phase_of(pk), stop, err) && ok;
                    fence_async();
                    tc_after();
                }
                if (elect_one()) {
                    if (more) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t in = (k & 3) * 32;
                            mma_ss_one(ts, q + (((k >> 2) * C::kQBlock + in) >> 4), kd + (((k >> 2) * C::kBlock + in) >> 4), idesc(kTile, false),
                                       k > 0);
                        }
                        mma_commit_one(saddr(&t.s_full[X]));
                        mma_commit_one(saddr(&t.empty[X][sk]));
                    } else {
                        if (product) mma_commit_one(saddr(&t.o_done[X]));
                        mma_commit_one(saddr(&t.q_empty));
                    }
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok);
                if (!more) break;
            }
            base += 2 * n;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
    }
    if (elect_one()) mma_commit_one(saddr(&t.drained));
    __syncwarp();
    drain_phase(&t.drained, 0);
}

template <int D, bool MAP>
__global__ void __launch_bounds__(kThreads, 1)
    pool_decode_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PoolArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    // (an offset and not a cast, so that the compiler knows it for shared memory)
    uint8_t* const smem = smem_raw + (-saddr(smem_raw) & 1023u);
    uint8_t* const sq = smem;
    uint8_t* const ring = smem + C::kQ;           // [kHeads][kStages][kBytes]
    typename C::Tail& t = *reinterpret_cast<typename C::Tail*>(ring + kHeads * C::kStages * C::kBytes + C::kOut);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = (a.Hkv + kHeads - 1) / kHeads, head0 = (int)(blockIdx.x % pairs) * kHeads, share = (int)(blockIdx.x / pairs);
    const bool alone = head0 + 1 == a.Hkv;        // the second head is not there
    Stop* const stop = &t.stop;

    if (threadIdx.x == 0) {
        mbar_init(&t.q_full, 1);
        mbar_init(&t.q_empty, 2);
        for (int x = 0; x < 2; ++x) {
            for (int i = 0; i < C::kStages; ++i) mbar_init(&t.full[x][i], 64), mbar_init(&t.empty[x][i], 1);
            mbar_init(&t.s_full[x], 1);
            mbar_init(&t.p_full[x][0], 1);
            mbar_init(&t.p_full[x][1], 1);
            mbar_init(&t.o_done[x], 1);
            mbar_init(&t.o_free[x][0], 1);
            mbar_init(&t.o_free[x][1], 1);
            mbar_init(&t.piece_full[x], 1);
            mbar_init(&t.piece_empty[x], 1 + 4 + 2 + 2);  // the queries, the loads, the issuers, the softmax warps
        }
        for (int i = 0; i < kLists; ++i) mbar_init(&t.lists.full[i], 1), mbar_init(&t.lists.empty[i], 4 + 2);  // the loads, the softmax warps
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
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = t.tmem;

    if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    if (warp == 0) {
        // ---- the share's pieces, and their lists ----
        unsigned err = 0;
        bool ok = true;
        uint32_t u = 0, made = 0;
        auto publish = [&](const typename C::Piece& w) {
            if (u >= 2 && !(ok = wait_idle(&t.piece_empty[u & 1], ((u >> 1) - 1) & 1, stop, a.err))) return;
            if (lane == 0) {
                t.piece[u & 1] = w;
                t.lists.progress[u & 1] = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.piece_full[u & 1]);
            ++u;
        };
        // The work, in keys: sessions of few tokens one after the other, kStart lists and their tokens.
        auto size_of = [&](const Session& x) { return x.count > 0 && x.count <= a.few ? (int64_t)x.len + kStart * kTile : 0; };
        int64_t total = 0;
        for (int s = lane; s < a.S; s += 32) {
            total += size_of(session_at(a.cu, a.lens, a.T, a.map.reach, s));
            if (blockIdx.x == 0) err |= session_errors(a.cu, a.lens, a.T, a.map.reach, s);
        }
        total = warp_sum(total);
        const int64_t quota = max((total + a.shares - 1) / a.shares, (int64_t)kLeast * kTile), from = share * quota, to = from + quota;
        int64_t at = 0;                 // where session s starts
        if (lane == 0) a.joints[blockIdx.x].sharers = 0;
        for (int s0 = 0; ok && s0 < a.S && at < to; s0 += 32) {
            Session mine{0, 0, 0};
            if (s0 + lane < a.S) mine = session_at(a.cu, a.lens, a.T, a.map.reach, s0 + lane);
            const int64_t size = size_of(mine), all = warp_sum(size);
            if (at + all <= from) {     // 32 sessions before the share
                at += all;
                continue;
            }
            for (int i = 0; ok && i < 32 && s0 + i < a.S && at < to; ++i) {
                const int64_t u0 = at, here = __shfl_sync(0xffffffffu, size, i), u1 = u0 + here;
                at = u1;
                if (here == 0 || u1 <= from) continue;
                typename C::Piece w;
                w.row = __shfl_sync(0xffffffffu, mine.first, i);
                w.tokens = __shfl_sync(0xffffffffu, mine.count, i);
                const int len = __shfl_sync(0xffffffffu, mine.len, i);
                const int lists = max(1, (int)(((int64_t)len + kTile - 1) / kTile));
                auto list_at = [&](int64_t p) {   // lists of the session that lie before place p of the work
                    return (int)min((int64_t)lists, max((int64_t)0, (p - u0) / kTile - kStart));
                };
                const int l0 = from <= u0 ? 0 : list_at(from), l1 = to >= u1 ? lists : list_at(to);
                if (l0 >= l1) continue;
                w.pos0 = len - w.tokens;
                w.session = s0 + i;
                w.stop = (int)min((int64_t)l1 * kTile, (int64_t)len);
                w.part = l0 > 0 ? 0 : l1 < lists ? 1 : -1;
                w.end = 0;
                if (w.part == 1 && lane == 0) {
                    // the last share with some of it starts before its last list does
                    const int64_t tail = min(u1, u0 + (int64_t)(lists + kStart) * kTile) - 1;
                    a.joints[blockIdx.x] = Joint{(int)(tail / quota) - share + 1, w.row, w.tokens};
                }
                publish(w);
                ok = ok && make_lists<MAP>(t.lists, a.map, a.map.map + (int64_t)(s0 + i) * a.map.ld, l0 * kTile, w.stop, w.pos0, made,
                                           &t.lists.progress[(u - 1) & 1], lane, stop, a.err, err);
            }
        }
        if (ok) {
            typename C::Piece w{};
            w.end = 1;
            publish(w);
        }
        if (err) atomicOr(a.err, err);
    } else if (warp == 1 || warp == 2) {
        issue_tiles<D>(t, sq, ring, warp - 1, warp == 2 && alone, lane, a.stuck && warp == 1, stop, a.err);
    } else if (warp == 3) {
        // ---- queries ----
        uint32_t loaded = 0;
        bool ok = true;
        for (uint32_t u = 0; ok; ++u) {
            if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
            const typename C::Piece w = t.piece[u & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
            if (w.end) break;
            if (u && !(ok = wait_idle(&t.q_empty, (u - 1) & 1, stop, a.err))) break;
            if (lane == 0) {
                const int heads = alone ? 1 : 2;
                mbar_expect_tx(&t.q_full, heads * (D / 64) * a.few * a.G * 128);
                for (int x = 0; x < heads; ++x)
                    for (int b = 0; b < D / 64; ++b)
                        tma_load(&map_q, &t.q_full, sq + (x * (D / 64) + b) * C::kQBlock, 64 * b, (head0 + x) * a.G, w.row);
            }
            ++loaded;
        }
        if (loaded) drain_phase(&t.q_full, (loaded - 1) & 1);
    } else {
        // ---- K and V tiles of a head: half of each a warp ----
        const int x = (warp - 4) >> 1;
        const bool idle = x == 1 && alone;
        uint32_t c = 0, l = 0;          // tiles and lists so far
        bool ok = true;
        for (uint32_t u = 0; ok; ++u) {
            if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
            const bool end = t.piece[u & 1].end;
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
            if (end) break;
            bool last = false;
            for (; ok && !last; ++l) {
                const uint32_t at = l % kLists;
                if (!(ok = wait_short(&t.lists.full[at], l / kLists & 1, stop, a.err))) break;
                const ListMeta meta = t.lists.meta[at];
                last = meta.last;
#pragma unroll 1
                for (int v = 0; ok && v < 2 && meta.n && !idle; ++v, ++c) {
                    const uint32_t st = stage_of(c);
                    if (!(ok = wait_short(&t.empty[x][st], phase_of(c) ^ 1, stop, a.err))) break;
                    load_rows<D, 2>(v ? &map_v : &map_k, v ? a.v : a.k, v ? a.v_bytes : a.k_bytes, (head0 + x) * D, t.lists.token + at * kTile,
                                    meta.n, meta.runs, ring + (x * C::kStages + st) * C::kBytes, &t.full[x][st], warp & 1, lane);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.lists.empty[at]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (uint32_t p = c > C::kStages ? c - C::kStages : 0; p < c; ++p) drain_phase(&t.full[x][stage_of(p)], phase_of(p));
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    if (warp < 10) {
        // ---- softmax: one row per thread ----
        const int x = warp - 8;
        const bool idle = x == 1 && alone;
        const int tok = lane / a.G, head = (head0 + x) * a.G + lane - tok * a.G;
        const uint32_t lanes = kTmem + ((uint32_t)(x * 32) << 16), ts = lanes + kColS + x * kTile, to = lanes + kColO + x * D;
        const float sc = a.scale2;
        uint32_t done = 0, mine = 0, base = 0, l = 0;  // this tile's steps and outputs, its tiles of K and V, and lists so far
        bool ok = true;
        for (uint32_t u = 0; ok; ++u) {
            if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
            const typename C::Piece w = t.piece[u & 1];
            __syncwarp();
            if (w.end) break;
            const int rows = w.tokens * a.G, row_pos = w.pos0 + tok;
            float ref = -3e38f;
            float2 sum = make_float2(0.f, 0.f);
            int n = 0, odd = INT_MAX;   // lists; the first key of a list with NaN or infinite values, set to zero
            bool last = false;
            for (; !last; ++l) {
                if (!(ok = wait_short(&t.lists.full[l % kLists], l / kLists & 1, stop, a.err))) break;
                const ListMeta meta = t.lists.meta[l % kLists];
                last = meta.last;
                if (meta.n && !idle) {
                    if (!(ok = wait_short(&t.s_full[x], done & 1, stop, a.err))) break;
                    const int2* const list = t.lists.token + l % kLists * kTile;
                    if (meta.causal) {
                        // NaN and infinities of V to zero
                        const uint32_t p = base + 2 * n + 1, st = stage_of(p);
                        if (!(ok = wait_short(&t.full[x][st], phase_of(p), stop, a.err))) break;
                        uint4* const tile = reinterpret_cast<uint4*>(ring + (x * C::kStages + st) * C::kBytes);
                        bool hits = false;
#pragma unroll 2
                        for (int e = lane; e < C::kBytes / 16; e += 32) {
                            const uint4 v = tile[e];
                            uint32_t y[4] = {v.x, v.y, v.z, v.w}, hit = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) hit |= (y[k] & 0x7F807F80u) + 0x00800080u;
                            if (hit & 0x80008000u) {
                                hits = true;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if ((y[k] & 0x7F80u) == 0x7F80u) y[k] &= 0xFFFF0000u;
                                    if ((y[k] & 0x7F800000u) == 0x7F800000u) y[k] &= 0x0000FFFFu;
                                }
                                tile[e] = make_uint4(y[0], y[1], y[2], y[3]);
                            }
                        }
                        if (__any_sync(0xffffffffu, hits)) odd = min(odd, list[0].y);
                        fence_async();
                    }
                    tc_after();
                    uint32_t s[kTile];
#pragma unroll
                    for (int b = 0; b < 4; ++b) tmem_ld32(ts + 32 * b, s + 32 * b);
                    tmem_wait_ld();
                    if (meta.causal || meta.n < kTile) {
                        // the row sees the list's tokens up to its own position: those before place `seen`
                        int seen = 0;
#pragma unroll
                        for (int step = kTile; step; step >>= 1)
                            if (seen + step <= meta.n && list[seen + step - 1].y <= row_pos) seen += step;
#pragma unroll
                        for (int c = 0; c < kTile; ++c)
                            if (c >= seen) s[c] = 0xFF800000u;
                    }
                    float m[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) m[b] = __uint_as_float(s[b]);
#pragma unroll
                    for (int c = 4; c + 8 <= kTile; c += 8)
#pragma unroll
                        for (int b = 0; b < 4; ++b) m[b] = max3(m[b], __uint_as_float(s[c + b]), __uint_as_float(s[c + 4 + b]));
#pragma unroll
                    for (int b = 0; b < 4; ++b) m[b] = fmaxf(m[b], __uint_as_float(s[kTile - 4 + b]));
                    // (rows of no token hold anything, and have no say in when references move)
                    const float top = lane < rows ? fmaxf(max3(m[0], m[1], m[2]), m[3]) * sc : -INFINITY;
                    if (n == 0) {
                        ref = fmaxf(top, -3e38f);  // of a row whose logits here are all -inf: low, and finite
                    } else if (__any_sync(0xffffffffu, top > ref + kSlack)) {
                        // references move up: the sums so far and O shrink with them
                        const float next = fmaxf(ref, top), f = ex2(ref - next);
                        ref = next;
                        sum.x *= f, sum.y *= f;
                        // (the commit that brought this S came after the last step's product: O is at rest)
#pragma unroll 1
                        for (int b = 0; b < D / 32; ++b) {
                            uint32_t o[32];
                            tmem_ld32(to + 32 * b, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                            tmem_st32(to + 32 * b, o);
                        }
                    }
                    const float2 sc2 = make_float2(sc, sc), nr = make_float2(-ref, -ref);
                    // in two halves, so that the product with V starts on the first while the second is worked out
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            uint32_t p[kTile / 8];
#pragma unroll
                            for (int c = 0; c < kTile / 8; ++c) {
                                const int e0 = half * (kTile / 2) + part * (kTile / 4) + 2 * c;
                                const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[e0]), __uint_as_float(s[e0 + 1])), sc2, nr);
                                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                                sum = __fadd2_rn(sum, e);
                                p[c] = pack_bf16(e.x, e.y);
                            }
                            tmem_st16(ts + 32 * half + 16 * part, p);
                        }
                        tmem_wait_st();
                        tc_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&t.p_full[x][half]);
                    }
                    ++done;
                }
                n += meta.n != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.lists.empty[l % kLists]);
            }
            if (!ok) break;
            base += 2 * n;
            // ---- output ----
            if (!idle) {
                if (n && !(ok = wait_short(&t.o_done[x], mine++ & 1, stop, a.err))) break;
                tc_after();
                uint32_t all[D];        // all at once, so that the next piece's products may start on O
                if (n) {
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) tmem_ld32(to + 32 * b, all + 32 * b);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int c = 0; c < D; ++c) all[c] = 0;
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.o_free[x][u & 1]);
                const float l_sum = sum.x + sum.y;
                const int64_t row_at = (int64_t)(w.row + tok) * a.Hq + head;
                float* const part = w.part < 0 ? nullptr : a.parts + ((size_t)blockIdx.x * 2 + w.part) * kPart + x * kPartHead;
                if (part) {
#pragma unroll
                    for (int c = 0; c < D / 4; ++c)
                        reinterpret_cast<uint4*>(part)[c * kRows + lane] = make_uint4(all[4 * c], all[4 * c + 1], all[4 * c + 2], all[4 * c + 3]);
                    part[kRows * 128 + lane] = ref;
                    part[kRows * 129 + lane] = l_sum;
                } else {
                    // through shared memory, as in pool_attention.cu
                    const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
                    const int row_off = tok * a.Hq + head;
                    uint8_t* const stage = ring + kHeads * C::kStages * C::kBytes + x * (32 * 64);
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) {
                        const uint32_t* const o = all + 32 * b;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t e[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                e[k] = pack_bf16(__uint_as_float(o[8 * c + 2 * k]) * inv, __uint_as_float(o[8 * c + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4*>(stage + lane * 64 + (c ^ ((lane >> 1) & 3)) * 16) = make_uint4(e[0], e[1], e[2], e[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int rr = 8 * c + (lane >> 2), off = __shfl_sync(0xffffffffu, row_off, rr);
                            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((lane & 3) ^ ((rr >> 1) & 3)) * 16);
                            if (rr < rows)
                                *reinterpret_cast<uint4*>(a.out + ((int64_t)w.row * a.Hq + off) * D + 32 * b + 8 * (lane & 3)) = v;
                        }
                        __syncwarp();
                    }
                    if (a.lse && lane < rows) a.lse[row_at] = l_sum == 0.f ? -INFINITY : (ref + log2f(l_sum)) * kLn2;
                }
                if (odd != INT_MAX)
                    add_odd<D, MAP>(a, w.session, head0 + x, odd, lane < rows ? min(row_pos, w.stop - 1) : -1, lane, [&](int d, float add) {
                        if (part)
                            part[((d >> 2) * kRows + lane) * 4 + (d & 3)] += add;
                        else
                            a.out[row_at * D + d] = __float2bfloat16_rn(__bfloat162float(a.out[row_at * D + d]) + add);
                    });
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
        }
    }
    tc_before();
    __syncthreads();
}

// Joins the session whose first keys block blockIdx.x has: one head's 32 dims a block, a row per lane, every eighth part a
// warp, so that the parts' loads are on their way together.
template <int D>
__global__ void __launch_bounds__(256) pool_decode_join_kernel(const PoolArgs a) {
    __shared__ float tops[8][kRows], sums[8][kRows];
    __shared__ float4 os[8][8][kRows];  // [warp][dims][row]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Joint u = a.joints[blockIdx.x];
    const int pairs = (a.Hkv + kHeads - 1) / kHeads, x = blockIdx.y / (D / 32), d0 = blockIdx.y % (D / 32) * 8;
    const int g = (int)(blockIdx.x % pairs) * kHeads + x;
    if (!u.sharers || g >= a.Hkv) return;
    const int warp = threadIdx.x >> 5, r = threadIdx.x & 31, rows = u.tokens * a.G;
    auto part = [&](int k) { return a.parts + ((size_t)(blockIdx.x + k * pairs) * 2 + (k == 0)) * kPart + x * kPartHead; };
    float top = -3e38f, sum = 0.f;
    float4 o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
#pragma unroll 2
        for (int k = warp; k < u.sharers; k += 8) {
            const float* const p = part(k);
            const float ref = p[kRows * 128 + r], l = p[kRows * 129 + r], next = fmaxf(top, ref), f0 = ex2(top - next), f1 = ex2(ref - next);
            top = next;
            sum = sum * f0 + l * f1;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float4 y = reinterpret_cast<const float4*>(p)[(d0 + c) * kRows + r];
                o[c].x = o[c].x * f0 + y.x * f1, o[c].y = o[c].y * f0 + y.y * f1;
                o[c].z = o[c].z * f0 + y.z * f1, o[c].w = o[c].w * f0 + y.w * f1;
            }
        }
    tops[warp][r] = top, sums[warp][r] = sum;
#pragma unroll
    for (int c = 0; c < 8; ++c) os[warp][c][r] = o[c];
    __syncthreads();
    if (r >= rows) return;
    // the warps' parts in order; warp w: dims d0 + w
    float all = tops[0][r], total = 0.f;
#pragma unroll
    for (int w = 1; w < 8; ++w) all = fmaxf(all, tops[w][r]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w >= u.sharers) break;      // (its part is nothing, whatever its reference)
        const float f = ex2(tops[w][r] - all);
        const float4 z = os[w][warp][r];
        total += f * sums[w][r];
        y.x += f * z.x, y.y += f * z.y, y.z += f * z.z, y.w += f * z.w;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int tok = r / a.G;
    const int64_t at = (int64_t)(u.row + tok) * a.Hq + g * a.G + r - tok * a.G;
    *reinterpret_cast<uint2*>(a.out + at * D + (d0 + warp) * 4) = make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
    if (a.lse && d0 == 0 && warp == 0) a.lse[at] = total == 0.f ? -INFINITY : (all + log2f(total)) * kLn2;
}

template <int D, bool MAP>
cudaError_t launch(kvsel_ctx* ctx, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PoolArgs& a,
                   cudaStream_t s) {
    auto* kernel = pool_decode_kernel<D, MAP>;
    constexpr uint64_t kBit = (uint64_t)KVSEL_READY_DECODE << (D / 64 - 1 + 2 * MAP);
    if (!(ctx->ready & kBit)) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split counts on it
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        ctx->ready |= kBit;
    }
    const unsigned blocks = (unsigned)a.shares * ((a.Hkv + kHeads - 1) / kHeads);
    kernel<<<blocks, kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.shares == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, kHeads * (D / 32));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pool_decode_join_kernel<D>, a);
}

}  // namespace decode
}  // namespace
