// kvsel_pool_attention: attention of packed new tokens over the bf16 page pools, on the 5th-generation tensor cores.
//
// Token i of a session sits at position pos = len - count + i and sees the live tokens j <= pos:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale log2e q . k_j - ref),  lse = ln sum_j e^(scale q . k_j).
//
// Rows.  A tile has the G = Hq/Hkv heads of one kv head for as many tokens as fit 128 rows (TMEM lanes), token by token, so
// that they share each key: a chunk of a prompt fills the tiles, a decode step has G rows.  A unit of work is two tiles of
// one session and kv head.
//
// Keys go through lists of 128 live tokens that one warp makes from the map (dropped tokens cost an entry's read and no
// more); their rows come by TMA where slots are consecutive, else by cp.async.  Per list and tile
//   S = Q K^T   tcgen05.mma, both operands from shared memory, 128 fp32 columns
//   P = 2^(S sc - ref) in bf16, written over S in TMEM
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory as it lies
// Where a unit fills both tiles, they share every K and V tile and take turns: one's softmax runs beside the other's
// products.  Where it has rows for one, TMEM's second half takes every other list for the same rows, and the two results
// are put together at the end.
//
// The softmax keeps per row a reference that only follows the running maximum when that has passed it by 8 (log2): weights
// are then at most 2^8, which bf16 and the fp32 sums hold as well as 1, and O is rescaled only then.  P is rounded to bf16
// since both operands of the product have one type and V's range is bf16's: 2^-8 at most per weight, at random, about the
// output's own rounding.
//
// 512 threads: warp 0 plans and makes the lists, warps 1 and 2 issue the MMAs of one tile each, warps 4-7 load, warps 8-11 and
// 12-15 are the softmax of the two tiles, a row per thread.  TMEM: S of tile 0 and 1 at columns 0 and 128, O at 256 and on.
//
// Shares.  The units' keys, laid end to end with some for the start of each, are cut into equal shares, found from the
// lengths on the device; neighbouring blocks take a share for one kv head each (the heads' rows of a slot lie side by side).
// What a block has of a unit that others have a part of goes to memory of a fixed size, and a second small kernel joins
// the parts in the order of the blocks.
//
// Masked places.  A weight of zero does not hide a NaN or an infinity in V.  In lists that not every row sees whole, the
// softmax warps set such values to zero in shared memory before the product, and if there were any, each row adds those it
// does see to its output at the end (what the sum would be: infinite or NaN).
//
// Measured: 2048 tokens behind 32768, 32/8 heads of 128, 0.84 to 0.86 ms (1.32 to 1.36 PFLOP/s, three quarters of a sustained
// matrix product's rate).  No unit is full: tensor pipe 66%, issue slots 50%, DRAM 32%.  Steps on the way there: rows by TMA gathers of four slots
// took 2.73 ms, an issuer's waits within its turn 1.09 and ahead of it 0.98, MMAs in a branch of one elected thread 0.97 -> 0.86;
// without turns it took 1.05 where turns took 0.98.
//
// Every wait is bounded (1 s); on a timeout the block flags KVSEL_ERR_TIMEOUT in the device error word, drains its own copies
// and MMAs, frees TMEM and returns.
#include <limits.h>

#include "pool_decode.cuh"

namespace {

constexpr int kThreads = 512;
// Registers per thread: at launch, then after the first warpgroup's setmaxnreg.dec and the softmax warpgroups' .inc.  An
// .inc beyond the launch's registers would wait forever; the launcher checks the compiled count.
constexpr int kRegsLaunch = 128, kRegsCtl = 72, kRegsSoft = 184;
static_assert(2 * kRegsCtl + 2 * kRegsSoft <= 4 * kRegsLaunch && kRegsLaunch * kThreads <= 65536, "register split");
constexpr int kLists = 8;
// Lists that the start of a unit counts as when shares are cut, and that a share has at least, so cut.  Measured: a start of 2
// costs a batch of 16 sessions of 1 to 1013 new tokens 2 to 5%, one of 8 changes nothing; no difference between shares of 1 to 8.
constexpr int kStart = 4, kLeast = 4;

template <int D>
struct Cfg {
    static constexpr int kBlock = kTile * 128;             // 128 rows x 64 dims, 128-byte swizzled
    static constexpr int kBytes = D / 64 * kBlock;         // one tile of Q, K or V
    static constexpr int kStages = 4;                      // K and V tiles share the ring (at_k and at_v count on four)
    static constexpr int kOut = 8 * 32 * 64;               // 32 rows of 32 dims for each softmax warp, on their way out
    // What a block does of one unit; end: there is nothing more.
    struct Piece {
        int row, tokens, pos0;          // first token in q, how many, the first one's position
        int session, stop;              // the piece's keys lie below position stop
        int part;                       // -1: the whole unit, else which partial result it is
        int two, end;
    };
    struct Tail {
        Lists<kLists> lists;
        uint64_t q_full, q_empty, full[kStages], empty[kStages], s_full[2], p_full[2][2], o_done[2], o_free[2][2], turn[2],
            piece_full[2], piece_empty[2], merge[2], drained;
        Stop stop;
        uint64_t never;                 // nothing completes it
        uint32_t tmem;
        int odd[2];                     // of the two pieces: the first key of a list with NaN or infinite values, set to zero
        Piece piece[2];
        float2 other[2][kTile];         // tile 1's references and sums, where both tiles have the same rows
    };
    static constexpr size_t kSmem = (size_t)(2 + kStages) * kBytes + kOut + sizeof(Tail) + 1024;
    static_assert(kSmem <= 232448, "shared memory per block");
};

// Places in the ring of list i's K and V tile, from the piece's first one on.  Where the two tiles share the lists (two): K0,
// K1, V0, K2, V1, ..., V(n-1) with the last list's V right behind its K.  Where they have every other list: K0, K1, V0, V1, K2,
// K3, ..., a place for each of a last pair, so that a stage of the ring is one tile's alone.
__device__ __forceinline__ int at_k(bool two, int i) { return !two ? (i >> 1) * 4 + (i & 1) : i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int at_v(bool two, int i, bool last) { return !two ? (i >> 1) * 4 + 2 + (i & 1) : last ? 2 * i + 1 : 2 * i + 2; }
__device__ __forceinline__ int places(bool two, int n) { return two ? 2 * n : (n + 1) / 2 * 4; }

// ---- MMAs: a warp per tile -------------------------------------------------
// Two issuers on two SM sub-partitions that take turns, so that one tile's products run beside the other's softmax.  One
// copy of the code for both.  Where they share lists, both see and release every tile of the ring; where they have every
// other list, a stage of the ring is one warp's alone for the whole piece.  A wait for a phase that is two behind would return
// at once, one for a phase with another one done behind it never: so such a piece begins, and ends, when all the tiles of the one
// before have been used, and the barriers of O are in pairs (a piece does not begin before the one two before it has been read).
template <int D>
__device__ __forceinline__ void issue_tiles(typename Cfg<D>::Tail& t, const uint8_t* sq, const uint8_t* ring, int tile, int lane,
                                            bool stuck, Stop* stop, unsigned* err) {
    using C = Cfg<D>;
    constexpr uint32_t kStages = C::kStages;
    const uint32_t lead = lane == 0, X = uniform(tile);
    uint32_t base = 0, turns = 0, steps = 0;  // ring places, turns and this tile's steps so far
    bool was_two = true;
    bool ok = !stuck || wait_short(&t.never, 0, stop, err);
    const uint32_t ts = uniform(kTmem + kColS + X * kTile), to = uniform(kTmem + kColO + X * D);
    for (uint32_t u = 0; ok; ++u) {
        if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, err))) break;
        const bool two = t.piece[u & 1].two;
        if (t.piece[u & 1].end) break;
        int n = 0;                                // lists of the piece that are known of
        bool ended = false;
        auto there_is = [&](int i) {              // list i; looks no more often than it has to
            if (ended || n > i) return i < n;
            uint32_t t0 = 0, tries = 0;
#pragma unroll 1
            for (;;) {
                const int p = t.lists.progress[u & 1];
                n = p >> 1;
                ended = p & 1;
                if (ended || n > i) break;
                __nanosleep(100);
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
        if (!(two && was_two) && u) {             // the tiles of the ring that the other warp alone has seen have landed
#pragma unroll 1
            for (int x = 0; x < 2; ++x) ok = ok && wait_short(&t.o_free[x][(u - 1) & 1], ((u - 1) >> 1) & 1, stop, err);
        }
        was_two = two;
        const int by = two ? 1 : 2, first = two ? 0 : (int)X;
        const uint32_t q = uniform(desc_low(saddr(sq) + (two ? X * C::kBytes : 0u), 16));
        // Round i: O += P V of list i (not before the first), then S of list i + by (while there is one).
#pragma unroll 1
        for (int i = first - by; ok; i += by) {
            const bool more = there_is(i + by), product = i >= first;
            if (!more) mma_commit(saddr(&t.q_empty), lead);  // no further S: Q is released when the ones issued have ended
            const uint32_t av = base + at_v(two, i, ended && i == n - 1), ak = base + at_k(two, i + by);
            const uint32_t vd = uniform(desc_low(saddr(ring) + av % kStages * C::kBytes, C::kBlock));
            const uint32_t kd = uniform(desc_low(saddr(ring) + ak % kStages * C::kBytes, 16));
            // one answer for the lanes at the end of the round
            uint64_t* const k_full = &t.full[ak % kStages];
            const uint32_t k_par = ak / kStages & 1;
            if (product) {
                // K, V, this tile's turn and the first half of P
                uint64_t* const v_full = &t.full[av % kStages];
                const uint32_t v_par = av / kStages & 1;
                const bool turn = two && (X == 1 || i > 0);
                if (u && i == first) ok = wait_lane(&t.o_free[X][(u - 1) & 1], ((u - 1) >> 1) & 1, stop, err) && ok;
                ok = wait_lane4(v_full, v_par, more ? k_full : v_full, more ? k_par : v_par, turn ? &t.turn[X] : v_full,
                                turn ? turns & 1 : v_par, &t.p_full[X][0], steps & 1, stop, err) && ok;
                turns += turn;
                fence_async();
                tc_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k)
                        mma_ts_one(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), k > 0 || i != first);
                }
                __syncwarp();
                ok = wait_lane(&t.p_full[X][1], steps & 1, stop, err) && ok;
                tc_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = kTile / 32; k < kTile / 16; ++k)
                        mma_ts_one(to, ts + k * 8, vd + k * (2048 >> 4), idesc(D, true), 1);
                }
                __syncwarp();
                ++steps;
            } else {
                if (more) ok = wait_lane(k_full, k_par, stop, err) && ok;
                fence_async();
                tc_after();
            }
            if (elect_one()) {
                if (more) {                       // writes over the P read above: one thread's MMAs run in the order of issue
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * C::kBlock + (k & 3) * 32) >> 4;
                        // the other tile's turn: its issuer is under way while the last of these are issued
                        if (k == D / 32 && two && product) mbar_arrive(&t.turn[X ^ 1]);
                        mma_ss_one(ts, q + off, kd + off, idesc(kTile, false), k > 0);
                    }
                    mma_commit_one(saddr(&t.s_full[X]));
                    mma_commit_one(saddr(&t.empty[ak % kStages]));
                    if (!two) mma_commit_one(saddr(&t.empty[ak % kStages]));  // for the other warp too
                } else if (product) {
                    if (two && X == 0) mbar_arrive(&t.turn[1]);
                    mma_commit_one(saddr(&t.o_done[X]));
                }
                if (product) {
                    mma_commit_one(saddr(&t.empty[av % kStages]));
                    if (!two) mma_commit_one(saddr(&t.empty[av % kStages]));
                }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            if (!more) break;
        }
        if (!two && X == 1 && (n & 1)) {          // the places of the list that is not there
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                const uint32_t at = base + (v ? at_v(false, n, true) : at_k(false, n));
                ok = ok && wait_short(&t.full[at % kStages], at / kStages & 1, stop, err);
                if (ok && lead) mbar_arrive(&t.empty[at % kStages]), mbar_arrive(&t.empty[at % kStages]);
            }
        }
        base += places(two, n);
        __syncwarp();
        if (lead) mbar_arrive(&t.piece_empty[u & 1]);
    }
    mma_commit(saddr(&t.drained), lead);
    drain_phase(&t.drained, 0);
}

// ---- shares ----------------------------------------------------------------
// The work of one kv head, in keys: units in the order of sessions and tokens, kStart lists for the start of each and then
// the keys that its last row sees, counted as if the last unit of a session were full (which makes a session's sum a
// closed form).
struct Cut {
    int64_t lead;                       // keys of the session before its new tokens, and the start
    int unit;                           // tokens of a unit
    __device__ __forceinline__ int64_t before(int64_t t) const { return t * lead + unit * (t * (t + 1) / 2); }
};
__device__ __forceinline__ Cut cut_of(const Session& x, int unit) {
    return Cut{(int64_t)max(0, x.len - x.count) + kStart * kTile, unit};
}
__device__ __forceinline__ int units_of(const Session& x, int unit) { return (int)(((int64_t)x.count + unit - 1) / unit); }

// ---- the kernel ------------------------------------------------------------

template <int D, bool MAP>
__global__ void __launch_bounds__(kThreads, 1)
    pool_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const PoolArgs a) {
    using C = Cfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    // (an offset and not a cast, so that the compiler knows it for shared memory)
    uint8_t* const smem = smem_raw + (-saddr(smem_raw) & 1023u);
    uint8_t* const sq = smem;                     // [2][kBytes]
    uint8_t* const ring = smem + 2 * C::kBytes;   // [kStages][kBytes]
    typename C::Tail& t = *reinterpret_cast<typename C::Tail*>(smem + (2 + kStages) * C::kBytes + C::kOut);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = (int)(blockIdx.x % a.Hkv), share = (int)(blockIdx.x / a.Hkv);
    Stop* const stop = &t.stop;

    if (threadIdx.x == 0) {
        mbar_init(&t.q_full, 1);
        mbar_init(&t.q_empty, 2);
        for (int i = 0; i < kStages; ++i) mbar_init(&t.full[i], 32), mbar_init(&t.empty[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t.s_full[i], 1);
            mbar_init(&t.p_full[i][0], 4);
            mbar_init(&t.p_full[i][1], 4);
            mbar_init(&t.o_done[i], 1);
            mbar_init(&t.o_free[i][0], 4);
            mbar_init(&t.o_free[i][1], 4);
            mbar_init(&t.turn[i], 1);
            mbar_init(&t.merge[i], 4);
            mbar_init(&t.piece_full[i], 1);
            mbar_init(&t.piece_empty[i], 4 + 2 + 8);  // the loads, the issuers, the softmax warps
        }
        for (int i = 0; i < kLists; ++i) mbar_init(&t.lists.full[i], 1), mbar_init(&t.lists.empty[i], 2 + 8);  // the loads of K and of V, the softmax warps
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
        if (warp >= 4) {
            // ---- loads ----
            const uint32_t mine = warp - 4;
            uint32_t c = 0, l = 0, loaded_q = 0;  // ring places and lists so far, Q loads
            uint32_t loaded = 0;                  // one behind the last place that this warp has filled
            bool ok = true;
            auto release = [&](uint32_t list) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.lists.empty[list % kLists]);
            };
            for (uint32_t u = 0; ok; ++u) {
                if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
                const typename C::Piece w = t.piece[u & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
                if (w.end) break;
                if (u && !(ok = wait_idle(&t.q_empty, (u - 1) & 1, stop, a.err))) break;
                if (warp == 4 && lane == 0) {
                    mbar_expect_tx(&t.q_full, (1 + w.two) * (D / 64) * a.tile_tokens * a.G * 128);
                    for (int x = 0; x < 1 + w.two; ++x)
                        for (int b = 0; b < D / 64; ++b)
                            tma_load(&map_q, &t.q_full, sq + x * C::kBytes + b * C::kBlock, 64 * b, g * a.G,
                                     w.row + x * a.tile_tokens);
                }
                ++loaded_q;
                int n = 0;                        // lists of the piece so far
                bool ended = false;
                auto there_is = [&](int i) {      // list i
#pragma unroll 1
                    while (ok && !ended && n <= i) {
                        const uint32_t at = (l + n) % kLists;
                        if (!(ok = wait_idle(&t.lists.full[at], (l + n) / kLists & 1, stop, a.err))) break;
                        ended = t.lists.meta[at].last;
                        if (t.lists.meta[at].n)
                            ++n;
                        else if (mine < 2)        // (as the two loads of a list would)
                            release(l);
                    }
                    return i < n;
                };
                // every kStages-th place of the ring: a stage of it is this warp's
#pragma unroll 1
                for (int p = (mine - c) % kStages; ok; p += kStages) {
                    int i = w.two ? (p + 1) / 2 : p / 4 * 2 + (p & 1);
                    bool v = w.two ? p > 0 && !(p & 1) : (p & 2) != 0, last = false;
                    if (w.two && v) i -= 1;
                    bool real = there_is(i);
                    if (w.two && v && !there_is(i + 1)) break;  // V of the last list is elsewhere
                    if (!real) {
                        if (!(p & 1) || !(w.two ? i == n : i - 1 < n)) break;
                        last = true;              // V of the last list, right behind its K; or a place without a list
                        if (w.two) i -= 1, v = real = true;
                    }
                    const uint32_t at = c + p, list = (l + i) % kLists;
                    if (!(ok = ok && wait_idle(&t.empty[mine], (at / kStages & 1) ^ 1u, stop, a.err))) break;
                    if (real) {
                        load_rows<D, 1>(v ? &map_v : &map_k, v ? a.v : a.k, v ? a.v_bytes : a.k_bytes, g * D, t.lists.token + list * kTile,
                                     t.lists.meta[list].n, t.lists.meta[list].runs, ring + mine * C::kBytes, &t.full[mine], 0, lane);
                        release(l + i);
                    } else {
                        mbar_arrive(&t.full[mine]);
                    }
                    loaded = at + 1;
                    if (last) break;
                }
                there_is(INT_MAX);                // (warps see every list)
                c += places(w.two, n);
                l += max(n, 1);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (loaded) drain_phase(&t.full[mine], (loaded - 1) / kStages & 1);
            if (warp == 4 && loaded_q) drain_phase(&t.q_full, (loaded_q - 1) & 1);
        } else if (warp == 1 || warp == 2) {
            issue_tiles<D>(t, sq, ring, warp - 1, lane, a.stuck && warp == 1, stop, a.err);
        } else if (warp == 0) {
            // ---- the share's pieces, and their lists ----
            unsigned err = 0;
            bool ok = true;
            uint32_t u = 0, made = 0;
            auto publish = [&](const typename C::Piece& w) {
                if (u >= 2 && !(ok = wait_idle(&t.piece_empty[u & 1], ((u >> 1) - 1) & 1, stop, a.err))) return;
                if (lane == 0) {
                    t.piece[u & 1] = w;
                    t.odd[u & 1] = INT_MAX;
                    t.lists.progress[u & 1] = 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.piece_full[u & 1]);
                ++u;
            };
            const int unit = 2 * a.tile_tokens;
            int64_t total = 0;
            for (int s = lane; s < a.S; s += 32) {
                Session x = session_at(a.cu, a.lens, a.T, a.map.reach, s);
                if (x.count <= a.few) x.count = 0;  // (another kernel's)
                total += cut_of(x, unit).before(units_of(x, unit));
                if (blockIdx.x == 0) err |= session_errors(a.cu, a.lens, a.T, a.map.reach, s);
            }
            total = warp_sum(total);
            const int64_t quota = max((total + a.shares - 1) / a.shares, (int64_t)kLeast * kTile);
            const int64_t from = share * quota, to = from + quota;
            int64_t at = 0;                       // where session s starts
            if (lane == 0) a.joints[blockIdx.x].sharers = 0;
            for (int s0 = 0; ok && s0 < a.S && at < to; s0 += 32) {
                Session mine{0, 0, 0};
                if (s0 + lane < a.S) mine = session_at(a.cu, a.lens, a.T, a.map.reach, s0 + lane);
                if (mine.count <= a.few) mine.count = 0;
                const int64_t size = cut_of(mine, unit).before(units_of(mine, unit));
                const int64_t all = warp_sum(size);
                if (at + all <= from) {           // 32 sessions before the share
                    at += all;
                    continue;
                }
                for (int i = 0; ok && i < 32 && s0 + i < a.S && at < to; ++i) {
                    Session x;
                    x.first = __shfl_sync(0xffffffffu, mine.first, i);
                    x.count = __shfl_sync(0xffffffffu, mine.count, i);
                    x.len = __shfl_sync(0xffffffffu, mine.len, i);
                    const int64_t here = __shfl_sync(0xffffffffu, size, i);
                    if (at + here <= from) {
                        at += here;
                        continue;
                    }
                    const Cut cut = cut_of(x, unit);
                    const int n = units_of(x, unit);
                    int k = 0;                    // the first unit that ends behind the share's start
                    for (int step = 1 << 24; step; step >>= 1)
                        if (k + step <= n && at + cut.before(k + step) <= from) k += step;
                    const int32_t* const row = a.map.map + (int64_t)(s0 + i) * a.map.ld;
                    for (; ok && k < n; ++k) {
                        const int64_t u0 = at + cut.before(k), u1 = at + cut.before(k + 1);
                        if (u0 >= to) break;
                        const int tok0 = k * unit, tokens = min(unit, x.count - tok0);
                        const int keys = max(0, x.len - x.count + tok0 + tokens);
                        const int lists = max(1, (int)(((int64_t)keys + kTile - 1) / kTile));
                        auto list_at = [&](int64_t p) {   // lists of the unit that lie before place p of the work
                            return (int)min((int64_t)lists, max((int64_t)0, (p - u0) / kTile - kStart));
                        };
                        const int l0 = from <= u0 ? 0 : list_at(from), l1 = to >= u1 ? lists : list_at(to);
                        if (l0 >= l1) continue;
                        typename C::Piece w;
                        w.row = x.first + tok0;
                        w.tokens = tokens;
                        w.pos0 = x.len - x.count + tok0;
                        w.session = s0 + i;
                        w.stop = (int)min((int64_t)l1 * kTile, (int64_t)keys);
                        w.part = l0 > 0 ? 0 : l1 < lists ? 1 : -1;
                        w.two = tokens > a.tile_tokens;
                        w.end = 0;
                        if (w.part == 1 && lane == 0) {
                            // the last share with some of it starts before its last list does
                            const int64_t tail = min(u1, u0 + (int64_t)(lists + kStart) * kTile) - 1;
                            a.joints[blockIdx.x] = Joint{(int)(tail / quota) - share + 1, w.row, tokens};
                        }
                        publish(w);
                        ok = ok && make_lists<MAP>(t.lists, a.map, row, l0 * kTile, w.stop, w.pos0, made, &t.lists.progress[(u - 1) & 1], lane, stop, a.err, err);
                    }
                    at += here;
                }
            }
            if (ok) {
                typename C::Piece w{};
                w.end = 1;
                publish(w);
            }
            if (err) atomicOr(a.err, err);
        }
        __syncwarp();
        tc_before();
        __syncthreads();
        tc_after();
        if (warp == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ---- softmax: one row per thread ----
    const int x = (warp - 8) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const int r_tok = r / a.G, r_head = g * a.G + r - r_tok * a.G;
    const uint32_t lane_base = kTmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t ts = lane_base + kColS + x * kTile, to = lane_base + kColO + x * D;
    const float sc = a.scale2;
    uint32_t done = 0, mine = 0, base = 0, l = 0;  // this tile's steps and outputs, ring places and lists so far
    bool ok = true;
    for (uint32_t u = 0; ok; ++u) {
        if (!(ok = wait_idle(&t.piece_full[u & 1], (u >> 1) & 1, stop, a.err))) break;
        const typename C::Piece w = t.piece[u & 1];
        __syncwarp();
        if (w.end) break;
        const int tok0 = w.two ? x * a.tile_tokens : 0, rows = min(a.tile_tokens, w.tokens - tok0) * a.G;
        const bool active = quarter * 32 < rows;        // the warp has rows
        const int row_pos = w.pos0 + tok0 + r_tok;
        float ref = -3e38f;
        float2 sum = make_float2(0.f, 0.f);
        int n = 0, steps = 0;
        bool last = false;
        for (; !last; ++l) {
            if (!(ok = wait_idle(&t.lists.full[l % kLists], l / kLists & 1, stop, a.err))) break;
            const ListMeta meta = t.lists.meta[l % kLists];
            last = meta.last;
            const int i = n;
            n += meta.n != 0;
            if (meta.n && (w.two || (i & 1) == x)) {
                if (!(ok = wait_short(&t.s_full[x], done & 1, stop, a.err))) break;
                if (meta.causal) {
                    // NaN and infinities of V to zero; both tiles look at all of it (a value may be set twice)
                    const uint32_t at = base + at_v(w.two, i, last), st = at % kStages;
                    if (!(ok = wait_short(&t.full[st], at / kStages & 1, stop, a.err))) break;
                    uint4* const tile = reinterpret_cast<uint4*>(ring + st * C::kBytes);
#pragma unroll 1
                    for (int e = r; e < C::kBytes / 16; e += kTile) {
                        const uint4 v = tile[e];
                        uint32_t y[4] = {v.x, v.y, v.z, v.w}, hit = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) hit |= (y[k] & 0x7F807F80u) + 0x00800080u;
                        if (hit & 0x80008000u) {
                            atomicMin(&t.odd[u & 1], t.lists.token[l % kLists * kTile].y);
                            __threadfence_block();
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((y[k] & 0x7F80u) == 0x7F80u) y[k] &= 0xFFFF0000u;
                                if ((y[k] & 0x7F800000u) == 0x7F800000u) y[k] &= 0x0000FFFFu;
                            }
                            tile[e] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                    fence_async();
                    __syncwarp();
                }
                tc_after();
                if (!active) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&t.p_full[x][0]), mbar_arrive(&t.p_full[x][1]);
                } else {
                    uint32_t s[kTile];
#pragma unroll
                    for (int b = 0; b < 4; ++b) tmem_ld32(ts + 32 * b, s + 32 * b);
                    tmem_wait_ld();
                    if (meta.causal || meta.n < kTile) {
                        // the row sees the list's tokens up to its own position: those before place `seen`
                        const int2* const list = t.lists.token + l % kLists * kTile;
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
                    const float top = r < rows ? fmaxf(max3(m[0], m[1], m[2]), m[3]) * sc : -INFINITY;
                    if (steps == 0) {
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
                }
                ++steps, ++done;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.lists.empty[l % kLists]);
        }
        if (!ok) break;
        base += places(w.two, n);
        // ---- output ----
        if (steps && !(ok = wait_short(&t.o_done[x], mine++ & 1, stop, a.err))) break;
        tc_after();
        float l_sum = sum.x + sum.y;
        if (x == 1) {                                   // to the thread that has the row's other part, if that is so
            t.other[u & 1][r] = make_float2(ref, l_sum);
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.merge[u & 1]);
        }
        if (w.two || x == 0) {
            uint32_t all[D];          // all at once, so that the next piece's products may start on O
            if (steps && active) {
#pragma unroll
                for (int b = 0; b < D / 32; ++b) tmem_ld32(to + 32 * b, all + 32 * b);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int c = 0; c < D; ++c) all[c] = 0;
            }
            if (!w.two) {
                if (!(ok = wait_short(&t.merge[u & 1], (u >> 1) & 1, stop, a.err))) break;
                tc_after();
                if (n > 1 && active) {
                    const float2 o = t.other[u & 1][r];
                    const float next = fmaxf(ref, o.x), f0 = ex2(ref - next), f1 = ex2(o.x - next);
                    ref = next;
                    l_sum = l_sum * f0 + o.y * f1;
#pragma unroll
                    for (int b = 0; b < D / 16; ++b) {
                        uint32_t y[16];
                        tmem_ld16(to + D + 16 * b, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            all[16 * b + c] = __float_as_uint(__uint_as_float(all[16 * b + c]) * f0 + __uint_as_float(y[c]) * f1);
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.o_free[1][u & 1]);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.o_free[x][u & 1]);
            const int64_t row_at = (int64_t)(w.row + tok0 + r_tok) * a.Hq + r_head;
            float* const part = w.part < 0 ? nullptr : a.parts + ((size_t)blockIdx.x * 2 + w.part) * kPart + x * kPartTile;
            if (active && part) {
#pragma unroll
                for (int c = 0; c < D / 4; ++c)
                    reinterpret_cast<uint4*>(part)[c * kTile + r] = make_uint4(all[4 * c], all[4 * c + 1], all[4 * c + 2], all[4 * c + 3]);
                part[kTile * 128 + r] = ref;
                part[kTile * 129 + r] = l_sum;
            } else if (active) {
                // through shared memory, so that a store covers 64 bytes of each of eight rows; 16-byte pieces are swizzled by
                // their row against bank conflicts
                const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
                const int row_off = (tok0 + r_tok) * a.Hq + r_head;
                uint8_t* const stage = smem + (2 + kStages) * C::kBytes + (warp - 8) * (32 * 64);
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
                        if (quarter * 32 + rr < rows)
                            *reinterpret_cast<uint4*>(a.out + ((int64_t)w.row * a.Hq + off) * D + 32 * b + 8 * (lane & 3)) = v;
                    }
                    __syncwarp();
                }
                if (a.lse && r < rows) a.lse[row_at] = l_sum == 0.f ? -INFINITY : (ref + log2f(l_sum)) * kLn2;
            }
            const int odd = __shfl_sync(0xffffffffu, *(volatile int*)&t.odd[u & 1], 0);
            if (odd != INT_MAX)
                add_odd<D, MAP>(a, w.session, g, odd, r < rows ? min(row_pos, w.stop - 1) : -1, lane, [&](int d, float add) {
                    if (part)
                        part[((d >> 2) * kTile + r) * 4 + (d & 3)] += add;
                    else
                        a.out[row_at * D + d] = __float2bfloat16_rn(__bfloat162float(a.out[row_at * D + d]) + add);
                });
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&t.piece_empty[u & 1]);
    }
    tc_before();
    __syncthreads();
}

// Joins the unit whose first keys block blockIdx.x has: 32 rows of a tile a block, a row per lane, four dims at a time.
template <int D>
__global__ void __launch_bounds__(256) pool_join_kernel(const PoolArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Joint u = a.joints[blockIdx.x];
    if (!u.sharers) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = blockIdx.y >> 2, r = (blockIdx.y & 3) * 32 + lane;
    const int rows = min(a.tile_tokens, u.tokens - x * a.tile_tokens) * a.G;
    if ((int)(blockIdx.y & 3) * 32 >= rows) return;
    auto part = [&](int k) {
        return a.parts + ((size_t)(blockIdx.x + k * a.Hkv) * 2 + (k == 0)) * kPart + x * kPartTile;
    };
    float top = -3e38f, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < u.sharers; ++k) top = fmaxf(top, part(k)[kTile * 128 + r]);
    float4 o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < u.sharers; ++k) {
        const float* const p = part(k);
        const float f = ex2(p[kTile * 128 + r] - top);
        sum += f * p[kTile * 129 + r];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const float4 y = reinterpret_cast<const float4*>(p)[(warp + 8 * c) * kTile + r];
            o[c].x += f * y.x, o[c].y += f * y.y, o[c].z += f * y.z, o[c].w += f * y.w;
        }
    }
    if (r >= rows) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = r / a.G;
    const int64_t at = (int64_t)(u.row + x * a.tile_tokens + tok) * a.Hq + (int)(blockIdx.x % a.Hkv) * a.G + r - tok * a.G;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        *reinterpret_cast<uint2*>(a.out + at * D + (warp + 8 * c) * 4) =
            make_uint2(pack_bf16(o[c].x * inv, o[c].y * inv), pack_bf16(o[c].z * inv, o[c].w * inv));
    if (a.lse && warp == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D, bool MAP>
cudaError_t launch(kvsel_ctx* ctx, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PoolArgs& a,
                   cudaStream_t s) {
    auto* kernel = pool_attention_kernel<D, MAP>;
    constexpr uint64_t kBit = (uint64_t)KVSEL_READY_POOL << (D / 64 - 1 + 2 * MAP);
    if (!(ctx->ready & kBit)) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split counts on it
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        ctx->ready |= kBit;
    }
    kernel<<<(unsigned)a.shares * a.Hkv, kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.shares == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.shares * a.Hkv, 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pool_join_kernel<D>, a);
}

int attention_call(kvsel_ctx* ctx, const void* q, int64_t q_stride, const int32_t* cu_new, int S, int T, int Hq, int Hkv, int D,
                   const void* k_pool, const void* v_pool, int64_t k_stride, int64_t v_stride, int P, int page,
                   const int32_t* seq_lens, const int32_t* slot_map, const int32_t* block_table, int ld, int dead_slot,
                   float scale, void* out, float* lse, void* stream, uint64_t wait_ns, int stuck) {
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    const void* pools[2] = {k_pool, v_pool};
    const int64_t strides[2] = {k_stride, v_stride};
    TokenMap map;
    rc = check_pool_call(ctx, "pool_attention", S, T, Hq, Hkv, D, q_stride, pools, strides, 2, P, page, slot_map, block_table,
                         ld, dead_slot, scale, &map);
    if (rc) return rc;
    if (S == 0 || T == 0) return KVSEL_OK;
    if (!q || !cu_new || !seq_lens || !out) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "pool_attention: null pointer");
    if ((reinterpret_cast<uintptr_t>(q) & 15u) || (reinterpret_cast<uintptr_t>(out) & 15u))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "pool_attention: q and out must be 16-byte aligned");
    const int G = Hq / Hkv, tile_tokens = kTile / G;
    const int most = decode::kRows / G;  // tokens that the rows of few hold
    // Sessions of few tokens go to the kernel for them where they may be most of the batch's; its launch is not worth it for
    // chunks, whose own kernel takes them too.  Where all tokens together are few, that one is not needed.  The host knows T and S
    // alone, so the rule goes by rows a session.  With and without the kernel, 36 sessions of 8192 tokens, 32/8 heads: new tokens
    // of 1 or 8 each 190 or 193 and 250 or 257 us; 8 and 16 by turns 260 and 260; 12, 16 or 24 each, where none are few, 291, 293
    // or 286 and 274, 276 or 271; 35 of one beside one of 256, 512 or 2048, 244, 265 or 404 and 305, 338 or 466.  The border at 64
    // rows lies behind 16 each and the one beside 512: two kernels for nothing cost 16 us there, and 62 are lost beside 2048.
    const bool few = most > 0 && (int64_t)T * G <= 2 * (int64_t)decode::kRows * S, all_few = T <= most;
    CUtensorMap mq, ms, mk, mv;
    if (!make_query_map(&mq, q, T, Hq, D, q_stride, G, tile_tokens) ||
        (few && !make_query_map(&ms, q, T, Hq, D, q_stride, G, most)) ||
        (P > 0 && (!make_pool_map(&mk, k_pool, P * page, Hkv, D, k_stride) ||
                   !make_pool_map(&mv, v_pool, P * page, Hkv, D, v_stride))))
        return kvsel_fail(ctx, KVSEL_ERR_CUDA, "pool_attention: tensor map encoding failed");
    if (P == 0) mk = mv = mq;           // nothing is live
    const int pairs = (Hkv + decode::kHeads - 1) / decode::kHeads;
    float* const parts = (float*)ctx->pool_parts;
    float* const few_parts = parts + (size_t)ctx->num_sms * 2 * kPart;
    Joint* const joints = (Joint*)(few_parts + (size_t)ctx->num_sms * 2 * decode::kPart);
    PoolArgs a{cu_new, seq_lens, S, T, Hq, Hkv, G, tile_tokens, few ? most : 0, (const __nv_bfloat16*)k_pool,
               (const __nv_bfloat16*)v_pool, (uint32_t)(k_stride * 2), (uint32_t)(v_stride * 2), map, scale * kLog2e,
               (__nv_bfloat16*)out, lse, ctx->dev_err, pairs < ctx->num_sms ? ctx->num_sms / pairs : 1, few_parts, joints,
               wait_ns, stuck};
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    auto run = [&](auto call, const CUtensorMap& m) { e = call(ctx, m, mk, mv, a, st); };
    if (few)
        slot_map ? D == 64 ? run(decode::launch<64, true>, ms) : run(decode::launch<128, true>, ms)
        : D == 64 ? run(decode::launch<64, false>, ms) : run(decode::launch<128, false>, ms);
    if (e == cudaSuccess && !(few && all_few)) {
        a.shares = Hkv < ctx->num_sms ? ctx->num_sms / Hkv : 1;
        a.parts = parts, a.joints = joints + 65536;
        slot_map ? D == 64 ? run(launch<64, true>, mq) : run(launch<128, true>, mq)
        : D == 64 ? run(launch<64, false>, mq) : run(launch<128, false>, mq);
    }
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "pool_attention launch");
}

}  // namespace

// Partial results and joints of the blocks: as many as there are SMs, or kv heads where those are more (their blocks have
// whole units and only clear their joints); of this kernel and of the one for few tokens.
size_t pool_parts_bytes(int num_sms) {
    return (size_t)num_sms * 2 * (kPart + decode::kPart) * sizeof(float) + (size_t)2 * 65536 * sizeof(Joint);
}

extern "C" int kvsel_pool_attention(kvsel_ctx* ctx, const void* q, int64_t q_stride, const int32_t* cu_new, int S, int T,
                                    int Hq, int Hkv, int D, const void* k_pool, const void* v_pool, int64_t k_stride,
                                    int64_t v_stride, int P, int page, const int32_t* seq_lens, const int32_t* slot_map,
                                    const int32_t* block_table, int ld, int dead_slot, float scale, void* out, float* lse,
                                    void* stream) {
    const kvsel_trace trace_("kvsel_pool_attention");
    return attention_call(ctx, q, q_stride, cu_new, S, T, Hq, Hkv, D, k_pool, v_pool, k_stride, v_stride, P, page, seq_lens,
                          slot_map, block_table, ld, dead_slot, scale, out, lse, stream, kWaitNs, 0);
}

// Test entry (not part of the public header): kvsel_pool_attention in which the issuer of tile 0 of every block waits on a
// barrier that nothing completes, with every wait limited to wait_ns.  It gives up while copies are in flight; out and lse
// hold no meaningful values afterwards.
extern "C" int kvsel_test_pool_attention_give_up(kvsel_ctx* ctx, const void* q, int64_t q_stride, const int32_t* cu_new, int S,
                                                 int T, int Hq, int Hkv, int D, const void* k_pool, const void* v_pool,
                                                 int64_t k_stride, int64_t v_stride, int P, int page, const int32_t* seq_lens,
                                                 const int32_t* slot_map, const int32_t* block_table, int ld, int dead_slot,
                                                 float scale, void* out, float* lse, uint64_t wait_ns, void* stream) {
    const kvsel_trace trace_("kvsel_test_pool_attention_give_up");
    if (wait_ns == 0 || wait_ns > kWaitNs)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "test_pool_attention_give_up: wait_ns must be in (0, 1 s]");
    return attention_call(ctx, q, q_stride, cu_new, S, T, Hq, Hkv, D, k_pool, v_pool, k_stride, v_stride, P, page, seq_lens,
                          slot_map, block_table, ld, dead_slot, scale, out, lse, stream, wait_ns, 1);
}
