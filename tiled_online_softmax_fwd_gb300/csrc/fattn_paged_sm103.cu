// fattn_paged_sm103.cu -- attention of new tokens over a paged key/value
// cache for GB300 (sm_103a): ragged batches, grouped heads, single tokens to
// long chunks in one call.
//
// For sequence b with n new tokens, the last of its L cached keys, and query
// head h reading key head h / G:
//
//   x_ij = scale q_i . k_j   for j < L and (causal) j <= L - n + i
//   o_i  = sum_j softmax(x_i)_j v_j,    lse_i = log sum_j exp(x_ij)
//
// by the online softmax (running maximum m and sum l, O rescaled when m
// grows; base 2, and m raised only past a threshold, which is exact algebra).
//
// Rows.  The G query heads of a key head attend to the same keys, so a Q tile
// packs them: row r of a tile is token r / G, head r % G, 128 / G tokens a
// tile.  A key tile is then read once for all of them: a decode step moves
// each key once, whatever G is.
//
// Bound.  With few new tokens the cache's bytes (HBM): 16 sequences of 16K to
// 32K keys, one token each, 32 query and 8 key heads, d = 128, bf16, take 247 us
// at 6.6 TB/s.  With many, the tensor cores and exponentials: two chunks of 2K
// tokens against 16K keys run at 1330 to 1480 TFLOP/s under the power cap (fp16,
// without the conversion of V, 1420 to 1470).  Short sequences are bound by a unit's start and end (see
// Costs).  One persistent CTA a SM serves all:
//   warps 0-7    two softmax warpgroups (thread = row)
//   warp 8       walks the CTA's work, publishes each piece of it to the other
//                warps, and copies: Q tiles, and pages into a ring of 128-key
//                tiles (TMA)
//   warp 9       MMA issuer: S = Q K^T and O += P V on tcgen05
//   warps 10-11  V in place: bf16 -> fp16 (P is fp16, and both operands of a
//                product share one type), and zeros behind the last key: a
//                slot no token has written may hold anything, and 0 * NaN
//                would reach every row
// A unit of work is a pair of Q tiles of one (sequence, key head).  Both tiles
// use each key tile (the warpgroups alternate, one in exponentials while the
// other's products run).  A unit with a single tile -- decode, drafts, the odd
// last tile -- has the two warpgroups take alternate key tiles of the same Q
// tile instead, into accumulators of their own that the epilogue merges, so
// the chain S -> softmax -> P V of one key tile overlaps the next one's.
//
// A single tile of at most 32 rows (decode steps) would leave one warp of each
// warpgroup with 128 exponentials a key tile, one after the other, and three
// idle: a warp reaches only its own 32 TMEM lanes.  So such rows are copied
// into all four lane quarters, and warp w takes keys 32 w .. 32 w + 31 of each
// key tile for its copy, with P zero at the others: four rows' statistics and
// accumulators instead of one, merged once a unit.
//
// Schedule.  Lengths live in device memory (a captured graph follows them),
// so the grid finds its own work: the units' costs, so much a key plus so much
// for a unit's start and end, have closed-form prefix sums; CTA c takes the
// c-th of equal ranges of their total.  A range may begin or end inside a
// unit: the unit is then split between CTAs by key tiles, each writes a
// partial O and log-sum-exp to its slot in the workspace (at most two a CTA),
// and combine_paged_kernel merges them in slot order.  Ranges depend only on
// the lengths and the SM count, so equal calls give equal bits.
//
// Code size.  Every role is code of its own, 127 KB in all at d = 64, and what
// the warps of a batch with units of several kinds run at a time does not fit
// the instruction caches: a CTA of quad units beside one of pairs took up to
// 1.5 times as long as beside its like.  So what does not stand in an inner
// loop is not unrolled, and divisions of 64 bits are calls.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "fattn_internal.h"
#include "ptx_sm103.cuh"

namespace fattn {
namespace {

using namespace ptx;

constexpr int kBM = 128;  // rows of a Q tile
constexpr int kBN = 128;  // keys of a key tile
constexpr int kThreads = 384;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpConv = 10;
constexpr int kPieces = 4;     // pieces published ahead
constexpr int kQuadRows = 32;  // rows of a tile that fit a lane quarter
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kChunkBytes = kBM * 128;  // 128 rows x 64 16-bit columns
// Epilogue staging of a softmax warp: 32 rows of 128 bytes, and room for the
// (m, l) of its rows, from the end.
constexpr uint32_t kStageBytes = 4096 + 128;
// Costs of a unit, in eighths of a key in a quad unit: its start and end, and
// each key it sees.  From a fit of the CTAs' cycles over eighteen ragged
// batches (16 to 40 sequences, up to 500 new tokens and 6000 keys): at d = 64 a
// quad unit took 4800 cycles and 1300 a key tile, another single tile 5800 and
// 1600, a pair of tiles 8300 and 2100; at d = 128 (bf16) 5800 and 2700, 9800 and
// 2700, 9800 and 3600.  With one cost for all, the slowest CTA of such a batch
// took 1.8 times the mean; with these 1.1 to 1.3 times.  The waits and copies
// have become shorter since (4200 and 1300, 4400 and 1600, 6100 and 2100 at d =
// 64), but costs fitted to that were no better over 24 such batches.  At d = 96
// equal whole units of 1 to 16 key tiles, keys from L2, take in these measures
// 2490, 3570 and 3860 and 8, 7.8 and 10.4 a key (a quad unit's tile: 0.96 us);
// the numbers here are within 15 % of that.  One set serves both types: fp16,
// without the conversion of V, takes 4 % less a tile of a quad unit and 8 to
// 15 % less of a pair, which moves the ratios by less than the fit is good for.
enum UnitKind { kQuad, kSingle, kPair };
struct Costs {
    int unit[3], key[3];
    // By a variable kind: selected, not indexed (the arrays stay constants).
    __device__ __forceinline__ int unit_of(int k) const
    {
        return k == kQuad ? unit[kQuad] : k == kSingle ? unit[kSingle] : unit[kPair];
    }
    __device__ __forceinline__ int key_of(int k) const
    {
        return k == kQuad ? key[kQuad] : k == kSingle ? key[kSingle] : key[kPair];
    }
};
template <int D> __device__ __forceinline__ constexpr Costs costs_of()
{
    return D == 64   ? Costs{{3750, 4530, 6550}, {8, 10, 13}}
           : D == 96 ? Costs{{2720, 3270, 4330}, {8, 9, 11}}
                     : Costs{{2190, 3730, 3740}, {8, 8, 11}};
}
// A CTA's share of the work is at least a quad unit of this many keys: below,
// the merge costs more than the shorter ranges save.  With 256 four decodes of
// 150 to 1100 keys took 16.7 us, with 128 15.2.
constexpr int kMinShareKeys = kBN;

template <int D, bool kF16> struct Cfg {
    static constexpr int kChunks = (D + 63) / 64;
    static constexpr uint32_t kTileBytes = kChunks * kChunkBytes;
    static constexpr int kStages = kChunks == 2 ? 4 : 8;
    static_assert(kStages % 2 == 0, "V is on the odd stages");
    static constexpr uint32_t kStageOffset = (2 + kStages) * kTileBytes;  // epilogue staging
    static constexpr uint32_t kBarsOffset = kStageOffset + 8 * kStageBytes;
    static constexpr uint32_t kColO0 = 256;  // O of warpgroup t at kColO0 + t D
};

// ------------------------------------------------------------------ schedule
struct Seq {
    int q0, n, L;  // first token, new tokens, keys
};

// A piece of work: key tiles [j0, j1) of a unit.
struct Piece {
    int h;        // key head; -1: no more work
    Seq s;
    int j0, j1;
    int slot;     // workspace slot of a partial result, or -1: the whole unit
    int alt;      // one Q tile: the warpgroups take alternate key tiles
    int lead;     // ... beginning with this one, which writes the result
    int quad;     // ... of at most 32 rows, copied to all four lane quarters
    int q_buf;    // a single tile's Q buffer: the two in turn
    int tile[2];  // Q tile of each warpgroup
    int rows[2];  // its rows
    int n[2];     // its key tiles in this piece
};

// A sequence's entries of the lists as they stand.
struct Raw {
    int c0, c1, L;
};

// Where a CTA starts: a unit (and its sequence's entries), the cost already
// behind in it, and how much of the total cost this CTA takes.
struct Start {
    int b, h, p;
    int snap;  // no split within this many key tiles of a unit's ends
    Raw raw;
    long long y, left;
};

struct Bars {
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[8], kv_empty[8], v_ready[8];
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2];
    uint64_t other_done;   // single-tile units: the statistics of the one that does not lead
    uint64_t quarters[2];  // quad units: merge steps of a warpgroup's four warps
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    Start start;
    Piece pieces[kPieces];
    long long warp_sum[kThreads / 32];
};

// A sequence's entries of the lists, and brought into range (bad: some value
// was not).
__device__ __forceinline__ Raw load_raw(const PagedArgs &a, int b)
{
    return Raw{a.cu_q[b], a.cu_q[b + 1], a.kv_len[b]};
}
__device__ __forceinline__ Seq in_range(const PagedArgs &a, Raw r, bool &bad)
{
    Seq s;
    s.q0 = min(max(r.c0, 0), a.T);
    s.n = min(max(r.c1, s.q0), a.T) - s.q0;
    s.n = min(s.n, a.max_q);
    s.L = min(max(r.L, 0), a.max_keys);
    bad = s.q0 != r.c0 || s.n != static_cast<long long>(r.c1) - r.c0 || s.L != r.L;
    return s;
}

__device__ __forceinline__ int tiles_of(const PagedArgs &a, const Seq &s)
{
    return (s.n + a.tile_tokens - 1) / a.tile_tokens;
}

// Keys that tokens before `end` see together.
__device__ __forceinline__ int keys_seen(const PagedArgs &a, const Seq &s, int end)
{
    return a.causal ? max(s.L - s.n + min(end, s.n), 0) : s.L;
}

// a / b of non-negative values, in 32 bits where they fit (64-bit division is a
// routine of some hundred instructions).
__device__ __noinline__ long long long_quotient(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    if (((a | b) >> 32) == 0)
        return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return long_quotient(a, b);
}

// The kind of a (sequence, head)'s unit p.
__device__ __forceinline__ int kind_of(const PagedArgs &a, const Seq &s, int tiles, int p)
{
    if (2 * p + 1 < tiles)
        return kPair;
    return (s.n - 2 * p * a.tile_tokens) * a.G <= kQuadRows && a.q_quad_tokens > 0 ? kQuad : kSingle;
}

// Cost of the first p of a (sequence, head)'s units.  Under the causal mask
// unit i sees off + (i + 1) R keys (none while that is negative), off = L - n,
// R tokens a unit; the last one sees L, and alone may be other than a pair.
__device__ __forceinline__ long long cost_before(const PagedArgs &a, const Costs &cost, const Seq &s,
                                                 int tiles, int p)
{
    const int units = (tiles + 1) / 2;
    if (units == 0)
        return 0;
    const long long i = min(p, units - 1);
    long long keys = i * s.L;
    if (a.causal) {
        const int over = s.n - s.L, per = 2 * a.tile_tokens;  // off = -over, R
        const long long off = -over, R = per;
        const long long z = over > 0 ? min(i, static_cast<long long>(over / per)) : 0;
        keys = (i - z) * off + R * ((i * (i + 1) - z * (z + 1)) / 2);
    }
    long long c = i * cost.unit[kPair] + keys * cost.key[kPair];
    if (p == units) {
        const int kind = kind_of(a, s, tiles, units - 1);
        c += cost.unit_of(kind) + static_cast<long long>(s.L) * cost.key_of(kind);
    }
    return c;
}

// Key tile that a cost of y inside a unit of `keys` keys falls on.
__device__ __forceinline__ int tile_at(long long y, int keys, int unit_cost, int key_cost, int snap)
{
    const int F = (keys + kBN - 1) / kBN;
    if (y <= 0)
        return 0;
    if (y >= unit_cost + static_cast<long long>(keys) * key_cost)
        return F;
    const int t = y < unit_cost ? 0 : static_cast<int>(quotient(y - unit_cost, kBN * key_cost));
    return t < snap ? 0 : F - t < snap ? F : t;
}

// The whole block finds this CTA's start: each thread sums the costs of a run
// of sequences, a scan gives the total and every run's place, and the thread
// whose run holds the CTA's first cost walks it.
__device__ void find_start(const PagedArgs &a, const Costs &cost, Bars &b)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    long long sum = 0;
    bool any_bad = false;
    Raw raw = {0, 0, 0};  // of the run's last sequence
#pragma unroll 1
    for (int i = b0; i < b1; ++i) {
        bool bad;
        raw = load_raw(a, i);
        const Seq s = in_range(a, raw, bad);
        any_bad = any_bad || bad || (i == 0 && raw.c0 != 0);
        const int tiles = tiles_of(a, s);
        sum += a.Hk * cost_before(a, cost, s, tiles, (tiles + 1) / 2);
    }
    if (any_bad && blockIdx.x == 0)
        atomicCAS(a.status, 0u, 6u /* FATTN_ERR_INDEX */ | (kRoleLoad << 8));
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += x;
    }
    if (lane == 31)
        b.warp_sum[warp] = incl;
    if (tid == 0) {
        b.start.b = -1;
        b.start.left = 0;
    }
    __syncthreads();
    long long before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? b.warp_sum[w] : 0;
        total += b.warp_sum[w];
    }
    const int least = cost.unit[kQuad] + kMinShareKeys * cost.key[kQuad];
    // CTA c takes [c total / shares, (c + 1) total / shares), formed without
    // long products.
    const int shares = static_cast<int>(
        min(static_cast<long long>(gridDim.x), max(quotient(total, least), 1LL)));
    const long long each = quotient(total, shares);
    const int rest = static_cast<int>(total - each * shares), c = blockIdx.x;
    const long long lo = c * each + c * rest / shares, hi = (c + 1) * each + (c + 1) * rest / shares;
    if (c < shares && lo < hi && before <= lo && lo < before + sum) {
        long long x = lo - before;
#pragma unroll 1
        for (int i = b0; i < b1; ++i) {
            bool bad;
            if (b1 - b0 > 1)
                raw = load_raw(a, i);
            const Seq s = in_range(a, raw, bad);
            const int tiles = tiles_of(a, s), units = (tiles + 1) / 2;
            const long long head = cost_before(a, cost, s, tiles, units);
            if (x >= head * a.Hk) {
                x -= head * a.Hk;
                continue;
            }
            Start st;
            st.b = i;
            st.raw = raw;
            st.h = static_cast<int>(quotient(x, head));
            x -= st.h * head;
            int p = 0, end = units;  // largest p with cost_before(p) <= x
#pragma unroll 1
            while (end - p > 1) {
                const int mid = (p + end) / 2;
                if (cost_before(a, cost, s, tiles, mid) <= x)
                    p = mid;
                else
                    end = mid;
            }
            st.p = p;
            st.y = x - cost_before(a, cost, s, tiles, p);
            st.left = hi - lo;
            st.snap = max(2, static_cast<int>(min(each / (64 * kBN * cost.key[kQuad]), 1LL << 20)));
            b.start = st;
            const int keys = keys_seen(a, s, (p + 1) * 2 * a.tile_tokens);
            const int kind = kind_of(a, s, tiles, p);
            const int t = tile_at(st.y, keys, cost.unit_of(kind), cost.key_of(kind), st.snap);
            const bool split = t > 0 && t < (keys + kBN - 1) / kBN;
            const int first = st.p * 2 * a.tile_tokens;
            a.starts[2 * c] = make_int4(st.b, st.h, st.p, split ? t : 0);
            a.starts[2 * c + 1] = make_int4(s.q0 + first, min(s.n - first, 2 * a.tile_tokens), 0, 0);
            break;
        }
    }
    if (tid == 0 && (c >= shares || lo >= hi))
        a.starts[2 * c] = make_int4(-1, 0, 0, 0);
}

// The same value on every lane of a converged warp, passed through a shuffle.
// Copy coordinates and descriptors are read from uniform registers; with a
// loop whose trip count comes from memory around it, a coordinate computed
// from values loaded outside the loop reached the copy without one of its
// terms (the rows of a later unit were then some other tokens'), although
// every lane held the right sum.  Why is not known; shuffled values are read
// afresh.  So every value of a copy or product that follows from the lists goes
// through one inside the loop that uses it: tokens, heads, slots, pages and
// ring positions here, tiles and ring positions in run_mma.  The shuffles and the
// votes of the waits also bring the warp's lanes together before each copy.
__device__ __forceinline__ int uniform(int x)
{
    return __shfl_sync(0xffffffffu, x, 0);
}
// The same where one lane runs alone: from `lane`, its own number as elect.sync
// gave it, which no compiler can tell from another lane's.
__device__ __forceinline__ int uniform_of(int x, uint32_t lane)
{
    return __shfl_sync(1u << lane, x, static_cast<int>(lane));
}
// The lane that elect_one picks.
__device__ __forceinline__ uint32_t elected_lane()
{
    uint32_t lane;
    asm volatile("{\n\t.reg .pred P1;\n\telect.sync %0|P1, 0xffffffff;\n\t}" : "=r"(lane));
    return lane;
}

// The pieces of this CTA in order.  The next sequence's list entries are
// fetched while the current one is worked on.
struct Walk {
    Start at;
    Seq s;
    int tiles, units;
    Raw next;
    int q_buf, lead;
    int at_b;        // sequence of the piece given last
    int again;       // heads that follow it with the same piece of their own
    long long cost;  // of that unit
};
__device__ __forceinline__ void enter(const PagedArgs &a, Walk &w, Raw r)
{
    bool bad;
    w.s = in_range(a, r, bad);
    w.tiles = tiles_of(a, w.s);
    w.units = (w.tiles + 1) / 2;
    if (w.at.b + 1 < a.B)
        w.next = Raw{r.c1, a.cu_q[w.at.b + 2], a.kv_len[w.at.b + 1]};
}
__device__ __forceinline__ Walk first_walk(const PagedArgs &a, const Bars &b)
{
    Walk w;
    w.at = b.start;
    w.q_buf = w.lead = w.again = 0;
    if (w.at.left > 0)
        enter(a, w, w.at.raw);
    return w;
}
// What changes from one single-tile piece to the next.
__device__ __forceinline__ void take_turn(Walk &w, Piece &u)
{
    const int n = u.j1 - u.j0;
    u.q_buf = w.q_buf;
    u.lead = w.lead;
    u.n[0] = (n + (w.lead == 0 ? 1 : 0)) / 2;
    u.n[1] = n - u.n[0];
    w.q_buf ^= 1;
    w.lead ^= n & 1;
}
__device__ __forceinline__ bool next_piece(const PagedArgs &a, const Costs &costs, Walk &w, Piece &u)
{
    if (w.again > 0) {  // the next head of the same sequence: all else is the same
        --w.again;
        ++w.at.h;
        w.at.left -= w.cost;
        u.h = w.at.h;
        if (u.alt)
            take_turn(w, u);
        return true;
    }
    while (w.at.left > 0) {
        if (w.at.p >= w.units) {  // past the head's (or an empty sequence's) last unit
            w.at.p = 0;
            if (w.units == 0 || ++w.at.h >= a.Hk) {
                w.at.h = 0;
                if (++w.at.b >= a.B)
                    return false;
                enter(a, w, w.next);
            }
            continue;
        }
        const int R = 2 * a.tile_tokens;
        const int keys = keys_seen(a, w.s, (w.at.p + 1) * R);
        const int F = (keys + kBN - 1) / kBN;
        const int kind = kind_of(a, w.s, w.tiles, w.at.p);
        const long long cost = costs.unit_of(kind) + static_cast<long long>(keys) * costs.key_of(kind);
        const long long y0 = w.at.y, y1 = min(y0 + w.at.left, cost);
        const int pair = w.at.p;
        w.at_b = w.at.b;
        u.h = w.at.h;
        u.s = w.s;
        u.j0 = tile_at(y0, keys, costs.unit_of(kind), costs.key_of(kind), w.at.snap);
        u.j1 = tile_at(y1, keys, costs.unit_of(kind), costs.key_of(kind), w.at.snap);
        w.at.left -= y1 - y0;
        w.at.y = 0;
        ++w.at.p;
        // Nothing of this unit falls to this CTA (a unit without keys belongs
        // to the CTA that holds its start).
        if (F == 0 ? y0 > 0 : u.j0 == u.j1)
            continue;
        const int cta = static_cast<int>(blockIdx.x);
        u.slot = u.j0 > 0 ? 2 * cta : u.j1 < F ? 2 * cta + 1 : -1;
        u.alt = kind != kPair;
        u.lead = u.q_buf = u.n[0] = u.n[1] = 0;
        u.tile[0] = 2 * pair;
        u.tile[1] = u.alt ? 2 * pair : 2 * pair + 1;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int first = u.tile[t] * a.tile_tokens;
            u.rows[t] = min(a.tile_tokens, u.s.n - first) * a.G;
            if (!u.alt) {
                const int ft = (keys_seen(a, u.s, first + a.tile_tokens) + kBN - 1) / kBN;
                u.n[t] = max(min(u.j1, ft) - u.j0, 0);
            }
        }
        if (u.alt && F > 0)
            take_turn(w, u);
        // One unit a head, given whole: the heads after it that fit into this
        // CTA's share whole get the same piece.
        w.cost = cost;
        if (w.units == 1 && u.slot < 0 && F > 0)
            w.again = static_cast<int>(min(quotient(w.at.left, cost), static_cast<long long>(a.Hk - 1 - u.h)));
        u.quad = kind == kQuad && F > 0;
        return true;
    }
    return false;
}

__device__ __forceinline__ void record_failure(const PagedArgs &a, Bars &b, uint32_t role)
{
    const uint32_t code = 4u /* FATTN_ERR_TIMEOUT */ | (role << 8) | ((blockIdx.x & 0xffffu) << 16);
    atomicCAS(a.status, 0u, code);
    *reinterpret_cast<volatile int *>(&b.abort) = 1;
}

__device__ __forceinline__ uint32_t timer_lo()
{
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
// Waits for a phase: false when the time is up or another role has given up.
// Few instructions, as there are some sixty of them (see Code size): 45 each, and
// the producer's copies unrolled throughout, made the kernel 150 KB, and the
// ragged d = 64 batch took 74 us instead of 62.
__device__ __forceinline__ bool lane_wait(uint64_t &bar, uint32_t parity, const volatile int *abort)
{
    const uint32_t at = smem_addr(&bar);
    bool ok = mbar_try_wait(at, parity);
    if (!ok) {
        const uint32_t t0 = timer_lo();
#pragma unroll 1
        do {
            ok = mbar_try_wait(at, parity);
        } while (!ok && *abort == 0 && timer_lo() - t0 < static_cast<uint32_t>(kWaitLimitNs));
    }
    return ok;
}
// The same by a whole warp; the outcome is uniform.
__device__ __forceinline__ bool warp_wait(uint64_t &bar, uint32_t parity, const volatile int *abort)
{
    return __all_sync(0xffffffffu, lane_wait(bar, parity, abort));
}

// The producer's end of the pieces: waits for a free place, writes, signals.
__device__ __forceinline__ bool publish(Bars &b, uint32_t k, const Piece &u)
{
    if (!warp_wait(b.piece_empty[k % kPieces], ((k / kPieces) & 1) ^ 1, &b.abort))
        return false;
    if ((threadIdx.x & 31) == 0)
        b.pieces[k % kPieces] = u;
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(smem_addr(&b.piece_full[k % kPieces]));
    return true;
}
// The k-th piece, read in place; false when there is none (ok) or the wait
// failed (!ok).  Held until given back.
__device__ __forceinline__ bool receive(Bars &b, uint32_t k, bool &ok)
{
    ok = ok && warp_wait(b.piece_full[k % kPieces], (k / kPieces) & 1, &b.abort);
    return ok && b.pieces[k % kPieces].h >= 0;
}
__device__ __forceinline__ void give_back(Bars &b, uint32_t k)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(smem_addr(&b.piece_empty[k % kPieces]));
}

template <bool kF16> __device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (kF16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// ------------------------------------------------------------------ producer
// K_j and V_j alternate through the ring, V on the odd stages.  A tile is 8
// pages of 16 slots down to part of one, a copy a page and 64-column box, all
// issued by one elected lane; the warp holds 32 table entries and the next 32.
template <int D, bool kF16>
__device__ void run_load(const PagedArgs &a, Bars &b, uint32_t smem_base, const CUtensorMap *mq,
                         const CUtensorMap *mq_quad, const CUtensorMap *mk, const CUtensorMap *mv)
{
    using C = Cfg<D, kF16>;
    const volatile int *abort = &b.abort;
    const int lane = threadIdx.x & 31;
    const bool leader = elect_one();
    const int shift = a.page_shift;
    const int per_tile = shift < 7 ? kBN >> shift : 1;  // pages a key tile touches
    const int box_rows = shift < 7 ? 1 << shift : kBN;
    const uint32_t q_row_bytes = C::kChunks * a.G * 128u;  // of a token
    uint32_t q_bits = 0, q_used = 0, pos = 0;  // of the Q buffers: phase, was ever filled
    bool ok = true;
    uint32_t pieces = 0;
    // The first table entries of the last piece: the next head's are the same.
    int held_b = -1, held_page = -1, held_cur = 0, held_ahead = 0;
    Walk w = first_walk(a, b);
    Piece u;
    while (ok && next_piece(a, costs_of<D>(), w, u)) {
        ok = publish(b, pieces++, u);
        if (!ok)
            break;
        // Copy coordinates, afresh (see uniform).
        const int head = uniform(u.h), q0 = uniform(u.s.q0);
        pos = uniform(pos);
        // The first table entries are on their way while the Q buffer is waited for.
        const int pages = (u.s.L + (1 << shift) - 1) >> shift;  // of the sequence
        const int *row = a.page_table + static_cast<long long>(w.at_b) * a.table_stride;
        auto entries = [&](int first) { return first + lane < pages ? row[first + lane] : 0; };
        const int first_page = static_cast<int>((static_cast<long long>(u.j0) * kBN) >> shift);
        if (w.at_b != held_b || first_page != held_page) {
            held_b = w.at_b;
            held_page = first_page;
            held_cur = entries(first_page);
            held_ahead = entries(first_page + 32);
        }
        int held = first_page, cur = held_cur, ahead = held_ahead;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            if (!ok || (u.alt ? u.j0 == u.j1 || u.q_buf != t : (t == 0 ? u.n[0] : u.n[1]) == 0))
                continue;
            ok = warp_wait(b.q_empty[t], ((q_bits >> t) & 1u) ^ 1u, abort);
            if (!ok)
                continue;
            const int token = uniform(q0 + (t == 0 ? u.tile[0] : u.tile[1]) * a.tile_tokens);
            if (leader) {
                const uint32_t full = smem_addr(&b.q_full[t]);
                const uint32_t dst = smem_base + t * C::kTileBytes;
                mbar_arrive_expect_tx(full, q_row_bytes * (u.quad ? 4 * a.q_quad_tokens : a.q_box_tokens));
                const CUtensorMap *map = u.quad ? mq_quad : mq;
                const uint32_t end = dst + (u.quad ? 4 * kQuadRows * 128 : 1);
#pragma unroll 1
                for (uint32_t at = dst; at < end; at += kQuadRows * 128) {
#pragma unroll
                    for (int c = 0; c < C::kChunks; ++c)
                        tma_load_4d(at + c * kChunkBytes, map, full, 64 * c, 0, head, token);
                }
            }
            q_used |= 1u << t;
            q_bits ^= 1u << t;
        }
        for (int j = u.j0; ok && j < u.j1; ++j) {
            const int p0 = (j * kBN) >> shift;
            if (p0 >= held + 32) {  // 32 is a multiple of per_tile
                held += 32;
                cur = ahead;
                ahead = entries(held + 32);
            }
            const int count = min(per_tile, pages - p0);
            // This lane's entry, brought into range: a page outside the pool
            // becomes the one behind it, which the copy fills with zeros.
            const bool stray = cur < 0 || cur >= a.num_pages;
            const int entry = stray ? a.num_pages : cur;
            if (stray && lane >= p0 - held && lane < p0 - held + count)
                atomicCAS(a.status, 0u,
                          6u /* FATTN_ERR_INDEX */ | (kRoleLoad << 8) | ((blockIdx.x & 0xffffu) << 16));
            const int slot = uniform(shift < 7 ? 0 : (j * kBN) & ((1 << shift) - 1));
            int page[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                page[i] = __shfl_sync(0xffffffffu, entry, min(p0 - held + i, 31));
#pragma unroll 1
            for (int which = 0; which < 2; ++which, ++pos) {
                const uint32_t stage = pos % C::kStages;
                ok = ok && warp_wait(b.kv_empty[stage], ((pos / C::kStages) & 1) ^ 1, abort);
                if (!ok)
                    break;
                const uint32_t full = smem_addr(&b.kv_full[stage]);
                const uint32_t dst = smem_base + (2 + stage) * C::kTileBytes;
                const CUtensorMap *map = which == 0 ? mk : mv;
                if (leader) {
                    mbar_arrive_expect_tx(full, count * box_rows * 128u * C::kChunks);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (i >= count)
                            break;
#pragma unroll
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_4d(dst + c * kChunkBytes + i * box_rows * 128, map, full, 64 * c, slot,
                                        head, page[i]);
                    }
                }
            }
        }
    }
    if (ok) {
        u.h = -1;
        ok = publish(b, pieces, u);
    }
    if (!ok) {
        if (leader)
            record_failure(a, b, kRoleLoad);
        // Copies already issued land before the CTA exits.
        const uint32_t first = pos > (uint32_t)C::kStages ? pos - C::kStages : 0;
        for (uint32_t q = first; q < pos; ++q)
            mbar_wait(smem_addr(&b.kv_full[q % C::kStages]), (q / C::kStages) & 1, kWaitLimitNs / 8,
                      nullptr);
        for (int t = 0; t < 2; ++t)
            if ((q_used >> t) & 1u)
                mbar_wait(smem_addr(&b.q_full[t]), ((q_bits >> t) & 1u) ^ 1u, kWaitLimitNs / 8, nullptr);
    }
}

// ------------------------------------------------------------------ V in place
// Exact for |v| < 65520 down to fp16's subnormals (off by at most 2^-25); a
// larger v becomes infinite, which the epilogue reports.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w)
{
    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint4 bf16x8_to_f16x8(uint4 w)
{
    return make_uint4(bf16x2_to_f16x2(w.x), bf16x2_to_f16x2(w.y), bf16x2_to_f16x2(w.z),
                      bf16x2_to_f16x2(w.w));
}

// One V tile by 64 threads: rows from `valid` on become zero, the others are
// converted (bf16).  Eight 16-byte steps in flight a thread; a thread writes
// only what it read.
template <int D, bool kF16, bool kRagged>
__device__ __forceinline__ void fix_v_tile(uint4 *tile, int tid, int valid)
{
    constexpr int kVecs = Cfg<D, kF16>::kTileBytes / 16, kBatch = 8;
#pragma unroll 1
    for (int base = tid; base < kVecs; base += 64 * kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            x[i] = tile[base + i * 64];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int at = base + i * 64;
            const bool keep = !kRagged || ((at / 8) % kBN) < valid;
            const uint4 y = kF16 ? x[i] : bf16x8_to_f16x8(x[i]);
            tile[at] = keep ? y : make_uint4(0, 0, 0, 0);
        }
    }
}

template <int D, bool kF16>
__device__ void run_convert(const PagedArgs &a, Bars &b, uint8_t *tiles, int cw)
{
    using C = Cfg<D, kF16>;
    const volatile int *abort = &b.abort;
    const int lane = threadIdx.x & 31, tid = cw * 32 + lane;
    uint32_t pos = 0;
    bool ok = true;
    for (uint32_t k = 0; receive(b, k, ok); ++k) {
        const Piece &u = b.pieces[k % kPieces];
        const int j0 = u.j0, j1 = u.j1, L = u.s.L;
        give_back(b, k);
        for (int j = j0; ok && j < j1; ++j, pos += 2) {
            const uint32_t at = pos + 1, stage = at % C::kStages;
            const int valid = L - j * kBN;
            // Every copy is waited for, and in fp16, whose whole tiles are used
            // as they land, said to have been: the stage is not filled again
            // before.  A phase is told by its parity, so a waiter two rounds
            // of the ring from the copies, on either side, would take another
            // for its own.
            ok = warp_wait(b.kv_full[stage], (at / C::kStages) & 1, abort);
            if (!ok)
                break;
            if (kF16) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&b.kv_empty[stage]));
                if (valid >= kBN)
                    continue;
            }
            uint4 *tile = reinterpret_cast<uint4 *>(tiles + (2 + stage) * C::kTileBytes);
            if (valid < kBN)
                fix_v_tile<D, kF16, true>(tile, tid, valid);
            else
                fix_v_tile<D, kF16, false>(tile, tid, valid);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&b.v_ready[stage]));
        }
    }
    if (!ok && lane == 0)
        record_failure(a, b, kRoleConvert);
}

// ------------------------------------------------------------------ MMA issue
// S = Q K^T: both operands K-major, 128-byte swizzled, 8-row groups 1024
// bytes apart; a K = 16 step is 32 bytes along d, or the next 16 KB box.
template <int D, bool kF16>
__device__ __forceinline__ void issue_s(uint32_t tmem_d, uint32_t q_smem, uint32_t k_smem)
{
    constexpr uint32_t idesc = idesc_f32acc(kBM, kBN, false, kF16);
    constexpr uint32_t hi = smem_desc_hi(1024);
    const uint32_t a_lo = smem_desc_lo(q_smem, 16), b_lo = smem_desc_lo(k_smem, 16);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
        mma_ss_w(tmem_d, a_lo + off, hi, b_lo + off, hi, idesc, kk > 0 ? 1u : 0u);
    }
}

// O (+)= P V, K-steps [kK0, kK1) of 16 keys: P from TMEM, V MN-major (64-column
// boxes 16 KB apart), both fp16.
template <int D, int kK0, int kK1>
__device__ __forceinline__ void issue_pv(uint32_t tmem_d, uint32_t tmem_p, uint32_t v_smem,
                                         bool accumulate)
{
    constexpr uint32_t idesc = idesc_f32acc(kBM, D, true, true);
    constexpr uint32_t hi = smem_desc_hi(1024);
    const uint32_t b_lo = smem_desc_lo(v_smem, D > 64 ? kChunkBytes : 1024);
#pragma unroll
    for (int kk = kK0; kk < kK1; ++kk)
        mma_ts_w(tmem_d, tmem_p + kk * 8, b_lo + ((kk * 16 * 128) >> 4), hi, idesc,
                 kk > 0 || accumulate ? 1u : 0u);
}

// Run by one lane: no votes after the waits and no branches around each product
// (127 KB of code instead of 133, 1.2 % over 24 ragged batches).
template <int D, bool kF16>
__device__ void run_mma(const PagedArgs &a, Bars &b, uint32_t smem_base, uint32_t tmem, uint32_t lane)
{
    using C = Cfg<D, kF16>;
    const volatile int *abort = &b.abort;
    bool ok = true;
    auto uniform = [&](int x) { return uniform_of(x, lane); };
    auto receive = [&](uint32_t k) {
        ok = ok && lane_wait(b.piece_full[k % kPieces], (k / kPieces) & 1, abort);
        return ok && b.pieces[k % kPieces].h >= 0;
    };
    auto give_back = [&](uint32_t k) { mbar_arrive(smem_addr(&b.piece_empty[k % kPieces])); };
    // Phases, a bit each (an array indexed by a variable would live in memory):
    // Q buffers, P halves and O by warpgroup, V by stage.
    uint32_t q_bits = 0, p_bits = 0, ph_bits = 0, oe_bits = 0, vr_bits = 0;
    uint32_t pos = 0;
    auto bit = [](uint32_t bits, int i) { return (bits >> i) & 1u; };
    auto stage_of = [&](uint32_t at) { return at % C::kStages; };
    auto kv_smem = [&](uint32_t at) { return smem_base + (2 + stage_of(at)) * C::kTileBytes; };
    auto k_wait = [&](uint32_t at) {
        return lane_wait(b.kv_full[stage_of(at)], (at / C::kStages) & 1, abort);
    };
    auto v_wait = [&](uint32_t at, bool whole) {
        if (kF16 && whole)
            return k_wait(at);
        const uint32_t st = stage_of(at);
        const bool r = lane_wait(b.v_ready[st], bit(vr_bits, st), abort);
        vr_bits ^= 1u << st;
        return r;
    };
    auto q_wait = [&](int buf) {
        const bool r = lane_wait(b.q_full[buf], bit(q_bits, buf), abort);
        q_bits ^= 1u << buf;
        return r;
    };
    auto commit = [&](uint64_t &bar) { mma_commit(smem_addr(&bar)); };
    // P V of one key tile into warpgroup t's accumulator; where a warp writes
    // a whole row of P, the keys in two halves: the first as soon as it is written.
    auto pv = [&](int t, uint32_t at_v, bool first, bool halves) {
        const uint32_t col_s = tmem + t * 128, col_o = tmem + C::kColO0 + t * D;
        const uint32_t v = kv_smem(at_v);
        if (first) {  // overwrites O: the last unit's has to be read
            if (!lane_wait(b.o_empty[t], bit(oe_bits, t) ^ 1, abort))
                return false;
            oe_bits ^= 1u << t;
        }
        if (halves) {
            if (!lane_wait(b.p_half[t], bit(ph_bits, t), abort))
                return false;
            ph_bits ^= 1u << t;
            tc_fence_after();
            issue_pv<D, 0, kBN / 32>(col_o, col_s, v, !first);
        }
        if (!lane_wait(b.p_full[t], bit(p_bits, t), abort))
            return false;
        p_bits ^= 1u << t;
        tc_fence_after();
        if (!halves)
            issue_pv<D, 0, kBN / 32>(col_o, col_s, v, !first);
        issue_pv<D, kBN / 32, kBN / 16>(col_o, col_s, v, true);
        return true;
    };
    auto s_product = [&](int t, int q_tile, uint32_t at_k) {
        issue_s<D, kF16>(tmem + t * 128, smem_base + q_tile * C::kTileBytes, kv_smem(at_k));
        commit(b.s_full[t]);
    };

    struct Unit {
        int n, alt, quad, q_buf;
        int whole;  // leading key tiles that lie in the sequence whole
        int nt[2];
    };
    auto read = [&](uint32_t k) {
        const Piece &u = b.pieces[k % kPieces];
        Unit x;
        x.n = uniform(u.j1 - u.j0);
        x.whole = uniform(u.s.L / kBN - u.j0);
        x.alt = uniform(u.alt);
        x.quad = uniform(u.quad);
        x.q_buf = uniform(u.q_buf);
        x.nt[0] = uniform(u.n[0]);
        x.nt[1] = uniform(u.n[1]);
        return x;
    };
    uint32_t turn = 0;  // key tiles of single-tile units so far: tile g is warpgroup g % 2's
    uint32_t k = 0;
    while (receive(k)) {
        Unit u = read(k);
        if (u.n == 0) {
            give_back(k++);
            continue;
        }
        if (u.alt) {
            // A run of single-tile units as one stream of key tiles: S goes up to
            // two tiles ahead of P V, across the units' ends.  The run's piece
            // at ks is where S is, the one at k where P V is.
            uint32_t ks = k, pos_s = pos, turn_s = turn;
            Unit us = u;
            int is = 0;
            bool open = true;  // S has not come to the run's end
            auto next_s = [&]() {
                // Tile g + 2 overwrites tile g's S and P.
                if (!open || turn_s - turn >= 2)
                    return;
                while (is == us.n) {
                    // The next piece, while the pieces held leave the producer a
                    // place to publish it in.
                    if (ks + 1 - k >= kPieces - 1)
                        return;
                    open = receive(ks + 1);
                    if (!open)
                        return;
                    us = read(++ks);
                    is = 0;
                    open = us.alt;
                    if (!open)
                        return;
                }
                if (is == 0) {
                    ok = q_wait(us.q_buf);
                    pos_s = uniform(pos_s);
                }
                ok = ok && k_wait(pos_s);
                if (!ok)
                    return;
                tc_fence_after();
                s_product(turn_s & 1, us.q_buf, pos_s);
                commit(b.kv_empty[stage_of(pos_s)]);
                if (++is == us.n)
                    commit(b.q_empty[us.q_buf]);
                pos_s += 2;
                ++turn_s;
            };
            next_s();
            for (;;) {  // the run's units
                pos = uniform(pos);
                for (int i = 0; ok && i < u.n; ++i) {
                    next_s();
                    const int t = turn & 1;
                    const uint32_t at_v = pos + 1;
                    ok = ok && v_wait(at_v, i < u.whole) && pv(t, at_v, i < 2, !u.quad);
                    if (!ok)
                        break;
                    commit(b.kv_empty[stage_of(at_v)]);
                    if (i + 2 >= u.n)
                        commit(b.o_full[t]);
                    pos = at_v + 1;
                    ++turn;
                    next_s();
                }
                if (!ok)
                    break;
                give_back(k++);
                if (ks < k)
                    next_s();
                if (!ok || ks < k || (ks == k && !us.alt))
                    break;  // no more work, or a unit of two tiles
                u = ks == k ? us : read(k);
            }
            continue;
        }
        give_back(k++);
        const int n = u.n;
        const uint32_t base = uniform(pos);  // K_(j0+i) at base + 2i, V_(j0+i) at base + 2i + 1
        pos = base + 2 * n;
        for (int t = 0; t < 2 && ok; ++t)
            if (u.nt[t] > 0) {
                ok = q_wait(t);
            }
        ok = ok && k_wait(base);
        if (!ok)
            break;
        tc_fence_after();
        for (int t = 0; t < 2; ++t) {
            if (u.nt[t] == 0)
                continue;
            s_product(t, t, base);
            if (u.nt[t] == 1)
                commit(b.q_empty[t]);
        }
        commit(b.kv_empty[stage_of(base)]);
        for (int i = 0; i < n && ok; ++i) {
            const uint32_t at_v = base + 2 * i + 1, at_k = base + 2 * (i + 1);
            const bool more = i + 1 < n;
            ok = v_wait(at_v, i < u.whole) && (!more || k_wait(at_k));
            for (int t = 0; t < 2 && ok; ++t) {
                if (i >= u.nt[t])
                    continue;
                ok = pv(t, at_v, i == 0, true);
                if (!ok)
                    break;
                if (i + 1 < u.nt[t]) {
                    s_product(t, t, at_k);
                    if (i + 2 == u.nt[t])
                        commit(b.q_empty[t]);
                } else {
                    commit(b.o_full[t]);
                }
            }
            if (!ok)
                break;
            commit(b.kv_empty[stage_of(at_v)]);
            if (more)
                commit(b.kv_empty[stage_of(at_k)]);
        }
    }
    if (!ok)
        record_failure(a, b, kRoleMma);
    commit(b.drain);
    mbar_wait(smem_addr(&b.drain), 0, kWaitLimitNs, nullptr);
}

// ------------------------------------------------------------------ softmax
// One key tile of one row: S from TMEM, mask (keys past `limit`, an index in
// the tile), row maximum, P (fp16) over the first 64 columns of S, l.
// pre(alpha) runs before any P is written, mid() once P of 64 keys is.
template <class Pre, class Mid>
__device__ __forceinline__ float softmax_tile(float sl2, uint32_t t_s, bool masked, int limit,
                                              bool first, float m, float &m_new, float &l, Pre pre,
                                              Mid mid)
{
    uint32_t raw[kBN / 32][32];
    float cmax[kBN / 32];
#pragma unroll
    for (int c = 0; c < kBN / 32; ++c)
        tmem_ld32_max(t_s + c * 32, raw[c], cmax[c]);
    tmem_wait_ld();
    float s[kBN];
#pragma unroll
    for (int i = 0; i < kBN; ++i)
        s[i] = __uint_as_float(raw[i / 32][i % 32]);
    float smax = fmaxf(fmaxf(cmax[0], cmax[1]), fmaxf(cmax[2], cmax[3]));
    if (masked) {  // uniform in the warp
#pragma unroll
        for (int i = 0; i < kBN; ++i)
            s[i] = i > limit ? -INFINITY : s[i];
        float mx[4] = {fmaxf(s[0], s[1]), fmaxf(s[2], s[3]), fmaxf(s[4], s[5]), fmaxf(s[6], s[7])};
#pragma unroll
        for (int i = 8; i < kBN; i += 8) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                mx[c] = fmax3(mx[c], s[i + 2 * c], s[i + 2 * c + 1]);
        }
        smax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    }
    // m starts at -FLT_MAX: a row that sees no key keeps it, with l = 0.
    const float cand = smax * sl2;
    m_new = (first || cand > m + kRescaleLog2) ? fmaxf(m, cand) : m;
    const float alpha = ex2(m - m_new);
    pre(alpha);
    const uint64_t sl2x2 = f2_pack(sl2, sl2), negm = f2_pack(-m_new, -m_new);
    uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < kBN / 32; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sl2x2, negm), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            pk[i] = pack2<true>(p0, p1);
            sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
        }
        tmem_st16(t_s + c * 16, pk);
        if (c == kBN / 64 - 1)
            mid();
    }
    float e0, e1, e2, e3;
    f2_unpack(sum[0], e0, e1);
    f2_unpack(sum[1], e2, e3);
    l = l * alpha + ((e0 + e1) + (e2 + e3));
    return alpha;
}

// The same for a quad unit: keys 32 w .. 32 w + 31 of the tile for this warp's
// copy of the rows (t_s: its lanes of S; limit: an index in the tile).
template <class Pre>
__device__ __forceinline__ float softmax_quarter(float sl2, uint32_t t_s, int w, bool masked, int limit,
                                                 bool first, float m, float &m_new, float &l, Pre pre)
{
    uint32_t raw[32];
    float smax;
    tmem_ld32_max(t_s + 32 * w, raw, smax);
    tmem_wait_ld();
    float s[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        s[i] = __uint_as_float(raw[i]);
    if (masked) {
        limit -= 32 * w;
        smax = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            s[i] = i > limit ? -INFINITY : s[i];
            s[i + 1] = i + 1 > limit ? -INFINITY : s[i + 1];
            smax = fmax3(smax, s[i], s[i + 1]);
        }
    }
    const float cand = smax * sl2;
    m_new = (first || cand > m + kRescaleLog2) ? fmaxf(m, cand) : m;
    const float alpha = ex2(m - m_new);
    pre(alpha);
    const uint64_t sl2x2 = f2_pack(sl2, sl2), negm = f2_pack(-m_new, -m_new);
    uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
    uint32_t pk[16], zero[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(s[2 * i], s[2 * i + 1]), sl2x2, negm), x0, x1);
        const float p0 = ex2(x0), p1 = ex2(x1);
        pk[i] = pack2<true>(p0, p1);
        sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
        zero[i] = 0;
    }
#pragma unroll
    for (int c = 0; c < kBN / 32; ++c) {
        if (c == w)
            tmem_st16(t_s + c * 16, pk);
        else
            tmem_st16(t_s + c * 16, zero);
    }
    float e0, e1, e2, e3;
    f2_unpack(sum[0], e0, e1);
    f2_unpack(sum[1], e2, e3);
    l = l * alpha + ((e0 + e1) + (e2 + e3));
    return alpha;
}

template <int D> __device__ __forceinline__ void rescale_o(uint32_t t_o, float alpha)
{
    const uint64_t alpha2 = f2_pack(alpha, alpha);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(t_o + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float x, y;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), alpha2), x, y);
            o[i] = __float_as_uint(x);
            o[i + 1] = __float_as_uint(y);
        }
        tmem_st32(t_o + c, o);
    }
}

// Row stores go through 4 KB of staging a warp: thread r puts a 128-byte
// piece of its row into staging row r, granule g at g ^ (r % 8), and eight
// lanes a row copy whole lines out.
__device__ __forceinline__ void stage_put(uint8_t *stage, int lane, int g, uint4 v)
{
    reinterpret_cast<uint4 *>(stage + lane * 128)[g ^ (lane & 7)] = v;
}
// `mine`: where this lane's row goes (null: nowhere); half: 64-byte pieces.
__device__ __forceinline__ void stage_flush(const uint8_t *stage, int lane, bool half, char *mine)
{
    __syncwarp();
    const int g = half ? lane % 4 : lane % 8, step = half ? 8 : 4;
#pragma unroll 2
    for (int r0 = 0; r0 < 32; r0 += step) {
        const int row = r0 + (half ? lane / 4 : lane / 8);
        const uint4 x = reinterpret_cast<const uint4 *>(stage + row * 128)[g ^ (row & 7)];
        char *dst = reinterpret_cast<char *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), row));
        if (dst != nullptr)
            *reinterpret_cast<uint4 *>(dst + g * 16) = x;
    }
    __syncwarp();
}

// Row r of a tile: token r / G, head r % G, by a multiplication (exact for r
// < 128 and G <= 128).
__device__ __forceinline__ int row_token(const PagedArgs &a, int r)
{
    return static_cast<int>((static_cast<uint32_t>(r) * a.g_inverse) >> 16);
}

// Writes warp rows [r0, r0 + 32) of tile t of the piece: O = w0 O_t0 + w1
// O_t1 (single-tile units merge two accumulators; w1 is ignored otherwise) and
// the base-2 log-sum-exp lse2.  To o and lse, or to the piece's slot.  A warp
// with at most kFewRows rows stores them from its registers: going through the
// staging area costs it 32 rows' steps whatever is in them.  So does one
// without keys (!some): nothing orders it behind the other warpgroup's reading
// of this one's (m, l).
constexpr int kFewRows = 8;
template <int D, bool kF16>
__device__ __forceinline__ void write_rows(const PagedArgs &a, const Piece &u, int t, int r0,
                                           uint32_t t_o0, uint32_t t_o1, bool two, float w0, float w1,
                                           float lse2, bool some, uint8_t *stage)
{
    const int lane = threadIdx.x & 31, rows = u.rows[t] - r0;
    const bool live = lane < rows, whole = u.slot < 0;
    const int tok = row_token(a, r0 + lane), g = r0 + lane - tok * a.G;
    const long long token = static_cast<long long>(u.s.q0) +
                            u.tile[t] * a.tile_tokens + tok;
    const int head = u.h * a.G + g;
    const long long slot_row = static_cast<long long>(u.slot) * a.slot_rows + (u.alt ? 0 : t * kBM) + r0 +
                               lane;
    char *dst = nullptr;
    if (live)
        dst = whole ? reinterpret_cast<char *>(static_cast<uint16_t *>(a.o) + token * a.o_st[0] +
                                               head * a.o_st[1])
                    : reinterpret_cast<char *>(a.ws_o + slot_row * D);
    // A sum over the row of O is finite unless some element is not: |O| < 2^8
    // keys * 65504.
    float nonfinite = 0.f;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        float y[32];
        if (some) {
            uint32_t o[32];
            tmem_ld32(t_o0 + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
                y[i] = __uint_as_float(o[i]) * w0;
            if (two) {
                tmem_ld32(t_o1 + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    y[i] = fmaf(__uint_as_float(o[i]), w1, y[i]);
            }
            if (!kF16) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    nonfinite += y[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                y[i] = 0.f;
        }
        if (whole) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = make_uint4(pack2<kF16>(y[8 * i], y[8 * i + 1]),
                                  pack2<kF16>(y[8 * i + 2], y[8 * i + 3]),
                                  pack2<kF16>(y[8 * i + 4], y[8 * i + 5]),
                                  pack2<kF16>(y[8 * i + 6], y[8 * i + 7]));
            if (rows <= kFewRows || !some) {
                if (live) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4 *>(dst)[c * 4 + i] = v[i];
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                stage_put(stage, lane, (c % 2) * 4 + i, v[i]);
            if (c % 2 == 1 || c + 1 == D / 32)
                stage_flush(stage, lane, c % 2 == 0, dst == nullptr ? dst : dst + (c / 2) * 128);
        } else {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]),
                                  __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]));
            if (rows <= kFewRows) {
                if (live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4 *>(dst)[c * 8 + i] = v[i];
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                stage_put(stage, lane, i, v[i]);
            stage_flush(stage, lane, false, dst == nullptr ? dst : dst + c * 128);
        }
    }
    if (!live)
        return;
    if (whole)
        a.lse[token * a.Hk * a.G + head] = lse2 * kLn2;
    else
        a.ws_l[slot_row] = lse2;
    if (!kF16 && !(fabsf(nonfinite) <= FLT_MAX))
        atomicCAS(a.status, 0u,
                  5u /* FATTN_ERR_RANGE */ | (kRoleEpilogue << 8) | ((blockIdx.x & 0xffffu) << 16));
}

// A step that the four warps of warpgroup t take together.
__device__ __forceinline__ bool quarters_meet(Bars &b, int t, uint32_t &phase)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(smem_addr(&b.quarters[t]));
    const bool ok = warp_wait(b.quarters[t], phase, &b.abort);
    phase ^= 1;
    return ok;
}

// (m, l) of row `lane` of a softmax warp, at the end of its staging area:
// written for the warpgroup that leads a unit, or for the other quarters.
__device__ __forceinline__ float2 *stats_of(uint8_t *stage, int lane)
{
    return reinterpret_cast<float2 *>(stage + kStageBytes) - (lane + 1);
}

// Epilogue of a quad unit: each warp has (m, l) and O (w0 O_0 + w1 O_1) of its
// keys for all rows, lane = row; the four are brought to one m, added through
// the staging areas (as many columns at a time as fit for the rows there are)
// and written, eight columns a thread.
template <int D, bool kF16>
__device__ __forceinline__ bool write_quad(const PagedArgs &a, Bars &b, const Piece &u, int t,
                                           uint8_t *stages, uint32_t t_o0, uint32_t t_o1, bool two, float w0, float w1,
                                           float m, float l, uint32_t &phase)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x / 32) & 3, rows = u.rows[0];
    const bool whole = u.slot < 0;
    if (lane < rows)
        *stats_of(stages + warp * kStageBytes, lane) = make_float2(m, l);
    if (!quarters_meet(b, t, phase))
        return false;
    float2 ml[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        ml[k] = lane < rows ? *stats_of(stages + k * kStageBytes, lane) : make_float2(-FLT_MAX, 0.f);
    const float mm = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        sum += ml[k].y * ex2(ml[k].x - mm);
    // Only a sum of zero means no key: a NaN or infinite score makes it NaN,
    // which goes on into o and lse (and the merge).
    const float f = sum == 0.f ? 0.f : ex2(m - mm) / sum;
    w0 *= f;
    w1 *= f;
    const long long first = static_cast<long long>(u.s.q0) + u.tile[0] * a.tile_tokens;
    if (warp == 0 && lane < rows) {
        const float lse2 = sum == 0.f ? -INFINITY : mm + log2f(sum);
        const int tok = row_token(a, lane);
        if (whole)
            a.lse[(first + tok) * a.Hk * a.G + u.h * a.G + lane - tok * a.G] = lse2 * kLn2;
        else
            a.ws_l[static_cast<long long>(u.slot) * a.slot_rows + lane] = lse2;
    }
    // Blocks of columns: put, meet, add and write, meet.
    int width = D;
    while (static_cast<uint32_t>(rows * (width * 4 + 8)) > kStageBytes)
        width = width > 32 ? width == 96 ? 32 : width / 2 : 16;
    const int each = width / 8;
    const int q = warp * 32 + lane, my_row = q / each, my_col = (q - my_row * each) * 8;
    const int swz = width == 16 ? 3 : 7;  // granules of a row trade places by row
    uint8_t *mine = stages + warp * kStageBytes + lane * width * 4;
    const uint8_t *theirs = stages + my_row * width * 4;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += width) {
#pragma unroll 1
        for (int c = 0; c < width; c += 16) {
            uint32_t o0[16], o1[16];
            tmem_ld16(t_o0 + c0 + c, o0);
            if (two)
                tmem_ld16(t_o1 + c0 + c, o1);
            tmem_wait_ld();
            if (lane >= rows)
                continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    y[k] = __uint_as_float(o0[4 * i + k]) * w0;
                    if (two)
                        y[k] = fmaf(__uint_as_float(o1[4 * i + k]), w1, y[k]);
                }
                *reinterpret_cast<float4 *>(mine + (((c / 4 + i) ^ (lane & swz)) << 4)) =
                    make_float4(y[0], y[1], y[2], y[3]);
            }
        }
        if (!quarters_meet(b, t, phase))
            return false;
        if (my_row < rows) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 x = *reinterpret_cast<const float4 *>(
                        theirs + k * kStageBytes + (((my_col / 4 + h) ^ (my_row & swz)) << 4));
                    y[4 * h] += x.x;
                    y[4 * h + 1] += x.y;
                    y[4 * h + 2] += x.z;
                    y[4 * h + 3] += x.w;
                }
            // Finite unless one of them is not.
            if (!kF16 && !(fabsf(((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]))) <= FLT_MAX))
                atomicCAS(a.status, 0u,
                          5u /* FATTN_ERR_RANGE */ | (kRoleEpilogue << 8) | ((blockIdx.x & 0xffffu) << 16));
            if (whole) {
                const int tok = row_token(a, my_row);
                uint16_t *dst = static_cast<uint16_t *>(a.o) + (first + tok) * a.o_st[0] +
                                (static_cast<long long>(u.h) * a.G + my_row - tok * a.G) * a.o_st[1] + c0 +
                                my_col;
                *reinterpret_cast<uint4 *>(dst) =
                    make_uint4(pack2<kF16>(y[0], y[1]), pack2<kF16>(y[2], y[3]), pack2<kF16>(y[4], y[5]),
                               pack2<kF16>(y[6], y[7]));
            } else {
                float *dst = a.ws_o + (static_cast<long long>(u.slot) * a.slot_rows + my_row) * D + c0 + my_col;
                reinterpret_cast<float4 *>(dst)[0] = make_float4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
        }
        if (!quarters_meet(b, t, phase))
            return false;
    }
    return true;
}

template <int D, bool kF16>
__device__ void run_softmax(const PagedArgs &a, Bars &b, uint32_t tmem, int t)
{
    using C = Cfg<D, kF16>;
    const int warp = (threadIdx.x / 32) & 3, lane = threadIdx.x & 31;
    const int r = warp * 32 + lane;
    // The inner loops need all but a few registers: what follows from `b` and
    // `tmem` (this warp's lanes of it) is formed where it is used, and the
    // phases share a word.
    tmem += static_cast<uint32_t>(warp * 32) << 16;
    auto t_o = [&](int of) { return tmem + C::kColO0 + of * D; };
    auto stages = [&](int of) {
        return reinterpret_cast<uint8_t *>(&b) - C::kBarsOffset + C::kStageOffset + of * 4 * kStageBytes;
    };
    enum { kPhaseS, kPhaseO, kPhaseOther, kPhaseQuarters };
    uint32_t phases = 0;
    auto wait = [&](uint64_t &bar, int phase) {
        const bool r = warp_wait(bar, (phases >> phase) & 1u, &b.abort);
        phases ^= 1u << phase;
        return r;
    };
    bool ok = true;
    for (uint32_t k = 0; receive(b, k, ok); ++k) {
        // Read in place where it is needed: the inner loops have no registers
        // to hold it.
        const Piece &u = b.pieces[k % kPieces];
        const int nt = u.n[t];
        const bool alt = u.alt, quad = u.quad;
        // Rows of this warp that exist (a warp without any only keeps step).
        const bool busy = quad || warp * 32 < u.rows[t];
        float m = -FLT_MAX, l = 0.f;
        {
            // Keys that this row sees in key tile j: its indexes 0 .. min(diag +
            // tok, tail), diag and tail counted from the tile's first key.
            const int step = alt ? 2 * kBN : kBN;
            const int tok = a.causal ? row_token(a, quad ? lane : r) : 0;
            int tail = u.s.L - 1 - (u.j0 + (alt && t != u.lead ? 1 : 0)) * kBN;
            int diag = a.causal ? tail + 1 - u.s.n + u.tile[t] * a.tile_tokens : tail;
            bool rescale = false, first = true;
            float m_new;
            auto pre = [&](float) { rescale = !first && __any_sync(0xffffffffu, m_new != m); };
            auto arrive = [&](uint64_t &bar) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&bar));
            };
            auto s_wait = [&]() {
                ok = wait(b.s_full[t], kPhaseS);
                tc_fence_after();
                __syncwarp();
                return ok;
            };
            if (quad) {
#pragma unroll 1
                for (int i = 0; i < nt && s_wait(); ++i) {
                    const bool masked = min(diag, tail) < kBN - 1;
                    const float alpha = softmax_quarter(a.sl2, tmem + t * 128, warp, masked, min(diag + tok, tail),
                                                        first, m, m_new, l, pre);
                    if (rescale)
                        rescale_o<D>(t_o(t), alpha);
                    m = m_new;
                    first = false;
                    diag -= step;
                    tail -= step;
                    arrive(b.p_full[t]);
                }
            } else if (busy) {
                auto mid = [&]() {
                    if (!rescale)
                        arrive(b.p_half[t]);
                };
#pragma unroll 1
                for (int i = 0; i < nt && s_wait(); ++i) {
                    const bool masked = min(diag, tail) < kBN - 1;
                    const float alpha = softmax_tile(a.sl2, tmem + t * 128, masked, min(diag + tok, tail), first, m,
                                                     m_new, l, pre, mid);
                    if (rescale) {
                        rescale_o<D>(t_o(t), alpha);
                        arrive(b.p_half[t]);
                    }
                    m = m_new;
                    first = false;
                    diag -= step;
                    tail -= step;
                    arrive(b.p_full[t]);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < nt && s_wait(); ++i)
                    if (lane == 0) {
                        mbar_arrive(smem_addr(&b.p_half[t]));
                        mbar_arrive(smem_addr(&b.p_full[t]));
                    }
            }
        }
        if (!ok)
            break;
        if (nt > 0) {
            ok = wait(b.o_full[t], kPhaseO);
            if (!ok)
                break;
        }
        const bool two = alt && u.n[t ^ 1] > 0 && nt > 0;
        if (alt && t != u.lead) {
            if (nt > 0) {
                *stats_of(stages(t) + warp * kStageBytes, lane) = make_float2(m, l);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&b.other_done));
                phases ^= 1u << kPhaseOther;
            }
            give_back(b, k);
            continue;
        }
        // O = w0 of the own accumulator + w1 of the other's, times 1 / l.
        float w0 = 1.f, w1 = 0.f;
        if (two) {
            ok = wait(b.other_done, kPhaseOther);
            if (!ok)
                break;
            const float2 ml = *stats_of(stages(t ^ 1) + warp * kStageBytes, lane);
            const float mm = fmaxf(m, ml.x);
            w0 = ex2(m - mm);
            w1 = ex2(ml.x - mm);
            l = l * w0 + ml.y * w1;
            m = mm;
        }
        tc_fence_after();
        __syncwarp();
        if (quad) {
            uint32_t phase = (phases >> kPhaseQuarters) & 1u;
            phases ^= phase << kPhaseQuarters;
            ok = write_quad<D, kF16>(a, b, u, t, stages(t), t_o(t), t_o(t ^ 1), two, w0, w1, m, l, phase);
            phases ^= phase << kPhaseQuarters;
            if (!ok)
                break;
        } else if (busy) {
            if (nt == 0 && u.slot >= 0) {  // no key tile of this piece: an empty partial
                if (r < u.rows[t])
                    a.ws_l[static_cast<long long>(u.slot) * a.slot_rows + t * kBM + r] = -INFINITY;
            } else {
                // l = 0: no key; NaN (a NaN or infinite score) goes on.
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
                write_rows<D, kF16>(a, u, t, warp * 32, t_o(t), t_o(t ^ 1), two, w0 * inv, w1 * inv,
                                    lse2, nt > 0, stages(t) + warp * kStageBytes);
            }
        }
        give_back(b, k);
        if (nt > 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&b.o_empty[t]));
                if (two)
                    mbar_arrive(smem_addr(&b.o_empty[t ^ 1]));
            }
        }
    }
    if (!ok)
        record_failure(a, b, kRoleSoftmax);
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mq_quad,
                 const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const PagedArgs a)
{
    using C = Cfg<D, kF16>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t smem_base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (smem_base - raw);
    Bars &b = *reinterpret_cast<Bars *>(smem + C::kBarsOffset);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_addr(&b.q_full[t]), 1);
            mbar_init(smem_addr(&b.q_empty[t]), 1);
            mbar_init(smem_addr(&b.s_full[t]), 1);
            mbar_init(smem_addr(&b.p_half[t]), 4);
            mbar_init(smem_addr(&b.p_full[t]), 4);
            mbar_init(smem_addr(&b.o_full[t]), 1);
            mbar_init(smem_addr(&b.o_empty[t]), 4);
        }
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_addr(&b.kv_full[s]), 1);
            // V stages (odd) in fp16: by both warps that look at V, too.
            mbar_init(smem_addr(&b.kv_empty[s]), kF16 && s % 2 == 1 ? 3 : 1);
            mbar_init(smem_addr(&b.v_ready[s]), 2);
        }
        for (int k = 0; k < kPieces; ++k) {
            mbar_init(smem_addr(&b.piece_full[k]), 1);
            mbar_init(smem_addr(&b.piece_empty[k]), kThreads / 32 - 1);
        }
        mbar_init(smem_addr(&b.other_done), 4);
        mbar_init(smem_addr(&b.quarters[0]), 4);
        mbar_init(smem_addr(&b.quarters[1]), 4);
        mbar_init(smem_addr(&b.drain), 1);
        b.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_addr(&b.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    if (warp == kWarpLoad && lane == 0) {
        prefetch_tensormap(&mq);
        prefetch_tensormap(&mq_quad);
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
    }
    // Launched ahead of the work before it in the stream: nothing above touches
    // global memory.
    grid_dependency_wait();
    find_start(a, costs_of<D>(), b);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem_base;
    if (warp < 8)
        run_softmax<D, kF16>(a, b, tmem, warp / 4);
    else if (warp == kWarpLoad)
        run_load<D, kF16>(a, b, smem_base, &mq, &mq_quad, &mk, &mv);
    else if (warp == kWarpMma) {
        const uint32_t leader = elected_lane();
        if (elect_one())
            run_mma<D, kF16>(a, b, smem_base, tmem, leader);
        __syncwarp();
    }
    else
        run_convert<D, kF16>(a, b, smem, warp - kWarpConv);
    // Here, not at the start: merge CTAs waiting on the SMs that finish first cost
    // the others 1 to 3 %.
    grid_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) {
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ combine
// Block x handles the unit that CTA x + 1 starts inside, if that is the first
// boundary in it: the partial of CTA x (its last slot) and those of CTAs x +
// 1, x + 2, ... that start inside the same unit.  With base-2 partial
// log-sum-exps e_s: lse = ln2 log2 sum 2^e_s, O = sum 2^(e_s - lse2) O_s.
// A warp takes kRows rows at a time and kSlots of their partials, all loads of
// such a group in flight together, D / 32 consecutive columns a lane: one row
// and eight partials where units are single tiles (few rows, long chains), two
// rows and two where they may be pairs (256 rows, mostly one boundary): the
// ragged d = 64 batch took 73 us with that, 80 with four rows, 83 with one.
template <int N> struct Cols;
template <> struct Cols<2> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[2])
    {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x;
        x[1] = v.y;
    }
};
template <> struct Cols<3> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[3])
    {
        x[0] = p[0];
        x[1] = p[1];
        x[2] = p[2];
    }
};
template <> struct Cols<4> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[4])
    {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    }
};

template <int D, bool kF16, int kRows, int kSlots>
__global__ void __launch_bounds__(128) combine_paged_kernel(const PagedArgs a, int grid)
{
    constexpr int kCols = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    grid_launch_dependents();
    grid_dependency_wait();
    // One round of loads: the starts from CTA c - 1 on, a lane each, and what
    // this unit's rows are.
    const int c = blockIdx.x + 1;
    int4 start = a.starts[2 * min(c - 1 + lane, grid - 1)];
    const int4 unit = a.starts[2 * c + 1];  // first token, tokens
    const int mine_b = __shfl_sync(0xffffffffu, start.x, 1), mine_h = __shfl_sync(0xffffffffu, start.y, 1),
              mine_p = __shfl_sync(0xffffffffu, start.z, 1), mine_t = __shfl_sync(0xffffffffu, start.w, 1);
    if (mine_b < 0 || mine_t == 0)
        return;
    // CTAs from c on that start inside this unit; c - 1 must not.
    int count = 0;
    for (int at = c - 1;;) {
        const bool same = start.x == mine_b && start.y == mine_h && start.z == mine_p && start.w > 0;
        const unsigned hit = __ballot_sync(0xffffffffu, at + lane < grid && same) | (at == c - 1 ? 1u : 0u);
        if (at == c - 1 && __shfl_sync(0xffffffffu, same ? 1 : 0, 0))
            return;
        const int run = hit == 0xffffffffu ? 32 : __ffs(~hit) - 1;
        count += run - (at == c - 1 ? 1 : 0);
        if (run < 32)
            break;
        at += 32;
        start = a.starts[2 * min(at + lane, grid - 1)];
    }
    const long long slot0 = 2LL * (c - 1) + 1;
    const int row0 = (blockIdx.y * 4 + warp) * kRows;
    bool live[kRows];
    bool any = false;
    float mx[kRows], se[kRows], acc[kRows][kCols];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = row0 + i, tok = row_token(a, row % kBM);
        live[i] = row < a.slot_rows && tok < a.tile_tokens && row / kBM * a.tile_tokens + tok < unit.y;
        any = any || live[i];
        mx[i] = -INFINITY;
        se[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            acc[i][j] = 0.f;
    }
    if (!any)
        return;
    for (int k0 = 0; k0 <= count; k0 += kSlots) {
        float e[kSlots][kRows], o[kSlots][kRows][kCols];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const long long slot = k0 + k == 0 ? slot0 : 2LL * (c + k0 + k - 1);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                e[k][i] = -INFINITY;
                if (k0 + k <= count && live[i]) {
                    const long long at = slot * a.slot_rows + row0 + i;
                    e[k][i] = a.ws_l[at];
                    Cols<kCols>::load(a.ws_o + at * D + lane * kCols, o[k][i]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (e[k][i] == -INFINITY)  // holds no key of this row (its O is not written)
                    continue;
                const float ne = fmaxf(mx[i], e[k][i]);
                const float f = ex2(mx[i] - ne), x = ex2(e[k][i] - ne);
                se[i] = se[i] * f + x;
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    acc[i][j] = fmaf(x, o[k][i][j], acc[i][j] * f);
                mx[i] = ne;
            }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (!live[i])
            continue;
        const int row = row0 + i, r = row % kBM, tok = row_token(a, r);
        const long long token = static_cast<long long>(unit.x) + row / kBM * a.tile_tokens + tok;
        const int head = mine_h * a.G + r - tok * a.G;
        const float inv = se[i] == 0.f ? 0.f : 1.f / se[i];  // NaN goes on
        uint16_t *dst = static_cast<uint16_t *>(a.o) + token * a.o_st[0] + head * a.o_st[1] + lane * kCols;
        if constexpr (kCols % 2 == 0) {
#pragma unroll
            for (int j = 0; j < kCols; j += 2)
                *reinterpret_cast<uint32_t *>(dst + j) = pack2<kF16>(acc[i][j] * inv, acc[i][j + 1] * inv);
        } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                dst[j] = static_cast<uint16_t>(pack2<kF16>(acc[i][j] * inv, 0.f) & 0xffffu);
        }
        if (lane == 0)
            a.lse[token * a.Hk * a.G + head] = se[i] == 0.f ? -INFINITY : (mx[i] + log2f(se[i])) * kLn2;
    }
}

template <int D, bool kF16>
cudaError_t launch(const PagedArgs &a, const PagedMaps &maps, int num_sms, cudaStream_t stream)
{
    using C = Cfg<D, kF16>;
    const size_t smem = C::kBarsOffset + sizeof(Bars) + 1024;
    cudaError_t e = cudaFuncSetAttribute(paged_kernel<D, kF16>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_kernel<D, kF16>, maps.q, maps.q_quad, maps.k, maps.v, a);
    if (e != cudaSuccess || num_sms < 2)
        return e;
    const bool pairs = a.slot_rows > kBM;
    const int rows = pairs ? 2 : 1;  // a warp
    cfg.gridDim = dim3(num_sms - 1, (a.slot_rows + 4 * rows - 1) / (4 * rows));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return pairs ? cudaLaunchKernelEx(&cfg, combine_paged_kernel<D, kF16, 2, 2>, a, num_sms)
                 : cudaLaunchKernelEx(&cfg, combine_paged_kernel<D, kF16, 1, 8>, a, num_sms);
}

template <int D>
cudaError_t launch_typed(const PagedArgs &a, const PagedMaps &maps, int num_sms, cudaStream_t stream)
{
    return a.f16 ? launch<D, true>(a, maps, num_sms, stream) : launch<D, false>(a, maps, num_sms, stream);
}

}  // namespace

cudaError_t launch_paged(const PagedArgs &a, const PagedMaps &maps, int num_sms, cudaStream_t stream)
{
    switch (a.d) {
    case 64: return launch_typed<64>(a, maps, num_sms, stream);
    case 96: return launch_typed<96>(a, maps, num_sms, stream);
    case 128: return launch_typed<128>(a, maps, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fattn
