// fattn_cross_bwd_sm103.cu -- gradients of cross attention on GB300 (sm_103a):
// batched queries against keys of another length, ragged, with shared heads.
//
// From the saved q, k, v, o and lse, with P = exp(scale Q K^T - lse) (zero
// behind a sequence's last key) and D_i = dO_i . o_i, for the G query heads h of
// a key head:
//   dV = sum_h P^T dO,     dP = dO V^T,   dS = P o (dP - D),
//   dQ = scale dS K,       dK = scale sum_h dS^T Q.
// Four kernels, each started under the tail of the one before:
//   prep     D (of few keys from P and dP), the norms of dO's rows and V's (fp16), and
//            zeros for key tiles without keys
//   dkdv     a unit is a tile of 128 keys of one (sequence, key head).  K, V
//            stay; the tiles of Q and dO of its G query heads stream by: S^T =
//            K Q^T and dP^T = V dO^T, keys on TMEM lanes, P^T over S^T, then dV
//            += P^T dO and dK += dS^T Q from TMEM
//   dq       a unit is a tile of 128 queries of one head.  Q and dO stay, in TMEM; K
//            and V stream by: S, dP, dS over dP, then dQ += dS K
//   merge    sums of units that were split
// S and dP are formed in both, so that neither needs atomics: 7 products where
// 5 would do, and equal calls give equal bits.
//
// Schedule.  Lengths live on the device.  Every CTA (one an SM) sums the units'
// costs, a step (tile pair) each and some for a unit's start and end, and takes
// an equal share of the total, which may begin or end inside a unit: that
// unit's sums go to the workspace in fp32, at most two a CTA, and the merge
// kernel adds them in order.  So few key tiles under many queries (a short text)
// fill the GPU as well as the reverse.  Where units are short they are dealt out
// whole, without a merge, and small calls run their passes side by side: dq starts on
// the SMs that dkdv leaves.
//
// Bound.  At d = 128 the tensor cores and the shared memory that feeds them: a tile
// of dkdv takes some 2520 cycles, its products 2048 and its reads and copies in
// shared memory 2350; a tile of dq 2005, its products 1536 (Q and dO in TMEM save it
// two reads of 32 KB).  4 sequences, 16 heads, 2048 queries, up to 4096 keys, bf16:
// 490 us alone in a graph, 970 TFLOP/s of the formulas' five products, 1355 of the
// seven; at the power cap's clocks 522 us.  fp16, whose prep reads V, too, takes 4 %
// longer (keys of one length, graphs at the cap: 697 and 666 us).  At d = 64
// the chain TMEM, exponential, conversion, TMEM of the
// elementwise warps, shortened by a second S or dP; with few tiles a unit its start
// and end: 2 sequences, 16 heads, 4096 queries, up to 154 keys 59 us, 1.2 TB/s.
//
// Types.  P and dS enter the second products in the inputs' type.  P in fp16 is
// multiplied by 2^15, in its exponent and so at no cost: with 10^5 keys it is below fp16's
// normal numbers, where dV would lose digits.  dS = P (dP - D) has that factor, and
// is scaled by a power of two that follows from the norm of dO's row (for dK, whose
// sums go over the rows, the largest of the key head's) and the largest norm of a row
// of V before the sequence's end: |dP| is at most their product N, and P (1 - P) at
// most 1/4, so |dS| is at most N / 2.  N is brought to 1 .. 2, so that no dS is
// infinite and small ones keep their digits whatever stands beside them.  The sums
// are scaled back in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "fattn_internal.h"
#include "ptx_sm103.cuh"

namespace fattn {
namespace {

using namespace ptx;

constexpr int kTile = 128;
// Warps 0-15 elementwise: four warpgroups, 32 of a tile's 128 columns each, so that
// four warps a scheduler hide one another's waits for TMEM and barriers (at d = 128
// two warpgroups of 64 columns are as fast); 16 the producer, 17 MMA.
constexpr int kElemWarps = 16;
constexpr int kWarpLoad = 16;
constexpr int kWarpMma = 17;
constexpr int kThreads = 18 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kChunkBytes = kTile * 64 * 2;
constexpr uint32_t kColS = 0, kColDP = 128;

// A unit's start and end, in steps (see Schedule): some 4000 cycles, where a step
// takes 1500 to 2800.  A split leaves at least kSnap steps on each side, and a share is
// at least a unit of one step: 30 calls of 2 to 2000 queries and 1 to 4000 keys, d =
// 64, 96 and 128, take 24.5, 20.1 and 22.6 us in the (geometric) mean, with kLeast 6
// 25.7, 21.8 and 24.0, with 3 24.2, 20.2 and 22.7, but whole units up to 10 % more.
constexpr int kUnitCost = 3, kSnap = 2, kLeast = kUnitCost + 1;
// What the merge kernel takes, in steps (see whole_units).
template <int D> constexpr int kMergeCost = D == 64 ? 6 : 3;
// A step of dkdv to one of dq; and the steps a SM up to which the passes run side by
// side, each on its part of the SMs: that saves the second start and end, in the calls
// above 1 to 3 % in the mean, in some a sixth (36 to 30 us).  In longer calls it is
// little, and the passes in turn need no guess of their steps' lengths.
constexpr int kStepKv = 4, kStepQ = 3, kTogether = 32;

// D = dO . o is off by h |dO| |o|, h half a step of the type.  Over many keys o is a
// mean, and small; of a few it is as large as their values, and its rounding the larger
// part of the gradients' error.  There D is summed up from P and dP in 32 bits.  Error
// of bf16 dQ in the norm (d = 64, the roundings alone): 2 keys 0.0023, from o 0.0041; 4
// keys 0.0023 and 0.0029; 16 keys 0.0024 and 0.0025; from 24 keys on the two are alike.
constexpr int kFewKeys = 16;

template <int D, bool kDkDv> struct BCfg {
    static constexpr int kChunks = (D + 63) / 64;
    static constexpr uint32_t kTileBytes = kChunks * kChunkBytes;  // one [128][D] tile
    // Slots of the resident tiles, which take turns (K_j, V_j, K_j', ... or Q_i, dO_i,
    // ...); dq copies them to TMEM, so a slot is free at once.  Then the streamed
    // tiles, dkdv: Q and dO; dq: K (held until dQ) and V.
    static constexpr int kRes = D == 64 ? 4 : 2;
    static constexpr int kStages = D == 64 ? 4 : kDkDv ? 2 : 3;
    static constexpr int kStages2 = kDkDv ? kStages : D == 64 ? 3 : 2;
    static constexpr uint32_t kRing = kRes * kTileBytes;
    static constexpr uint32_t kRing2 = kRing + kStages * kTileBytes;
    static constexpr uint32_t kTilesBytes = kRing2 + kStages2 * kTileBytes;
    // TMEM: S, dP; at d = 64 a second S (dkdv) or dP (dq), so that the next one is
    // there when the elementwise pass is done with this; the sums; dq: Q and dO.
    static constexpr int kTwo = D == 64;
    static constexpr uint32_t kColAcc = kTwo ? 384 : 256;
    static constexpr uint32_t kAccCols = kDkDv ? 2 * D : D;
    static constexpr uint32_t kColQ = kColAcc + kAccCols, kColDO = kColQ + D / 2;
    static_assert((kDkDv ? kColQ : kColDO + D / 2) <= kTmemCols, "TMEM columns");
    static __device__ __forceinline__ uint32_t s_col(uint32_t pos)
    {
        return kDkDv && kTwo && (pos & 1) ? 256 : kColS;
    }
    static __device__ __forceinline__ uint32_t dp_col(uint32_t pos)
    {
        return !kDkDv && kTwo && (pos & 1) ? 256 : kColDP;
    }
};

// Where a CTA starts: a sequence, the cost already behind in it, and its share.
struct Start {
    int b;
    long long y, left;
};

// A piece of work: steps [t0, t1) of a unit.
struct Piece {
    int b, h, tile;  // h < 0: no more work
    int L;           // keys of the sequence
    int t0, t1;      // dkdv: (query head of the group, query tile); dq: key tiles
    int slot;        // workspace slot of a partial result, or -1: the whole unit
};
constexpr int kPieces = 4;  // published ahead

struct alignas(16) BBars {
    uint64_t res_full[4], res_empty[4], q_full;  // q_full: dq, Q and dO are in TMEM
    uint64_t st_full[4], st_empty[4];  // dkdv: Q stages; dq: K stages
    uint64_t v_full[4], v_empty[4];    // dkdv: dO stages; dq: V stages
    // Of tile n on n % 2: S and dP computed, P^T (dq: S is in registers) and dS
    // written.  With two S or two dP the elementwise pass can be done with the tile
    // after the one that the MMA lane is about to wait for: on one barrier that
    // would be two phases, which a parity does not tell from none.
    uint64_t s_full[2], dp_full[2], p1_full[2], p_full[2];
    uint64_t o_full, o_empty;
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    Start start;
    Piece pieces[kPieces];
};
// dkdv, behind the barriers: each warp's -lse log2(e) and -D (scaled) of the 32
// queries of its columns, two tiles deep.
struct BXch {
    float lse2[kElemWarps][2][32], dd[kElemWarps][2][32];
};

__device__ __forceinline__ int clamp_len(const CrossBwdArgs &a, int b)
{
    const int L = a.kv_len != nullptr ? __ldcg(a.kv_len + b) : a.Nk;
    return min(max(L, 0), a.Nk);
}

// Units of a sequence with L keys, and the steps of each.  Units without steps
// are none: the prep kernel writes their zeros.
template <bool kDkDv>
__device__ __forceinline__ void units_of(const CrossBwdArgs &a, int L, int &units, int &steps)
{
    const int F = (L + kTile - 1) / kTile;
    steps = kDkDv ? a.G * a.Tq : F;
    units = steps == 0 ? 0 : kDkDv ? a.Hk * F : a.Hk * a.G * a.Tq;
}
// Step that a cost of y inside a unit falls on.
__device__ __forceinline__ int step_at(long long y, int steps, int snap)
{
    if (y >= steps + kUnitCost)
        return steps;
    const int t = y < kUnitCost ? 0 : static_cast<int>(y - kUnitCost);
    return t < snap ? 0 : steps - t < snap ? steps : t;
}

// a / b of non-negative values, in 32 bits where they fit.
__device__ __noinline__ long long long_quotient(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long quotient(long long a, int b)
{
    return (a >> 32) == 0 ? static_cast<unsigned>(a) / static_cast<unsigned>(b) : long_quotient(a, b);
}

struct Walk {
    Start at;
    int L, units, steps, u;
};
template <bool kDkDv> __device__ __forceinline__ void enter(const CrossBwdArgs &a, Walk &w)
{
    w.L = clamp_len(a, w.at.b);
    units_of<kDkDv>(a, w.L, w.units, w.steps);
}
template <bool kDkDv> __device__ __forceinline__ Walk first_walk(const CrossBwdArgs &a, const BBars &b)
{
    Walk w;
    w.at = b.start;
    w.u = w.units = 0;
    if (w.at.left > 0) {
        enter<kDkDv>(a, w);
        const int cost = w.steps + kUnitCost;
        w.u = static_cast<int>(quotient(w.at.y, cost));
        w.at.y -= static_cast<long long>(w.u) * cost;
    }
    return w;
}
template <bool kDkDv> __device__ __forceinline__ bool next_piece(const CrossBwdArgs &a, Walk &w, Piece &p)
{
    while (w.at.left > 0) {
        if (w.u >= w.units) {
            w.u = 0;
            if (++w.at.b >= a.B)
                return false;
            enter<kDkDv>(a, w);
            continue;
        }
        const int cost = w.steps + kUnitCost;
        const long long y0 = w.at.y, y1 = min(y0 + w.at.left, static_cast<long long>(cost));
        const int u = w.u++;
        w.at.left -= y1 - y0;
        w.at.y = 0;
        p.t0 = step_at(y0, w.steps, a.snap);
        p.t1 = step_at(y1, w.steps, a.snap);
        if (p.t0 == p.t1)  // nothing of it falls to this CTA
            continue;
        const int per = kDkDv ? w.units / a.Hk : a.Tq;
        p.b = w.at.b;
        p.h = u / per;
        p.tile = u - p.h * per;
        p.L = w.L;
        const int cta = static_cast<int>(blockIdx.x);
        p.slot = p.t0 > 0 ? 2 * cta : p.t1 < w.steps ? 2 * cta + 1 : -1;
        return true;
    }
    return false;
}

// Finds this CTA's start: warp 0 alone, 32 sequences at a time.
template <bool kDkDv> __device__ void find_start(const CrossBwdArgs &a, BBars &b)
{
    if (threadIdx.x >= 32)
        return;
    const int lane = threadIdx.x;
    // Cost of sequence i, whose lengths the second walk finds in the cache.
    auto cost_of = [&](int i, int &units, int &steps) {
        units = steps = 0;
        if (i < a.B)
            units_of<kDkDv>(a, clamp_len(a, i), units, steps);
        return static_cast<long long>(units) * (steps + kUnitCost);
    };
    int units, steps;
    long long total = 0, other = 0;  // of this pass and of the other one
    for (int i = lane; i < a.B; i += 32) {
        total += cost_of(i, units, steps);
        units_of<!kDkDv>(a, clamp_len(a, i), units, steps);
        other += static_cast<long long>(units) * (steps + kUnitCost);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        other += __shfl_xor_sync(0xffffffffu, other, o);
    }
    const int c = blockIdx.x;
    // A small call's passes run side by side, each on its part of the SMs.
    const long long mine = total * (kDkDv ? kStepKv : kStepQ), both = mine + other * (kDkDv ? kStepQ : kStepKv);
    int most = gridDim.x;
    if (both <= static_cast<long long>(kTogether) * kStepKv * most && total > 0 && other > 0) {
        const int kv = static_cast<int>(quotient((kDkDv ? mine : both - mine) * most + both / 2, static_cast<int>(both)));
        most = max(kDkDv ? kv : most - kv, 1);
    }
    const int shares = static_cast<int>(min(static_cast<long long>(most), max(quotient(total, kLeast), 1LL)));
    const long long each = quotient(total, shares);
    const int rest = static_cast<int>(total - each * shares);
    const long long lo = c * each + c * rest / shares, hi = (c + 1) * each + (c + 1) * rest / shares;
    int4 *starts = a.starts + (kDkDv ? 0 : a.grid);
    if (c >= shares || lo >= hi) {
        if (lane == 0) {
            b.start = Start{0, 0, 0};
            starts[c] = make_int4(-1, 0, 0, 0);
        }
        return;
    }
    // The sequence that holds this CTA's first cost.
    long long before = 0;
    for (int b0 = 0; b0 < a.B && before <= lo; b0 += 32) {
        const long long mine = cost_of(b0 + lane, units, steps);
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            incl += lane >= o ? x : 0;
        }
        const long long first = before + incl - mine;
        if (first <= lo && lo < first + mine) {
            b.start = Start{b0 + lane, lo - first, hi - lo};
            const int cost = steps + kUnitCost, u = static_cast<int>(quotient(lo - first, cost));
            const int t = step_at(lo - first - static_cast<long long>(u) * cost, steps, a.snap);
            const int per = kDkDv ? units / a.Hk : a.Tq, h = u / per;
            starts[c] = make_int4(b0 + lane, h, u - h * per, t < steps ? t : 0);
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ __forceinline__ void fail(const CrossBwdArgs &a, BBars &b, uint32_t role)
{
    const uint32_t code = 4u /* FATTN_ERR_TIMEOUT */ | (role << 8) | ((blockIdx.x & 0xffffu) << 16);
    atomicCAS(a.status, 0u, code);
    *reinterpret_cast<volatile int *>(&b.abort) = 1;
}
__device__ __forceinline__ bool warp_wait(uint64_t &bar, uint32_t parity, const volatile int *abort)
{
    const bool ok = mbar_wait(smem_addr(&bar), parity, kWaitLimitNs, abort);
    return __all_sync(0xffffffffu, ok);
}
// The same value on every lane of a converged warp, read afresh: copy
// coordinates that follow from the lists go through it inside the loop that uses
// them (see paged_sm103.cuh).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// The same where one lane runs alone, by its number as elect.sync gave it.
__device__ __forceinline__ uint32_t uniform_of(uint32_t x, uint32_t lane)
{
    return __shfl_sync(1u << lane, x, static_cast<int>(lane));
}
__device__ __forceinline__ uint32_t elected_lane()
{
    uint32_t lane;
    asm volatile("{\n\t.reg .pred P1;\n\telect.sync %0|P1, 0xffffffff;\n\t}" : "=r"(lane));
    return lane;
}

// The pieces, published by the producer.  The k-th, read in place; false when
// there is none (ok) or a wait failed (!ok).  Held until given back.
__device__ __forceinline__ bool receive(BBars &b, uint32_t k, bool &ok)
{
    ok = ok && warp_wait(b.piece_full[k % kPieces], (k / kPieces) & 1, &b.abort);
    return ok && b.pieces[k % kPieces].h >= 0;
}
__device__ __forceinline__ void give_back(BBars &b, uint32_t k)
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

// ------------------------------------------------------------------ products
// [128 x D] x [128 x D]^T, both K-major, into 128 fp32 columns.
template <int D, bool kF16>
__device__ __forceinline__ void mma_nt(uint32_t tmem_d, uint32_t a_smem, uint32_t b_smem)
{
    constexpr uint32_t idesc = idesc_f32acc(kTile, kTile, false, kF16);
    constexpr uint32_t hi = smem_desc_hi(1024);
    const uint32_t a_lo = smem_desc_lo(a_smem, 16), b_lo = smem_desc_lo(b_smem, 16);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
        mma_ss_w(tmem_d, a_lo + off, hi, b_lo + off, hi, idesc, kk > 0 ? 1u : 0u);
    }
}
// The same with A in TMEM, D / 2 packed columns.
template <int D, bool kF16>
__device__ __forceinline__ void mma_nt_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_smem)
{
    constexpr uint32_t idesc = idesc_f32acc(kTile, kTile, false, kF16);
    constexpr uint32_t hi = smem_desc_hi(1024);
    const uint32_t b_lo = smem_desc_lo(b_smem, 16);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        mma_ts_w(tmem_d, tmem_a + kk * 8, b_lo + (((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4), hi, idesc,
                 kk > 0 ? 1u : 0u);
}
// A from TMEM: 16 packed columns at the head of each 32-column chunk of a score
// region, K = 16 step kk at column 32 (kk / 2) + 8 (kk % 2).  B MN-major.
template <int D, bool kF16>
__device__ __forceinline__ void mma_tn(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_smem, bool accumulate)
{
    constexpr uint32_t idesc = idesc_f32acc(kTile, D, true, kF16);
    constexpr uint32_t hi = smem_desc_hi(1024);
    const uint32_t b_lo = smem_desc_lo(b_smem, D > 64 ? kChunkBytes : 1024);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
        mma_ts_w(tmem_d, tmem_a + 32 * (kk >> 1) + 8 * (kk & 1), b_lo + ((kk * 16 * 128) >> 4), hi, idesc,
                 kk > 0 || accumulate ? 1u : 0u);
}

// ------------------------------------------------------------------ producer
template <int D, bool kDkDv>
__device__ void bwd_load(const CrossBwdArgs &a, BBars &b, uint32_t smem, const CUtensorMap *mq,
                         const CUtensorMap *mk, const CUtensorMap *mv, const CUtensorMap *mdo)
{
    using C = BCfg<D, kDkDv>;
    const volatile int *abort = &b.abort;
    const bool leader = elect_one();
    uint32_t rpos = 0, kpos = 0, vpos = 0;  // resident, streamed and other streamed tiles
    // A tile, when its slot is free.
    auto load = [&](uint64_t *full, uint64_t *empty, uint32_t &pos, int slots, uint32_t base,
                    const CUtensorMap *map, int row, int head, int batch) {
        const uint32_t slot = pos % slots;
        if (!warp_wait(empty[slot], ((pos / slots) & 1) ^ 1, abort))
            return false;
        if (leader) {
            const uint32_t bar = smem_addr(&full[slot]), dst = smem + base + slot * C::kTileBytes;
            mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
                tma_load_4d(dst + c * kChunkBytes, map, bar, 64 * c, row, head, batch);
        }
        ++pos;
        return true;
    };
    bool ok = true;
    uint32_t k = 0;
    Walk w = first_walk<kDkDv>(a, b);
    Piece p;
    bool more = true;
    while (ok && more) {
        more = next_piece<kDkDv>(a, w, p);
        ok = warp_wait(b.piece_empty[k % kPieces], ((k / kPieces) & 1) ^ 1, abort);
        if (!ok)
            break;
        if (!more)
            p.h = -1;
        if ((threadIdx.x & 31) == 0) {
            b.pieces[k % kPieces] = p;
            mbar_arrive(smem_addr(&b.piece_full[k % kPieces]));
        }
        ++k;
        if (!more)
            break;
        const int head = uniform(p.h), batch = uniform(p.b), own = uniform(p.tile * kTile);
        ok = load(b.res_full, b.res_empty, rpos, C::kRes, 0, kDkDv ? mk : mq, own, head, batch) &&
             load(b.res_full, b.res_empty, rpos, C::kRes, 0, kDkDv ? mv : mdo, own, head, batch);
        int g = kDkDv ? p.t0 / a.Tq : 0, i = kDkDv ? p.t0 - g * a.Tq : 0;
        for (int t = p.t0; ok && t < p.t1; ++t) {
            if constexpr (kDkDv) {
                // dO first: its slot is released (after dV) before Q's (after dK).
                const int row = uniform(i * kTile), qh = uniform(p.h * a.G + g);
                ok = load(b.v_full, b.v_empty, vpos, C::kStages2, C::kRing2, mdo, row, qh, batch) &&
                     load(b.st_full, b.st_empty, kpos, C::kStages, C::kRing, mq, row, qh, batch);
                if (++i == a.Tq) {
                    i = 0;
                    ++g;
                }
            } else {
                const int row = uniform(t * kTile), kh = uniform(p.h / a.G);
                ok = load(b.st_full, b.st_empty, kpos, C::kStages, C::kRing, mk, row, kh, batch) &&
                     load(b.v_full, b.v_empty, vpos, C::kStages2, C::kRing2, mv, row, kh, batch);
            }
        }
    }
    if (!ok) {
        if (leader)
            fail(a, b, kRoleLoad);
        // Copies already issued land before the CTA exits.
        auto land = [&](uint64_t *full, uint32_t pos, uint32_t slots) {
            for (uint32_t q = pos > slots ? pos - slots : 0; q < pos; ++q)
                mbar_wait(smem_addr(&full[q % slots]), (q / slots) & 1, kWaitLimitNs / 8, nullptr);
        };
        land(b.st_full, kpos, C::kStages);
        land(b.v_full, vpos, C::kStages2);
        land(b.res_full, rpos, C::kRes);
    }
}

// ------------------------------------------------------------------ MMA issue
// The CTA's tiles as one stream, across the pieces' ends: the first products of
// a tile go out while the elementwise pass is at the one before, be it the last
// of another unit.  Run by one lane, and what is between two products is short:
// the tensor cores wait for it (with votes, shuffles and remainders for each
// place in a ring, a fifth of the time).
template <int kSlots> struct Ring {  // a place in a ring and its phase
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void step()
    {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
    }
};
template <int D, bool kF16, bool kDkDv>
__device__ void bwd_mma(const CrossBwdArgs &a, BBars &b, uint32_t smem, uint32_t tmem, uint32_t lane)
{
    using C = BCfg<D, kDkDv>;
    const volatile int *abort = &b.abort;
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        return mbar_wait(smem_addr(&bar), parity & 1, kWaitLimitNs, abort);
    };
    auto commit = [&](uint64_t &bar) { mma_commit(smem_addr(&bar)); };
    bool ok = true;
    uint32_t piece = 0, pos = 0;
    // Tiles of the piece, 0: there is none.
    auto tiles_of = [&](uint32_t k) {
        ok = ok && wait(b.piece_full[k % kPieces], k / kPieces);
        if (!ok || b.pieces[k % kPieces].h < 0)
            return 0;
        return static_cast<int>(uniform_of(b.pieces[k % kPieces].t1 - b.pieces[k % kPieces].t0, lane));
    };
    Ring<C::kRes> res0, res1;  // dkdv: of the piece that S and dP are at
    res1.step();
    Ring<C::kStages> st_s, st_k;  // of S, and of dK or dQ
    Ring<C::kStages2> v_d, v_v;   // of dP, and of dV
    auto step2 = [](auto &x) {
        x.step();
        x.step();
    };
    auto at = [&](uint32_t base, uint32_t slot) {
        return uniform_of(smem + base + slot * C::kTileBytes, lane);
    };
    // S (S^T) of a tile, the `t`-th of the `n` of piece `k`, `pos`-th of all; dP (dP^T).
    auto scores = [&](uint32_t k, uint32_t pos, int t, int n) {
        ok = ok && (t > 0 || (kDkDv ? wait(b.res_full[res0.slot], res0.phase) : wait(b.q_full, k))) &&
             wait(b.st_full[st_s.slot], st_s.phase);
        if (!ok)
            return;
        tc_fence_after();
        if constexpr (kDkDv)
            mma_nt<D, kF16>(tmem + C::s_col(pos), at(0, res0.slot), at(C::kRing, st_s.slot));
        else
            mma_nt_ts<D, kF16>(tmem + kColS, tmem + C::kColQ, at(C::kRing, st_s.slot));
        commit(b.s_full[pos & 1]);
        if (kDkDv && t + 1 == n) {
            commit(b.res_empty[res0.slot]);
            step2(res0);
        }
        st_s.step();
    };
    auto grads = [&](uint32_t pos, int t, int n) {
        ok = ok && (t > 0 || !kDkDv || wait(b.res_full[res1.slot], res1.phase)) &&
             wait(b.v_full[v_d.slot], v_d.phase);
        if (!ok)
            return;
        tc_fence_after();
        if constexpr (kDkDv)
            mma_nt<D, kF16>(tmem + kColDP, at(0, res1.slot), at(C::kRing2, v_d.slot));
        else
            mma_nt_ts<D, kF16>(tmem + C::dp_col(pos), tmem + C::kColDO, at(C::kRing2, v_d.slot));
        commit(b.dp_full[pos & 1]);
        if (!kDkDv)
            commit(b.v_empty[v_d.slot]);
        if (kDkDv && t + 1 == n) {
            commit(b.res_empty[res1.slot]);
            step2(res1);
        }
        v_d.step();
    };
    int n = tiles_of(0);
    if (n > 0) {
        scores(0, 0, 0, n);
        grads(0, 0, n);
    }
    const uint32_t acc = tmem + C::kColAcc;
    while (ok && n > 0) {
        int next = 0;
        for (int t = 0; ok && t < n; ++t, ++pos) {
            // The tile after this one: of this piece or the first of the next.
            const bool last = t + 1 == n;
            const int t_next = last ? 0 : t + 1;
            auto acc_wait = [&]() { return t > 0 || wait(b.o_empty, piece ^ 1); };
            if constexpr (!kDkDv) {
                // dS is written over dP.  S of the next tile once this one's is in
                // registers, dP of it after dQ (with another dP at once); another
                // piece's Q and dO are written after this one's last dS.
                ok = ok && wait(b.p1_full[pos & 1], pos >> 1);
                if (!last) {
                    scores(piece, pos + 1, t_next, n);
                    if (C::kTwo)
                        grads(pos + 1, t_next, n);
                }
                ok = ok && wait(b.p_full[pos & 1], pos >> 1) && acc_wait();
                if (!ok)
                    break;
                tc_fence_after();
                mma_tn<D, kF16>(acc, tmem + C::dp_col(pos), at(C::kRing, st_k.slot), t > 0);  // dQ += dS K
                commit(b.st_empty[st_k.slot]);
                st_k.step();
                if (last) {
                    commit(b.o_full);
                    next = tiles_of(piece + 1);
                    if (next > 0)
                        scores(piece + 1, pos + 1, 0, next);
                }
                if (last ? next > 0 : !C::kTwo)
                    grads(pos + 1, t_next, last ? next : n);
            } else {
                // P^T is written over S^T, dS^T over dP^T: the next S^T follows dV
                // (with another S it is ahead), the next dP^T dK.  Behind a piece's last
                // tile dK goes first where the next piece's K is still to be loaded.
                int n_next = n;
                auto next_scores = [&]() {
                    if (last)
                        n_next = next = tiles_of(piece + 1);
                    if (n_next > 0)
                        scores(last ? piece + 1 : piece, pos + 1, t_next, n_next);
                };
                if constexpr (C::kTwo)
                    next_scores();
                ok = ok && wait(b.p1_full[pos & 1], pos >> 1) && acc_wait();
                if (!ok)
                    break;
                tc_fence_after();
                mma_tn<D, kF16>(acc, tmem + C::s_col(pos), at(C::kRing2, v_v.slot), t > 0);  // dV += P^T dO
                commit(b.v_empty[v_v.slot]);
                v_v.step();
                if (!C::kTwo && !last)
                    next_scores();
                ok = ok && wait(b.p_full[pos & 1], pos >> 1);
                if (!ok)
                    break;
                tc_fence_after();
                mma_tn<D, kF16>(acc + D, tmem + kColDP, at(C::kRing, st_k.slot), t > 0);  // dK += dS^T Q
                commit(b.st_empty[st_k.slot]);
                st_k.step();
                if (last) {
                    commit(b.o_full);
                    if (!C::kTwo)
                        next_scores();
                }
                if (n_next > 0)
                    grads(pos + 1, t_next, n_next);
            }
        }
        if (!ok)
            break;
        mbar_arrive(smem_addr(&b.piece_empty[piece % kPieces]));
        ++piece;
        n = next;
    }
    if (!ok)
        fail(a, b, kRoleMma);
    commit(b.drain);
    mbar_wait(smem_addr(&b.drain), 0, kWaitLimitNs, nullptr);
}

// What fp16's P is multiplied by (see Types): P is at most 1, and 2^16 too large.
template <bool kF16> constexpr float kPExponent = kF16 ? 15.f : 0.f;
template <bool kF16> constexpr float kPInverse = kF16 ? 1.f / 32768.f : 1.f;

// -lse log2(e), with which P = 2^(s scale log2(e) + it), and P's factor; of a row
// that saw no key (lse = -inf) -inf, so that its P is 0.
template <bool kF16> __device__ __forceinline__ float neg_lse2(float lse)
{
    return lse == -INFINITY ? lse : kF16 ? fmaf(-lse, kLog2e, kPExponent<kF16>) : -lse * kLog2e;
}

// Four lanes' 16-byte pieces change places: v[j] of lane i of four becomes v[i]
// of lane j.  Rows held a lane each are then stored 64 bytes at a time, eight rows
// an instruction (16 bytes at a time, half a sector each, the end of a unit took
// 9400 cycles at d = 128).
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane)
{
    auto trade = [&](uint4 &a, uint4 &b, int by) {
        const bool up = lane & by;
        uint4 x = up ? a : b;
        x.x = __shfl_xor_sync(0xffffffffu, x.x, by);
        x.y = __shfl_xor_sync(0xffffffffu, x.y, by);
        x.z = __shfl_xor_sync(0xffffffffu, x.z, by);
        x.w = __shfl_xor_sync(0xffffffffu, x.w, by);
        if (up)
            a = x;
        else
            b = x;
    };
    trade(v[0], v[1], 1);
    trade(v[2], v[3], 1);
    trade(v[0], v[2], 2);
    trade(v[1], v[3], 2);
}

// What dQ's and dK's sums are multiplied by.  With one key P is 1 whatever q and k
// are, and dS is zero: D, from o in 16 bits and in another order of sums, would leave
// some 1e-6 |dO| |v| of it.
template <bool kF16> __device__ __forceinline__ float grad_scale(const CrossBwdArgs &a, int keys, float ds_scale)
{
    return keys == 1 ? 0.f : a.scale / ds_scale * kPInverse<kF16>;
}

// The largest of some values, NaN aside, each lane some of them; and of the lanes'.
__device__ __forceinline__ float lanes_max(const float *x, int n, int lane)
{
    float m = lane < n ? __ldcg(x + lane) : 0.f;  // of up to 32 not waited for here
#pragma unroll 2
    for (int i = lane + 32; i < n; i += 32)
        m = fmaxf(m, __ldcg(x + i));
    return m;
}
__device__ __forceinline__ float warp_max(float m)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
// The power of two that brings the product of two norms to 1 .. 2: 1 where it is zero
// or not finite.
__device__ __forceinline__ float scale_of(float x)
{
    const uint32_t e = __float_as_uint(x) >> 23;  // of fp16 rows' norms 79 .. 167
    return x > 0.f && e >= 1 && e <= 253 ? __uint_as_float((254u - e) << 23) : 1.f;
}

// ------------------------------------------------------------------ elementwise
// Thread r of a warpgroup owns TMEM lane r, row 128 tile + r of the resident tile;
// warpgroup g works on columns 32 g .. 32 g + 31 of it.
template <int D, bool kF16, bool kDkDv>
__device__ void bwd_elem(const CrossBwdArgs &a, BBars &b, BXch &xch, uint8_t *tiles, uint32_t tmem)
{
    using C = BCfg<D, kDkDv>;
    const volatile int *abort = &b.abort;
    const int warp = (threadIdx.x / 32) & 3, lane = threadIdx.x & 31;
    const int quarter = threadIdx.x / 128;
    const int r = warp * 32 + lane;
    tmem += static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t col = quarter * 32;
    uint32_t pos = 0;  // tiles so far
    bool ok = true;
    // What dS is multiplied by, twice: dkdv, of the piece; dq, of the row.
    uint64_t dss = f2_pack(1.f, 1.f);
    auto ds_scale = [&]() {
        float x, y;
        f2_unpack(dss, x, y);
        return x;
    };
    const uint64_t sl2x2 = f2_pack(a.sl2, a.sl2);
    auto wait = [&](uint64_t &bar, uint32_t phase) {
        return mbar_wait(smem_addr(&bar), phase & 1, kWaitLimitNs, abort);
    };
    auto arrive = [&](uint64_t &bar) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&bar));
    };
    // dkdv: lse and D of the query of this lane's column, fetched a tile ahead, the
    // next piece's first one too.
    float next_lse = 0.f, next_d = 0.f;
    // fp16: norms of dO (dkdv: a lane's part of the piece's; dq: the row's) and of V (a
    // lane's part).  Read and used outside the loop over tiles: inside of it, in what is
    // done once at its end, their shuffles cost dq an eighth of its time.
    float norm = 0.f, v_norm = 0.f;
    auto fetch_norms = [&](const Piece &p) {
        if constexpr (kF16) {
            const long long head = static_cast<long long>(p.b) * a.Hk + (kDkDv ? p.h : p.h / a.G);
            const int row = p.tile * kTile + r;
            v_norm = lanes_max(a.v_max + head * a.v_parts, a.v_parts, lane);
            if (kDkDv)
                norm = lanes_max(a.do_max + head * a.do_parts, a.do_parts, lane);
            else
                norm = row < a.Nq ? __ldcg(a.norms + (static_cast<long long>(p.b) * a.Hk * a.G + p.h) * a.Nq + row)
                                  : 0.f;
        }
    };
    auto set_scale = [&]() {
        if constexpr (kF16) {
            const float x = scale_of((kDkDv ? warp_max(norm) : norm) * warp_max(v_norm));
            dss = f2_pack(x, x);
        }
    };
    auto fetch = [&](const Piece &p, int t) {
        const int g = t / a.Tq, q = (t - g * a.Tq) * kTile + col + lane;
        const long long at = ((static_cast<long long>(p.b) * a.Hk + p.h) * a.G + g) * a.Nq + q;
        next_lse = q < a.Nq ? __ldcg(a.lse + at) : 0.f;
        next_d = q < a.Nq ? __ldcg((p.L <= kFewKeys ? a.dfew : a.dvec) + at) : 0.f;
    };
    // dq: the k-th piece's Q and dO into TMEM, 32 elements of a row a job, a lane a
    // row; and the row's lse and D, fetched before.
    float row_nl2 = 0.f, row_nd = 0.f;
    auto fetch_row = [&](const Piece &p) {
        const int row = p.tile * kTile + r;
        const long long at = (static_cast<long long>(p.b) * a.Hk * a.G + p.h) * a.Nq + row;
        next_lse = row < a.Nq ? __ldcg(a.lse + at) : 0.f;
        next_d = row < a.Nq ? __ldcg((p.L <= kFewKeys ? a.dfew : a.dvec) + at) : 0.f;
    };
    auto make_resident = [&](uint32_t k) {
        constexpr int kJobs = D / 32;  // of each tensor
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t slot = (2 * k + i) % C::kRes;
            ok = ok && wait(b.res_full[slot], (2 * k + i) / C::kRes);
#pragma unroll
            for (int j = 0; j < (kJobs + 3) / 4; ++j) {
                // dO's jobs begin where Q's end (kColDO follows kColQ).
                const int job = (quarter + 4 * j + (i == 0 ? 0 : 4 - kJobs % 4)) % 4 + 4 * j;
                if (!ok || job >= kJobs)
                    continue;
                const uint8_t *tile = tiles + slot * C::kTileBytes + (job / 2) * kChunkBytes + r * 128;
                uint32_t x[16];
#pragma unroll
                for (int g = 0; g < 4; ++g) {  // 16-byte piece g of the row is at g ^ (r % 8)
                    const uint4 v = reinterpret_cast<const uint4 *>(tile)[((job % 2) * 4 + g) ^ (r & 7)];
                    x[4 * g] = v.x;
                    x[4 * g + 1] = v.y;
                    x[4 * g + 2] = v.z;
                    x[4 * g + 3] = v.w;
                }
                __syncwarp();
                tmem_st16(tmem + (i == 0 ? C::kColQ : C::kColDO) + job * 16, x);
            }
            arrive(b.res_empty[slot]);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(b.q_full);
    };
    for (uint32_t k = 0; receive(b, k, ok); ++k) {
        const Piece &p = b.pieces[k % kPieces];
        const int t0 = p.t0, t1 = p.t1;
        if (k == 0) {
            if (kDkDv) {
                fetch(p, t0);
                fetch_norms(p);
            } else {
                fetch_row(p);
                fetch_norms(p);
                make_resident(k);
            }
        }
        set_scale();
        if (!kDkDv) {
            row_nl2 = neg_lse2<kF16>(next_lse);
            row_nd = -next_d * ds_scale();
        }
        for (int t = t0; ok && t < t1; ++t, ++pos) {
            if constexpr (kDkDv) {
                float *lse2 = xch.lse2[threadIdx.x / 32][pos & 1], *dd = xch.dd[threadIdx.x / 32][pos & 1];
                lse2[lane] = neg_lse2<kF16>(next_lse);
                dd[lane] = -next_d * ds_scale();
                if (t + 1 < t1)
                    fetch(p, t + 1);
                else if (receive(b, k + 1, ok))
                    fetch(b.pieces[(k + 1) % kPieces], b.pieces[(k + 1) % kPieces].t0);
                __syncwarp();
                ok = ok && wait(b.s_full[pos & 1], pos >> 1);
                if (!ok)
                    break;
                tc_fence_after();
                // P^T, kept in registers and written over the first 16 columns of
                // the S^T chunk.  Queries behind Nq are zero rows of Q and dO and
                // add nothing; keys behind the last one are lanes of their own, not
                // stored.
                float pr[32];
                {
                    uint32_t sr[32], pk[16];
                    __syncwarp();
                    tmem_ld32(tmem + C::s_col(pos) + col, sr);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const ulonglong2 nl2 = *reinterpret_cast<const ulonglong2 *>(&lse2[2 * i]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * (i + j)]),
                                                     __uint_as_float(sr[2 * (i + j) + 1])),
                                             sl2x2, j == 0 ? nl2.x : nl2.y),
                                      x0, x1);
                            pr[2 * (i + j)] = ex2(x0);
                            pr[2 * (i + j) + 1] = ex2(x1);
                            pk[i + j] = pack2<kF16>(pr[2 * (i + j)], pr[2 * (i + j) + 1]);
                        }
                    }
                    tmem_st16(tmem + C::s_col(pos) + col, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(b.p1_full[pos & 1]);
                // dS^T = P^T (dP^T - D) over the first 16 columns of the chunk.
                ok = wait(b.dp_full[pos & 1], pos >> 1);
                if (!ok)
                    break;
                tc_fence_after();
                {
                    uint32_t dr[32], dk[16];
                    __syncwarp();
                    tmem_ld32(tmem + kColDP + col, dr);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const ulonglong2 nd = *reinterpret_cast<const ulonglong2 *>(&dd[2 * i]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int c = 2 * (i + j);
                            float d0, d1;
                            f2_unpack(f2_mul(f2_pack(pr[c], pr[c + 1]),
                                             f2_fma(f2_pack(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1])), dss,
                                                    j == 0 ? nd.x : nd.y)),
                                      d0, d1);
                            dk[i + j] = pack2<kF16>(d0, d1);
                        }
                    }
                    tmem_st16(tmem + kColDP + col, dk);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(b.p_full[pos & 1]);
            } else {
                ok = wait(b.s_full[pos & 1], pos >> 1);
                if (!ok)
                    break;
                tc_fence_after();
                const int valid = p.L - t * kTile;  // keys of this tile
                if (t + 1 == t1 && receive(b, k + 1, ok))
                    fetch_row(b.pieces[(k + 1) % kPieces]);
                // P in registers, so that the next S is computed meanwhile.
                float pr[32];
                {
                    uint32_t sr[32];
                    __syncwarp();
                    tmem_ld32(tmem + kColS + col, sr);
                    tmem_wait_ld();
                    tc_fence_before();
                    arrive(b.p1_full[pos & 1]);
                    const uint64_t nl2 = f2_pack(row_nl2, row_nl2);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), sl2x2, nl2), x0,
                                  x1);
                        pr[i] = ex2(x0);
                        pr[i + 1] = ex2(x1);
                    }
                }
                if (valid < kTile) {
                    // What lies behind the last key may be anything: dS is zero
                    // there, and so must K be (S has read it).
                    uint4 *k_tile = reinterpret_cast<uint4 *>(tiles + C::kRing + pos % C::kStages * C::kTileBytes);
                    for (int at = threadIdx.x; at < C::kChunks * kTile * 8; at += kElemWarps * 32)
                        if ((at / 8) % kTile >= valid)
                            k_tile[at] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                ok = wait(b.dp_full[pos & 1], pos >> 1);
                if (!ok)
                    break;
                tc_fence_after();
                {
                    uint32_t dr[32], dk[16];
                    __syncwarp();
                    tmem_ld32(tmem + C::dp_col(pos) + col, dr);
                    tmem_wait_ld();
                    const uint64_t nd = f2_pack(row_nd, row_nd);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float d0, d1;
                        f2_unpack(f2_mul(f2_pack(pr[2 * i], pr[2 * i + 1]),
                                         f2_fma(f2_pack(__uint_as_float(dr[2 * i]), __uint_as_float(dr[2 * i + 1])),
                                                dss, nd)),
                                  d0, d1);
                        if (valid < kTile) {  // uniform
                            d0 = static_cast<int>(col) + 2 * i < valid ? d0 : 0.f;
                            d1 = static_cast<int>(col) + 2 * i + 1 < valid ? d1 : 0.f;
                        }
                        dk[i] = pack2<kF16>(d0, d1);
                    }
                    // dS over the first half of its own chunk of dP.
                    tmem_st16(tmem + C::dp_col(pos) + col, dk);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(b.p_full[pos & 1]);
                // S and dP of this piece are done: the next one's rows.
                if (t + 1 == t1 && receive(b, k + 1, ok))
                    make_resident(k + 1);
            }
        }
        if (!ok)
            break;
        if (kF16 && receive(b, k + 1, ok))
            fetch_norms(b.pieces[(k + 1) % kPieces]);
        ok = ok && wait(b.o_full, k);
        if (!ok)
            break;
        tc_fence_after();
        // dkdv: dV by warpgroups 0 and 1, dK by 2 and 3, alternate 32-column
        // chunks; dq: a chunk a warpgroup.
        const bool is_dv = kDkDv && quarter < 2;
        const uint32_t acc = tmem + C::kColAcc + (kDkDv && !is_dv ? D : 0);
        const float f = is_dv ? kPInverse<kF16> : grad_scale<kF16>(a, p.L, ds_scale());
        const bool whole = p.slot < 0;
        const bool zero = kDkDv && p.tile * kTile + r >= p.L;
        const long long *st = kDkDv ? (is_dv ? a.dv_st : a.dk_st) : a.dq_st;
        // This lane's piece of the first of its four rows, and the rows there are.
        const int r4 = r & ~3, rows = (kDkDv ? a.Nk : a.Nq) - p.tile * kTile - r4;
        uint16_t *dst = static_cast<uint16_t *>(kDkDv ? (is_dv ? a.dv : a.dk) : a.dq) + p.b * st[0] + p.h * st[1] +
                        (static_cast<long long>(p.tile) * kTile + r4) * st[2] + (lane & 3) * 8;
        float *part = (kDkDv ? a.ws_kv : a.ws_q) +
                      ((static_cast<long long>(p.slot) * (kDkDv ? 2 : 1) + (kDkDv && !is_dv ? 1 : 0)) * kTile + r4) * D +
                      (lane & 3) * 4;
#pragma unroll 1
        for (int c = kDkDv ? quarter & 1 : quarter; c < D / 32; c += kDkDv ? 2 : 4) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(acc + c * 32, o);
            tmem_wait_ld();
            uint4 v[4];
            if (whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = zero ? 0u
                                    : pack2<kF16>(__uint_as_float(o[8 * i + 2 * j]) * f,
                                                  __uint_as_float(o[8 * i + 2 * j + 1]) * f);
                    v[i] = make_uint4(x[0], x[1], x[2], x[3]);
                }
                transpose4(v, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < rows)
                        *reinterpret_cast<uint4 *>(dst + c * 32 + j * st[2]) = v[j];
            } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = make_uint4(o[16 * half + 4 * i], o[16 * half + 4 * i + 1], o[16 * half + 4 * i + 2],
                                          o[16 * half + 4 * i + 3]);
                    transpose4(v, lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < rows)
                            *reinterpret_cast<uint4 *>(part + c * 32 + half * 16 + j * D) = v[j];
                }
            }
        }
        give_back(b, k);
        tc_fence_before();
        arrive(b.o_empty);
    }
    if (!ok)
        fail(a, b, kRoleSoftmax);
}

template <int D, bool kF16, bool kDkDv>
__global__ void __launch_bounds__(kThreads, 1)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                     const CrossBwdArgs a)
{
    using C = BCfg<D, kDkDv>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t smem = (raw + 1023u) & ~1023u;
    uint8_t *tiles = smem_raw + (smem - raw);
    BBars &b = *reinterpret_cast<BBars *>(tiles + C::kTilesBytes);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&b.res_full[i]), 1);
            mbar_init(smem_addr(&b.res_empty[i]), kDkDv ? 1 : kElemWarps);
            mbar_init(smem_addr(&b.st_full[i]), 1);
            mbar_init(smem_addr(&b.st_empty[i]), 1);
            mbar_init(smem_addr(&b.v_full[i]), 1);
            mbar_init(smem_addr(&b.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&b.s_full[i]), 1);
            mbar_init(smem_addr(&b.dp_full[i]), 1);
            mbar_init(smem_addr(&b.p1_full[i]), kElemWarps);
            mbar_init(smem_addr(&b.p_full[i]), kElemWarps);
        }
        mbar_init(smem_addr(&b.o_full), 1);
        mbar_init(smem_addr(&b.o_empty), kElemWarps);
        mbar_init(smem_addr(&b.q_full), kElemWarps);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_addr(&b.piece_full[i]), 1);
            mbar_init(smem_addr(&b.piece_empty[i]), kElemWarps + 1);
        }
        mbar_init(smem_addr(&b.drain), 1);
        b.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_addr(&b.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    if (warp == kWarpLoad && (threadIdx.x & 31) == 0) {
        prefetch_tensormap(&mq);
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
        prefetch_tensormap(&mdo);
    }
    // The kernel ahead has begun, so what it waited for is there: the lengths, and
    // for dq, behind dkdv, all that it reads; dq only ends behind dkdv.  What is
    // read without a wait of this kernel's own is read past the first-level cache.
    find_start<kDkDv>(a, b);
    if (kDkDv) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem_base;
    if (warp < kElemWarps)
        bwd_elem<D, kF16, kDkDv>(a, b, *reinterpret_cast<BXch *>(&b + 1), tiles, tmem);
    else if (warp == kWarpLoad)
        bwd_load<D, kDkDv>(a, b, smem, &mq, &mk, &mv, &mdo);
    else if (warp == kWarpMma) {
        const uint32_t lane = elected_lane();
        if (elect_one())
            bwd_mma<D, kF16, kDkDv>(a, b, smem, tmem, lane);
        __syncwarp();
    }
    if (!kDkDv) {
        grid_launch_dependents();
        grid_dependency_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) {
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ prep
constexpr int kPrepThreads = 256;
constexpr int kPrepBlocks = 760;  // at most: 5 a SM
constexpr int kPrepRows = 2;       // of a group of lanes in flight

template <bool kF16> __device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (kF16)
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// Zeros into 128 rows (as far as there are any) of a tensor's tile.
template <int kGroup, int kLanes>
__device__ __forceinline__ void zero_tile(void *t, const long long *st, int b, int h, int tile, int rows)
{
    const int part = threadIdx.x % kGroup, end = min(rows, (tile + 1) * kTile);
    for (int n = tile * kTile + threadIdx.x / kGroup; n < end; n += kPrepThreads / kGroup)
        if (part < kLanes)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(t) + b * st[0] + h * st[1] + n * st[2] + part * 8) =
                make_uint4(0, 0, 0, 0);
}

// Sums over d of 16 rows of x with 16 keys' rows of y, on the tensor cores: c[n] is rows
// lane / 4 and 8 behind it, keys 8 n + 2 (lane % 4) and the next.  The elements of a row
// may come in any order, the same for both, so a lane takes 16 bytes at a time.
template <int D, bool kF16, class X, class Y>
__device__ __forceinline__ void product16(const X &x, const Y &y, float (&c)[2][4])
{
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[n][i] = 0.f;
    auto mma = [](float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
        if constexpr (kF16)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                "{%0, %1, %2, %3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                "{%0, %1, %2, %3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    };
#pragma unroll 1
    for (int e = 0; e < D; e += 32) {
        const uint4 x0 = x(0, e), x1 = x(8, e);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const uint4 w = y(8 * n, e);
            mma(c[n], x0.x, x1.x, x0.y, x1.y, w.x, w.y);
            mma(c[n], x0.z, x1.z, x0.w, x1.w, w.z, w.w);
        }
    }
}

// D of a tile's rows of one head, which have the same few keys: a warp 16 rows.  Bound by
// reading q and dO once more: 8 sequences, 16 heads, 4096 queries, 16 keys, d = 64, bf16
// 169 us in all, 141 with D from o (with sums on the CUDA cores, a row a group of lanes,
// 351).
template <int D, bool kF16>
__device__ __forceinline__ void few_keys(const CrossBwdArgs &a, int b, int h, int tile, int L)
{
    static_assert(kFewKeys == 16 && kPrepThreads / 32 * 16 == kTile, "a product is 16 keys, a block's warps a tile");
    const int lane = threadIdx.x & 31, quad = lane / 4;
    const int row = tile * kTile + threadIdx.x / 32 * 16 + quad, piece = lane % 4 * 8;
    auto rows_of = [&](const void *p, const long long *st) {
        const uint16_t *at = static_cast<const uint16_t *>(p) + b * st[0] + h * st[1] + row * st[2] + piece;
        return [at, st, left = a.Nq - row](int r, int e) {
            return r < left ? *reinterpret_cast<const uint4 *>(at + r * st[2] + e) : make_uint4(0, 0, 0, 0);
        };
    };
    auto keys_of = [&](const void *p, const long long *st) {
        const uint16_t *at = static_cast<const uint16_t *>(p) + b * st[0] + h / a.G * st[1] + quad * st[2] + piece;
        return [at, st, left = L - quad](int j, int e) {
            return j < left ? *reinterpret_cast<const uint4 *>(at + j * st[2] + e) : make_uint4(0, 0, 0, 0);
        };
    };
    float s[2][4], dp[2][4];
    product16<D, kF16>(rows_of(a.q, a.q_st), keys_of(a.k, a.k_st), s);
    product16<D, kF16>(rows_of(a.dout, a.do_st), keys_of(a.v, a.v_st), dp);
    const long long at = (static_cast<long long>(b) * a.Hk * a.G + h) * a.Nq + row;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const bool live = row + 8 * half < a.Nq;
        const float nl2 = live ? neg_lse2<false>(a.lse[at + 8 * half]) : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = i / 2, c = 2 * half + i % 2;
            if (8 * n + lane % 4 * 2 + i % 2 < L)
                sum = fmaf(ex2(fmaf(s[n][c], a.sl2, nl2)), dp[n][c], sum);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (live && lane % 4 == 0)
            a.dfew[at + 8 * half] = sum;
    }
}

// D of all rows, a group of lanes a row (16 bytes a lane), in the order in which
// they lie in memory; in fp16 a run of a key head's rows at a time, with their norms
// and the run's largest, and the same of V's rows.  Then D of the rows with few keys,
// and zeros for what no unit covers: key tiles behind a sequence's last key (all,
// without queries) and the queries of a sequence without keys.
template <int D, bool kF16> __global__ void __launch_bounds__(kPrepThreads, 5) cross_prep_kernel(const CrossBwdArgs a)
{
    constexpr int kLanes = D / 8, kGroup = D == 64 ? 8 : 16;
    __shared__ float warp_max_of[kPrepThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, part = lane % kGroup;
    const int groups = kPrepThreads / kGroup;
    const int Hq = a.Hk * a.G;
    const long long rows = static_cast<long long>(a.B) * Hq * a.Nq;
    const bool heads_inside = a.do_st[1] < a.do_st[2];
    const bool some_few = a.kv_len != nullptr || a.Nk <= kFewKeys;  // as far as can be told
    auto block_max = [&](float x, float *to) {
        x = warp_max(x);
        if (lane == 0)
            warp_max_of[threadIdx.x / 32] = x;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kPrepThreads / 32; ++w)
                x = fmaxf(x, warp_max_of[w]);
            *to = x;
        }
        __syncthreads();
    };
    // bf16: one item a block, all rows in turns.
    const long long head_rows = static_cast<long long>(a.G) * a.Nq, per = (head_rows + a.do_parts - 1) / a.do_parts;
    const long long items = !kF16 ? gridDim.x : rows > 0 ? static_cast<long long>(a.B) * a.Hk * a.do_parts : 0;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        long long begin = item * groups, end = rows, stride = static_cast<long long>(gridDim.x) * groups, run = 0;
        int batch = 0, key_head = 0;
        if (kF16) {  // heads side by side
            const long long q1 = quotient(item, a.Hk);
            batch = static_cast<int>(quotient(q1, a.do_parts));
            key_head = static_cast<int>(item - q1 * a.Hk);
            const int c = static_cast<int>(q1 - static_cast<long long>(batch) * a.do_parts);
            run = (static_cast<long long>(batch) * a.Hk + key_head) * a.do_parts + c;
            begin = c * per;
            end = min(begin + per, head_rows);
            stride = groups;
        }
        float top = 0.f;
        for (long long row0 = begin + threadIdx.x / kGroup; row0 - threadIdx.x / kGroup < end;
             row0 += stride * kPrepRows) {
            uint4 x[kPrepRows], y[kPrepRows];
            long long to[kPrepRows];
#pragma unroll
            for (int i = 0; i < kPrepRows; ++i) {
                const long long row = row0 + i * stride;
                x[i] = y[i] = make_uint4(0, 0, 0, 0);
                to[i] = -1;
                if (row < end) {
                    const int heads = kF16 ? a.G : Hq;
                    const int inner = heads_inside ? heads : a.Nq, outer = heads_inside ? a.Nq : heads;
                    const long long q1 = quotient(row, inner), q2 = kF16 ? batch : quotient(q1, outer);
                    const int i0 = static_cast<int>(row - q1 * inner);
                    const int i1 = static_cast<int>(kF16 ? q1 : q1 - q2 * outer);
                    const int h = (heads_inside ? i0 : i1) + key_head * a.G, n = heads_inside ? i1 : i0;
                    to[i] = (q2 * Hq + h) * a.Nq + n;
                    if (part < kLanes) {
                        x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.o) + q2 * a.o_st[0] +
                                                                h * a.o_st[1] + n * a.o_st[2] + part * 8);
                        y[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.dout) +
                                                                q2 * a.do_st[0] + h * a.do_st[1] + n * a.do_st[2] +
                                                                part * 8);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kPrepRows; ++i) {
                const uint32_t xv[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, yv[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
                float acc = 0.f, squares = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = unpack2<kF16>(xv[j]), v = unpack2<kF16>(yv[j]);
                    acc = fmaf(u.x, v.x, acc);
                    acc = fmaf(u.y, v.y, acc);
                    if (kF16)
                        squares = fmaf(v.x, v.x, fmaf(v.y, v.y, squares));
                }
#pragma unroll
                for (int o = kGroup / 2; o > 0; o /= 2) {
                    acc += __shfl_xor_sync(0xffffffffu, acc, o);
                    if (kF16)
                        squares += __shfl_xor_sync(0xffffffffu, squares, o);
                }
                if (to[i] >= 0 && part == 0) {
                    a.dvec[to[i]] = acc;
                    if (kF16) {
                        const float norm = sqrtf(squares);
                        a.norms[to[i]] = norm;
                        top = fmaxf(top, norm);
                    }
                }
            }
        }
        if (kF16)
            block_max(top, a.do_max + run);
    }
    if constexpr (kF16) {
        // Rows of V before the sequence's end, runs as above, the first ones to the last
        // blocks, which have had fewer of dO's.
        const long long v_items = a.Nk > 0 ? static_cast<long long>(a.B) * a.Hk * a.v_parts : 0;
        const int v_per = (a.Nk + a.v_parts - 1) / a.v_parts;
        for (long long item = gridDim.x - 1 - blockIdx.x; item < v_items; item += gridDim.x) {
            const long long q1 = quotient(item, a.Hk);
            const int b = static_cast<int>(quotient(q1, a.v_parts)), h = static_cast<int>(item - q1 * a.Hk);
            const int c = static_cast<int>(q1 - static_cast<long long>(b) * a.v_parts);
            const long long begin = static_cast<long long>(c) * v_per;
            const long long end = min(begin + v_per, static_cast<long long>(clamp_len(a, b)));
            const uint16_t *v = static_cast<const uint16_t *>(a.v) + b * a.v_st[0] + h * a.v_st[1] + part * 8;
            float top = 0.f;
            for (long long row0 = begin + threadIdx.x / kGroup; row0 - threadIdx.x / kGroup < end; row0 += 4 * groups) {
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (row0 + i * groups < end && part < kLanes)
                        x[i] = *reinterpret_cast<const uint4 *>(v + (row0 + i * groups) * a.v_st[2]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    float squares = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<kF16>(w[j]);
                        squares = fmaf(f.x, f.x, fmaf(f.y, f.y, squares));
                    }
#pragma unroll
                    for (int o = kGroup / 2; o > 0; o /= 2)
                        squares += __shfl_xor_sync(0xffffffffu, squares, o);
                    top = fmaxf(top, sqrtf(squares));
                }
            }
            block_max(top, a.v_max + (static_cast<long long>(b) * a.Hk + h) * a.v_parts + c);
        }
    }
    if (!some_few && rows > 0)
        return;
    const int Tk = (a.Nk + kTile - 1) / kTile;
    const long long k_tiles = static_cast<long long>(a.Hk) * Tk, tiles = k_tiles + static_cast<long long>(Hq) * a.Tq;
    for (long long i = blockIdx.x; i < tiles * a.B; i += gridDim.x) {
        const int b = static_cast<int>(i / tiles), L = clamp_len(a, b);
        const long long at = i - b * tiles;
        if (at == 0 && threadIdx.x == 0 && a.kv_len != nullptr && a.kv_len[b] != L)
            atomicCAS(a.status, 0u, 6u /* FATTN_ERR_INDEX */ | (kRoleCross << 8));
        if (at < k_tiles) {
            const int h = static_cast<int>(at / Tk), tile = static_cast<int>(at - static_cast<long long>(h) * Tk);
            if (tile * kTile >= L || rows == 0) {
                zero_tile<kGroup, kLanes>(a.dk, a.dk_st, b, h, tile, a.Nk);
                zero_tile<kGroup, kLanes>(a.dv, a.dv_st, b, h, tile, a.Nk);
            }
        } else if (L <= kFewKeys) {
            const int h = static_cast<int>((at - k_tiles) / a.Tq);
            const int tile = static_cast<int>(at - k_tiles - static_cast<long long>(h) * a.Tq);
            if (L == 0)
                zero_tile<kGroup, kLanes>(a.dq, a.dq_st, b, h, tile, a.Nq);
            else
                few_keys<D, kF16>(a, b, h, tile, L);
        }
    }
}

// ------------------------------------------------------------------ merge
// Block (x, y) adds up the unit that CTA x + 1 starts inside, if that is the
// first boundary in it: the partial of CTA x (its last slot) and those of CTAs
// x + 1, x + 2, ... that start inside it.  y: dK, dV or dQ, and 32 rows of it.
constexpr int kMergeThreads = 256, kMergeRows = 32;
template <int D, bool kF16> __global__ void __launch_bounds__(kMergeThreads) cross_merge_kernel(const CrossBwdArgs a)
{
    grid_dependency_wait();
    const int which = blockIdx.y / (kTile / kMergeRows);  // 0: dV, 1: dK, 2: dQ
    const int r0 = blockIdx.y % (kTile / kMergeRows) * kMergeRows;
    const int4 *starts = a.starts + (which == 2 ? a.grid : 0);
    const int c = blockIdx.x + 1;
    const int4 me = starts[c], last = starts[c - 1];
    auto inside = [&](const int4 &s) { return s.x == me.x && s.y == me.y && s.z == me.z && s.w > 0; };
    if (me.x < 0 || me.w == 0 || inside(last))
        return;
    int count = 1;
    while (c + count < a.grid && inside(starts[c + count]))
        ++count;
    const float *ws = which == 2 ? a.ws_q : a.ws_kv;
    const int parts = which == 2 ? 1 : 2, part = which == 1 ? 1 : 0;
    const long long *st = which == 2 ? a.dq_st : which == 1 ? a.dk_st : a.dv_st;
    uint16_t *out = static_cast<uint16_t *>(which == 2 ? a.dq : which == 1 ? a.dk : a.dv);
    const int keys = clamp_len(a, me.x), rows = which == 2 ? a.Nq : a.Nk, L = which == 2 ? a.Nq : keys;
    const float *norms = a.norms + (static_cast<long long>(me.x) * a.Hk * a.G + me.y) * a.Nq;
    float scale = 1.f, v_norm = 0.f;
    if (kF16 && which != 0) {
        const long long head = static_cast<long long>(me.x) * a.Hk + (which == 1 ? me.y : me.y / a.G);
        v_norm = warp_max(lanes_max(a.v_max + head * a.v_parts, a.v_parts, threadIdx.x & 31));
        if (which == 1)
            scale = scale_of(
                warp_max(lanes_max(a.do_max + head * a.do_parts, a.do_parts, threadIdx.x & 31)) * v_norm);
    }
    constexpr int kVecs = D / 4;
    for (int at = threadIdx.x; at < kMergeRows * kVecs; at += kMergeThreads) {
        const int r = r0 + at / kVecs, v = at % kVecs, row = me.z * kTile + r;
        if (row >= rows)
            continue;
        auto slot = [&](int k) {
            const long long s = k == 0 ? 2LL * (c - 1) + 1 : 2LL * (c + k - 1);
            return reinterpret_cast<const float4 *>(ws + ((s * parts + part) * kTile + r) * D)[v];
        };
        float4 x = slot(0);
#pragma unroll 4
        for (int k = 1; k <= count; ++k) {
            const float4 y = slot(k);
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        if (kF16 && which == 2)
            scale = scale_of(norms[row] * v_norm);
        const float f = which == 0 ? kPInverse<kF16> : grad_scale<kF16>(a, keys, scale);
        const uint2 packed = row < L ? make_uint2(pack2<kF16>(x.x * f, x.y * f), pack2<kF16>(x.z * f, x.w * f))
                                     : make_uint2(0, 0);
        *reinterpret_cast<uint2 *>(out + me.x * st[0] + me.y * st[1] + row * st[2] + v * 4) = packed;
    }
}

template <class... Params, class... Args>
cudaError_t start(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                  const Args &...args)
{
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, bool kF16, bool kDkDv>
cudaError_t launch_pass(const CrossBwdArgs &a, const CrossBwdMaps &m, cudaStream_t stream)
{
    const size_t smem = BCfg<D, kDkDv>::kTilesBytes + sizeof(BBars) + (kDkDv ? sizeof(BXch) : 0) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(
        cross_bwd_kernel<D, kF16, kDkDv>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    return e != cudaSuccess ? e
                            : start(cross_bwd_kernel<D, kF16, kDkDv>, dim3(a.grid), kThreads, smem, stream, m.q,
                                    m.k, m.v, m.dout, a);
}

// Whether the units are dealt out whole, so that there is nothing to merge: where a
// unit of each pass takes no longer than the least shares and the merge, whatever the
// lengths (3 x 333 queries of 12 heads, 4 key heads, up to 501 keys, d = 64: 23.5 us,
// split and merged 28; 4 x 500 queries and keys of 16 heads, d = 128: 39.6 and 46.7).
template <int D> bool whole_units(const CrossBwdArgs &a)
{
    const long long keys = (a.Nk + kTile - 1) / kTile, queries = static_cast<long long>(a.G) * a.Tq;
    auto longer = [](long long steps) { return steps > kLeast ? steps - kLeast : 0; };
    return a.grid == 1 || longer(keys) + longer(queries) <= kMergeCost<D>;
}

template <int D, bool kF16>
cudaError_t launch(const CrossBwdArgs &args, const CrossBwdMaps &m, cudaStream_t stream)
{
    CrossBwdArgs a = args;
    constexpr int kRows = kPrepThreads / (D == 64 ? 8 : 16) * kPrepRows;  // of a block
    const long long rows = static_cast<long long>(a.B) * a.Hk * a.G * a.Nq;
    const long long blocks = (rows + kRows - 1) / kRows;
    // The zeros of short sequences, and fp16's runs, want hands, too.
    const bool most = kF16 || a.kv_len != nullptr || a.Nk == 0 || rows == 0 || blocks > kPrepBlocks;
    a.prep_blocks = most ? kPrepBlocks : static_cast<int>(blocks);
    const bool whole = whole_units<D>(a);
    a.snap = whole ? 0x7fffffff : kSnap;
    cudaError_t e = start(cross_prep_kernel<D, kF16>, dim3(a.prep_blocks), kPrepThreads, 0, stream, a);
    if (e == cudaSuccess)
        e = launch_pass<D, kF16, true>(a, m, stream);
    if (e == cudaSuccess)
        e = launch_pass<D, kF16, false>(a, m, stream);
    if (e == cudaSuccess && !whole)
        e = start(cross_merge_kernel<D, kF16>, dim3(a.grid - 1, 3 * (kTile / kMergeRows)), kMergeThreads, 0, stream,
                  a);
    return e;
}

template <int D> cudaError_t launch_typed(const CrossBwdArgs &a, const CrossBwdMaps &m, cudaStream_t stream)
{
    return a.f16 ? launch<D, true>(a, m, stream) : launch<D, false>(a, m, stream);
}

}  // namespace

CrossBwdSizes cross_bwd_sizes(int d, int num_sms)
{
    return CrossBwdSizes{2 * num_sms, 2LL * num_sms * 2 * kTile * d, 2LL * num_sms * kTile * d};
}

// A run a prep block, or where the heads alone are some hundred four, so that no round
// of the blocks is half empty; of 64 rows at least.  A warp of the passes reads one
// key head's at most 256 where its piece starts.
int cross_bwd_parts(long long heads, long long rows)
{
    const long long want = heads > 0 ? (heads > kPrepBlocks / 4 ? 4 : 1) * kPrepBlocks / heads : 1;
    return static_cast<int>(std::max(std::min({want, (rows + 63) / 64, 256LL}), 1LL));
}

cudaError_t launch_cross_bwd(const CrossBwdArgs &a, const CrossBwdMaps &m, cudaStream_t stream)
{
    switch (a.d) {
    case 64: return launch_typed<64>(a, m, stream);
    case 96: return launch_typed<96>(a, m, stream);
    case 128: return launch_typed<128>(a, m, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fattn
