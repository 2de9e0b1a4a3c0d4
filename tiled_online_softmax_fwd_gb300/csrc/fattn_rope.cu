// fattn_rope.cu -- the per-head norm and position rotation of queries and
// keys, its backward pass, and the append of rotated keys and values to a
// paged cache.
//
// With x one head's row of d elements, w the norm's weights and R(p) the
// rotation by the angles of position p (pairs (x_a, x_b) -> (x_a cos - x_b
// sin, x_b cos + x_a sin)):
//
//   forward   r = (mean x^2 + eps)^-1/2,   y = R(p) (r x w)
//   backward  g = R(p)^T dy,  dw = sum_rows g r x,
//             dx = r (g w - x r^2 mean(g w x))
//   append    k_cache[page, head, slot] = R(p) k,   v_cache[...] = v
//
// All are bound by HBM: a forward row is read and written once, some 12 flops
// an element pair.  Layout: a lane holds two 16-byte vectors of a row, a
// rotation pair's first elements and its second ones (8 lanes a row at d =
// 128), so the turn needs no exchange between lanes and one set of angles
// serves both; a warp holds 2 to 8 rows, one token each, and walks over the
// heads of its tokens, so the angles (64 bytes a lane) are read once a token,
// not once a row.  With one vector a lane, partners fetched by shuffles, the
// backward pass ran at 152 registers and issued twice the instructions: 143 us
// for B4 H16 N4096 d128 (405 MB).  Arithmetic is fp32, two elements an
// instruction, with one rounding, at the store.  A row lives in one lane group
// from load to store, so the outputs may be the inputs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>

#include "fattn_internal.h"
#include "ptx_sm103.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Residency that the registers are capped for: forward and append 5 blocks a
// SM (96 registers), backward 4 (128).
constexpr int kBlocksPerSm = 5, kBwdBlocksPerSm = 4;

template <int D> struct Geo {
    static constexpr int kLanes = D / 16;        // lanes that hold a row, two vectors each
    static constexpr int kTokens = 32 / kLanes;  // tokens (rows) a warp holds
    // d = 96: five rows of six lanes; the last two lanes hold none.
    static __device__ __forceinline__ bool in_row(int lane)
    {
        return kLanes * kTokens == 32 || lane < kLanes * kTokens;
    }
};

// Eight 16-bit elements as four fp32 pairs, and back.
using F8 = uint64_t[4];
template <bool kF16> __device__ __forceinline__ void widen(uint4 u, F8 &x)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kF16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[i] = ptx::f2_pack(f.x, f.y);
        } else {
            x[i] = ptx::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        }
    }
}
template <bool kF16> __device__ __forceinline__ uint4 narrow(const F8 &x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        ptx::f2_unpack(x[i], lo, hi);
        if constexpr (kF16) {
            const __half2 h = __floats2half2_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint64_t both(float x) { return ptx::f2_pack(x, x); }
__device__ __forceinline__ float add_pair(uint64_t x)
{
    float a, b;
    ptx::f2_unpack(x, a, b);
    return a + b;
}
__device__ __forceinline__ uint64_t swapped(uint64_t x)
{
    float a, b;
    ptx::f2_unpack(x, a, b);
    return ptx::f2_pack(b, a);
}

__device__ __forceinline__ const uint16_t *elem_ptr(const void *base, long long elem)
{
    return static_cast<const uint16_t *>(base) + elem;
}
__device__ __forceinline__ uint4 load16(const void *base, long long elem)
{
    return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + elem);
}
__device__ __forceinline__ void store16(void *base, long long elem, uint4 v)
{
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + elem) = v;
}

__device__ __forceinline__ void record_index(uint32_t *status, uint32_t role)
{
    const uint32_t code = 6u /* FATTN_ERR_INDEX */ | (role << 8) | ((blockIdx.x & 0xffffu) << 16);
    atomicCAS(status, 0u, code);
}

// The two vectors of lane `l` of a group.  rot is a multiple of 16: the first
// rot / 16 lanes hold vectors l and l + rot / 16 (half-split pairs face each
// other), the others the unturned rest in the same manner.
struct Place {
    int a, b;     // element offsets in the row
    bool turned;
};
template <int D> __device__ __forceinline__ Place place_of(int l, int rot)
{
    const int half = rot / 16, rest = D / 16 - half;
    if (l < half)
        return Place{l * 8, (l + half) * 8, true};
    return Place{(l + half) * 8, (l + half + rest) * 8, false};
}

// Factors of a lane's turn, y_a = x_a ca + o_a sa and y_b = x_b cb + o_b sb:
// half-split, o_a = x_b and o_b = x_a; neighbouring pairs, o = x with each
// pair swapped.  dir = -1 turns back.
struct Turn {
    F8 ca, sa, cb, sb;
};
template <bool kInter>
__device__ __forceinline__ void load_turn(const float *table, long long pos, int rot, Place at,
                                          float dir, Turn &t)
{
    const float *row = table + pos * rot;
    if constexpr (kInter) {
        auto one = [&](int elem, F8 &c, F8 &s) {
            const float4 cc = *reinterpret_cast<const float4 *>(row + elem / 2);
            const float4 ss = *reinterpret_cast<const float4 *>(row + rot / 2 + elem / 2);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = both(cv[i]);
                s[i] = ptx::f2_pack(-dir * sv[i], dir * sv[i]);
            }
        };
        one(at.a, t.ca, t.sa);
        one(at.b, t.cb, t.sb);
    } else {
        const float *p = row + at.a;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 cc = *reinterpret_cast<const float4 *>(p + 4 * i);
            const float4 ss = *reinterpret_cast<const float4 *>(p + rot / 2 + 4 * i);
            t.ca[2 * i] = t.cb[2 * i] = ptx::f2_pack(cc.x, cc.y);
            t.ca[2 * i + 1] = t.cb[2 * i + 1] = ptx::f2_pack(cc.z, cc.w);
            t.sa[2 * i] = ptx::f2_pack(-dir * ss.x, -dir * ss.y);
            t.sa[2 * i + 1] = ptx::f2_pack(-dir * ss.z, -dir * ss.w);
            t.sb[2 * i] = ptx::f2_pack(dir * ss.x, dir * ss.y);
            t.sb[2 * i + 1] = ptx::f2_pack(dir * ss.z, dir * ss.w);
        }
    }
}
template <bool kInter> __device__ __forceinline__ void turn(const Turn &t, F8 &a, F8 &b)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t oa = kInter ? swapped(a[i]) : b[i], ob = kInter ? swapped(b[i]) : a[i];
        const uint64_t ya = ptx::f2_fma(oa, t.sa[i], ptx::f2_mul(a[i], t.ca[i]));
        b[i] = ptx::f2_fma(ob, t.sb[i], ptx::f2_mul(b[i], t.cb[i]));
        a[i] = ya;
    }
}

// Sum over the lanes of a row, on each of them.
template <int kLanes> __device__ __forceinline__ float group_sum(float x)
{
    if constexpr (kLanes == 6) {
        const int lane = threadIdx.x & 31, l = lane % 6, base = lane - l;
        x += __shfl_sync(0xffffffffu, x, base + (l + 3) % 6);
        return x + __shfl_sync(0xffffffffu, x, base + (l + 1) % 6) +
               __shfl_sync(0xffffffffu, x, base + (l + 2) % 6);
    } else {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2)
            x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
}
// Sum over the warp's rows, on the lanes of the first.
template <int D> __device__ __forceinline__ float row_total(float x)
{
    constexpr int kLanes = Geo<D>::kLanes;
    float sum = x;
#pragma unroll
    for (int g = 1; g < Geo<D>::kTokens; ++g)
        sum += __shfl_down_sync(0xffffffffu, x, g * kLanes);
    return sum;
}

// A lane's token in block `block` of kTokens consecutive tokens (of the
// flattened batch).
struct Item {
    int b, n;
    long long pos;
    bool live;  // the token exists, and has a position in the table
};
template <int D>
__device__ __forceinline__ Item item_at(const NormRopeArgs &a, int block, int lane)
{
    Item x;
    const unsigned tok = static_cast<unsigned>(block) * Geo<D>::kTokens + lane / Geo<D>::kLanes;
    x.live = tok < static_cast<unsigned>(a.tokens) && Geo<D>::in_row(lane);
    const unsigned b = x.live ? tok / static_cast<unsigned>(a.N) : 0u;
    x.b = static_cast<int>(b);
    x.n = x.live ? static_cast<int>(tok - b * static_cast<unsigned>(a.N)) : 0;
    x.pos = 0;
    if (x.live && a.rot > 0) {
        x.pos = a.positions != nullptr ? a.positions[tok] : x.n;
        if (x.pos < 0 || x.pos >= a.max_pos) {
            x.live = false;
            if (lane % Geo<D>::kLanes == 0)
                record_index(a.status, kRoleRotate);
        }
    }
    return x;
}
__device__ __forceinline__ long long row_at(const long long (&st)[3], const Item &x)
{
    return x.b * st[0] + x.n * st[2];
}

// ------------------------------------------------------------------ forward
// B4 H16 N4096 d128, q and k (268 MB): 44 us, 6.2 TB/s; a decode step's 16
// tokens 3.3 us in a graph.
template <int D, bool kF16, bool kInter>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_rope_kernel(const NormRopeArgs a)
{
    using G = Geo<D>;
    constexpr int kBatch = 4;  // rows in flight a lane group
    const int lane = threadIdx.x & 31;
    long long it = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (it >= a.items[0] + a.items[1])
        return;
    const int w = it < a.items[0] ? 0 : 1;
    it -= w == 0 ? 0 : a.items[0];
    const int block = static_cast<int>(it / a.chunks[w]);
    const int chunk = static_cast<int>(it - static_cast<long long>(block) * a.chunks[w]);
    const int h0 = chunk * a.heads_per_chunk, h1 = min(h0 + a.heads_per_chunk, a.H[w]);
    const Item x = item_at<D>(a, block, lane);
    const Place at = place_of<D>(lane % G::kLanes, a.rot);
    const uint16_t *x_at = elem_ptr(a.x[w], row_at(a.x_st[w], x) + h0 * a.x_st[w][1]);
    uint16_t *y_at = static_cast<uint16_t *>(a.y[w]) + row_at(a.y_st[w], x) + h0 * a.y_st[w][1];
    const long long x_step = a.x_st[w][1], y_step = a.y_st[w][1];
    const bool norm = a.w[w] != nullptr;
    // The weights are folded into the turn: y_a = r (x_a ca w_a + o_a sa w_o).
    Turn t;
    if (x.live) {
        if (at.turned) {
            load_turn<kInter>(a.table, x.pos, a.rot, at, 1.f, t);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t.ca[i] = t.cb[i] = both(1.f);
        }
        if (norm) {
            F8 wa, wb;
            widen<kF16>(load16(a.w[w], at.a), wa);
            widen<kF16>(load16(a.w[w], at.b), wb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                t.ca[i] = ptx::f2_mul(t.ca[i], wa[i]);
                t.cb[i] = ptx::f2_mul(t.cb[i], wb[i]);
                t.sa[i] = ptx::f2_mul(t.sa[i], kInter ? swapped(wa[i]) : wb[i]);
                t.sb[i] = ptx::f2_mul(t.sb[i], kInter ? swapped(wb[i]) : wa[i]);
            }
        }
    }
    for (int h = h0; h < h1; h += kBatch) {
        uint4 u[kBatch][2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            u[k][0] = u[k][1] = make_uint4(0, 0, 0, 0);
            if (x.live && h + k < h1) {
                u[k][0] = load16(x_at, at.a);
                u[k][1] = load16(x_at, at.b);
                x_at += x_step;
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            F8 xa, xb;
            widen<kF16>(u[k][0], xa);
            widen<kF16>(u[k][1], xb);
            uint64_t r = both(1.f);
            if (norm) {
                uint64_t ss = ptx::f2_mul(xa[0], xa[0]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i > 0)
                        ss = ptx::f2_fma(i < 4 ? xa[i] : xb[i - 4], i < 4 ? xa[i] : xb[i - 4], ss);
                r = both(rsqrtf(group_sum<G::kLanes>(add_pair(ss)) * (1.f / D) + a.eps));
            }
            if (at.turned) {
                turn<kInter>(t, xa, xb);
            } else if (norm) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xa[i] = ptx::f2_mul(xa[i], t.ca[i]);
                    xb[i] = ptx::f2_mul(xb[i], t.cb[i]);
                }
            }
            if (norm) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xa[i] = ptx::f2_mul(xa[i], r);
                    xb[i] = ptx::f2_mul(xb[i], r);
                }
            }
            if (x.live && h + k < h1) {
                store16(y_at, at.a, narrow<kF16>(xa));
                store16(y_at, at.b, narrow<kF16>(xb));
                y_at += y_step;
            }
        }
    }
}

// ------------------------------------------------------------------ backward
// A persistent grid, its first blocks for q and the others for k in the ratio
// of their rows, and each warp with one of equal runs of the tensor's (block of
// tokens, head) rows, in that order.  With items of 8 heads dealt in turn the
// slowest warp had 10 % more than the mean: B3 H32/4 N4096 d96 took 54 us, now
// 51 (5.0 TB/s).  Every warp keeps the weight gradients of its rows in
// registers (fp32), the block adds its warps' sums in a fixed order and writes
// one partial; dw_reduce_kernel adds those, also in a fixed order, so equal
// calls give equal bits.
//
// A row's two reductions stand between its loads and its stores, and with the
// rows in flight held in registers (two a lane group) a warp spent most of its
// time waiting: 80 us for B4 H16 N4096 d128.  So each lane copies its own
// vectors ahead into its own shared-memory slots (cp.async, no barrier: nobody
// else reads them), across the ends of blocks, and its addresses step from head
// to head: 65.5 us, 6.2 TB/s.  A ring of 3 rows; with 4 and 5 it was 66 and 69.
constexpr int kRing = 3;
// Rows of a warp where there are few: 1021 tokens of 24 and 6 heads, d = 64,
// take 6.9 us with 3 rows, 7.7 with 2 and 8.1 with 4.
constexpr int kMinRows = 3;

__device__ __forceinline__ void copy_ahead(uint32_t dst, const void *src, bool live)
{
    // Zero bytes read fill the slot with zeros.
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}

template <int D, bool kF16, bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm) norm_rope_bwd_kernel(const NormRopeArgs a)
{
    using G = Geo<D>;
    __shared__ uint4 ring[kRing][kWarps][4][32];  // g_a, g_b, x_a, x_b of each lane
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const Place at = place_of<D>(lane % G::kLanes, a.rot);
    const int w = static_cast<int>(blockIdx.x) < a.blocks[0] ? 0 : 1;
    const int block = w == 0 ? blockIdx.x : blockIdx.x - a.blocks[0];
    // This warp's rows: the first rows_over warps have one more than the others.
    const int self = block * kWarps + warp, over = a.rows_over[w];
    const long long row0 = self * a.rows_each[w] + min(self, over);
    const bool norm = a.w[w] != nullptr, in_row = G::in_row(lane);
    F8 wa, wb, acc_a, acc_b;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        wa[i] = wb[i] = acc_a[i] = acc_b[i] = both(0.f);
    if (norm && in_row) {
        widen<kF16>(load16(a.w[w], at.a), wa);
        widen<kF16>(load16(a.w[w], at.b), wb);
    }
    // Two walks over the rows: `ahead` copies, `now` computes.
    struct Walk {
        int blk, head, left, rest;  // rows left in this block of tokens, and behind it
        Item x;
    };
    auto enter = [&](Walk &k) {
        k.left = min(a.H[w] - k.head, k.rest);
        k.rest -= k.left;
        if (k.left > 0)
            k.x = item_at<D>(a, k.blk, lane);
    };
    auto next_block = [&](Walk &k) {
        ++k.blk;
        k.head = 0;
        enter(k);
    };
    Walk ahead, now;
    const unsigned H = static_cast<unsigned>(a.H[w]);
    ahead.blk = static_cast<int>(row0 >> 32 == 0 ? static_cast<unsigned>(row0) / H : row0 / H);
    ahead.head = static_cast<int>(row0 - static_cast<long long>(ahead.blk) * H);
    ahead.rest = static_cast<int>(a.rows_each[w]) + (self < over ? 1 : 0);
    enter(ahead);
    now = ahead;
    // Where the copies read: stepped from head to head.  A lane without a row
    // stays at the tensor's base, of which it reads nothing.
    const uint16_t *g_at, *x_at;
    long long g_step, x_step;
    auto point = [&]() {
        if (ahead.left == 0)
            return;
        const bool live = ahead.x.live;
        g_at = elem_ptr(a.g[w], live ? row_at(a.g_st[w], ahead.x) + ahead.head * a.g_st[w][1] + at.a : 0);
        g_step = live ? a.g_st[w][1] : 0;
        if (norm) {
            x_at = elem_ptr(a.x[w], live ? row_at(a.x_st[w], ahead.x) + ahead.head * a.x_st[w][1] + at.a : 0);
            x_step = live ? a.x_st[w][1] : 0;
        }
    };
    point();
    const int b_off = in_row ? at.b - at.a : 0;
    const uint32_t ring0 = ptx::smem_addr(&ring[0][warp][0][lane]);
    constexpr uint32_t kSlot = sizeof(ring[0]);
    uint32_t put = ring0;
    int get = 0;
    auto copy_row = [&]() {
        if (ahead.left > 0) {
            const bool live = ahead.x.live;
            copy_ahead(put, g_at, live);
            copy_ahead(put + 512, g_at + b_off, live);
            g_at += g_step;
            if (norm) {
                copy_ahead(put + 1024, x_at, live);
                copy_ahead(put + 1536, x_at + b_off, live);
                x_at += x_step;
            }
            put = put == ring0 + (kRing - 1) * kSlot ? ring0 : put + kSlot;
            if (--ahead.left == 0) {
                next_block(ahead);
                point();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kRing - 1; ++i)
        copy_row();
    while (now.left > 0) {
        const bool live = now.x.live;
        uint16_t *y_at = static_cast<uint16_t *>(a.y[w]) + row_at(a.y_st[w], now.x) +
                         now.head * a.y_st[w][1] + at.a;
        Turn t;
        if (live && at.turned)
            load_turn<kInter>(a.table, now.x.pos, a.rot, at, -1.f, t);
#pragma unroll 1
        for (; now.left > 0; --now.left) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            const uint4(&slot)[4][32] = ring[get][warp];
            F8 ga, gb;
            widen<kF16>(slot[0][lane], ga);
            widen<kF16>(slot[1][lane], gb);
            if (at.turned && live)
                turn<kInter>(t, ga, gb);
            if (norm) {
                F8 xa, xb;
                widen<kF16>(slot[2][lane], xa);
                widen<kF16>(slot[3][lane], xb);
                uint64_t ss = both(0.f), gx = both(0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ss = ptx::f2_fma(xa[i], xa[i], ss);
                    gx = ptx::f2_fma(ptx::f2_mul(ga[i], wa[i]), xa[i], gx);
                    ss = ptx::f2_fma(xb[i], xb[i], ss);
                    gx = ptx::f2_fma(ptx::f2_mul(gb[i], wb[i]), xb[i], gx);
                }
                const float r = rsqrtf(group_sum<G::kLanes>(add_pair(ss)) * (1.f / D) + a.eps);
                const float m = group_sum<G::kLanes>(add_pair(gx)) * (1.f / D) * r * r;
                const uint64_t rr = both(r), mr = both(-m * r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t ra = ptx::f2_mul(ga[i], rr), rb = ptx::f2_mul(gb[i], rr);
                    acc_a[i] = ptx::f2_fma(ra, xa[i], acc_a[i]);
                    acc_b[i] = ptx::f2_fma(rb, xb[i], acc_b[i]);
                    ga[i] = ptx::f2_fma(ra, wa[i], ptx::f2_mul(xa[i], mr));
                    gb[i] = ptx::f2_fma(rb, wb[i], ptx::f2_mul(xb[i], mr));
                }
            }
            if (live) {
                store16(y_at, 0, narrow<kF16>(ga));
                store16(y_at, b_off, narrow<kF16>(gb));
                y_at += a.y_st[w][1];
            }
            get = get + 1 == kRing ? 0 : get + 1;
            copy_row();
        }
        next_block(now);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!norm)  // no weights: nothing to sum
        return;
    // Groups of the warp, then the block's warps (the ring's memory is free).
    float(&part)[kWarps][D] = *reinterpret_cast<float(*)[kWarps][D]>(ring);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float lo, hi;
        ptx::f2_unpack(i < 4 ? acc_a[i] : acc_b[i - 4], lo, hi);
        lo = row_total<D>(lo);
        hi = row_total<D>(hi);
        if (lane < G::kLanes) {
            float *dst = &part[warp][(i < 4 ? at.a : at.b) + 2 * (i % 4)];
            dst[0] = lo;
            dst[1] = hi;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            x += part[k][i];
        a.partial[static_cast<size_t>(blockIdx.x) * D + i] = x;
    }
}

// dw[t][c] = sum over the partials of tensor t's blocks, kept to twice fp32's
// length by carrying each addition's rounding error along (Knuth's two-sum);
// fp64 additions, at this chip's rate, took 8 to 14 us here.  Eight columns a
// CTA, 32 rows of threads over the blocks.
constexpr int kReduceRows = 32, kReduceCols = 8;
struct Sum2 {
    float s = 0.f, e = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = s + x, z = t - s;
        e += (s - (t - z)) + (x - z);
        s = t;
    }
};
__global__ void __launch_bounds__(kReduceCols *kReduceRows)
    dw_reduce_kernel(const float *partial, int q_blocks, int k_blocks, int D, float *dwq, float *dwk)
{
    __shared__ float2 part[kReduceRows][kReduceCols];
    const int t = blockIdx.x * kReduceCols >= D ? 1 : 0;
    const int col = blockIdx.x * kReduceCols - t * D + threadIdx.x;
    float *dst = t == 0 ? dwq : dwk;
    ptx::grid_dependency_wait();  // before any way out: what follows this grid relies on it
    if (dst == nullptr)
        return;
    const int b0 = t == 0 ? 0 : q_blocks, b1 = t == 0 ? q_blocks : q_blocks + k_blocks;
    Sum2 x;
#pragma unroll 8
    for (int b = b0 + threadIdx.y; b < b1; b += kReduceRows)
        x.add(partial[static_cast<size_t>(b) * D + col]);
    part[threadIdx.y][threadIdx.x] = make_float2(x.s, x.e);
    __syncthreads();
    if (threadIdx.y != 0)
        return;
    x = Sum2();
#pragma unroll
    for (int r = 0; r < kReduceRows; ++r) {
        x.add(part[r][threadIdx.x].x);
        x.e += part[r][threadIdx.x].y;
    }
    dst[col] = x.s + x.e;
}

// ------------------------------------------------------------------ append
// Whether cu_q is not a list of starts: from 0, none before the one ahead of
// it, the last within the tokens.  Each thread's share of it.
__device__ __forceinline__ bool list_is_bad(const int *cu, int B, long long T)
{
    bool bad = false;
    for (int i = threadIdx.x; i <= B; i += kThreads) {
        const int at = cu[i];
        bad = bad || (i == 0 ? at != 0 : at < cu[i - 1]) || at > T;
    }
    return bad;
}

// The largest b in [0, B] with cu[b] <= t (-1: none), found by the lanes of a
// group together: each step cuts the range into kLanes parts, so 256
// sequences take two dependent loads where halving takes eight.  The number
// of steps depends on B alone, so the groups of a warp stay together.  In a
// list out of order it ends at some entry, or none: list_is_bad reports that.
template <int kLanes>
__device__ __forceinline__ int find_sequence(const int *cu, int B, long long t, int v, int base)
{
    int lo = 0, n = B + 1;
    bool none = false;
    do {
        const int step = (n + kLanes - 1) / kLanes;
        const int i = lo + v * step;
        const bool below = v * step < n && i <= B && cu[i] <= t;
        const unsigned all = __ballot_sync(0xffffffffu, below);
        const unsigned mine = (all >> base) & (0xffffffffu >> (32 - kLanes));
        none = none || mine == 0;
        lo += none ? 0 : (31 - __clz(mine)) * step;
        n = step;
    } while (n > 1);
    return none ? -1 : lo;
}

// Token t = cu_q[b] + i of sequence b goes to position kv_len[b] - (new
// tokens of b) + i of its pages, a key turned by that position's angles.  24
// prompts of 500 to 4096 tokens, 8 heads, d = 128 (483 MB): 69 us, 7.0 TB/s; 64
// single tokens 3.1 us in a graph (3.0 without the block for the list).
template <int D, bool kF16, bool kInter>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) kv_append_kernel(const KvAppendArgs a)
{
    using G = Geo<D>;
    constexpr int kBatch = 4;
    const int lane = threadIdx.x & 31, l = lane % G::kLanes, base = lane - l;
    // The last block looks the list over, beside the others: a search finds no
    // sequence for some tokens of a list out of order, as for padding.
    if (blockIdx.x == gridDim.x - 1) {
        if (list_is_bad(a.cu_q, a.B, a.T))
            record_index(a.status, kRoleAppend);
        return;
    }
    const long long it = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (it >= a.items)
        return;
    // Items: for each block of tokens its chunks of key heads, then of value heads.
    const long long blk = it / (2 * a.chunks);
    int c = static_cast<int>(it - blk * 2 * a.chunks);
    const bool is_v = c >= a.chunks;
    if (is_v)
        c -= a.chunks;
    const int h0 = c * a.heads_per_chunk, h1 = min(h0 + a.heads_per_chunk, a.H);
    const long long tok = blk * G::kTokens + lane / G::kLanes;
    const bool exists = tok < a.T && G::in_row(lane);
    const Place at = place_of<D>(l, is_v ? 0 : a.rot);
    const void *src = is_v ? a.v : a.k;
    const long long tok_stride = is_v ? a.v_st[0] : a.k_st[0];
    const long long head_stride = is_v ? a.v_st[1] : a.k_st[1];
    const long long in0 = (exists ? tok : 0) * tok_stride;
    // The rows do not depend on where they go: the first batch is in flight
    // while the token's sequence, page and angles are looked up.
    uint4 u[kBatch][2];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            u[k][0] = u[k][1] = make_uint4(0, 0, 0, 0);
            if (exists && h + k < h1) {
                const long long row = in0 + (h + k) * head_stride;
                u[k][0] = load16(src, row + at.a);
                u[k][1] = load16(src, row + at.b);
            }
        }
    };
    load(h0);
    bool live = exists, bad = false;
    const int b = find_sequence<G::kLanes>(a.cu_q, a.B, tok, l, base);
    long long pos = 0, out0 = 0;
    if (live && b >= 0 && b < a.B) {
        const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
        pos = static_cast<long long>(a.kv_len[b]) - q1 + tok;
        const long long col = pos >> a.page_shift;
        bad = q0 < 0 || q1 > a.T || tok >= q1 || pos < 0 || col >= a.max_pages ||
              (a.rot > 0 && pos >= a.max_pos);
        if (!bad) {
            const int page = a.page_table[static_cast<long long>(b) * a.table_stride + col];
            bad = page < 0 || page >= a.num_pages;
            const long long slot = pos & ((1LL << a.page_shift) - 1);
            out0 = is_v ? a.vc_st[0] * page + a.vc_st[2] * slot
                        : a.kc_st[0] * page + a.kc_st[2] * slot;
        }
        if (bad && l == 0 && h0 == 0 && !is_v)
            record_index(a.status, kRoleAppend);
        live = !bad;
    } else {
        live = false;  // behind the last sequence (or before the first)
    }
    void *dst = is_v ? a.v_cache : a.k_cache;
    const long long out_head = is_v ? a.vc_st[1] : a.kc_st[1];
    Turn t;
    if (live && at.turned)
        load_turn<kInter>(a.table, pos, a.rot, at, 1.f, t);
    for (int h = h0;;) {
        if (live) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (at.turned) {  // unturned elements keep their bits
                    F8 xa, xb;
                    widen<kF16>(u[k][0], xa);
                    widen<kF16>(u[k][1], xb);
                    turn<kInter>(t, xa, xb);
                    u[k][0] = narrow<kF16>(xa);
                    u[k][1] = narrow<kF16>(xb);
                }
                if (h + k < h1) {
                    const long long row = out0 + (h + k) * out_head;
                    store16(dst, row + at.a, u[k][0]);
                    store16(dst, row + at.b, u[k][1]);
                }
            }
        }
        h += kBatch;
        if (h >= h1)
            break;
        load(h);
    }
}

// Heads an item: enough items to give every SM kItemsPerSm warps, at least
// kMinHeads heads each.  More heads an item read the angles less often.
constexpr int kItemsPerSm = 64, kMinHeads = 4;
int heads_per_item(long long token_blocks, int heads, int num_sms)
{
    const long long want = static_cast<long long>(num_sms) * kItemsPerSm;
    int n = kMinHeads;
    while (n < heads && token_blocks * ((heads + 2 * n - 1) / (2 * n)) >= want)
        n *= 2;
    return n;
}

template <int D, bool kF16, bool kInter>
cudaError_t norm_rope(NormRopeArgs a, int num_sms, cudaStream_t stream)
{
    const long long blocks = (a.tokens + Geo<D>::kTokens - 1) / Geo<D>::kTokens;
    if (a.g[0] == nullptr && a.g[1] == nullptr) {
        a.heads_per_chunk = heads_per_item(blocks, a.H[0] + a.H[1], num_sms);
        for (int t = 0; t < 2; ++t) {
            a.chunks[t] = (a.H[t] + a.heads_per_chunk - 1) / a.heads_per_chunk;
            a.items[t] = blocks * a.chunks[t];
        }
        const long long grid = (a.items[0] + a.items[1] + kWarps - 1) / kWarps;
        if (grid > 0x7fffffffLL)
            return cudaErrorInvalidConfiguration;
        norm_rope_kernel<D, kF16, kInter><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    // kMinRows rows a warp while all blocks fit on the SMs, else the SMs' blocks
    // in the ratio of the rows, each tensor at least one.
    long long need[2];
    for (int t = 0; t < 2; ++t) {
        a.items[t] = blocks * a.H[t];
        need[t] = (a.items[t] + kWarps * kMinRows - 1) / (kWarps * kMinRows);
    }
    const int all = norm_rope_bwd_blocks(num_sms);
    if (need[0] + need[1] <= all) {
        a.blocks[0] = static_cast<int>(need[0]);
        a.blocks[1] = static_cast<int>(need[1]);
    } else {
        const long long q = (static_cast<long long>(all) * a.H[0] + (a.H[0] + a.H[1]) / 2) /
                            (static_cast<long long>(a.H[0]) + a.H[1]);
        a.blocks[0] = static_cast<int>(a.H[0] == 0 ? 0 : a.H[1] == 0 ? all : q < 1 ? 1 : q > all - 1 ? all - 1 : q);
        a.blocks[1] = all - a.blocks[0];
    }
    for (int t = 0; t < 2; ++t) {
        const int warps = std::max(a.blocks[t] * kWarps, 1);
        a.rows_each[t] = a.items[t] / warps;
        a.rows_over[t] = static_cast<int>(a.items[t] - a.rows_each[t] * warps);
    }
    const int grid = a.blocks[0] + a.blocks[1];
    norm_rope_bwd_kernel<D, kF16, kInter><<<grid, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.partial == nullptr)
        return e;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * D / kReduceCols);
    cfg.blockDim = dim3(kReduceCols, kReduceRows);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dw_reduce_kernel, static_cast<const float *>(a.partial),
                              a.blocks[0], a.blocks[1], D, a.dw[0], a.dw[1]);
}

template <int D, bool kF16, bool kInter>
cudaError_t kv_append(KvAppendArgs a, int num_sms, cudaStream_t stream)
{
    const long long blocks = (static_cast<long long>(a.T) + Geo<D>::kTokens - 1) / Geo<D>::kTokens;
    a.heads_per_chunk = heads_per_item(2 * blocks, a.H, num_sms);
    a.chunks = (a.H + a.heads_per_chunk - 1) / a.heads_per_chunk;
    a.items = blocks * 2 * a.chunks;
    const long long grid = (a.items + kWarps - 1) / kWarps + 1;
    if (grid > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    kv_append_kernel<D, kF16, kInter><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D> cudaError_t norm_rope_typed(const NormRopeArgs &a, int num_sms, cudaStream_t stream)
{
    if (a.f16)
        return a.interleaved ? norm_rope<D, true, true>(a, num_sms, stream)
                             : norm_rope<D, true, false>(a, num_sms, stream);
    return a.interleaved ? norm_rope<D, false, true>(a, num_sms, stream)
                         : norm_rope<D, false, false>(a, num_sms, stream);
}
template <int D> cudaError_t kv_append_typed(const KvAppendArgs &a, int num_sms, cudaStream_t stream)
{
    if (a.f16)
        return a.interleaved ? kv_append<D, true, true>(a, num_sms, stream)
                             : kv_append<D, true, false>(a, num_sms, stream);
    return a.interleaved ? kv_append<D, false, true>(a, num_sms, stream)
                         : kv_append<D, false, false>(a, num_sms, stream);
}

}  // namespace

int norm_rope_bwd_blocks(int num_sms) { return kBwdBlocksPerSm * num_sms; }

cudaError_t launch_norm_rope(const NormRopeArgs &a, int num_sms, cudaStream_t stream)
{
    switch (a.d) {
    case 64: return norm_rope_typed<64>(a, num_sms, stream);
    case 96: return norm_rope_typed<96>(a, num_sms, stream);
    case 128: return norm_rope_typed<128>(a, num_sms, stream);
    case 256: return norm_rope_typed<256>(a, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, cudaStream_t stream)
{
    switch (a.d) {
    case 64: return kv_append_typed<64>(a, num_sms, stream);
    case 96: return kv_append_typed<96>(a, num_sms, stream);
    case 128: return kv_append_typed<128>(a, num_sms, stream);
    case 256: return kv_append_typed<256>(a, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fattn
