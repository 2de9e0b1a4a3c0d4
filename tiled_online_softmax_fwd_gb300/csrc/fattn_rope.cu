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
// All are bound by HBM: a forward row is read and written once, 12 flops an
// element pair.  Layout: a row's 16-byte vectors sit on consecutive lanes (8
// lanes for d = 64, 16 for 96 and 128, 32 for 256), so a warp holds 1 to 4
// rows, one token each, and walks over the heads of its tokens: the angles
// (64 bytes a lane, four times the row's own 16) are read once a token, not
// once a row.  A row's rotation partner is d-dependent lanes away and comes
// by shuffles of the packed 16-bit words, before any arithmetic.  A row lives
// in one lane group from load to store, so the outputs may be the inputs.
// Arithmetic is fp32 with one rounding, at the store.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fattn_internal.h"
#include "ptx_sm103.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Rows in flight per lane group: four 16-byte loads a lane, issued together.
constexpr int kBatch = 4;

template <int D> struct Geo {
    static constexpr int kVecs = D / 8;  // 16-byte vectors of a row
    static constexpr int kLanes = D == 64 ? 8 : D == 256 ? 32 : 16;
    static constexpr int kTokens = 32 / kLanes;  // tokens (rows) a warp holds
};

template <bool kF16> __device__ __forceinline__ float2 widen(uint32_t w)
{
    if constexpr (kF16) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}

template <bool kF16> __device__ __forceinline__ uint32_t narrow(float lo, float hi)
{
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool kF16> __device__ __forceinline__ void widen8(uint4 u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = widen<kF16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <bool kF16> __device__ __forceinline__ uint4 narrow8(const float (&x)[8])
{
    return make_uint4(narrow<kF16>(x[0], x[1]), narrow<kF16>(x[2], x[3]),
                      narrow<kF16>(x[4], x[5]), narrow<kF16>(x[6], x[7]));
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

// Where a lane's vector v takes its rotation partner from.  rot is a multiple
// of 16, so both halves of a half-split row are whole vectors.
struct Partner {
    int vec;     // vector that holds the partners (v itself: none, or in the vector)
    float sign;  // of the partner's sine term: -1 first of a pair, +1 second, 0 not rotated
};
__device__ __forceinline__ Partner partner_of(int v, int rot, int interleaved)
{
    const int half = rot / 16;
    if (v >= 2 * half)
        return Partner{v, 0.f};
    if (interleaved)
        return Partner{v, 1.f};  // the sign alternates inside the vector
    return v < half ? Partner{v + half, -1.f} : Partner{v - half, 1.f};
}

// Cosines and signed sines for the 8 elements of vector v at position pos:
// forward y = x cos + x_partner sin_signed.
__device__ __forceinline__ void load_angles(const float *table, long long pos, int v, int rot,
                                            int interleaved, Partner pr, float (&c)[8],
                                            float (&s)[8])
{
    if (pr.sign == 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        return;
    }
    const float *row = table + pos * rot;
    if (interleaved) {
        const float4 cc = *reinterpret_cast<const float4 *>(row + v * 4);
        const float4 ss = *reinterpret_cast<const float4 *>(row + rot / 2 + v * 4);
        const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[2 * i] = c[2 * i + 1] = cv[i];
            s[2 * i] = -sv[i];
            s[2 * i + 1] = sv[i];
        }
    } else {
        const float *p = row + min(v, pr.vec) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 cc = *reinterpret_cast<const float4 *>(p + 4 * i);
            const float4 ss = *reinterpret_cast<const float4 *>(p + rot / 2 + 4 * i);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c[4 * i + k] = cv[k];
                s[4 * i + k] = pr.sign * sv[k];
            }
        }
    }
}

// The partner elements of a lane's vector: another lane's words, or for
// neighbouring pairs the vector's own with each pair swapped.
__device__ __forceinline__ uint4 partner_words(uint4 u, int src_lane, int interleaved)
{
    if (interleaved)
        return make_uint4(__funnelshift_l(u.x, u.x, 16), __funnelshift_l(u.y, u.y, 16),
                          __funnelshift_l(u.z, u.z, 16), __funnelshift_l(u.w, u.w, 16));
    return make_uint4(__shfl_sync(0xffffffffu, u.x, src_lane), __shfl_sync(0xffffffffu, u.y, src_lane),
                      __shfl_sync(0xffffffffu, u.z, src_lane), __shfl_sync(0xffffffffu, u.w, src_lane));
}

template <int kLanes> __device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = kLanes / 2; o > 0; o /= 2)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One tensor of a norm call: its rows and their layout (batch, head, token
// strides in elements).
__device__ __forceinline__ long long row_at(const long long (&st)[3], int b, int h, int n)
{
    return b * st[0] + h * st[1] + n * st[2];
}

// A warp's work: kTokens consecutive tokens (of the flattened batch) and a
// run of heads of q (which = 0) or k (which = 1).
struct Item {
    int which, h0, h1;
    long long tok0;
};
__device__ __forceinline__ Item item_at(const NormRopeArgs &a, long long it, int tokens)
{
    Item x;
    const int chunks = a.chunks[0] + a.chunks[1];
    const long long blk = it / chunks;
    int c = static_cast<int>(it - blk * chunks);
    x.which = c >= a.chunks[0] ? 1 : 0;
    if (x.which)
        c -= a.chunks[0];
    x.h0 = c * a.heads_per_chunk;
    x.h1 = min(x.h0 + a.heads_per_chunk, a.H[x.which]);
    x.tok0 = blk * tokens;
    return x;
}

// Position of a token; false where it has none in the table.
__device__ __forceinline__ bool position_of(const NormRopeArgs &a, long long tok, int n, long long &pos)
{
    pos = 0;
    if (a.rot == 0)
        return true;
    pos = a.positions != nullptr ? a.positions[tok] : n;
    return pos >= 0 && pos < a.max_pos;
}

// ------------------------------------------------------------------ forward
template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a)
{
    using G = Geo<D>;
    const int lane = threadIdx.x & 31, v = lane % G::kLanes, base = lane - v;
    const long long it = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (it >= a.items)
        return;
    const Item item = item_at(a, it, G::kTokens);
    const int w = item.which;
    const long long tok = item.tok0 + lane / G::kLanes;
    const bool in_row = v < G::kVecs;  // d = 96: lanes 12-15 of a group idle
    bool live = tok < a.tokens;
    const int b = live ? static_cast<int>(tok / a.N) : 0;
    const int n = live ? static_cast<int>(tok - static_cast<long long>(b) * a.N) : 0;
    long long pos;
    if (live && !position_of(a, tok, n, pos)) {
        live = false;
        if (v == 0 && item.h0 == 0)
            record_index(a.status, kRoleRotate);
    }
    live = live && in_row;
    const void *src = a.x[w];
    void *dst = a.y[w];
    const long long in0 = row_at(a.x_st[w], b, 0, n) + v * 8;
    const long long out0 = row_at(a.y_st[w], b, 0, n) + v * 8;
    // y = r (x ca + x_partner sb), the weights folded into the angles.
    float ca[8], sb[8];
    const Partner pr = partner_of(v, a.rot, a.interleaved);
    const bool norm = a.w[w] != nullptr;
    if (live) {
        load_angles(a.table, pos, v, a.rot, a.interleaved, pr, ca, sb);
        if (norm) {
            float own[8], other[8];
            const uint4 wo = load16(a.w[w], v * 8);
            widen8<kF16>(wo, own);
            widen8<kF16>(a.interleaved ? partner_words(wo, 0, 1) : load16(a.w[w], pr.vec * 8), other);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ca[i] *= own[i];
                sb[i] *= other[i];
            }
        }
    }
    const int src_lane = base + pr.vec;
    for (int h = item.h0; h < item.h1; h += kBatch) {
        uint4 u[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            u[k] = make_uint4(0, 0, 0, 0);
            if (live && h + k < item.h1)
                u[k] = load16(src, in0 + (h + k) * a.x_st[w][1]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            float x[8], xp[8], y[8];
            widen8<kF16>(u[k], x);
            float r = 1.f;
            if (norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = fmaf(x[i], x[i], ss);
                r = rsqrtf(group_sum<G::kLanes>(ss) * (1.f / D) + a.eps);
            }
            if (a.rot > 0) {
                widen8<kF16>(partner_words(u[k], src_lane, a.interleaved), xp);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = r * fmaf(x[i], ca[i], pr.sign != 0.f ? xp[i] * sb[i] : 0.f);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = r * (x[i] * ca[i]);
            }
            if (live && h + k < item.h1)
                store16(dst, out0 + (h + k) * a.y_st[w][1], narrow8<kF16>(y));
        }
    }
}

// ------------------------------------------------------------------ backward
// A persistent grid: every warp keeps the weight gradients of its rows in
// registers (fp32) over all its items, the block adds its warps' sums in a
// fixed order and writes one partial a block; dw_reduce_kernel adds those in
// fp64, also in a fixed order, so equal calls give equal bits.
template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeArgs a)
{
    using G = Geo<D>;
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31, v = lane % G::kLanes, base = lane - v;
    const bool in_row = v < G::kVecs;
    const Partner pr = partner_of(v, a.rot, a.interleaved);
    const int src_lane = base + pr.vec;
    float dw[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        dw[0][i] = dw[1][i] = 0.f;
    const long long stride = static_cast<long long>(gridDim.x) * kWarps;
    for (long long it = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32; it < a.items;
         it += stride) {
        const Item item = item_at(a, it, G::kTokens);
        const int w = item.which;
        const long long tok = item.tok0 + lane / G::kLanes;
        bool live = tok < a.tokens;
        const int b = live ? static_cast<int>(tok / a.N) : 0;
        const int n = live ? static_cast<int>(tok - static_cast<long long>(b) * a.N) : 0;
        long long pos;
        if (live && !position_of(a, tok, n, pos)) {
            live = false;
            if (v == 0 && item.h0 == 0)
                record_index(a.status, kRoleRotate);
        }
        live = live && in_row;
        const bool norm = a.w[w] != nullptr;
        const long long x0 = row_at(a.x_st[w], b, 0, n) + v * 8;
        const long long g0 = row_at(a.g_st[w], b, 0, n) + v * 8;
        const long long y0 = row_at(a.y_st[w], b, 0, n) + v * 8;
        float c[8], s[8], wt[8], acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = wt[i] = 1.f;
            s[i] = acc[i] = 0.f;
        }
        if (live) {
            load_angles(a.table, pos, v, a.rot, a.interleaved, pr, c, s);
            if (norm)
                widen8<kF16>(load16(a.w[w], v * 8), wt);
        }
        for (int h = item.h0; h < item.h1; h += kBatch) {
            uint4 ux[kBatch], ug[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                ux[k] = ug[k] = make_uint4(0, 0, 0, 0);
                if (live && h + k < item.h1) {
                    ug[k] = load16(a.g[w], g0 + (h + k) * a.g_st[w][1]);
                    if (norm)
                        ux[k] = load16(a.x[w], x0 + (h + k) * a.x_st[w][1]);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float g[8];
                widen8<kF16>(ug[k], g);
                if (a.rot > 0) {  // the transposed rotation: the sines change sign
                    float gp[8];
                    widen8<kF16>(partner_words(ug[k], src_lane, a.interleaved), gp);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        g[i] = fmaf(g[i], c[i], pr.sign != 0.f ? -gp[i] * s[i] : 0.f);
                }
                if (norm) {
                    float x[8], ss = 0.f, gx = 0.f;
                    widen8<kF16>(ux[k], x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ss = fmaf(x[i], x[i], ss);
                        gx = fmaf(g[i] * wt[i], x[i], gx);
                    }
                    const float r = rsqrtf(group_sum<G::kLanes>(ss) * (1.f / D) + a.eps);
                    const float m = group_sum<G::kLanes>(gx) * (1.f / D) * r * r;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        acc[i] = fmaf(g[i], x[i] * r, acc[i]);
                        g[i] = r * fmaf(-x[i], m, g[i] * wt[i]);
                    }
                }
                if (live && h + k < item.h1)
                    store16(a.y[w], y0 + (h + k) * a.y_st[w][1], narrow8<kF16>(g));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[0][i] += w == 0 ? acc[i] : 0.f;
            dw[1][i] += w == 1 ? acc[i] : 0.f;
        }
    }
    if (a.partial == nullptr)  // no weights: nothing to sum
        return;
    // Groups of a warp first, then the block's warps through shared memory.
    __shared__ float part[kWarps][2][D];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = dw[t][i];
#pragma unroll
            for (int o = G::kLanes; o < 32; o *= 2)
                x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane < G::kVecs)
                part[threadIdx.x / 32][t][lane * 8 + i] = x;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            x += part[k][i / D][i % D];
        a.partial[static_cast<size_t>(blockIdx.x) * 2 * D + i] = x;
    }
}

// dw[t][c] = sum over the blocks' partials.  32 columns a CTA, 32 rows of
// threads over the blocks.
constexpr int kReduceRows = 32;
__global__ void __launch_bounds__(32 * kReduceRows)
    dw_reduce_kernel(const float *partial, int blocks, int D, float *dwq, float *dwk)
{
    __shared__ double part[kReduceRows][33];
    ptx::grid_dependency_wait();
    const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 D, a multiple of 32
    double x = 0.0;
    for (int b = threadIdx.y; b < blocks; b += kReduceRows)
        x += partial[static_cast<size_t>(b) * 2 * D + col];
    part[threadIdx.y][threadIdx.x] = x;
    __syncthreads();
    if (threadIdx.y != 0)
        return;
    x = 0.0;
#pragma unroll
    for (int r = 0; r < kReduceRows; ++r)
        x += part[r][threadIdx.x];
    float *dst = col < D ? dwq : dwk;
    if (dst != nullptr)
        dst[col < D ? col : col - D] = static_cast<float>(x);
}

// ------------------------------------------------------------------ append
// The largest b in [0, B] with cu[b] <= t (-1: none), found by the lanes of a
// group together: each step cuts the range into kLanes parts, so 256
// sequences take two dependent loads where halving takes eight.  The number
// of steps depends on B alone, so the groups of a warp stay together.
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
// tokens of b) + i of its pages, a key turned by that position's angles.
template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a)
{
    using G = Geo<D>;
    const int lane = threadIdx.x & 31, v = lane % G::kLanes, base = lane - v;
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
    const bool exists = tok < a.T && v < G::kVecs;
    const void *src = is_v ? a.v : a.k;
    const long long tok_stride = is_v ? a.v_st[0] : a.k_st[0];
    const long long head_stride = is_v ? a.v_st[1] : a.k_st[1];
    const long long in0 = (exists ? tok : 0) * tok_stride + v * 8;
    // The rows do not depend on where they go: the first batch is in flight
    // while the token's sequence, page and angles are looked up.
    uint4 u[kBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            u[k] = make_uint4(0, 0, 0, 0);
            if (exists && h + k < h1)
                u[k] = load16(src, in0 + (h + k) * head_stride);
        }
    };
    load(h0);
    bool live = tok < a.T, bad = false;
    const int b = find_sequence<G::kLanes>(a.cu_q, a.B, tok, v, base);
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
            out0 = (is_v ? a.vc_st[0] * page + a.vc_st[2] * slot
                         : a.kc_st[0] * page + a.kc_st[2] * slot) + v * 8;
        }
        if (bad && v == 0 && h0 == 0 && !is_v)
            record_index(a.status, kRoleAppend);
        live = !bad && v < G::kVecs;
    } else {
        live = false;  // behind the last sequence (or before the first)
    }
    void *dst = is_v ? a.v_cache : a.k_cache;
    const long long out_head = is_v ? a.vc_st[1] : a.kc_st[1];
    const bool turn = !is_v && a.rot > 0;
    const Partner pr = partner_of(v, turn ? a.rot : 0, a.interleaved);
    float ca[8], sa[8];
    if (turn && live)
        load_angles(a.table, pos, v, a.rot, a.interleaved, pr, ca, sa);
    for (int h = h0;;) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            uint4 y = u[k];
            if (turn) {
                const uint4 up = partner_words(u[k], base + pr.vec, a.interleaved);
                if (pr.sign != 0.f) {  // unrotated elements keep their bits
                    float x[8], xp[8];
                    widen8<kF16>(u[k], x);
                    widen8<kF16>(up, xp);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = fmaf(x[i], ca[i], xp[i] * sa[i]);
                    y = narrow8<kF16>(x);
                }
            }
            if (live && h + k < h1)
                store16(dst, out0 + (h + k) * out_head, y);
        }
        h += kBatch;
        if (h >= h1)
            break;
        load(h);
    }
}

// Heads an item: enough items to give every SM kItemsPerSm warps, at least
// one batch of rows each.  More heads an item read the angles less often.
constexpr int kItemsPerSm = 32;
int heads_per_item(long long token_blocks, int heads, int num_sms)
{
    const long long want = static_cast<long long>(num_sms) * kItemsPerSm;
    int n = kBatch;
    while (n < heads && token_blocks * ((heads + 2 * n - 1) / (2 * n)) >= want)
        n *= 2;
    return n;
}

cudaError_t grid_of(long long items, unsigned *grid)
{
    const long long blocks = (items + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    *grid = static_cast<unsigned>(blocks);
    return cudaSuccess;
}

template <int D, bool kF16>
cudaError_t norm_rope(NormRopeArgs a, int num_sms, cudaStream_t stream)
{
    const long long blocks = (a.tokens + Geo<D>::kTokens - 1) / Geo<D>::kTokens;
    a.heads_per_chunk = heads_per_item(blocks, a.H[0] + a.H[1], num_sms);
    for (int t = 0; t < 2; ++t)
        a.chunks[t] = (a.H[t] + a.heads_per_chunk - 1) / a.heads_per_chunk;
    a.items = blocks * (a.chunks[0] + a.chunks[1]);
    if (a.g[0] == nullptr && a.g[1] == nullptr) {
        unsigned grid;
        cudaError_t e = grid_of(a.items, &grid);
        if (e != cudaSuccess)
            return e;
        norm_rope_kernel<D, kF16><<<grid, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const long long want = (a.items + kWarps - 1) / kWarps;
    const int grid = static_cast<int>(want < norm_rope_bwd_blocks(num_sms)
                                          ? want : norm_rope_bwd_blocks(num_sms));
    norm_rope_bwd_kernel<D, kF16><<<grid, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.partial == nullptr)
        return e;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * D / 32);
    cfg.blockDim = dim3(32, kReduceRows);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dw_reduce_kernel, static_cast<const float *>(a.partial), grid, D,
                              a.dw[0], a.dw[1]);
}

template <int D, bool kF16>
cudaError_t kv_append(KvAppendArgs a, int num_sms, cudaStream_t stream)
{
    const long long blocks = (a.T + Geo<D>::kTokens - 1) / Geo<D>::kTokens;
    a.heads_per_chunk = heads_per_item(2 * blocks, a.H, num_sms);
    a.chunks = (a.H + a.heads_per_chunk - 1) / a.heads_per_chunk;
    a.items = blocks * 2 * a.chunks;
    unsigned grid;
    cudaError_t e = grid_of(a.items, &grid);
    if (e != cudaSuccess)
        return e;
    kv_append_kernel<D, kF16><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D> cudaError_t norm_rope_typed(const NormRopeArgs &a, int num_sms, cudaStream_t stream)
{
    return a.f16 ? norm_rope<D, true>(a, num_sms, stream) : norm_rope<D, false>(a, num_sms, stream);
}
template <int D> cudaError_t kv_append_typed(const KvAppendArgs &a, int num_sms, cudaStream_t stream)
{
    return a.f16 ? kv_append<D, true>(a, num_sms, stream) : kv_append<D, false>(a, num_sms, stream);
}

}  // namespace

// Eight blocks of four warps a SM fill it at the backward kernel's registers.
int norm_rope_bwd_blocks(int num_sms) { return 8 * num_sms; }

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
