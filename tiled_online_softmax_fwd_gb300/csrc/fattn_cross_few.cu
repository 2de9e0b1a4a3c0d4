// fattn_cross_few.cu -- cross attention of few rows: a decoder's single tokens
// (or a few beams) against long keys, on the CUDA cores.
//
// With R = Nq Hq / Hk rows to a key head each key takes R d multiply-adds and as
// many for its value, against 4 d bytes: at R <= 4 the memory is the bound.  The
// tensor-core kernel spends its time on copies, hand-overs and 128-row tiles
// that are mostly empty (37.5 us for 32 sequences of 500 to 1500 keys, 16 heads,
// d = 64, 128 MB, where this one takes 24.8: 5.2 TB/s).
//
// Copies (cp.async) run two batches of 16 or 8 keys ahead of a warp, some 64 KB
// a SM on their way: with plain loads, a batch of each warp at a time, it took a
// quarter longer.
//
// A warp takes keys in turns: a group of d / 8 lanes (rounded up to a power of
// two) holds a key's 16-byte pieces and the same pieces of the R queries.  Each
// group keeps a softmax of its own over its keys, (m, l, O) in fp32; groups are
// merged by shuffles, warps through shared memory, and the blocks of a cluster,
// which share the keys of one (sequence, key head), through distributed shared
// memory: one launch, and an order of sums that depends on the lengths alone.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include "fattn_internal.h"
#include "ptx_sm103.cuh"

namespace fattn {
namespace {

namespace cg = cooperative_groups;
using namespace ptx;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSteps = 4;   // of a batch: that many pieces of K and of V a lane
constexpr int kStages = 3;  // batches of a warp in shared memory, on their way or in use
constexpr uint32_t kRingBytes = kWarps * kStages * kSteps * 2 * 32 * 16;
constexpr float kLn2 = 0.6931471805599453f;

template <bool kF16> __device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (kF16)
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
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
// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint4 *to, const uint16_t *from, bool some)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(some ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n> __device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// Two softmaxes become one: factors of the first and the second, and the new m.
__device__ __forceinline__ void join(float m0, float m1, float &m, float &f0, float &f1)
{
    m = fmaxf(m0, m1);
    f0 = ex2(m0 - m);
    f1 = ex2(m1 - m);
}

template <int D, bool kF16, int R>
__global__ void __launch_bounds__(kThreads, 2) cross_few_kernel(const PagedArgs a, const CrossFew x)
{
    constexpr int kLanes = D / 8, kGroup = D == 64 ? 8 : 16, kKeys = 32 / kGroup;  // of a warp's step
    // A block's result: R rows of D sums, then (m, l) of each.
    constexpr int kPart = R * D + (2 * R + 3) / 4 * 4;  // in whole 16 bytes
    __shared__ alignas(16) float part[kWarps][kPart];
    __shared__ alignas(16) float whole[kPart];
    cg::cluster_group cluster = cg::this_cluster();
    const int splits = x.splits, rank = blockIdx.x % splits;
    const int unit = blockIdx.x / splits, place = unit / a.Hk, h = unit - place * a.Hk;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int piece = lane % kGroup, group = lane / kGroup;
    const bool real = piece < kLanes;
    grid_dependency_wait();
    grid_launch_dependents();
    // The longest sequences first, up to 32 of them, so that the last blocks to start
    // are short (24.8 us for the batch above, in the given order 28).  More than a warp's
    // lanes are taken as given; that was not measured.
    int b = place, given = a.max_keys;
    if (a.kv_len != nullptr) {
        if (a.B <= 32) {
            const int mine = lane < a.B ? a.kv_len[lane] : INT_MIN;
            int before = 0;
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {
                const int other = __shfl_sync(0xffffffffu, mine, j);
                before += other > mine || (other == mine && j < lane);
            }
            b = __ffs(__ballot_sync(0xffffffffu, before == place)) - 1;
            given = __shfl_sync(0xffffffffu, mine, b);
        } else {
            given = a.kv_len[b];
        }
    }
    const int L = min(max(given, 0), a.max_keys);
    if (given != L && h == 0 && rank == 0 && tid == 0)
        atomicCAS(a.status, 0u, 6u /* FATTN_ERR_INDEX */ | (kRoleLoad << 8));
    float q[R][8], acc[R][8], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int tok = r / a.G, g = r - tok * a.G;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < x.rows && real)
            w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x.q) + b * x.q_st[0] +
                                                 (h * a.G + g) * x.q_st[1] + tok * x.q_st[2] + piece * 8);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<kF16>(v[i]);
            q[r][2 * i] = f.x * a.sl2;
            q[r][2 * i + 1] = f.y * a.sl2;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[r][i] = 0.f;
        m[r] = -FLT_MAX;
        l[r] = 0.f;
    }
    // This block's keys, and a warp's turns in them.
    const int per = (L + splits - 1) / splits, k0 = min(rank * per, L), k1 = min(k0 + per, L);
    const uint16_t *kp = static_cast<const uint16_t *>(x.k) + b * x.k_st[0] + h * x.k_st[1] + (real ? piece * 8 : 0);
    const uint16_t *vp = static_cast<const uint16_t *>(x.v) + b * x.v_st[0] + h * x.v_st[1] + (real ? piece * 8 : 0);
    // A lane reads what it has copied itself, so the ring needs no barriers.
    extern __shared__ uint4 ring[];
    uint4 *mine = ring + warp * (kStages * kSteps * 2 * 32) + lane;
    constexpr int kBatch = kSteps * kKeys;
    const int first = k0 + warp * kBatch, turn = kWarps * kBatch;
    const int batches = first < k1 ? (k1 - first + turn - 1) / turn : 0;
    auto issue = [&](int i) {
        if (i < batches) {
            uint4 *to = mine + i % kStages * (kSteps * 2 * 32);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int key = first + i * turn + s * kKeys + group;
                const bool some = key < k1 && real;
                const int at = some ? key : k0;
                copy16(to + 64 * s, kp + at * x.k_st[2], some);
                copy16(to + 64 * s + 32, vp + at * x.v_st[2], some);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        issue(i);
#pragma unroll 1
    for (int it = 0; it < batches; ++it) {
        const int base = first + it * turn;
        issue(it + kStages - 1);
        copies_wait<kStages - 1>();
        uint4 kw[kSteps], vw[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            kw[s] = mine[it % kStages * (kSteps * 2 * 32) + 64 * s];
            vw[s] = mine[it % kStages * (kSteps * 2 * 32) + 64 * s + 32];
        }
        float p[kSteps][R];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const uint32_t w[4] = {kw[s].x, kw[s].y, kw[s].z, kw[s].w};
#pragma unroll
            for (int r = 0; r < R; ++r)
                p[s][r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<kF16>(w[i]);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    p[s][r] = fmaf(f.y, q[r][2 * i + 1], fmaf(f.x, q[r][2 * i], p[s][r]));
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int o = kGroup / 2; o > 0; o /= 2)
                    p[s][r] += __shfl_xor_sync(0xffffffffu, p[s][r], o);
                if (base + s * kKeys + group >= k1)
                    p[s][r] = -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = m[r];
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                top = fmaxf(top, p[s][r]);
            const float f = ex2(m[r] - top);
            m[r] = top;
            l[r] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[r][i] *= f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                p[s][r] = ex2(p[s][r] - top);
                l[r] += p[s][r];
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const uint32_t w[4] = {vw[s].x, vw[s].y, vw[s].z, vw[s].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<kF16>(w[i]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[r][2 * i] = fmaf(p[s][r], f.x, acc[r][2 * i]);
                    acc[r][2 * i + 1] = fmaf(p[s][r], f.y, acc[r][2 * i + 1]);
                }
            }
        }
    }
    // The warp's groups, then the block's warps.
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int o = kGroup; o < 32; o *= 2) {
            const float m1 = __shfl_xor_sync(0xffffffffu, m[r], o), l1 = __shfl_xor_sync(0xffffffffu, l[r], o);
            float mm, f0, f1;
            join(m[r], m1, mm, f0, f1);
            // The lower lane's sum first on both sides: equal bits in all lanes.
            const bool low = (lane & o) == 0;
            m[r] = mm;
            l[r] = low ? fmaf(l1, f1, l[r] * f0) : fmaf(l[r], f0, l1 * f1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __shfl_xor_sync(0xffffffffu, acc[r][i], o);
                acc[r][i] = low ? fmaf(y, f1, acc[r][i] * f0) : fmaf(acc[r][i], f0, y * f1);
            }
        }
        if (group == 0 && real) {
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<float4 *>(&part[warp][r * D + piece * 8 + i]) =
                    make_float4(acc[r][i], acc[r][i + 1], acc[r][i + 2], acc[r][i + 3]);
            if (piece == 0) {
                part[warp][R * D + 2 * r] = m[r];
                part[warp][R * D + 2 * r + 1] = l[r];
            }
        }
    }
    __syncthreads();
    auto merge = [&](auto get, int count, int r, int c, float &mm, float &ll) {
        mm = -FLT_MAX;
        for (int w = 0; w < count; ++w)
            mm = fmaxf(mm, get(w)[R * D + 2 * r]);
        float sum = 0.f;
        ll = 0.f;
        for (int w = 0; w < count; ++w) {
            const float *p = get(w);
            const float f = ex2(p[R * D + 2 * r] - mm);
            sum = fmaf(p[r * D + c], f, sum);
            ll = fmaf(p[R * D + 2 * r + 1], f, ll);
        }
        return sum;
    };
    for (int i = tid; i < R * D; i += kThreads) {
        const int r = i / D, c = i - r * D;
        float mm, ll;
        const float y = merge([&](int w) { return part[w]; }, kWarps, r, c, mm, ll);
        whole[i] = y;
        if (c == 0) {
            whole[R * D + 2 * r] = mm;
            whole[R * D + 2 * r + 1] = ll;
        }
    }
    if (splits > 1)
        cluster.sync();
    else
        __syncthreads();
    // The cluster's blocks: each writes a share of the rows' columns, in pairs.
    for (int i = rank * kThreads + tid; i < x.rows * D / 2; i += splits * kThreads) {
        const int r = 2 * i / D, c = 2 * i - r * D;
        float mm, ll, y[2];
        auto get = [&](int w) {
            return splits > 1 ? static_cast<const float *>(cluster.map_shared_rank(whole, w)) : whole;
        };
        y[0] = merge(get, splits, r, c, mm, ll);
        y[1] = merge(get, splits, r, c + 1, mm, ll);
        const float inv = ll == 0.f ? 0.f : 1.f / ll;  // no key; NaN goes on
        const int tok = r / a.G, head = h * a.G + r - tok * a.G;
        uint16_t *o = static_cast<uint16_t *>(a.o) + b * a.o_batch + head * a.o_st[1] + tok * a.o_st[0];
        *reinterpret_cast<uint32_t *>(o + c) = pack2<kF16>(y[0] * inv, y[1] * inv);
        if (c == 0)
            a.lse[(static_cast<long long>(b) * a.Hk * a.G + head) * a.Nq + tok] =
                ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
        // Each for itself: the sum of two that fit may not.
        if (!kF16 && !(fabsf(y[0] * inv) <= FLT_MAX && fabsf(y[1] * inv) <= FLT_MAX))
            atomicCAS(a.status, 0u,
                      5u /* FATTN_ERR_RANGE */ | (kRoleEpilogue << 8) | ((blockIdx.x & 0xffffu) << 16));
    }
    if (splits > 1)
        cluster.sync();  // the others read this block's memory
}

template <int D, bool kF16, int R>
cudaError_t launch_rows(const PagedArgs &a, const CrossFew &x, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(
        cross_few_kernel<D, kF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes));
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = x.splits;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.Hk * x.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRingBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = x.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, cross_few_kernel<D, kF16, R>, a, x);
}
template <int D, bool kF16> cudaError_t launch_typed(const PagedArgs &a, const CrossFew &x, cudaStream_t stream)
{
    return x.rows == 1   ? launch_rows<D, kF16, 1>(a, x, stream)
           : x.rows == 2 ? launch_rows<D, kF16, 2>(a, x, stream)
                         : launch_rows<D, kF16, 4>(a, x, stream);
}
template <int D> cudaError_t launch(const PagedArgs &a, const CrossFew &x, cudaStream_t stream)
{
    return a.f16 ? launch_typed<D, true>(a, x, stream) : launch_typed<D, false>(a, x, stream);
}

}  // namespace

int cross_few_splits(int B, int Hk, int rows, int Nk, int d, int num_sms)
{
    const long long units = static_cast<long long>(B) * Hk;
    if (rows > kCrossFewRows || units * 8 > 0x7fffffffLL)
        return 0;
    // A block for every SM, while each has some keys to read; a second one an SM
    // only for long keys (a cluster's start and its merge cost some 3 us).
    int splits = 1;
    while (splits < 8 && Nk / (2 * splits) >= 64 &&
           (units * splits < num_sms || (units * splits < 2 * num_sms && Nk / splits >= 2048)))
        splits *= 2;
    // Measured against the tensor-core kernel (us, this one first).  Few units of
    // long keys leave SMs idle, which that one fills: 8 units of 30000 keys, d =
    // 64, 24.0 and 21.6, d = 128 41.6 and 33.6; of 6000 8.0 and 13.6, 12.5 and
    // 17.1.  More rows take more arithmetic, four at d = 128 more registers than
    // there are: 128 units of 300 keys 18.0 and 15.3, 8 units of 1500 9.1 and 13.8;
    // at d = 64 512 units of 1500 keys 52.8 and 50.6, of 300 18.7 and 24.1.
    if (units * splits < num_sms && Nk / splits > 1536)
        return 0;
    if (rows > 2 && units * Nk > (d == 64 ? 65536 : 16384))
        return 0;
    return splits;
}

cudaError_t launch_cross_few(const PagedArgs &a, const CrossFew &x, cudaStream_t stream)
{
    switch (a.d) {
    case 64: return launch<64>(a, x, stream);
    case 96: return launch<96>(a, x, stream);
    case 128: return launch<128>(a, x, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fattn
