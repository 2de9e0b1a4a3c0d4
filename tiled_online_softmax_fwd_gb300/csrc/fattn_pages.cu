// fattn_pages.cu -- the sequences of a paged cache between the steps of a
// search: keeping the accepted tokens of a drafted tree, and forking, growing
// and freeing sequences.
//
// Keep.  Of a sequence's n new tokens those listed stay, moved together:
//   slot L - n + j  <-  slot L - n + kept[j],   j = 0, 1, ...;   L' = L - n + m
// with kept ascending, so kept[j] >= j and a block that goes through j in order
// never reads a slot it has written: it loads a batch of rows, meets, and
// stores them.  Bound by latency at a step's few tokens (a chain of four loads:
// lengths, kept, pages, rows), by bytes at many.
//
// Fork.  Sequence b goes on as its parent's copy with room for new tokens:
//   table'[b] = the parent's entries, L'[b] = L[parent] + n_b.
// Whole pages are shared.  A last page that is partly filled has one owner, the
// parent itself where it goes on and else its first child; every other child
// gets a copy of it in a page of its own.  refs counts the entries that name a
// page; pages that none names after the step are free, and the lowest of them
// are given out in the order of sequences and columns, so equal calls give equal
// tables whatever the order of the atomic counts.  One cluster of blocks does
// the lists in steps between cluster barriers (a block alone where they are
// short), a second kernel copies the pages' rows.
#include <cooperative_groups.h>
#include <stdint.h>

#include "fattn_internal.h"
#include "ptx_sm103.cuh"

namespace fattn {
namespace {

namespace cg = cooperative_groups;
using namespace ptx;

// ------------------------------------------------------------------ keep
constexpr int kKeepThreads = 256;
constexpr int kKeepBatch = 4;  // 16-byte pieces of a thread in flight

// A block: one sequence, some heads, one of the two caches; a cluster: a
// sequence, so that its length is written (in place, too) behind every reading.
__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const KvKeepArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int chunk = blockIdx.x % a.chunks, which = blockIdx.x / a.chunks % 2;
    const int b = blockIdx.x / a.chunks / 2;
    const int tid = threadIdx.x;
    const int L = a.kv_len[b], count = a.kept_len[b];
    const long long n = static_cast<long long>(a.cu_q[b + 1]) - a.cu_q[b];
    const long long max_keys = static_cast<long long>(a.max_pages) << a.page_shift;
    const int *kept = a.kept + b * a.kept_stride;
    const int *table = a.page_table + b * a.table_stride;
    bool bad = n < 0 || L < n || L > max_keys || count < 0 || count > n || count > a.max_kept;
    const int prefix = bad ? 0 : static_cast<int>(L - n);
    const int m = bad ? 0 : count;
    // The list's own faults, and where the moves begin.
    int stay = m;
    for (int j = tid; j < m; j += kKeepThreads) {
        const int at = kept[j];
        const bool in = at >= 0 && at < n && (j == 0 || kept[j - 1] < at);
        bad = bad || !in;
        if (in && at != j) {
            const int src = table[(prefix + at) >> a.page_shift], dst = table[(prefix + j) >> a.page_shift];
            bad = bad || src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages;
            stay = min(stay, j);
        }
    }
    // In ascending order the tokens that stay in place come first.
    __shared__ int first;
    if (tid == 0)
        first = m;
    bad = __syncthreads_or(bad);
    if (stay < m)
        atomicMin(&first, stay);
    cg::this_cluster().sync();
    if (chunk == 0 && which == 0 && tid == 0) {
        a.kv_len_out[b] = bad ? L : prefix + m;
        if (bad)
            atomicCAS(a.status, 0u, 6u /* FATTN_ERR_INDEX */ | (kRoleKeep << 8));
    }
    if (bad)
        return;
    const int h0 = chunk * a.heads_per_chunk, heads = max(min(a.heads_per_chunk, a.H - h0), 0);
    const int vecs = a.d / 8, each = heads * vecs;  // of a row, of a token
    const long long *st = which == 0 ? a.kc_st : a.vc_st;
    uint16_t *cache = static_cast<uint16_t *>(which == 0 ? a.k_cache : a.v_cache);
    const int slots = (1 << a.page_shift) - 1;
    auto at = [&](int pos, int h, int c) {
        return reinterpret_cast<uint4 *>(cache + table[pos >> a.page_shift] * st[0] + (h0 + h) * st[1] +
                                         (pos & slots) * st[2] + c * 8);
    };
    const long long total = static_cast<long long>(m - first) * each;
    for (long long base = 0; base < total; base += kKeepThreads * kKeepBatch) {
        uint4 x[kKeepBatch], *to[kKeepBatch];
#pragma unroll
        for (int i = 0; i < kKeepBatch; ++i) {
            const long long item = base + i * kKeepThreads + tid;
            to[i] = nullptr;
            if (item < total) {
                const int t = static_cast<int>(item / each), rest = static_cast<int>(item - static_cast<long long>(t) * each);
                const int h = rest / vecs, c = rest - h * vecs, j = first + t;
                x[i] = *at(prefix + kept[j], h, c);
                to[i] = at(prefix + j, h, c);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kKeepBatch; ++i)
            if (to[i] != nullptr)
                *to[i] = x[i];
    }
}

// ------------------------------------------------------------------ fork
constexpr int kForkThreads = 512;
constexpr int kForkWarps = kForkThreads / 32;

// What becomes of a sequence.
struct Next {
    int parent;  // -1: none
    bool keeps;  // goes on with the parent's own pages
    int whole;   // pages that it shares (or keeps) whole
    int part;    // filled slots of the page behind them
    int total, want;  // keys and pages afterwards
    bool bad;
};
__device__ __forceinline__ int parent_of(const KvForkArgs &a, int b, bool &bad)
{
    const int p = a.parents != nullptr ? a.parents[b] : b;
    bad = p < -1 || p >= a.B;
    return bad ? b : p;
}
__device__ __forceinline__ Next next_of(const KvForkArgs &a, const int *old_len, int b)
{
    Next x;
    x.parent = parent_of(a, b, x.bad);
    x.keeps = x.parent >= 0 && __ldcg(&a.first[x.parent]) == b;
    const long long max_keys = static_cast<long long>(a.max_pages) << a.page_shift;
    long long base = 0;
    if (x.parent >= 0) {
        const int L = __ldcg(&old_len[x.parent]);
        base = min(max(static_cast<long long>(L), 0LL), max_keys);
        x.bad = x.bad || base != L;
    }
    long long total = base;
    if (a.cu_q != nullptr) {
        const long long n = static_cast<long long>(a.cu_q[b + 1]) - a.cu_q[b];
        total = min(base + max(n, 0LL), max_keys);
        x.bad = x.bad || n < 0 || total != base + n;
    }
    x.whole = static_cast<int>(base >> a.page_shift);
    x.part = static_cast<int>(base & ((1 << a.page_shift) - 1));
    x.total = static_cast<int>(total);
    x.want = static_cast<int>((total + (1 << a.page_shift) - 1) >> a.page_shift);
    return x;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int block_sum(int x, int *scratch)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        scratch[threadIdx.x / 32] = x;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kForkWarps; ++w)
        sum += scratch[w];
    return sum;
}
// Exclusive prefix over the block's threads, and the total.
__device__ __forceinline__ int block_prefix(int x, int *scratch, int &total)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? y : 0;
    }
    __syncthreads();
    if (lane == 31)
        scratch[warp] = incl;
    __syncthreads();
    int before = incl - x;
    total = 0;
#pragma unroll
    for (int w = 0; w < kForkWarps; ++w) {
        before += w < warp ? scratch[w] : 0;
        total += scratch[w];
    }
    return before;
}

// The lists.  What one step writes the next reads past the first-level cache.
// Blocks of the one cluster meet between the steps; rows and pages
// are dealt to the cluster's warps and blocks.
__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(const KvForkArgs a)
{
    __shared__ int scratch[kForkWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x, ranks = gridDim.x;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int all = rank * kForkThreads + tid, threads = ranks * kForkThreads;
    const int my_warp = rank * kForkWarps + warp, warps = ranks * kForkWarps;
    grid_launch_dependents();
    grid_dependency_wait();
    auto meet = [&]() {
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    bool bad = false;
    // 1. Copies of what is overwritten in place; counts; no child yet.
    const int *old_table = a.page_table, *old_len = a.kv_len;
    long long old_stride = a.table_stride;
    if (a.staged) {
        for (int b = my_warp; b < a.B; b += warps)
            for (int c = lane; c < a.max_pages; c += 32)
                a.stage[static_cast<long long>(b) * a.max_pages + c] = a.page_table[b * a.table_stride + c];
        for (int b = all; b < a.B; b += threads)
            a.stage_len[b] = a.kv_len[b];
        old_table = a.stage;
        old_len = a.stage_len;
        old_stride = a.max_pages;
    }
    if (a.refs_out != a.refs)
        for (int i = all; i < a.num_pages; i += threads)
            a.refs_out[i] = a.refs[i];
    for (int b = all; b < a.B; b += threads)
        a.first[b] = 0x7fffffff;
    meet();
    // 2. Each parent's page owner: itself (as -1, below all), or the first child.
    for (int b = all; b < a.B; b += threads) {
        bool stray;
        const int p = parent_of(a, b, stray);
        if (p >= 0)
            atomicMin(&a.first[p], p == b ? -1 : b);
    }
    meet();
    for (int b = all; b < a.B; b += threads)
        if (__ldcg(&a.first[b]) == -1)
            a.first[b] = b;
    meet();
    // 3. The new rows as far as they follow from the old ones, the counts, and
    // how many pages each lacks.
    for (int b = my_warp; b < a.B; b += warps) {
        const Next x = next_of(a, old_len, b);
        bad = bad || x.bad;
        const int *mine = old_table + b * old_stride;
        const int *theirs = x.parent >= 0 ? old_table + x.parent * old_stride : mine;
        const bool same = x.parent == b;
        int lacks = 0;
        for (int c0 = 0; c0 < a.max_pages; c0 += 32) {
            const int c = c0 + lane;
            int e = -1, was = -1;
            if (c < a.max_pages) {
                was = __ldcg(&mine[c]);
                if (x.parent >= 0 && (x.keeps || c < x.whole))
                    e = __ldcg(&theirs[c]);
                bad = bad || was < -1 || was >= a.num_pages;
                was = was >= a.num_pages ? -1 : was;
                e = e >= a.num_pages ? -1 : max(e, -1);
                a.table_out[b * a.table_out_stride + c] = e;
                if (!same) {
                    if (was >= 0)
                        atomicSub(&a.refs_out[was], 1);
                    if (e >= 0)
                        atomicAdd(&a.refs_out[e], 1);
                }
            }
            lacks += __popc(__ballot_sync(0xffffffffu, c < x.want && e < 0));
        }
        if (lane == 0) {
            a.lacks[b] = lacks;
            a.len_out[b] = x.total;
            // The page to copy, if any; its place is filled in below.
            int src = -1;
            if (x.parent >= 0 && !x.keeps && x.part > 0) {
                src = __ldcg(&theirs[x.whole]);
                if (src < 0 || src >= a.num_pages) {
                    src = -1;
                    bad = true;
                }
            }
            a.copies[b] = make_int4(src, -1, x.part, x.whole);
        }
    }
    meet();
    // 4. Free pages among each block's range of them, and the lacks before its rows.
    const int page0 = static_cast<int>(static_cast<long long>(a.num_pages) * rank / ranks);
    const int page1 = static_cast<int>(static_cast<long long>(a.num_pages) * (rank + 1) / ranks);
    int mine = 0, need = 0;
    for (int i = page0 + tid; i < page1; i += kForkThreads)
        mine += __ldcg(&a.refs_out[i]) == 0;
    for (int b = tid; b < a.B; b += kForkThreads)
        need += __ldcg(&a.lacks[b]);
    mine = block_sum(mine, scratch);
    need = block_sum(need, scratch);
    if (tid == 0)
        a.counts[rank] = mine;
    meet();
    if (need > 0) {
        int at = 0;
        for (int r = 0; r < rank; ++r)
            at += __ldcg(&a.counts[r]);
        for (int i0 = page0; i0 < page1 && at < need; i0 += kForkThreads) {
            const int i = i0 + tid;
            const bool is = i < page1 && __ldcg(&a.refs_out[i]) == 0;
            int found;
            const int k = at + block_prefix(is ? 1 : 0, scratch, found);
            if (is && k < need)
                a.free_list[k] = i;
            at += found;
        }
        // Where each row's pages begin in the list: every block all of them, in
        // its own copy.
        int before = 0;
        for (int b0 = 0; b0 < a.B; b0 += kForkThreads) {
            const int b = b0 + tid;
            int sum;
            const int k = block_prefix(b < a.B ? __ldcg(&a.lacks[b]) : 0, scratch, sum);
            if (b < a.B && b % ranks == rank)
                a.first[b] = before + k;
            before += sum;
        }
    }
    int have = 0;
    for (int r = 0; r < ranks; ++r)
        have += __ldcg(&a.counts[r]);
    meet();
    // 5. The lacking entries, in order.
    if (need > 0)
        for (int b = my_warp; b < a.B; b += warps) {
            if (__ldcg(&a.lacks[b]) == 0)
                continue;
            int at = __ldcg(&a.first[b]);
            const int4 copy = __ldcg(&a.copies[b]);
            const int want = (__ldcg(&a.len_out[b]) + (1 << a.page_shift) - 1) >> a.page_shift;
            int *row = a.table_out + b * a.table_out_stride;
            for (int c0 = 0; c0 < want; c0 += 32) {
                const int c = c0 + lane;
                const bool lack = c < want && __ldcg(&row[c]) < 0;
                const unsigned who = __ballot_sync(0xffffffffu, lack);
                if (lack) {
                    const int k = at + __popc(who & ((1u << lane) - 1u));
                    if (k < have) {
                        const int page = __ldcg(&a.free_list[k]);
                        row[c] = page;
                        a.refs_out[page] = 1;
                        if (c == copy.w && copy.x >= 0)
                            a.copies[b].y = page;
                    } else {
                        bad = true;
                    }
                }
                at += __popc(who);
            }
        }
    if (bad)
        atomicCAS(a.status, 0u, 6u /* FATTN_ERR_INDEX */ | (kRoleFork << 8));
}

// The copied pages' filled slots: a block takes a run of one page's pieces, of
// one cache.
constexpr int kCopyThreads = 256, kCopyBatch = 4;
__global__ void __launch_bounds__(kCopyThreads) kv_fork_copy_kernel(const KvForkArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int chunk = blockIdx.x % a.chunks, which = blockIdx.x / a.chunks % 2;
    const int4 copy = a.copies[blockIdx.x / a.chunks / 2];
    if (copy.x < 0 || copy.y < 0)
        return;
    const int vecs = a.d / 8, each = copy.z * vecs, total = a.H * each;
    const long long *st = which == 0 ? a.kc_st : a.vc_st;
    uint16_t *cache = static_cast<uint16_t *>(which == 0 ? a.k_cache : a.v_cache);
    const uint16_t *src = cache + copy.x * st[0];
    uint16_t *dst = cache + copy.y * st[0];
    uint4 x[kCopyBatch];
    long long off[kCopyBatch];
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i) {
        const int item = (chunk * kCopyBatch + i) * kCopyThreads + threadIdx.x;
        off[i] = -1;
        if (item < total) {
            const int h = item / each, rest = item - h * each, slot = rest / vecs;
            off[i] = h * st[1] + slot * st[2] + (rest - slot * vecs) * 8;
            x[i] = *reinterpret_cast<const uint4 *>(src + off[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i)
        if (off[i] >= 0)
            *reinterpret_cast<uint4 *>(dst + off[i]) = x[i];
}

template <class Args>
cudaError_t start(void (*kernel)(Args), const Args &a, long long blocks, int threads, int cluster,
                  cudaStream_t stream)
{
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_keep(const KvKeepArgs &args, cudaStream_t stream)
{
    KvKeepArgs a = args;
    // One, two or four blocks for the heads of a cache (a cluster has at most
    // eight): more while each has a batch of its threads' pieces to move at the
    // most tokens kept.
    const long long pieces = static_cast<long long>(a.max_kept) * a.H * (a.d / 8);
    a.chunks = pieces <= kKeepThreads * kKeepBatch ? 1 : pieces <= 2 * kKeepThreads * kKeepBatch ? 2 : 4;
    a.heads_per_chunk = (a.H + a.chunks - 1) / a.chunks;
    return start(kv_keep_kernel, a, 2LL * a.B * a.chunks, kKeepThreads, 2 * a.chunks, stream);
}

cudaError_t launch_kv_fork(const KvForkArgs &args, cudaStream_t stream)
{
    KvForkArgs a = args;
    // One block up to some thousand entries: its barriers are shorter than a
    // cluster's, which has more hands for long lists.
    const long long entries = static_cast<long long>(a.B) * a.max_pages + a.num_pages;
    const int ranks = entries <= 4096 ? 1 : kForkRanks;
    cudaError_t e = start(kv_fork_kernel, a, ranks, kForkThreads, ranks, stream);
    if (e != cudaSuccess || a.parents == nullptr || a.H == 0)
        return e;
    const long long pieces = static_cast<long long>(a.H) * ((1 << a.page_shift) - 1) * (a.d / 8);
    a.chunks = static_cast<int>((pieces + kCopyThreads * kCopyBatch - 1) / (kCopyThreads * kCopyBatch));
    return start(kv_fork_copy_kernel, a, 2LL * a.B * a.chunks, kCopyThreads, 1, stream);
}

}  // namespace fattn
