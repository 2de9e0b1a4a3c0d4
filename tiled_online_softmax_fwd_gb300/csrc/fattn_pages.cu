// fattn_pages.cu -- the sequences of a paged cache between the steps of a
// search: keeping the accepted tokens of a drafted tree, and forking, growing
// and freeing sequences.
//
// Keep.  Of a sequence's n new tokens those listed stay, moved together:
//   slot L - n + j  <-  slot L - n + kept[j],   j = 0, 1, ...;   L' = L - n + m
// with kept ascending, so kept[j] >= j and a block that goes through j in order
// never reads a slot it has written: it loads a batch of rows, meets, and
// stores them.  Bound by latency at a step's few tokens (a chain of four loads:
// lengths, kept, pages, rows): 6 us on the GPU, in a graph, with the append before it
// for 4 sequences of 26 tokens (plain calls 12, the host's); 8.7 us for 192 of up to
// 129, up to 24 of them kept (8 key heads, d = 128; the rows were written just before
// and come from L2).
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
// short), a second kernel copies the pages' rows.  Bound by latency: the lists are
// a few KB, read in four dependent steps (entries, their counts, the counts' sums,
// the free pages) with a meeting of the blocks between two: 9.3 us in a graph for 8
// sequences of up to 900 keys, 16.7 for 256 of up to 4000 and 700 new ones; pages of 16
// and 32.  A sequence that goes on with its own pages adds a walk by one thread along
// the columns that it grows by, a read each: 64 sequences that grow by a page 8.3 us
// (with 50000 pages in the pool, all looked at, 12.0), one by 1000 pages 62, 16 by 1000
// each 81.
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
    // Some tokens at a time, as many as the threads' pieces hold, or parts of one.
    constexpr int kWave = kKeepThreads * kKeepBatch;
    const int group = max(kWave / max(each, 1), 1);
    for (int j0 = first; each > 0 && j0 < m; j0 += min(group, m - j0)) {
        const int pieces = min(group, m - j0) * each;
        for (int base = 0; base < pieces; base += kWave) {
            uint4 x[kKeepBatch], *to[kKeepBatch];
#pragma unroll
            for (int i = 0; i < kKeepBatch; ++i) {
                const int item = base + i * kKeepThreads + tid;
                to[i] = nullptr;
                if (item < pieces) {
                    const int t = item / each, rest = item - t * each, h = rest / vecs, c = rest - h * vecs;
                    x[i] = *at(prefix + kept[j0 + t], h, c);
                    to[i] = at(prefix + j0 + t, h, c);
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kKeepBatch; ++i)
                if (to[i] != nullptr)
                    *to[i] = x[i];
        }
    }
}

// ------------------------------------------------------------------ fork
constexpr int kForkThreads = 1024;
constexpr int kForkWarps = kForkThreads / 32;
constexpr int kForkSmall = 4096;
constexpr int kForkRecount = 32 * kForkThreads;
constexpr int kForkBatch = 2;  // 32-column runs of rows that a warp has in flight

// The sequences' lists, in range, and what follows from them.  Every block has
// all of them, in shared memory where they fit, else in its own part of the
// workspace.
struct Seqs {
    int *parent;  // -1: none
    int *base;    // the parent's keys
    int *total;   // keys afterwards
    int *heir;    // of a parent: the child that keeps its pages, -1: itself
    int *given;   // where its new pages begin among all that are given out
};

// Exclusive prefix over the block's threads, and the total.
__device__ __noinline__ int block_prefix(int x, int *scratch, int &total)
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
    int w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        w += lane >= o ? y : 0;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return incl - x + (warp > 0 ? before : 0);
}
static_assert(kForkWarps == 32, "a warp scans the warps' sums");

// The lists, by one cluster of blocks that meet between the steps (or one block,
// where they are short).  What another block has written is read past the
// first-level cache.
__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(const KvForkArgs a)
{
    extern __shared__ int shared[];
    __shared__ int scratch[kForkWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x, ranks = gridDim.x;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int all = rank * kForkThreads + tid, threads = ranks * kForkThreads;
    grid_launch_dependents();
    grid_dependency_wait();
    auto meet = [&]() {
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    int *mem = a.in_shared ? shared : a.seqs + static_cast<long long>(rank) * 5 * a.B;
    const Seqs s{mem, mem + a.B, mem + 2LL * a.B, mem + 3LL * a.B, mem + 4LL * a.B};
    const int page = 1 << a.page_shift;
    const long long max_keys = static_cast<long long>(a.max_pages) << a.page_shift;
    auto heir_of = [&](int p) { return *static_cast<volatile int *>(&s.heir[p]); };
    auto keeps = [&](int b, int p) { return p >= 0 && (p == b || heir_of(p) == b); };
    auto in_pool = [&](int e) { return e >= 0 && e < a.num_pages; };
    bool bad = false;
    // 1. The lists, checked; each parent's heir; copies of what is overwritten in
    // place, and the counts.
    for (int b = tid; b < a.B; b += kForkThreads) {
        const int p = a.parents != nullptr ? a.parents[b] : b;
        const bool stray = p < -1 || p >= a.B;
        s.parent[b] = stray ? b : p;
        const int L = a.kv_len[b];
        const long long n = a.cu_q != nullptr ? static_cast<long long>(a.cu_q[b + 1]) - a.cu_q[b] : 0;
        s.total[b] = static_cast<int>(min(max(n, 0LL), max_keys));  // of the new tokens, so far
        s.given[b] = static_cast<int>(min(max(static_cast<long long>(L), 0LL), max_keys));  // own keys
        s.heir[b] = 0x7fffffff;
        bad = bad || stray || s.given[b] != L || s.total[b] != n;
    }
    const int *old_table = a.page_table;
    long long old_stride = a.table_stride;
    if (a.staged) {
        const long long cells = static_cast<long long>(a.B) * a.max_pages;
        for (long long i = all; i < cells; i += threads) {
            const long long b = i / a.max_pages;
            a.stage[i] = a.page_table[b * a.table_stride + (i - b * a.max_pages)];
        }
        old_table = a.stage;
        old_stride = a.max_pages;
    }
    if (a.refs_out != a.refs)
        for (int i = all; i < a.num_pages; i += threads)
            a.refs_out[i] = a.refs[i];
    __syncthreads();
    for (int b = tid; b < a.B; b += kForkThreads) {
        const int p = s.parent[b];
        if (p >= 0)
            atomicMin(&s.heir[p], p == b ? -1 : b);
        const int base = p >= 0 ? s.given[p] : 0;
        const long long total = static_cast<long long>(base) + s.total[b];
        s.base[b] = base;
        s.total[b] = static_cast<int>(min(total, max_keys));
        bad = bad || total > max_keys;
    }
    meet();
    // 2. The new rows as far as they follow from the old ones, and the counts: the
    // block's own rows, a warp some runs of 32 columns at a time.
    const int row0 = static_cast<int>(static_cast<long long>(a.B) * rank / ranks);
    const int row1 = static_cast<int>(static_cast<long long>(a.B) * (rank + 1) / ranks);
    const int runs = (a.max_pages + 31) / 32;
    const long long items = static_cast<long long>(row1 - row0) * runs;
    for (long long i0 = static_cast<long long>(warp) * kForkBatch; i0 < items; i0 += kForkWarps * kForkBatch) {
        int mine[kForkBatch], theirs[kForkBatch], row[kForkBatch], col[kForkBatch];
        int at = static_cast<int>(i0 / runs), run = static_cast<int>(i0 - static_cast<long long>(at) * runs);
#pragma unroll
        for (int k = 0; k < kForkBatch; ++k) {
            mine[k] = theirs[k] = -1;
            const int b = row[k] = row0 + at, c = col[k] = run * 32 + lane;
            if (++run == runs) {
                run = 0;
                ++at;
            }
            if (i0 + k < items && c < a.max_pages) {
                const int p = s.parent[b];
                mine[k] = __ldcg(&old_table[b * old_stride + c]);
                if (p >= 0)
                    theirs[k] = p == b ? mine[k] : __ldcg(&old_table[p * old_stride + c]);
            }
        }
#pragma unroll
        for (int k = 0; k < kForkBatch; ++k) {
            const int b = row[k], c = col[k];
            if (i0 + k >= items || c >= a.max_pages)
                continue;
            const int p = s.parent[b], base = s.base[b], whole = base >> a.page_shift;
            const bool kept = keeps(b, p);
            const int e = in_pool(theirs[k]) && (kept || c < whole) ? theirs[k] : -1;
            a.table_out[b * a.table_out_stride + c] = e;
            if (p != b) {
                if (in_pool(mine[k]))
                    atomicSub(&a.refs_out[mine[k]], 1);
                if (e >= 0)
                    atomicAdd(&a.refs_out[e], 1);
            }
            // An entry of no page, or none where the parent has keys.
            bad = bad || (mine[k] != -1 && !in_pool(mine[k])) ||
                  (p >= 0 && static_cast<long long>(c) * page < base && !in_pool(theirs[k]));
        }
    }
    // How many pages each sequence lacks behind its whole ones, and where those
    // begin among all that are given out: every block for all sequences.
    int need = 0;
    for (int b0 = 0; b0 < a.B; b0 += kForkThreads) {
        const int b = b0 + tid;
        int lacks = 0, sum;
        if (b < a.B) {
            const int p = s.parent[b], whole = s.base[b] >> a.page_shift;
            const int want = static_cast<int>((static_cast<long long>(s.total[b]) + page - 1) >> a.page_shift);
            lacks = want - whole;
            if (keeps(b, p))
                for (int c = whole; c < want; ++c)
                    lacks -= in_pool(__ldcg(&old_table[p * old_stride + c]));
        }
        const int k = block_prefix(lacks, scratch, sum);
        if (b < a.B)
            s.given[b] = need + k;
        need += sum;
    }
    meet();
    // 3. The free pages in each block's part of them.
    int have = 0;
    if (need > 0) {
        const int page0 = static_cast<int>(static_cast<long long>(a.num_pages) * rank / ranks);
        const int page1 = static_cast<int>(static_cast<long long>(a.num_pages) * (rank + 1) / ranks);
        auto free_pages = [&](int from, int to) {
            int n = 0, sum;
#pragma unroll 4
            for (int i = from + tid; i < to; i += kForkThreads)
                n += __ldcg(&a.refs_out[i]) == 0;
            block_prefix(n, scratch, sum);
            return sum;
        };
        // Those of the blocks before: counted again while that is less than
        // another meeting.
        int at = 0;
        if (rank > 0 && a.num_pages <= kForkRecount) {
            at = free_pages(0, page0);
        } else if (ranks > 1 && a.num_pages > kForkRecount) {
            const int n = free_pages(page0, page1);
            if (tid == 0)
                a.counts[rank] = n;
            meet();
            for (int r = 0; r < rank; ++r)
                at += __ldcg(&a.counts[r]);
        }
        for (int i0 = page0; i0 < page1 && at < need; i0 += kForkThreads) {
            const int i = i0 + tid;
            const bool is = i < page1 && __ldcg(&a.refs_out[i]) == 0;
            int found;
            const int k = at + block_prefix(is ? 1 : 0, scratch, found);
            if (is && k < need)
                a.free_list[k] = i;
            at += found;
        }
        // Known to the last block: all that are needed, or all there are.
        if (tid == 0 && rank == ranks - 1)
            a.counts[kForkRanks] = min(at, need);
        meet();
        have = __ldcg(&a.counts[kForkRanks]);
    }
    // 4. The lacking entries, in order, and what is to be copied.
    for (int b = row0 + warp; b < row1; b += kForkWarps) {
        const int p = s.parent[b], base = s.base[b], whole = base >> a.page_shift, part = base & (page - 1);
        const int want = static_cast<int>((static_cast<long long>(s.total[b]) + page - 1) >> a.page_shift);
        const bool kept = keeps(b, p);
        int *row = a.table_out + b * a.table_out_stride;
        const int *old = old_table + max(p, 0) * old_stride;
        int k = s.given[b];
        if (lane == 0) {
            a.len_out[b] = s.total[b];
            // A partly filled page of a parent's that another child keeps.
            const int src = p >= 0 && !kept && part > 0 ? __ldcg(&old[whole]) : -1;
            a.copies[b] = make_int4(src, in_pool(src) && k < have ? __ldcg(&a.free_list[k]) : -1, part, 0);
        }
        for (int c0 = whole; c0 < want; c0 += 32) {
            const int c = c0 + lane;
            const bool lack = c < want && !(kept && in_pool(__ldcg(&old[c])));
            const unsigned who = __ballot_sync(0xffffffffu, lack);
            if (lack) {
                const int at = k + __popc(who & ((1u << lane) - 1u));
                if (at < have) {
                    const int x = __ldcg(&a.free_list[at]);
                    row[c] = x;
                    a.refs_out[x] = 1;
                } else {
                    bad = true;
                }
            }
            k += __popc(who);
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
cudaError_t start(void (*kernel)(Args), const Args &a, long long blocks, int threads, int cluster, size_t smem,
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
    cfg.dynamicSmemBytes = smem;
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
    a.chunks = pieces <= kKeepThreads * kKeepBatch ? 1 : pieces <= 4 * kKeepThreads * kKeepBatch ? 2 : 4;
    a.heads_per_chunk = (a.H + a.chunks - 1) / a.chunks;
    return start(kv_keep_kernel, a, 2LL * a.B * a.chunks, kKeepThreads, 2 * a.chunks, 0, stream);
}

cudaError_t launch_kv_fork(const KvForkArgs &args, cudaStream_t stream)
{
    KvForkArgs a = args;
    // One block up to some thousand entries: its barriers are shorter than a
    // cluster's, which has more hands for long lists.
    const long long entries = static_cast<long long>(a.B) * a.max_pages + a.num_pages;
    const int ranks = entries <= kForkSmall ? 1 : kForkRanks;
    // The sequences' lists fit shared memory without asking for more of it.
    const size_t lists = static_cast<size_t>(a.B) * 5 * sizeof(int);
    a.in_shared = lists <= 40960;
    cudaError_t e = start(kv_fork_kernel, a, ranks, kForkThreads, ranks, a.in_shared ? lists : 0, stream);
    if (e != cudaSuccess || a.parents == nullptr || a.H == 0)
        return e;
    const long long pieces = static_cast<long long>(a.H) * ((1 << a.page_shift) - 1) * (a.d / 8);
    a.chunks = static_cast<int>((pieces + kCopyThreads * kCopyBatch - 1) / (kCopyThreads * kCopyBatch));
    return start(kv_fork_copy_kernel, a, 2LL * a.B * a.chunks, kCopyThreads, 1, 0, stream);
}

}  // namespace fattn
