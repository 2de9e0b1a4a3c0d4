// fattn_tree_sm103.cu -- trees of drafted tokens: attention over a paged cache
// with a mask among the new tokens (see paged_sm103.cuh), and the masks and
// positions that follow from each token's parent.
#include "paged_sm103.cuh"

namespace fattn {
namespace {

// A block a sequence, a thread a token.  Parents come before their children.  What
// a token sees among its own 32 (a warp's) follows from the others of them in five
// steps of twice the length: each lane takes over the tokens, and the one to go on
// from, of the lane that it has come to.  Then its path is walked 32 tokens at a
// step, and the words of its row are written from the last to the first, each once.
// Bound by latency: 24 trees of up to 200 tokens, some 57 deep, 3.6 us (walked
// token by token 9.3 us).  A tree beyond the shared memory is walked so.
constexpr int kMaskThreads = 256;
constexpr int kMaskTokens = 4096;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const TreeMaskArgs a)
{
    __shared__ unsigned own[kMaskTokens];  // of its 32, those that a token sees
    __shared__ int before[kMaskTokens];    // and the first before them, or -1
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = blockIdx.x, lane = threadIdx.x % 32;
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], L = a.kv_len[b];
    const int q0 = min(max(c0, 0), a.T);
    const int all = min(max(c1, q0), a.T) - q0;
    const int n = static_cast<int>(min(static_cast<long long>(all), 32LL * a.words));
    bool bad = q0 != c0 || n != static_cast<long long>(c1) - c0 || (b == 0 && c0 != 0) || L < all;
    const int prefix = L > all ? L - all : 0;  // keys before the new tokens
    const int *parents = a.parents + q0;
    auto parent_of = [&](int i) {
        const int p = parents[i];
        return p < 0 || p >= i ? -1 : p;
    };
    for (int i0 = threadIdx.x - lane; i0 < n; i0 += kMaskThreads) {
        const int i = i0 + lane, given = i < n ? parents[i] : -1;
        const int p = given < 0 || given >= i ? -1 : given;
        bad = bad || p != given;
        if (n > kMaskTokens)
            continue;
        unsigned sees = 1u << lane;
        int next = p >= i0 ? p - i0 : -1;  // among the 32
        int out = next >= 0 ? -1 : p;
#pragma unroll
        for (int step = 0; step < 5; ++step) {
            const int from = next >= 0 ? next : lane;
            const unsigned s = __shfl_sync(0xffffffffu, sees, from);
            const int m = __shfl_sync(0xffffffffu, next, from), e = __shfl_sync(0xffffffffu, out, from);
            if (next >= 0) {
                sees |= s;
                out = e;
                next = m;
            }
        }
        if (i < n) {
            own[i] = sees;
            before[i] = out;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kMaskThreads) {
        unsigned *row = a.mask + (static_cast<long long>(q0) + i) * a.words;
        int w = a.words - 1, tokens = 0;
        unsigned bits = 0;
        for (int at = i; at >= 0;) {
            for (; w > at >> 5; --w, bits = 0)
                row[w] = bits;
            const unsigned s = n <= kMaskTokens ? own[at] : 1u << (at & 31);
            bits |= s;
            tokens += __popc(s);
            at = n <= kMaskTokens ? before[at] : parent_of(at);
        }
        for (; w >= 0; --w, bits = 0)
            row[w] = bits;
        a.positions[q0 + i] = prefix + tokens - 1;
    }
    if (bad)
        atomicCAS(a.status, 0u, 6u /* FATTN_ERR_INDEX */ | (kRoleTree << 8));
}

}  // namespace

cudaError_t launch_tree(const PagedArgs &a, const PagedMaps &maps, int num_sms, cudaStream_t stream)
{
    return launch_mode<kTree>(a, maps, num_sms, stream);
}

cudaError_t launch_tree_mask(const TreeMaskArgs &a, cudaStream_t stream)
{
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.B);
    cfg.blockDim = dim3(kMaskThreads);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_mask_kernel, a);
}

}  // namespace fattn
