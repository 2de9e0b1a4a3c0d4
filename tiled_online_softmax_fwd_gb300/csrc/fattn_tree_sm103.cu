// fattn_tree_sm103.cu -- trees of drafted tokens: attention over a paged cache
// with a mask among the new tokens (see paged_sm103.cuh), and the masks and
// positions that follow from each token's parent.
#include "paged_sm103.cuh"

namespace fattn {
namespace {

// A block a sequence, a thread a token: it walks to the tree's root, and sets
// the bit of every token on the way.  Parents come before their children, so
// the words of a row are finished from the last to the first and each is
// written once.  Bound by latency: a step of the walk waits for the one before,
// as many as the tree is deep.  So the parents are brought into shared memory
// first (trees that do not fit it are walked in the caches).  24 trees of up to 200
// tokens, some 57 deep: 13.2 us in the caches, 4 so.
constexpr int kMaskThreads = 256;
constexpr int kMaskShared = 4096;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const TreeMaskArgs a)
{
    __shared__ int near[kMaskShared];
    grid_launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x;
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], L = a.kv_len[b];
    const int q0 = min(max(c0, 0), a.T);
    const int all = min(max(c1, q0), a.T) - q0;
    const int n = static_cast<int>(min(static_cast<long long>(all), 32LL * a.words));
    bool bad = q0 != c0 || n != static_cast<long long>(c1) - c0 || (b == 0 && c0 != 0);
    const int *parents = a.parents + q0;
    if (n <= kMaskShared) {
        for (int i = threadIdx.x; i < n; i += kMaskThreads)
            near[i] = parents[i];
        __syncthreads();
        parents = near;
    }
    for (int i = threadIdx.x; i < n; i += kMaskThreads) {
        unsigned *row = a.mask + (static_cast<long long>(q0) + i) * a.words;
        int w = a.words - 1, depth = 0;
        unsigned bits = 0;
        for (int at = i;;) {
            for (; w > at >> 5; --w, bits = 0)
                row[w] = bits;
            bits |= 1u << (at & 31);
            const int p = parents[at];
            if (p < 0 || p >= at) {
                bad = bad || p != -1;
                break;
            }
            at = p;
            ++depth;
        }
        for (; w >= 0; --w, bits = 0)
            row[w] = bits;
        a.positions[q0 + i] = L - all + depth;
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
