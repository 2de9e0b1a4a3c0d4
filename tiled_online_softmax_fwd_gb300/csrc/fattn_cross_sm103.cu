// fattn_cross_sm103.cu -- cross attention: batched queries over the contiguous
// keys and values of sequences of other lengths (see paged_sm103.cuh).
#include "paged_sm103.cuh"

namespace fattn {

cudaError_t launch_cross(const PagedArgs &a, const PagedMaps &maps, int num_sms, cudaStream_t stream)
{
    return launch_mode<kCross>(a, maps, num_sms, stream);
}

}  // namespace fattn
