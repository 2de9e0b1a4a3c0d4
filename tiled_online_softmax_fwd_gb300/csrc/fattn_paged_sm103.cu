// fattn_paged_sm103.cu -- attention of new tokens over a paged cache, causal or
// full (see paged_sm103.cuh).
#include "paged_sm103.cuh"

namespace fattn {

cudaError_t launch_paged(const PagedArgs &a, const PagedMaps &maps, int num_sms, cudaStream_t stream)
{
    return launch_mode<kPaged>(a, maps, num_sms, stream);
}

}  // namespace fattn
