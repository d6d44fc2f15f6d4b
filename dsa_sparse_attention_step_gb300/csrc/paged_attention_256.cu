// paged_attention_256.cu -- the paged attention kernels for 256 head dims and requests of one
// token.
#include "paged_attention.cuh"

namespace dsa {

cudaError_t launch_paged_attention_256(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                     int format, int* launches, cudaStream_t stream) {
    return paged::launch_dim<256, false>(p, cache, format, launches, stream);
}

}  // namespace dsa
