// paged_attention_128.cu -- the paged attention kernels for 128 head dims and requests of one
// token.
#include "paged_attention.cuh"

namespace dsa {

cudaError_t launch_paged_attention_128(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                     int format, int* launches, cudaStream_t stream) {
    return paged::launch_dim<128, false>(p, cache, format, launches, stream);
}

}  // namespace dsa
