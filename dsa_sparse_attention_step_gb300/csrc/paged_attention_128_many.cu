// paged_attention_128_many.cu -- the paged attention kernels for 128 head dims and requests
// of several tokens.
#include "paged_attention.cuh"

namespace dsa {

cudaError_t launch_paged_attention_128_many(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                            int format, int* launches, cudaStream_t stream) {
    return paged::launch_dim<128, true>(p, cache, format, launches, stream);
}

}  // namespace dsa
