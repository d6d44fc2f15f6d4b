// quant_attention_128_e4m3.cu -- the paged attention kernels for 128 head dims held as E4M3 codes
// with a scale for every 16 tokens, and requests of one token.
#include "paged_attention.cuh"

namespace dsa {

cudaError_t launch_quant_attention_128_e4m3(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                        int format, int* launches, cudaStream_t stream) {
    return paged::launch_codes<128, paged::kCodeE4m3, false>(p, cache, format, launches, stream);
}

}  // namespace dsa
