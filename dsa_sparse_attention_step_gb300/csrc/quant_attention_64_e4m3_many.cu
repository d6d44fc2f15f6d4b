// quant_attention_64_e4m3_many.cu -- the paged attention kernels for 64 head dims held as E4M3
// codes with a scale for every 16 tokens, and requests of several tokens.
#include "paged_attention.cuh"

namespace dsa {

cudaError_t launch_quant_attention_64_e4m3_many(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                        int format, int* launches, cudaStream_t stream) {
    return paged::launch_codes<64, paged::kCodeE4m3, true>(p, cache, format, launches, stream);
}

}  // namespace dsa
