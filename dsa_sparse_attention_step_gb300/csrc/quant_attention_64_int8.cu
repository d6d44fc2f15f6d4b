// quant_attention_64_int8.cu -- the paged attention kernels for 64 head dims held as INT8 codes
// with a scale for every 16 tokens.
#include "paged_attention.cuh"

namespace dsa {

cudaError_t launch_quant_attention_64_int8(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                        int format, int* launches, cudaStream_t stream) {
    return paged::launch_codes<64, paged::kCodeInt8, false>(p, cache, format, launches, stream);
}

}  // namespace dsa
