// quant_attention_tc_64.cu -- the tcgen05 kernels of quant_attention_tc.cuh for 64 head dims.
#include "quant_attention_tc.cuh"

namespace dsa {

cudaError_t launch_quant_attention_tc_64(const paged::AttnParams& p, const dsa_kv_cache& cache,
                                        int format, bool int8, int* launches,
                                        cudaStream_t stream) {
    return int8 ? paged::launch_tensor<64, paged::kCodeInt8>(p, cache, format, launches, stream)
                : paged::launch_tensor<64, paged::kCodeE4m3>(p, cache, format, launches, stream);
}

}  // namespace dsa
