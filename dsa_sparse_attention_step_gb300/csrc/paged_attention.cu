// paged_attention.cu -- workspace, limits and dispatch of the paged attention
// kernels (paged_attention.cuh), which are compiled per head dim.
#include "paged_attention.cuh"

namespace dsa {

using namespace paged;

// _many: for requests of several tokens (kMany).
using Launch = cudaError_t(const AttnParams& p, const dsa_kv_cache& cache, int format,
                           int* launches, cudaStream_t stream);
Launch launch_paged_attention_64, launch_paged_attention_128, launch_paged_attention_256;
Launch launch_paged_attention_64_many, launch_paged_attention_128_many,
    launch_paged_attention_256_many;

// Positions in the list of key tiles are 32-bit (kUnitCost is at most 8).
bool paged_attention_supported(const BatchArgs& bt, int kv_heads, int group) {
    const double tiles = ((double)bt.max_seq + kPage - 1) / kPage;
    return most_units(bt, kv_heads, group, 16) * (tiles + 1 + 8) < 2147483648.0;
}

// The factor of q . k codes, in units of log2.
float paged_score_scale(float sm_scale, const dsa_kv_cache& cache) {
    return sm_scale * cache.k_scale * kLog2e;
}

// Of the default plan, which needs more than the whole one.
size_t paged_attention_workspace_bytes(int64_t max_rows, int head_dim) {
    return ws_layout(head_dim, row_tile(head_dim, max_rows, false)).total;
}

cudaError_t launch_paged_attention(const BatchArgs& bt, const dsa_kv_cache& cache, int format,
                                   int num_q_heads, const void* q, int64_t q_stride,
                                   float sm_scale, void* out, float* lse, void* ws, bool whole,
                                   bool wait_test, int32_t* status, int* launches,
                                   cudaStream_t stream) {
    AttnParams p;
    p.bt = bt;
    p.kv_heads = cache.num_kv_heads;
    p.group = num_q_heads / cache.num_kv_heads;
    p.inv_group = 1.0f / (float)p.group;
    p.whole = whole;
    p.withhold = wait_test;
    p.min_length = p.cluster = p.row_tiles = 0;  // set by the launch
    p.q_stride = q_stride;
    p.q = q;
    p.v_pages = cache.v_pages;
    p.out = out;
    p.lse = lse;
    p.score_scale = paged_score_scale(sm_scale, cache);
    p.v_scale = cache.v_scale;
    const WsLayout w = ws_layout(
        cache.head_dim, row_tile(cache.head_dim, (int64_t)bt.max_q * p.group, false));
    uint8_t* base = static_cast<uint8_t*>(ws);
    p.part_o = reinterpret_cast<float*>(base);
    p.part_ml = reinterpret_cast<float*>(base + w.ml);
    p.joins = reinterpret_cast<int32_t*>(base + w.joins);
    p.status = status;
    *launches = 1;
    // a request's results may not depend on the others' token counts when it runs whole
    const bool many = bt.max_q > 1 || whole;
    Launch* launch;
    switch (cache.head_dim) {
        case 64: launch = many ? launch_paged_attention_64_many : launch_paged_attention_64; break;
        case 128:
            launch = many ? launch_paged_attention_128_many : launch_paged_attention_128;
            break;
        default: launch = many ? launch_paged_attention_256_many : launch_paged_attention_256;
    }
    return launch(p, cache, format, launches, stream);
}

}  // namespace dsa
