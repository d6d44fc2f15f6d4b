// paged_attention.cu -- workspace, limits and dispatch of the paged attention
// kernels (paged_attention.cuh), which are compiled per head dim.
#include "quant_attention_tc.cuh"

namespace dsa {

using namespace paged;

// The parameters that do not depend on how the cache holds its elements; part_rows: rows of
// a tile that pieces are kept for.
AttnParams attention_params(const BatchArgs& bt, int kv_heads, int head_dim, int num_q_heads,
                            const void* q, int64_t q_stride, void* out, float* lse, void* ws,
                            int part_rows, bool whole, bool wait_test, int32_t* status) {
    AttnParams p;
    p.bt = bt;
    p.kv_heads = kv_heads;
    p.group = num_q_heads / kv_heads;
    p.inv_group = 1.0f / (float)p.group;
    p.whole = whole;
    p.withhold = wait_test;
    p.min_length = p.cluster = p.row_tiles = 0;  // set by the launch
    p.q_stride = q_stride;
    p.q = q;
    p.scales = nullptr;
    p.out = out;
    p.lse = lse;
    const WsLayout w = ws_layout(head_dim, part_rows);
    uint8_t* base = static_cast<uint8_t*>(ws);
    p.part_o = reinterpret_cast<float*>(base);
    p.part_ml = reinterpret_cast<float*>(base + w.ml);
    p.joins = reinterpret_cast<int32_t*>(base + w.joins);
    p.status = status;
    return p;
}

using Launch = cudaError_t(const AttnParams& p, const dsa_kv_cache& cache, int format,
                           int* launches, cudaStream_t stream);
// _many: for requests of several tokens (kMany).
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
    const int64_t rows = (int64_t)bt.max_q * (num_q_heads / cache.num_kv_heads);
    AttnParams p = attention_params(bt, cache.num_kv_heads, cache.head_dim, num_q_heads, q,
                                    q_stride, out, lse, ws, row_tile(cache.head_dim, rows, false),
                                    whole, wait_test, status);
    p.v_pages = cache.v_pages;
    p.score_scale = paged_score_scale(sm_scale, cache);
    p.v_scale = cache.v_scale;
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

Launch launch_quant_attention_64_e4m3, launch_quant_attention_128_e4m3,
    launch_quant_attention_256_e4m3;
Launch launch_quant_attention_64_e4m3_many, launch_quant_attention_128_e4m3_many,
    launch_quant_attention_256_e4m3_many;
Launch launch_quant_attention_64_int8, launch_quant_attention_128_int8,
    launch_quant_attention_256_int8;

using TensorLaunch = cudaError_t(const AttnParams& p, const dsa_kv_cache& cache, int format,
                                 bool int8, int* launches, cudaStream_t stream);
TensorLaunch launch_quant_attention_tc_64, launch_quant_attention_tc_128,
    launch_quant_attention_tc_256;

float quant_score_scale(float sm_scale) { return sm_scale * kLog2e; }

// Rows of a tile whose pieces the workspace has room for, whatever the switch says.
static int quant_part_rows(const BatchArgs& bt, int num_q_heads, int kv_heads, int head_dim) {
    return takes_tensor_cores(bt, num_q_heads, kv_heads, head_dim, false)
               ? 128
               : row_tile(head_dim, (int64_t)bt.max_q * (num_q_heads / kv_heads), false);
}

size_t quant_attention_workspace_bytes(const BatchArgs& bt, int num_q_heads, int kv_heads,
                                       int head_dim) {
    return ws_layout(head_dim, quant_part_rows(bt, num_q_heads, kv_heads, head_dim)).total;
}

cudaError_t launch_quant_attention(const BatchArgs& bt, const dsa_quant_cache& cache, int format,
                                   int num_q_heads, const void* q, int64_t q_stride,
                                   float sm_scale, void* out, float* lse, void* ws, bool whole,
                                   bool wait_test, int32_t* status, int* launches,
                                   cudaStream_t stream) {
    AttnParams p = attention_params(
        bt, cache.num_kv_heads, cache.head_dim, num_q_heads, q, q_stride, out, lse, ws,
        quant_part_rows(bt, num_q_heads, cache.num_kv_heads, cache.head_dim), whole,
        wait_test, status);
    p.v_pages = cache.v_pages;
    p.scales = cache.scales;
    p.score_scale = quant_score_scale(sm_scale);
    p.v_scale = 1.f;
    *launches = 1;
    // the pools as bytes
    const dsa_kv_cache bytes = {cache.num_pages, cache.num_kv_heads, cache.head_dim,
                                DSA_KV_FP8_E4M3, cache.k_pages, cache.v_pages, 1.f, 1.f};
    const bool int8 = cache.format == DSA_QUANT_INT8;
    if (takes_tensor_cores(bt, num_q_heads, cache.num_kv_heads, cache.head_dim, whole)) {
        TensorLaunch* launch = cache.head_dim == 64    ? launch_quant_attention_tc_64
                               : cache.head_dim == 128 ? launch_quant_attention_tc_128
                                                       : launch_quant_attention_tc_256;
        return launch(p, bytes, format, int8, launches, stream);
    }
    const bool many = bt.max_q > 1 || whole;
    Launch* launch;
    switch (cache.head_dim) {
        case 64:
            launch = int8   ? launch_quant_attention_64_int8
                     : many ? launch_quant_attention_64_e4m3_many
                            : launch_quant_attention_64_e4m3;
            break;
        case 128:
            launch = int8   ? launch_quant_attention_128_int8
                     : many ? launch_quant_attention_128_e4m3_many
                            : launch_quant_attention_128_e4m3;
            break;
        default:
            launch = int8   ? launch_quant_attention_256_int8
                     : many ? launch_quant_attention_256_e4m3_many
                            : launch_quant_attention_256_e4m3;
    }
    return launch(p, bytes, format, launches, stream);
}

}  // namespace dsa
