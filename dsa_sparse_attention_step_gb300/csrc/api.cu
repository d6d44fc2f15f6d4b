// api.cu -- the extern "C" boundary of libdsa.so: argument validation,
// workspace arithmetic and kernel launches.  See include/dsa.h.
#include <atomic>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "../../include/dsa_testing.h"

namespace dsa {
cudaError_t launch_index_scores(const BatchArgs& bt, const uint8_t* q8, const float* qscale,
                                const float* w, const void* pages, int key_format,
                                float* scores, int64_t ld, int32_t* status, cudaStream_t stream);
bool indexer_supported(const BatchArgs& bt);
cudaError_t launch_topk(const BatchArgs& bt, const float* scores, int64_t ld, int K,
                        int32_t* out, void* ws, bool pdl, cudaStream_t stream);
size_t topk_workspace_bytes(int total_q, int max_seq);
int topk_launches(int total_q, int max_seq);
bool topk_supported(int max_seq);
cudaError_t launch_sparse_mla(const BatchArgs& bt, const uint16_t* q_lat, const void* latent_pages,
                              float kv_scale, float sm_scale, const int32_t* indices, int K,
                              uint16_t* out, float* lse, void* ws, int32_t* status, bool pdl,
                              cudaStream_t stream, bool wait_test, int latent_format,
                              bool whole_only);
size_t sparse_mla_workspace_bytes(int total_q, int K);
int sparse_mla_launches(int total_q, int K, bool whole_only);
cudaError_t launch_append_cache(const BatchArgs& bt, const float* keys, const float* lat,
                                float kv_scale, void* index_pages, void* latent_pages,
                                int32_t* status, cudaStream_t stream);

int dcp_default_cand(int world, int K);
struct DcpWs {
    size_t sent, sent_n, full, full_n, flags, total;
};
DcpWs dcp_ws_layout(int total_q, int world, int cand, int K);
bool dcp_supported(int world, int max_seq);
cudaError_t launch_dcp_topk(const BatchArgs& bt, const float* scores, int64_t ld, int world,
                            int cand, int K, int32_t* indices, int32_t* rank_indices,
                            int32_t* resent, void* ws, cudaStream_t stream);
cudaError_t launch_lse_combine(int total_q, int world, const uint16_t* part, const float* part_lse,
                               uint16_t* out, float* lse, cudaStream_t stream);

cudaError_t launch_indexer_front(const BatchArgs& bt, const uint16_t* q_c, const uint16_t* x,
                                 const uint16_t* w_q, const uint16_t* w_k, const uint16_t* w_w,
                                 uint8_t* q8, float* qscale, float* w, void* index_pages,
                                 float* q_f32, float* k_f32, int32_t* status, cudaStream_t stream);

bool build_tables_supported(int num_requests);
cudaError_t launch_build_tables(int num_requests, const int32_t* cached, const int32_t* added,
                                const int32_t* free_pages, int num_free, int num_pages,
                                int max_pages, int max_tokens, int32_t* block_table,
                                int32_t* q_offsets, int32_t* seq_lens, int64_t* slots,
                                int32_t* positions, int32_t* token_requests, int32_t* pages_taken,
                                int32_t* status, cudaStream_t stream);
cudaError_t launch_rope_append(int num_tokens, const dsa_kv_cache& cache, int format,
                               const dsa_rope& rope, const int32_t* positions,
                               const int64_t* slots, int num_q_heads, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, void* q_out, int64_t q_out_stride,
                               int32_t* status, cudaStream_t stream);

bool paged_attention_supported(const BatchArgs& bt, int kv_heads, int group);
float paged_score_scale(float sm_scale, const dsa_kv_cache& cache);
size_t paged_attention_workspace_bytes(int64_t max_rows, int head_dim);
cudaError_t launch_paged_attention(const BatchArgs& bt, const dsa_kv_cache& cache, int format,
                                   int num_q_heads, const void* q, int64_t q_stride,
                                   float sm_scale, void* out, float* lse, void* ws, bool whole,
                                   bool wait_test, int32_t* status, int* launches,
                                   cudaStream_t stream);

std::atomic<uint64_t> g_launches{0};
std::atomic<int32_t> g_batch_invariant{0};  // dsa_set_batch_invariant
}  // namespace dsa

using namespace dsa;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// padded: requests may have more query rows than context (or none at all).
dsa_status check_batch(const dsa_batch* bt, bool padded = false) {
    if (bt == nullptr) return DSA_ERR_INVALID_ARG;
    if (bt->page_size != kPage) return DSA_ERR_UNSUPPORTED;
    if (bt->num_requests < 1 || bt->total_q < 0 || bt->max_q_per_request < 0 ||
        bt->max_seq_len < (padded ? 0 : 1) || bt->num_pages < 1 || bt->max_pages < 1)
        return DSA_ERR_INVALID_ARG;
    if ((int64_t)bt->max_pages * kPage < bt->max_seq_len) return DSA_ERR_INVALID_ARG;
    if (!padded && bt->max_q_per_request > bt->max_seq_len) return DSA_ERR_INVALID_ARG;
    if ((int64_t)bt->total_q > (int64_t)bt->num_requests * bt->max_q_per_request)
        return DSA_ERR_INVALID_ARG;
    if (!bt->q_offsets || !bt->seq_lens || !bt->block_table) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

BatchArgs to_args(const dsa_batch* bt) {
    BatchArgs a;
    a.num_requests = bt->num_requests;
    a.total_q = bt->total_q;
    a.max_q = bt->max_q_per_request;
    a.max_seq = bt->max_seq_len;
    a.num_pages = bt->num_pages;
    a.max_pages = bt->max_pages;
    a.q_offsets = bt->q_offsets;
    a.seq_lens = bt->seq_lens;
    a.block_table = bt->block_table;
    return a;
}

inline dsa_status cuda_status(cudaError_t e) {
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline int64_t score_ld_for(const dsa_batch* bt) {
    return (int64_t)align_up((size_t)bt->max_seq_len, 128);
}

dsa_status check_index_args(const dsa_batch* bt, const uint8_t* q8, const float* qscale,
                            const float* w, const void* pages, dsa_key_format fmt,
                            const float* scores, int64_t ld) {
    if (fmt != DSA_KEYS_FP8_E4M3 && fmt != DSA_KEYS_MXFP4) return DSA_ERR_UNSUPPORTED;
    if (!indexer_supported(to_args(bt))) return DSA_ERR_UNSUPPORTED;
    if (!q8 || !qscale || !w || !pages || !scores) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q8) || !aligned16(pages) || !aligned16(scores) || !aligned16(qscale) ||
        !aligned16(w))
        return DSA_ERR_INVALID_ARG;
    if (ld < bt->max_seq_len || (ld % 4) != 0) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

dsa_status check_mla_args(const dsa_batch* bt, const uint16_t* q_lat, const void* lat,
                          const int32_t* indices, int32_t topk, const uint16_t* out,
                          float kv_scale, float sm_scale) {
    (void)bt;
    if (topk != kTopK) return DSA_ERR_UNSUPPORTED;
    if (!q_lat || !lat || !indices || !out) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_lat) || !aligned16(lat) || !aligned16(indices) || !aligned16(out))
        return DSA_ERR_INVALID_ARG;
    if (!(kv_scale > 0.f) || !(sm_scale > 0.f)) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

// A 16-bit cache holds the type of the queries, unscaled; an FP8 cache serves
// both types.
dsa_status check_kv_cache(const dsa_kv_cache* c, dsa_float_format format) {
    if (c == nullptr) return DSA_ERR_INVALID_ARG;
    if (format != DSA_FLOAT_BF16 && format != DSA_FLOAT_F16) return DSA_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DSA_ERR_UNSUPPORTED;
    if (c->format != DSA_KV_FP8_E4M3 &&
        c->format != (format == DSA_FLOAT_BF16 ? DSA_KV_BF16 : DSA_KV_F16))
        return DSA_ERR_UNSUPPORTED;
    if (c->num_pages < 1 || c->num_kv_heads < 1 ||
        (int64_t)c->num_pages * c->num_kv_heads > INT32_MAX)
        return DSA_ERR_INVALID_ARG;
    if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages))
        return DSA_ERR_INVALID_ARG;
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !std::isfinite(c->k_scale) ||
        !std::isfinite(c->v_scale))
        return DSA_ERR_INVALID_ARG;
    if (c->format != DSA_KV_FP8_E4M3 && (c->k_scale != 1.f || c->v_scale != 1.f))
        return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

// Token rows of `heads` heads: 16-byte accesses need 8-element strides.
bool row_ok(const void* p, int64_t stride, int64_t heads, int head_dim) {
    return p && aligned16(p) && stride % 8 == 0 && stride >= heads * head_dim;
}

// An array of `count` elements; whether two of them share bytes.
struct Span {
    uintptr_t begin, end;
    Span(const void* p, int64_t count, size_t size)
        : begin(reinterpret_cast<uintptr_t>(p)), end(p ? begin + (uintptr_t)count * size : begin) {}
};
bool overlap(const Span& a, const Span& b) {
    return a.begin < b.end && b.begin < a.end && a.begin < a.end && b.begin < b.end;
}

constexpr int kMaxHeads = 1 << 14;  // query heads, and KV heads, of one layer

}  // namespace

extern "C" {

const char* dsa_status_string(dsa_status s) {
    switch (s) {
        case DSA_OK: return "ok";
        case DSA_ERR_INVALID_ARG: return "invalid argument";
        case DSA_ERR_UNSUPPORTED: return "unsupported shape or format";
        case DSA_ERR_WORKSPACE: return "workspace too small";
        case DSA_ERR_CUDA: return "CUDA error";
        case DSA_ERR_DEVICE_CHECK: return "device check failed (page id or position out of range)";
        case DSA_ERR_TIMEOUT: return "device wait timed out";
    }
    return "unknown status";
}

int32_t dsa_set_batch_invariant(int32_t enabled) {
    return g_batch_invariant.exchange(enabled != 0 ? 1 : 0);
}

uint64_t dsa_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

dsa_status dsa_index_scores(const dsa_batch* batch, const uint8_t* q_fp8, const float* q_scale,
                            const float* w, const void* index_pages, dsa_key_format key_format,
                            float* scores, int64_t score_ld, int32_t* dev_status,
                            dsa_stream_t stream) {
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    st = check_index_args(batch, q_fp8, q_scale, w, index_pages, key_format, scores, score_ld);
    if (st != DSA_OK) return st;
    if (batch->total_q == 0) return DSA_OK;
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_status(launch_index_scores(to_args(batch), q_fp8, q_scale, w, index_pages,
                                           (int)key_format, scores, score_ld, dev_status,
                                           (cudaStream_t)stream));
}

size_t dsa_topk_workspace_size(const dsa_batch* batch, int32_t topk) {
    if (check_batch(batch) != DSA_OK || topk != kTopK) return 0;
    return topk_workspace_bytes(batch->total_q, batch->max_seq_len);
}

dsa_status dsa_topk(const dsa_batch* batch, const float* scores, int64_t score_ld, int32_t topk,
                    int32_t* indices, void* ws, size_t ws_bytes, dsa_stream_t stream) {
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    if (topk != kTopK || !topk_supported(batch->max_seq_len)) return DSA_ERR_UNSUPPORTED;
    if (!scores || !indices) return DSA_ERR_INVALID_ARG;
    if (!aligned16(scores) || !aligned16(indices) || score_ld < batch->max_seq_len ||
        (score_ld % 4) != 0)
        return DSA_ERR_INVALID_ARG;
    const size_t need = dsa_topk_workspace_size(batch, topk);
    if (ws_bytes < need || (need > 0 && (!ws || !aligned16(ws)))) return DSA_ERR_WORKSPACE;
    if (batch->total_q == 0) return DSA_OK;
    g_launches.fetch_add((uint64_t)topk_launches(batch->total_q, batch->max_seq_len),
                         std::memory_order_relaxed);
    return cuda_status(launch_topk(to_args(batch), scores, score_ld, topk, indices, ws, false,
                                   (cudaStream_t)stream));
}

size_t dsa_sparse_mla_workspace_size(const dsa_batch* batch, int32_t topk) {
    if (check_batch(batch) != DSA_OK || topk != kTopK) return 0;
    return sparse_mla_workspace_bytes(batch->total_q, topk);
}

dsa_status dsa_sparse_mla(const dsa_batch* batch, const uint16_t* q_lat, const void* latent_pages,
                          float kv_scale, float sm_scale, const int32_t* indices, int32_t topk,
                          uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                          int32_t* dev_status, dsa_stream_t stream) {
    return dsa_sparse_mla_ex(batch, q_lat, latent_pages, DSA_LATENT_FP8_E4M3, kv_scale, sm_scale,
                             indices, topk, out, lse, ws, ws_bytes, dev_status, stream);
}

dsa_status dsa_sparse_mla_ex(const dsa_batch* batch, const uint16_t* q_lat,
                             const void* latent_pages, dsa_latent_format latent_format,
                             float kv_scale, float sm_scale, const int32_t* indices, int32_t topk,
                             uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                             int32_t* dev_status, dsa_stream_t stream) {
    if (latent_format != DSA_LATENT_FP8_E4M3 && latent_format != DSA_LATENT_NVFP4)
        return DSA_ERR_UNSUPPORTED;
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    st = check_mla_args(batch, q_lat, latent_pages, indices, topk, out, kv_scale, sm_scale);
    if (st != DSA_OK) return st;
    const size_t need = dsa_sparse_mla_workspace_size(batch, topk);
    if (ws_bytes < need || (need > 0 && (!ws || !aligned16(ws)))) return DSA_ERR_WORKSPACE;
    if (batch->total_q == 0) return DSA_OK;
    const bool whole_only = g_batch_invariant.load(std::memory_order_relaxed) != 0;
    g_launches.fetch_add((uint64_t)sparse_mla_launches(batch->total_q, topk, whole_only),
                         std::memory_order_relaxed);
    return cuda_status(launch_sparse_mla(to_args(batch), q_lat, latent_pages, kv_scale, sm_scale,
                                         indices, topk, out, lse, ws, dev_status, false,
                                         (cudaStream_t)stream, false, (int)latent_format,
                                         whole_only));
}

size_t dsa_decode_workspace_size(const dsa_batch* batch, int32_t topk) {
    if (check_batch(batch) != DSA_OK) return 0;
    size_t scores = align_up((size_t)batch->total_q * score_ld_for(batch) * sizeof(float), 256);
    return scores + align_up(dsa_topk_workspace_size(batch, topk), 256) +
           align_up(dsa_sparse_mla_workspace_size(batch, topk), 256);
}

dsa_status dsa_decode(const dsa_batch* batch, const uint8_t* q_fp8, const float* q_scale,
                      const float* w, const void* index_pages, dsa_key_format key_format,
                      const uint16_t* q_lat, const void* latent_pages, float kv_scale,
                      float sm_scale, int32_t topk, uint16_t* out, float* lse, int32_t* indices,
                      void* ws, size_t ws_bytes, int32_t* dev_status, dsa_stream_t stream) {
    return dsa_decode_ex(batch, q_fp8, q_scale, w, index_pages, key_format, q_lat, latent_pages,
                         DSA_LATENT_FP8_E4M3, kv_scale, sm_scale, topk, out, lse, indices, ws,
                         ws_bytes, dev_status, stream);
}

dsa_status dsa_decode_ex(const dsa_batch* batch, const uint8_t* q_fp8, const float* q_scale,
                         const float* w, const void* index_pages, dsa_key_format key_format,
                         const uint16_t* q_lat, const void* latent_pages,
                         dsa_latent_format latent_format, float kv_scale, float sm_scale,
                         int32_t topk, uint16_t* out, float* lse, int32_t* indices, void* ws,
                         size_t ws_bytes, int32_t* dev_status, dsa_stream_t stream) {
    if (latent_format != DSA_LATENT_FP8_E4M3 && latent_format != DSA_LATENT_NVFP4)
        return DSA_ERR_UNSUPPORTED;
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    const int64_t ld = score_ld_for(batch);
    float* scores = static_cast<float*>(ws);
    st = check_index_args(batch, q_fp8, q_scale, w, index_pages, key_format,
                          scores ? scores : reinterpret_cast<float*>(16), ld);
    if (st != DSA_OK) return st;
    st = check_mla_args(batch, q_lat, latent_pages, indices, topk, out, kv_scale, sm_scale);
    if (st != DSA_OK) return st;
    if (!topk_supported(batch->max_seq_len)) return DSA_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws) || ws_bytes < dsa_decode_workspace_size(batch, topk))
        return DSA_ERR_WORKSPACE;
    if (batch->total_q == 0) return DSA_OK;
    const BatchArgs a = to_args(batch);
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t* base = static_cast<uint8_t*>(ws);
    const size_t off_topk = align_up((size_t)batch->total_q * ld * sizeof(float), 256);
    const size_t off_mla = off_topk + align_up(dsa_topk_workspace_size(batch, topk), 256);
    const bool whole_only = g_batch_invariant.load(std::memory_order_relaxed) != 0;
    g_launches.fetch_add(1 + (uint64_t)topk_launches(batch->total_q, batch->max_seq_len) +
                             (uint64_t)sparse_mla_launches(batch->total_q, topk, whole_only),
                         std::memory_order_relaxed);
    cudaError_t e = launch_index_scores(a, q_fp8, q_scale, w, index_pages, (int)key_format,
                                        scores, ld, dev_status, s);
    // the later kernels only read what the kernel before them writes after
    // their grid-dependency wait, so each may start while its predecessor runs
    if (e == cudaSuccess) e = launch_topk(a, scores, ld, topk, indices, base + off_topk, true, s);
    if (e == cudaSuccess)
        e = launch_sparse_mla(a, q_lat, latent_pages, kv_scale, sm_scale, indices, topk, out, lse,
                              base + off_mla, dev_status, true, s, false, (int)latent_format,
                              whole_only);
    return cuda_status(e);
}

size_t dsa_dcp_topk_workspace_size(const dsa_batch* batch, int32_t world, int32_t cand,
                                   int32_t topk) {
    if (check_batch(batch) != DSA_OK || topk != kTopK || world < 1 || world > 8) return 0;
    if (cand == 0) cand = dcp_default_cand(world, topk);
    if (cand < 1 || cand > topk) return 0;
    return dcp_ws_layout(batch->total_q, world, cand, topk).total;
}

dsa_status dsa_dcp_topk(const dsa_batch* batch, const float* scores, int64_t score_ld,
                        int32_t world, int32_t cand, int32_t topk, int32_t* indices,
                        int32_t* rank_indices, int32_t* resent, void* ws, size_t ws_bytes,
                        dsa_stream_t stream) {
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    if (topk != kTopK) return DSA_ERR_UNSUPPORTED;
    if (world < 1 || world > 8) return DSA_ERR_UNSUPPORTED;
    if (cand == 0) cand = dcp_default_cand(world, topk);
    if (cand < 1 || cand > topk) return DSA_ERR_INVALID_ARG;
    if (!dcp_supported(world, batch->max_seq_len)) return DSA_ERR_UNSUPPORTED;
    if (!scores || !indices || !aligned16(scores) || !aligned16(indices)) return DSA_ERR_INVALID_ARG;
    if ((rank_indices && !aligned16(rank_indices)) || (resent && !aligned16(resent)))
        return DSA_ERR_INVALID_ARG;
    if (score_ld < batch->max_seq_len || (score_ld % 4) != 0) return DSA_ERR_INVALID_ARG;
    const size_t need = dsa_dcp_topk_workspace_size(batch, world, cand, topk);
    if (!ws || !aligned16(ws) || ws_bytes < need) return DSA_ERR_WORKSPACE;
    if (batch->total_q == 0) return DSA_OK;
    g_launches.fetch_add(4, std::memory_order_relaxed);
    return cuda_status(launch_dcp_topk(to_args(batch), scores, score_ld, world, cand, topk,
                                       indices, rank_indices, resent, ws, (cudaStream_t)stream));
}

dsa_status dsa_lse_combine(int32_t total_q, int32_t world, const uint16_t* part_out,
                           const float* part_lse, uint16_t* out, float* lse,
                           dsa_stream_t stream) {
    if (total_q < 0) return DSA_ERR_INVALID_ARG;
    if (world < 1 || world > 8) return DSA_ERR_UNSUPPORTED;
    if (!part_out || !part_lse || !out || !aligned16(part_out) || !aligned16(out))
        return DSA_ERR_INVALID_ARG;
    if (total_q == 0) return DSA_OK;
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_status(launch_lse_combine(total_q, world, part_out, part_lse, out, lse,
                                          (cudaStream_t)stream));
}

dsa_status dsa_indexer_front(const dsa_batch* batch, const uint16_t* q_c, const uint16_t* x,
                             const uint16_t* w_q, const uint16_t* w_k, const uint16_t* w_w,
                             uint8_t* q_fp8, float* q_scale, float* w, void* index_pages,
                             dsa_key_format key_format, float* q_f32, float* k_f32,
                             int32_t* dev_status, dsa_stream_t stream) {
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    if (index_pages && key_format != DSA_KEYS_FP8_E4M3) return DSA_ERR_UNSUPPORTED;
    if (!q_c || !x || !w_q || !w_k || !w_w || !q_fp8 || !q_scale || !w) return DSA_ERR_INVALID_ARG;
    const void* ptrs[] = {q_c, x, w_q, w_k, w_w, q_fp8, q_scale, w};
    for (const void* q : ptrs)
        if (!aligned16(q)) return DSA_ERR_INVALID_ARG;
    if ((index_pages && !aligned16(index_pages)) || (q_f32 && !aligned16(q_f32)) ||
        (k_f32 && !aligned16(k_f32)))
        return DSA_ERR_INVALID_ARG;
    if (batch->total_q == 0) return DSA_OK;
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_status(launch_indexer_front(to_args(batch), q_c, x, w_q, w_k, w_w, q_fp8, q_scale,
                                            w, index_pages, q_f32, k_f32, dev_status,
                                            (cudaStream_t)stream));
}

dsa_status dsa_test_sparse_mla_wait_timeout(const dsa_batch* batch, const uint16_t* q_lat,
                                           const void* latent_pages, float kv_scale,
                                           float sm_scale, const int32_t* indices, int32_t topk,
                                           uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                           int32_t* dev_status, dsa_stream_t stream) {
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    st = check_mla_args(batch, q_lat, latent_pages, indices, topk, out, kv_scale, sm_scale);
    if (st != DSA_OK) return st;
    const size_t need = dsa_sparse_mla_workspace_size(batch, topk);
    if (ws_bytes < need || (need > 0 && (!ws || !aligned16(ws)))) return DSA_ERR_WORKSPACE;
    if (batch->total_q == 0) return DSA_OK;
    g_launches.fetch_add((uint64_t)sparse_mla_launches(batch->total_q, topk, false),
                         std::memory_order_relaxed);
    return cuda_status(launch_sparse_mla(to_args(batch), q_lat, latent_pages, kv_scale, sm_scale,
                                         indices, topk, out, lse, ws, dev_status, false,
                                         (cudaStream_t)stream, true, DSA_LATENT_FP8_E4M3, false));
}

dsa_status dsa_append_cache(const dsa_batch* batch, const float* new_keys,
                            const float* new_latent, float kv_scale, void* index_pages,
                            void* latent_pages, dsa_key_format key_format, int32_t* dev_status,
                            dsa_stream_t stream) {
    dsa_status st = check_batch(batch);
    if (st != DSA_OK) return st;
    if (new_keys && key_format != DSA_KEYS_FP8_E4M3) return DSA_ERR_UNSUPPORTED;
    if ((new_keys && !index_pages) || (new_latent && !latent_pages)) return DSA_ERR_INVALID_ARG;
    if ((new_keys && (!aligned16(new_keys) || !aligned16(index_pages))) ||
        (new_latent && (!aligned16(new_latent) || !aligned16(latent_pages))))
        return DSA_ERR_INVALID_ARG;
    if (new_latent && !(kv_scale > 0.f)) return DSA_ERR_INVALID_ARG;
    if (batch->total_q == 0 || (!new_keys && !new_latent)) return DSA_OK;
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_status(launch_append_cache(to_args(batch), new_keys, new_latent, kv_scale,
                                           index_pages, latent_pages, dev_status,
                                           (cudaStream_t)stream));
}

dsa_status dsa_build_tables(int32_t num_requests, const int32_t* cached_lens,
                            const int32_t* new_lens, const int32_t* free_pages, int32_t num_free,
                            int32_t num_pages, int32_t max_pages, int32_t max_tokens,
                            int32_t* block_table, int32_t* q_offsets, int32_t* seq_lens,
                            int64_t* slots, int32_t* positions, int32_t* token_requests,
                            int32_t* pages_taken, int32_t* dev_status, dsa_stream_t stream) {
    if (num_requests < 1 || num_free < 0 || num_pages < 1 || max_pages < 1 || max_tokens < 0)
        return DSA_ERR_INVALID_ARG;
    if (!build_tables_supported(num_requests)) return DSA_ERR_UNSUPPORTED;
    if (!cached_lens || !new_lens || (num_free > 0 && !free_pages) || !block_table ||
        !q_offsets || !seq_lens || !pages_taken)
        return DSA_ERR_INVALID_ARG;
    if ((slots && !aligned16(slots)) || (positions && !aligned16(positions)) ||
        (token_requests && !aligned16(token_requests)))
        return DSA_ERR_INVALID_ARG;
    // every CTA reads all lengths while others write: outputs (first) and inputs apart
    const Span spans[] = {Span(block_table, (int64_t)num_requests * max_pages, 4),
                          Span(q_offsets, (int64_t)num_requests + 1, 4),
                          Span(seq_lens, num_requests, 4), Span(slots, max_tokens, 8),
                          Span(positions, max_tokens, 4), Span(token_requests, max_tokens, 4),
                          Span(pages_taken, 1, 4), Span(dev_status, 1, 4),
                          Span(cached_lens, num_requests, 4), Span(new_lens, num_requests, 4),
                          Span(free_pages, num_free, 4)};
    constexpr int kOutputs = 8;
    for (int i = 0; i < kOutputs; ++i)
        for (int j = i + 1; j < (int)(sizeof(spans) / sizeof(spans[0])); ++j)
            if (overlap(spans[i], spans[j])) return DSA_ERR_INVALID_ARG;
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_status(launch_build_tables(num_requests, cached_lens, new_lens, free_pages,
                                           num_free, num_pages, max_pages, max_tokens, block_table,
                                           q_offsets, seq_lens, slots, positions, token_requests,
                                           pages_taken, dev_status, (cudaStream_t)stream));
}

dsa_status dsa_rope_append(int32_t num_tokens, const dsa_kv_cache* cache, dsa_float_format format,
                           const dsa_rope* rope, const int32_t* positions, const int64_t* slots,
                           int32_t num_q_heads, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                           int64_t q_out_stride, int32_t* dev_status, dsa_stream_t stream) {
    const dsa_status st = check_kv_cache(cache, format);
    if (st != DSA_OK) return st;
    if (rope == nullptr || num_tokens < 0 || num_q_heads < 0) return DSA_ERR_INVALID_ARG;
    if (num_q_heads > kMaxHeads || cache->num_kv_heads > kMaxHeads) return DSA_ERR_UNSUPPORTED;
    if (rope->num_axes < 0 || rope->num_axes > 3) return DSA_ERR_UNSUPPORTED;
    int64_t pairs = 0;
    for (int i = 0; i < rope->num_axes; ++i) {
        if (rope->sections[i] < 0) return DSA_ERR_INVALID_ARG;
        pairs += rope->sections[i];
    }
    if (2 * pairs > cache->head_dim) return DSA_ERR_INVALID_ARG;
    if (pairs % 8 != 0) return DSA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return DSA_OK;
    if ((pairs > 0 && (!rope->inv_freq || !positions)) || !slots) return DSA_ERR_INVALID_ARG;
    const int dim = cache->head_dim;
    if (!row_ok(k, k_stride, cache->num_kv_heads, dim) ||
        !row_ok(v, v_stride, cache->num_kv_heads, dim))
        return DSA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!row_ok(q, q_stride, num_q_heads, dim) ||
                            !row_ok(q_out, q_out_stride, num_q_heads, dim)))
        return DSA_ERR_INVALID_ARG;
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_status(launch_rope_append(num_tokens, *cache, (int)format, *rope, positions, slots,
                                          num_q_heads, q, q_stride, k, k_stride, v, v_stride, q_out,
                                          q_out_stride, dev_status, (cudaStream_t)stream));
}

size_t dsa_paged_attention_workspace_size(const dsa_batch* batch, const dsa_kv_cache* cache,
                                          int32_t num_q_heads) {
    if (check_batch(batch, true) != DSA_OK || cache == nullptr || cache->num_kv_heads < 1 ||
        num_q_heads < 1 || num_q_heads % cache->num_kv_heads != 0 ||
        (cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256))
        return 0;
    return paged_attention_workspace_bytes(
        (int64_t)batch->max_q_per_request * (num_q_heads / cache->num_kv_heads), cache->head_dim);
}

static dsa_status paged_attention(const dsa_batch* batch, const dsa_kv_cache* cache,
                                  dsa_float_format format, int32_t num_q_heads, const void* q,
                                  int64_t q_stride, float sm_scale, void* out, float* lse,
                                  void* ws, size_t ws_bytes, bool wait_test, int32_t* dev_status,
                                  dsa_stream_t stream) {
    dsa_status st = check_batch(batch, true);
    if (st != DSA_OK) return st;
    st = check_kv_cache(cache, format);
    if (st != DSA_OK) return st;
    if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads != 0 ||
        batch->num_pages != cache->num_pages)
        return DSA_ERR_INVALID_ARG;
    const int group = num_q_heads / cache->num_kv_heads;
    if (num_q_heads > kMaxHeads || (int64_t)batch->max_q_per_request * group > (1 << 30) ||
        !paged_attention_supported(to_args(batch), cache->num_kv_heads, group))
        return DSA_ERR_UNSUPPORTED;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
    if (!std::isnormal(paged_score_scale(sm_scale, *cache))) return DSA_ERR_INVALID_ARG;
    if (batch->total_q == 0) return DSA_OK;
    if (!row_ok(q, q_stride, num_q_heads, cache->head_dim) || !out || !aligned16(out))
        return DSA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws) ||
        ws_bytes < dsa_paged_attention_workspace_size(batch, cache, num_q_heads))
        return DSA_ERR_WORKSPACE;
    const bool whole = g_batch_invariant.load(std::memory_order_relaxed) != 0;
    int launches = 0;
    const dsa_status rc = cuda_status(
        launch_paged_attention(to_args(batch), *cache, (int)format, num_q_heads, q, q_stride,
                               sm_scale, out, lse, ws, whole, wait_test, dev_status, &launches,
                               (cudaStream_t)stream));
    g_launches.fetch_add((uint64_t)launches, std::memory_order_relaxed);
    return rc;
}

dsa_status dsa_paged_attention(const dsa_batch* batch, const dsa_kv_cache* cache,
                               dsa_float_format format, int32_t num_q_heads, const void* q,
                               int64_t q_stride, float sm_scale, void* out, float* lse, void* ws,
                               size_t ws_bytes, int32_t* dev_status, dsa_stream_t stream) {
    return paged_attention(batch, cache, format, num_q_heads, q, q_stride, sm_scale, out, lse, ws,
                           ws_bytes, false, dev_status, stream);
}

dsa_status dsa_test_paged_attention_wait_timeout(const dsa_batch* batch, const dsa_kv_cache* cache,
                                                 dsa_float_format format, int32_t num_q_heads,
                                                 const void* q, int64_t q_stride, float sm_scale,
                                                 void* out, float* lse, void* ws, size_t ws_bytes,
                                                 int32_t* dev_status, dsa_stream_t stream) {
    return paged_attention(batch, cache, format, num_q_heads, q, q_stride, sm_scale, out, lse, ws,
                           ws_bytes, true, dev_status, stream);
}

}  // extern "C"
