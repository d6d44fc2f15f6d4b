// build_tables.cu -- block tables, offsets and cache slots from request lengths.
//
// With held = ceil(cached / 64) and grown = ceil((cached + new) / 64) - held,
// two exclusive sums over the requests (new tokens, new pages) place every
// output: page i of the step's new pages goes to the request whose range of the
// second sum holds i, token t to the request whose range of the first holds t.
//
// Every CTA forms both sums over all requests by itself (at most 4096 pairs of
// lengths, read through L2) and keeps them in shared memory, then fills its own
// tile of tokens and its share of the new pages by binary search.  That repeats
// up to 32 KB of reads per CTA but needs one launch and no ordering between
// CTAs.  The work is bound by latency: the outputs are 16 bytes per token.
#include "common.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxRequests = 4096;
constexpr int kTokensPerThread = 4;
constexpr int kTile = kThreads * kTokensPerThread;

struct TablesArgs {
    int32_t num_requests, num_free, num_pages, max_pages, max_tokens;
    const int32_t* cached;
    const int32_t* added;
    const int32_t* free_pages;
    int32_t* block_table;
    int32_t* q_offsets;
    int32_t* seq_lens;
    int64_t* slots;
    int32_t* positions;
    int32_t* token_requests;
    int32_t* pages_taken;
    int32_t* status;
};

// What a request brings.  `fits` is false for negative lengths and for more
// pages than a table row holds: such a request takes no pages and no slots.
struct Growth {
    int32_t cached, added, held, grown;
    bool fits;
};

__device__ __forceinline__ Growth growth_of(const TablesArgs& a, int b) {
    const int cached = __ldg(a.cached + b), added = __ldg(a.added + b);
    Growth g;
    g.cached = max(cached, 0);
    g.added = max(added, 0);
    const int64_t held = ((int64_t)g.cached + kPage - 1) / kPage;
    const int64_t pages = ((int64_t)g.cached + g.added + kPage - 1) / kPage;
    g.fits = cached >= 0 && added >= 0 && pages <= a.max_pages;
    g.held = (int32_t)held;
    g.grown = g.fits ? (int32_t)(pages - held) : 0;
    return g;
}

// Page i of the step's new pages, or -1 when the list is too short or the id is
// outside the pool.
__device__ __forceinline__ int new_page(const TablesArgs& a, int64_t i) {
    if (i >= a.num_free) return -1;
    const int p = __ldg(a.free_pages + i);
    return p >= 0 && p < a.num_pages ? p : -1;
}

// The last b with sums[b] <= x (sums is non-decreasing, sums[0] = 0): the
// request whose range holds x, since ranges before the last equal entry are empty.
__device__ __forceinline__ int owner_of(const int32_t* sums, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) build_tables_kernel(TablesArgs a) {
    __shared__ int32_t s_tokens[kMaxRequests];
    __shared__ int32_t s_pages[kMaxRequests];
    __shared__ int64_t s_warp[2][kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = a.num_requests;
    grid_dependents_launch();
    grid_dependency_wait();

    // both sums in 64 bits: each thread sums a run of requests, then a scan over
    // the threads' totals
    const int per = (n + kThreads - 1) / kThreads;
    int64_t tokens = 0, pages = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < n) {
            const Growth g = growth_of(a, b);
            tokens += g.added;
            pages += g.grown;
            bad |= !g.fits;
        }
    }
    int64_t ti = tokens, pi = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, pi, o);
        if (lane >= o) {
            ti += x;
            pi += y;
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = ti;
        s_warp[1][warp] = pi;
    }
    __syncthreads();
    int64_t t0 = 0, p0 = 0, all_tokens = 0, all_pages = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int64_t x = s_warp[0][w], y = s_warp[1][w];
        if (w < warp) {
            t0 += x;
            p0 += y;
        }
        all_tokens += x;
        all_pages += y;
    }
    t0 += ti - tokens;
    p0 += pi - pages;
    const bool first = blockIdx.x == 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < n) {
            const Growth g = growth_of(a, b);
            const int32_t at = (int32_t)min(t0, (int64_t)a.max_tokens);
            s_tokens[b] = at;
            s_pages[b] = (int32_t)min(p0, (int64_t)INT32_MAX);
            if (first) {
                a.q_offsets[b] = at;
                a.seq_lens[b] = (int32_t)min((int64_t)g.cached + g.added, (int64_t)INT32_MAX);
            }
            t0 += g.added;
            p0 += g.grown;
        }
    }
    const int T = (int)min(all_tokens, (int64_t)a.max_tokens);
    if (first) {
        if (bad) record_error(a.status, DSA_ERR_DEVICE_CHECK);
        if (tid == 0) {
            a.q_offsets[n] = T;
            *a.pages_taken = (int32_t)min(all_pages, (int64_t)INT32_MAX);
            if (all_tokens > a.max_tokens || all_pages > a.num_free)
                record_error(a.status, DSA_ERR_DEVICE_CHECK);
        }
    }
    __syncthreads();

    // new table entries
    const int64_t step = (int64_t)gridDim.x * kThreads;
    const int64_t end = min(all_pages, (int64_t)INT32_MAX);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < end; i += step) {
        const int b = owner_of(s_pages, n, (int)i);
        const int held = growth_of(a, b).held;
        const int page = new_page(a, i);
        if (page < 0) record_error(a.status, DSA_ERR_DEVICE_CHECK);
        a.block_table[(int64_t)b * a.max_pages + held + (i - s_pages[b])] = page;
    }

    // tokens
    if (!a.slots && !a.positions && !a.token_requests) return;
    for (int i = 0; i < kTokensPerThread; ++i) {
        const int64_t t64 = (int64_t)blockIdx.x * kTile + i * kThreads + tid;
        if (t64 >= a.max_tokens) break;
        const int t = (int)t64;
        int b = -1, pos = 0;
        int64_t slot = -1;
        if (t < T) {
            b = owner_of(s_tokens, n, t);
            const Growth g = growth_of(a, b);
            pos = (int)min((int64_t)g.cached + (t - s_tokens[b]), (int64_t)INT32_MAX);
            if (g.fits) {
                const int lp = pos / kPage;
                int page;
                if (lp >= g.held) {
                    page = new_page(a, (int64_t)s_pages[b] + lp - g.held);
                } else {  // the page the cached tokens left open
                    page = __ldg(a.block_table + (int64_t)b * a.max_pages + lp);
                    if (page < 0 || page >= a.num_pages) {
                        page = -1;
                        record_error(a.status, DSA_ERR_DEVICE_CHECK);
                    }
                }
                if (page >= 0) slot = (int64_t)page * kPage + pos % kPage;
            }
        }
        if (a.slots) a.slots[t] = slot;
        if (a.positions) a.positions[t] = pos;
        if (a.token_requests) a.token_requests[t] = b;
    }
}

}  // namespace

bool build_tables_supported(int num_requests) { return num_requests <= kMaxRequests; }

cudaError_t launch_build_tables(int num_requests, const int32_t* cached, const int32_t* added,
                                const int32_t* free_pages, int num_free, int num_pages,
                                int max_pages, int max_tokens, int32_t* block_table,
                                int32_t* q_offsets, int32_t* seq_lens, int64_t* slots,
                                int32_t* positions, int32_t* token_requests, int32_t* pages_taken,
                                int32_t* status, cudaStream_t stream) {
    TablesArgs a;
    a.num_requests = num_requests;
    a.num_free = num_free;
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.max_tokens = max_tokens;
    a.cached = cached;
    a.added = added;
    a.free_pages = free_pages;
    a.block_table = block_table;
    a.q_offsets = q_offsets;
    a.seq_lens = seq_lens;
    a.slots = slots;
    a.positions = positions;
    a.token_requests = token_requests;
    a.pages_taken = pages_taken;
    a.status = status;
    const bool per_token = slots || positions || token_requests;
    const int64_t grid = per_token ? ((int64_t)max_tokens + kTile - 1) / kTile : 1;
    return launch_kernel(build_tables_kernel, dim3((unsigned)(grid < 1 ? 1 : grid)), dim3(kThreads),
                         0, stream, true, 1, a);
}

}  // namespace dsa
