// build_tables.cu -- block tables, offsets and cache slots from request lengths.
//
// With held = ceil(cached / 64) and grown = ceil((cached + new) / 64) - held,
// two exclusive sums over the requests (new tokens, new pages) place every
// output: page i of the step's new pages goes to the request whose range of the
// second sum holds i, token t to the request whose range of the first holds t.
//
// Every CTA forms both sums over all requests by itself (at most 4096 pairs of
// lengths, read through L2) and keeps them in shared memory, then fills its own
// tiles of tokens and its share of the new pages.  That repeats up to 32 KB of reads
// per CTA but needs one launch and no ordering between CTAs.  A warp writes 64
// consecutive tokens, two a lane (a 16-byte store of slots, 8-byte ones of positions
// and requests); it looks its request up once where one request holds them all.
//
// Bound by latency up to some 100,000 tokens, then by the writes of 16 bytes a token.
#include "common.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxRequests = 4096;
constexpr int kPerThread = kMaxRequests / kThreads;  // requests summed by one thread
constexpr int kTile = kThreads * 2;                  // tokens written at a time
constexpr int kMaxCtas = 2 * 152;                    // resident at once

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

// The last b in [lo, hi] with sums[b] <= x (sums is non-decreasing, sums[lo] <= x):
// the request whose range holds x, since ranges before the last equal entry are empty.
__device__ __forceinline__ int owner_of(const int32_t* sums, int lo, int hi, int x) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Sums stop at the largest int32 (associative for values of 0 and more).
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    return min(a + b, (uint32_t)INT32_MAX);
}

// The cache slot of position pos of request b, whose new pages begin at first_new.
__device__ __forceinline__ int64_t slot_of(const TablesArgs& a, const Growth& g, int b,
                                           int first_new, int pos) {
    if (!g.fits) return -1;
    const int lp = pos / kPage;
    int page;
    if (lp >= g.held) {
        page = new_page(a, (int64_t)first_new + lp - g.held);
    } else {  // the page the cached tokens left open
        page = __ldg(a.block_table + (int64_t)b * a.max_pages + lp);
        if (page < 0 || page >= a.num_pages) {
            page = -1;
            record_error(a.status, DSA_ERR_DEVICE_CHECK);
        }
    }
    return page < 0 ? -1 : (int64_t)page * kPage + pos % kPage;
}

__global__ void __launch_bounds__(kThreads, 2) build_tables_kernel(TablesArgs a) {
    __shared__ int32_t s_tokens[kMaxRequests];
    __shared__ int32_t s_pages[kMaxRequests];
    __shared__ uint32_t s_warp[2][kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = a.num_requests;
    grid_dependents_launch();
    grid_dependency_wait();

    // each thread sums a run of requests, then a scan over the threads' totals
    const int per = (n + kThreads - 1) / kThreads;
    uint32_t added[kPerThread], grown[kPerThread], length[kPerThread];
    uint32_t tokens = 0, pages = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = tid * per + i;
        added[i] = grown[i] = length[i] = 0;
        if (i < per && b < n) {
            const Growth g = growth_of(a, b);
            added[i] = g.added;
            grown[i] = g.grown;
            length[i] = add(g.cached, g.added);
            bad |= !g.fits;
        }
        tokens = add(tokens, added[i]);
        pages = add(pages, grown[i]);
    }
    uint32_t ti = tokens, pi = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, ti, o);
        const uint32_t y = __shfl_up_sync(0xffffffffu, pi, o);
        if (lane >= o) {
            ti = add(ti, x);
            pi = add(pi, y);
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = ti;
        s_warp[1][warp] = pi;
    }
    // exclusive within the warp
    uint32_t t0 = __shfl_up_sync(0xffffffffu, ti, 1), p0 = __shfl_up_sync(0xffffffffu, pi, 1);
    if (lane == 0) t0 = p0 = 0;
    __syncthreads();
    uint32_t all_tokens = 0, all_pages = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const uint32_t x = s_warp[0][w], y = s_warp[1][w];
        if (w < warp) {
            t0 = add(t0, x);
            p0 = add(p0, y);
        }
        all_tokens = add(all_tokens, x);
        all_pages = add(all_pages, y);
    }
    const uint32_t cap = a.max_tokens;
    const bool writes = tid % gridDim.x == blockIdx.x;  // the offsets, spread over the CTAs
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = tid * per + i;
        if (i < per && b < n) {
            const int32_t at = (int32_t)min(t0, cap);
            s_tokens[b] = at;
            s_pages[b] = (int32_t)p0;
            if (writes) {
                a.q_offsets[b] = at;
                a.seq_lens[b] = (int32_t)length[i];
            }
            t0 = add(t0, added[i]);
            p0 = add(p0, grown[i]);
        }
    }
    const int T = (int)min(all_tokens, cap);
    if (blockIdx.x == 0) {
        if (bad) record_error(a.status, DSA_ERR_DEVICE_CHECK);
        if (tid == 0) {
            a.q_offsets[n] = T;
            *a.pages_taken = (int32_t)all_pages;
            if (all_tokens > cap || all_pages > (uint32_t)a.num_free)
                record_error(a.status, DSA_ERR_DEVICE_CHECK);
        }
    }
    __syncthreads();

    // new table entries
    const uint32_t step = gridDim.x * kThreads;
    for (uint32_t i = blockIdx.x * kThreads + tid; i < all_pages; i += step) {
        const int b = owner_of(s_pages, 0, n - 1, (int)i);
        const int held = growth_of(a, b).held;
        const int page = new_page(a, i);
        if (page < 0) record_error(a.status, DSA_ERR_DEVICE_CHECK);
        a.block_table[(int64_t)b * a.max_pages + held + ((int)i - s_pages[b])] = page;
    }

    // tokens
    if (!a.slots && !a.positions && !a.token_requests) return;
    for (int64_t tile = (int64_t)blockIdx.x * kTile; tile < a.max_tokens;
         tile += (int64_t)gridDim.x * kTile) {
        const int64_t first = tile + warp * 64;  // of the warp's 64 tokens
        if (first >= a.max_tokens) break;
        int lo = 0, hi = n - 1;
        if (first < T) {
            lo = owner_of(s_tokens, 0, n - 1, (int)first);
            if (lo == n - 1 || s_tokens[lo + 1] >= first + 64) hi = lo;
        }
        const int64_t t = first + 2 * lane;
        int b[2], pos[2];
        int64_t slot[2];
        Growth g = {};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            b[x] = -1;
            pos[x] = 0;
            slot[x] = -1;
            if (t + x < T) {
                const int tx = (int)t + x;
                b[x] = owner_of(s_tokens, x ? b[0] : lo, hi, tx);
                if (x == 0 || b[1] != b[0]) g = growth_of(a, b[x]);
                pos[x] = (int)add(g.cached, tx - s_tokens[b[x]]);
                if (x == 1 && b[1] == b[0] && pos[1] % kPage != 0)
                    slot[1] = slot[0] < 0 ? -1 : slot[0] + 1;  // the same page
                else
                    slot[x] = slot_of(a, g, b[x], s_pages[b[x]], pos[x]);
            }
        }
        if (t + 1 < a.max_tokens) {
            if (a.slots)
                *reinterpret_cast<longlong2*>(a.slots + t) = make_longlong2(slot[0], slot[1]);
            if (a.positions) *reinterpret_cast<int2*>(a.positions + t) = make_int2(pos[0], pos[1]);
            if (a.token_requests)
                *reinterpret_cast<int2*>(a.token_requests + t) = make_int2(b[0], b[1]);
        } else if (t < a.max_tokens) {
            if (a.slots) a.slots[t] = slot[0];
            if (a.positions) a.positions[t] = pos[0];
            if (a.token_requests) a.token_requests[t] = b[0];
        }
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
    const int64_t tiles = per_token ? ((int64_t)max_tokens + kTile - 1) / kTile : 1;
    // every CTA the same number of tiles
    const int64_t each = (tiles + kMaxCtas - 1) / kMaxCtas;
    const int64_t grid = tiles > 0 ? (tiles + each - 1) / each : 1;
    return launch_kernel(build_tables_kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, true,
                         1, a);
}

}  // namespace dsa
