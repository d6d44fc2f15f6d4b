// quant_cache.cu -- the 8-bit cache with a scale for every 16 tokens of a head: rotary
// positions and quantisation as tokens are written, and the values read back.
#include <climits>

#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = DSA_QUANT_BLOCK;
constexpr int kPageBlocks = kPage / kBlock;
constexpr int kMaxTokens = 16;  // of a CTA
constexpr int kSpan = kMaxTokens + kBlock - 1;  // tokens whose angles a CTA may need
constexpr int kAhead = 2;       // 16-value units of queries that a thread has in flight
constexpr float kMinScale = 0x1p-48f, kMaxNeed = 0x1p32f, kMaxScale = 0x1p33f;

struct QuantArgs {
    int32_t num_tokens, q_heads, kv_heads, interleaved, pairs;
    int32_t tokens;      // of a CTA
    int32_t axes;
    int32_t end0, end1;  // first pair of the second and of the third section
    int64_t slot_end;
    const double* inv_freq;
    const int32_t* positions;
    const int64_t* slots;
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    uint8_t* k_pages;
    uint8_t* v_pages;
    float* scales;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int32_t* status;
};

template <bool kInt8>
__device__ __forceinline__ float largest() {
    return kInt8 ? 127.f : 448.f;
}

// Four values as codes, the first in the low byte; INT8: within +-127.49 already, rounded
// by the addition of 1.5 * 2^23, whose low bits then hold the integer.
template <bool kInt8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if (kInt8) {
        constexpr float kMagic = 12582912.f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, kMagic)),
                                        __float_as_uint(__fadd_rn(b, kMagic)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, kMagic)),
                                        __float_as_uint(__fadd_rn(d, kMagic)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <bool kInt8>
__device__ __forceinline__ void decode4(uint32_t codes, float (&x)[4]) {
    if (kInt8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(codes >> (8 * i));
    } else {
        const float2 lo = e4m3x2_to_float2((uint16_t)codes);
        const float2 hi = e4m3x2_to_float2((uint16_t)(codes >> 16));
        x[0] = lo.x;
        x[1] = lo.y;
        x[2] = hi.x;
        x[3] = hi.y;
    }
}

template <bool kInt8>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float by) {
    return make_uint2(encode4<kInt8>(__fmul_rn(x[0], by), __fmul_rn(x[1], by),
                                     __fmul_rn(x[2], by), __fmul_rn(x[3], by)),
                      encode4<kInt8>(__fmul_rn(x[4], by), __fmul_rn(x[5], by),
                                     __fmul_rn(x[6], by), __fmul_rn(x[7], by)));
}

// The least k >= 0 with scale * 2^k >= need (normal numbers).
__device__ __forceinline__ int doublings(float scale, float need) {
    const uint32_t s = __float_as_uint(scale), n = __float_as_uint(need);
    return max(0, (int)(n >> 23) - (int)(s >> 23) + ((n & 0x7fffffu) > (s & 0x7fffffu)));
}

// The larger, or NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Nothing; but values formed from these before are not known to be those formed after, and
// so not kept, at twice the registers.
__device__ __forceinline__ void opaque(uint4& a, uint4& b) {
    asm volatile("" : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w), "+r"(b.x), "+r"(b.y), "+r"(b.z),
                      "+r"(b.w));
}

// The tokens of one block that stand together: the first of them, from the CTA's first
// token on, how many, and which of them are stored.
struct Run {
    int32_t first, count;
    uint32_t stored;
    int32_t pad;
};

// A way through [tokens][each] in steps, without a division for each.
struct Stride2 {
    int token, rest, each, step_token, step_rest;
    __device__ __forceinline__ Stride2(int each_, int begin, int step) : each(each_) {
        token = begin / each;
        rest = begin - token * each;
        step_token = step / each;
        step_rest = step - step_token * each;
    }
    __device__ __forceinline__ bool next() {  // whether it has wrapped
        token += step_token;
        rest += step_rest;
        if (rest < each) return false;
        rest -= each;
        ++token;
        return true;
    }
};

// A thread's way over the queries of a CTA's tokens, 16 values of a head at a time (the two
// halves of eight pairs, or neighbours): its unit of the heads stays the same, as the steps
// are multiples of a head's units.
template <typename T, int kDim>
struct Queries {
    static constexpr int kUnits = kDim / 16;
    Stride2 way;
    T* p;
    int64_t step, wrap;  // of p
    __device__ __forceinline__ Queries(const T* base, int64_t stride, int heads, int begin,
                                       int by)
        : way(heads * kUnits, begin, by) {
        p = const_cast<T*>(base) + way.token * stride + way.rest / kUnits * kDim;
        step = way.step_token * stride + way.step_rest / kUnits * kDim;
        wrap = stride - (int64_t)heads * kDim;
    }
    __device__ __forceinline__ void next() { p += way.next() ? step + wrap : step; }
};

// The largest magnitude of 8 values, NaN if there is one, in both halves of a pair.
template <typename T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_abs2<__nv_bfloat16>(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t max_abs2<__half>(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2_nan(__habs2(*reinterpret_cast<const __half2*>(&a)),
                                  __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t max_abs8(uint32_t m, const uint4& u) {
    return max_abs2<T>(max_abs2<T>(max_abs2<T>(max_abs2<T>(m, u.x), u.y), u.z), u.w);
}

// The last slot of slots[0 .. at] within the pool, -1 if there is none, by the whole CTA (*near
// in shared memory: INT_MAX).  2048 slots at a time: where the first 28672 of a prompt's 32768
// tokens are not stored the call takes 100 us (without the search 96, by a warp's 32 slots at a
// time 515).  Not inline: prompts of 7 requests 106.1 us, so 105.6, without the search 105.1.
__device__ __noinline__ int64_t slot_before(const int64_t* slots, int64_t at, int64_t slot_end,
                                            int* near) {
    constexpr int kLook = 8;
    const int tid = threadIdx.x;
#pragma unroll 1
    for (; at >= 0; at -= kThreads * kLook) {
        int64_t s[kLook];
#pragma unroll
        for (int i = 0; i < kLook; ++i) {
            const int64_t t = at - tid - kThreads * i;
            s[i] = t >= 0 ? __ldg(slots + t) : -1;
        }
        int mine = INT_MAX;
#pragma unroll
        for (int i = kLook - 1; i >= 0; --i)
            if (s[i] >= 0 && s[i] < slot_end) mine = tid + kThreads * i;
        if (!__syncthreads_or(mine != INT_MAX)) continue;
        atomicMin(near, mine);
        __syncthreads();
        return __ldg(slots + at - *near);
    }
    return -1;
}

// kShort: for small calls, a token or two to a CTA.  With one its keys and values are on
// their way, too, before it is known where they go.
template <typename T, bool kInt8, int kDim, bool kShort>
__global__ void __launch_bounds__(kThreads, 3) quant_append_kernel(const QuantArgs a) {
    constexpr int kUnits = kDim / 16;     // 16 values of a row to a lane
    constexpr int kRows = 32 / kUnits;    // of a warp at a time
    constexpr int kSteps = kBlock / kRows;
    // Steps in flight.  Of 256 dims two (prompts of 7 requests 80 us, with four and so 200
    // bytes spilled 86); in a small call, which mostly has one row to a run, one: short code,
    // which has to be fetched, is the faster (one token: 5.6 -> 3.95 us; 256 requests of up
    // to five tokens 11.5 -> 10.4, a prompt of 500 alone 8.5 -> 9.5).
    constexpr int kLoads = kShort ? 1 : kDim == 256 ? 2 : kSteps < 4 ? kSteps : 4;
    constexpr int kUnroll = kShort ? 1 : kSteps / kLoads;
    extern __shared__ float2 s_turn[];    // of each token, turn_at()
    __shared__ int64_t s_slot[kMaxTokens + kBlock];  // from the token before the CTA's on
    __shared__ Run s_run[kMaxTokens];
    __shared__ int s_runs, s_reach, s_near;
    __shared__ int64_t s_apart;
    __shared__ unsigned long long s_rate[kDim / 2];
    __shared__ int32_t s_pos[3 * kSpan];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = (int64_t)blockIdx.x * a.tokens;
    const int count = (int)min((int64_t)a.tokens, a.num_tokens - first);
    // a run may go on behind the CTA's tokens
    const int reach = (int)min((int64_t)count + kBlock - 1, a.num_tokens - first);
    grid_dependents_launch();
    grid_dependency_wait();

    // the first queries are on their way while slots are looked at and angles formed
    const int unit = lane % kUnits, row0 = lane / kUnits;  // of a block's rows
    struct Source {
        const void* base;
        int64_t stride;
        int head, at0, at1;
        bool turned;
    };
    auto source = [&](int which, int head) {
        Source x;
        x.base = which ? a.v : a.k;
        x.stride = which ? a.v_stride : a.k_stride;
        x.head = head;
        x.turned = !which && unit < a.pairs / 8;
        const bool halves = x.turned && !a.interleaved;
        x.at0 = halves ? unit * 8 : unit * 16;
        x.at1 = halves ? unit * 8 + a.pairs : unit * 16 + 8;
        return x;
    };
    uint4 own_lo, own_hi;
    const int own = warp + kWarps * blockIdx.y;  // first item
    if (kShort && a.tokens == 1 && row0 == 0 && own < 2 * a.kv_heads) {
        const int which = own >= a.kv_heads;
        const Source x = source(which, own - which * a.kv_heads);
        const T* p = static_cast<const T*>(x.base) + first * x.stride + x.head * kDim;
        own_lo = *reinterpret_cast<const uint4*>(p + x.at0);
        own_hi = *reinterpret_cast<const uint4*>(p + x.at1);
    }
    const int q_end = a.q_heads > 0 ? count : 0;
    const int begin = tid + kThreads * blockIdx.y, step = kThreads * gridDim.y;
    const int q_unit = tid % kUnits;
    const bool q_turned = q_unit < a.pairs / 8, q_halves = q_turned && !a.interleaved;
    const int q_at0 = q_halves ? q_unit * 8 : q_unit * 16;
    const int q_at1 = q_halves ? q_unit * 8 + a.pairs : q_unit * 16 + 8;
    Queries<T, kDim> ahead(static_cast<const T*>(a.q) + first * a.q_stride, a.q_stride,
                           max(a.q_heads, 1), begin, step);
    uint4 q_lo[kAhead], q_hi[kAhead];
    auto load_query = [&](int x) {
        if (ahead.way.token < q_end) {
            q_lo[x] = *reinterpret_cast<const uint4*>(ahead.p + q_at0);
            q_hi[x] = *reinterpret_cast<const uint4*>(ahead.p + q_at1);
        }
        ahead.next();
    };
#pragma unroll
    for (int x = 0; x < kAhead; ++x) load_query(x);

    if (warp == 0) {
        static_assert(kSpan < 32, "a lane to each token");
        int64_t slot = -1;
        const int64_t t = first + lane - 1;
        if (lane <= reach && t >= 0) {
            slot = __ldg(a.slots + t);
            if (slot >= a.slot_end) {
                if (lane > 0 && lane <= count) record_error(a.status, DSA_ERR_DEVICE_CHECK);
                slot = -1;
            }
        }
        if (lane <= reach) s_slot[lane] = slot;
        __syncwarp();
        // lane i: the CTA's token i
        const int64_t own = lane < reach ? s_slot[lane + 1] : -1;
        const int64_t before = lane < reach ? s_slot[lane] : -1;
        const bool joined = own >= 0 && before >= 0 && own / kBlock == before / kBlock;
        const bool ascends = !joined || own > before;
        if (lane < count && !ascends) record_error(a.status, DSA_ERR_DEVICE_CHECK);
        const uint32_t all_joined = __ballot_sync(0xffffffffu, joined);
        const uint32_t all_ascend = __ballot_sync(0xffffffffu, ascends);
        bool leads = lane < count && own >= 0 && !joined;
        // Behind tokens that are not stored the block of the last one that is may come up
        // again: whoever writes that block may be at it now, so these tokens are left out.
        const bool behind_gap = leads && before < 0 && first + lane > 0;
        if (lane == 0) {
            s_apart = -1;
            s_near = INT_MAX;
        }
        if (__any_sync(0xffffffffu, behind_gap)) {
            const uint32_t kept = __ballot_sync(0xffffffffu, lane <= reach && slot >= 0) &
                                  ((2u << lane) - 1u);  // of s_slot[0 .. lane]
            __syncwarp();
            if (behind_gap && kept == 0) {
                s_apart = own;  // the first run's: the last slot kept lies before the window
            } else if (behind_gap && s_slot[31 - __clz(kept)] / kBlock == own / kBlock) {
                record_error(a.status, DSA_ERR_DEVICE_CHECK);
                leads = false;
            }
        }
        const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
        int end = 0;
        if (leads) {
            Run r;
            r.first = lane;
            // tokens behind this one that are joined to their predecessor
            r.count = min(__ffs(~(all_joined >> (lane + 1))), kBlock);
            const uint32_t all = (1u << r.count) - 1u;
            r.stored = (all_ascend >> lane) & all;
            if (r.stored != all) {  // those that exceed every one before, so that no row comes twice
                int64_t most = own;
                for (int i = 1; i < r.count; ++i) {
                    const int64_t s = s_slot[lane + 1 + i];
                    if (s > most) most = s;
                    else r.stored &= ~(1u << i);
                }
            }
            end = lane + r.count;
            s_run[__popc(leaders & ((1u << lane) - 1u))] = r;
        }
        end = __reduce_max_sync(0xffffffffu, end);
        if (lane == 0) {
            s_runs = __popc(leaders);
            s_reach = max(end, a.q_heads > 0 ? count : 0);
        }
    } else if (warp < kWarps / 2) {
        if (a.pairs > 0)
            for (int i = tid - 32; i < a.axes * kSpan; i += kThreads / 2 - 32)
                if (i % kSpan < reach)
                    s_pos[i] = __ldg(a.positions + (int64_t)(i / kSpan) * a.num_tokens + first +
                                     i % kSpan);
    } else {
        // double precision is slow here: once for a pair, not for each of its angles
        for (int i = tid - kThreads / 2; i < a.pairs; i += kThreads / 2)
            s_rate[i] = turn_rate(__ldg(a.inv_freq + i));
    }
    __syncthreads();
    if (s_apart >= 0) {  // the same for slots before the window
        const int64_t last = slot_before(a.slots, first - 2, a.slot_end, &s_near);
        if (tid == 0 && last >= 0 && last / kBlock == s_apart / kBlock) {
            record_error(a.status, DSA_ERR_DEVICE_CHECK);
            s_run[0] = s_run[--s_runs];
        }
    }
    if (a.pairs > 0) {
        int j = tid / a.pairs, pair = tid - j * a.pairs;
        const int step_j = kThreads / a.pairs, step_pair = kThreads - step_j * a.pairs;
        while (j < s_reach) {
            const int axis = (pair >= a.end0 ? 1 : 0) + (pair >= a.end1 ? 1 : 0);
            s_turn[j * a.pairs + turn_at(pair, a.pairs)] =
                fine_turn_of(s_rate[pair], s_pos[axis * kSpan + j]);
            j += step_j;
            pair += step_pair;
            if (pair >= a.pairs) {
                pair -= a.pairs;
                ++j;
            }
        }
    }
    __syncthreads();

    // Queries: a thread to 16 values.
    Queries<T, kDim> here(static_cast<const T*>(a.q_out) + first * a.q_out_stride, a.q_out_stride,
                          max(a.q_heads, 1), begin, step);
    while (here.way.token < q_end) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (here.way.token < q_end) {
                float v[8], w[8];
                unpack8<T>(q_lo[x], v);
                unpack8<T>(q_hi[x], w);
                if (q_turned)
                    turn16(v, w, s_turn + here.way.token * a.pairs, a.pairs / 8, q_unit,
                           a.interleaved);
                store8(here.p + q_at0, v);
                store8(here.p + q_at1, w);
            }
            here.next();
            load_query(x);
        }
    }

    // Keys and values: a warp to a run's head.
    bool loaded = kShort && a.tokens == 1;  // the first row of the first item
    for (Stride2 item(2 * a.kv_heads, warp + kWarps * blockIdx.y, kWarps * gridDim.y);
         item.token < s_runs; item.next()) {
        const int i_run = item.token, rest = item.rest;
        const int which = rest >= a.kv_heads, head = rest - which * a.kv_heads;
        const Run run = s_run[i_run];
        const int64_t slot0 = s_slot[run.first + 1];
        const int64_t page_head = slot0 / kPage * a.kv_heads + head;
        const int part = (int)(slot0 % kPage) / kBlock;
        float* const scale_at = a.scales + (page_head * 2 + which) * kPageBlocks + part;
        uint8_t* const block =
            (which ? a.v_pages : a.k_pages) + (page_head * kPage + part * kBlock) * kDim;
        const bool fresh = slot0 % kBlock == 0;
        const float begun = *scale_at;
        const Source x = source(which, head);
        const bool turned = x.turned;
        const int at0 = x.at0, at1 = x.at1;
        // Two passes over the values.  Up to 128 dims their 16-bit forms stay in registers
        // in between; 256 read them once more, from the caches.
        const T* const from = static_cast<const T*>(x.base) +
                              (first + run.first + row0) * x.stride + head * kDim;
        auto load = [&](int s, uint4& lo, uint4& hi) {
            lo = hi = make_uint4(0, 0, 0, 0);
            if (kShort && loaded && s == 0 && row0 == 0) {
                lo = own_lo;
                hi = own_hi;
            } else if (run.stored >> (s * kRows + row0) & 1) {
                const T* p = from + s * kRows * x.stride;
                lo = *reinterpret_cast<const uint4*>(p + at0);
                hi = *reinterpret_cast<const uint4*>(p + at1);
            }
        };
        auto values = [&](int s, const uint4& lo, const uint4& hi, float (&x)[8], float (&y)[8]) {
            unpack8<T>(lo, x);
            unpack8<T>(hi, y);
            if (turned)
                turn16(x, y, s_turn + (run.first + s * kRows + row0) * a.pairs, a.pairs / 8, unit,
                       a.interleaved);
        };
        const int steps = kShort ? (run.count + kRows - 1) / kRows : kSteps;
        // the largest magnitude; NaN if there is one
        float most = 0.f;
        uint32_t most2 = 0;  // of a pair of values as they are
        const bool as_is = which || a.pairs == 0;
        uint4 lo[kLoads], hi[kLoads];
#pragma unroll kUnroll
        for (int s0 = 0; s0 < steps; s0 += kLoads) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load(s0 + i, lo[i], hi[i]);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                if (as_is) {
                    most2 = max_abs8<T>(max_abs8<T>(most2, lo[i]), hi[i]);
                    continue;
                }
                float x[8], y[8];
                values(s0 + i, lo[i], hi[i], x, y);
                // of a row that is not stored the values are 0, or 0 turned by what its
                // place in shared memory holds
                if (run.stored >> ((s0 + i) * kRows + row0) & 1)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        most = max_nan(most, max_nan(fabsf(x[e]), fabsf(y[e])));
            }
        }
        if (as_is) {
            const float2 m = to_float2<T>(most2);
            most = max_nan(m.x, m.y);
        }
        uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu);
        const bool odd = top >= 0x7f800000u;
        if (odd) {  // of the finite values only
            if (lane == 0) record_error(a.status, DSA_ERR_DEVICE_CHECK);
            top = 0;
#pragma unroll 1
            for (int s = 0; s < kSteps; ++s) {
                uint4 l, h;
                load(s, l, h);
                float x[8], y[8];
                values(s, l, h, x, y);
                if (run.stored >> (s * kRows + row0) & 1)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (isfinite(x[i])) top = max(top, __float_as_uint(fabsf(x[i])));
                        if (isfinite(y[i])) top = max(top, __float_as_uint(fabsf(y[i])));
                    }
            }
            top = __reduce_max_sync(0xffffffffu, top);
        }
        const float all = __fdiv_rn(__uint_as_float(top), largest<kInt8>());
        const float need = fminf(fmaxf(all, kMinScale), kMaxNeed);
        if (!fresh && !(begun >= kMinScale && begun <= kMaxScale)) {
            if (lane == 0) record_error(a.status, DSA_ERR_DEVICE_CHECK);
            loaded = false;
            continue;
        }
        const int k = fresh ? 0 : doublings(begun, need);
        const float scale = fresh ? need : __uint_as_float(__float_as_uint(begun) + (k << 23));
        const float by = __frcp_rn(scale);

        uint32_t written = 0;  // which of the block's rows this call writes
        auto write = [&](int s, const float (&x)[8], const float (&y)[8]) {
            const int row = (int)(s_slot[run.first + s * kRows + row0 + 1]) % kBlock;
            written |= 1u << row;
            uint8_t* dst = block + row * kDim;
            *reinterpret_cast<uint2*>(dst + at0) = encode8<kInt8>(x, by);
            *reinterpret_cast<uint2*>(dst + at1) = encode8<kInt8>(y, by);
        };
        if (kInt8 && (odd || all > kMaxNeed)) {
            // values that have no code (E4M3's conversion knows what to do with them)
            const float most = __fmul_rn(scale, largest<kInt8>());
#pragma unroll 1
            for (int s = 0; s < kSteps; ++s) {
                if (!(run.stored >> (s * kRows + row0) & 1)) continue;
                uint4 l, h;
                load(s, l, h);
                float x[8], y[8];
                values(s, l, h, x, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = x[e] != x[e] ? 0.f : fminf(fmaxf(x[e], -most), most);
                    y[e] = y[e] != y[e] ? 0.f : fminf(fmaxf(y[e], -most), most);
                }
                write(s, x, y);
            }
        } else {
#pragma unroll kUnroll
            for (int s0 = 0; s0 < steps; s0 += kLoads) {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    if (kSteps > kLoads) load(s0 + i, lo[i], hi[i]);
                    else opaque(lo[i], hi[i]);
                }
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    if (run.stored >> ((s0 + i) * kRows + row0) & 1) {
                        float x[8], y[8];
                        values(s0 + i, lo[i], hi[i], x, y);
                        write(s0 + i, x, y);
                    }
            }
        }
        if (k > 0) {
            written = __reduce_or_sync(0xffffffffu, written);
            const float down = __uint_as_float((uint32_t)max(127 - k, 1) << 23);
#pragma unroll 1
            for (int s = 0; s < kSteps; ++s) {
                const int row = s * kRows + row0;
                if (written >> row & 1) continue;
                uint4* at = reinterpret_cast<uint4*>(block + row * kDim) + unit;
                uint4 u = *at;
                uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float c[4];
                    decode4<kInt8>(w[i], c);
                    w[i] = encode4<kInt8>(c[0] * down, c[1] * down, c[2] * down, c[3] * down);
                }
                *at = u;
            }
        }
        if (lane == 0 && (fresh || k > 0)) *scale_at = scale;
        loaded = false;
    }
}

template <typename T, bool kInt8, int kDim>
cudaError_t launch_append(QuantArgs a, cudaStream_t stream) {
    // As few tokens to a CTA as one wave of three CTAs an SM holds, up to eight, from 16384
    // on sixteen: more spare angles, which tokens of a block behind a CTA's last cost twice,
    // fewer keep the last wave full (32768 tokens: 135 us with eight, 134 with sixteen; 8192:
    // 41 and 46; 773 tokens of 256 requests: with one 13.1, two 11.6, four 16.6).
    a.tokens = 1;
    const int most_tokens = a.num_tokens < 16384 ? 8 : kMaxTokens;
    while (a.tokens < most_tokens && (a.num_tokens + a.tokens - 1) / a.tokens > 456) a.tokens *= 2;
    const int ctas = (a.num_tokens + a.tokens - 1) / a.tokens;
    // few tokens: several CTAs share the heads of each
    const int most = max((2 * a.kv_heads + kWarps - 1) / kWarps,
                         (a.q_heads * (kDim / 16) + kThreads - 1) / kThreads);
    int splits = 1;
    while (splits < most && splits < 16 && ctas * splits < 304) splits *= 2;
    const size_t smem = (size_t)(a.tokens + kBlock - 1) * a.pairs * sizeof(float2);  // <= 32 KB
    return launch_kernel(a.tokens <= 2 ? quant_append_kernel<T, kInt8, kDim, true>
                                       : quant_append_kernel<T, kInt8, kDim, false>,
                         dim3((unsigned)ctas, (unsigned)splits), dim3(kThreads), smem, stream,
                         true, 1, a);
}

// ---- reading back ---------------------------------------------------------------

constexpr int kReadTokens = 16;  // of a CTA

struct ReadArgs {
    BatchArgs bt;
    int32_t kv_heads;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* scales;
    void* k_out;
    void* v_out;
    int64_t k_stride, v_stride;
    int32_t* status;
};

// A scale as the reading calls take it.
__device__ __forceinline__ float taken_scale(float s) {
    return fminf(fmaxf(s, kMinScale), kMaxScale);
}

template <typename T, bool kInt8, int kDim>
__global__ void __launch_bounds__(kThreads) quant_read_kernel(const ReadArgs a) {
    constexpr int kUnits = kDim / 16;
    __shared__ int64_t s_slot[kReadTokens];
    const int tid = threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * kReadTokens;
    const int count = (int)min((int64_t)kReadTokens, a.bt.total_q - first);
    grid_dependents_launch();
    grid_dependency_wait();
    if (tid < 32) {
        // the requests of the CTA's first and last token, by 32 at a time, and between them
        // each token's own: a binary search of 256 would wait eight times
        auto request = [&](int t) {
            int lo = 0, n = a.bt.num_requests;
            while (n > 1) {
                const int step = (n + 31) / 32, at = lo + min(tid * step, n - 1);
                const bool below = __ldg(a.bt.q_offsets + at) <= t;
                const int part = max(__popc(__ballot_sync(0xffffffffu, below && tid * step < n)), 1);
                lo += (part - 1) * step;
                n = min(step, n - (part - 1) * step);
            }
            return lo;
        };
        const int from = request((int)first), to = request((int)first + count - 1);
        const int t = (int)first + min(tid, count - 1);
        int b = from, last = to;
        while (b < last) {
            const int mid = (b + last + 1) >> 1;
            if (__ldg(a.bt.q_offsets + mid) <= t) b = mid;
            else last = mid - 1;
        }
        const int q0 = __ldg(a.bt.q_offsets + b), q1 = __ldg(a.bt.q_offsets + b + 1);
        const int seq = __ldg(a.bt.seq_lens + b);
        int64_t slot = -1;
        // rows behind the last request's are nobody's: a step of fixed size has such
        const bool spare = b + 1 == a.bt.num_requests && q0 >= 0 && q0 <= q1 && q1 <= t;
        if (spare) {
            // keeps what it has
        } else if (q0 < 0 || t < q0 || t >= q1 || q1 > a.bt.total_q || q1 - q0 > a.bt.max_q ||
                   seq < 0 || seq > a.bt.max_seq) {
            if (tid < count) record_error(a.status, DSA_ERR_DEVICE_CHECK);
        } else if (tid < count) {
            const int pos = seq - (q1 - t);
            if (pos >= 0) {
                const int page = page_lookup(a.bt, b, pos / kPage, a.status);
                if (page >= 0) slot = (int64_t)page * kPage + pos % kPage;
            }
        }
        if (tid < count) s_slot[tid] = slot;
    }
    __syncthreads();
    // neighbouring lanes: units of a row, then rows of a head, which lie together in a page
    const int items = 2 * a.kv_heads * kReadTokens * kUnits;
    for (int i = tid + kThreads * blockIdx.y; i < items; i += kThreads * gridDim.y) {
        const int unit = i % kUnits, j = i / kUnits % kReadTokens;
        const int rest = i / (kUnits * kReadTokens);
        const int which = rest >= a.kv_heads, head = rest - which * a.kv_heads;
        T* out = static_cast<T*>(which ? a.v_out : a.k_out);
        const int64_t slot = j < count ? s_slot[j] : -1;
        if (out == nullptr || slot < 0) continue;
        const int64_t page_head = slot / kPage * a.kv_heads + head;
        const int row = (int)(slot % kPage);
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(
                                  (which ? a.v_pages : a.k_pages) +
                                  (page_head * kPage + row) * kDim) + unit);
        const float scale = taken_scale(
            __ldg(a.scales + (page_head * 2 + which) * kPageBlocks + row / kBlock));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float x[8], y[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float v[4];
            decode4<kInt8>(w[c], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) (c < 2 ? x : y)[4 * (c & 1) + e] = v[e] * scale;
        }
        T* dst = out + (first + j) * (which ? a.v_stride : a.k_stride) + head * kDim + unit * 16;
        store8(dst, x);
        store8(dst + 8, y);
    }
}

template <typename T, bool kInt8, int kDim>
cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream) {
    const int ctas = (a.bt.total_q + kReadTokens - 1) / kReadTokens;
    const int items = 2 * a.kv_heads * kReadTokens * (kDim / 16);
    int splits = 1;
    while (splits < 64 && ctas * splits < 608 && splits * kThreads < items) splits *= 2;
    return launch_kernel(quant_read_kernel<T, kInt8, kDim>,
                         dim3((unsigned)ctas, (unsigned)splits), dim3(kThreads), 0, stream, true, 1,
                         a);
}

// f.run<T, kInt8, kDim>() for a cache and a 16-bit type.
template <typename T, bool kInt8, typename F>
cudaError_t by_dim(int head_dim, const F& f) {
    switch (head_dim) {
        case 64: return f.template run<T, kInt8, 64>();
        case 128: return f.template run<T, kInt8, 128>();
        default: return f.template run<T, kInt8, 256>();
    }
}

template <typename F>
cudaError_t by_type(const dsa_quant_cache& cache, int format, const F& f) {
    const bool int8 = cache.format == DSA_QUANT_INT8;
    if (format == DSA_FLOAT_BF16)
        return int8 ? by_dim<__nv_bfloat16, true>(cache.head_dim, f)
                    : by_dim<__nv_bfloat16, false>(cache.head_dim, f);
    return int8 ? by_dim<__half, true>(cache.head_dim, f)
                : by_dim<__half, false>(cache.head_dim, f);
}

struct Append {
    QuantArgs a;
    cudaStream_t stream;
    template <typename T, bool kInt8, int kDim>
    cudaError_t run() const {
        return launch_append<T, kInt8, kDim>(a, stream);
    }
};

struct Read {
    ReadArgs a;
    cudaStream_t stream;
    template <typename T, bool kInt8, int kDim>
    cudaError_t run() const {
        return launch_read<T, kInt8, kDim>(a, stream);
    }
};

}  // namespace

cudaError_t launch_quant_append(int num_tokens, const dsa_quant_cache& cache, int format,
                                const dsa_rope& rope, const int32_t* positions,
                                const int64_t* slots, int num_q_heads, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, void* q_out, int64_t q_out_stride,
                                int32_t* status, cudaStream_t stream) {
    QuantArgs a;
    a.num_tokens = num_tokens;
    a.q_heads = num_q_heads;
    a.kv_heads = cache.num_kv_heads;
    a.interleaved = rope.interleaved != 0;
    a.pairs = 0;
    int ends[3] = {0, 0, 0};
    for (int i = 0; i < 3; ++i) {
        if (i < rope.num_axes) a.pairs += rope.sections[i];
        ends[i] = a.pairs;
    }
    a.end0 = ends[0];
    a.end1 = ends[1];
    a.tokens = 0;  // set by the launch
    a.axes = rope.num_axes;
    a.slot_end = (int64_t)cache.num_pages * kPage;
    a.inv_freq = rope.inv_freq;
    a.positions = positions;
    a.slots = slots;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_pages = static_cast<uint8_t*>(cache.k_pages);
    a.v_pages = static_cast<uint8_t*>(cache.v_pages);
    a.scales = cache.scales;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.status = status;
    return by_type(cache, format, Append{a, stream});
}

cudaError_t launch_quant_read(const BatchArgs& bt, const dsa_quant_cache& cache, int format,
                              void* k_out, int64_t k_stride, void* v_out, int64_t v_stride,
                              int32_t* status, cudaStream_t stream) {
    ReadArgs a;
    a.bt = bt;
    a.kv_heads = cache.num_kv_heads;
    a.k_pages = static_cast<const uint8_t*>(cache.k_pages);
    a.v_pages = static_cast<const uint8_t*>(cache.v_pages);
    a.scales = cache.scales;
    a.k_out = k_out;
    a.v_out = v_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.status = status;
    return by_type(cache, format, Read{a, stream});
}

}  // namespace dsa
