// rope_append.cu -- rotary positions on queries and keys, and the write of keys
// and values into the paged cache, in one pass.
//
// Pair i of a head is turned by positions[axis(i), t] * inv_freq[i]:
//   (x, y) -> (x cos - y sin, y cos + x sin).
// The angle is reduced in fixed point (rope.cuh): two double-precision operations per
// pair, none per value.
//
// Memory bound: every value is read and written once.  A thread moves units of 16
// values (two 16-byte loads: the two halves of eight pairs, or 16 consecutive
// values).  A CTA forms its tokens' cosines and sines, once for all heads, in shared
// memory, with its first loads in flight, and then keeps two units a thread in
// flight.  Below a million units a CTA takes as few tokens as give its threads four
// units each, so that they fill the GPU, else at least four (1024 tokens of 48 heads
// of 128: 5.9 us; 2053 of 80: 17.7 us).  From eight million on DRAM is busy anyway and
// one unit a thread, which leaves registers for a fifth CTA on the SM, is the faster
// (32768 tokens of 40 heads of 256: 206 us, 6.5 TB/s, with two 213; 4096 tokens of 48
// such heads: 44.7 and 39.4 us).
#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;       // units of a thread in flight
constexpr int kMaxTokens = 16;  // of a CTA

struct RopeArgs {
    int32_t num_tokens, q_heads, kv_heads, interleaved, pairs;
    int32_t tokens;  // of a CTA
    int32_t end0, end1;  // first pair of the second and of the third section
    int64_t slot_end;
    const double* inv_freq;
    const int32_t* positions;
    const int64_t* slots;
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_pages;
    void* v_pages;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    float k_scale, v_scale;
    int32_t* status;
};

// Eight values as E4M3 codes of x / scale (IEEE division, so that the codes are
// those of the definition), round to nearest even, saturating.
__device__ __forceinline__ void store8_fp8(uint8_t* p, const float (&x)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)), __NV_SATFINITE,
            __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)),
            __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// A unit of work: 16 values of a token's head.
template <typename T>
struct Unit {
    uint4 a, b;        // the values
    int64_t row;       // of the destination: the token for q, the cache row else
    int32_t at0, at1;  // first values of a and b in the head
    int32_t kind;      // -1: nothing to do; 0: q; 1: k; 2: v
    int32_t token, head, unit;
};

template <typename T, bool kFp8, int kDim>
__device__ __forceinline__ Unit<T> load_unit(const RopeArgs& a, int64_t first, int items, int count,
                                             int i) {
    constexpr int kUnits = kDim / 16;
    Unit<T> u;
    u.kind = -1;
    if (i >= count * items) return u;
    const int j = i / items, rest = i - j * items;
    const int head = rest / kUnits, unit = rest % kUnits;
    const int64_t t = first + j;
    u.token = j;
    u.unit = unit;
    const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.kv_heads ? 1 : 2;
    const int h = kind == 0 ? head : head - a.q_heads - (kind == 2 ? a.kv_heads : 0);
    u.head = h;
    u.row = t;
    if (kind != 0) {
        const int64_t slot = __ldg(a.slots + t);
        if (slot < 0) return u;
        if (slot >= a.slot_end) {
            record_error(a.status, DSA_ERR_DEVICE_CHECK);
            return u;
        }
        u.row = ((slot / kPage) * a.kv_heads + h) * kPage + slot % kPage;
    }
    u.kind = kind;
    const T* src = (kind == 0   ? static_cast<const T*>(a.q) + t * a.q_stride
                    : kind == 1 ? static_cast<const T*>(a.k) + t * a.k_stride
                                : static_cast<const T*>(a.v) + t * a.v_stride) +
                   h * kDim;
    const bool halves = kind != 2 && unit < a.pairs / 8 && !a.interleaved;
    u.at0 = halves ? unit * 8 : unit * 16;
    u.at1 = halves ? unit * 8 + a.pairs : unit * 16 + 8;
    u.a = *reinterpret_cast<const uint4*>(src + u.at0);
    u.b = *reinterpret_cast<const uint4*>(src + u.at1);
    return u;
}

template <typename T, bool kFp8, int kDim>
__device__ __forceinline__ void finish_unit(const RopeArgs& a, const Unit<T>& u,
                                            const float2* turns) {
    if (u.kind < 0) return;
    float x[8], y[8];
    unpack8<T>(u.a, x);
    unpack8<T>(u.b, y);
    if (u.kind != 2 && u.unit < a.pairs / 8) {
        turn16(x, y, turns + u.token * a.pairs, a.pairs / 8, u.unit, a.interleaved);
    }
    if (u.kind == 0) {
        T* dst = static_cast<T*>(a.q_out) + u.row * a.q_out_stride + u.head * kDim;
        store8(dst + u.at0, x);
        store8(dst + u.at1, y);
    } else if (kFp8) {
        uint8_t* dst = static_cast<uint8_t*>(u.kind == 1 ? a.k_pages : a.v_pages) + u.row * kDim;
        const float scale = u.kind == 1 ? a.k_scale : a.v_scale;
        store8_fp8(dst + u.at0, x, scale);
        store8_fp8(dst + u.at1, y, scale);
    } else {
        T* dst = static_cast<T*>(u.kind == 1 ? a.k_pages : a.v_pages) + u.row * kDim;
        store8(dst + u.at0, x);
        store8(dst + u.at1, y);
    }
}

template <typename T, bool kFp8, int kDim, bool kAhead>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(RopeArgs a) {
    // (cos, sin) as [tokens][4][units][2]: pair 8 u + 2 p + e of a token at [p][u][e]
    extern __shared__ float2 s_turn[];
    const int tid = threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * a.tokens;
    const int count = (int)min((int64_t)a.tokens, a.num_tokens - first);
    const int items = (a.q_heads + 2 * a.kv_heads) * (kDim / 16);
    grid_dependents_launch();
    grid_dependency_wait();

    Unit<T> u[kBatch];
    if (kAhead)
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
            u[x] = load_unit<T, kFp8, kDim>(a, first, items, count, tid + x * kThreads);
    for (int i = tid; i < count * a.pairs; i += kThreads) {
        const int j = i / a.pairs, pair = i - j * a.pairs;
        const int axis = (pair >= a.end0 ? 1 : 0) + (pair >= a.end1 ? 1 : 0);
        const int pos = __ldg(a.positions + (int64_t)axis * a.num_tokens + first + j);
        s_turn[j * a.pairs + turn_at(pair, a.pairs)] = turn_of(__ldg(a.inv_freq + pair), pos);
    }
    __syncthreads();
    if constexpr (kAhead) {
        for (int i = tid; i < count * items;) {
            i += kBatch * kThreads;
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                finish_unit<T, kFp8, kDim>(a, u[x], s_turn);
                u[x] = load_unit<T, kFp8, kDim>(a, first, items, count, i + x * kThreads);
            }
        }
    } else {
        for (int i = tid; i < count * items; i += kThreads)
            finish_unit<T, kFp8, kDim>(a, load_unit<T, kFp8, kDim>(a, first, items, count, i),
                                       s_turn);
    }
}

template <typename T, bool kFp8, int kDim>
cudaError_t launch_units(RopeArgs a, cudaStream_t stream) {
    const int items = (a.q_heads + 2 * a.kv_heads) * (kDim / 16);
    const int64_t units = (int64_t)a.num_tokens * items;
    const bool ahead = units < (1 << 23);
    const int few = 4 * kThreads / items;
    a.tokens = few < 1 ? 1 : few > kMaxTokens ? kMaxTokens : few;
    if (units >= (1 << 20) && a.tokens < 4) a.tokens = 4;
    const dim3 grid((unsigned)(((int64_t)a.num_tokens + a.tokens - 1) / a.tokens));
    const size_t smem = (size_t)a.tokens * a.pairs * sizeof(float2);  // at most 16 KB
    return launch_kernel(ahead ? rope_append_kernel<T, kFp8, kDim, true>
                               : rope_append_kernel<T, kFp8, kDim, false>,
                         grid, dim3(kThreads), smem, stream, true, 1, a);
}

template <typename T, bool kFp8>
cudaError_t launch_dim(const RopeArgs& a, int head_dim, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return launch_units<T, kFp8, 64>(a, stream);
        case 128: return launch_units<T, kFp8, 128>(a, stream);
        default: return launch_units<T, kFp8, 256>(a, stream);
    }
}

}  // namespace

cudaError_t launch_rope_append(int num_tokens, const dsa_kv_cache& cache, int format,
                               const dsa_rope& rope, const int32_t* positions,
                               const int64_t* slots, int num_q_heads, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, void* q_out, int64_t q_out_stride,
                               int32_t* status, cudaStream_t stream) {
    RopeArgs a;
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
    a.slot_end = (int64_t)cache.num_pages * kPage;
    a.inv_freq = rope.inv_freq;
    a.positions = positions;
    a.slots = slots;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_pages = cache.k_pages;
    a.v_pages = cache.v_pages;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.k_scale = cache.k_scale;
    a.v_scale = cache.v_scale;
    a.status = status;
    const bool fp8 = cache.format == DSA_KV_FP8_E4M3;
    if (format == DSA_FLOAT_BF16)
        return fp8 ? launch_dim<__nv_bfloat16, true>(a, cache.head_dim, stream)
                   : launch_dim<__nv_bfloat16, false>(a, cache.head_dim, stream);
    return fp8 ? launch_dim<__half, true>(a, cache.head_dim, stream)
               : launch_dim<__half, false>(a, cache.head_dim, stream);
}

}  // namespace dsa
