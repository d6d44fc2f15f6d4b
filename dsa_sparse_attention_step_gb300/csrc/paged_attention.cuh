// paged_attention.cuh -- attention of new tokens over every cached position they
// see, keys and values in 64-token pages, G query heads to a KV head.
//
//   z[s] = sm_scale q . k_s,  out = sum_s e^(z[s] - m) v_s / sum_s e^(z[s] - m)
//
// One pass over the cache with a running maximum m and sum per row (a row is
// one query token's one head).  The G n_b rows of a request that share a KV head
// form row tiles of 16 to 64, so the cache is read once per row tile: at decode (at
// most 64 rows) 2 G n_b / element size flop per byte, below what the tensor cores
// need to keep up with HBM.  The kernel is bound by the reads.
//
// Work is counted in key tiles (one page of one KV head against one row tile)
// over all requests, and every CTA of a resident grid takes an equal, contiguous
// run of that list: short and long requests share the SMs evenly without the
// host knowing their lengths, and the copies of the next request run while the
// last one is finished.  A unit (request, row tile, KV head) cut by a CTA's border
// leaves unnormalised pieces in the workspace, which a second kernel joins
// (launched early, it waits for the first): piece order is fixed, so results do
// not change from run to run.  Short contexts do without the list: a cluster to a
// unit where units are few, half-size CTAs where they are many (launch_cfg).
//
// One warp or four per CTA issue the copies (TMA, 128-byte swizzled page tiles into
// a ring of stages); each consumer warp takes 16 rows and a share of a page's
// tokens with a softmax of its own, so the warps meet only when a unit is done.
// m16n8k16 MMAs with fp32 accumulation: at 16 rows a tcgen05 tile of 128 rows would
// be seven eighths empty, and the fragments' register layout lets P go from scores
// to operand without leaving the registers.  FP8 keys and values are lifted to f16
// exactly; bf16 queries then are scaled by a power of two per row, so that f16 holds
// them.  f16 probabilities are held at 2^15 times their size.  So are INT8 codes, and
// caches whose codes have a scale for every 16 tokens (kCode) bring the scales with each
// page: the keys' multiply the scores, the values' go into the exponent.
//
// Measured: one token over 2^20 positions of 32/8 heads of 128, bf16, 593 us, 7.24
// TB/s; 64 ragged FP8 requests, 64/8 heads, 335 us, 6.74 TB/s; five tokens to verify
// in each of 16 requests of up to 131072, 587 us, 6.74 TB/s.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "sm100.cuh"

namespace dsa {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace paged {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    BatchArgs bt;
    int32_t kv_heads, group;
    float inv_group;
    int32_t min_length;  // least length of a CTA's run of the list
    int32_t whole;       // every (request, row tile, KV head) by one CTA
    // without the list: CTAs of a cluster, row tiles that a request may have
    int32_t cluster, row_tiles;
    int32_t withhold;  // test only: the first page's copy is not issued
    int64_t q_stride;
    const void* q;
    const void* v_pages;
    const float* scales;  // [pages][KV heads][2][4]: of 16 tokens' keys and values (kCode)
    void* out;
    float* lse;
    float score_scale;  // sm_scale * k_scale * log2 e
    float v_scale;
    float* part_o;    // [2 * CTAs][rows][dim] unnormalised pieces
    float* part_ml;   // [2 * CTAs][rows][2]: maximum (log2 units), sum
    int32_t* joins;   // [CTAs][8]
    int32_t* status;
};

// What a joining block needs to know of the row tile whose first piece a CTA wrote.
// The first four are read as one vector.
enum { kJoinPieces, kJoinToken, kJoinRow, kJoinRows, kJoinHead, kJoinInts = 8 };

// How a cache holds its elements: by the configuration's kFp8 with one scale for all, or
// as 8-bit codes with a scale for every 16 tokens.
enum { kCodePlain, kCodeE4m3, kCodeInt8 };
constexpr int kBlock = DSA_QUANT_BLOCK;
constexpr float kMinBlockScale = 0x1p-48f, kMaxBlockScale = 0x1p33f;

// The consumer warps: kNG groups, each taking every kNG-th page of the CTA's run;
// within a group kWM warps along the rows (16 each) by kWN warps along the page's
// tokens.  8 or 12 warps, or 4 of each of an SM's two CTAs, as many as the
// accumulators' registers allow: a warp's softmax is a chain of dependent
// instructions, and only other warps fill its gaps.
// kKvFp8: elements of one byte, lifted to f16.
template <int kD, bool kKvFp8, int kWM_, int kWN_, int kNG_, bool kDirect_ = false,
          int kCtas_ = 1, int kCode_ = kCodePlain>
struct AttnCfg {
    static constexpr int kDim = kD;
    static constexpr bool kDirect = kDirect_;  // a cluster to a unit, no list
    static constexpr int kCtas = kCtas_;       // of an SM
    static constexpr int kCode = kCode_;
    static constexpr bool kScaled = kCode != kCodePlain, kInt8 = kCode == kCodeInt8;
    using Direct = AttnCfg<kD, kKvFp8, kWM_, kWN_, kNG_, true, 1, kCode>;
    static constexpr bool kFp8 = kKvFp8;
    static constexpr int kWM = kWM_, kWN = kWN_, kNG = kNG_;
    static constexpr int kRows = 16 * kWM;
    static constexpr int kConsumers = kWM * kWN * kNG;
    static constexpr int kTokenWarps = kWN * kNG;  // warps that share a row
    static constexpr int kThreads = 32 * (kConsumers + 4);
    static constexpr int kRowBytes = kD * (kKvFp8 ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;
    static constexpr int kBoxes = kRowBytes / kBoxBytes;
    static constexpr int kTileBytes = kPage * kRowBytes;  // keys or values of one page
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kScaleBytes = kScaled ? 2 * kPage / kBlock * 4 : 0;  // of a page
    static constexpr int kTokens = kPage / kWN;                       // of a page, per warp
    static constexpr int kSub = kD == 256 || kTokens < 32 ? 16 : 32;  // softmax step
    static constexpr int kPairs = kRowBytes / 32;  // pairs of 16-byte chunks in a row
    static constexpr int kTilesD = kD / 8;         // accumulator tiles along the dims
    // Q fragments stay in registers where they fit beside the accumulators and the
    // 32-token softmax step, which is worth more (verification of five tokens: 622
    // us with both in registers and 16-token steps, 587 so)
    static constexpr bool kQSmem = kD == 256 || (kD == 128 && kConsumers == 12);
    static constexpr int kQBytes = kRows * kD * 2;
    // The join of the warps takes so many dims at a time; 64 keep all threads busy
    // where the buffer then takes no stage that is needed.
    static constexpr int kMergeDims = kRows == 16 && (kD < 256 || kKvFp8) ? 64 : 32;
    static constexpr int kMergeLd = kMergeDims + 8;  // floats; keeps fragment stores apart
    static constexpr int kMergeBytes = kTokenWarps * kRows * kMergeLd * 4;
    static constexpr int kMlBytes = kTokenWarps * kRows * 8 + kRows * 4;
    static constexpr int kFixed = 1024 + kQBytes + kMergeBytes + kMlBytes;
    static constexpr int kFit = ((kCtas == 1 ? 226 : 111) * 1024 - kFixed) / kStageBytes;
    // A copying warp takes about 500 cycles a page (wait, arm, issue).  FP8 pages of
    // up to 16 KB come faster than that: four warps copy every fourth page each (64
    // dims: 92.5 -> 55.7 us for 152 requests of 16384; 128: 357 -> 350 us for the
    // ragged batch of 64).  16-bit pages of 16 KB gain nothing in long requests and
    // lose 13% in short ones to the shallower ring.  The stages then are a multiple
    // of four, so that each warp keeps its own, and of kNG, so that full barriers and
    // stages go together (below).
    static constexpr int kMost = kFit < 12 ? kFit : 12;
    static constexpr int kProducers =
        kKvFp8 && kStageBytes <= 16384 && kMost >= 4 && kMost / 4 * 4 % kNG == 0 ? 4 : 1;
    static constexpr int kStages = kMost / kProducers * kProducers;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    // Page n of a CTA's run lands in stage n mod kStages but signals full barrier
    // n mod kFull, a multiple of kNG: a barrier then belongs to one group, which sees
    // each of its phases.  (Copies may finish out of order; a group that waited on a
    // barrier another group's page still has to complete would take the phase before
    // for its own.)  A barrier may be armed again once its page has been released:
    // one copying warp has waited for the release of all pages up to n - kStages, so
    // kFull >= kStages will do; of several each knows its own stage only.
    static constexpr int kFull = (kStages + kNG - 1) / kNG * kNG;
    static_assert(kProducers == 1 || kFull == kStages, "");
    // What a unit costs besides its tiles (queries, the join of the warps: about 2000
    // to 5000 cycles), in tiles at the rate at which HBM brings them (24 bytes a cycle).
    static constexpr int kUnitCost =
        ((kD == 64 ? 2000 : 5000) * 24 + kStageBytes / 2) / kStageBytes;
    static_assert(kUnitCost <= 8, "");
    // The launch gives every thread kLaunchRegs registers (launch bounds); the copying
    // warpgroup then hands most of its share to the consumers.
    static constexpr int kLaunchRegs = 65536 / (kThreads * kCtas) / 8 * 8;
    static constexpr int kProducerRegs =
        kConsumers == 12 ? 56 : kD == 256 || kConsumers == 4 ? 40 : 72;
    static constexpr int kConsumerRegs = kConsumers == 12 ? 152 : kD == 256 ? 232 : 208;
    static_assert(128 * kProducerRegs + 32 * kConsumers * kConsumerRegs <= kThreads * kLaunchRegs,
                  "setmaxnreg.inc would wait forever");
    static_assert(kConsumers == 4 * (3 - kCtas) || kConsumers == 12, "");
    static_assert(kStages >= 2 && kStages * kStageBytes >= kRows * (kD + 2) * 4, "");
};

// ---- the list of key tiles ----------------------------------------------------

// Row number / group: the token of a row within its request.
__device__ __forceinline__ int token_of(const AttnParams& p, int row) {
    if (row >= 1 << 24) return row / p.group;
    int t = (int)((float)row * p.inv_group);  // off by one at most
    const int rest = row - t * p.group;
    t += rest >= p.group;
    t -= rest < 0;
    return t;
}

// One request as the schedule sees it; rows = 0 when it brings no tokens or its
// metadata contradict the host sizes.  Unlike the other kernels' check this
// takes seq < n_b (rows that see nothing).
struct Request {
    int q0, nb, seq, rows;
};

struct RawRequest {
    int q0, q1, seq;
};

__device__ __forceinline__ RawRequest raw_request(const AttnParams& p, int b) {
    return {__ldg(p.bt.q_offsets + b), __ldg(p.bt.q_offsets + b + 1), __ldg(p.bt.seq_lens + b)};
}

__device__ __forceinline__ Request request_of(const AttnParams& p, const RawRequest& x,
                                              int32_t* status) {
    const bool ok = x.q0 >= 0 && x.q1 >= x.q0 && x.q1 <= p.bt.total_q &&
                    x.q1 - x.q0 <= p.bt.max_q && x.seq >= 0 && x.seq <= p.bt.max_seq;
    if (!ok) record_error(status, DSA_ERR_DEVICE_CHECK);
    const int nb = ok ? x.q1 - x.q0 : 0;
    return {x.q0, nb, x.seq, nb * p.group};
}

// Key tiles that row tile rt of a request needs: pages up to the last position
// its last row sees.
template <int kRows>
__device__ __forceinline__ int tiles_of(const AttnParams& p, const Request& r, int rt) {
    const int last = min(r.rows, (rt + 1) * kRows) - 1;
    const int vis = last == r.rows - 1 ? r.seq : r.seq - r.nb + token_of(p, last) + 1;
    return vis > 0 ? (vis + kPage - 1) / kPage : 0;
}

// A place in the list.  Units run over requests, row tiles, KV heads.  A unit
// without key tiles counts as one tile, so that somebody writes its empty rows.
// The next request's metadata are loaded one request ahead.
template <int kRows>
struct Cursor {
    int b, rt, h, tiles;
    Request r;
    RawRequest ahead;

    __device__ __forceinline__ int cost() const { return tiles > 0 ? tiles : 1; }
    __device__ __forceinline__ void look_ahead(const AttnParams& p) {
        ahead = raw_request(p, min(b + 1, p.bt.num_requests - 1));
    }
    // False at the end of the list.
    __device__ __forceinline__ bool next(const AttnParams& p) {
        if (++h < p.kv_heads) return true;
        h = 0;
        if ((rt + 1) * kRows < r.rows) {
            ++rt;
        } else {
            rt = 0;
            do {
                if (++b >= p.bt.num_requests) return false;
                r = request_of(p, ahead, nullptr);
                look_ahead(p);
            } while (r.rows == 0);
        }
        tiles = tiles_of<kRows>(p, r, rt);
        return true;
    }
};

// In the list a unit is as long as its tiles and kUnitCost more in front of them,
// for what a unit costs a CTA besides its tiles.  Positions are 32-bit: the host
// refuses longer lists.  (Offsets that run back and forth could still make one, and
// a wrong cut of it; every walk therefore ends with the last request, and pieces
// with the last CTA.)
template <int kRows>
struct Share {
    uint32_t begin, end, per;  // this CTA's run of the list
    uint32_t offset;           // of the first position, in the unit at
    Cursor<kRows> at;
};

// A CTA's way through its run.  Copying and consuming warps each take their own,
// after they have parted: with the start in shared variables the compiler moves
// common subexpressions above the fork and spills them in both.
template <typename C>
struct Walk {
    uint32_t pos, end, offset;  // offset of pos in u
    int tile, count;            // of u in this run: first tile, tiles
    Cursor<C::kRows> u;

    __device__ __forceinline__ Walk(const AttnParams& p, const Share<C::kRows>& s)
        : pos(s.begin), end(s.end), offset(s.offset), u(s.at) {
        if (C::kDirect) {
            tile = s.offset;
            count = s.per;
        } else {
            u.look_ahead(p);
            settle(p);
        }
    }
    // Makes (tile, count) this run's part of u, passing over units of which it has
    // none.  With `whole` a unit belongs to the run that holds its first position.
    __device__ __forceinline__ void settle(const AttnParams& p) {
        while (pos < end) {
            const uint32_t length = C::kUnitCost + u.cost();
            const uint32_t stop = p.whole ? length : min(length, offset + (end - pos));
            tile = max((int)offset - C::kUnitCost, 0);
            count = max((int)stop - C::kUnitCost, 0) - tile;
            if (p.whole && offset > 0) count = 0;
            if (count > 0) return;
            advance(p);
        }
    }
    __device__ __forceinline__ void advance(const AttnParams& p) {
        pos += C::kUnitCost + u.cost() - offset;
        offset = 0;
        if (pos < end && !u.next(p)) pos = end;
    }
    __device__ __forceinline__ void next(const AttnParams& p) {
        if (C::kDirect) {
            pos = end;
        } else {
            advance(p);
            settle(p);
        }
    }
    __device__ __forceinline__ bool complete(const AttnParams& p) const {
        return C::kDirect ? p.cluster == 1 : count == u.cost();
    }
};

// The unit of this CTA's cluster and the CTA's part of its tiles, without a list:
// begin = end where the request has no such row tile.
template <typename C>
__device__ void find_unit(const AttnParams& p, Share<C::kRows>* s) {
    if (threadIdx.x == 0) {
        const int unit = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
        const int each = p.row_tiles * p.kv_heads;
        const int b = unit / each, rt = unit % each / p.kv_heads;
        const Request r = request_of(p, raw_request(p, b), p.status);
        const int tiles = rt * C::kRows < r.rows ? tiles_of<C::kRows>(p, r, rt) : 0;
        s->begin = 0;
        s->end = rt * C::kRows < r.rows;
        s->offset = (uint32_t)(tiles * rank / p.cluster);
        s->per = (uint32_t)(tiles * (rank + 1) / p.cluster) - s->offset;
        s->at.b = b;
        s->at.rt = rt;
        s->at.h = unit % p.kv_heads;
        s->at.tiles = tiles;
        s->at.r = r;
    }
    __syncthreads();
}

// Whole CTA: this CTA's share of the list.  Each thread adds up a run of
// requests; sums over the warps place the warps, and in the warp whose run holds
// the CTA's first position a scan finds the thread, which looks it up.
template <typename C>
__device__ void find_share(const AttnParams& p, Share<C::kRows>* s, uint32_t* s_warp) {
    constexpr int kWarps = C::kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = p.bt.num_requests;
    const int each = (n + C::kThreads - 1) / C::kThreads;
    const int first = tid * each;
    uint32_t sum = 0;
    Request r = {0, 0, 0, 0};
    for (int b = first; b < min(n, first + each); ++b) {
        r = request_of(p, raw_request(p, b), blockIdx.x == 0 ? p.status : nullptr);
        for (int rt = 0; rt * C::kRows < r.rows; ++rt)
            sum += (max(1, tiles_of<C::kRows>(p, r, rt)) + C::kUnitCost) * p.kv_heads;
    }
    const uint32_t warp_sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) s_warp[warp] = warp_sum;
    if (tid == 0) s->begin = s->end = 0;  // for a CTA without work
    __syncthreads();
    uint32_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    const uint32_t per = max((total + gridDim.x - 1) / gridDim.x, (uint32_t)p.min_length);
    const uint32_t begin = (uint32_t)min((unsigned long long)per * blockIdx.x,
                                         (unsigned long long)total);
    if (begin < total && before <= begin && begin < before + warp_sum) {
        uint32_t upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        before += upto - sum;
        if (before <= begin && begin < before + sum) {
            for (int b = first; b < min(n, first + each); ++b) {
                if (each > 1) r = request_of(p, raw_request(p, b), nullptr);
                int rt = 0;
                for (; rt * C::kRows < r.rows; ++rt) {
                    const int tiles = tiles_of<C::kRows>(p, r, rt);
                    const uint32_t length = max(1, tiles) + C::kUnitCost;
                    if (begin < before + length * p.kv_heads) {
                        const uint32_t h = (begin - before) / length;
                        s->begin = begin;
                        s->end = min(total, begin + per);
                        s->per = per;
                        s->offset = begin - before - h * length;
                        s->at.b = b;
                        s->at.rt = rt;
                        s->at.h = (int)h;
                        s->at.tiles = tiles;
                        s->at.r = r;
                        break;
                    }
                    before += length * p.kv_heads;
                }
                if (rt * C::kRows < r.rows) break;  // found
            }
        }
    }
    __syncthreads();
}

// ---- fragments -----------------------------------------------------------------

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Infinite and NaN elements in 16 bytes of a cache: whether there are any, and the rest
// with zeros in their place.
template <bool kFp8, bool kBf16>
__device__ __forceinline__ bool any_not_finite(const uint4& u) {
    if (kFp8)  // magnitude 0x7f
        return (((u.x & 0x7f7f7f7fu) + 0x01010101u | (u.y & 0x7f7f7f7fu) + 0x01010101u |
                 (u.z & 0x7f7f7f7fu) + 0x01010101u | (u.w & 0x7f7f7f7fu) + 0x01010101u) &
                0x80808080u) != 0;
    const uint32_t top = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                  __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    constexpr uint32_t kInf = kBf16 ? 0x7f80 : 0x7c00;
    return max(top & 0xffffu, top >> 16) >= kInf;
}

template <bool kFp8, bool kBf16>
__device__ __forceinline__ uint4 finite_part(const uint4& u) {
    constexpr uint32_t kMask = kFp8 ? 0x7f7f7f7fu : kBf16 ? 0x7f807f80u : 0x7c007c00u;
    auto part = [](uint32_t w) {
        return w & ~(kFp8 ? __vcmpeq4(w & kMask, kMask) : __vcmpeq2(w & kMask, kMask));
    };
    return make_uint4(part(u.x), part(u.y), part(u.z), part(u.w));
}

// Four codes as two pairs of f16, exact.  INT8: with the sign bit flipped a code is c +
// 128, as the low byte of an f16 in 1024 .. 2047 it is c + 1152.
template <bool kInt8>
__device__ __forceinline__ void lift(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    if (kInt8) {
        const uint32_t u = codes ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
        auto pair = [&](uint32_t select) {
            const uint32_t w = __byte_perm(u, 0x64646464u, select);
            const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&w), bias);
            return *reinterpret_cast<const uint32_t*>(&r);
        };
        lo = pair(0x4140);
        hi = pair(0x4342);
        return;
    }
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if (kBf16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// An unnormalised output as a result; 0 where the sum is 0 (factor 0), whatever x is.
__device__ __forceinline__ float result(float x, float factor) {
    return factor == 0.f ? 0.f : x * factor;
}

// A maximum as a subtrahend: 0 for a row that has seen nothing yet.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

// 3-D tiled TMA load of one box at (x, y, z).
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* tmap, int x, int y, int z,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Barrier over the threads of a cluster that have not exited.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Loads from the shared memory of the cluster's CTA `rank`, at this CTA's address.
__device__ __forceinline__ float2 cluster_load2(uint32_t addr, int rank) {
    float2 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
                 "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr), "r"(rank));
    return v;
}

__device__ __forceinline__ float4 cluster_load4(uint32_t addr, int rank) {
    float4 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr), "r"(rank));
    return v;
}

template <bool kBf16>
__device__ __forceinline__ float unpack(uint16_t bits) {
    return kBf16 ? __uint_as_float((uint32_t)bits << 16) : __half2float(__ushort_as_half(bits));
}

// The value at a unit's position, if it is infinite or NaN, else 0: added to a row that
// sees it, as good as its product with the probability.
template <typename C, bool kBf16>
__device__ __forceinline__ float not_finite_value(const AttnParams& p, const Cursor<C::kRows>& u,
                                                  int position, int dim) {
    const int page = __ldg(p.bt.block_table + (int64_t)u.b * p.bt.max_pages + position / kPage);
    if (page < 0 || page >= p.bt.num_pages) return 0.f;
    const int64_t at =
        (((int64_t)page * p.kv_heads + u.h) * kPage + position % kPage) * C::kDim + dim;
    const float x =
        C::kFp8 ? e4m3x2_to_float2(static_cast<const uint8_t*>(p.v_pages)[at]).x
                : unpack<kBf16>(static_cast<const uint16_t*>(p.v_pages)[C::kFp8 ? 0 : at]);
    return isfinite(x) ? 0.f : x;
}

template <int kCount>
__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kCount) : "memory");
}

// ---- the kernel ----------------------------------------------------------------

// kMany: requests may bring several tokens, so that positions of the context are hidden
// from some rows.  With one token none is, and what it takes (below: values that are not
// finite) would cost short calls 1 to 4%; with several it costs long ones nothing and the
// shortest 0.2 to 0.7 us (186 requests of up to 226, 8 tokens: 9.3 -> 10.0 us).
template <typename C, bool kQBf16, bool kMany>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
paged_attention_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
    // operands of the MMAs: the cache's own type, or f16 lifted from FP8
    constexpr bool kBf16 = kQBf16 && !C::kFp8;
    // Probabilities that become f16 are held at 2^15 times their size, the row's largest
    // at 2^15: f16 has normal numbers down to 2^-29 of it then, and steps of 2^-39 below
    // (at their own size 2^-14 and 2^-24, where the positions beside a large one, 2^-25
    // each, would vanish from the product but not from the sum).
    constexpr float kPExp = kBf16 ? 0.f : 15.f, kPUnit = kBf16 ? 1.f : 0x1p-15f;
    constexpr int kD = C::kDim;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t s_full[C::kFull], s_empty[C::kStages];
    __shared__ int s_valid[C::kStages];
    __shared__ alignas(16) float s_scale[C::kScaled ? C::kStages : 1][2 * kPage / kBlock];
    __shared__ uint32_t s_warp[C::kThreads / 32];
    __shared__ Share<C::kRows> s_share;
    __shared__ int s_abort;
    __shared__ int s_cleared;  // n of the unit some of whose values were cleared
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                               ~(uintptr_t)1023);
    uint8_t* tail = ring + C::kStages * C::kStageBytes;
    uint4* s_q = reinterpret_cast<uint4*>(tail);
    float* s_merge = reinterpret_cast<float*>(tail + C::kQBytes);
    float2* s_ml = reinterpret_cast<float2*>(tail + C::kQBytes + C::kMergeBytes);
    float* s_factor = reinterpret_cast<float*>(s_ml + C::kTokenWarps * C::kRows);  // of a row

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < C::kFull; ++i) mbar_init(&s_full[i], 1);
        for (int i = 0; i < C::kStages; ++i) mbar_init(&s_empty[i], C::kWM * C::kWN);
        fence_mbar_init();
        s_abort = 0;
        s_cleared = -1;
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    grid_dependents_launch();
    grid_dependency_wait();
    if (C::kDirect) find_unit<C>(p, &s_share);
    else find_share<C>(p, &s_share, s_warp);
    volatile int* abort_flag = &s_abort;

    if (s_share.begin >= s_share.end) {
        if (tid == 0 && !C::kDirect) p.joins[blockIdx.x * kJoinInts + kJoinPieces] = 0;
        return;
    }

    if (warp >= C::kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kProducerRegs));
        const int me = warp - C::kConsumers;
        if (me >= C::kProducers) return;
        Walk<C> walk(p, s_share);
        // Copies: every kProducers-th page of the run.  The warp holds 32 table
        // entries of the unit and the first 32 of the one after it; its first lane
        // issues.
        auto entries = [&](const Cursor<C::kRows>& x, int t) {
            return t + lane < x.tiles
                       ? __ldg(p.bt.block_table + (int64_t)x.b * p.bt.max_pages + t + lane)
                       : -1;
        };
        int pieces = 0;
        // the first lane's next page: its number in the run, stage, full barrier and
        // empty parity (a fresh barrier's phase before the first counts as complete)
        int n = me, st = me, fb = me;
        uint32_t parity = 1;
        int skip = me;  // pages until this warp's next one
        bool ok = true;
        int ahead = walk.pos < walk.end ? entries(walk.u, walk.tile) : -1;
        while (walk.pos < walk.end) {
            const Cursor<C::kRows>& u = walk.u;
            const int tile = walk.tile, count = min(u.tiles, tile + walk.count) - tile;
            Walk<C> v = walk;
            v.next(p);
            const int ahead_v = v.pos < v.end ? entries(v.u, v.tile) : -1;
            int i = skip, held = 0;
            for (; i < count; i += C::kProducers) {
                if (i - held >= 32) {
                    held = i & ~31;
                    ahead = entries(u, tile + held);
                }
                const int page = __shfl_sync(0xffffffffu, ahead, i & 31);
                if (lane == 0 && ok && (ok = mbar_wait(&s_empty[st], parity, abort_flag))) {
                    const bool valid = page >= 0 && page < p.bt.num_pages;
                    s_valid[st] = valid;
                    if (p.withhold && n == 0) {
                        // nobody will arrive on this page's barrier
                    } else if (valid) {
                        mbar_arrive_expect_tx(&s_full[fb], C::kStageBytes + C::kScaleBytes);
                        uint8_t* dst = ring + st * C::kStageBytes;
                        const int z = page * p.kv_heads + u.h;
                        if constexpr (C::kScaled)
                            bulk_copy_g2s(s_scale[st], p.scales + (int64_t)z * (2 * kPage / kBlock),
                                          C::kScaleBytes, &s_full[fb]);
#pragma unroll
                        for (int x = 0; x < C::kBoxes; ++x)
                            tma_load_3d(dst + x * (kPage * C::kBoxBytes), &tm_k, x * C::kBoxBytes,
                                        0, z, &s_full[fb]);
#pragma unroll
                        for (int x = 0; x < C::kBoxes; ++x)
                            tma_load_3d(dst + C::kTileBytes + x * (kPage * C::kBoxBytes), &tm_v,
                                        x * C::kBoxBytes, 0, z, &s_full[fb]);
                    } else {
                        record_error(p.status, DSA_ERR_DEVICE_CHECK);
                        mbar_arrive(&s_full[fb]);
                    }
                    n += C::kProducers;
                    if ((fb += C::kProducers) >= C::kFull) fb -= C::kFull;
                    if ((st += C::kProducers) >= C::kStages) {
                        st -= C::kStages;
                        parity ^= 1;
                    }
                }
                __syncwarp();
            }
            skip = i - max(count, 0);
            if (me == 0 && lane == 0 && !C::kDirect && tile == 0 && !walk.complete(p)) {
                // first piece of a row tile that other CTAs finish
                int32_t* j = p.joins + blockIdx.x * kJoinInts;
                pieces = 1 + (int)((u.cost() - walk.count + s_share.per - 1) / s_share.per);
                pieces = min(pieces, (int)(gridDim.x - blockIdx.x));
                j[kJoinToken] = u.r.q0;
                j[kJoinRow] = u.rt * C::kRows;
                j[kJoinRows] = min(C::kRows, u.r.rows - u.rt * C::kRows);
                j[kJoinHead] = u.h * p.group;
            }
            walk = v;
            ahead = ahead_v;
        }
        if (me == 0 && lane == 0 && !C::kDirect)
            p.joins[blockIdx.x * kJoinInts + kJoinPieces] = pieces;
        if (lane == 0) {
            // the CTA must not exit under copies in flight, which it would if a consumer
            // gave up after the last page had been issued: wait for what was issued last
            for (int i = n - C::kProducers; i >= 0 && i > n - C::kProducers - C::kStages;
                 i -= C::kProducers)
                mbar_drain(&s_full[i % C::kFull], (i / C::kFull) & 1);
            if (*abort_flag) record_error(p.status, DSA_ERR_TIMEOUT);
        }
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kConsumerRegs));

    Walk<C> walk(p, s_share);
    const int grp = warp / (C::kWM * C::kWN);
    const int wn = warp / C::kWM % C::kWN, wm = warp % C::kWM;
    const int g = lane >> 2, c = lane & 3;
    // ldmatrix addresses of this lane: for keys the matrices are token halves by
    // chunk of a pair, for values (transposed) chunks by token halves.  The swizzle
    // XORs a row's low bits into the chunk number, so the pairs of a 128-byte row
    // have up to four different offsets and the rest is an immediate.
    constexpr int kPairsBox = C::kBoxBytes / 32;
    uint32_t k_at[kPairsBox], v_at[kPairsBox];
    {
        const int sw = C::kBoxBytes == 128 ? lane & 7 : (lane >> 1) & 3;
        const int k_row = wn * C::kTokens + ((lane >> 4) << 3) + (lane & 7);
        const int v_row = wn * C::kTokens + (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
        for (int j = 0; j < kPairsBox; ++j) {
            k_at[j] = k_row * C::kBoxBytes + (((2 * j + ((lane >> 3) & 1)) ^ sw) << 4);
            v_at[j] = C::kTileBytes + v_row * C::kBoxBytes + (((2 * j + (lane >> 4)) ^ sw) << 4);
        }
    }
    constexpr auto pair_offset = [](int j, int token) {
        return (uint32_t)(j / kPairsBox * (kPage * C::kBoxBytes) + token * C::kBoxBytes);
    };
    const uint32_t ring_u32 = smem_u32(ring);
    int n = 0;  // pages of the CTA's run before the current unit
    bool dead = false;

    // Queries of this warp's rows of a row tile, one row a warp at a time.
    constexpr int kWords = kD / 64;  // pairs of values of a row in a lane
    constexpr int kRowsWarp = (C::kRows + C::kConsumers - 1) / C::kConsumers;
    uint32_t qw[kRowsWarp][kWords];
    auto load_q = [&](const Cursor<C::kRows>& u) {
#pragma unroll
        for (int x = 0; x < kRowsWarp; ++x) {
            const int r = u.rt * C::kRows + warp + x * C::kConsumers;
            const int j = token_of(p, r);
            const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                                (int64_t)(u.r.q0 + j) * p.q_stride +
                                (int64_t)(u.h * p.group + r - j * p.group) * kD;
#pragma unroll
            for (int i = 0; i < kWords; ++i) qw[x][i] = 0;
            if (warp + x * C::kConsumers < C::kRows && r < u.r.rows) {
                if (kWords == 1) {
                    qw[x][0] = *(reinterpret_cast<const uint32_t*>(q) + lane);
                } else if (kWords == 2) {
                    const uint2 w = *(reinterpret_cast<const uint2*>(q) + lane);
                    qw[x][0] = w.x;
                    qw[x][kWords > 1 ? 1 : 0] = w.y;
                } else {
                    const uint4 w = *(reinterpret_cast<const uint4*>(q) + lane);
                    qw[x][0] = w.x;
                    qw[x][kWords > 1 ? 1 : 0] = w.y;
                    qw[x][kWords > 2 ? 2 : 0] = w.z;
                    qw[x][kWords > 2 ? 3 : 0] = w.w;
                }
            }
        }
    };
    // loaded a unit ahead where the registers allow it
    constexpr bool kQAhead = kRowsWarp * kWords <= 4;
    if (kQAhead && walk.pos < walk.end) load_q(walk.u);

    while (walk.pos < walk.end) {
        const Cursor<C::kRows>& u = walk.u;
        const int tile = walk.tile;
        const int tile_row = u.rt * C::kRows;  // first row of the row tile in its request

        if (!kQAhead) load_q(u);
        // Queries to shared memory as A fragments; a row's score factor beside them.
        // For FP8 the columns of a 16-value group are taken in the order in which the
        // lifted keys come, 4 c .. 4 c + 3.
#pragma unroll
        for (int x = 0; x < kRowsWarp; ++x) {
            const int r = warp + x * C::kConsumers;
            if (r >= C::kRows) break;
            float factor = p.score_scale;
            if (C::kFp8 && kQBf16) {
                // bf16 to f16: scale the row by a power of two that brings its
                // largest value to 1..2 (what then falls below f16's range is
                // below 2^-25 of that value), and undo it in the score factor
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    top = max(top, max(qw[x][i] & 0x7fffu, (qw[x][i] >> 16) & 0x7fffu));
                top = __reduce_max_sync(0xffffffffu, top);
                // biased exponent; infinite and NaN rows stay unscaled, and rows below
                // 2^-63, whose scores are 0 in fp32 next to any other
                const uint32_t e = top >> 7;
                float up = 1.f;
                if (e >= 64 && e < 255) {
                    const uint32_t by = min(e, 253u);  // 2^-127 is no normal number: 2..4 then
                    up = __uint_as_float((254 - by) << 23);
                    // (not below fp32's normal range, where the scores are 0 anyway: a
                    // factor of 0 would make NaN of a masked -inf)
                    factor = fmaxf(factor * __uint_as_float(by << 23), 0x1p-126f);
                }
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    qw[x][i] = pack2<false>(__uint_as_float(qw[x][i] << 16) * up,
                                            __uint_as_float(qw[x][i] & 0xffff0000u) * up);
            }
            // times any block's scale it stays within fp32's normal range
            if (C::kScaled) factor = fminf(fmaxf(factor, 0x1p-78f), 0x1p94f);
            if (lane == 0) s_factor[r] = factor;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int pair = lane * kWords + i, at = pair & 7;
                const int column = C::kFp8 ? at >> 1 : at & 3, half = C::kFp8 ? at & 1 : at >> 2;
                reinterpret_cast<uint32_t*>(
                    s_q)[(((r >> 4) * (kD / 16) + (pair >> 3)) * 32 + (r & 7) * 4 + column) * 4 +
                         2 * half + ((r >> 3) & 1)] = qw[x][i];
            }
        }
        if (kQAhead) {  // the next unit's, for which there is time until this one is done
            Walk<C> v = walk;
            v.next(p);
            if (v.pos < v.end) load_q(v.u);
        }
        consumer_sync<32 * C::kConsumers>();
        const float f[2] = {s_factor[16 * wm + g], s_factor[16 * wm + g + 8]};
        uint32_t qf[C::kQSmem ? 1 : kD / 16][4];
        if (!C::kQSmem) {
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                const uint4 w = s_q[(wm * (kD / 16) + ks) * 32 + lane];
                qf[C::kQSmem ? 0 : ks][0] = w.x;
                qf[C::kQSmem ? 0 : ks][1] = w.y;
                qf[C::kQSmem ? 0 : ks][2] = w.z;
                qf[C::kQSmem ? 0 : ks][3] = w.w;
            }
        }

        // what this thread's rows, g and g + 8 of the warp's 16, see
        int vis[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = tile_row + 16 * wm + g + 8 * x;
            vis[x] = r < u.r.rows ? u.r.seq - u.r.nb + token_of(p, r) + 1 : 0;
        }
        // and what the row tile's first row, and so every row of it, sees
        const int vis_first = u.r.seq - u.r.nb + token_of(p, tile_row) + 1;

        float o[C::kTilesD][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < C::kTilesD; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

        const int last = min(u.tiles, tile + walk.count);
        // this group's pages: those whose number in the run is grp modulo kNG.  The join
        // takes the groups from the one with the unit's first page on, so that the
        // order of its sums does not depend on the units before this one.
        const int turn = (grp + C::kNG - n % C::kNG) % C::kNG;
        const int tw = turn * C::kWN + wn;  // of the warps that share rows
        for (int t = tile + turn; t < last; t += C::kNG) {
            const int i_run = n + (t - tile), st = i_run % C::kStages;
            if (!dead)
                dead = !mbar_wait(&s_full[i_run % C::kFull], (i_run / C::kFull) & 1, abort_flag);
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;
            if (s_valid[st]) {
                const uint32_t stage = ring_u32 + st * C::kStageBytes;
                const int first = t * kPage + wn * C::kTokens;  // this warp's first position
                if (!C::kInt8 && first + C::kTokens > u.r.seq) {
                    // stale rows past the context may hold anything: p is 0 there, but
                    // 0 * NaN is not
                    const int keep = max(0, u.r.seq - first);
                    uint8_t* v = ring + st * C::kStageBytes + C::kTileBytes;
                    for (int i = lane; i < (C::kTokens - keep) * (C::kRowBytes / 16); i += 32) {
                        const int r = wn * C::kTokens + keep + i / (C::kRowBytes / 16);
                        const int x = i % (C::kRowBytes / 16), per = C::kBoxBytes / 16;
                        *reinterpret_cast<uint4*>(v + (x / per) * (kPage * C::kBoxBytes) +
                                                  r * C::kBoxBytes + (x % per) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();  // the next copy into this stage comes after
                    __syncwarp();
                }
                const int shown = min(first + C::kTokens, u.r.seq);
                if (kMany && !C::kInt8 && max(first, vis_first) < shown) {
                    // the same for infinite and NaN values of new tokens that some of the
                    // row tile's rows do not see; the others get them when the unit is done
                    constexpr int kChunks = C::kRowBytes / 16, kPer = C::kBoxBytes / 16;
                    const int x = lane % kChunks, r0 = max(first, vis_first) + lane / kChunks;
                    uint8_t* v = ring + st * C::kStageBytes + C::kTileBytes +
                                 (x / kPer) * (kPage * C::kBoxBytes) + (x % kPer) * 16;
                    bool bad = false;
#pragma unroll 1
                    for (int r = r0; r < shown; r += 32 / kChunks)
                        bad |= any_not_finite<C::kFp8, kBf16>(
                            *reinterpret_cast<const uint4*>(v + r % kPage * C::kBoxBytes));
                    if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                        for (int r = r0; r < shown; r += 32 / kChunks) {
                            uint4* at = reinterpret_cast<uint4*>(v + r % kPage * C::kBoxBytes);
                            *at = finite_part<C::kFp8, kBf16>(*at);
                        }
                        *static_cast<volatile int*>(&s_cleared) = n;
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int sub = 0; sub < C::kTokens; sub += C::kSub) {
                    constexpr int kNt = C::kSub / 8;
                    float s[kNt][4];
#pragma unroll
                    for (int i = 0; i < kNt; ++i)
                        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
                    constexpr int kSteps = C::kFp8 ? 2 : 1;  // MMA steps in a chunk pair
#pragma unroll
                    for (int j = 0; j < C::kPairs; ++j) {
                        uint32_t qa[kSteps][4];
#pragma unroll
                        for (int x = 0; x < kSteps; ++x) {
                            if (C::kQSmem) {
                                const uint4 w =
                                    s_q[(wm * (kD / 16) + kSteps * j + x) * 32 + lane];
                                qa[x][0] = w.x;
                                qa[x][1] = w.y;
                                qa[x][2] = w.z;
                                qa[x][3] = w.w;
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    qa[x][i] = qf[C::kQSmem ? 0 : kSteps * j + x][i];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < C::kSub / 16; ++i) {
                            uint32_t k[4];
                            ldmatrix4(k,
                                      stage + k_at[j % kPairsBox] + pair_offset(j, sub + 16 * i));
                            if (C::kFp8) {
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    uint32_t k0, k1, k2, k3;
                                    lift<C::kInt8>(k[x], k0, k1);
                                    lift<C::kInt8>(k[2 + x], k2, k3);
                                    mma16816<false>(s[2 * i], qa[x % kSteps], k0, k1);
                                    mma16816<false>(s[2 * i + 1], qa[x % kSteps], k2, k3);
                                }
                            } else {
                                mma16816<kBf16>(s[2 * i], qa[0], k[0], k[1]);
                                mma16816<kBf16>(s[2 * i + 1], qa[0], k[2], k[3]);
                            }
                        }
                    }
                    if (t * kPage + kPage > vis_first) {
#pragma unroll
                        for (int i = 0; i < kNt; ++i)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (first + sub + 8 * i + 2 * c + (x & 1) >= vis[x >> 1])
                                    s[i][x] = -INFINITY;
                    }
                    // With a scale k, v to a block, z = s f k; the maximum is that of z +
                    // log2 v, and what becomes the operand is p = 2^(z + log2 v - m), the
                    // probability as the codes of the values want it.  p / v is summed.
                    constexpr int kBlocks = C::kScaled ? C::kSub / kBlock : 1;
                    float fk[kBlocks][2], lv[kBlocks], iv[kBlocks];
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i) {
                        fk[i][0] = f[0];
                        fk[i][1] = f[1];
                        lv[i] = 0.f;
                        iv[i] = 1.f;
                        if (C::kScaled) {
                            const float* at = s_scale[C::kScaled ? st : 0] +
                                              (wn * C::kTokens + sub) / kBlock + i;
                            const float k = fminf(fmaxf(at[0], kMinBlockScale), kMaxBlockScale);
                            const float v = fminf(fmaxf(at[kPage / kBlock], kMinBlockScale),
                                                  kMaxBlockScale);
                            fk[i][0] *= k;
                            fk[i][1] *= k;
                            lv[i] = lg2(v);
                            iv[i] = rcp(v);
                        }
                    }
                    float top[2];
                    bool grew = false;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // rounded up, as the bases below, so that no p exceeds 2^kPExp
                        if (C::kScaled) {
                            float y = -INFINITY;
#pragma unroll
                            for (int b = 0; b < kBlocks; ++b) {
                                const float(&u)[4] = s[2 * b];
                                const float(&w)[4] = s[C::kScaled ? 2 * b + 1 : 0];
                                y = fmaxf(y, __fmaf_ru(fmaxf(fmaxf(u[2 * x], u[2 * x + 1]),
                                                             fmaxf(w[2 * x], w[2 * x + 1])),
                                                       fk[b][x], lv[b]));
                            }
                            top[x] = fmaxf(m[x], quad_max(y));
                        } else {
                            float y = -INFINITY;
#pragma unroll
                            for (int i = 0; i < kNt; ++i)
                                y = fmaxf(y, fmaxf(s[i][2 * x], s[i][2 * x + 1]));
                            top[x] = fmaxf(m[x], __fmul_ru(quad_max(y), f[x]));
                        }
                        grew |= top[x] > m[x];
                    }
                    if (__any_sync(0xffffffffu, grew)) {
                        const float a0 = ex2(m[0] - base_of(top[0]));
                        const float a1 = ex2(m[1] - base_of(top[1]));
                        l[0] *= a0;
                        l[1] *= a1;
#pragma unroll
                        for (int i = 0; i < C::kTilesD; ++i) {
                            o[i][0] *= a0;
                            o[i][1] *= a0;
                            o[i][2] *= a1;
                            o[i][3] *= a1;
                        }
                        m[0] = top[0];
                        m[1] = top[1];
                    }
                    // P rounded to the operand type, by half a step at most: 2^-8 of a
                    // probability in bf16, 2^-11 in f16 (2^-40 of the row's largest for
                    // those below 2^-29 of it).  The sums are of the unrounded values.
                    uint32_t pf[C::kSub / 16][4];
                    const float b0 = __fsub_ru(base_of(m[0]), kPExp);
                    const float b1 = __fsub_ru(base_of(m[1]), kPExp);
#pragma unroll
                    for (int i = 0; i < kNt; ++i) {
                        const int b = C::kScaled ? i / 2 : 0;
                        const float c0 = C::kScaled ? __fsub_ru(b0, lv[b]) : b0;
                        const float c1 = C::kScaled ? __fsub_ru(b1, lv[b]) : b1;
                        const float p0 = ex2(fmaf(s[i][0], fk[b][0], -c0));
                        const float p1 = ex2(fmaf(s[i][1], fk[b][0], -c0));
                        const float p2 = ex2(fmaf(s[i][2], fk[b][1], -c1));
                        const float p3 = ex2(fmaf(s[i][3], fk[b][1], -c1));
                        if (C::kScaled) {
                            l[0] = fmaf(p0 + p1, iv[b], l[0]);
                            l[1] = fmaf(p2 + p3, iv[b], l[1]);
                        } else {
                            l[0] += p0 + p1;
                            l[1] += p2 + p3;
                        }
                        pf[i / 2][2 * (i & 1)] = pack2<kBf16>(p0, p1);
                        pf[i / 2][2 * (i & 1) + 1] = pack2<kBf16>(p2, p3);
                    }
#pragma unroll
                    for (int i = 0; i < C::kSub / 16; ++i) {
#pragma unroll
                        for (int j = 0; j < C::kPairs; ++j) {
                            uint32_t v[4];
                            ldmatrix4_t(v,
                                        stage + v_at[j % kPairsBox] + pair_offset(j, sub + 16 * i));
                            if (C::kFp8) {
                                // each register: two tokens by two dims; split by dim
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    uint32_t v0, v1, v2, v3;
                                    lift<C::kInt8>(__byte_perm(v[2 * x], 0, 0x3120), v0, v2);
                                    lift<C::kInt8>(__byte_perm(v[2 * x + 1], 0, 0x3120), v1, v3);
                                    constexpr int kStep = C::kFp8 ? 4 : 2;
                                    constexpr int kHalf = C::kFp8 ? 2 : 0;
                                    mma16816<false>(o[kStep * j + kHalf * x], pf[i], v0, v1);
                                    mma16816<false>(o[kStep * j + kHalf * x + 1], pf[i], v2, v3);
                                }
                            } else {
                                constexpr int kStep = C::kFp8 ? 0 : 2;
                                mma16816<kBf16>(o[kStep * j], pf[i], v[0], v[1]);
                                mma16816<kBf16>(o[kStep * j + 1], pf[i], v[2], v[3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[st]);
        }
        n += max(0, last - tile);

        // Join the warps that share rows, kMergeDims at a time through shared memory:
        // each thread adds four dims of a row over the warps, weighted by what their
        // maxima lack to the common one.  (The next unit's barriers keep its writes
        // from overtaking the last pass's reads.)
        const int r = 16 * wm + g;
        l[0] = quad_sum(l[0]);
        l[1] = quad_sum(l[1]);
        if (c == 0) {
            s_ml[tw * C::kRows + r] = make_float2(m[0], l[0] * kPUnit);
            s_ml[tw * C::kRows + r + 8] = make_float2(m[1], l[1] * kPUnit);
        }
        const bool complete = walk.complete(p);
        // a cluster's pieces stay in the ring, which its only unit is done with
        float* piece_o = reinterpret_cast<float*>(ring);
        float2* piece_ml = reinterpret_cast<float2*>(piece_o + C::kRows * kD);
        const int rows = min(C::kRows, u.r.rows - tile_row);
        constexpr int kQuads = C::kMergeDims / 4;
        constexpr int kThreads = 32 * C::kConsumers;
        constexpr int kItems = (C::kRows * kQuads + kThreads - 1) / kThreads;  // rows of a thread
        const int quad = tid % kQuads * 4;
        float weight[kItems][C::kTokenWarps];
        int64_t at[kItems];  // output row, or row of the piece
        float inv[kItems];
#pragma unroll
        for (int d0 = 0; d0 < kD; d0 += C::kMergeDims) {
            if (d0 > 0) consumer_sync<32 * C::kConsumers>();  // the last pass has been read
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float* dst = s_merge + (tw * C::kRows + 16 * wm + g + 8 * x) * C::kMergeLd;
                constexpr int kPer = C::kMergeDims / 8;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float(&e)[4] = o[d0 / 8 + i];
                    if (C::kFp8) {  // tiles of even and odd dims in turn
                        if (i % 2 == 0) {
                            const float(&q)[4] = o[d0 / 8 + (C::kFp8 ? i + 1 : 0)];
                            *reinterpret_cast<float4*>(dst + 8 * i + 4 * c) = make_float4(
                                e[2 * x], q[2 * x], e[2 * x + 1], q[2 * x + 1]);
                        }
                    } else {
                        *reinterpret_cast<float2*>(dst + 8 * i + 2 * c) =
                            make_float2(e[2 * x], e[2 * x + 1]);
                    }
                }
            }
            consumer_sync<32 * C::kConsumers>();
#pragma unroll
            for (int x = 0; x < kItems; ++x) {
                const int r = (tid + kThreads * x) / kQuads;
                if (r >= rows) continue;
                if (d0 == 0) {
                    float top = -INFINITY, total = 0.f;
#pragma unroll
                    for (int w = 0; w < C::kTokenWarps; ++w)
                        top = fmaxf(top, s_ml[w * C::kRows + r].x);
                    const float base = base_of(top);
#pragma unroll
                    for (int w = 0; w < C::kTokenWarps; ++w) {
                        const float2 ml = s_ml[w * C::kRows + r];
                        const float a = ex2(ml.x - base);
                        total += ml.y * a;
                        weight[x][w] = a * kPUnit;
                    }
                    if (complete) {
                        const int j = token_of(p, tile_row + r);
                        at[x] = (int64_t)(u.r.q0 + j) * (p.kv_heads * p.group) + u.h * p.group +
                                tile_row + r - j * p.group;
                        inv[x] = total == 0.f ? 0.f : p.v_scale / total;
                        if (p.lse && quad == 0)
                            p.lse[at[x]] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
                    } else if (C::kDirect) {
                        at[x] = r;
                        if (quad == 0) piece_ml[r] = make_float2(top, total);
                    } else {
                        at[x] = (2 * (int64_t)blockIdx.x + (tile == 0 ? 1 : 0)) * C::kRows + r;
                        if (quad == 0)
                            *reinterpret_cast<float2*>(p.part_ml + 2 * at[x]) =
                                make_float2(top, total);
                    }
                }
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::kTokenWarps; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(
                        s_merge + (w * C::kRows + r) * C::kMergeLd + quad);
                    sum.x += weight[x][w] * v.x;
                    sum.y += weight[x][w] * v.y;
                    sum.z += weight[x][w] * v.z;
                    sum.w += weight[x][w] * v.w;
                }
                if (complete)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at[x] * kD + d0 +
                                              quad) =
                        make_uint2(pack2<kQBf16>(result(sum.x, inv[x]), result(sum.y, inv[x])),
                                   pack2<kQBf16>(result(sum.z, inv[x]), result(sum.w, inv[x])));
                else
                    *reinterpret_cast<float4*>((C::kDirect ? piece_o : p.part_o) + at[x] * kD + d0 +
                                               quad) = sum;
            }
        }
        if (kMany && !C::kInt8 && s_cleared == n - max(0, last - tile)) {
            // values of this run's tiles were cleared: add them to the rows that see them
            consumer_sync<32 * C::kConsumers>();
#pragma unroll 1
            for (int i = tid; i < rows * kD; i += kThreads) {
                const int row = tile_row + i / kD, d = i % kD, j = token_of(p, row);
                const int to = min(min(u.r.seq, last * kPage), u.r.seq - u.r.nb + j + 1);
                float bad = 0.f;
#pragma unroll 1
                for (int x = max(vis_first, tile * kPage); x < to; ++x)
                    bad += not_finite_value<C, kBf16>(p, u, x, d);
                if (bad == 0.f) continue;
                if (complete) {
                    const int64_t at = (int64_t)(u.r.q0 + j) * (p.kv_heads * p.group) +
                                       u.h * p.group + row - j * p.group;
                    uint16_t* out = static_cast<uint16_t*>(p.out) + at * kD + d;
                    *out = (uint16_t)pack2<kQBf16>(unpack<kQBf16>(*out) + bad, 0.f);
                } else if (C::kDirect) {
                    piece_o[i] += bad;
                } else {
                    p.part_o[(2 * (int64_t)blockIdx.x + (tile == 0 ? 1 : 0)) * C::kRows * kD + i] +=
                        bad;
                }
            }
        }
        if (C::kDirect && p.cluster > 1) {
            // the cluster's pieces, read from its CTAs' shared memory
            constexpr int kRowQuads = kD / 4;
            const uint32_t o_at = smem_u32(piece_o), ml_at = smem_u32(piece_ml);
            cluster_sync();
            for (int i = (int)(blockIdx.x % p.cluster) * 32 * C::kConsumers + tid;
                 i < rows * kRowQuads; i += p.cluster * 32 * C::kConsumers) {
                const int r = i / kRowQuads, d = i % kRowQuads * 4;
                float top = -INFINITY, total = 0.f;
                for (int k = 0; k < p.cluster; ++k)
                    top = fmaxf(top, cluster_load2(ml_at + 8 * r, k).x);
                const float base = base_of(top);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int k = 0; k < p.cluster; ++k) {
                    const float2 ml = cluster_load2(ml_at + 8 * r, k);
                    const float4 v = cluster_load4(o_at + 4 * (r * kD + d), k);
                    const float a = ex2(ml.x - base);
                    total += ml.y * a;
                    sum.x += v.x * a;
                    sum.y += v.y * a;
                    sum.z += v.z * a;
                    sum.w += v.w * a;
                }
                const int j = token_of(p, tile_row + r);
                const int64_t row = (int64_t)(walk.u.r.q0 + j) * (p.kv_heads * p.group) +
                                    walk.u.h * p.group + tile_row + r - j * p.group;
                const float scale = total == 0.f ? 0.f : p.v_scale / total;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kD + d) =
                    make_uint2(pack2<kQBf16>(result(sum.x, scale), result(sum.y, scale)),
                               pack2<kQBf16>(result(sum.z, scale), result(sum.w, scale)));
                if (p.lse && d == 0)
                    p.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
            }
            cluster_sync();  // nobody leaves while its memory is read
        }
        walk.next(p);
    }
    if (dead && lane == 0) record_error(p.status, DSA_ERR_TIMEOUT);
}

// Joins the pieces of a row tile: block (CTA that wrote the first piece, row modulo
// the grid's rows).  Groups of kDim / 4 threads take every kGroups-th piece with a
// running maximum each, then the groups are added in order.
constexpr int kJoinThreads = 128;
constexpr int kJoinRowBlocks = 16;  // most CTAs have nothing to join: few blocks for each

// One more piece (m, l, o) of a row into the sums so far.
__device__ __forceinline__ void join_piece(float& m, float& l, float4& o, const float2& ml,
                                           const float4& v) {
    const float top = fmaxf(m, ml.x), base = base_of(top);
    const float a = ex2(m - base), b = ex2(ml.x - base);
    m = top;
    l = l * a + ml.y * b;
    o.x = o.x * a + v.x * b;
    o.y = o.y * a + v.y * b;
    o.z = o.z * a + v.z * b;
    o.w = o.w * a + v.w * b;
}

template <int kDim, bool kQBf16>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const AttnParams p, int rows) {
    constexpr int kLanes = kDim / 4, kGroups = kJoinThreads / kLanes;
    __shared__ float4 s_o[kGroups][kLanes];
    __shared__ float2 s_ml[kGroups];
    grid_dependents_launch();
    grid_dependency_wait();
    const int cta = blockIdx.x;
    const int4 join = __ldcg(reinterpret_cast<const int4*>(p.joins + cta * kJoinInts));
    const int join_head = __ldcg(p.joins + cta * kJoinInts + kJoinHead);
    const int pieces = join.x;
    if (pieces == 0) return;
    const int x = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    for (int row = blockIdx.y; row < join.w; row += gridDim.y) {
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = grp; i < pieces; i += kGroups) {
            const int64_t at = (2 * (int64_t)(cta + i) + (i == 0 ? 1 : 0)) * rows + row;
            join_piece(m, l, o, __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at),
                       __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kDim) + x));
        }
        s_o[grp][x] = o;
        if (x == 0) s_ml[grp] = make_float2(m, l);
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int i = 1; i < kGroups; ++i) join_piece(m, l, o, s_ml[i], s_o[i][x]);
            const int r = join.z + row, t = token_of(p, r);
            const int64_t at =
                (int64_t)(join.y + t) * (p.kv_heads * p.group) + join_head + r - t * p.group;
            const float inv = l == 0.f ? 0.f : p.v_scale / l;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * kDim + 4 * x) =
                make_uint2(pack2<kQBf16>(result(o.x, inv), result(o.y, inv)),
                           pack2<kQBf16>(result(o.z, inv), result(o.w, inv)));
            if (p.lse && x == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        __syncthreads();
    }
}

// ---- launch --------------------------------------------------------------------

// A pool as [pages x KV heads][64 tokens][row bytes], boxes of 64 tokens by up to 128
// bytes, swizzled so that eight rows' chunks of one column fall into all banks.
inline bool encode_pool(CUtensorMap* tm, const void* base, const dsa_kv_cache& c, int row_bytes) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int box_bytes = row_bytes < 128 ? row_bytes : 128;
    cuuint64_t dims[3] = {(cuuint64_t)row_bytes, kPage, (cuuint64_t)c.num_pages * c.num_kv_heads};
    cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)row_bytes * kPage};
    cuuint32_t box[3] = {(cuuint32_t)box_bytes, kPage, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxCtas = 160;  // pieces are kept for this many CTAs
constexpr int kMinTiles = 2;

// Rows of a tile for requests of up to max_rows rows: the smallest that holds
// them, so that the cache is read once, but 16 when every request runs whole
// (a row's arithmetic must not depend on the other requests' row counts).  The
// kernel's kRows and the workspace both follow it.
inline int row_tile(int dim, int64_t max_rows, bool whole) {
    if (whole || max_rows <= 16) return 16;
    if (max_rows <= 32) return 32;
    return max_rows <= 48 && dim < 256 ? 48 : 64;  // 256 dims: eight warps, no 3 x 4
}

// At most so many units: a request of n_b tokens has n_b group / rows row tiles,
// and one more for what is left.
inline double most_units(const BatchArgs& bt, int kv_heads, int group, int rows) {
    const double each = (double)(((int64_t)bt.max_q * group + rows - 1) / rows) * bt.num_requests;
    const double all = (double)bt.total_q * group / rows + bt.num_requests;
    return (each < all ? each : all) * kv_heads;
}

struct WsLayout {
    size_t ml, joins, total;
};
inline WsLayout ws_layout(int dim, int rows) {
    WsLayout w;
    w.ml = (size_t)2 * kMaxCtas * rows * dim * sizeof(float);
    w.joins = w.ml + (size_t)2 * kMaxCtas * rows * 2 * sizeof(float);
    w.total = w.joins + (size_t)kMaxCtas * kJoinInts * sizeof(int32_t);
    return w;
}

// The kernel's attributes, set once: its dynamic shared memory, and its registers,
// of which the consumers would wait forever for more than the launch brings.
template <typename C, bool kQBf16, bool kMany>
cudaError_t prepare_kernel() {
    static const cudaError_t ready = [] {
        cudaFuncAttributes a;
        cudaError_t e = cudaFuncGetAttributes(&a, paged_attention_kernel<C, kQBf16, kMany>);
        if (e == cudaSuccess && a.numRegs < C::kLaunchRegs) e = cudaErrorInvalidConfiguration;
        return e;
    }();
    if (ready != cudaSuccess) return ready;
    return cudaFuncSetAttribute(paged_attention_kernel<C, kQBf16, kMany>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
}

template <typename C, bool kQBf16, bool kMany>
cudaError_t launch_cfg(AttnParams p, const dsa_kv_cache& cache, int* launches,
                       cudaStream_t stream) {
    CUtensorMap tm_k, tm_v;
    if (!encode_pool(&tm_k, cache.k_pages, cache, C::kRowBytes) ||
        !encode_pool(&tm_v, cache.v_pages, cache, C::kRowBytes))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    const int64_t tiles = ((int64_t)p.bt.max_seq + kPage - 1) / kPage;
    const int64_t row_tiles = ((int64_t)p.bt.max_q * p.group + C::kRows - 1) / C::kRows;
    // A unit to every SM or less, and short ones: a cluster to a unit, joined through
    // shared memory.  That spares the list's share search and the joining kernel,
    // 3 to 4 us (one request of 700: 8.4 -> 7.4 us, 152 requests of 64: 10.3 -> 4.9
    // us), but leaves a CTA alone with the longest unit: no more than 512 KB of it,
    // which a ragged batch may lose to the list as the 4 us at most.
    const int64_t units = row_tiles * p.bt.num_requests * p.kv_heads;
    // 256 dims, of which only one CTA fits an SM, also in two or three waves (107
    // requests of 146, 4 heads: 29.9 -> 26.8 us).
    if (!p.whole && units <= (C::kDim == 256 ? 3 * sms : sms)) {
        using D = typename C::Direct;
        p.cluster = 1;
        while (p.cluster < 8 && units * p.cluster * 2 <= sms) p.cluster *= 2;
        p.row_tiles = (int)row_tiles;
        if (tiles * C::kStageBytes <= (int64_t)p.cluster * (units <= sms ? 524288 : 262144)) {
            if ((e = prepare_kernel<D, kQBf16, kMany>()) != cudaSuccess) return e;
            return launch_kernel(paged_attention_kernel<D, kQBf16, kMany>,
                                 dim3((unsigned)(units * p.cluster)), dim3(D::kThreads),
                                 (size_t)D::kSmem, stream, true, p.cluster, tm_k, tm_v, p);
        }
    }
    // Many short units: a CTA to a unit, two to an SM, so that the fixed costs of one
    // overlap the other's tiles (64 requests of up to 256 positions, 4 heads of 128:
    // 13.8 -> 7.1 us).  The longest unit alone bounds the time where the list would
    // spread it: the sides meet at 13 to 16 pages of 32 KB, 16 to 30 of 16 KB and 25
    // to 35 of 8 KB, for 1 to 7 units an SM.  256 dims need more registers than half
    // an SM has for them.
    if constexpr (C::kDim < 256) {
        constexpr int kWM = C::kRows == 16 ? 1 : C::kRows == 32 ? 2 : 4;
        // 16 rows: four warps to a page for 128 16-bit dims (5.5 -> 5.2 us for the
        // shortest), else two groups of two (64 FP8 requests of 500: 9.2 us, with four
        // 10.9)
        constexpr int kWN = kWM == 1 && (C::kDim == 64 || C::kFp8) ? 2 : 4 / kWM;
        using S = AttnCfg<C::kDim, C::kFp8, kWM, kWN, 4 / (kWM * kWN), true, 2, C::kCode>;
        const int64_t small_tiles = ((int64_t)p.bt.max_q * p.group + S::kRows - 1) / S::kRows;
        const int64_t small_units = small_tiles * p.bt.num_requests * p.kv_heads;
        if (!p.whole && small_units > sms && small_units < (1 << 24) &&
            tiles * (C::kStageBytes + 8192) <= 524288) {
            p.cluster = 1;
            p.row_tiles = (int)small_tiles;
            if ((e = prepare_kernel<S, kQBf16, kMany>()) != cudaSuccess) return e;
            return launch_kernel(paged_attention_kernel<S, kQBf16, kMany>, dim3((unsigned)small_units),
                                 dim3(S::kThreads), (size_t)S::kSmem, stream, true, 1, tm_k, tm_v,
                                 p);
        }
    }
    // the workspace was laid out for this tile
    const int64_t rows = (int64_t)p.bt.max_q * p.group;
    if (C::kRows != row_tile(C::kDim, rows, p.whole != 0)) return cudaErrorInvalidValue;
    if ((e = prepare_kernel<C, kQBf16, kMany>()) != cudaSuccess) return e;
    // no more CTAs than the longest list that these host sizes allow has work for
    p.min_length = C::kUnitCost + kMinTiles;
    const double length =
        most_units(p.bt, p.kv_heads, p.group, C::kRows) * (double)(tiles + C::kUnitCost);
    int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    if (length < (double)ctas * p.min_length) ctas = (int)(length / p.min_length) + 1;
    e = launch_kernel(paged_attention_kernel<C, kQBf16, kMany>, dim3((unsigned)ctas), dim3(C::kThreads),
                      (size_t)C::kSmem, stream, true, 1, tm_k, tm_v, p);
    if (e != cudaSuccess || p.whole || ctas == 1) return e;
    *launches = 2;
    const dim3 grid((unsigned)ctas, (unsigned)(rows < kJoinRowBlocks ? rows : kJoinRowBlocks));
    return launch_kernel(paged_join_kernel<C::kDim, kQBf16>, grid, dim3(kJoinThreads), 0, stream,
                         true, 1, p, (int)C::kRows);
}

// The plan with the list: a CTA to an SM.
template <int kD, bool kFp8, int kCode, int kWM, int kWN, int kNG>
using ListCfg = AttnCfg<kD, kFp8, kWM, kWN, kNG, false, 1, kCode>;

template <int kD, bool kFp8, bool kQBf16, bool kMany, int kCode = kCodePlain>
cudaError_t launch_rows(const AttnParams& p, const dsa_kv_cache& cache, int* launches,
                        cudaStream_t stream) {
    // D = 256 has 128 accumulators a thread for 16 rows and so eight warps.  At 16 rows
    // four warps to a page halve its latency where their 16-token steps are enough to
    // keep up (one wide FP8 head: 38.4 -> 35.3 us); 64 dims and FP8 need the longer
    // steps of two (64 ragged FP8 requests: 331 us, with four 381).
    constexpr bool kFour = kD == 256 || (kD == 128 && !kFp8), kWide = kD == 256;
    switch (row_tile(kD, (int64_t)p.bt.max_q * p.group, p.whole != 0)) {
        case 16:
            return launch_cfg<ListCfg<kD, kFp8, kCode, 1, kFour ? 4 : 2, kFour ? 2 : 4>, kQBf16,
                              kMany>(p, cache, launches, stream);
        case 32:
            return launch_cfg<ListCfg<kD, kFp8, kCode, 2, 2, kWide ? 2 : 3>, kQBf16, kMany>(
                p, cache, launches, stream);
        case 48:
            if constexpr (!kWide)
                return launch_cfg<ListCfg<kD, kFp8, kCode, 3, kFour ? 2 : 1, kFour ? 2 : 4>,
                                  kQBf16, kMany>(p, cache, launches, stream);
            return cudaErrorInvalidValue;  // row_tile gives 256 dims no 48
        default:
            return launch_cfg<ListCfg<kD, kFp8, kCode, 4, kWide ? 2 : 1, kWide ? 1 : 3>, kQBf16,
                              kMany>(p, cache, launches, stream);
    }
}

template <int kD, bool kMany>
cudaError_t launch_dim(const AttnParams& p, const dsa_kv_cache& cache, int format, int* launches,
                       cudaStream_t stream) {
    const bool fp8 = cache.format == DSA_KV_FP8_E4M3;
    if (format == DSA_FLOAT_BF16)
        return fp8 ? launch_rows<kD, true, true, kMany>(p, cache, launches, stream)
                   : launch_rows<kD, false, true, kMany>(p, cache, launches, stream);
    return fp8 ? launch_rows<kD, true, false, kMany>(p, cache, launches, stream)
               : launch_rows<kD, false, false, kMany>(p, cache, launches, stream);
}

// Caches of 8-bit codes with a scale for every 16 tokens.  INT8 has no NaN, so that kMany
// changes nothing and is false; E4M3 gains by it as above (64 requests of up to 500: 16.6 ->
// 16.0 us, 200 of up to 300 19.6 -> 18.5).
template <int kD, int kCode, bool kMany>
cudaError_t launch_codes(const AttnParams& p, const dsa_kv_cache& cache, int format, int* launches,
                         cudaStream_t stream) {
    return format == DSA_FLOAT_BF16
               ? launch_rows<kD, true, true, kMany, kCode>(p, cache, launches, stream)
               : launch_rows<kD, true, false, kMany, kCode>(p, cache, launches, stream);
}

}  // namespace paged
}  // namespace dsa
