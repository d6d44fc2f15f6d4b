// quant_attention_tc.cuh -- attention of many query rows over an 8-bit cache with a scale
// for every 16 tokens, on tcgen05: verification of several tokens a request and prompt
// chunks.  The definition is paged_attention.cuh's, and so are the list of key tiles, the
// CTAs' shares of it and the joining of pieces; a row tile has 128 rows here.
//
//   S = Q K^T    M = 128 rows, N = 128 positions (64 for 256 dims); S in TMEM
//   O += P V     A = P from TMEM (f16, in the place of S), B = V; O in TMEM
//
// Codes are lifted to f16 once for all 128 rows: where mma.sync has every warp of 16 rows
// lift for itself, which bounds it (up to 40 rows of 16 requests over INT8 codes: 746 us
// where HBM takes 313; here 591), eight warps here write the lifted tiles into the swizzled
// layout that both products read (K as K-major, V as MN-major operand).  A thread of the
// softmax has half a row of S to itself: no shuffles.  A block's key scale multiplies its 16
// columns of S, its value scale goes into the exponent, as in paged_attention.cuh.
//
// Measured: 1000 tokens of 32/8 heads of 128 over 16384 E4M3 positions, 356 us, 0.73
// PFLOP/s (mma.sync: 857 us).  A step of 128 positions takes some 2900 cycles, of which a
// softmax warp works 2400 and waits 500: maxima, the meeting of a row's halves, exponentials
// and the store of P follow one another, and the products and lifts (1030 and 1300 cycles)
// run beside them.
//
// Warps: 0-7 softmax and epilogue (two threads to a row), 8-11 lift K, 12-15 lift V (and
// all eight bring Q), 16 and 18 copy (TMA into a ring of code tiles, K and V in turn), 17 issues the MMAs: S
// of the next step before O of this one, so that the tensor cores run while the softmax
// does.
#pragma once

#include "paged_attention.cuh"

namespace dsa {
namespace paged {

// What a unit costs besides its pages (its queries, its first step alone, its epilogue), in
// pages of about 1450 cycles (counted as 7: 1000 tokens over 2000 positions 92 us, so 81).
constexpr int kTcUnitCost = 20;

template <int kD, int kCode_>
struct TcCfg {
    static constexpr int kDim = kD, kCode = kCode_;
    static constexpr bool kInt8 = kCode == kCodeInt8, kDirect = false;
    static constexpr int kRows = 128;
    static constexpr int kStep = kD == 256 ? 64 : 128;  // positions
    static constexpr int kPages = kStep / kPage;
    static constexpr int kBlocks = kStep / kBlock;
    static constexpr int kThreads = 640;
    static constexpr int kLiftThreads = 128;  // of K, and of V
    static constexpr int kSlabs = kD / 64;    // 64 f16 dims are a 128-byte row of a slab
    static constexpr int kSlabBytes = kStep * 128, kQSlabBytes = kRows * 128;
    static constexpr int kQBytes = kSlabs * kQSlabBytes, kTileBytes = kSlabs * kSlabBytes;
    static constexpr int kPageBytes = kPage * kD, kEntryBytes = kPages * kPageBytes;
    static constexpr int kBoxBytes = kD < 128 ? kD : 128, kBoxes = kD / kBoxBytes;
    static constexpr int kKBufs = kD == 256 ? 1 : 2, kVBufs = kD == 64 ? 2 : 1;
    // even: a slot then always holds keys or always values, and whoever waits for one sees
    // each phase of its barrier
    static constexpr int kRing = kD == 64 ? 8 : 4;
    static_assert(kRing % 2 == 0, "");
    static constexpr int kMeta = 4;  // steps whose scales, and units whose factors, are kept
    static constexpr int kSmem = 1024 + kQBytes + (kKBufs + kVBufs) * kTileBytes +
                                 kRing * kEntryBytes;
    static constexpr uint32_t kColO = 2 * kStep, kCols = 512;
    static_assert(kColO + kD <= kCols, "");
    static constexpr int kUnitCost = kTcUnitCost;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kSoftmaxRegs = 104, kLiftRegs = 96, kControlRegs = 80;
    static_assert(256 * kSoftmaxRegs + 256 * kLiftRegs + 128 * kControlRegs <=
                      kThreads * kLaunchRegs, "setmaxnreg.inc would wait forever");
    static constexpr int kHalf = kStep / 2;  // positions of a softmax warp
    static constexpr uint32_t kIdescS = make_idesc(kFmtF16, kFmtF16, 128, kStep, false, false);
    static constexpr uint32_t kIdescO = make_idesc(kFmtF16, kFmtF16, 128, kD, false, true);
};

// What becomes f16 is held at 2^12 times the probability; a row's reference maximum
// moves when a new one exceeds it by more than 2^3, so that it stays below 2^15.
constexpr float kTcPExp = 12.f, kTcPUnit = 0x1p-12f, kTcLag = 3.f;

template <typename C>
struct TcShared {
    uint64_t code_full[C::kRing], code_empty[C::kRing];
    uint64_t k_full[C::kKBufs], k_empty[C::kKBufs], v_full[C::kVBufs], v_empty[C::kVBufs];
    uint64_t v_seen[C::kMeta], s_full[2], p_full[2], o_done[2];
    uint64_t o_free, q_free, q_full, all_done;
    uint64_t pair[4];                // the two softmax warps of 32 rows
    uint32_t tmem;
    int abort;
    int valid[C::kRing][C::kPages];  // whether a page of the entry is there
    int cleared[C::kMeta];           // unit + 1 if values of it were cleared
    alignas(16) float scales[C::kRing][C::kPages][2 * kPage / kBlock];
    alignas(16) float4 meta[C::kMeta][C::kBlocks];  // key scale, log2 and 1 / of the value scale
    float factor[C::kMeta][C::kRows];
    float top[2][2][C::kRows];       // of a step's halves
    float sum[C::kRows];             // of the upper half's probabilities
    uint32_t warp_sums[C::kThreads / 32];
    Share<C::kRows> share;
};

// D[tmem] (+)= A[tmem] x B[smem]; issued by a single thread.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Wait for a phase of a barrier, as mbar_wait, in few instructions: what the warps of an SM
// quarter run has to fit its instruction cache.  Up to 2^15 attempts of kSuspendNs each.
__device__ __forceinline__ bool phase_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\tmov.u32 n, 32768;\n\t"
        "again: mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra done;\n\tsub.u32 n, n, 1;\n\tsetp.ne.u32 p, n, 0;\n\t@p bra again;\n\t"
        "done: selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r));
    return r != 0;
}

// The wait for TMEM loads, tied to what was loaded.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// A role's way through the steps of its CTA's run.  g counts steps, unit the units that
// have any.
template <typename C>
struct Steps {
    Walk<C> w;
    int step, steps, g, unit;
    __device__ __forceinline__ Steps(const AttnParams& p, const Share<C::kRows>& s)
        : w(p, s), step(0), g(0), unit(0) {
        find(p);
    }
    __device__ __forceinline__ static int pages(const Walk<C>& w) {
        return max(0, min(w.u.tiles, w.tile + w.count) - w.tile);
    }
    __device__ __forceinline__ void find(const AttnParams& p) {
        for (; w.pos < w.end; w.next(p)) {
            steps = (pages(w) + C::kPages - 1) / C::kPages;
            if (steps > 0) return;
        }
    }
    __device__ __forceinline__ bool more() const { return w.pos < w.end; }
    __device__ __forceinline__ void next(const AttnParams& p) {
        ++g;
        if (++step < steps) return;
        step = 0;
        ++unit;
        w.next(p);
        find(p);
    }
    __device__ __forceinline__ int first_position() const {
        return (w.tile + step * C::kPages) * kPage;
    }
    __device__ __forceinline__ bool last() const { return step + 1 == steps; }
};

// Lifts this thread's part of an entry's codes into a tile.  Eight lanes take four chunks
// of 16 codes of rows r and r ^ 5: the swizzles then put both what they read and what they
// write into all banks.  A thread's rows are 32 apart, so that all its addresses are two
// and constants.  kChecked: rows from `rows` on, and of pages that are not there, become 0,
// and so do NaN codes of rows from `from` on; returns whether there were any.
template <typename C, bool kChecked>
__device__ __forceinline__ bool lift_tile(const uint8_t* entry, uint8_t* tile, const int* valid,
                                          int rows, int from, int thread) {
    const int c4 = thread & 3, pair = thread >> 3;  // 16 pairs of rows: 32
    const int r0 = pair / 4 * 8 + pair % 4, row0 = thread & 4 ? r0 ^ 5 : r0;
    constexpr int kRowBytes = C::kBoxBytes;  // of codes, in a box
    // chunks of a row in a box: by their slab's four the swizzle leaves together
    const int at = row0 * kRowBytes +
                   ((kRowBytes == 64 ? c4 ^ (row0 >> 1 & 3) : c4 ^ (row0 & 3)) << 4);
    const int half = kRowBytes == 64 ? 0 : row0 & 4 ? 64 : 0;  // where slab 0 of a box is
    const int to = row0 * 128 + (((2 * c4) ^ (row0 & 7)) << 4);
    bool bad = false;
#pragma unroll 1
    for (int slab = 0; slab < C::kSlabs; ++slab) {
        const uint8_t* src = entry + slab / 2 * (kPage * 128) + at + (slab % 2 ? half ^ 64 : half);
        uint8_t* dst = tile + slab * C::kSlabBytes + to;
        constexpr int kTimes = C::kStep / 32;
        uint4 u[kTimes];
#pragma unroll
        for (int i = 0; i < kTimes; ++i)
            u[i] = *reinterpret_cast<const uint4*>(src + i / 2 * C::kPageBytes +
                                                   i % 2 * (32 * kRowBytes));
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
            uint4 lo, hi;
            if (kChecked) {
                const int row = row0 + 32 * i;
                if (row >= rows || !valid[i / 2]) u[i] = make_uint4(0, 0, 0, 0);
                if (!C::kInt8 && row >= from && any_not_finite<true, false>(u[i])) {
                    u[i] = finite_part<true, false>(u[i]);
                    bad = true;
                }
            }
            lift<C::kInt8>(u[i].x, lo.x, lo.y);
            lift<C::kInt8>(u[i].y, lo.z, lo.w);
            lift<C::kInt8>(u[i].z, hi.x, hi.y);
            lift<C::kInt8>(u[i].w, hi.z, hi.w);
            // the second chunk of a pair is the neighbour of the first, swizzled alike
            *reinterpret_cast<uint4*>(dst + i * 4096) = lo;
            *reinterpret_cast<uint4*>(tile + slab * C::kSlabBytes + (to ^ 16) + i * 4096) = hi;
        }
    }
    return bad;
}

// max(a, b, c) in one instruction
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename C, bool kQBf16>
__global__ void __launch_bounds__(C::kThreads, 1)
quant_attention_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
    constexpr int kD = C::kDim;
    constexpr int kLiftWarp = 8, kCopyWarp = 16, kMmaWarp = 17;
    extern __shared__ uint8_t raw[];
    __shared__ TcShared<C> sh;
    uint8_t* const s_q = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                    ~(uintptr_t)1023);
    uint8_t* const s_k = s_q + C::kQBytes;
    uint8_t* const s_v = s_k + C::kKBufs * C::kTileBytes;
    uint8_t* const ring = s_v + C::kVBufs * C::kTileBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&sh.code_full[i], 1);
            mbar_init(&sh.code_empty[i], 4);
        }
        for (int i = 0; i < C::kKBufs; ++i) {
            mbar_init(&sh.k_full[i], 4);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < C::kVBufs; ++i) {
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int i = 0; i < C::kMeta; ++i) {
            mbar_init(&sh.v_seen[i], 4);
            sh.cleared[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 2);
            mbar_init(&sh.o_done[i], 1);
            mbar_init(&sh.p_full[i], 8);
        }
        mbar_init(&sh.o_free, 8);
        mbar_init(&sh.q_free, 1);
        mbar_init(&sh.q_full, 8);
        mbar_init(&sh.all_done, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&sh.pair[i], 2);
        fence_mbar_init();
        sh.abort = 0;
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    grid_dependents_launch();
    grid_dependency_wait();
    find_share<C>(p, &sh.share, sh.warp_sums);
    if (sh.share.begin >= sh.share.end) {
        if (tid == 0) p.joins[blockIdx.x * kJoinInts + kJoinPieces] = 0;
        return;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    bool ok = true;

    if (warp >= kCopyWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kControlRegs));
        if (warp == kCopyWarp || warp == kCopyWarp + 2) {
            // ---- copies: one warp brings the codes of a step's keys, with all its scales, one
            // those of its values (an entry takes a warp about 1400 cycles to issue)
            const int kind = warp != kCopyWarp;
            Walk<C> walk(p, sh.share);
            int n = kind;  // the warp's next entry
            int pieces = 0;
            auto entries = [&](const Cursor<C::kRows>& x, int t) {
                return t + lane < x.tiles
                           ? __ldg(p.bt.block_table + (int64_t)x.b * p.bt.max_pages + t + lane)
                           : -1;
            };
            int ahead = walk.pos < walk.end ? entries(walk.u, walk.tile) : -1;
            while (walk.pos < walk.end) {
                const Cursor<C::kRows>& u = walk.u;
                const int tile = walk.tile, count = Steps<C>::pages(walk);
                Walk<C> v = walk;
                v.next(p);
                const int ahead_v = v.pos < v.end ? entries(v.u, v.tile) : -1;
                for (int i = 0; i < count; i += C::kPages) {
                    if (i > 0 && i % 32 == 0) ahead = entries(u, tile + i);
                    int page[C::kPages];
                    bool here[C::kPages];
                    int there = 0;
#pragma unroll
                    for (int x = 0; x < C::kPages; ++x) {
                        page[x] = __shfl_sync(0xffffffffu, ahead, (i + x) % 32);
                        here[x] = i + x < count && page[x] >= 0 && page[x] < p.bt.num_pages;
                        there += here[x];
                        if (i + x < count && !here[x] && lane == 0 && kind == 0)
                            record_error(p.status, DSA_ERR_DEVICE_CHECK);
                    }
                    const int st = n % C::kRing;
                    if (lane == 0 && ok &&
                        (ok = phase_wait(&sh.code_empty[st], (n / C::kRing & 1) ^ 1))) {
#pragma unroll
                        for (int x = 0; x < C::kPages; ++x) sh.valid[st][x] = here[x];
                        const bool withheld = p.withhold && n == 0;  // by the test only
                        const int each = C::kPageBytes + (kind == 0 ? 2 * kPage / kBlock * 4 : 0);
                        if (!withheld) mbar_arrive_expect_tx(&sh.code_full[st], there * each);
#pragma unroll
                        for (int x = 0; x < C::kPages; ++x) {
                            if (!here[x] || withheld) continue;
                            const int z = page[x] * p.kv_heads + u.h;
                            uint8_t* dst = ring + st * C::kEntryBytes + x * C::kPageBytes;
#pragma unroll
                            for (int b = 0; b < C::kBoxes; ++b)
                                tma_load_3d(dst + b * (kPage * C::kBoxBytes),
                                            kind == 0 ? &tm_k : &tm_v, b * C::kBoxBytes, 0, z,
                                            &sh.code_full[st]);
                            if (kind == 0)
                                bulk_copy_g2s(sh.scales[st][x],
                                              p.scales + (int64_t)z * (2 * kPage / kBlock),
                                              2 * kPage / kBlock * 4, &sh.code_full[st]);
                        }
                    }
                    n += 2;
                    __syncwarp();
                }
                if (lane == 0 && kind == 0 && tile == 0 && !walk.complete(p)) {
                    // first piece of a row tile that other CTAs finish
                    int32_t* j = p.joins + blockIdx.x * kJoinInts;
                    pieces =
                        1 + (int)((u.cost() - walk.count + sh.share.per - 1) / sh.share.per);
                    pieces = min(pieces, (int)(gridDim.x - blockIdx.x));
                    j[kJoinToken] = u.r.q0;
                    j[kJoinRow] = u.rt * C::kRows;
                    j[kJoinRows] = min(C::kRows, u.r.rows - u.rt * C::kRows);
                    j[kJoinHead] = u.h * p.group;
                }
                walk = v;
                ahead = ahead_v;
            }
            if (lane == 0 && kind == 0) p.joins[blockIdx.x * kJoinInts + kJoinPieces] = pieces;
        } else if (warp == kMmaWarp) {
            // ---- MMAs: the warp goes along as one, so that what it computes stays in uniform
            // registers, and one lane issues
            const uint64_t qd = smem_desc(smem_u32(s_q), 16, 1024, kSwizzle128B);
            const uint64_t kd = smem_desc(smem_u32(s_k), 16, 1024, kSwizzle128B);
            const uint64_t vd = smem_desc(smem_u32(s_v), C::kSlabBytes, 1024, kSwizzle128B);
            const bool leader = elect_one();
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xffffffffu, phase_wait(bar, parity)) != 0;
            };
            auto issue_s = [&](const Steps<C>& x) {
                const int b = x.g % C::kKBufs;
                // the buffer's P has been read: MMAs of other accumulators and shapes are
                // not kept in order
                if (x.g >= 2 && !wait(&sh.o_done[x.g & 1], (x.g - 2) >> 1 & 1)) return false;
                if (x.step == 0 && !wait(&sh.q_full, x.unit & 1)) return false;
                if (!wait(&sh.k_full[b], x.g / C::kKBufs & 1)) return false;
                tc_fence_after();
                const uint32_t d = tmem + (x.g & 1) * C::kStep;
                const uint64_t kb = kd + (uint64_t)(b * C::kTileBytes >> 4);
                const bool last = x.last();
                if (leader) {
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16(d, qd + (uint64_t)((s * C::kQSlabBytes + k * 32) >> 4),
                                    kb + (uint64_t)((s * C::kSlabBytes + k * 32) >> 4),
                                    C::kIdescS, s + k > 0);
                    mma_commit(&sh.s_full[x.g & 1]);
                    mma_commit(&sh.k_empty[b]);
                    // and what this warp has seen: the scales and factors
                    mbar_arrive(&sh.s_full[x.g & 1]);
                    if (last) mma_commit(&sh.q_free);
                }
                __syncwarp();
                return true;
            };
            Steps<C> now(p, sh.share), ahead = now;
            if (ahead.more()) {
                ok = issue_s(ahead);
                ahead.next(p);
            }
            for (; ok && now.more(); now.next(p)) {
                if (ahead.more()) {
                    if (!(ok = issue_s(ahead))) break;
                    ahead.next(p);
                }
                const int b = now.g % C::kVBufs;
                if (now.step == 0 && now.unit > 0) ok = wait(&sh.o_free, (now.unit - 1) & 1);
                ok = ok && wait(&sh.v_full[b], now.g / C::kVBufs & 1) &&
                     wait(&sh.p_full[now.g & 1], now.g >> 1 & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t pt = tmem + (now.g & 1) * C::kStep;
                const uint64_t vb = vd + (uint64_t)(b * C::kTileBytes >> 4);
                const uint32_t more = now.step > 0;
                if (leader) {
#pragma unroll
                    for (int k = 0; k < C::kStep / 16; ++k)
                        mma_f16_ta(tmem + C::kColO,
                                   pt + k * 16 / C::kHalf * C::kHalf + k * 16 % C::kHalf / 2,
                                   vb + (uint64_t)(k * 2048 >> 4), C::kIdescO, k > 0 ? 1 : more);
                    mma_commit(&sh.v_empty[b]);
                    mma_commit(&sh.o_done[now.g & 1]);
                }
                __syncwarp();
            }
            // TMEM and shared memory stay until the last MMA is done
            if (leader) mma_commit(&sh.all_done);
            __syncwarp();
            mbar_drain(&sh.all_done, 0);
        }
    } else if (warp >= kLiftWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLiftRegs));
        const bool values = warp >= kLiftWarp + 4;
        const int thread = tid % C::kLiftThreads;
        Steps<C> x(p, sh.share);
        for (; ok && x.more(); x.next(p)) {
            const Cursor<C::kRows>& u = x.w.u;
            const int tile_row = u.rt * C::kRows;
            if (x.step == 0) {
                // Queries, a warp of either group to a row; their scaling as in
                // paged_attention.cuh.
                if (x.unit > 0) {
                    ok = phase_wait(&sh.q_free, (x.unit - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                constexpr int kWords = kD / 64;
#pragma unroll 8
                for (int r = warp - kLiftWarp; r < C::kRows; r += 8) {
                    const int row = tile_row + r, j = token_of(p, row);
                    uint32_t w[kWords];
#pragma unroll
                    for (int i = 0; i < kWords; ++i) w[i] = 0;
                    if (row < u.r.rows) {
                        const uint32_t* q = reinterpret_cast<const uint32_t*>(
                                                static_cast<const uint16_t*>(p.q) +
                                                (int64_t)(u.r.q0 + j) * p.q_stride +
                                                (int64_t)(u.h * p.group + row - j * p.group) * kD) +
                                            lane * kWords;
                        if (kWords == 1) {
                            w[0] = *q;
                        } else if (kWords == 2) {
                            const uint2 y = *reinterpret_cast<const uint2*>(q);
                            w[0] = y.x;
                            w[kWords > 1 ? 1 : 0] = y.y;
                        } else {
                            const uint4 y = *reinterpret_cast<const uint4*>(q);
                            w[0] = y.x;
                            w[kWords > 1 ? 1 : 0] = y.y;
                            w[kWords > 2 ? 2 : 0] = y.z;
                            w[kWords > 2 ? 3 : 0] = y.w;
                        }
                    }
                    float factor = p.score_scale;
                    if (kQBf16) {
                        uint32_t top = 0;
#pragma unroll
                        for (int i = 0; i < kWords; ++i)
                            top = max(top, max(w[i] & 0x7fffu, w[i] >> 16 & 0x7fffu));
                        const uint32_t e = __reduce_max_sync(0xffffffffu, top) >> 7;
                        float up = 1.f;
                        if (e >= 64 && e < 255) {
                            const uint32_t by = min(e, 253u);
                            up = __uint_as_float((254 - by) << 23);
                            factor = factor * __uint_as_float(by << 23);
                        }
#pragma unroll
                        for (int i = 0; i < kWords; ++i)
                            w[i] = pack2<false>(__uint_as_float(w[i] << 16) * up,
                                                __uint_as_float(w[i] & 0xffff0000u) * up);
                    }
                    if (lane == 0)
                        sh.factor[x.unit % C::kMeta][r] = fminf(fmaxf(factor, 0x1p-78f), 0x1p94f);
                    const int byte = lane * kWords * 4;  // of the f16 row
                    uint8_t* dst = s_q + byte / 128 * C::kQSlabBytes + sw128(r, byte % 128);
                    if (kWords == 1)
                        *reinterpret_cast<uint32_t*>(dst) = w[0];
                    else if (kWords == 2)
                        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[kWords > 1 ? 1 : 0]);
                    else
                        *reinterpret_cast<uint4*>(dst) =
                            make_uint4(w[0], w[kWords > 1 ? 1 : 0], w[kWords > 2 ? 2 : 0],
                                       w[kWords > 2 ? 3 : 0]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full);
            }
            const int n = 2 * x.g + values, st = n % C::kRing;
            const int bufs = values ? C::kVBufs : C::kKBufs, b = x.g % bufs;
            uint64_t* const full = values ? &sh.v_full[b] : &sh.k_full[b];
            uint64_t* const empty = values ? &sh.v_empty[b] : &sh.k_empty[b];
            uint8_t* const tile = (values ? s_v : s_k) + b * C::kTileBytes;
            ok = phase_wait(empty, (x.g / bufs & 1) ^ 1) &&
                 phase_wait(&sh.code_full[st], n / C::kRing & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t* entry = ring + st * C::kEntryBytes;
            const int first = x.first_position();
            bool there = true;  // all pages
#pragma unroll
            for (int i = 0; i < C::kPages; ++i) there = there && sh.valid[st][i];
            // Values past the context may hold anything, and p there is 0; E4M3 has NaN, which
            // not all rows may see: cleared here, given back in the epilogue.  (Keys there are
            // masked.)
            const int rows = values ? u.r.seq - first : C::kStep;
            const int vis_first = u.r.seq - u.r.nb + token_of(p, tile_row) + 1;
            const int from = values && !C::kInt8 ? max(0, vis_first - first) : C::kStep;
            if (there && rows >= C::kStep && from >= C::kStep)
                lift_tile<C, false>(entry, tile, nullptr, 0, 0, thread);
            else if (lift_tile<C, true>(entry, tile, sh.valid[st], rows, from, thread))
                *static_cast<volatile int*>(&sh.cleared[x.unit % C::kMeta]) = x.unit + 1;
            if (!values && thread < C::kBlocks) {
                const int page = thread / (kPage / kBlock), i = thread % (kPage / kBlock);
                // positions of a page that is not there are left out: 2^-infinity
                float4 m = make_float4(1.f, -INFINITY, 1.f, 0.f);
                if (sh.valid[st][page]) {
                    const float* s = sh.scales[st][page];
                    const float v =
                        fminf(fmaxf(s[kPage / kBlock + i], kMinBlockScale), kMaxBlockScale);
                    m = make_float4(fminf(fmaxf(s[i], kMinBlockScale), kMaxBlockScale), lg2(v),
                                    rcp(v), 0.f);
                }
                sh.meta[x.g % C::kMeta][thread] = m;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(&sh.code_empty[st]);
                if (values) mbar_arrive(&sh.v_seen[x.g % C::kMeta]);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        // Two threads to a row: warps w and w + 4 take a half of a step's positions each,
        // with one reference maximum and sums of their own, and a half of the dims.
        constexpr int kBlocks = C::kHalf / kBlock;  // of a half
        const int half = warp >> 2, r = tid & 127;
        const uint32_t lanes = tmem_addr(tmem, (warp & 3) * 32, 0);
        int g = 0, unit = 0, meetings = 0;
        // The warps of a pair meet, with what they have read of TMEM and written to shared
        // memory (by a barrier whose waits end, unlike bar.sync's).
        auto meet = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pair[warp & 3]);
            ok = phase_wait(&sh.pair[warp & 3], meetings++ & 1);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        for (Walk<C> walk(p, sh.share); ok && walk.pos < walk.end; walk.next(p)) {
            const Cursor<C::kRows>& u = walk.u;
            const int pages = Steps<C>::pages(walk), steps = (pages + C::kPages - 1) / C::kPages;
            const int tile_row = u.rt * C::kRows, rows = min(C::kRows, u.r.rows - tile_row);
            const int row = tile_row + r, j = token_of(p, row);
            const int vis = r < rows ? u.r.seq - u.r.nb + j + 1 : 0;
            const int vis_first = u.r.seq - u.r.nb + token_of(p, tile_row) + 1;
            const bool idle = (warp & 3) * 32 >= rows;  // a warp without a row
            float m = -INFINITY, l = 0.f, f = 0.f;
            for (int step = 0; step < steps; ++step, ++g) {
                ok = phase_wait(&sh.s_full[g & 1], g >> 1 & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (!idle) {
                    if (step == 0) f = sh.factor[unit % C::kMeta][r];
                    // Two passes, 32 positions at a time: the loops have to stay small (the
                    // warps of an SM quarter run four programs, and what they run of them
                    // has to fit its instruction cache), so S is loaded twice.
                    const uint32_t s_at = lanes + (g & 1) * C::kStep + half * C::kHalf;
                    const int first = (walk.tile + step * C::kPages) * kPage + half * C::kHalf;
                    const float4* meta = sh.meta[g % C::kMeta] + half * kBlocks;
                    float most = -INFINITY;
#pragma unroll 1
                    for (int i = 0; i < C::kHalf / 32; ++i) {
                        uint32_t s[32];
                        tmem_ld32(s_at + 32 * i, s);
                        tmem_wait_ld(s);
                        if (first + 32 * i + 32 > vis_first) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (first + 32 * i + e >= vis) s[e] = 0xff800000u;
                            tmem_st32(s_at + 32 * i, s);
                            tmem_wait_st();
                        }
                        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < kBlock; e += 2)
#pragma unroll
                            for (int b = 0; b < 2; ++b)
                                top[b] = max3(top[b], __uint_as_float(s[b * kBlock + e]),
                                              __uint_as_float(s[b * kBlock + e + 1]));
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            most = fmaxf(most, __fmaf_ru(top[b], f * meta[2 * i + b].x,
                                                         meta[2 * i + b].y));
                    }
                    sh.top[g & 1][half][r] = most;
                    meet();
                    if (!ok) break;
                    const float top = fmaxf(most, sh.top[g & 1][half ^ 1][r]);
                    // the reference moves rarely, and O with it
                    const bool grew = top > m + kTcLag;
                    if (__any_sync(0xffffffffu, grew)) {
                        const float a = grew ? ex2(m - base_of(top)) : 1.f;
                        l *= a;
                        if (grew) m = top;
                        if (step > 0) {
                            ok = phase_wait(&sh.o_done[(g - 1) & 1], (g - 1) >> 1 & 1);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int d = half * (kD / 2); d < (half + 1) * (kD / 2); d += 32) {
                                uint32_t o[32];
                                tmem_ld32(lanes + C::kColO + d, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                                tmem_st32(lanes + C::kColO + d, o);
                            }
                        }
                    }
                    const float base = __fsub_ru(base_of(m), kTcPExp);
#pragma unroll 1
                    for (int i = 0; i < C::kHalf / 32; ++i) {
                        uint32_t s[32], pk[16];
                        tmem_ld32(s_at + 32 * i, s);
                        float fk[2], c[2], sum[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            fk[b] = f * meta[2 * i + b].x;
                            c[b] = -__fsub_ru(base, meta[2 * i + b].y);
                            sum[b] = 0.f;
                        }
                        tmem_wait_ld(s);
#pragma unroll
                        for (int e = 0; e < kBlock; e += 2)
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const uint32_t* z = s + b * kBlock + e;
                                const float x = ex2(fmaf(__uint_as_float(z[0]), fk[b], c[b]));
                                const float y = ex2(fmaf(__uint_as_float(z[1]), fk[b], c[b]));
                                sum[b] += x + y;
                                pk[(b * kBlock + e) / 2] = pack2<false>(x, y);
                            }
#pragma unroll
                        for (int b = 0; b < 2; ++b) l = fmaf(sum[b], meta[2 * i + b].z, l);
                        tmem_st16(s_at + 16 * i, pk);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[g & 1]);
            }
            if (!ok) break;
            // ---- the unit's rows
            const bool complete = walk.complete(p);
            uint32_t nan[kD / 64];  // of this half's dims: where its row sees a cleared NaN
#pragma unroll
            for (int i = 0; i < kD / 64; ++i) nan[i] = 0;
            if (steps > 0) {
                ok = phase_wait(&sh.o_done[(g - 1) & 1], (g - 1) >> 1 & 1) &&
                     phase_wait(&sh.v_seen[(g - 1) % C::kMeta], (g - 1) / C::kMeta & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (!C::kInt8 &&
                    *static_cast<volatile int*>(&sh.cleared[unit % C::kMeta]) == unit + 1) {
                    const int to = min(min(u.r.seq, (walk.tile + pages) * kPage), vis);
#pragma unroll 1
                    for (int x = max(vis_first, walk.tile * kPage); x < to; ++x) {
                        const int page = __ldg(p.bt.block_table +
                                               (int64_t)u.b * p.bt.max_pages + x / kPage);
                        if (page < 0 || page >= p.bt.num_pages) continue;
                        const uint8_t* v = static_cast<const uint8_t*>(p.v_pages) +
                                           (((int64_t)page * p.kv_heads + u.h) * kPage +
                                            x % kPage) * kD + half * (kD / 2);
#pragma unroll
                        for (int i = 0; i < kD / 8; ++i) {
                            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(v) + i);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if ((w >> (8 * y) & 0x7f) == 0x7f)
                                    nan[i / 8] |= 1u << (i % 8 * 4 + y);
                        }
                    }
                }
            }
            if (!idle) {
                // both halves' sums, in this order in both
                if (half) sh.sum[r] = l;
                else sh.top[0][0][r] = l;
                meet();
                l = sh.top[0][0][r] + sh.sum[r];
                if (ok) meet();  // before either is written again
                if (!ok) break;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            int64_t at;
            if (complete) {
                at = (int64_t)(u.r.q0 + j) * (p.kv_heads * p.group) + u.h * p.group + row -
                     j * p.group;
                if (p.lse && half == 0 && r < rows)
                    p.lse[at] = l == 0.f ? -INFINITY : (m + (log2f(l) - kTcPExp)) * kLn2;
            } else {
                at = (2 * (int64_t)blockIdx.x + (walk.tile == 0 ? 1 : 0)) * C::kRows + r;
                if (half == 0 && r < rows)
                    *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m, l * kTcPUnit);
            }
            if (!idle) {
#pragma unroll 1
                for (int x = 0; x < kD / 64; ++x) {
                    const int d = half * (kD / 2) + 32 * x;
                    uint32_t o[32];
                    if (steps > 0) {
                        tmem_ld32(lanes + C::kColO + d, o);
                        tmem_wait_ld(o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0;
                    }
                    uint32_t bad = 0;
#pragma unroll
                    for (int i = 0; i < kD / 64; ++i) bad |= x == i ? nan[i] : 0;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float y = __uint_as_float(o[i]);
                        v[i] = complete ? result(y, inv) : y * kTcPUnit;
                        if (bad >> i & 1) v[i] = __uint_as_float(0x7fffffffu);
                    }
                    if (r < rows) {
                        if (complete) {
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                                                  at * kD + d);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                dst[i] = make_uint4(pack2<kQBf16>(v[8 * i], v[8 * i + 1]),
                                                    pack2<kQBf16>(v[8 * i + 2], v[8 * i + 3]),
                                                    pack2<kQBf16>(v[8 * i + 4], v[8 * i + 5]),
                                                    pack2<kQBf16>(v[8 * i + 6], v[8 * i + 7]));
                        } else {
                            float4* dst = reinterpret_cast<float4*>(p.part_o + at * kD + d);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2],
                                                     v[4 * i + 3]);
                        }
                    }
                }
            }
            if (steps > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.o_free);
                ++unit;
            }
        }
    }
    if (!ok && (warp < kCopyWarp || lane == 0)) {
        sh.abort = 1;
        record_error(p.status, DSA_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.abort) {
        // the CTA must not exit under copies in flight.  Where all went well their readers
        // have waited for them; here each slot's last one (or none, which costs the budget)
        if (tid < C::kRing) {
            mbar_drain<kWaitCycles / 64>(&sh.code_full[tid], 0);
            mbar_drain<kWaitCycles / 64>(&sh.code_full[tid], 1);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        __syncwarp();
        tmem_dealloc(tmem, C::kCols);
    }
}

// Whether a call takes this kernel.  mma.sync takes a request's rows in tiles of up to 64,
// each of which lifts for itself; it is the faster up to 32 rows (48 of 64 dims: 886 us and
// here 1022 for five tokens of eight heads over 16 x 131072 positions of INT8; 128 dims
// 1493 and 1192, with four tokens 1109 and 1147).  A launch here costs some 25 us more
// (first steps alone, 128 rows to join), which it makes up for at 2.4 times the rate: the
// sides meet between 8 and 10 * 10^9 operations by the host's sizes (16 requests of 2000
// positions, 64 rows, 8.4 * 10^9: 48 and 47 us; of 1000: 29 and 37; 500 new tokens over 1000,
// 8.2 * 10^9: 41 and 44, 1000: 62 and 60).
// The largest request decides for all, and total_q tokens are counted over max_seq positions
// each.  Both err towards this kernel where requests differ: of 64 requests of one token over up
// to 32768 positions, 64 / 8 heads of 128 and E4M3, 278 us by themselves, one with five tokens
// makes it 507 (two calls 295), and a chunk of 1000 over 16384 beside them 1208 (two calls 940).
inline bool takes_tensor_cores(const BatchArgs& bt, int num_q_heads, int kv_heads, int head_dim,
                               bool whole) {
    const int64_t rows = (int64_t)bt.max_q * (num_q_heads / kv_heads);
    const double work = 4.0 * bt.total_q * num_q_heads * head_dim * (double)bt.max_seq;
    // positions in the list are 32-bit
    const double list = most_units(bt, kv_heads, num_q_heads / kv_heads, 128) *
                        ((double)bt.max_seq / kPage + 2 + kTcUnitCost);
    return !whole && rows > (head_dim == 64 ? 48 : 32) && work >= 9e9 && list < 2147483648.0;
}

template <typename C, bool kQBf16>
cudaError_t launch_tc(AttnParams p, const dsa_kv_cache& cache, int* launches,
                      cudaStream_t stream) {
    CUtensorMap tm_k, tm_v;
    if (!encode_pool(&tm_k, cache.k_pages, cache, C::kDim) ||
        !encode_pool(&tm_v, cache.v_pages, cache, C::kDim))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    // the consumers of registers would wait forever for more than the launch brings
    static const cudaError_t ready = [] {
        cudaFuncAttributes a;
        cudaError_t e = cudaFuncGetAttributes(&a, quant_attention_tc_kernel<C, kQBf16>);
        if (e == cudaSuccess && a.numRegs < C::kLaunchRegs) e = cudaErrorInvalidConfiguration;
        return e;
    }();
    if (ready != cudaSuccess) return ready;
    if ((e = cudaFuncSetAttribute(quant_attention_tc_kernel<C, kQBf16>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) !=
        cudaSuccess)
        return e;
    p.min_length = C::kUnitCost + 2 * C::kPages;
    const int64_t tiles = ((int64_t)p.bt.max_seq + kPage - 1) / kPage;
    const double length =
        most_units(p.bt, p.kv_heads, p.group, C::kRows) * (double)(tiles + C::kUnitCost);
    int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    if (length < (double)ctas * p.min_length) ctas = (int)(length / p.min_length) + 1;
    e = launch_kernel(quant_attention_tc_kernel<C, kQBf16>, dim3((unsigned)ctas),
                      dim3(C::kThreads), (size_t)C::kSmem, stream, true, 1, tm_k, tm_v, p);
    if (e != cudaSuccess || ctas == 1) return e;
    *launches = 2;
    const dim3 grid((unsigned)ctas, (unsigned)kJoinRowBlocks);
    return launch_kernel(paged_join_kernel<C::kDim, kQBf16>, grid, dim3(kJoinThreads), 0, stream,
                         true, 1, p, (int)C::kRows);
}

template <int kD, int kCode>
cudaError_t launch_tensor(const AttnParams& p, const dsa_kv_cache& cache, int format,
                          int* launches, cudaStream_t stream) {
    using C = TcCfg<kD, kCode>;
    return format == DSA_FLOAT_BF16 ? launch_tc<C, true>(p, cache, launches, stream)
                                    : launch_tc<C, false>(p, cache, launches, stream);
}

}  // namespace paged
}  // namespace dsa
