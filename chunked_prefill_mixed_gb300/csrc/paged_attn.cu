// paged_attn.cu -- attention of a planned ragged batch over its pages, with
// capped scores, a bias by distance and an interval of visible keys per token:
//   s_j = q . K_j scale;  s_j = cap tanh(s_j / cap);  s_j -= slope |p - j|;
//   out = sum_{lo <= j < hi} softmax_j(s_j) V_j.
//
// One persistent launch, one CTA an SM, takes work items from the plan's two
// queues:
//
//   TILE    up to two tiles of 128 query rows (token x q head of one kv head's
//           group) over a range of keys in blocks (80 keys at d = 128, 128 at
//           d = 64): a chunk's tokens over their row's pages, or all the
//           tokens of a group of requests over the pages that they share.  S
//           = Q K^T and O += P V run on the tensor cores (tcgen05,
//           accumulators and P in tensor memory), K and V come by TMA straight
//           from the pages, and each tile's softmax is done by a warpgroup of
//           its own, one thread a row, so that one tile's exponentials run
//           while the other tile's products do.
//   STREAM  a range of a one-token row's pages for one kv head, by one warp:
//           TMA page loads that run on into the warp's next item, warp-level MMA
//           for the 16 padded rows of a group.  The bytes are the bound there,
//           and 16 x 16 x d products per page are far below a tcgen05 tile.
//
// An item that is one of several for its tokens writes partial rows (sum, its
// base and weight); a second small kernel joins them in a fixed order, so the
// bits do not depend on which item ended first.  No item waits for another.
//
// What bounds them, on a GB300 that copies at 6.8 TB/s and multiplies bf16 at 1.9
// PFLOP/s: streams, HBM (80 decodes of 32 / 8 heads, 732 MB, 116 us, 6.3 TB/s);
// tiles of long chunks, softmax and products that overlap in part only (pages in
// order: 4096-token prompt, 32 / 8 heads, d 128, 106 us, 1.30 PFLOP/s; 2048 tokens
// behind 6144 keys with a bias, 200 us, 1.20 PFLOP/s, the tensor pipe active in 60% of
// the cycles, and 250 us with scattered pages, a copy each); short key ranges, 1.5 us
// an item beside 1 to 1.7 us a block (4001 tokens of 9 documents, 29 us).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "device_util.cuh"
#include "paged_internal.h"
#include "sarathi.h"

namespace sarathi {
namespace paged {

using namespace dev;

struct Params {
    const uint16_t* q;
    const uint16_t* k_cache;
    const uint16_t* v_cache;
    uint16_t* out;
    float* lse;
    const float* slopes;
    int64_t q_stride;
    const int32_t* plan;
    int off_pages, off_tokens, off_items, off_merge;
    int n_items, n_first, first_sms, n_merge;
    int Hq, Hkv, group, num_pages;
    float raw_scale;  // of q . K: sm_scale log2(e), or sm_scale / cap under a cap
    float cap2;       // cap log2(e); 0: no cap
    int cap_fine;     // the cap is above kCapFine
    int next_early;   // the stream's next kernel may begin while this one runs
    int32_t* ws;
    float2* part_ml;  // {max, sum} of each partial row
    float* part_o;    // its weighted sum of values, [n_partials][d]
};

constexpr int kThreads = 384;      // 12 warps: 0-7 softmax / streams, 8-11 copies and MMA issue
constexpr int kMainThreads = 256;
// Registers: a softmax thread holds its row's 80 or 128 scores of a block.  Both
// shares together are what the block is launched with (384 x 168): 256 x 216 + 128 x 72.
constexpr int kMainRegs = 216, kAuxRegs = 72, kLaunchRegs = 168;
static_assert(kMainThreads * kMainRegs + (kThreads - kMainThreads) * kAuxRegs <= kThreads * kLaunchRegs,
              "register split");
constexpr unsigned long long kWaitNs = 2000000000ull;  // bound on any wait

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kKeys = block_keys(D);                // keys of a K/V block
    static constexpr int kPages = kKeys / kPage;
    static constexpr int kQBytes = kTileRows * D * 2;          // a Q tile
    static constexpr int kBlkBytes = kKeys * D * 2;            // a K or V block
    static constexpr int kBlkHalf = kKeys * 128;               // one 64-column half of a block
    static constexpr int kStages = D == 128 ? 6 : 8;           // K/V ring
    static constexpr int kQ = kStages * kBlkBytes;             // two Q tiles behind the ring
    static constexpr int kStage = kQ + 2 * kQBytes;            // 32 rows x 128 B a softmax warp, for its stores
    static constexpr int kPageBytes = kPage * D * 2;           // one page of a kv head
    // tensor memory columns of tile x: scores S, weights P (two a column), sums O
    __host__ __device__ static constexpr uint32_t s_col(int x) { return D == 128 ? 128u * x : 256u * x; }
    __host__ __device__ static constexpr uint32_t p_col(int x) { return s_col(x) + kKeys; }
    __host__ __device__ static constexpr uint32_t o_col(int x) { return D == 128 ? 256u + 128u * x : 256u * x + 192u; }
    static constexpr int kStreamStages = 3;                    // pages (K and V) a streaming warp keeps in flight
    static constexpr int kStreamQ = kStreamWarps * kStreamStages * 2 * kPageBytes;  // then a query tile a warp
    static constexpr int kTileEnd = kStage + 8 * 4096, kStreamEnd = kStreamQ + kStreamWarps * kPageBytes;
    static constexpr int kBytes = kTileEnd > kStreamEnd ? kTileEnd : kStreamEnd;
    static constexpr int kAlloc = kBytes + 1024;               // + alignment slack
    static_assert(kAlloc + 1024 <= 227 * 1024, "shared memory per CTA");
    static_assert(kBlkBytes % 1024 == 0 && kBlkHalf % 1024 == 0 && kPages <= 8, "swizzle atoms, page lanes");
};
constexpr int kMaxStages = 8;
constexpr int kItemSlots = 2;  // tile items that a CTA's roles are in at once
enum Bar {
    kKvFull = 0,
    kKvEmpty = kKvFull + kMaxStages,
    kSFull = kKvEmpty + kMaxStages,  // per tile: a block's scores are in tensor memory
    kSFree = kSFull + 2,             // per tile: they have been loaded (4 warps)
    kPFull = kSFree + 2,             // per tile: its weights are in tensor memory (4 warps)
    kPvDone = kPFull + 2,            // per tile: its P V is done
    kQFull = kPvDone + 2,
    kQFree = kQFull + 1,             // the item's last S = Q K^T is done
    kVLast = kQFree + 1,             // block 0's V is there, to be cleaned ...
    kVFix = kVLast + 1,              // ... and is clean: rows past the keys are zero (32 arrivals)
    kItemFull = kVFix + 1,           // per slot: an item has been claimed
    kItemFree = kItemFull + kItemSlots,  // per slot: every role is done with it
    kStreamBar = kItemFree + kItemSlots,  // [warp][stage]
    kNumBars = kStreamBar + kStreamWarps * 3
};
constexpr uint32_t kItemReaders = 8 + 2 + 1;  // softmax warps, product warps, the cleaning warp
constexpr uint32_t kTmemCols = 512;

struct Shared {
    __align__(16) int item[kItemSlots][8];
    uint64_t bars[kNumBars];
    int abort;
    uint32_t tmem;
};

__device__ __forceinline__ void raise(const Params& P, int code, int detail) {
    if (atomicCAS(&P.ws[kError], 0, code) == 0) P.ws[kDetail] = detail;
}
// Bounded wait for a barrier's phase; false once the block gives up.
__device__ __forceinline__ bool wait_slow(const Params& P, uint32_t bar, uint32_t parity, Shared* sh, int code) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (*(volatile int*)&sh->abort) return false;
        if (globaltimer() - t0 > kWaitNs) {
            raise(P, kErrWait, code);
            *(volatile int*)&sh->abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(const Params& P, uint32_t bar, uint32_t parity, Shared* sh, int code) {
    return mbar_try_wait(bar, parity) || wait_slow(P, bar, parity, sh, code);
}
// The same for a whole warp whose next step is collective: all lanes agree.
__device__ __forceinline__ bool wait_warp(const Params& P, uint32_t bar, uint32_t parity, Shared* sh, int code) {
    return __all_sync(0xffffffffu, wait(P, bar, parity, sh, code));
}
__device__ __forceinline__ int page_id(const Params& P, int entry) {
    const int page = P.plan[P.off_pages + entry];
    if ((uint32_t)page < (uint32_t)P.num_pages) return page;
    raise(P, kErrBounds, page);
    return 0;
}

// cap2 tanh(x) by exponential and reciprocal, within a few 2^-23 of cap2; caps
// above kCapFine, for which that is more than an fp16 output's rounding shows,
// take tanh's series below 0.3 (within 2^-24 there), so that the error goes by the
// score and not by the cap.
constexpr float kCapFine = 128.f;
__device__ __forceinline__ float tanh_fine(float x) {
    const float u = x * x;
    float p = fmaf(u, 62.f / 2835.f, -17.f / 315.f);
    p = fmaf(u, p, 2.f / 15.f);
    p = fmaf(u, p, -1.f / 3.f);
    p = fmaf(u * p, x, x);
    return fabsf(x) < 0.3f ? p : tanh_abs(x);
}

// Weights are taken 2^kUp larger than they are relative to their base (fp16: up
// to 2^15 once the maximum has passed the base by 2^8), so that small ones round
// to fp16 as they do to bf16: relatively, down to 2^-21 of the base, and to steps
// of 2^-31 below.  At 2^0 a tail of many keys each 2^-23 of the largest is off by
// a third.
template <bool F16>
__device__ constexpr float weight_up() { return F16 ? 7.f : 0.f; }

// A visible score in base-2 logits.
__device__ __forceinline__ float score(const Params& P, float raw, float slope2, int pos, int key) {
    float t = raw * P.raw_scale;
    if (P.cap2 > 0.f) t = P.cap2 * (P.cap_fine ? tanh_fine(t) : tanh_abs(t));
    return fmaf(-slope2, fabsf((float)(pos - key)), t);
}

// One query row by one warp, eight keys a step: running maximum m and sum l
// (base-2 logits) and the weighted sum acc (lane holds dims D/32 lane ...) over
// the keys [lo, hi).
template <int D, bool F16>
__device__ __forceinline__ void attend_row(const Params& P, const uint16_t* q, int kvp0, int pos, int g, float slope2,
                                           int lo, int hi, float& m, float& l, float (&acc)[D / 32]) {
    constexpr int N = D / 32, W = N / 2, B = 8;
    const int lane = threadIdx.x & 31;
    float2 qf[W];
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        qf[i] = unpack2<F16>(*reinterpret_cast<const uint32_t*>(q + lane * N + 2 * i));
        acc[2 * i] = acc[2 * i + 1] = 0.f;
    }
    for (int j = lo / B * B; j < hi; j += B) {
        const size_t row = (((size_t)page_id(P, kvp0 + j / kPage) * P.Hkv + g) * kPage + j % kPage) * D + lane * N;
        uint32_t kw[B][W], vw[B][W];
#pragma unroll
        for (int e = 0; e < B; ++e) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                kw[e][i] = *reinterpret_cast<const uint32_t*>(P.k_cache + row + e * D + 2 * i);
                vw[e][i] = *reinterpret_cast<const uint32_t*>(P.v_cache + row + e * D + 2 * i);
            }
        }
        float s[B], mn = m;
#pragma unroll
        for (int e = 0; e < B; ++e) {
            s[e] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 k2 = unpack2<F16>(kw[e][i]);
                s[e] = fmaf(qf[i].x, k2.x, fmaf(qf[i].y, k2.y, s[e]));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
#pragma unroll
            for (int e = 0; e < B; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
        }
#pragma unroll
        for (int e = 0; e < B; ++e) {
            s[e] = j + e >= lo && j + e < hi ? score(P, s[e], slope2, pos, j + e) : -INFINITY;
            mn = fmaxf(mn, s[e]);
        }
        const float base = mn == -INFINITY ? 0.f : mn, al = ex2(m - base);
        m = mn;
        l *= al;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] *= al;
#pragma unroll
        for (int e = 0; e < B; ++e) {
            if (j + e < lo || j + e >= hi) continue;
            const float w = ex2(s[e] - base);
            l += w;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 v2 = unpack2<F16>(vw[e][i]);
                acc[2 * i] = fmaf(w, v2.x, acc[2 * i]);
                acc[2 * i + 1] = fmaf(w, v2.y, acc[2 * i + 1]);
            }
        }
    }
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Where a tile item stands in the CTA's barriers: counts carried across items.
struct Counts {
    uint32_t kv = 0;            // K and V loads into the ring
    uint32_t s[2] = {0, 0};     // blocks of each tile
    uint32_t items = 0;         // tile items with keys
    uint32_t fixes = 0;         // ... whose last keys' block needed clean V rows
};
struct Tile {
    int kind, g, t0, nt, kvp0, kb, ke, part;
    int nb, tok[2];             // blocks, tokens of each tile
    bool fix;
};
template <int D>
__device__ __forceinline__ Tile tile_of(const Params& P, const int* it) {
    Tile T;
    T.kind = it[kKind];
    T.g = it[kG];
    T.t0 = it[kT0];
    T.nt = it[kNt];
    T.kvp0 = it[kKvp0];
    T.kb = it[kKb];
    T.ke = it[kKe];
    T.part = it[kPart];
    T.nb = (T.ke - T.kb + Layout<D>::kKeys - 1) / Layout<D>::kKeys;
    const int tpt = kTileRows / P.group;
    T.tok[0] = min(tpt, T.nt);
    T.tok[1] = T.nt - T.tok[0];
    T.fix = (T.ke - T.kb) % Layout<D>::kKeys != 0;
    return T;
}
__device__ __forceinline__ void count_item(Counts& c, const Tile& T) {
    if (T.nb == 0) return;
    c.kv += 2u * (uint32_t)T.nb;
    c.s[0] += (uint32_t)T.nb;
    if (T.tok[1]) c.s[1] += (uint32_t)T.nb;
    ++c.items;
    c.fixes += T.fix;
}

// ---------------------------------------------------------------------------
// TILE, warp 8: K and V blocks into the ring, in the order in which the products
// take them: K0, K1 V0, K2 V1, ..., V(n-1).  Block 0 holds the item's last keys:
// from there on a bias by distance only falls, so that the largest scores come
// first and the sums are not rescaled at every block (with slopes up to 0.84 a
// block of 2 x 128 x 80 scores took 2550 cycles in the keys' own order).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t k_load(const Counts& c, int j) { return c.kv + (j ? 2u * (uint32_t)j - 1u : 0u); }
__device__ __forceinline__ uint32_t v_load(const Counts& c, int j, int nb) {
    return c.kv + 2u * (uint32_t)j + (j == nb - 1 ? 1u : 2u);
}
template <int D>
__device__ void tile_loads(const Params& P, const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                           const CUtensorMap* tmK5, const CUtensorMap* tmV5, const Tile& T, const Counts& c,
                           uint8_t* smem, uint32_t bars, Shared* sh) {
    using L = Layout<D>;
    const int lane = threadIdx.x & 31;
    const int G = P.group, tpt = kTileRows / G;
    // lane 8 hf + i holds the id of the block's page i, and issues the box of
    // that page and column half where the pages are not consecutive in the pool
    const int hf = lane >> 3, pi = lane & 7;
    const int p_first = T.kb / kPage, p_end = (T.ke + kPage - 1) / kPage;
    auto ids_of = [&](int j) {
        const int e = p_first + L::kPages * (T.nb - 1 - j) + pi;
        return j < T.nb && pi < L::kPages && e < p_end ? page_id(P, T.kvp0 + e) : 0;
    };
    auto load = [&](uint32_t kv, int j, int id, const CUtensorMap* map, const CUtensorMap* map5) {
        const int npg = min(L::kPages, p_end - (p_first + L::kPages * (T.nb - 1 - j)));
        const int id0 = __shfl_sync(0xffffffffu, id, 0);
        const bool one_box = __all_sync(0xffffffffu, pi >= npg || id == id0 + pi);
        const int st = (int)(kv % L::kStages);
        const uint32_t full = bars + 8 * (kKvFull + st);
        if (!wait_warp(P, bars + 8 * (kKvEmpty + st), ((kv / L::kStages) & 1u) ^ 1u, sh, 1000 + j)) return false;
        uint8_t* dst = smem + st * L::kBlkBytes;
        if (one_box) {
            // one box for the block (pages past the row's come along unused)
            if (lane == 0) {
                mbar_expect_tx(full, (uint32_t)L::kBlkBytes);
                tma_load_5d(smem_u32(dst), map5, 0, 0, T.g, id0, 0, full);
            }
        } else {
            if (lane == 0) mbar_expect_tx(full, (uint32_t)(npg * L::kPageBytes));
            __syncwarp();
            if (hf < L::kHalves && pi < npg)
                tma_load_2d(smem_u32(dst + hf * L::kBlkHalf + pi * kPage * 128), map, hf * 64,
                            (id * P.Hkv + T.g) * kPage, full);
        }
        __syncwarp();
        return true;
    };
    int id = ids_of(0), prev = 0;
    // the Q tiles once the item before is done with its scores
    if (!wait_warp(P, bars + 8 * kQFree, (c.items & 1u) ^ 1u, sh, 900)) return;
    if (lane == 0) {
        const int tiles = T.tok[1] ? 2 : 1;
        mbar_expect_tx(bars + 8 * kQFull, (uint32_t)(tiles * L::kHalves * G * tpt * 128));
        for (int x = 0; x < tiles; ++x)
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_3d(smem_u32(smem + L::kQ + x * L::kQBytes + h * kTileRows * 128), tmQ, h * 64, T.g * G,
                            T.t0 + x * tpt, bars + 8 * kQFull);
    }
    __syncwarp();
    for (int j = 0; j <= T.nb; ++j) {
        const int nxt = ids_of(j + 1);
        if (j < T.nb && !load(k_load(c, j), j, id, tmK, tmK5)) return;
        if (j > 0 && !load(v_load(c, j - 1, T.nb), j - 1, prev, tmV, tmV5)) return;
        prev = id;
        id = nxt;
    }
}

// ---------------------------------------------------------------------------
// TILE, warps 9 and 10: the products, S = Q K^T of a block as soon as the softmax
// has loaded the block before's scores, O += P V once its weights are stored, so
// that both run while the softmax works.  Two warps, since one that issues both
// spends a third of the time waiting for one kind while the other could go.
// 80 keys a block at d = 128: tensor memory holds P beside S in 2 x (80 S + 40 P +
// 128 O) columns.  With 128 keys P has to lie over S, and S of block j + 1 waits
// for P V of block j, 1850 of the 4250 cycles that 2 x 128 x 128 scores took.
// ---------------------------------------------------------------------------
template <int D, bool F16>
__device__ void tile_scores(const Params& P, const Tile& T, const Counts& c, uint8_t* smem, uint32_t bars,
                            uint32_t tmem, Shared* sh) {
    using L = Layout<D>;
    constexpr uint32_t idesc = umma_idesc<F16>(L::kKeys, false), hi = umma_desc_hi(1024);
    const int tiles = (int)uniform(T.tok[1] ? 2u : 1u);
    const uint32_t ring = smem_u32(smem), tm = uniform(tmem), q_lo = uniform(umma_desc_lo(ring + L::kQ, 16));
    if (!wait_warp(P, bars + 8 * kQFull, c.items & 1u, sh, 2000)) return;
    for (int j = 0; j < T.nb; ++j) {
        const uint32_t kv = k_load(c, j), st = kv % L::kStages;
        if (!wait_warp(P, bars + 8 * (kKvFull + st), (kv / L::kStages) & 1u, sh, 2100 + j)) return;
        const uint32_t k_lo = uniform(umma_desc_lo(ring + st * L::kBlkBytes, 16));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x >= tiles) break;
            if (!wait_warp(P, bars + 8 * (kSFree + x), ((c.s[x] + (uint32_t)j) & 1u) ^ 1u, sh, 3000 + j)) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_ss(tm + L::s_col(x),
                            umma_desc(q_lo + ((x * L::kQBytes + (kk >> 2) * kTileRows * 128 + (kk & 3) * 32) >> 4), hi),
                            umma_desc(k_lo + (((kk >> 2) * L::kBlkHalf + (kk & 3) * 32) >> 4), hi), idesc, kk > 0);
                umma_commit(bars + 8 * (kSFull + x));
                if (x == tiles - 1) {
                    umma_commit(bars + 8 * (kKvEmpty + st));
                    if (j == T.nb - 1) umma_commit(bars + 8 * kQFree);
                }
            }
            __syncwarp();
        }
    }
}
template <int D, bool F16>
__device__ void tile_sums(const Params& P, const Tile& T, const Counts& c, uint8_t* smem, uint32_t bars, uint32_t tmem,
                          Shared* sh) {
    using L = Layout<D>;
    constexpr uint32_t idesc = umma_idesc<F16>(D, true), hi = umma_desc_hi(1024);
    const int tiles = (int)uniform(T.tok[1] ? 2u : 1u);
    const uint32_t ring = smem_u32(smem), tm = uniform(tmem);
    for (int j = 0; j < T.nb; ++j) {
        const uint32_t kv = v_load(c, j, T.nb), st = kv % L::kStages;
        if (!wait_warp(P, bars + 8 * (kKvFull + st), (kv / L::kStages) & 1u, sh, 4000 + j)) return;
        if (j == 0 && T.fix) {
            if (elect_one()) mbar_arrive(bars + 8 * kVLast);
            __syncwarp();
            if (!wait_warp(P, bars + 8 * kVFix, c.fixes & 1u, sh, 4500)) return;
        }
        const uint32_t v_lo = uniform(umma_desc_lo(ring + st * L::kBlkBytes, L::kBlkHalf));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x >= tiles) break;
            if (!wait_warp(P, bars + 8 * (kPFull + x), (c.s[x] + (uint32_t)j) & 1u, sh, 5000 + j)) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < L::kPages; ++kk)
                    // P from tensor memory (16 keys = 8 columns a step), V MN-major as the pages hold it
                    umma_ts(tm + L::o_col(x), tm + L::p_col(x) + 8u * kk, umma_desc(v_lo + ((kk * 16 * 128) >> 4), hi),
                            idesc, kk > 0 ? 1u : (uint32_t)(j > 0));
                umma_commit(bars + 8 * (kPvDone + x));
                if (x == tiles - 1) umma_commit(bars + 8 * (kKvEmpty + st));
            }
            __syncwarp();
        }
    }
}

// TILE, warp 11: V rows past the item's last key hold other bytes; zeros, so
// that a weight of 0 gives 0.
template <int D>
__device__ void tile_clean(const Params& P, const Tile& T, const Counts& c, uint8_t* smem, uint32_t bars, Shared* sh) {
    using L = Layout<D>;
    // (not the ring's own barrier: its parity says nothing to a thread that did
    // not wait for the stage's earlier loads)
    if (!wait(P, bars + 8 * kVLast, c.fixes & 1u, sh, 7000)) return;
    uint8_t* dst = smem + (v_load(c, 0, T.nb) % L::kStages) * L::kBlkBytes;
    const int first = (T.ke - T.kb) % L::kKeys;
    for (int hf = 0; hf < L::kHalves; ++hf)
        for (int i = first * 128 + (int)(threadIdx.x & 31) * 16; i < L::kBlkHalf; i += 32 * 16)
            *reinterpret_cast<uint4*>(dst + hf * L::kBlkHalf + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
    mbar_arrive(bars + 8 * kVFix);
}

// cap2 tanh(scale v) = v p(v^2) while |scale v| is small, p the polynomial with the
// smallest largest error there (fitted by iterated weighted least squares), its
// coefficients times the powers of the scale: degree 2 up to 0.35 (within 5e-7 of
// tanh), degree 3 up to 0.6 (6e-7).  Four or five multiply-adds of two lanes for
// two scores, where the exponential and the reciprocal of tanh_abs keep the
// special-function unit twice as long as the softmax's own exponentials do: 2048
// tokens behind 2048 keys (32 heads, d 128, cap 30) take 121 us with queries and keys
// of deviation 2 and 1 (scores below 0.35 of the cap), 142 with 3 and 1, 196 with 6 and
// 1 (most warps' largest pass 0.6); 91 uncapped.
// A warp takes it where all of a block's scores allow; scales whose seventh power
// would leave fp32 do not.  The scores of keys that a row does not see are left out:
// past an item's last key they are products with whatever the ring held, and the
// formulas differ in the last bits.  The maximum of the seen ones is taken only
// where the block's largest score of all is above the first bound: the same tokens
// with a window of 500 take 41.9 us, 46.5 where every block with a hidden key takes
// it.  A choice by row instead of by warp takes 1.15 to 1.4 times as long.
constexpr float kTanhLow = 0.35f, kTanhHigh = 0.6f;
constexpr float kScaleLow = 2e-4f, kScaleHigh = 50.f;
struct CapPoly {
    float low[3], high[4];
};
__device__ __forceinline__ CapPoly cap_poly(float cap2, float scale) {
    const float q = scale * scale;
    float f = cap2 * scale;
    CapPoly c;
    c.high[0] = f * 0.9999909996986389f;
    c.low[0] = f * 0.9999902248382568f;
    f *= q;
    c.high[1] = f * -0.33298975229263306f;
    c.low[1] = f * -0.33268409967422485f;
    f *= q;
    c.high[2] = f * 0.1297455132007599f;
    c.low[2] = f * 0.1224803775548935f;
    f *= q;
    c.high[3] = f * -0.03961123153567314f;
    return c;
}
template <int N>
__device__ __forceinline__ float2 odd_poly(float2 v, const float (&c)[N]) {
    const float2 u = fmul2(v, v);
    float2 p = make_float2(c[N - 1], c[N - 1]);
#pragma unroll
    for (int k = N - 2; k >= 0; --k) p = ffma2(p, u, make_float2(c[k], c[k]));
    return fmul2(v, p);
}

// Bits [a, z) of 32.
__device__ __forceinline__ uint32_t bit_range(int a, int z) {
    const uint32_t below_z = z >= 32 ? 0xFFFFFFFFu : z <= 0 ? 0u : (1u << z) - 1u;
    const uint32_t below_a = a >= 32 ? 0xFFFFFFFFu : a <= 0 ? 0u : (1u << a) - 1u;
    return below_z & ~below_a;
}

// ---------------------------------------------------------------------------
// TILE, warps 4 x .. 4 x + 3: the softmax of tile x, one thread a query row.
// The exponent base moves only when a block's maximum passes it by 2^8, so O is
// rarely rescaled (weights stay below 2^8; their sum and O are fp32).
// ---------------------------------------------------------------------------
// What a tile's scores may be, as far as a kernel knows.  The code of other kinds
// costs time even where no call takes it: 2048 tokens behind 6144 keys with a bias
// take 200 us with a kernel of their own, 217 with the one for all; 2048 behind 2048
// at d = 64 64 us plain (70) and 83 biased (87).  Plain scores at d = 128 (95 against
// 91 us) and capped ones (2% less) have none.
enum Scores { kAny = 0, kBiased = 1, kPlain = 2 };

// A thread's query row of its tile.
struct TileRow {
    int rows;          // of the tile
    int t, h;          // token and q head (rows past the tile's stand for its last one)
    int lo, hi, pos;   // keys of the item that it sees; its position
    float slope2;
};
__device__ __forceinline__ TileRow row_of(const Params& P, const Tile& T) {
    TileRow R;
    const int x = threadIdx.x >> 7;
    R.rows = T.kind < 0 ? 0 : (x ? T.tok[1] : T.tok[0]) * P.group;
    if (R.rows == 0) return R;
    const int rr = min((int)threadIdx.x & 127, R.rows - 1);
    R.t = T.t0 + (x ? T.tok[0] : 0) + rr / P.group;
    R.h = T.g * P.group + rr % P.group;
    const int4 tok = *reinterpret_cast<const int4*>(P.plan + P.off_tokens + (size_t)R.t * kTokenWords);
    R.slope2 = P.slopes ? P.slopes[R.h] * 1.4426950408889634f : 0.f;
    R.lo = max(tok.x, T.kb);
    R.hi = min(tok.y, T.ke);
    R.pos = tok.z;
    return R;
}
template <int D, bool F16, int KIND, typename Next>
__device__ void tile_softmax(const Params& P, const Tile& T, const TileRow& R, const Counts& c, uint8_t* smem,
                             uint32_t bars, uint32_t tmem, Shared* sh, Next next) {
    using L = Layout<D>;
    constexpr int N = L::kKeys;
    const int x = threadIdx.x >> 7, r = threadIdx.x & 127, lane = threadIdx.x & 31;
    if (R.rows == 0) {
        next();
        return;
    }
    const uint32_t blocks = x ? c.s[1] : c.s[0];
    const uint32_t base = tmem + ((uint32_t)(r & 96) << 16);
    const uint32_t s_col = base + L::s_col(x), p_col = base + L::p_col(x), o_col = base + L::o_col(x);
    const int t = R.t, h = R.h, lo = R.lo, hi = R.hi;
    const float slope2 = R.slope2;
    const bool capped = KIND == kAny && P.cap2 > 0.f, biased = KIND == kBiased || (KIND == kAny && P.slopes);
    const float mul = capped || biased ? 1.f : P.raw_scale;  // of what v holds when the weights are taken
    const bool poly = P.raw_scale >= kScaleLow && P.raw_scale <= kScaleHigh && !P.cap_fine;
    const CapPoly cp = cap_poly(P.cap2, P.raw_scale);
    const bool idle = r >= R.rows;  // (what such a thread holds has no say)
    float m_run = -INFINITY, l_run = 0.f;
    for (int j = 0; j < T.nb; ++j) {
        const uint32_t odd = (blocks + (uint32_t)j) & 1u;
        if (!wait_warp(P, bars + 8 * (kSFull + x), odd, sh, 8000 + j)) return;
        tc_fence_after();
        float v[N];
        tmem_ld<N>(s_col, v);
        tmem_wait_ld(v);
        // the scores are in registers: the next block's may come
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kSFree + x));
        const int key0 = T.kb + (T.nb - 1 - j) * N;
        if (capped) {
            float am[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < N; e += 8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) am[q] = fmax3(am[q], fabsf(v[e + 2 * q]), fabsf(v[e + 2 * q + 1]));
            }
            float top = fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3])) * P.raw_scale;
            bool low = __all_sync(0xffffffffu, top <= kTanhLow || idle);
            // (else the largest that the row sees)
            if (!low && __any_sync(0xffffffffu, key0 < lo || key0 + N > hi)) {
                top = 0.f;
#pragma unroll
                for (int q = 0; q < N; q += 16) {
                    const uint32_t seen = bit_range(lo - key0 - q, hi - key0 - q);
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, seen & (1u << e) ? fabsf(v[q + e]) : 0.f);
                }
                top *= P.raw_scale;
                low = __all_sync(0xffffffffu, top <= kTanhLow || idle);
            }
            if (poly && low) {
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float2 w = odd_poly(make_float2(v[e], v[e + 1]), cp.low);
                    v[e] = w.x;
                    v[e + 1] = w.y;
                }
            } else if (poly && __all_sync(0xffffffffu, top <= kTanhHigh || idle)) {
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float2 w = odd_poly(make_float2(v[e], v[e + 1]), cp.high);
                    v[e] = w.x;
                    v[e + 1] = w.y;
                }
            } else if (!P.cap_fine) {
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = P.cap2 * tanh_abs(v[e] * P.raw_scale);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = P.cap2 * tanh_fine(v[e] * P.raw_scale);
            }
        }
        if (biased) {
            const float a = capped ? 1.f : P.raw_scale;
            const float2 a2 = make_float2(a, a);
            const int d0 = R.pos - key0;  // distance of the block's first key
            if (__all_sync(0xffffffffu, d0 >= N - 1)) {
                // the whole block at or before the rows' positions: -slope (d0 - e), two at a time
                const float2 s2 = make_float2(slope2, slope2);
                const float c0 = -slope2 * (float)d0;
                const float2 c2 = make_float2(c0, c0 + slope2);
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float2 b = ffma2(s2, make_float2((float)e, (float)e), c2);
                    const float2 y = ffma2(make_float2(v[e], v[e + 1]), a2, b);
                    v[e] = y.x;
                    v[e + 1] = y.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = fmaf(-slope2, fabsf((float)(d0 - e)), v[e] * a);
            }
        }
        if (__any_sync(0xffffffffu, key0 < lo || key0 + N > hi)) {
#pragma unroll
            for (int q = 0; q < N; q += 16) {
                const uint32_t seen = bit_range(lo - key0 - q, hi - key0 - q);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[q + e] = seen & (1u << e) ? v[q + e] : -INFINITY;
            }
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < N; e += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) mq[q] = fmax3(mq[q], v[e + 2 * q], v[e + 2 * q + 1]);
        }
        const float mx = fmax3(fmaxf(mq[0], mq[1]), mq[2], mq[3]) * mul;
        const float m_use = mx > m_run + 8.f ? mx : m_run;
        const float m_exp = m_use == -INFINITY ? 0.f : m_use - weight_up<F16>();  // (no key seen yet: weights 0)
        const float2 mul2 = make_float2(mul, mul), nm2 = make_float2(-m_exp, -m_exp);
        float2 sum2 = make_float2(0.f, 0.f);
        uint32_t pk[N / 2];
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 y = ffma2(make_float2(v[e], v[e + 1]), mul2, nm2);
            const float2 w = make_float2(ex2(y.x), ex2(y.y));
            sum2 = fadd2(sum2, w);
            pk[e >> 1] = pack2<F16>(w.x, w.y);
        }
        // P's columns and O are free once the P V of the block before is done
        if (!wait_warp(P, bars + 8 * (kPvDone + x), odd ^ 1u, sh, 8500 + j)) return;
        tc_fence_after();
        tmem_st<N / 2>(p_col, pk);
        const bool moved = m_use != m_run;
        const float alpha = moved ? ex2(m_run - m_use) : 1.f;
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
#pragma unroll 1
            for (int q = 0; q < D; q += 32) {
                float o[32];
                tmem_ld32(o_col + q, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                tmem_st32(o_col + q, reinterpret_cast<const uint32_t*>(o));
            }
        }
        l_run = l_run * alpha + (sum2.x + sum2.y);
        m_run = m_use;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kPFull + x));
    }
    next();  // (the next item's row is on its way while this one's is stored)
    // the item's rows
    if (T.nb > 0) {
        if (!wait_warp(P, bars + 8 * (kPvDone + x), (blocks + (uint32_t)T.nb - 1u) & 1u, sh, 9000)) return;
        tc_fence_after();
    }
    const bool mine = r < R.rows;
    const int part_row = T.part < 0 ? -1 : T.part + (x ? T.tok[0] * P.group : 0) + r;
    const size_t out_row = (size_t)t * P.Hq + h;
    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
    // A thread holds a row, but a row's 128 bytes should leave together: each
    // warp passes its 32 rows through shared memory (16-byte chunk c of row r at
    // c ^ (r & 7)), 32 columns of a partial row or 64 of out at a time, and 8
    // lanes store a row's piece.  Stored by rows straight from the registers a
    // tile's 256 partial rows took 6 us.
    uint8_t* stg = smem + L::kStage + (threadIdx.x >> 5) * 4096;
    const uint64_t row_at = T.part < 0 ? reinterpret_cast<uint64_t>(P.out + out_row * D)
                                       : reinterpret_cast<uint64_t>(P.part_o + (size_t)part_row * D);
    const int warp_rows = min(32, R.rows - (r & 96));  // (may be negative)
    float check = 0.f;
#pragma unroll 1
    for (int q = 0; q < D; q += 32) {
        float o[32];
        if (T.nb > 0) {
            tmem_ld32(o_col + q, o);
            tmem_wait_ld(o);
            // A row that sees none of the item's keys has weights of 0, and 0 times an
            // infinite value of a key that other rows see is NaN: zeros, whatever O holds.
            if (lo >= hi) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) check = fmaf(o[e], 0.f, check);  // NaN once one is infinite or NaN
        uint4* mine_at = reinterpret_cast<uint4*>(stg + lane * 128);
        if (T.part >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mine_at[i ^ (lane & 7)] = make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                                                     __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mine_at[(i + (q & 32) / 8) ^ (lane & 7)] =
                    make_uint4(pack2<F16>(o[8 * i] * inv, o[8 * i + 1] * inv),
                               pack2<F16>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                               pack2<F16>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                               pack2<F16>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        }
        if (T.part < 0 && !(q & 32)) continue;  // (half of the 128 bytes)
        __syncwarp();
        const int byte = T.part >= 0 ? q * 4 : (q & ~32) * 2;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const int row = i + (lane >> 3);
            const uint64_t at = __shfl_sync(0xffffffffu, row_at, row);
            if (row < warp_rows)
                *reinterpret_cast<uint4*>(at + byte + (lane & 7) * 16) =
                    *reinterpret_cast<const uint4*>(stg + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
        }
        __syncwarp();
    }
    if (mine) {
        if (part_row >= 0)
            P.part_ml[part_row] = make_float2(m_run - weight_up<F16>(), l_run);
        else if (P.lse)
            P.lse[out_row] = lse_of(m_run - weight_up<F16>(), l_run);
    }
    // A row that is not finite although keys are hidden from it: 0 times an
    // infinite value of a hidden key is NaN.  Such rows again, over their own
    // keys only.
    uint32_t again = __ballot_sync(0xffffffffu, mine && check != 0.f && (lo > T.kb || hi < T.ke));
    for (; again; again &= again - 1) {
        const int src = __ffs(again) - 1;
        const int t2 = __shfl_sync(0xffffffffu, t, src), h2 = __shfl_sync(0xffffffffu, h, src);
        const int lo2 = __shfl_sync(0xffffffffu, lo, src), hi2 = __shfl_sync(0xffffffffu, hi, src);
        const int pr2 = __shfl_sync(0xffffffffu, part_row, src);
        const float sl2 = __shfl_sync(0xffffffffu, slope2, src);
        const int pos2 = __shfl_sync(0xffffffffu, R.pos, src);
        float m, l, acc[D / 32];
        attend_row<D, F16>(P, P.q + t2 * P.q_stride + (size_t)h2 * D, T.kvp0, pos2, T.g, sl2, lo2, hi2, m, l, acc);
        const float inv2 = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < D / 32; i += 2) {
            const int col = lane * (D / 32) + i;
            if (pr2 >= 0)
                *reinterpret_cast<float2*>(P.part_o + (size_t)pr2 * D + col) = make_float2(acc[i], acc[i + 1]);
            else
                *reinterpret_cast<uint32_t*>(P.out + ((size_t)t2 * P.Hq + h2) * D + col) =
                    pack2<F16>(acc[i] * inv2, acc[i + 1] * inv2);
        }
        if (lane == 0) {
            if (pr2 >= 0)
                P.part_ml[pr2] = make_float2(m, l);
            else if (P.lse)
                P.lse[(size_t)t2 * P.Hq + h2] = lse_of(m, l);
        }
    }
}

// ---------------------------------------------------------------------------
// STREAM, each of warps 0-7 by itself: pages of a one-token row for one kv head
// through the warp's TMA ring.  The loads run ahead of the work by the ring's
// depth and on into the warp's next item, so that a short item costs little more
// than its bytes; the item after that is being claimed meanwhile.
// ---------------------------------------------------------------------------
struct Stream {
    int g, t, part, lo, hi;      // keys [lo, hi) of the item that the token sees
    int entry, np;               // page-list entry of its first page, pages (-1: no item)
    int key0;                    // first key of the first page
    int pos;
    int issued;                  // pages whose loads have been issued
    int ids;                     // lane i: id of page 32 (issued / 32) + i
};
__device__ __forceinline__ void load_ids(const Params& P, Stream& it) {
    const int k = (it.issued & ~31) + ((int)threadIdx.x & 31);
    it.ids = k < it.np ? page_id(P, it.entry + k) : 0;
}

template <int D, bool F16>
__device__ void run_streams(const Params& P, const CUtensorMap* tmK, const CUtensorMap* tmV, uint8_t* smem,
                            uint32_t bars, Shared* sh, bool preferred) {
    using L = Layout<D>;
    constexpr int NST = L::kStreamStages, PB = L::kPageBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mi = lane >> 3, G = P.group;
    const int n_second = P.n_items - P.n_first;
    // The first items need no atomic: warp w of the b-th CTA that prefers the
    // queue takes item w n + b of it, and the head counts the claims after those.
    const int ctas = (int)gridDim.x - P.first_sms, given = min(kStreamWarps * ctas, n_second);
    uint8_t* qtile = smem + L::kStreamQ + warp * PB;
    // An item comes in three steps, each with what the one before has loaded: its
    // index, from the queue's head; its record; its token, page ids and queries.
    // While an item is in work the next one takes a step a page, so that none of
    // the loads is waited for.  (Only one is claimed ahead: more would leave the
    // last ones with few warps.)
    int asked = 0;
    int4 ra, rb, tok;
    auto ask = [&] {
        if (lane == 0) asked = given + atomicAdd(&P.ws[kHead1], 1);
    };
    auto fetch = [&](int k) {  // item k of the queue; false: there is none
        if (k >= n_second) return false;
        const int4* src = reinterpret_cast<const int4*>(P.plan + P.off_items + (size_t)(P.n_first + k) * kItemWords);
        ra = __ldg(src);      // kind g t0 nt
        rb = __ldg(src + 1);  // kvp0 kb ke part
        return true;
    };
    auto open = [&](Stream& s) {
        s.g = ra.y;
        s.t = ra.z;
        s.part = rb.w;
        s.key0 = rb.y;
        s.entry = rb.x + rb.y / kPage;
        s.np = (rb.z + kPage - 1) / kPage - rb.y / kPage;
        s.issued = 0;
        load_ids(P, s);
        tok = __ldg(reinterpret_cast<const int4*>(P.plan + P.off_tokens + (size_t)s.t * kTokenWords));
        // its queries into the tile, whose rows past the group's stay zero (the
        // item in work holds its own in registers)
        const uint16_t* q = P.q + s.t * P.q_stride + (size_t)s.g * G * D;
        for (int i = lane; i < G * (D / 8); i += 32)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(qtile + sw128_chunk(16, i / (D / 8), i % (D / 8)))),
                         "l"(q + (size_t)i * 8)
                         : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto see = [&](Stream& s) {
        s.lo = max(tok.x, rb.y);
        s.hi = min(tok.y, rb.z);
        s.pos = tok.z;
    };
    for (int i = G * (D / 8) + lane; i < 16 * (D / 8); i += 32)
        *reinterpret_cast<uint4*>(qtile + sw128_chunk(16, i / (D / 8), i % (D / 8))) = make_uint4(0, 0, 0, 0);
    Stream cur, nxt;
    {
        int k = warp * ctas + (int)blockIdx.x - P.first_sms;
        if (!preferred) {
            ask();
            k = __shfl_sync(0xffffffffu, asked, 0);
        }
        if (!fetch(k)) return;
        open(cur);
        see(cur);
    }
    ask();
    int steps = 0;  // that the next item has taken; 3: it is there, or there is none
    nxt.np = -1;
    nxt.issued = 0;
    auto advance = [&] {
        if (steps == 0) {
            const int k = __shfl_sync(0xffffffffu, asked, 0);
            steps = fetch(k) ? 1 : 3;
        } else if (steps == 1) {
            open(nxt);
            steps = 2;
        } else if (steps == 2) {
            see(nxt);
            steps = 3;
        }
    };

    uint8_t* ring = smem + warp * NST * 2 * PB;
    const uint32_t wbar = bars + 8 * (kStreamBar + 3 * warp);
    uint32_t fill = 0, use = 0;  // pages issued and taken, in all
    auto issue_from = [&](Stream& it) {
        const int page = __shfl_sync(0xffffffffu, it.ids, it.issued & 31);
        if (lane == 0) {
            const uint32_t st = fill % NST, dst = smem_u32(ring + st * 2 * PB), bar = wbar + 8 * st;
            mbar_expect_tx(bar, 2 * PB);
            const int y = (page * P.Hkv + it.g) * kPage;
            if (D == 128) {  // {64 columns, 16 rows, 2 halves}: a page of the head in one box
                tma_load_3d(dst, tmK, 0, y, 0, bar);
                tma_load_3d(dst + PB, tmV, 0, y, 0, bar);
            } else {
                tma_load_2d(dst, tmK, 0, y, bar);
                tma_load_2d(dst + PB, tmV, 0, y, bar);
            }
        }
        ++fill;
        ++it.issued;
        if ((it.issued & 31) == 0) load_ids(P, it);
    };
    auto issue = [&] {
        while (fill - use < (uint32_t)NST) {
            if (cur.issued < cur.np)
                issue_from(cur);
            else if (steps == 3 && nxt.issued < nxt.np)
                issue_from(nxt);
            else
                break;
        }
    };
    issue();
    const int rA = lane >> 2, rB = rA + 8;          // this lane's rows of the fragments
    while (cur.np >= 0) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            ldsm_x4(smem_u32(qtile + sw128_chunk(16, (mi & 1) * 8 + (lane & 7), 2 * kk + (mi >> 1))), qf[kk][0],
                    qf[kk][1], qf[kk][2], qf[kk][3]);
        __syncwarp();  // (the next item's queries may overwrite the tile)
        const float slA = P.slopes && rA < G ? P.slopes[cur.g * G + rA] * 1.4426950408889634f : 0.f;
        const float slB = P.slopes && rB < G ? P.slopes[cur.g * G + rB] * 1.4426950408889634f : 0.f;
        float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f;
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        for (int k = 0; k < cur.np; ++k) {
            const uint32_t st = use % NST;
            if (!wait_warp(P, wbar + 8 * st, (use / NST) & 1u, sh, k)) return;
            uint8_t* kbuf = ring + st * 2 * PB;
            uint8_t* vbuf = kbuf + PB;
            const int key0 = cur.key0 + kPage * k;
            const bool edge = key0 < cur.lo || key0 + kPage > cur.hi;
            if (edge) {
                // values of keys that the token does not see: zeros, so that their weight 0 gives 0
                for (int i = lane; i < kPage * (D / 8); i += 32) {
                    const int row = i / (D / 8);
                    if (key0 + row < cur.lo || key0 + row >= cur.hi)
                        *reinterpret_cast<uint4*>(vbuf + sw128_chunk(kPage, row, i % (D / 8))) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
            // (two accumulators a score: half as long a chain of products)
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, s2[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(smem_u32(kbuf + sw128_chunk(kPage, (mi >> 1) * 8 + (lane & 7), 2 * kk + (mi & 1))), b0, b1, b2,
                        b3);
                mma_16816<F16>(kk & 1 ? s2[0] : sc[0], qf[kk], b0, b1);
                mma_16816<F16>(kk & 1 ? s2[1] : sc[1], qf[kk], b2, b3);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = (sc[n][e] + s2[n][e]) * P.raw_scale;
            }
            if (P.cap2 > 0.f) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[n][e] = P.cap2 * (P.cap_fine ? tanh_fine(sc[n][e]) : tanh_abs(sc[n][e]));
                }
            }
            const int lk = 2 * (lane & 3);  // this lane's keys of the page: lk, lk + 1, lk + 8, lk + 9
            if (P.slopes) {
                const float d0 = (float)(cur.pos - key0 - lk);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[n][e] = fmaf(e < 2 ? -slA : -slB, fabsf(d0 - (float)(8 * n + (e & 1))), sc[n][e]);
                }
            }
            if (edge) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + lk + 8 * n + (e & 1);
                        sc[n][e] = key >= cur.lo && key < cur.hi ? sc[n][e] : -INFINITY;
                    }
                }
            }
            float mxA = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
            float mxB = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
            mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, 1));
            mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, 1));
            mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, 2));
            mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, 2));
            // the base moves when the maximum passes it by 2^8, as in a tile
            const float nA = mxA > mA + 8.f ? mxA : mA, nB = mxB > mB + 8.f ? mxB : mB;
            if (__any_sync(0xffffffffu, nA != mA || nB != mB)) {
                const float alA = nA == mA ? 1.f : ex2(mA - nA), alB = nB == mB ? 1.f : ex2(mB - nB);
                lA *= alA;
                lB *= alB;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= alA;
                    o[n][1] *= alA;
                    o[n][2] *= alB;
                    o[n][3] *= alB;
                }
                mA = nA;
                mB = nB;
            }
            const float bA = mA == -INFINITY ? 0.f : mA - weight_up<F16>();
            const float bB = mB == -INFINITY ? 0.f : mB - weight_up<F16>();
            const float p00 = ex2(sc[0][0] - bA), p01 = ex2(sc[0][1] - bA), p02 = ex2(sc[0][2] - bB),
                        p03 = ex2(sc[0][3] - bB), p10 = ex2(sc[1][0] - bA), p11 = ex2(sc[1][1] - bA),
                        p12 = ex2(sc[1][2] - bB), p13 = ex2(sc[1][3] - bB);
            lA += (p00 + p01) + (p10 + p11);
            lB += (p02 + p03) + (p12 + p13);
            const uint32_t pa[4] = {pack2<F16>(p00, p01), pack2<F16>(p02, p03), pack2<F16>(p10, p11),
                                    pack2<F16>(p12, p13)};
#pragma unroll
            for (int n2 = 0; n2 < D / 16; ++n2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(smem_u32(vbuf + sw128_chunk(kPage, (mi & 1) * 8 + (lane & 7), 2 * n2 + (mi >> 1))), b0, b1,
                          b2, b3);
                mma_16816<F16>(o[2 * n2], pa, b0, b1);
                mma_16816<F16>(o[2 * n2 + 1], pa, b2, b3);
            }
            ++use;
            if (edge) fence_proxy_async_shared();  // the zeroed rows are next written by TMA
            __syncwarp();
            advance();
            issue();
        }
        while (steps < 3) advance();  // (a short item)
        issue();
        lA += __shfl_xor_sync(0xffffffffu, lA, 1);
        lA += __shfl_xor_sync(0xffffffffu, lA, 2);
        lB += __shfl_xor_sync(0xffffffffu, lB, 1);
        lB += __shfl_xor_sync(0xffffffffu, lB, 2);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = half ? rB : rA;
            if (row >= G) continue;
            const float m = (half ? mB : mA) - weight_up<F16>(), l = half ? lB : lA;
            const size_t out_row = (size_t)cur.t * P.Hq + cur.g * G + row;
            if (cur.part >= 0) {
                float* dst = P.part_o + (size_t)(cur.part + row) * D + 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * half], o[n][2 * half + 1]);
                if ((lane & 3) == 0) P.part_ml[cur.part + row] = make_float2(m, l);
            } else {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint16_t* dst = P.out + out_row * D + 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<uint32_t*>(dst + 8 * n) = pack2<F16>(o[n][2 * half] * inv, o[n][2 * half + 1] * inv);
                if ((lane & 3) == 0 && P.lse) P.lse[out_row] = lse_of(m, l);
            }
        }
        cur = nxt;
        if (cur.np >= 0) {
            ask();
            steps = 0;
            nxt.np = -1;
            nxt.issued = 0;
        }
    }
}

// TILES, STREAMS: which of the two kinds of item the plan has.  (A kernel with
// both is 2 to 3% slower on either alone.)
template <int D, bool F16, int KIND, bool TILES, bool STREAMS>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmK3, const __grid_constant__ CUtensorMap tmV3,
                      const __grid_constant__ CUtensorMap tmK5, const __grid_constant__ CUtensorMap tmV5) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Shared shared;
    Shared* sh = &shared;
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t bars = smem_u32(sh->bars);
    if (tid == 0) {
        sh->abort = 0;
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t n = 1;
            if (i == kPFull || i == kPFull + 1 || i == kSFree || i == kSFree + 1) n = 4;
            if (i == kVFix) n = 32;
            if (i >= kItemFree && i < kItemFree + kItemSlots) n = kItemReaders;
            mbar_init(bars + 8 * i, n);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (TILES && warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh->tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // This launch may begin while the stream's kernel before it ends, and the next
    // one while it does; both wait here for what is before them.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (P.next_early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = TILES ? sh->tmem : 0u;
    // CTAs below first_sms take tiles first and then streams, the others the
    // other way round; a CTA is in one of the two at a time.
    const bool tiles_first = TILES && (!STREAMS || (int)blockIdx.x < P.first_sms);
    auto between = [&] {  // what one part wrote to shared memory is next written by TMA
        fence_proxy_async_shared();
        tc_fence_before();
        bar_sync<1, kThreads>();
        tc_fence_after();
    };
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
        if (!tiles_first) between();
        Counts c;
        for (uint32_t n = 0; TILES; ++n) {
            const uint32_t slot = n % kItemSlots, phase = (n / kItemSlots) & 1u;
            if (warp == 8) {
                if (!wait_warp(P, bars + 8 * (kItemFree + slot), phase ^ 1u, sh, 100)) break;
                if ((threadIdx.x & 31) == 0) {
                    // (the first round needs no atomic: CTA b takes tile b)
                    int idx = tiles_first && n == 0 ? (int)blockIdx.x
                                                    : min(P.first_sms, P.n_first) + atomicAdd(&P.ws[kHead0], 1);
                    int4 a = make_int4(-1, 0, 0, 0), b = a;
                    if (idx < P.n_first) {
                        const int4* src = reinterpret_cast<const int4*>(P.plan + P.off_items + (size_t)idx * kItemWords);
                        a = src[0];
                        b = src[1];
                    }
                    reinterpret_cast<int4*>(sh->item[slot])[0] = a;
                    reinterpret_cast<int4*>(sh->item[slot])[1] = b;
                    mbar_arrive(bars + 8 * (kItemFull + slot));
                }
                __syncwarp();
            }
            if (!wait_warp(P, bars + 8 * (kItemFull + slot), phase, sh, 200)) break;
            const Tile T = tile_of<D>(P, sh->item[slot]);
            if (T.kind < 0) break;
            if (T.nb > 0) {
                if (warp == 8)
                    tile_loads<D>(P, &tmQ, &tmK, &tmV, &tmK5, &tmV5, T, c, smem, bars, sh);
                else if (warp == 9)
                    tile_scores<D, F16>(P, T, c, smem, bars, tmem, sh);
                else if (warp == 10)
                    tile_sums<D, F16>(P, T, c, smem, bars, tmem, sh);
                else if (T.fix)
                    tile_clean<D>(P, T, c, smem, bars, sh);
            }
            count_item(c, T);
            __syncwarp();
            if (warp >= 9 && (threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (kItemFree + slot));
        }
        if (tiles_first) between();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMainRegs));
        if (STREAMS && !tiles_first) {
            run_streams<D, F16>(P, &tmK3, &tmV3, smem, bars, sh, true);
        }
        if (!tiles_first) between();
        if (TILES) {
            Counts c;
            auto item = [&](uint32_t n) {
                const uint32_t slot = n % kItemSlots;
                Tile T;
                T.kind = -1;
                if (wait_warp(P, bars + 8 * (kItemFull + slot), (n / kItemSlots) & 1u, sh, 300))
                    T = tile_of<D>(P, sh->item[slot]);
                return T;
            };
            Tile T = item(0);
            TileRow R = row_of(P, T);
            for (uint32_t n = 0; T.kind >= 0; ++n) {
                Tile Tn;
                Tn.kind = -1;
                TileRow Rn;
                tile_softmax<D, F16, KIND>(P, T, R, c, smem, bars, tmem, sh, [&] {
                    Tn = item(n + 1);
                    Rn = row_of(P, Tn);
                });
                count_item(c, T);
                __syncwarp();
                if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (kItemFree + n % kItemSlots));
                T = Tn;
                R = Rn;
            }
        }
        if (tiles_first) {
            between();
            if (STREAMS) run_streams<D, F16>(P, &tmK3, &tmV3, smem, bars, sh, false);
        }
    }
    // (after a wait that ran out: let copies and products in flight end)
    if (*(volatile int*)&sh->abort) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 5000000ull) __nanosleep(10000);
    }
    tc_fence_before();
    bar_sync<1, kThreads>();
    tc_fence_after();
    if (TILES && warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    // the last CTA out leaves the counters at zero for the next launch
    if (tid == 0) {
        __threadfence();
        if (atomicAdd(&P.ws[kOut], 1) == (int)gridDim.x - 1) {
            P.ws[kHead0] = 0;
            P.ws[kHead1] = 0;
            P.ws[kOut] = 0;
        }
    }
}

// ---------------------------------------------------------------------------
// Joins a split token's partial rows: out = sum_k O_k 2^(m_k - M) / sum_k l_k
// 2^(m_k - M).  W warps take a (token, q head), warp w the pieces w, w + W, ...
// of the shared pages and of the token's own: W = 1 (four rows a block) for a
// few pieces a row, 4 for more, 16 for a long context's hundreds.  The launch
// overlaps the end of the first kernel and waits for it here.
// ---------------------------------------------------------------------------
template <int D, bool F16, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) paged_join_kernel(const __grid_constant__ Params P) {
    constexpr int N = D / 32, kRows = W == 1 ? 4 : 1;
    const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : (int)threadIdx.x >> 5;
    const int row = (int)blockIdx.x * kRows + (W == 1 ? (int)threadIdx.x >> 5 : 0);
    const bool mine = row < P.n_merge * P.Hq;
    const int h = row % P.Hq, hkv = h / P.group;
    if (P.next_early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int* rec = P.plan + P.off_merge + (size_t)(mine ? row / P.Hq : 0) * kMergeWords;
    const int4 ra = reinterpret_cast<const int4*>(rec)[0], rb = reinterpret_cast<const int4*>(rec)[1];
    const int t = ra.x, n0 = ra.y, n = mine ? n0 + rb.x : 0;
    const int row0 = ra.z + hkv * ra.w + h % P.group, step0 = P.Hkv * ra.w;
    const int row1 = rb.y + hkv * rb.z + h % P.group, step1 = P.Hkv * rb.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    constexpr int B = W == 16 ? 8 : 4;  // pieces loaded at once
    for (int k0 = warp; k0 < n; k0 += W * B) {
        float2 ml[B];
        float o[B][N];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int k = k0 + W * b;
            ml[b] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < N; ++i) o[b][i] = 0.f;
            if (k < n) {
                const size_t p = (size_t)(k < n0 ? row0 + k * step0 : row1 + (k - n0) * step1);
                ml[b] = __ldcg(P.part_ml + p);
                if (N == 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(P.part_o + p * D + lane * N));
                    o[b][0] = y.x; o[b][1] = y.y; o[b][N - 2] = y.z; o[b][N - 1] = y.w;
                } else {
                    const float2 y = __ldcg(reinterpret_cast<const float2*>(P.part_o + p * D + lane * N));
                    o[b][0] = y.x; o[b][1] = y.y;
                }
            }
        }
        float mn = m;
#pragma unroll
        for (int b = 0; b < B; ++b) mn = fmaxf(mn, ml[b].x);
        const float base = mn == -INFINITY ? 0.f : mn, fa = ex2(m - base);
        m = mn;
        l *= fa;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] *= fa;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float f = ex2(ml[b].x - base);
            l += ml[b].y * f;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += o[b][i] * f;
        }
    }
    if (W > 1) {
        __shared__ float s_m[W], s_l[W], s_o[W][D];
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s_o[warp][lane * N + i] = acc[i];
        __syncthreads();
        if (warp) return;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[w]);
        const float base = M == -INFINITY ? 0.f : M;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = ex2(s_m[w] - base);
            l += s_l[w] * f;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += s_o[w][lane * N + i] * f;
        }
        m = M;
    }
    if (!mine) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(P.out + ((size_t)t * P.Hq + h) * D + lane * N);
#pragma unroll
    for (int i = 0; i < N; i += 2) dst[i / 2] = pack2<F16>(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0 && P.lse) P.lse[(size_t)t * P.Hq + h] = lse_of(m, l);
}

namespace {

int32_t cuda_fail(cudaError_t e, const char* what);

// A launch; overlap: it may begin while the kernel before it on the stream ends,
// which the kernel itself waits for.
int32_t launch(const void* kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, void** params,
               bool overlap, const char* what) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, params);
    return e == cudaSuccess ? SARATHI_OK : cuda_fail(e, what);
}

constexpr int kJoinSome = 4, kJoinMany = 48;  // pieces a row above which 4 and 16 warps join it

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int32_t cuda_fail(cudaError_t e, const char* what) {
    char msg[256];
    std::snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return fail(SARATHI_ERR_CUDA, msg);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A tensor map of rank n over 16-bit elements with the 128-byte swizzle.
int32_t make_map(CUtensorMap* m, const void* base, bool f16, int n, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    auto enc = encode_fn();
    if (!enc) return fail(SARATHI_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const CUresult r =
        enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n, const_cast<void*>(base),
            dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char msg[128];
        std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (%d) for a map of rank %d", (int)r, n);
        return fail(SARATHI_ERR_CUDA, msg);
    }
    return SARATHI_OK;
}
// Views of a page pool [pages][H_kv][16][d]: {d, rows} with a box of one page's
// 64-column half; {64, rows, d/64} with a box of one page of a head; {64, slots,
// heads, pages, d/64} with a box of a block's consecutive pages of a head.
int32_t pool_map2(CUtensorMap* m, const void* base, bool f16, int64_t pages, int Hkv, int d) {
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)(pages * Hkv * kPage)}, strides[1] = {(cuuint64_t)d * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)kPage};
    return make_map(m, base, f16, 2, dims, strides, box);
}
int32_t pool_map3(CUtensorMap* m, const void* base, bool f16, int64_t pages, int Hkv, int d) {
    const cuuint64_t dims[3] = {64, (cuuint64_t)(pages * Hkv * kPage), (cuuint64_t)(d / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)kPage, (cuuint32_t)(d / 64)};
    return make_map(m, base, f16, 3, dims, strides, box);
}
int32_t pool_map5(CUtensorMap* m, const void* base, bool f16, int64_t pages, int Hkv, int d) {
    const cuuint64_t dims[5] = {64, (cuuint64_t)kPage, (cuuint64_t)Hkv, (cuuint64_t)pages, (cuuint64_t)(d / 64)};
    const cuuint64_t strides[4] = {(cuuint64_t)d * 2, (cuuint64_t)kPage * d * 2, (cuuint64_t)Hkv * kPage * d * 2, 128};
    const cuuint32_t box[5] = {64, (cuuint32_t)kPage, 1, (cuuint32_t)(block_keys(d) / kPage), (cuuint32_t)(d / 64)};
    return make_map(m, base, f16, 5, dims, strides, box);
}
// The queries {d, H_q, T}, a box of one tile's rows (token-major), 64 columns.
int32_t query_map(CUtensorMap* m, const void* q, bool f16, int T, int Hq, int G, int d, int64_t stride) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hq, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTileRows / G)};
    return make_map(m, q, f16, 3, dims, strides, box);
}

struct Kernels {
    const void* attn[3];  // tiles, streams, both
    const void* join[3];  // 1, 4 and 16 warps a row
    int smem, id;         // id: of these, in 0 .. 11
};
template <int D, bool F16, int KIND>
Kernels kernels() {
    return Kernels{{(const void*)paged_attn_kernel<D, F16, KIND, true, false>,
                    (const void*)paged_attn_kernel<D, F16, kAny, false, true>,
                    (const void*)paged_attn_kernel<D, F16, KIND, true, true>},
                   {(const void*)paged_join_kernel<D, F16, 1>, (const void*)paged_join_kernel<D, F16, 4>,
                    (const void*)paged_join_kernel<D, F16, 16>},
                   Layout<D>::kAlloc,
                   3 * ((D == 128 ? 2 : 0) + (F16 ? 1 : 0)) + KIND};
}
template <bool F16>
Kernels kernels_for(int d, bool capped, bool biased) {
    if (d == 128) return biased && !capped ? kernels<128, F16, kBiased>() : kernels<128, F16, kAny>();
    if (capped) return kernels<64, F16, kAny>();
    return biased ? kernels<64, F16, kBiased>() : kernels<64, F16, kPlain>();
}

// The device's SM count, once the kernel is known to run there: its shared
// memory granted, one block fitting an SM, and launched with the registers that
// its split hands out (a smaller launch would leave setmaxnreg waiting).
int32_t ready(const void* attn, int smem, int which, int* sms) {
    static std::mutex mu;
    static int sm_count[128] = {};
    static bool done[128][36] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 128) return fail(SARATHI_ERR_UNSUPPORTED, "device index >= 128");
    std::lock_guard<std::mutex> lk(mu);
    if (!done[dev][which]) {
        e = cudaDeviceGetAttribute(&sm_count[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, attn);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
        if (fa.numRegs < kLaunchRegs)
            return fail(SARATHI_ERR_CUDA, "paged_attn_kernel built with fewer registers than it shares out");
        e = cudaFuncSetAttribute(attn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        int resident = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, attn, kThreads, smem);
        if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
        if (resident < 1) return fail(SARATHI_ERR_CUDA, "paged_attn_kernel does not fit one SM");
        done[dev][which] = true;
    }
    *sms = sm_count[dev];
    return SARATHI_OK;
}

}  // namespace
}  // namespace paged
}  // namespace sarathi

using namespace sarathi;

extern "C" int32_t sarathi_paged_attn(const sarathi_paged_args* a, void* cuda_stream) {
    using namespace paged;
    if (!a) return fail(SARATHI_ERR_INVALID_ARG, "args is NULL");
    int32_t st = check_shape(&a->shape);
    if (st) return st;
    const sarathi_paged_info* in = a->info;
    if (!in) return fail(SARATHI_ERR_INVALID_ARG, "info is NULL");
    const int Hq = a->shape.num_heads_q, Hkv = a->shape.num_heads_kv, d = a->shape.head_dim;
    if (in->shape.num_heads_q != Hq || in->shape.num_heads_kv != Hkv || in->shape.head_dim != d)
        return fail(SARATHI_ERR_INVALID_ARG, "the plan was made for another shape");
    if (a->dtype != SARATHI_BF16 && a->dtype != SARATHI_FP16) return fail(SARATHI_ERR_UNSUPPORTED, "unknown dtype");
    if (!(a->sm_scale > 0.f) || !std::isfinite(a->sm_scale))
        return fail(SARATHI_ERR_INVALID_ARG, "sm_scale must be positive and finite");
    if (!(a->score_cap >= 0.f) || !std::isfinite(a->score_cap))
        return fail(SARATHI_ERR_INVALID_ARG, "score_cap must be 0 or positive and finite");
    const double log2e = 1.4426950408889634;
    const float raw_scale = a->score_cap > 0.f ? a->sm_scale / a->score_cap : (float)(a->sm_scale * log2e);
    const float cap2 = (float)(a->score_cap * log2e);
    if (!std::isnormal(raw_scale) || (a->score_cap > 0.f && !std::isnormal(cap2)))
        return fail(SARATHI_ERR_INVALID_ARG, "sm_scale and score_cap leave the range of fp32");
    if (a->num_pages <= 0) return fail(SARATHI_ERR_INVALID_ARG, "num_pages must be positive");
    if (in->num_tokens < 0 || in->n_items < 0 || in->n_merge < 0 || in->n_partials < 0 || in->packed_ints < 0)
        return fail(SARATHI_ERR_INVALID_ARG, "inconsistent plan info");
    if (in->num_tokens == 0) return SARATHI_OK;
    if (!a->q || !a->k_cache || !a->v_cache || !a->out || !a->plan || !a->workspace)
        return fail(SARATHI_ERR_INVALID_ARG, "NULL device pointer");
    if (!aligned(a->q, 16) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->out, 16) ||
        !aligned(a->plan, 16) || !aligned(a->lse, 4) || !aligned(a->slopes, 4) || !aligned(a->workspace, 256))
        return fail(SARATHI_ERR_INVALID_ARG, "misaligned pointer (tensors 16 B, workspace 256 B)");
    if (a->q_stride < (int64_t)Hq * d || (a->q_stride & 7))
        return fail(SARATHI_ERR_INVALID_ARG, "q_stride is shorter than a token's heads or no multiple of 8");
    const auto q0 = reinterpret_cast<uintptr_t>(a->q), o0 = reinterpret_cast<uintptr_t>(a->out);
    const uint64_t q_bytes = ((uint64_t)(in->num_tokens - 1) * a->q_stride + (uint64_t)Hq * d) * 2;
    if (q0 < o0 + (uint64_t)in->num_tokens * Hq * d * 2 && o0 < q0 + q_bytes)
        return fail(SARATHI_ERR_INVALID_ARG, "out overlaps q");
    if (a->workspace_bytes < in->workspace_bytes) return fail(SARATHI_ERR_CAPACITY, "workspace too small");
    if ((int64_t)a->num_pages * Hkv * kPage >= (int64_t)1 << 31)
        return fail(SARATHI_ERR_UNSUPPORTED, "page pool too large for 32-bit row coordinates");
    if (in->n_first < 0 || in->n_first > in->n_items || in->first_sms < 0 || (in->off_items & 3) ||
        (in->off_tokens & 3) || in->workspace_bytes < workspace_size(in->n_partials, d))
        return fail(SARATHI_ERR_INVALID_ARG, "inconsistent plan info");
    const bool f16 = a->dtype == SARATHI_FP16;
    const Kernels kern = f16 ? kernels_for<true>(d, a->score_cap > 0.f, a->slopes)
                             : kernels_for<false>(d, a->score_cap > 0.f, a->slopes);
    int sms = 0;
    const int kind = in->n_first == in->n_items ? 0 : in->n_first == 0 ? 1 : 2;
    st = ready(kern.attn[kind], kern.smem, 3 * kern.id + kind, &sms);
    if (st) return st;
    Params P;
    P.q = static_cast<const uint16_t*>(a->q);
    P.k_cache = static_cast<const uint16_t*>(a->k_cache);
    P.v_cache = static_cast<const uint16_t*>(a->v_cache);
    P.out = static_cast<uint16_t*>(a->out);
    P.lse = a->lse;
    P.slopes = a->slopes;
    P.q_stride = a->q_stride;
    P.plan = a->plan;
    P.off_pages = in->off_pages;
    P.off_tokens = in->off_tokens;
    P.off_items = in->off_items;
    P.off_merge = in->off_merge;
    P.n_items = in->n_items;
    P.n_first = in->n_first;
    P.n_merge = in->n_merge;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.group = Hq / Hkv;
    P.num_pages = a->num_pages;
    P.raw_scale = raw_scale;
    P.cap2 = cap2;
    P.cap_fine = a->score_cap > kCapFine;
    P.ws = static_cast<int32_t*>(a->workspace);
    P.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a->workspace) + ml_offset());
    P.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + o_offset(in->n_partials));
    cudaStream_t stream = (cudaStream_t)cuda_stream;
    // (two threads' calls on one stream: a join follows its own partial rows)
    static std::mutex pair;
    std::lock_guard<std::mutex> lk(pair);
    if (in->n_items > 0) {
        const int n_second = in->n_items - in->n_first;
        const int grid = std::min(sms, in->n_items);
        P.first_sms = kind == 0 ? grid : kind == 1 ? 0 : std::min(in->first_sms, grid - 1);
        // the views that the plan's items use
        CUtensorMap tmQ = {}, tmK = {}, tmV = {}, tmK3 = {}, tmV3 = {}, tmK5 = {}, tmV5 = {};
        if (in->n_first > 0) {
            st = query_map(&tmQ, a->q, f16, in->num_tokens, Hq, Hq / Hkv, d, a->q_stride);
            if (!st) st = pool_map2(&tmK, a->k_cache, f16, a->num_pages, Hkv, d);
            if (!st) st = pool_map2(&tmV, a->v_cache, f16, a->num_pages, Hkv, d);
            if (!st) st = pool_map5(&tmK5, a->k_cache, f16, a->num_pages, Hkv, d);
            if (!st) st = pool_map5(&tmV5, a->v_cache, f16, a->num_pages, Hkv, d);
        }
        if (!st && n_second > 0) {
            st = d == 128 ? pool_map3(&tmK3, a->k_cache, f16, a->num_pages, Hkv, d)
                          : pool_map2(&tmK3, a->k_cache, f16, a->num_pages, Hkv, d);
            if (!st)
                st = d == 128 ? pool_map3(&tmV3, a->v_cache, f16, a->num_pages, Hkv, d)
                              : pool_map2(&tmV3, a->v_cache, f16, a->num_pages, Hkv, d);
        }
        if (st) return st;
        void* params[] = {&P, &tmQ, &tmK, &tmV, &tmK3, &tmV3, &tmK5, &tmV5};
        // An early start saves 2 us of launch and prologue.  It also hands out the SMs
        // in the order in which they come free, and where tiles and streams fill all
        // of them that order matters: 192 requests behind 2000-key prefixes take 50
        // us when the kernel before lets them begin at its end, 58 when it does sooner.
        const bool sooner = kind != 2 || in->n_items <= sms;
        P.next_early = sooner || in->n_merge > 0;
        st = launch(kern.attn[kind], (unsigned)grid, (unsigned)kThreads, (size_t)kern.smem, stream, params, true,
                    "paged_attn_kernel launch");
        P.next_early = sooner;
        if (st) return st;
    }
    if (in->n_merge > 0) {
        const int64_t rows = (int64_t)in->n_merge * Hq;
        const int wide = in->n_partials > kJoinMany * rows ? 2 : in->n_partials > kJoinSome * rows ? 1 : 0;
        if (in->n_items == 0) P.next_early = 1;
        void* params[] = {&P};
        st = launch(kern.join[wide], (unsigned)(wide ? rows : (rows + 3) / 4), wide == 2 ? 512 : 128, 0, stream, params,
                    in->n_items > 0, "paged_join_kernel launch");
        if (st) return st;
    }
    return SARATHI_OK;
}
