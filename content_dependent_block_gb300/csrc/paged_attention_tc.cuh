// New tokens over the paged cache, many query rows at a time, on the tensor
// cores: prompts in chunks, trees of drafted tokens, many heads to a cache head
// (the mathematics is in paged_attention.cuh).
//
// A tile is 128 query rows: the G heads that share a cache head, times 128 / G
// tokens of one sequence.  K and V arrive in tiles of 128 keys, page by page
// (TMA straight from the 16-bit pages; from 8-bit pages the codes come by
// asynchronous copies and four warps turn them into fp16, which is exact).  A
// CTA runs two streams of
//   S = Q K^T (M 128, N 128, into tensor memory), softmax by one thread per
//   row, P, O += P V (N = d, in tensor memory),
// and the scores of a step are issued as soon as those of the one before are
// read, so that the softmax finds the next ones waiting:
//   pair  two tiles of rows over the same keys (K and V loaded once for 256 rows);
//   dual  one tile of rows, the streams taking key tiles in turn.
// The keys of either may be dealt to a cluster of CTAs; the states of the
// streams of a row, and of the cluster, are merged through shared memory.
// At d 128 tensor memory is full (two S, two O) and P lies in shared memory; at
// d 64 it lies in tensor memory.  The running maximum of a row follows only when
// it has grown by 2^8 (any shift gives the same softmax; weights stay below 2^8),
// so O is seldom rescaled.  Masks are bit sets of 32 keys, built only where a
// tile is not seen whole.  P is one bf16 number (off by 2^-8 at most, as in the
// prompt's sparse forward): with its remainder as a second one, as few rows
// take it (paged_tiles.cuh), the products with V would double, and at d 128 there
// is no room for it (at d 64 there is; not tried).  8-bit pages: P in fp16, as there.
//
// Measured: 3 prompts of 8191 tokens in all, 32 heads over 8, d 128, a window of 4096:
// 402 to 431 us on several cards, 1.28 to 1.37 PFLOP/s (67 to 71 % of cuBLAS's
// burst), over 8-bit pages 1290 us; 16 trees of 64 tokens behind 4096 to 32768
// keys, the same heads: 292 to 341 us against 184 us of traffic, over 8-bit pages
// 668 against 161; 24 trees of 13 tokens, 24 heads over 4, d 64, over 8-bit pages:
// 208 to 222 us against 36.  A step of a pair took about 3000 cycles with both
// streams in step: the softmax (loads 200, maximum 480, exponentials and P 2000, waits
// 400), and the products, which at d 128 read 128 bytes a cycle of shared
// memory for 2500.
//
//   warps 0-3, 4-7   softmax of streams 0 and 1
//   warps 8, 9       MMA of streams 0 and 1, each issued by one thread (in dual one
//                    thread issues both; in pair it would wait where it could issue)
//   warps 10, 11     producers: of K and of V, page by page into the ring (16-bit
//                    pages); codes and scales into a ring of their own (8-bit)
//   warps 12-15      8-bit pages: codes to fp16, into the ring
#pragma once

#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include "bsa_device.cuh"
#include "bsa_internal.h"
#include "paged_common.cuh"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace bsa {
namespace {

constexpr int kRows = 128;               // rows of a stream
constexpr int kKeys = 128;               // keys of a tile
constexpr int kNotes = 16;               // tiles whose notes are kept: more than the ring holds
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kMinusInf = -__builtin_huge_valf();
constexpr float kLazy = 8.f;             // growth of a row's maximum that is let pass, log2
constexpr int kWeightShift = 6;          // 8-bit pages: weights times 2^(6 - E), below 2^(8 + 1 + 6)

template <int D, bool kPair, bool Q8>
struct TCfg {
    static constexpr int kSub = D / 64;
    static constexpr int kPanel = kKeys * 128;              // 128 rows x 64 channels
    static constexpr int kStage = kSub * kPanel;            // K or V of a tile, or a stream's Q
    static constexpr int kStages = D == 64 ? (Q8 ? 4 : 7) : Q8 ? 2 : kPair ? 3 : 4;
    static constexpr int kRaw = !Q8 ? 0 : D == 64 ? 5 : 3;  // 8-bit pages: tiles of codes on their way
    static constexpr int kRawStage = kKeys * D + 2 * kKeys * 4;     // codes, and with K the scales of both
    static constexpr bool kPShared = D == 128;              // P in shared memory, else in tensor memory
    static constexpr int kPBytes = 2 * kPanel;              // 128 rows x 128 keys
    static constexpr int kQTiles = kPair ? 2 : 1;
    static constexpr int kSoft = 8;                         // softmax warps
    static constexpr int kWarps = kSoft + (Q8 ? 8 : 4);
    static constexpr int oQ = 0;
    static constexpr int oP = oQ + kQTiles * kStage;
    static constexpr int oRing = oP + (kPShared ? 2 * kPBytes : 0);
    static constexpr int oRaw = oRing + kStages * kStage;
    static constexpr int oNotes = oRaw + kRaw * kRawStage;  // uint32 [kNotes]: which 16-key groups are there
    static constexpr int oTops = oNotes + kNotes * 4;       // uint32 [kNotes][4]: largest vs (bits) of a quarter's keys
    static constexpr int oScales = oTops + (Q8 ? kNotes * 16 : 0);   // float [8][2][128]
    static constexpr int oBar = oScales + (Q8 ? 8 * 2 * kKeys * 4 : 0);
    static constexpr int oStat = oQ;                        // float2 [2][128], for the merge
    enum { bQ = 0, bTail, bGo, bFull, bEmpty = bFull + kStages, bRawFull = bEmpty + kStages, bRawEmpty = bRawFull + kRaw,
           bS = bRawEmpty + kRaw, bSFree = bS + 2, bP = bSFree + 2, bPv = bP + 2, bCount = bPv + 2 };
    static constexpr int oMisc = oBar + bCount * 8;
    static constexpr int kTotal = oMisc + 16 + 1024;
    static constexpr uint32_t cS = 0, cO = 2 * kKeys, cP = cO + 2 * D;      // columns of tensor memory
    static constexpr int kOStride = D + 4;                  // floats of a row of the merge
};
static_assert(TCfg<128, true, false>::kTotal <= 227 * 1024 && TCfg<128, false, false>::kTotal <= 227 * 1024 &&
                  TCfg<128, false, true>::kTotal <= 227 * 1024 && TCfg<64, true, false>::kTotal <= 227 * 1024 &&
                  TCfg<64, false, false>::kTotal <= 227 * 1024 && TCfg<64, true, true>::kTotal <= 227 * 1024 &&
                  TCfg<64, false, true>::kTotal <= 227 * 1024,
              "shared memory");
template <int D, bool kPair, bool Q8>
constexpr bool merge_fits() {
    using C = TCfg<D, kPair, Q8>;
    return 2 * kRows * C::kOStride * 4 <= C::oNotes - C::oP && 2 * kRows * 8 <= C::kStage;
}
static_assert(merge_fits<64, false, false>() && merge_fits<64, false, true>() && merge_fits<128, false, false>() &&
                  merge_fits<128, false, true>() && merge_fits<64, true, false>() && merge_fits<64, true, true>() &&
                  merge_fits<128, true, false>(),
              "the merge uses P and the rings");
static_assert(TCfg<128, true, false>::cO + 256 <= 512 && TCfg<64, true, false>::cP + 128 <= 512, "tensor memory");

struct TilesPlan {
    int64_t items_each;
    int32_t cluster;
    int32_t tokens;           // of a stream's tile: 128 / G, or as many as a sequence has
    int32_t size;             // of a CTA's
};

__device__ __forceinline__ float exp2_ftz(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two numbers at a time.
__device__ __forceinline__ uint64_t as_pair(float2 x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
    return r;
}
__device__ __forceinline__ float2 of_pair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_pair(x)), "l"(as_pair(y)), "l"(as_pair(z)));
    return of_pair(r);
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_pair(x)), "l"(as_pair(y)));
    return of_pair(r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_pair(x)), "l"(as_pair(y)));
    return of_pair(r);
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Bits [lo, hi) of a word, the bounds clamped to [0, 32].
__device__ __forceinline__ uint32_t bits_from_to(int lo, int hi) {
    const int l = min(max(lo, 0), 32), h = min(max(hi, 0), 32);
    if (l >= h) return 0u;
    return (kAll >> (32 - h)) & (kAll << l);
}

// Which of the 32 keys from j on a row sees.
__device__ __forceinline__ uint32_t seen_bits(const Sight &s, int32_t start, int32_t sinks, int32_t j) {
    uint32_t m = bits_from_to(s.lo - j, s.hi - j) | bits_from_to(-j, min(sinks, s.hi) - j);
    const int64_t off = int64_t(j) - start;
    if (s.tree != 0 && off > -32 && off < 64)
        m |= uint32_t(off >= 0 ? s.tree >> off : s.tree << -off);
    return m;
}

// The tiles of keys that a CTA takes, of those that some of its rows see.
struct KeyTiles {
    int sinks, gap, first, count;
    __device__ __forceinline__ KeyTiles(const Reach &r, int rank, int cluster) {
        sinks = min((r.sinks_end + kKeys - 1) / kKeys, r.first / kKeys);
        gap = r.first / kKeys - sinks;
        const int all = (r.end + kKeys - 1) / kKeys - gap;
        const int each = (all + cluster - 1) / cluster;
        first = min(all, rank * each);
        count = min(all, first + each) - first;
    }
    __device__ __forceinline__ int32_t key0(int i) const {
        const int u = first + i;
        return (u < sinks ? u : u + gap) * kKeys;
    }
};

// A tile's `i`-th page: whether some row sees any of it, and if so its entry in
// the table (0 where not, without a look).
__device__ __forceinline__ bool page_seen(const AttentionArgs &a, const Reach &r, int32_t key0, int i) {
    const int32_t k0 = key0 + i * a.c.page;
    return i * a.c.page < kKeys && k0 < r.end && (k0 < r.sinks_end || k0 + a.c.page > r.first);
}
__device__ __forceinline__ int32_t page_entry(const AttentionArgs &a, const Reach &r, int32_t key0, int i) {
    return page_seen(a, r, key0, i) ? __ldg(a.table + r.seq * a.width + (key0 / a.c.page + i)) : 0;
}

// The page of an entry: -1 where no row sees it, -2 where it is not in the cache.
__device__ __forceinline__ int32_t page_checked(const AttentionArgs &a, bool seen, int32_t entry) {
    if (!seen) return -1;
    if (entry >= 0 && entry < a.c.num_pages) return entry;
    report_status(a.status, kStatusBadIndex);
    return -2;
}

// A row by itself, by one warp: every key it sees, online in fp32; out[e] =
// channel lane * D / 32 + e.  For rows whose tile's products met a masked value
// that is not finite.
template <int D>
__device__ __noinline__ void row_alone(const AttentionArgs &a, const Reach &r, const Sight &s, int head,
                                       const uint16_t *q_row, float (&out)[D / 32]) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float q[E], m = kMinusInf, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float(uint32_t(q_row[lane * E + e]) << 16);
        out[e] = 0.f;
    }
    for (int32_t j = 0; j < r.end; j += 32) {
        if (j >= r.sinks_end && j + 32 <= r.first) {
            j = r.first / 32 * 32 - 32;
            continue;
        }
        for (uint32_t left = seen_bits(s, int32_t(r.start), a.window > 0 ? a.sinks : 0, j); left != 0;
             left &= left - 1) {
            const int32_t key = j + __ffs(left) - 1;
            const int32_t pid = a.table[r.seq * a.width + key / a.c.page];
            if (pid < 0 || pid >= a.c.num_pages) continue;
            const int64_t at = ((int64_t(pid) * a.c.heads + head) * a.c.page + key % a.c.page) * D + lane * E;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(q[e], __uint_as_float(uint32_t(a.c.k[at + e]) << 16), x);
            x = warp_sum(x) * a.scale_log2;
            const float mn = fmaxf(m, x), base = mn == kMinusInf ? 0.f : mn;
            const float corr = exp2_ftz(m - base), p = exp2_ftz(x - base);
            m = mn;
            l = fmaf(l, corr, p);
#pragma unroll
            for (int e = 0; e < E; ++e)
                out[e] = fmaf(p, __uint_as_float(uint32_t(a.c.v[at + e]) << 16), out[e] * corr);
        }
    }
    const float inv = l > 0.f || l != l ? __fdiv_rn(1.f, l) : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] *= inv;
}

// Sixteen codes of a key, as fp16, to their two chunks of a swizzled row.
__device__ __forceinline__ void store_codes(uint8_t *row, int chunk, int r, const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = w[i] ^ 0x80808080u;              // a byte plus 128: the low byte of 1024 + it
        const uint32_t lo = __byte_perm(b, 0x64646464u, 0x4140), hi = __byte_perm(b, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * i]) : "r"(lo), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * i + 1]) : "r"(hi), "r"(0x64806480u));
    }
    *reinterpret_cast<uint4 *>(row + ((chunk ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(row + (((chunk + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// The largest |scale| (bits) of those of 32 keys whose bits are set.  A call: in
// line it takes registers from every step at d 128 (3 prompts over 8-bit pages
// 1356 us, so 1290; 1251 with the largest of the whole tile, which is wrong where
// it is that of a key which the row does not see).
__device__ __noinline__ uint32_t largest_scale(const float4 *scales, uint32_t keys) {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 v4 = scales[j];
        const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (((keys >> (4 * j + k)) & 1u) && fabsf(v[k]) < -kMinusInf) top = max(top, __float_as_uint(fabsf(v[k])));
    }
    return top;
}

template <int D, bool kPair, bool Q8>
__global__ void __launch_bounds__(TCfg<D, kPair, Q8>::kWarps * 32, 1)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const AttentionArgs a, const TilesPlan p) {
    using C = TCfg<D, kPair, Q8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = tc::align_smem_1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::oBar);
    uint32_t *notes = reinterpret_cast<uint32_t *>(sm + C::oNotes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::oMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = int(blockIdx.x % unsigned(p.cluster));
    const unsigned cluster = blockIdx.x / unsigned(p.cluster);
    const int64_t number = cluster / unsigned(a.c.heads);
    const int head = int(cluster - unsigned(number) * unsigned(a.c.heads));
    const int group = a.q_heads / a.c.heads;
    int32_t *status = a.status;
    check_bounds(a.cu, a.seqs, a.tokens, int64_t(blockIdx.x) * (C::kWarps * 32) + tid, status);
    Reach r;
    // the whole cluster leaves together
    if (!find_reach(a, p.size, p.items_each, number, rank == 0 && tid == 0, &r)) return;
    const int32_t sinks = a.window > 0 ? a.sinks : 0;
    const KeyTiles tiles(r, rank, p.cluster);
    const int n = tiles.count;
    // rows and key tiles of a stream; key tile of its t-th step
    const auto rows_of = [&](int s) {
        return kPair ? max(0, min(p.tokens, r.nt - s * p.tokens)) * group : r.nt * group;
    };
    const auto steps_of = [&](int s) { return kPair ? (rows_of(s) > 0 ? n : 0) : (n + 1 - s) / 2; };
    const auto tile_of = [&](int s, int t) { return kPair ? t : 2 * t + s; };
    const bool merges = !kPair || p.cluster > 1;            // of states: of both streams, or of the cluster

    if (tid == 0) {
        tc::mbar_init(bars + C::bQ, 32 * C::kSoft);
        tc::mbar_init(bars + C::bTail, 1);
        tc::mbar_init(bars + C::bGo, kRows);
        const uint32_t users = kPair && rows_of(1) > 0 ? 2 : 1;
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(bars + C::bFull + i, Q8 ? 128 : 1);
            tc::mbar_init(bars + C::bEmpty + i, users);
        }
        for (int i = 0; i < C::kRaw; ++i) {
            tc::mbar_init(bars + C::bRawFull + i, 33);      // a lane's copies each, and the tile's note
            tc::mbar_init(bars + C::bRawEmpty + i, 128);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(bars + C::bS + s, 1);
            tc::mbar_init(bars + C::bSFree + s, kRows);
            tc::mbar_init(bars + C::bP + s, kRows);
            tc::mbar_init(bars + C::bPv + s, 1);
        }
        tc::fence_barrier_init();
        if (!Q8) {
            tc::prefetch_tensormap(&tm_k);
            tc::prefetch_tensormap(&tm_v);
        }
    }
    if (warp == C::kSoft) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const auto token_row = [&](int s, int row, int64_t stride) {
        const int t = row / group;
        return (r.lo + r.t0 + (kPair ? s * p.tokens : 0) + t) * stride + int64_t(head * group + row - t * group) * D;
    };
    const auto sight_at = [&](int s, int row) {
        return sight_of(a, r.start, r.lo, r.n, min(r.n - 1, r.t0 + (kPair ? s * p.tokens : 0) + row / group));
    };

    // The order in which K and V tiles are loaded and used: a stream's scores of
    // the next step come before the products of this one, and in dual the
    // streams take turns.
    constexpr int kAhead = kPair ? 1 : 2;                   // tiles of a step
    // for the thread that issues products, with as little as possible between them
    const auto schedule = [](int count, const auto &use) {
        int q = 0;
        for (int i = 0; i < min(kAhead, count); ++i)
            if (!use(false, i, q++)) return;
        for (int i = 0; i < count; ++i) {
            if (i + kAhead < count && !use(false, i + kAhead, q++)) return;
            if (!use(true, i, q++)) return;
        }
    };
    // the same for larger bodies, which it has once (24 trees over 8-bit pages:
    // 342 us with three copies, 267 us)
    const auto schedule_once = [](int count, const auto &use) {
        const int lead = min(kAhead, count), both = 2 * (count - lead);
        for (int q = 0; q < 2 * count; ++q) {
            const int j = q - lead;
            const bool v = j >= both || (j >= 0 && (j & 1) != 0);
            const int i = j < 0 ? q : j >= both ? count - lead + j - both : v ? j / 2 : lead + j / 2;
            if (!use(v, i, q)) return;
        }
    };

    if (warp < C::kSoft) {
        // ---------------------------------------------------- softmax of stream s
        const int s = warp >> 2, row = tid & 127;
        const int rows = rows_of(s), steps = steps_of(s);
        const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + C::cS + uint32_t(s * kKeys) + lane_off, tO = tmem + C::cO + uint32_t(s * D) + lane_off;
        float back = a.scale_log2;                          // times a row's raw scores
        {
            // Q into shared memory, swizzled, by the threads of its rows (in dual of both streams)
            const bool there = row < rows;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + token_row(s, there ? row : 0, a.q_stride));
            uint8_t *dst = sm + C::oQ + (kPair ? s * C::kStage : 0) + row * 128;
            float to = 1.f;
            if (Q8) {
                uint32_t top = 0u;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = there ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                 __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                }
                // the power of two that brings the largest |q| to [2^14, 2^15), as in paged_tiles.cuh
                const int e = min(max(int(max(top & 0xffffu, top >> 16) >> 7), 15), 254) - 127;
                back *= exp2_int(e - 14);
                to = exp2_int(14 - e);
            }
            constexpr int kMine = D / 8 / (kPair ? 1 : 2);
            const int c0 = kPair ? 0 : s * kMine;
#pragma unroll 4
            for (int c = c0; c < c0 + kMine; ++c) {
                uint4 x = there ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
                if (Q8) {
                    x.x = pack_f16x2(bf16_low_half(x.x) * to, bf16_high_half(x.x) * to);
                    x.y = pack_f16x2(bf16_low_half(x.y) * to, bf16_high_half(x.y) * to);
                    x.z = pack_f16x2(bf16_low_half(x.z) * to, bf16_high_half(x.z) * to);
                    x.w = pack_f16x2(bf16_low_half(x.w) * to, bf16_high_half(x.w) * to);
                }
                *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kPanel + (((c & 7) ^ (row & 7)) << 4)) = x;
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bars + C::bQ);
        }
        const Sight sight = sight_at(s, max(0, min(row, rows - 1)));
        const bool active = (warp & 3) * 32 < rows;         // any row in this warp
        const int32_t lo_max = __reduce_max_sync(kAll, sight.lo), hi_min = __reduce_min_sync(kAll, sight.hi);
        float m = kMinusInf, l = 0.f;
        int big = -110;                                     // E of the row's weights (8-bit pages)
        bool ok = true;
        for (int t = 0; t < steps; ++t) {
            const int i = tile_of(s, t);
            const int32_t key0 = tiles.key0(i);
            // a wait that ran out is on record, and the ones behind it end at
            // once: the steps go on, so that the barriers below stay paired
            ok &= tc::mbar_wait(bars + C::bS + s, t & 1, status);
            tc::tc_fence_after();
            if (kPair && s == 0 && t == 0) tc::mbar_arrive(bars + C::bGo);
            if (active) {
                const uint32_t there = notes[i % kNotes];
                const bool full = key0 >= lo_max && key0 + kKeys <= hi_min && there == 0xffu;
                const float4 *ks = reinterpret_cast<const float4 *>(sm + C::oScales) + (i % 8) * 64;
                const float4 *vs = ks + 32;
                const auto admitted = [&](int c) {
                    const uint32_t g = there >> (2 * c);
                    return seen_bits(sight, int32_t(r.start), sinks, key0 + c * 32) &
                           ((g & 1u ? 0xffffu : 0u) | (g & 2u ? 0xffff0000u : 0u));
                };
                const auto mask = [&](uint32_t adm, float *x) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!((adm >> j) & 1u)) x[j] = kMinusInf;
                };
                const float2 back2 = make_float2(back, back);
                // 8-bit pages: scores of 32 keys in log2 units
                const auto scores8 = [&](int c, float *x) {
                    uint32_t raw[32];
                    tc::tmem_ld32(tS + uint32_t(c * 32), raw);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 k4 = ks[c * 8 + j / 4];
                        const float2 y0 = mul2(make_float2(__uint_as_float(raw[j]), __uint_as_float(raw[j + 1])),
                                               mul2(make_float2(k4.x, k4.y), back2));
                        const float2 y1 = mul2(make_float2(__uint_as_float(raw[j + 2]), __uint_as_float(raw[j + 3])),
                                               mul2(make_float2(k4.z, k4.w), back2));
                        x[j] = y0.x;
                        x[j + 1] = y0.y;
                        x[j + 2] = y1.x;
                        x[j + 3] = y1.y;
                    }
                };
                float mx[4] = {kMinusInf, kMinusInf, kMinusInf, kMinusInf};
                const auto largest = [&](const float *x) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[j + e], x[j + 4 + e]);
                };
                // 16-bit pages: the scores are held from the maximum to the
                // weights; 8-bit pages read them with their scales, find the
                // maximum on the way and start again where it had grown
                float x[Q8 ? 32 : kKeys];
                if constexpr (!Q8) {
                    uint32_t raw[kKeys / 32][32];
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) tc::tmem_ld32(tS + uint32_t(c * 32), raw[c]);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < kKeys; ++j) x[j] = __uint_as_float(raw[j / 32][j % 32]);
                    tc::tc_fence_before();
                    tc::mbar_arrive(bars + C::bSFree + s);  // the next scores may come
                    if (!full)
#pragma unroll
                        for (int c = 0; c < kKeys / 32; ++c) mask(admitted(c), x + c * 32);
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) largest(x + c * 32);
                }
                // The row's maximum, once it has grown enough.
                float corr = 1.f, base;
                const auto follow = [&] {
                    float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                    if (!Q8) top *= back;
                    const bool grown = top > m + kLazy || (m == kMinusInf && top > kMinusInf);
                    if (grown) {
                        const float c = exp2_ftz(m - top);
                        corr *= c;
                        l *= c;
                        m = top;
                    }
                    base = m == kMinusInf ? 0.f : m;
                    return grown;
                };
                float vf = 1.f;
                if (Q8) {
                    const uint4 tops = *reinterpret_cast<const uint4 *>(sm + C::oTops + (i % kNotes) * 16);
                    int e = int(max(max(tops.x, tops.y), max(tops.z, tops.w)) >> 23) - 127;
                    if (e > big && !full) {
                        // the largest scale may be that of a key which this row
                        // does not see: the largest of those that it does
                        uint32_t own = 0u;
#pragma unroll 1
                        for (int c = 0; c < kKeys / 32; ++c) {
                            const uint32_t adm = admitted(c);
                            const uint32_t all = reinterpret_cast<const uint32_t *>(sm + C::oTops)[(i % kNotes) * 4 + c];
                            own = max(own, adm == kAll ? all : adm != 0u ? largest_scale(vs + c * 8, adm) : 0u);
                        }
                        e = int(own >> 23) - 127;
                    }
                    if (e > big) {
                        corr = exp2_int(max(big - e, -126));
                        big = e;
                    }
                    vf = exp2_int(kWeightShift - big);
                }
                follow();                                   // (8-bit pages: nothing yet, the base as it is)
                // O and P are this step's once the product of the last is done
                const auto rescale = [&] {
                    if (t == 0 || !__any_sync(kAll, corr != 1.f)) return;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16(tO + uint32_t(c), o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
                        tc::tmem_st16(tO + uint32_t(c), o);
                    }
                };
                const auto settle = [&] {
                    if (t > 0) ok &= tc::mbar_wait(bars + C::bPv + s, (t - 1) & 1, status);
                    tc::tc_fence_after();
                };
                const float2 f2 = make_float2(vf, vf);
                float2 ls[2];
                uint32_t pk[32];                            // weights of 64 keys
                const auto weights = [&](int c, const float *x, uint32_t *to) {
                    const float2 n2 = make_float2(-base, -base);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 v4 = Q8 ? vs[c * 8 + j / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float2 y = make_float2(x[j + e], x[j + e + 1]);
                            y = Q8 ? add2(y, n2) : fma2(y, back2, n2);
                            y.x = exp2_ftz(y.x);
                            y.y = exp2_ftz(y.y);
                            ls[e / 2] = add2(ls[e / 2], y);
                            if (Q8) {
                                y = mul2(y, mul2(e == 0 ? make_float2(v4.x, v4.y) : make_float2(v4.z, v4.w), f2));
                                to[(j + e) / 2] = pack_f16x2(y.x, y.y);
                            } else {
                                to[(j + e) / 2] = pack_bf16x2(y.x, y.y);
                            }
                        }
                    }
                };
                const auto publish = [&](int panel) {       // 64 keys
                    if (C::kPShared) {
                        uint8_t *dst = sm + C::oP + s * C::kPBytes + panel * C::kPanel + row * 128;
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<uint4 *>(dst + ((v ^ (row & 7)) << 4)) =
                                make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                    } else {
                        const uint32_t tP = tmem + C::cP + uint32_t(s * 64 + panel * 32) + lane_off;
                        tc::tmem_st32(tP, pk);
                    }
                };
                if constexpr (Q8) {
                    settle();
                    for (;;) {
                        rescale();
                        corr = 1.f;
                        ls[0] = ls[1] = make_float2(0.f, 0.f);
#pragma unroll 1
                        for (int p64 = 0; p64 < kKeys / 64; ++p64) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int c = 2 * p64 + k;
                                scores8(c, x);
                                const uint32_t adm = full ? kAll : admitted(c);
                                if (!full) mask(adm, x);
                                largest(x);
                                weights(c, x, pk + 16 * k);
                                if (!full)                  // the scale of a masked key may be anything
#pragma unroll
                                    for (int j = 0; j < 16; ++j)
                                        pk[16 * k + j] &= (((adm >> (2 * j)) & 1u) ? 0xffffu : 0u) |
                                                          (((adm >> (2 * j + 1)) & 1u) ? 0xffff0000u : 0u);
                            }
                            publish(p64);
                        }
                        // once more at most: the maximum is that of all keys now
                        if (!__any_sync(kAll, follow())) break;
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(bars + C::bSFree + s);
                } else {
                    ls[0] = ls[1] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int p64 = 0; p64 < kKeys / 64; ++p64) {
                        weights(2 * p64, x + p64 * 64, pk);
                        weights(2 * p64 + 1, x + p64 * 64 + 32, pk + 16);
                        if (p64 == 0) {
                            settle();
                            rescale();
                        }
                        publish(p64);
                    }
                }
                l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                if (C::kPShared) tc::fence_proxy_async_smem();
                tc::tmem_st_wait();
            } else {
                tc::mbar_arrive(bars + C::bSFree + s);
                // as above: P of this step may be announced once the last one's was used
                if (t > 0) ok &= tc::mbar_wait(bars + C::bPv + s, (t - 1) & 1, status);
            }
            tc::tc_fence_before();
            tc::mbar_arrive(bars + C::bP + s);
        }
        if (steps > 0) ok &= tc::mbar_wait(bars + C::bPv + s, (steps - 1) & 1, status);
        tc::tc_fence_after();
        const float un = Q8 ? exp2_int(big - kWeightShift) : 1.f;
        if (merges) tc::named_bar_sync(1, 32 * C::kSoft);   // nothing reads Q, P and the rings any more
        if (!merges) {
            const float inv = (l > 0.f || l != l ? __fdiv_rn(1.f, l) : 0.f) * un;
            bool finite = true;
            if (ok && active) {
                uint16_t *dst = a.out + token_row(s, min(row, rows - 1), int64_t(a.q_heads) * D);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(tO + uint32_t(c), o);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float x = l != 0.f ? __uint_as_float(o[j]) * inv : 0.f;
                        finite = finite && fabsf(x) < -kMinusInf;
                        o[j] = __float_as_uint(x);
                    }
                    if (row < rows)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w[j] = pack_bf16x2(__uint_as_float(o[8 * v + 2 * j]), __uint_as_float(o[8 * v + 2 * j + 1]));
                            *reinterpret_cast<uint4 *>(dst + c + 8 * v) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                }
                if (!Q8) {
                    // a sum that is not a number comes from the row's own scores;
                    // other lanes write over what this one wrote above
                    __syncwarp();
                    for (uint32_t again = __ballot_sync(kAll, row < rows && !finite && l == l); again != 0;
                         again &= again - 1) {
                        const int which = (warp & 3) * 32 + __ffs(again) - 1;
                        float x[D / 32];
                        row_alone<D>(a, r, sight_at(s, which), head, a.q + token_row(s, which, a.q_stride), x);
                        uint16_t *to = a.out + token_row(s, which, int64_t(a.q_heads) * D) + lane * (D / 32);
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) to[e] = f32_to_bf16_bits(x[e]);
                    }
                }
            }
        } else {
            // the stream's state, for the merge
            const bool any = ok && steps > 0 && l != 0.f;
            reinterpret_cast<float2 *>(sm + C::oStat)[s * kRows + row] =
                any ? make_float2(m, l) : make_float2(kMinusInf, 0.f);
            float *dst = reinterpret_cast<float *>(sm + C::oP) + (s * kRows + row) * C::kOStride;
            if (ok && steps > 0 && active)
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(tO + uint32_t(c), o);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(dst + c + j) =
                            make_float4(__uint_as_float(o[j]) * un, __uint_as_float(o[j + 1]) * un,
                                        __uint_as_float(o[j + 2]) * un, __uint_as_float(o[j + 3]) * un);
                }
        }
        tc::tc_fence_before();
    } else {
        if (warp < C::kSoft + 2) {
            // ----------- MMA, in pair of stream s, in dual (where each tile is one
            // stream's, and a barrier's phases have to be seen in order) of both
            if (lane == 0 && (kPair || warp == C::kSoft)) {
                constexpr uint32_t idesc_s = Q8 ? tc::idesc_f16_f32(kRows, kKeys) : tc::idesc_bf16_f32(kRows, kKeys);
                constexpr uint32_t idesc_o = Q8 ? tc::idesc_f16_f32(kRows, D, true) : tc::idesc_bf16_f32(kRows, D, true);
                const uint32_t ring = tc::smem_u32(sm + C::oRing);
                // S = Q K^T of a stream's step t, once the scores of the last are read
                const auto scores = [&](int s, int t, int q) {
                    const int st = q % C::kStages;
                    if (!tc::mbar_wait(bars + C::bFull + st, (q / C::kStages) & 1, status)) return false;
                    if (t > 0 && !tc::mbar_wait(bars + C::bSFree + s, (t - 1) & 1, status)) return false;
                    tc::tc_fence_after();
                    const uint32_t ak = ring + uint32_t(st * C::kStage);
                    const uint32_t aq = tc::smem_u32(sm + C::oQ + (kPair ? s * C::kStage : 0));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = uint32_t((k >> 2) * C::kPanel + (k & 3) * 32);
                        tc::mma_bf16(tmem + C::cS + uint32_t(s * kKeys), tc::smem_desc_sw128(aq + off, 1024),
                                     tc::smem_desc_sw128(ak + off, 1024), idesc_s, k > 0);
                    }
                    tc::mma_commit(bars + C::bS + s);
                    tc::mma_commit(bars + C::bEmpty + st);
                    return true;
                };
                // O += P V, once V is there and P is written
                const auto output = [&](int s, int t, int q) {
                    const int st = q % C::kStages;
                    if (!tc::mbar_wait(bars + C::bFull + st, (q / C::kStages) & 1, status)) return false;
                    if (!Q8 && tile_of(s, t) == n - 1 && !tc::mbar_wait(bars + C::bTail, 0, status)) return false;
                    if (!tc::mbar_wait(bars + C::bP + s, t & 1, status)) return false;
                    tc::tc_fence_after();
                    const uint32_t av = ring + uint32_t(st * C::kStage);
                    const uint32_t tO = tmem + C::cO + uint32_t(s * D), ap = tc::smem_u32(sm + C::oP + s * C::kPBytes);
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k) {
                        const uint64_t dv = tc::smem_desc_sw128_mn(av + k * 2048, C::kPanel, 1024);
                        const uint32_t more = (t > 0 || k > 0) ? 1u : 0u;
                        if (C::kPShared)
                            tc::mma_bf16(tO, tc::smem_desc_sw128(ap + (k >> 2) * C::kPanel + (k & 3) * 32, 1024), dv,
                                         idesc_o, more);
                        else
                            tc::mma_bf16_ts(tO, tmem + C::cP + uint32_t(s * 64 + k * 8), dv, idesc_o, more);
                    }
                    tc::mma_commit(bars + C::bPv + s);
                    tc::mma_commit(bars + C::bEmpty + st);
                    return true;
                };
                // Stream 1 starts once stream 0 has its first scores: out of
                // step, one's exponentials run under the other's loads and maxima
                // (3 prompts: 446 us in step, 404 so, 428 and more with later starts).
                if (steps_of(warp - C::kSoft) > 0 && tc::mbar_wait(bars + C::bQ, 0, status) &&
                    (!kPair || warp == C::kSoft || tc::mbar_wait(bars + C::bGo, 0, status)))
                    schedule(n, [&](bool v, int i, int q) {
                        const int s = kPair ? warp - C::kSoft : i & 1, t = kPair ? i : i >> 1;
                        return v ? output(s, t, q) : scores(s, t, q);
                    });
            }
            __syncwarp();
        } else if (!Q8) {
            // ------------------------------- producers, one of K and one of V
            const bool of_v = warp == C::kSoft + 3;
            const int pages = kKeys / a.c.page, per16 = a.c.page / 16, tiles_at_once = 32 / pages;
            // entries of the tiles from i on, one to a lane
            const auto look_up = [&](int i) {
                const int u = i + lane / pages;
                return u < n ? page_entry(a, r, tiles.key0(u), lane % pages) : 0;
            };
            int32_t ids = -1, next = look_up(0);
            bool ok = true;
            uint32_t mine = 0u, odd = 0u;                   // stages last loaded by this warp, and their phases
            schedule_once(n, [&](bool v, int i, int q) {
                if (v != of_v) return true;
                const int at = i % tiles_at_once * pages, st = q % C::kStages;
                if (at == 0) {
                    const int u = i + lane / pages;
                    ids = page_checked(a, u < n && page_seen(a, r, tiles.key0(u), lane % pages), next);
                    next = look_up(i + tiles_at_once);
                }
                if (q >= C::kStages)
                    ok = __all_sync(kAll, tc::mbar_wait(bars + C::bEmpty + st, (q / C::kStages - 1) & 1, status));
                if (!ok) return false;
                mine |= 1u << st;
                odd = (odd & ~(1u << st)) | uint32_t((q / C::kStages) & 1) << st;
                const uint32_t gone = (__ballot_sync(kAll, ids == -2) >> at) & ((1u << pages) - 1);
                if (lane == 0) {
                    if (!v) {
                        uint32_t there = 0xffu;
                        for (uint32_t g = gone; g != 0; g &= g - 1)
                            there &= ~(((1u << per16) - 1) << ((__ffs(g) - 1) * per16));
                        notes[i % kNotes] = there;
                    }
                    tc::mbar_arrive_expect_tx(bars + C::bFull + st, C::kStage);
                }
                __syncwarp();
                for (int g = 0; g < pages; ++g) {
                    const int32_t pid = __shfl_sync(kAll, ids, at + g);
                    if (lane == 0)
#pragma unroll
                        for (int sub = 0; sub < C::kSub; ++sub)     // what is not there arrives as zeros
                            tc::tma_load_4d(sm + C::oRing + st * C::kStage + sub * C::kPanel + g * a.c.page * 128,
                                            v ? &tm_v : &tm_k, bars + C::bFull + st, sub * 64, 0, head, pid < 0 ? -1 : pid);
                }
                __syncwarp();
                return true;
            });
            if (!ok)                                        // copies in flight land before the CTA ends
                for (int st = 0; st < C::kStages; ++st)
                    for (int poll = 0; ((mine >> st) & 1u) && poll < (1 << 20); ++poll)
                        if (tc::mbar_test_wait(bars + C::bFull + st, (odd >> st) & 1u)) break;
            if (of_v && ok && n > 0) {
                // rows past the last key hold anything, and 0 times NaN must not reach O
                const int q = 2 * n - 1, st = q % C::kStages, tail = r.end - tiles.key0(n - 1);
                if (tail < kKeys && tc::mbar_wait(bars + C::bFull + st, (q / C::kStages) & 1, status))
                    for (int i = lane; i < (kKeys - tail) * 8 * C::kSub; i += 32) {
                        const int row = tail + i / (8 * C::kSub), c = i % (8 * C::kSub);
                        *reinterpret_cast<uint4 *>(sm + C::oRing + st * C::kStage + (c >> 3) * C::kPanel + row * 128 +
                                                   (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + C::bTail);
            }
        } else if (warp < C::kSoft + 4) {
            // ---- 8-bit pages: codes and scales into a ring of their own, a warp for K
            // and one for V, in pieces of 16 and 4 bytes (bulk copies, one for
            // each page and its scales, take one thread 200 cycles each)
            const bool of_v = warp == C::kSoft + 3;
            constexpr int kPer = D / 16;                    // pieces of a row
            constexpr int kRaw = C::kRaw > 0 ? C::kRaw : 1;
            const int page = a.c.page, shift = 31 - __clz(page);
            // entries of tile i, one to each of eight lanes; used a tile later
            const auto entries = [&](int i) { return i < n && lane < 8 ? page_entry(a, r, tiles.key0(i), lane) : 0; };
            int32_t next = entries(0);
            schedule_once(n, [&](bool v, int i, int q) {
                if (v != of_v) return true;
                const int32_t key0 = tiles.key0(i);
                const int raw = q % kRaw;
                const int32_t ids = page_checked(a, lane < 8 && page_seen(a, r, key0, lane), next);
                next = entries(i + 1);
                const uint32_t gone = __ballot_sync(kAll, ids == -2), here = __ballot_sync(kAll, ids >= 0);
                // this lane's page: its first row in the cache
                const int64_t base = ids < 0 ? -1 : (int64_t(ids) * a.c.heads + head) * page;
                const int end = r.end - key0, hide = r.sinks_end - key0, show = r.first - key0;
                if (q >= kRaw &&
                    !__all_sync(kAll, tc::mbar_wait(bars + C::bRawEmpty + raw, (q / kRaw - 1) & 1, status)))
                    return false;
                uint8_t *dst = sm + C::oRaw + raw * C::kRawStage;
                const int8_t *src = reinterpret_cast<const int8_t *>(v ? a.c.v : a.c.k);
                float *sc = reinterpret_cast<float *>(dst + kKeys * D);
                if (here == (1u << (kKeys >> shift)) - 1 && end >= kKeys && (hide >= kKeys || show <= 0 || show <= hide)) {
                    // every row is there: sixteen at a time, of one page
                    const int8_t *mine = src + (lane / kPer) * D + lane % kPer * 16;
#pragma unroll
                    for (int g = 0; g < kKeys / 16; ++g) {
                        const int64_t row0 = __shfl_sync(kAll, base, g * 16 >> shift) + (g * 16 & (page - 1));
#pragma unroll
                        for (int j = 0; j < kPer / 2; ++j)
                            tc::cp_async16(dst + (g * 16 * kPer + j * 32 + lane) * 16, mine + row0 * D + j * (32 / kPer) * D);
                    }
                    if (!v) {
                        const int64_t row0 = __shfl_sync(kAll, base, lane * 4 >> shift) + (lane * 4 & (page - 1));
                        tc::cp_async16(sc + lane * 4, a.ks + row0);
                        tc::cp_async16(sc + kKeys + lane * 4, a.vs + row0);
                    }
                } else {
                    const auto row_in = [&](int x) -> int64_t {     // -1: nothing sees it
                        const int64_t row0 = __shfl_sync(kAll, base, x >> shift);
                        return row0 < 0 || x >= end || (x >= hide && x < show) ? -1 : row0 + (x & (page - 1));
                    };
#pragma unroll 1
                    for (int j = 0; j < kPer * 4; ++j) {
                        const int c = j * 32 + lane;
                        const int64_t at = row_in(c / kPer);
                        tc::cp_async16_zfill(dst + c * 16, src + (at < 0 ? 0 : at) * D + c % kPer * 16, at >= 0);
                    }
                    if (!v)
#pragma unroll 1
                        for (int x = lane; x < kKeys; x += 32) {
                            const int64_t at = row_in(x);
                            tc::cp_async4_zfill(sc + x, a.ks + (at < 0 ? 0 : at), at >= 0);
                            tc::cp_async4_zfill(sc + kKeys + x, a.vs + (at < 0 ? 0 : at), at >= 0);
                        }
                }
                if (!v && lane == 0) {
                    uint32_t there = 0xffu;
                    for (uint32_t g = gone; g != 0; g &= g - 1)
                        there &= ~(((1u << (page / 16)) - 1) << ((__ffs(g) - 1) * (page / 16)));
                    notes[i % kNotes] = there;
                }
                // the copies' arrivals come when they end and say nothing of the
                // stores before them: the note has one of its own
                tc::cp_async_arrive(bars + C::bRawFull + raw);
                if (lane == 0) tc::mbar_arrive(bars + C::bRawFull + raw);
                return true;
            });
            tc::cp_async_wait_all();
        } else {
            // ----------------------------------------- codes to fp16, into the ring
            constexpr int kPer = D / 16;
            constexpr int kRaw = C::kRaw > 0 ? C::kRaw : 1;
            const int w = tid - (C::kSoft + 4) * 32;
            float *scales = reinterpret_cast<float *>(sm + C::oScales);
            schedule_once(n, [&](bool v, int i, int q) {
                const int st = q % C::kStages, raw = q % kRaw;
                const bool ok =
                    tc::mbar_wait(bars + C::bRawFull + raw, (q / kRaw) & 1, status) &&
                    (q < C::kStages || tc::mbar_wait(bars + C::bEmpty + st, (q / C::kStages - 1) & 1, status));
                if (!__all_sync(kAll, ok)) return false;
                const uint8_t *src = sm + C::oRaw + raw * C::kRawStage;
                uint8_t *stage = sm + C::oRing + st * C::kStage;
                if (!v) {
                    const float *sc = reinterpret_cast<const float *>(src + kKeys * D) + w;
                    const float sv = sc[kKeys];
                    scales[(i % 8) * 2 * kKeys + w] = sc[0];
                    scales[((i % 8) * 2 + 1) * kKeys + w] = sv;
                    const uint32_t top = __reduce_max_sync(kAll, fabsf(sv) < -kMinusInf ? __float_as_uint(fabsf(sv)) : 0u);
                    if (lane == 0) reinterpret_cast<uint32_t *>(sm + C::oTops)[(i % kNotes) * 4 + (w >> 5)] = top;
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int c = j * 128 + w, row = c / kPer, ch = c % kPer;
                    store_codes(stage + (ch >> 2) * C::kPanel + row * 128, (ch & 3) * 2, row,
                                *reinterpret_cast<const uint4 *>(src + c * 16));
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(bars + C::bFull + st);
                tc::mbar_arrive(bars + C::bRawEmpty + raw);
                return true;
            });
        }
    }

    if (merges) {
        // rows are dealt to the cluster's CTAs and their warps; each merges the
        // states of every CTA, in dual of both streams
        cg::cluster_group peers = cg::this_cluster();
        if (p.cluster > 1)
            peers.sync();
        else
            __syncthreads();
        const int rows0 = rows_of(0), rows = kPair ? rows0 + rows_of(1) : rows0;
        constexpr int kOf = kPair ? 1 : 2;                  // states of a row in a CTA
        constexpr int E = D / 32;
        for (int u = rank + p.cluster * warp; u < rows; u += p.cluster * C::kWarps) {
            const int s = u < rows0 ? 0 : 1, row = u - s * rows0;
            float2 st = make_float2(kMinusInf, 0.f);
            if (lane < kOf * p.cluster)
                st = *peers.map_shared_rank(
                    reinterpret_cast<float2 *>(sm + C::oStat) + (kPair ? s : lane & 1) * kRows + row, lane / kOf);
            const float top = warp_max(st.x);
            const float w = st.x == kMinusInf && st.y == 0.f ? 0.f : exp2_ftz(st.x - (top == kMinusInf ? 0.f : top));
            const float l = warp_sum(w * st.y);
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.f;
            for (int i = 0; i < kOf * p.cluster; ++i) {
                const float wi = __shfl_sync(kAll, w, i);
                if (__shfl_sync(kAll, st.y, i) == 0.f) continue;          // nothing there
                const float *o = peers.map_shared_rank(
                    reinterpret_cast<float *>(sm + C::oP) + ((kPair ? s : i & 1) * kRows + row) * C::kOStride, i / kOf);
                if (E == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(o + lane * 4);
                    x[0] = fmaf(wi, v.x, x[0]);
                    x[1] = fmaf(wi, v.y, x[1]);
                    x[E - 2] = fmaf(wi, v.z, x[E - 2]);
                    x[E - 1] = fmaf(wi, v.w, x[E - 1]);
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(o + lane * 2);
                    x[0] = fmaf(wi, v.x, x[0]);
                    x[E - 1] = fmaf(wi, v.y, x[E - 1]);
                }
            }
            const float inv = l > 0.f || l != l ? __fdiv_rn(1.f, l) : 0.f;
            bool finite = true;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[e] *= inv;
                finite = finite && fabsf(x[e]) < -kMinusInf;
            }
            // a sum that is not a number comes from the row's own scores
            if (!Q8 && l == l && !__all_sync(kAll, finite))
                row_alone<D>(a, r, sight_at(s, row), head, a.q + token_row(s, row, a.q_stride), x);
            uint16_t *to = a.out + token_row(s, row, int64_t(a.q_heads) * D) + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(to + e) = pack_bf16x2(x[e], x[e + 1]);
        }
        if (p.cluster > 1) peers.sync();                    // peers read this CTA's shared memory
    }
    __syncthreads();
    if (warp == C::kSoft) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 paged_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                                            &qr) == cudaSuccess && qr == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// Pages as a 4-D tensor, box 64 channels x page rows, 128-byte swizzle.
bool make_page_map(CUtensorMap *m, const void *base, const CacheView &c) {
    auto fn = paged_encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t row = cuuint64_t(c.d) * 2;
    cuuint64_t dims[4] = {cuuint64_t(c.d), cuuint64_t(c.page), cuuint64_t(c.heads), cuuint64_t(c.num_pages)};
    cuuint64_t strides[3] = {row, row * c.page, row * c.page * c.heads};
    cuuint32_t box[4] = {64, cuuint32_t(c.page), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kPair, bool Q8>
cudaError_t launch_tiles(const AttentionArgs &a, const TilesPlan &p, int64_t items, cudaStream_t st) {
    using C = TCfg<D, kPair, Q8>;
    auto kernel = attention_tiles_kernel<D, kPair, Q8>;
    // once per device: calls on other threads set the same values
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || ((ready.load() >> dev) & 1u) == 0u) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
    CUtensorMap mk = {}, mv = {};
    if (!Q8 && (!make_page_map(&mk, a.c.k, a.c) || !make_page_map(&mv, a.c.v, a.c))) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(items * p.cluster));
    cfg.blockDim = dim3(C::kWarps * 32);
    cfg.dynamicSmemBytes = C::kTotal;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(p.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, a, p);
    if (e != cudaSuccess) cudaGetLastError();           // reported here, not by the next launch
    return e;
}

template <bool Q8>
cudaError_t launch_tiles_form(const AttentionArgs &a, cudaStream_t st) {
    const int group = a.q_heads / a.c.heads;
    const int64_t mean = (a.tokens + a.seqs - 1) / a.seqs;
    TilesPlan p;
    // A CTA costs what its key tiles do (a tile of a dual one as much as of a
    // pair, which has twice the rows) and about as much as three besides.  With a window
    // the keys are much the same everywhere, and the turns that the card
    // takes count; without one lengths are ragged, of which the host knows
    // only the table's width, and what counts is the longest CTA and the sum of all.
    p.tokens = std::max(1, kRows / group);
    int64_t keys = int64_t(a.width) * a.c.page;
    if (a.window > 0) keys = std::min<int64_t>(keys, int64_t(a.window) + a.sinks + p.tokens);
    const int64_t tiles = (keys + kKeys - 1) / kKeys, slots = 152, besides = 3;
    const auto cost = [&](int64_t ctas, int64_t one) {
        return a.window > 0 ? (ctas + slots - 1) / slots * (one + besides)
                            : std::max(one + besides, ctas * (one * 3 / 5 + besides) / slots);
    };
    // CTAs that have rows, as far as the host knows
    const auto busy = [&](int64_t size) { return (a.tokens + size - 1) / size * a.c.heads; };
    const int single = int(std::min<int64_t>(p.tokens, mean));
    bool pair = false;
    int64_t least = INT64_MAX;
    for (int c = 1; c <= 8; c *= 2)
        for (int two = mean > p.tokens && !(Q8 && a.c.d == 128) ? 1 : 0; two >= 0; --two) {
            const int64_t now = cost(busy(two != 0 ? 2 * p.tokens : single) * c, (tiles + c - 1) / c);
            if (now < least) {
                least = now;
                pair = two != 0;
                p.cluster = c;
            }
        }
    if (!pair) p.tokens = single;
    p.size = pair ? 2 * p.tokens : p.tokens;
    p.items_each = (a.tokens / a.seqs + p.size - 1) / p.size;
    const int64_t items = (a.cu != nullptr ? a.tokens / p.size + 2 * a.seqs : a.seqs * p.items_each) * a.c.heads;
    if (items * p.cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (a.c.d == 64) return pair ? launch_tiles<64, true, Q8>(a, p, items, st) : launch_tiles<64, false, Q8>(a, p, items, st);
    if constexpr (!Q8)
        if (pair) return launch_tiles<128, true, Q8>(a, p, items, st);
    return launch_tiles<128, false, Q8>(a, p, items, st);
}

}  // namespace
}  // namespace bsa
