// Single tokens over the paged cache: score every block mean of the token's
// sequence, keep the top-k blocks of each query head (or of each group of
// heads), softmax attention over their keys -- the two stages of page
// "sparse-attention-triton-bench" (Two-stage block indexer) for decoding, in
// one launch.
//
// One thread-block cluster of C CTAs serves one (token, cache head) with the
// up to 16 query heads that share it:
//   1. scores   each CTA scores a contiguous share of the blocks: a block
//               mean is one 16-byte load per lane, used by all heads of the
//               group; fp32 dot products, reduced over the lanes by an
//               exchange that halves the number of values at each step.
//               The scores stay in shared memory as order-preserving keys.
//   2. top-k    each row's scores gather in the shared memory of one CTA of the
//               cluster, whose warps find t, the k-th best, with a histogram
//               between the smallest and the largest score (64 equal
//               intervals, so that only a few scores share the one of t) and hand the selection back to the cluster.
//               A score is off its true value by at most e (a bound from the
//               sums of |q| and the largest |mean|), so blocks above t + 2e
//               are selected for certain and blocks below t - 2e are not.
//               Where more blocks than wanted lie between, those are scored
//               again in fp64 (ties to the lower id).  The selection is
//               therefore that of the exact scores, whatever the order of the
//               sums.
//   3. attention over the union of the heads' selected blocks, each loaded
//               once: a warp takes 16 keys at a time straight from global
//               memory into mma fragments (no shared memory between), S^T =
//               K Q^T and O^T += V^T P^T with the group's heads as the
//               8-wide side; a head that did not select the block is masked.
//               K of the next keys is requested as soon as the scores of
//               these are done, V as soon as their product is.  Online
//               softmax per warp, merged over the warps and then over the
//               cluster, each CTA receiving its share of the outputs.
// Bound: memory (block means and selected K, V once); with one sequence, the
// latency of the chain table -> means -> k-th best -> keys.  m16n8k16 mma.sync
// carries it: 8 or 16 rows against 16 keys is far below a tcgen05 tile (128
// rows), and the keys arrive at about 23 bytes a clock and SM, for which the
// tensor pipe is busy 7 to 8 % of the time, each weight entering twice (5 to
// 7 % and the same times with the weights rounded to bf16 once).
// Measured, device time: 96 sequences up to 32768 tokens, 64 heads over 8
// sharing selections, d 128, top-32: 158 us, 5.8 TB/s (86 % of a plain copy's
// rate); 32 such sequences, 32 heads over 8, d 64, top-16, each head for
// itself: 57 us, 4.7 TB/s (the CTAs run in step, so memory idles while they
// select: a fifth of a CTA's time); one sequence of 131072 tokens, 64 heads
// over 8, top-32: 31 us against 11 us of traffic.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cstddef>

#include "bsa_device.cuh"
#include "bsa_internal.h"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace bsa {
namespace {

constexpr int kMaxRows = 16;        // query heads of one cluster
constexpr int kMaxK = 32;
constexpr int kMaxItems = kMaxRows * kMaxK;
constexpr int kMaxWarps = 12;
constexpr int kMaxCluster = 16;
constexpr int kBins = 64;
constexpr int kListCap = 256;       // candidates a team lists
constexpr int kMaxKeys = 32768;     // scores one CTA holds
constexpr int kMaxSmem = 227 * 1024;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();

struct Plan {
    int32_t cluster;      // CTAs per (token, cache head, part of the group)
    int32_t takers;       // CTAs that write outputs: a power of two
    int32_t group;        // query heads per cache head
    int32_t parts;        // clusters a group is dealt to
    int32_t rows;         // query heads per cluster
    int32_t score_rows;   // rows, or 1 when the group shares the selection
    int32_t part_off, main_off;
};

// Scratch of the warps that select for one row.
struct Team {
    uint32_t hist[kBins];
    uint32_t near[32];        // the keys of t's interval
    uint32_t low[kMaxWarps], high[kMaxWarps], floor[kMaxWarps];
    uint16_t list[kListCap];  // blocks of the intervals from just below t's up
    uint16_t sel[kMaxK], sure[kMaxK];
    int32_t count, near_count;
};

struct Fixed {
    int32_t fin[kMaxRows][kMaxK];    // the row's selection without the forced block
    int32_t fin_page[kMaxRows][kMaxK];
    float qabs[kMaxRows];            // sum of |q| over a row's channels and heads
    uint32_t bits[kDecodeMaxWidth / 32], pref[kDecodeMaxWidth / 32];
    int32_t pages[kMaxItems];
    uint32_t masks[kMaxItems];
    uint16_t items[kMaxItems];
    float wm[kMaxWarps][kMaxRows], wl[kMaxWarps][kMaxRows];
    float pm[kMaxCluster][kMaxRows], pl[kMaxCluster][kMaxRows];   // of every CTA
    uint32_t kmax;                   // bits of the largest |mean| of all blocks
    int32_t n_items;
    uint32_t redo;                   // rows whose output is not finite
    float redo_m[kMaxRows], redo_inv[kMaxRows];
    Team teams[kMaxWarps];           // as many as the CTA has warps
};

// Order-preserving image of a float (NaN as -inf, -0 as +0); 0 is below all.
__device__ __forceinline__ uint32_t key_of(float x) {
    x = x == x ? x + 0.f : kNegInf;
    const uint32_t u = __float_as_uint(x);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sums each of NV values over the LPB lanes of a lane group: at each step a
// lane keeps half of the values and gives the other half to its partner, so
// NV - 1 exchanges do what NV log2 LPB would.  The lane ends with the value
// of index (lane % LPB) / (LPB / NV).
template <int NV, int LPB>
__device__ __forceinline__ float reduce_exchange(float (&v)[NV], int lane) {
    static_assert(NV <= LPB, "one value per lane at most");
    int o = LPB / 2;
#pragma unroll
    for (int n = NV; n > 1; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = up ? v[i] : v[i + n / 2];
            const float keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(kFull, give, o);
        }
    }
    float r = v[0];
#pragma unroll
    for (; o > 0; o /= 2) r += __shfl_xor_sync(kFull, r, o);
    return r;
}

// The cluster's barrier in two halves.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t word(const uint4 &u, int j) {
    return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
}

// Everything a CTA of the cluster knows about its share of the work.
struct Job {
    int32_t token, head, part, row0, rows, rank, nb, own, own_page, ne, kk;
    int64_t len;
    const int32_t *table;     // the sequence's page ids
};

// q . mean in fp64 for one or two blocks (their loads in flight together);
// lanes hold D / 32 channels of q (summed over the group when it shares the
// selection).
template <int D>
__device__ __forceinline__ void score_fp64(const DecodeArgs &a, const Job &w, const int (&block)[2],
                                           int count, const double (&q)[D / 32], double (&s)[2],
                                           int lane) {
    float m[2][D / 32];
    bool good[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t pid = i < count ? w.table[block[i]] : -1;
        good[i] = pid >= 0 && pid < a.c.num_pages;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            m[i][e] = good[i] ? __ldg(a.c.kbar + (pid * a.c.heads + w.head) * D + lane * (D / 32) + e)
                              : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s[i] = 0.0;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) s[i] += q[e] * double(m[i][e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s[i] += __shfl_xor_sync(kFull, s[i], o);
        if (!good[i] || s[i] != s[i]) s[i] = double(kNegInf);
    }
}

// A row's q in fp64, summed over the group when it shares the selection.
template <int D>
__device__ __forceinline__ void load_fp64(const DecodeArgs &a, const Plan &p, const Job &w, int row,
                                          double (&q)[D / 32], int lane) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) q[e] = 0.0;
    const int h0 = w.head * p.group + (a.share ? 0 : w.row0 + row);
    const uint16_t *src = a.q + int64_t(w.token) * a.q_stride + int64_t(h0) * D + lane * (D / 32);
#pragma unroll 4
    for (int g = 0; g < (a.share ? p.group : 1); ++g)
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            q[e] += double(__uint_as_float(uint32_t(src[g * D + e]) << 16));
}

// Puts (x, b) in front of lane `at`'s entry; the last entry falls out.
__device__ __forceinline__ void insert_at(double &best, int &id, int at, double x, int b, int lane) {
    const double bu = __shfl_up_sync(kFull, best, 1);
    const int iu = __shfl_up_sync(kFull, id, 1);
    best = lane > at ? bu : lane == at ? x : best;
    id = lane > at ? iu : lane == at ? b : id;
}

// Stage 1: the keys of the CTA's n blocks from b0 on, each put into keys[row /
// C][block] of CTA row % C.  With up to four rows a lane takes eight channels of
// a block, in two loads: half the lanes share a block's sums, which halves the
// exchanges (96 sequences that share selections: 167 -> 160 us; with eight rows
// the registers run out and nothing is gained).
template <int D, int RP, int W>
__device__ __forceinline__ void score_blocks(const DecodeArgs &a, const Plan &p, const Job &w,
                                             Fixed &f, uint32_t *keys, int b0, int n) {
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int L = RP <= 4 ? 2 : 1;  // 16-byte loads of a lane for a block
    constexpr int LPB = D / 4 / L;      // lanes per block
    constexpr int BPL = 32 / LPB;       // blocks a warp takes at a time
    constexpr int U = (RP <= 2 ? 16 : 8) / L;          // such steps in flight
    constexpr int J = U < LPB / RP ? U : LPB / RP;
    constexpr int NV = J * RP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ch = (lane % LPB) * 4;    // and, for l > 0, 4 l LPB further
    constexpr int kStep = W * U * BPL;
    static_assert(U * BPL <= 32, "a lane looks up one page");
    const int ahead = lane < U * BPL ? lane : n;       // this lane's block of a batch
    int base = warp * U * BPL;
    int entry = base + ahead < n ? w.table[b0 + base + ahead] : 0;
    float q[RP][L][4];
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
        for (int l = 0; l < L; ++l)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[r][l][e] = 0.f;
    const uint16_t *qt = a.q + int64_t(w.token) * a.q_stride + int64_t(w.head) * p.group * D + ch;
    const auto row_sum = [&](float x, int row) {       // over the block's lanes
#pragma unroll
        for (int o = LPB / 2; o > 0; o /= 2) x += __shfl_xor_sync(kFull, x, o);
        if (lane == 0) f.qabs[row] = x;
    };
    if (RP == 1 && a.share) {
        float qa = 0.f;
#pragma unroll 8
        for (int g = 0; g < p.group; ++g)
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const uint2 x = *reinterpret_cast<const uint2 *>(qt + g * D + l * LPB * 4);
                const float v[4] = {bf16_low_half(x.x), bf16_high_half(x.x), bf16_low_half(x.y),
                                    bf16_high_half(x.y)};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    q[0][l][e] += v[e];
                    qa += fabsf(v[e]);
                }
            }
        if (warp == 0) row_sum(qa, 0);
    } else {
        uint2 raw[RP][L];               // all rows requested before any is used
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int l = 0; l < L; ++l)
                raw[r][l] = *reinterpret_cast<const uint2 *>(
                    qt + (w.row0 + min(r, w.rows - 1)) * D + l * LPB * 4);
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            float qa = 0.f;
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const uint2 x = r < w.rows ? raw[r][l] : make_uint2(0u, 0u);
                q[r][l][0] = bf16_low_half(x.x);
                q[r][l][1] = bf16_high_half(x.x);
                q[r][l][2] = bf16_low_half(x.y);
                q[r][l][3] = bf16_high_half(x.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) qa += fabsf(q[r][l][e]);
            }
            if (r % W == warp) row_sum(qa, r);
        }
    }
    const int srows = a.share ? 1 : w.rows;
    if (p.cluster > 1) cluster_wait();
    // where this lane's sums go: block `sub` of a step's J * BPL, one row
    const int at = (lane % LPB) / (LPB / NV), row = at % RP;
    const int sub = at / RP * BPL + lane / LPB;
    const bool writes = lane % (LPB / NV) == 0 && row < srows;
    uint32_t *dst = cluster.map_shared_rank(keys, row % p.cluster) + row / p.cluster * a.width + b0 + sub;
    float big = 0.f;
    bool unknown = false;
    for (; base < n; base += kStep) {
        int mine = -1;
        if (base + ahead < n) {
            mine = entry;
            if (mine < 0 || mine >= a.c.num_pages) {
                report_status(a.status, kStatusBadIndex);
                mine = -1;
            }
        }
        if (base + kStep + ahead < n) entry = w.table[b0 + base + kStep + ahead];
        float4 x[U][L];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t pid = __shfl_sync(kFull, mine, u * BPL + lane / LPB);
            const float *m = a.c.kbar + (pid * a.c.heads + w.head) * D + ch;
#pragma unroll
            for (int l = 0; l < L; ++l)
                x[u][l] = pid >= 0 ? __ldg(reinterpret_cast<const float4 *>(m + l * LPB * 4))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int l = 0; l < L; ++l)
                big = fmaxf(fmaxf(fmaxf(big, fabsf(x[u][l].x)), fmaxf(fabsf(x[u][l].y), fabsf(x[u][l].z))),
                            fabsf(x[u][l].w));
#pragma unroll
        for (int j0 = 0; j0 < U; j0 += J) {
            float v[NV];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    float s = 0.f;
#pragma unroll
                    for (int l = 0; l < L; ++l) {
                        const float4 y = x[j0 + j][l];
                        s = fmaf(q[r][l][0], y.x, s);
                        s = fmaf(q[r][l][1], y.y, s);
                        s = fmaf(q[r][l][2], y.z, s);
                        s = fmaf(q[r][l][3], y.w, s);
                    }
                    v[j * RP + r] = s;
                }
            const float s = reduce_exchange<NV, LPB>(v, lane);
            const bool good = __shfl_sync(kFull, mine, j0 * BPL + sub) >= 0;
            unknown |= s != s;
            if (writes && base + j0 * BPL + sub < n) dst[base + j0 * BPL] = key_of(good ? s : kNegInf);
        }
    }
    // a NaN score (from means that are not finite) leaves the bound unknown
    const uint32_t most = __reduce_max_sync(kFull, unknown ? 0x7fffffffu : __float_as_uint(big));
    if (lane < p.cluster) atomicMax(&cluster.map_shared_rank(&f, lane)->kmax, most);
}

// Where a row's kk-th largest key lies.
struct Found {
    int in, above;            // keys in its interval, keys above that
    bool listed;              // t.list has every key from `floor` up
    uint32_t floor;
};

// Narrows keys[0, n), kk < n, down to an interval with the kk-th largest and
// at most 32 keys (or equal ones only), which go to t.near, and lists the
// blocks of that interval, the one below it and all above.  Done by the team
// of `size` threads (whole warps; `me` is this one's index).  Intervals are
// equal in value, or in the keys where values are not finite; either way the
// smallest and the largest key part, so the loop ends.
template <typename Sync>
__device__ __forceinline__ Found narrow(const uint32_t *keys, int n, int kk, Team &t, int me, int size,
                                        Sync sync) {
    const int lane = me & 31, warps = size >> 5;
    uint32_t from = 0u, to = kFull;     // the keys still in question
    int above = 0;                      // how many lie above those
    bool first = true;
    for (;;) {
        for (int i = me; i < kBins; i += size) t.hist[i] = 0u;
        if (me == 0) t.count = t.near_count = 0;
        uint32_t lo = kFull, hi = 0u;
#pragma unroll 4
        for (int i = me; i < n; i += size) {
            const uint32_t x = keys[i];
            if (x >= from && x <= to) {
                lo = min(lo, x);
                hi = max(hi, x);
            }
        }
        lo = __reduce_min_sync(kFull, lo);
        hi = __reduce_max_sync(kFull, hi);
        if (warps > 1) {
            if (lane == 0) {
                t.low[me >> 5] = lo;
                t.high[me >> 5] = hi;
            }
            sync();
            lo = __reduce_min_sync(kFull, lane < warps ? t.low[lane] : kFull);
            hi = __reduce_max_sync(kFull, lane < warps ? t.high[lane] : 0u);
        } else {
            sync();
        }
        from = lo;
        to = hi;
        const float base = key_value(from), width = key_value(to) - base;
        const float scale = __fdividef(float(kBins) - 0.01f, width);
        const bool linear = width < 1e30f && width > 1e-30f;
        const int shift = max(0, 26 - __clz(to - from));
        const auto bin = [&](uint32_t x) {
            return linear ? int((key_value(x) - base) * scale) : int((x - from) >> shift);
        };
#pragma unroll 4
        for (int i = me; i < n; i += size) {
            const uint32_t x = keys[i];
            if (x >= from && x <= to) atomicAdd(&t.hist[bin(x)], 1u);
        }
        sync();
        // every warp for itself: lane l has the l-th pair of bins from the top
        const int top = kBins - 1 - 2 * lane;
        const int c0 = int(t.hist[top]), c1 = int(t.hist[top - 1]);
        int run = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, run, o);
            if (lane >= o) run += y;
        }
        const int who = __ffs(__ballot_sync(kFull, above + run >= kk)) - 1;
        const int over = above + run - c0 - c1;         // above this lane's bins
        const bool upper = over + c0 >= kk;
        above = __shfl_sync(kFull, upper ? over : over + c0, who);
        const int pivot = __shfl_sync(kFull, upper ? top : top - 1, who);
        const int in = __shfl_sync(kFull, upper ? c0 : c1, who);
        const int below = pivot > 0 ? int(t.hist[pivot - 1]) : 0;
        if (in > 32 && from != to) {
            // again within the interval; intervals are in order, so no other
            // key lies between its ends
            lo = kFull;
            hi = 0u;
            for (int i = me; i < n; i += size) {
                const uint32_t x = keys[i];
                if (x >= from && x <= to && bin(x) == pivot) {
                    lo = min(lo, x);
                    hi = max(hi, x);
                }
            }
            lo = __reduce_min_sync(kFull, lo);
            hi = __reduce_max_sync(kFull, hi);
            sync();
            if (lane == 0) {
                t.low[me >> 5] = lo;
                t.high[me >> 5] = hi;
            }
            sync();
            from = __reduce_min_sync(kFull, lane < warps ? t.low[lane] : kFull);
            to = __reduce_max_sync(kFull, lane < warps ? t.high[lane] : 0u);
            sync();
            first = false;
            continue;
        }
        Found r;
        r.in = min(in, 32);             // more only if all are equal
        r.above = above;
        r.listed = first && above + in + below <= kListCap;
        const int least = r.listed ? max(0, pivot - 1) : pivot;
        uint32_t floor = 0u;            // the largest key that is not listed
#pragma unroll 4
        for (int i = me; i < n; i += size) {
            const uint32_t x = keys[i];
            if (x >= from && x <= to) {
                const int b = bin(x);
                if (b < least) {
                    floor = max(floor, x);
                    continue;
                }
                if (b == pivot) {
                    const int at = atomicAdd(&t.near_count, 1);
                    if (at < 32) t.near[at] = x;
                }
                if (r.listed) t.list[atomicAdd(&t.count, 1)] = uint16_t(i);
            }
        }
        floor = __reduce_max_sync(kFull, floor);
        if (warps > 1) {
            if (lane == 0) t.floor[me >> 5] = floor;
            sync();
            floor = __reduce_max_sync(kFull, lane < warps ? t.floor[lane] : 0u);
        } else {
            sync();
        }
        r.floor = floor + 1u;
        return r;
    }
}

// Stage 2: fills f.fin with the kk selected ids of every score row,
// ascending, and f.fin_page with their pages, in every CTA of the cluster.
// Row r is selected by CTA r % C, whose keys[r / C] has all its scores.
template <int D, int W>
__device__ __forceinline__ void select_blocks(const DecodeArgs &a, const Plan &p, const Job &w,
                                              Fixed &f, const uint32_t *own_keys) {
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int srows = a.share ? 1 : w.rows, kk = w.kk, C = p.cluster, n = w.ne;
    // the warps are dealt to the rows in teams of `per`: as large as still
    // leave a team for each row
    const int mine = (srows - w.rank + C - 1) / C;
    int per = 1, team = warp, teams = W;
    if (mine <= 1) {
        per = W;
        team = 0;
        teams = 1;
    } else if (mine == 2) {
        per = W / 2;
        team = warp / (W / 2);
        teams = 2;
    } else if (mine <= W / 2) {
        per = 2;
        team = warp / 2;
        teams = W / 2;
    }
    const int size = per * 32, me = threadIdx.x - team * size;
    const auto sync = [&] {
        if (per == 1)
            __syncwarp();
        else
            tc::named_bar_sync(1 + team, size);
    };
    for (int k = team; k < mine; k += teams) {
        const int row = w.rank + k * C;
        const uint32_t *keys = own_keys + k * a.width;
        Team &t = f.teams[team];
        // 32 blocks are one interval (1024 tokens: 10.7 us, narrowed 11.7)
        const bool tiny = n <= 32;
        const Found r = tiny ? Found{n, 0, false, 0u} : narrow(keys, n, kk, t, me, size, sync);
        if (me >= 32) continue;     // the next row's syncs come before the scratch is reused
        // t, the kk-th largest: rank r.above + (keys above it in the interval,
        // or equal and before it)
        const uint32_t x = lane < r.in ? (tiny ? keys[lane] : t.near[lane]) : 0u;
        int rank = r.above;
        for (int j = 0; j < r.in; ++j) {
            const uint32_t y = __shfl_sync(kFull, x, j);
            rank += y > x || (y == x && j < lane);
        }
        const uint32_t hit = __ballot_sync(kFull, lane < r.in && rank == kk - 1);
        const uint32_t kth = __shfl_sync(kFull, x, hit != 0 ? __ffs(hit) - 1 : 0);
        // |computed - true| <= e: at most 8 + 4 roundings on a path of the sum
        // (4 + 5 with a lane's four channels), 2^-24 each of sum |q||mean|,
        // which is at most sum |q| times the largest |mean|; a shared row's q
        // is itself a sum of `group` terms.  The last unit leaves room for
        // this bound's own roundings.
        const float e = (f.qabs[row] * __uint_as_float(f.kmax)) *
                            (float(13 + (a.share ? p.group : 0)) * 5.9604645e-8f) + 1e-36f;
        uint32_t lo = 0u, hi = kFull;           // unknown: every block is open
        if (e < -kNegInf) {
            lo = key_of(key_value(kth) - 2.f * e);
            hi = key_of(key_value(kth) + 2.f * e);
        }
        const bool listed = r.listed && lo >= r.floor;
        const int m = listed ? t.count : n;
        int found = 0, have = 0;                // at or above lo, above hi
        for (int i0 = 0; i0 < m; i0 += 32) {
            const int b = i0 + lane < m ? (listed ? int(t.list[i0 + lane]) : i0 + lane) : 0;
            const uint32_t y = i0 + lane < m ? keys[b] : 0u;
            const uint32_t v = __ballot_sync(kFull, y >= lo && y != 0u);
            const uint32_t u = __ballot_sync(kFull, y > hi);
            const int at = found + __popc(v & ((1u << lane) - 1));
            const int ut = have + __popc(u & ((1u << lane) - 1));
            if (y >= lo && y != 0u && at < kMaxK) t.sel[at] = uint16_t(b);
            if (y > hi && ut < kMaxK) t.sure[ut] = uint16_t(b);
            found += __popc(v);
            have += __popc(u);
        }
        __syncwarp();
        int id = 0x7fffffff;
        if (found == kk) {
            if (lane < kk) id = t.sel[lane];
        } else if (!(f.qabs[row] > 0.f) || f.kmax == 0u) {
            // q or all means zero, or a NaN in q: the scores are exact (0, or
            // -inf for a page that is not there and for NaN), so the ids decide
            int got = 0;
            for (int pass = 0; pass < 2; ++pass)        // above the kk-th, then equal to it
                for (int i0 = 0; i0 < n && got < kk; i0 += 32) {
                    const uint32_t y = i0 + lane < n ? keys[i0 + lane] : 0u;
                    const uint32_t v = __ballot_sync(kFull, pass == 0 ? y > kth : y == kth);
                    const int at = got + __popc(v & ((1u << lane) - 1));
                    if ((v >> lane & 1u) && at < kk) t.sel[at] = uint16_t(i0 + lane);
                    got += __popc(v);
                }
            __syncwarp();
            if (lane < kk) id = t.sel[lane];
        } else {
            // more than wanted: those above t + 2e, then the best of the
            // others by their fp64 scores, lane i holding the i-th of these
            double q[D / 32], best = 0.0;
            load_fp64<D>(a, p, w, row, q, lane);
            int held = 0, open_id = 0;
            if (lane < have) id = t.sure[lane];
            for (int i0 = 0; i0 < m; i0 += 32) {
                const int b = i0 + lane < m ? (listed ? int(t.list[i0 + lane]) : i0 + lane) : 0;
                const uint32_t y0 = i0 + lane < m ? keys[b] : 0u;
                uint32_t open = __ballot_sync(kFull, y0 != 0u && y0 >= lo && !(y0 > hi));
                while (open != 0) {
                    int y[2], cnt = 0;
                    double v[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        y[j] = __shfl_sync(kFull, b, open != 0 ? __ffs(open) - 1 : 0);
                        cnt += open != 0;
                        open &= open - 1;
                    }
                    score_fp64<D>(a, w, y, cnt, q, v, lane);
#pragma unroll 1
                    for (int j = 0; j < cnt; ++j) {
                        const double vj = j == 0 ? v[0] : v[1];
                        const int yj = j == 0 ? y[0] : y[1];
                        const int at = __popc(__ballot_sync(
                            kFull, lane < held && (best > vj || (best == vj && open_id < yj))));
                        insert_at(best, open_id, at, vj, yj, lane);
                        held = min(held + 1, kMaxK);
                    }
                }
            }
            const int y = __shfl_sync(kFull, open_id, (lane - have) & 31);
            if (lane >= have && lane < kk) id = y;
        }
        const int page = lane < kk ? w.table[id] : 0;
        int before = 0;                         // ascending ids
#pragma unroll 8
        for (int j = 0; j < kMaxK; ++j) before += __shfl_sync(kFull, id, j) < id;
        if (lane < kk)
            for (int c = 0; c < C; ++c) {
                Fixed *peer = cluster.map_shared_rank(&f, c);
                peer->fin[row][before] = id;
                peer->fin_page[row][before] = page;
            }
    }
}

// The union of the rows' lists: items (ascending ids), their pages and the
// rows that selected each.  f.bits and f.masks are zero.
template <int W>
__device__ __forceinline__ void make_items(const DecodeArgs &a, const Plan &p, const Job &w,
                                           Fixed &f) {
    constexpr int kThreads = W * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool all = w.ne <= w.kk;                       // every block is selected
    const int sel = all ? w.ne : w.kk;
    const int cnt = sel + (w.own >= 0 ? 1 : 0);
    const uint32_t every = (1u << w.rows) - 1;
    const auto put = [&](int at, int id, int pid) {
        if (pid < 0 || pid >= a.c.num_pages) {
            report_status(a.status, kStatusBadIndex);
            pid = -1;
        }
        f.items[at] = uint16_t(id);
        f.pages[at] = pid;
    };
    if (all || a.share || w.rows == 1) {
        for (int i = tid; i < cnt; i += kThreads) {
            put(i, i == sel ? w.own : all ? i : f.fin[0][i],
                i == sel ? w.own_page : all ? w.table[i] : f.fin_page[0][i]);
            f.masks[i] = every;
        }
        if (tid == 0) f.n_items = cnt;
    } else {
        const int words = (w.nb + 31) / 32;
        for (int i = tid; i < w.rows * cnt; i += kThreads) {
            const int r = i / cnt, j = i - r * cnt;
            const int id = j == sel ? w.own : f.fin[r][j];
            atomicOr(&f.bits[id >> 5], 1u << (id & 31));
        }
        __syncthreads();
        if (warp == 0) {
            const int per = (words + 31) / 32, w0 = min(words, lane * per);
            const int w1 = min(words, w0 + per);
            int sum = 0;
            for (int i = w0; i < w1; ++i) sum += __popc(f.bits[i]);
            int run = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, run, o);
                if (lane >= o) run += y;
            }
            if (lane == 31) f.n_items = run;
            run -= sum;
            for (int i = w0; i < w1; ++i) {
                f.pref[i] = uint32_t(run);
                run += __popc(f.bits[i]);
            }
        }
        __syncthreads();
        for (int i = tid; i < w.rows * cnt; i += kThreads) {
            const int r = i / cnt, j = i - r * cnt;
            const int id = j == sel ? w.own : f.fin[r][j];
            const int at = int(f.pref[id >> 5]) + __popc(f.bits[id >> 5] & ((1u << (id & 31)) - 1));
            if (atomicOr(&f.masks[at], 1u << r) == 0u)       // the first row to come
                put(at, id, j == sel ? w.own_page : f.fin_page[r][j]);
        }
    }
    if (a.idx != nullptr && w.rank == 0 && (!a.share || w.part == 0)) {
        const int srows = a.share ? 1 : w.rows;
        for (int i = tid; i < srows * a.topk; i += kThreads) {
            const int r = i / a.topk, j = i - r * a.topk;
            const int id = j < sel ? (all ? j : f.fin[r][j]) : j < cnt ? w.own : -1;
            const int64_t row = a.share ? int64_t(w.token) * a.c.heads + w.head
                                        : int64_t(w.token) * a.q_heads + w.head * p.group + w.row0 + r;
            a.idx[row * a.topk + j] = id;
        }
    }
    __syncthreads();
}

// A row whose output is not finite, again and alone: the tiles multiply a
// masked key's weight 0, or the remainder of a weight, which may be 0 or below,
// with the key's value, which must not count where that is infinite or NaN.
// Every warp takes keys of the row's own blocks; `sum` has
// W + 1 rows of D.
template <int D, int W>
__device__ __forceinline__ void attend_alone(const DecodeArgs &a, const Plan &p, const Job &w,
                                          const Fixed &f, int row, float mx, float *sum) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *qr = a.q + int64_t(w.token) * a.q_stride +
                         int64_t(w.head * p.group + w.row0 + row) * D + lane * E;
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float(uint32_t(qr[e]) << 16);
        acc[e] = 0.f;
    }
    for (int i = 0; i < f.n_items; ++i) {
        const int64_t pid = f.pages[i];
        if (!(f.masks[i] >> row & 1u) || pid < 0) continue;
        const int keys = int(i64min(a.c.page, w.len - int64_t(f.items[i]) * a.c.page));
        for (int j = warp; j < keys; j += W) {
            const int64_t at = ((pid * a.c.heads + w.head) * a.c.page + j) * D + lane * E;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(q[e], __uint_as_float(uint32_t(a.c.k[at + e]) << 16), s);
            const float x = exp2_fast(warp_sum(s) * a.scale_log2 - (mx == kNegInf ? 0.f : mx));
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = fmaf(x, __uint_as_float(uint32_t(a.c.v[at + e]) << 16), acc[e]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) sum[warp * D + lane * E + e] = acc[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += W * 32) {
        float x = 0.f;
        for (int k = 0; k < W; ++k) x += sum[k * D + c];
        sum[W * D + c] = x;
    }
    __syncthreads();
}

// Stage 3 and the merge.  `part` is where the cluster leaves this CTA's share
// of the outputs, [CTA][rows][D / takers].
template <int D, int NT, int W>
__device__ __forceinline__ void attend(const DecodeArgs &a, const Plan &p, const Job &w, Fixed &f,
                                       float *part, float *po) {
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int kThreads = W * 32;
    constexpr int PS = D + 1;           // row stride of the warps' outputs
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n8 = lane >> 2, kq = lane & 3;
    uint4 q[NT][D / 32];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = t * 8 + n8;
        const uint16_t *src = a.q + int64_t(w.token) * a.q_stride +
                              int64_t(w.head * p.group + w.row0 + min(r, w.rows - 1)) * D + kq * 8;
#pragma unroll
        for (int g = 0; g < D / 32; ++g)
            q[t][g] = r < w.rows ? *reinterpret_cast<const uint4 *>(src + g * 32)
                                 : make_uint4(0u, 0u, 0u, 0u);
    }
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
        m[t][0] = m[t][1] = kNegInf;
        l[t][0] = l[t][1] = 0.f;
    }
    const int tpp = a.c.page / 16;      // 16-key tiles of a page, a power of two
    const int shift = 31 - __clz(tpp);
    const int units = f.n_items << shift, step = p.cluster * W;
    uint4 kr[2][D / 32], vr[4][D / 64];
    // the next unit from u on that has keys: its first row in the cache
    int64_t row0 = 0;
    int valid = 0, item = 0;
    const auto find = [&](int u) {
        for (; u < units; u += step) {
            item = u >> shift;
            const int tile = u & (tpp - 1);
            const int64_t pid = f.pages[item];
            const int64_t left = w.len - (int64_t(f.items[item]) * a.c.page + tile * 16);
            if (pid < 0 || left <= 0) continue;
            valid = int(i64min(16, left));
            row0 = (pid * a.c.heads + w.head) * a.c.page + tile * 16;
            return u;
        }
        return units;
    };
    const auto load_k = [&] {
        const uint16_t *kp = a.c.k + (row0 + n8) * D + kq * 8;
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
            kr[0][g] = __ldg(reinterpret_cast<const uint4 *>(kp + g * 32));
            kr[1][g] = __ldg(reinterpret_cast<const uint4 *>(kp + 8 * D + g * 32));
        }
    };
    const auto load_v = [&](int64_t row) {
        const uint16_t *vp = a.c.v + (row + 2 * kq) * D + n8 * 8;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
            vr[0][g] = __ldg(reinterpret_cast<const uint4 *>(vp + g * 64));
            vr[1][g] = __ldg(reinterpret_cast<const uint4 *>(vp + D + g * 64));
            vr[2][g] = __ldg(reinterpret_cast<const uint4 *>(vp + 8 * D + g * 64));
            vr[3][g] = __ldg(reinterpret_cast<const uint4 *>(vp + 9 * D + g * 64));
        }
    };
    int unit = find(w.rank * W + warp);
    if (unit < units) {
        load_k();
        load_v(row0);
    }
    while (unit < units) {
        const int now_valid = valid;
        const uint32_t mask = f.masks[item];
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
                mma_bf16(s[t], kr[0][g].x, kr[1][g].x, kr[0][g].y, kr[1][g].y, q[t][g].x, q[t][g].y);
                mma_bf16(s[t], kr[0][g].z, kr[1][g].z, kr[0][g].w, kr[1][g].w, q[t][g].z, q[t][g].w);
            }
        }
        unit = find(unit + step);
        if (unit < units) load_k();     // in flight during the softmax and P V
        uint32_t b0[NT], b1[NT], r0[NT], r1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float corr[2];
            bool moved = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool in = (mask >> (t * 8 + 2 * kq + e)) & 1u;
                // s[e]: key n8, s[2 + e]: key n8 + 8
                s[t][e] = in && n8 < now_valid ? s[t][e] * a.scale_log2 : kNegInf;
                s[t][2 + e] = in && n8 + 8 < now_valid ? s[t][2 + e] * a.scale_log2 : kNegInf;
                float x = fmaxf(s[t][e], s[t][2 + e]);
                x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                const float mn = fmaxf(m[t][e], x);
                const float base = mn == kNegInf ? 0.f : mn;     // nothing admitted yet
                moved |= mn != m[t][e];
                corr[e] = exp2_fast(m[t][e] - base);
                m[t][e] = mn;
                s[t][e] = exp2_fast(s[t][e] - base);
                s[t][2 + e] = exp2_fast(s[t][2 + e] - base);
                l[t][e] = l[t][e] * corr[e] + (s[t][e] + s[t][2 + e]);
            }
            if (__any_sync(kFull, moved)) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[t][i][0] *= corr[0];
                    o[t][i][1] *= corr[1];
                    o[t][i][2] *= corr[0];
                    o[t][i][3] *= corr[1];
                }
            }
            // P for the product is its bf16 value and what that leaves, again
            // in bf16: off by 2^-18 of p at most (of one bf16 value, 2^-9)
            const uint32_t p0 = pack_bf16x2(s[t][0], s[t][1]), p1 = pack_bf16x2(s[t][2], s[t][3]);
            b0[t] = transpose_8x8(p0);
            b1[t] = transpose_8x8(p1);
            r0[t] = transpose_8x8(pack_bf16x2(s[t][0] - bf16_low_half(p0), s[t][1] - bf16_high_half(p0)));
            r1[t] = transpose_8x8(pack_bf16x2(s[t][2] - bf16_low_half(p1), s[t][3] - bf16_high_half(p1)));
        }
        if (now_valid < 16) {
            // rows past the end hold anything: 0 * NaN must not reach O
            const int rows[4] = {2 * kq, 2 * kq + 1, 2 * kq + 8, 2 * kq + 9};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (rows[i] >= now_valid)
#pragma unroll
                    for (int g = 0; g < D / 64; ++g) vr[i][g] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w0 = word(vr[0][g], j), w1 = word(vr[1][g], j);
                const uint32_t w2 = word(vr[2][g], j), w3 = word(vr[3][g], j);
                const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
                const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma_bf16(o[t][g * 4 + j], a0, a1, a2, a3, b0[t], b1[t]);
                    mma_bf16(o[t][g * 4 + j], a0, a1, a2, a3, r0[t], r1[t]);
                }
            }
        if (unit < units) load_v(row0);
    }
    // merge the warps' states
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = t * 8 + 2 * kq + e;
            float x = l[t][e];
            x += __shfl_xor_sync(kFull, x, 4);
            x += __shfl_xor_sync(kFull, x, 8);
            x += __shfl_xor_sync(kFull, x, 16);
            if (r < w.rows) {
                if (n8 == 0) {
                    f.wm[warp][r] = m[t][e];
                    f.wl[warp][r] = x;
                }
                float *dst = po + (warp * p.rows + r) * PS + n8 * 8;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    dst[(i / 4) * 64 + (i % 4) * 2] = o[t][i][e];
                    dst[(i / 4) * 64 + (i % 4) * 2 + 1] = o[t][i][2 + e];
                }
            }
        }
    __syncthreads();
    uint16_t *out = a.out + (int64_t(w.token) * a.q_heads + w.head * p.group + w.row0) * D;
    const int C = p.cluster, share = D / p.takers;      // channels of each that writes
    const int shift_c = 31 - __clz(share);
    // a row with no key to attend to is zero
    const auto put = [&](int i, int r, float mx, float ls, float x0, float x1) {
        const float inv = ls > 0.f || ls != ls ? __fdiv_rn(1.f, ls) : 0.f;
        x0 *= inv;
        x1 *= inv;
        *reinterpret_cast<uint32_t *>(out + i) = pack_bf16x2(x0, x1);
        // a sum that is not a number comes from the row's own scores
        if (ls == ls && !(fabsf(x0) < -kNegInf && fabsf(x1) < -kNegInf)) {
            f.redo_m[r] = mx;
            f.redo_inv[r] = inv;
            atomicOr(&f.redo, 1u << r);
        }
    };
    for (int i = 2 * tid; i < w.rows * D; i += 2 * kThreads) {
        const int r = i / D, c = i % D;
        float mx = kNegInf;
#pragma unroll
        for (int k = 0; k < W; ++k) mx = fmaxf(mx, f.wm[k][r]);
        const float base = mx == kNegInf ? 0.f : mx;
        float x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float x = exp2_fast(f.wm[k][r] - base);
            x0 = fmaf(x, po[(k * p.rows + r) * PS + c], x0);
            x1 = fmaf(x, po[(k * p.rows + r) * PS + c + 1], x1);
            ls = fmaf(x, f.wl[k][r], ls);
        }
        if (C == 1) {
            put(i, r, mx, ls, x0, x1);
        } else {
            float *dst = cluster.map_shared_rank(part, c >> shift_c);
            *reinterpret_cast<float2 *>(dst + ((w.rank * w.rows + r) << shift_c) + (c & (share - 1))) =
                make_float2(x0, x1);
            if (c < 2 * p.takers) {     // one thread of the row for each
                Fixed *peer = cluster.map_shared_rank(&f, c / 2);
                peer->pm[w.rank][r] = mx;
                peer->pl[w.rank][r] = ls;
            }
        }
    }
    if (C > 1) {
        cluster.sync();
        if (w.rank >= p.takers) return;
        for (int j = 2 * tid; j < w.rows * share; j += 2 * kThreads) {
            const int r = j >> shift_c, i = r * D + w.rank * share + (j & (share - 1));
            float mx = kNegInf;
#pragma unroll 4
            for (int k = 0; k < C; ++k) mx = fmaxf(mx, f.pm[k][r]);
            const float base = mx == kNegInf ? 0.f : mx;
            float x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll 4
            for (int k = 0; k < C; ++k) {
                const float2 y = *reinterpret_cast<const float2 *>(part + k * w.rows * share + j);
                const float x = exp2_fast(f.pm[k][r] - base);
                x0 = fmaf(x, y.x, x0);
                x1 = fmaf(x, y.y, x1);
                ls = fmaf(x, f.pl[k][r], ls);
            }
            put(i, r, mx, ls, x0, x1);
        }
    }
    __syncthreads();
    if (f.redo == 0u) return;
    for (int r = 0; r < w.rows; ++r) {
        if (!(f.redo >> r & 1u)) continue;
        attend_alone<D, W>(a, p, w, f, r, f.redo_m[r], po);
        for (int c = tid; c < share; c += kThreads) {
            const float x = po[W * D + w.rank * share + c] * f.redo_inv[r];
            out[r * D + w.rank * share + c] = f32_to_bf16_bits(x);
        }
    }
}

// Warps of a CTA, and CTAs an SM holds by their registers (sixteen heads'
// accumulators take twice the registers).
constexpr int kWarpsSmall = 4;
constexpr int warps_large(int nt) { return nt == 1 ? 12 : 8; }
constexpr int ctas_per_sm(int d, int nt) { return nt == 2 ? 2 : d == 64 ? 4 : 3; }

// Clusters of 5 to 16 CTAs the card holds with one CTA to an SM (its SMs come
// in groups of unequal size, and a cluster lies within one).  Asked of one
// GB300; where another holds fewer, the last clusters take a second turn.
constexpr int kFewItems = 28;
constexpr int8_t kClustersFit[kMaxCluster + 1] = {0, 0, 0, 0, 0, 28, 23, 15, 15, 15, 13, 8, 8, 7, 7, 7, 7};

template <int D, int RP, int NT, int W>
__global__ void __launch_bounds__(W * 32, W == kWarpsSmall ? ctas_per_sm(D, NT) : 1)
    decode_kernel(DecodeArgs a, Plan p) {
    extern __shared__ __align__(16) char smem[];
    constexpr int kThreads = W * 32;
    Fixed &f = *reinterpret_cast<Fixed *>(smem);
    float *part = reinterpret_cast<float *>(smem + p.part_off);
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem + p.main_off);
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x;
    Job w;
    w.rank = int(blockIdx.x % unsigned(p.cluster));
    const unsigned item = blockIdx.x / unsigned(p.cluster);
    const unsigned per = unsigned(a.c.heads * p.parts);
    w.token = int32_t(item / per);
    const int hp = int(item - unsigned(w.token) * per);
    w.head = hp / p.parts;
    w.part = hp - w.head * p.parts;
    w.row0 = w.part * p.rows;
    w.rows = min(p.rows, p.group - w.row0);
    const int64_t seq = a.token_seq != nullptr ? a.token_seq[w.token] : w.token;
    w.len = a.lens[w.token];
    for (int i = tid; i < kDecodeMaxWidth / 32; i += kThreads) f.bits[i] = 0u;
    for (int i = tid; i < kMaxItems; i += kThreads) f.masks[i] = 0u;
    if (tid == 0) f.kmax = f.redo = 0u;
    if (seq < 0 || seq >= a.seqs) {
        if (tid == 0) report_status(a.status, kStatusBadIndex);
        w.len = 0;
    }
    const int64_t most = int64_t(a.width) * a.c.page;
    if (w.len < 0 || w.len > most) {
        if (tid == 0) report_status(a.status, kStatusInvalidArg);
        w.len = w.len < 0 ? 0 : most;
    }
    w.nb = int((w.len + a.c.page - 1) >> (31 - __clz(a.c.page)));      // a power of two
    if (w.nb == 0) {                    // the same for the whole cluster
        if (w.rank != 0) return;
        uint16_t *out = a.out + (int64_t(w.token) * a.q_heads + w.head * p.group + w.row0) * D;
        for (int i = tid; i < w.rows * D; i += kThreads) out[i] = 0;
        if (a.idx != nullptr && (!a.share || w.part == 0)) {
            const int64_t row = a.share ? int64_t(w.token) * a.c.heads + w.head
                                        : int64_t(w.token) * a.q_heads + w.head * p.group + w.row0;
            for (int i = tid; i < (a.share ? 1 : w.rows) * a.topk; i += kThreads)
                a.idx[row * a.topk + i] = -1;
        }
        return;
    }
    w.table = a.table + seq * a.width;
    w.own = a.local ? w.nb - 1 : -1;
    w.own_page = a.local ? w.table[w.own] : -1;
    w.ne = w.nb - (a.local ? 1 : 0);
    w.kk = a.topk - (a.local ? 1 : 0);
    // peers may write to this CTA's shared memory once all have come this far
    if (p.cluster > 1) cluster_arrive();
    __syncthreads();
    if (w.ne > w.kk && w.kk > 0) {
        const int each = (w.ne + p.cluster - 1) / p.cluster;
        const int b0 = min(w.ne, w.rank * each), n = min(w.ne, b0 + each) - b0;
        score_blocks<D, RP, W>(a, p, w, f, keys, b0, n);
        p.cluster > 1 ? cluster.sync() : __syncthreads();
        select_blocks<D, W>(a, p, w, f, keys);
        p.cluster > 1 ? cluster.sync() : __syncthreads();
    } else if (p.cluster > 1) {
        cluster_wait();
    }
    make_items<W>(a, p, w, f);
    attend<D, NT, W>(a, p, w, f, part, reinterpret_cast<float *>(keys));
}

template <int D, int RP, int NT, int W>
cudaError_t launch(const DecodeArgs &a, const Plan &p, size_t smem, int64_t items, cudaStream_t st) {
    auto kernel = decode_kernel<D, RP, NT, W>;
    // once per device: calls on other threads set the same values
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || ((ready.load() >> dev) & 1u) == 0u) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(items * p.cluster));
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(p.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, p);
    if (e != cudaSuccess) cudaGetLastError();           // reported here, not by the next launch
    return e;
}

template <int D, int RP, int NT>
cudaError_t pick(const DecodeArgs &a, const Plan &p, bool large, size_t smem, int64_t items,
                 cudaStream_t st) {
    if (large) return launch<D, RP, NT, warps_large(NT)>(a, p, smem, items, st);
    return launch<D, RP, NT, kWarpsSmall>(a, p, smem, items, st);
}

template <int D>
cudaError_t dispatch(const DecodeArgs &a, const Plan &p, bool large, size_t smem, int64_t items,
                     cudaStream_t st) {
    if (p.score_rows == 1) {
        if (p.rows > 8) return pick<D, 1, 2>(a, p, large, smem, items, st);
        return pick<D, 1, 1>(a, p, large, smem, items, st);
    }
    if (p.rows <= 2) return pick<D, 2, 1>(a, p, large, smem, items, st);
    if (p.rows <= 4) return pick<D, 4, 1>(a, p, large, smem, items, st);
    if (p.rows <= 8) return pick<D, 8, 1>(a, p, large, smem, items, st);
    return pick<D, 16, 2>(a, p, large, smem, items, st);
}

}  // namespace

cudaError_t launch_paged_decode(const DecodeArgs &a, cudaStream_t st) {
    Plan p;
    p.group = a.q_heads / a.c.heads;
    p.parts = (p.group + kMaxRows - 1) / kMaxRows;
    p.rows = (p.group + p.parts - 1) / p.parts;
    p.score_rows = a.share ? 1 : p.rows;
    const int64_t items = a.tokens * a.c.heads * p.parts;
    // Few items: large CTAs, one to an SM, in the largest clusters that fit the
    // card all at once.  Many: small CTAs, three or four to an SM, so that some
    // load while others select, in clusters as large as leave all CTAs on the
    // card at once (52 drafted tokens, 4 heads: 62 us in pairs; 70 in fours,
    // which take two turns; 90 alone).  That counts registers; tables of many
    // blocks take shared memory besides, up to one CTA to an SM (32 sequences
    // of 131072 tokens in pages of 32: 606 us against 184 us of traffic).  No
    // more warps than have two 16-key tiles to attend to or sixteen blocks to
    // score (1024 tokens, top-4: one CTA, 10.7 us; two, 11.1).
    const bool large = items <= kFewItems;
    const int warps = large ? warps_large(p.rows > 8 ? 2 : 1) : kWarpsSmall;
    const int64_t picked = int64_t(p.score_rows) * a.topk;
    const int64_t tiles = (picked < a.width ? picked : a.width) * (a.c.page / 16);
    const int64_t pairs = (tiles > a.width / 8 ? tiles : a.width / 8) / 2;
    if (large) {
        p.cluster = kMaxCluster;
        while (kClustersFit[p.cluster] < items) --p.cluster;
        while (p.cluster > 1 && (p.cluster - 1) * warps >= pairs) --p.cluster;
    } else {
        p.cluster = 1;
        while (p.cluster < 8 && p.cluster * warps < pairs &&
               items * p.cluster * 2 <= 152 * ctas_per_sm(a.c.d, p.rows > 8 ? 2 : 1))
            p.cluster *= 2;
    }
    const auto kept = [&] {         // scores a CTA holds
        return int64_t((p.score_rows + p.cluster - 1) / p.cluster) * a.width;
    };
    while (kept() > kMaxKeys) p.cluster *= 2;
    if (items * p.cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.takers = p.cluster >= 8 ? 8 : p.cluster >= 4 ? 4 : p.cluster >= 2 ? 2 : 1;
    const auto up = [](size_t x) { return (x + 15) / 16 * 16; };
    size_t off = up(offsetof(Fixed, teams) + warps * sizeof(Team));
    p.part_off = int32_t(off);
    if (p.cluster > 1) off = up(off + size_t(p.cluster) * p.rows * (a.c.d / p.takers) * 4);
    p.main_off = int32_t(off);
    const size_t scores = size_t(kept()) * 4;
    // the warps' outputs, or the W + 1 rows of a row that is attended to alone
    const size_t merge = size_t(warps) * p.rows * (a.c.d + 1) * 4;
    const size_t alone = size_t(warps + 1) * a.c.d * 4;
    const size_t smem = off + up(std::max({scores, merge, alone}));
    return a.c.d == 64 ? dispatch<64>(a, p, large, smem, items, st)
                       : dispatch<128>(a, p, large, smem, items, st);
}

}  // namespace bsa
