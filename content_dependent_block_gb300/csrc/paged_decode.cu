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
//   2. top-k    a warp sorts its share's best 32 (key, id) and each CTA gives
//               its list to the whole cluster (distributed shared memory), so
//               that every CTA merges all lists and knows t, the k-th best.
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
// latency of the chain table -> means -> merge -> table -> keys.  m16n8k16
// mma.sync carries it: 8 or 16 rows against 16 keys is far below a tcgen05
// tile (128 rows), and the keys arrive at about 23 bytes a clock and SM.
#include <cooperative_groups.h>

#include <utility>

#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace cg = cooperative_groups;

namespace bsa {
namespace {

constexpr int kMaxRows = 16;        // query heads of one cluster
constexpr int kMaxK = 32;
constexpr int kMaxItems = kMaxRows * kMaxK;
constexpr int kMaxWarps = 12;
constexpr int kMaxCluster = 8;
constexpr int kListCap = 256;       // candidates of a filtered list
constexpr int kMaxLocal = 2048;     // blocks one CTA scores
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();

struct Plan {
    int32_t cluster;      // CTAs per (token, cache head, part of the group)
    int32_t group;        // query heads per cache head
    int32_t parts;        // clusters a group is dealt to
    int32_t rows;         // query heads per cluster
    int32_t score_rows;   // rows, or 1 when the group shares the selection
    int32_t segs;         // warps that share a row's local top-k
    int32_t nloc;         // score slots of a row
    int32_t list_off, part_off, main_off;
};

// A CTA's best of one row, largest key first; `next` is the largest key that
// is not in the list (0: none).
struct List {
    uint32_t key[kMaxK];
    uint16_t id[kMaxK];
    uint32_t next;
};

struct Fixed {
    double dscore[kMaxRows][kMaxK];
    uint64_t seg[kMaxWarps][kMaxK];     // sorted lists of a row's parts
    uint32_t seg_next[kMaxWarps];
    uint16_t cand[kMaxWarps][kListCap];
    int32_t def[kMaxRows][kMaxK];    // re-scoring: own blocks above t + 2e
    int32_t did[kMaxRows][kMaxK];    // own best re-scored blocks
    int32_t fin[kMaxRows][kMaxK];    // the row's selection without the forced block
    int32_t ndef[kMaxRows], nd[kMaxRows], slow[kMaxRows];
    uint32_t lo[kMaxRows], hi[kMaxRows];
    uint32_t bits[kDecodeMaxWidth / 32], pref[kDecodeMaxWidth / 32];
    int32_t pages[kMaxItems];
    uint32_t masks[kMaxItems];
    uint16_t items[kMaxItems];
    float wm[kMaxWarps][kMaxRows], wl[kMaxWarps][kMaxRows];
    float pm[kMaxCluster][kMaxRows], pl[kMaxCluster][kMaxRows];   // of every CTA
    uint32_t kmaxes[kMaxCluster];
    uint32_t kmax;
    int32_t any_slow, n_items;
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

// Bitonic networks over the 32 lanes, largest first, B independent lists at
// once (the exchanges of one hide the latency of the others').
template <typename T, int B>
__device__ __forceinline__ void sort32(T (&x)[B], int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int j = size / 2; j > 0; j /= 2) {
            const bool larger = ((lane & j) == 0) == ((lane & size) == 0);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const T y = __shfl_xor_sync(kFull, x[b], j);
                x[b] = larger == (x[b] > y) ? x[b] : y;
            }
        }
}

// Merges pairs of sorted lists, x[i] with x[i + N], into their best 32;
// `low` keeps the largest of what falls out.
template <typename T, int B, int N>
__device__ __forceinline__ void merge32(T (&x)[B], T &low, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const T y = __shfl_sync(kFull, x[i + N], 31 - lane);
        const T out = x[i] > y ? y : x[i];
        x[i] = x[i] > y ? x[i] : y;
        low = low > out ? low : out;
    }
#pragma unroll
    for (int j = 16; j > 0; j /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const T y = __shfl_xor_sync(kFull, x[i], j);
            x[i] = ((lane & j) == 0) == (x[i] > y) ? x[i] : y;
        }
}
template <typename T, int B>
__device__ __forceinline__ void merge_all(T (&x)[B], T &low, int lane) {
    if constexpr (B >= 16) merge32<T, B, 8>(x, low, lane);
    if constexpr (B >= 8) merge32<T, B, 4>(x, low, lane);
    if constexpr (B >= 4) merge32<T, B, 2>(x, low, lane);
    if constexpr (B >= 2) merge32<T, B, 1>(x, low, lane);
}

// (key, index) as one number: a larger key first, then a lower index.
__device__ __forceinline__ uint64_t composite(uint32_t key, int i) {
    return (uint64_t(key) << 32) | uint32_t(0xffff - i);
}

// B batches of 32 keys a[index(i)], i < m, sorted and merged.
template <int B, typename F>
__device__ __forceinline__ uint64_t best32(const uint32_t *a, int m, F index, uint64_t &low, int lane) {
    uint64_t x[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int i = b * 32 + lane;
        x[b] = 0;
        if (i < m) {
            const int j = index(i);
            x[b] = composite(a[j], j);
        }
    }
    sort32(x, lane);
    merge_all(x, low, lane);
    return x[0];
}

// The best 32 of a[0, n) (lane i has the i-th) and the largest key left out.
// For many keys only those are sorted that are at or above the k-th largest
// of the 32 lanes' maxima: k of the keys are, and few others (some 20 to 100
// of 2048).
__device__ uint64_t top32(const uint32_t *a, int n, int k, uint16_t *cand, uint32_t &next, int lane) {
    const auto same = [](int i) { return i; };
    uint64_t low = 0, best;
    uint32_t rest = 0;
    if (n <= 32) {
        best = best32<1>(a, n, same, low, lane);
    } else if (n <= 64) {
        best = best32<2>(a, n, same, low, lane);
    } else if (n <= 128) {
        best = best32<4>(a, n, same, low, lane);
    } else {
        uint32_t mx[1] = {0u};
#pragma unroll 8
        for (int i = lane; i < n; i += 32) mx[0] = max(mx[0], a[i]);
        sort32(mx, lane);
        const uint32_t bound = __shfl_sync(kFull, mx[0], k - 1);
        int m = 0;
#pragma unroll 4
        for (int i0 = 0; i0 < n; i0 += 32) {
            const uint32_t x = i0 + lane < n ? a[i0 + lane] : 0u;
            const bool in = i0 + lane < n && x >= bound;
            const uint32_t b = __ballot_sync(kFull, in);
            const int at = m + __popc(b & ((1u << lane) - 1));
            if (in) {
                if (at < kListCap) cand[at] = uint16_t(i0 + lane);
            } else {
                rest = max(rest, x);
            }
            m += __popc(b);
        }
        __syncwarp();
        const auto listed = [cand](int i) { return int(cand[i]); };
        if (m <= 32) {
            best = best32<1>(a, m, listed, low, lane);
        } else if (m <= 64) {
            best = best32<2>(a, m, listed, low, lane);
        } else if (m <= 128) {
            best = best32<4>(a, m, listed, low, lane);
        } else if (m <= kListCap) {
            best = best32<8>(a, m, listed, low, lane);
        } else {                                // many equal scores
            rest = 0;
            best = 0;
            for (int i0 = 0; i0 < n; i0 += 32) {
                uint64_t x[2] = {best, i0 + lane < n ? composite(a[i0 + lane], i0 + lane) : 0};
                const uint64_t worst = __shfl_sync(kFull, best, 31);
                if (!__any_sync(kFull, x[1] > worst)) {
                    low = low > x[1] ? low : x[1];
                    continue;
                }
                uint64_t y[1] = {x[1]};
                sort32(y, lane);
                x[1] = y[0];
                merge32<uint64_t, 2, 1>(x, low, lane);
                best = x[0];
            }
        }
        __syncwarp();
    }
    next = __reduce_max_sync(kFull, max(rest, uint32_t(low >> 32)));
    return best;
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
    int32_t token, head, part, row0, rows, rank, nb, own, ne, kk;
    int64_t len;
    const int32_t *table;     // the sequence's page ids
};

// q . mean of one block in fp64; lanes hold D / 32 channels of q (summed over
// the group when it shares the selection).
template <int D>
__device__ __forceinline__ double score_fp64(const DecodeArgs &a, const Job &w, int block,
                                             const double (&q)[D / 32], int lane) {
    const int64_t pid = w.table[block];
    if (pid < 0 || pid >= a.c.num_pages) return double(kNegInf);
    const float *m = a.c.kbar + (pid * a.c.heads + w.head) * D + lane * (D / 32);
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s += q[e] * double(__ldg(m + e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    return s == s ? s : double(kNegInf);
}

// Stage 1: the keys of the CTA's n blocks from b0 on, sc[row][nloc].
template <int D, int RP, int W>
__device__ __forceinline__ void score_blocks(const DecodeArgs &a, const Plan &p, const Job &w,
                                             Fixed &f, uint32_t *sc, int b0, int n) {
    constexpr int LPB = D / 4;          // lanes per block
    constexpr int BPL = 32 / LPB;       // blocks per load instruction
    constexpr int U = 8;                // loads in flight
    constexpr int J = U < LPB / RP ? U : LPB / RP;
    constexpr int NV = J * RP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ch = (lane % LPB) * 4;
    float q[RP][4];
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) q[r][e] = 0.f;
    const uint16_t *qt = a.q + int64_t(w.token) * a.q_stride + int64_t(w.head) * p.group * D + ch;
    if (RP == 1 && a.share) {
        for (int g = 0; g < p.group; ++g) {
            const uint2 x = *reinterpret_cast<const uint2 *>(qt + g * D);
            q[0][0] += bf16_low_half(x.x);
            q[0][1] += bf16_high_half(x.x);
            q[0][2] += bf16_low_half(x.y);
            q[0][3] += bf16_high_half(x.y);
        }
    } else {
#pragma unroll
        for (int r = 0; r < RP; ++r)
            if (r < w.rows) {
                const uint2 x = *reinterpret_cast<const uint2 *>(qt + (w.row0 + r) * D);
                q[r][0] = bf16_low_half(x.x);
                q[r][1] = bf16_high_half(x.x);
                q[r][2] = bf16_low_half(x.y);
                q[r][3] = bf16_high_half(x.y);
            }
    }
    const int srows = a.share ? 1 : w.rows;
    uint32_t big = 0;
    constexpr int kStep = W * U * BPL;
    const int ahead = lane < U * BPL ? lane : n;       // this lane's block of a batch
    int base = warp * U * BPL;
    int entry = base + ahead < n ? w.table[b0 + base + ahead] : 0;
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
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t pid = __shfl_sync(kFull, mine, u * BPL + lane / LPB);
            x[u] = pid >= 0 ? __ldg(reinterpret_cast<const float4 *>(
                                  a.c.kbar + (pid * a.c.heads + w.head) * D + ch))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // as integers, so that a NaN counts as larger than everything
            big = max(big, __float_as_uint(x[u].x) & 0x7fffffffu);
            big = max(big, __float_as_uint(x[u].y) & 0x7fffffffu);
            big = max(big, __float_as_uint(x[u].z) & 0x7fffffffu);
            big = max(big, __float_as_uint(x[u].w) & 0x7fffffffu);
        }
#pragma unroll
        for (int j0 = 0; j0 < U; j0 += J) {
            float v[NV];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    float s = q[r][0] * x[j0 + j].x;
                    s = fmaf(q[r][1], x[j0 + j].y, s);
                    s = fmaf(q[r][2], x[j0 + j].z, s);
                    v[j * RP + r] = fmaf(q[r][3], x[j0 + j].w, s);
                }
            const float s = reduce_exchange<NV, LPB>(v, lane);
            const int at = (lane % LPB) / (LPB / NV);
            const int slot = (j0 + at / RP) * BPL + lane / LPB, row = at % RP;
            const bool good = __shfl_sync(kFull, mine, slot) >= 0;
            if (lane % (LPB / NV) == 0 && row < srows && base + slot < n)
                sc[row * p.nloc + base + slot] = key_of(good ? s : kNegInf);
        }
    }
    big = __reduce_max_sync(kFull, big);
    if (lane == 0) atomicMax(&f.kmax, big);
}

// Stage 2: fills f.fin with the kk selected ids of every score row,
// ascending.  Every CTA of the cluster ends with the same lists.
// lists[CTA][row] is filled by the cluster.
template <int D, int W>
__device__ __forceinline__ void select_blocks(const DecodeArgs &a, const Plan &p, const Job &w,
                                              Fixed &f, uint32_t *sc, List *lists, int b0, int n) {
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int srows = a.share ? 1 : w.rows, kk = w.kk, C = p.cluster;
    if (threadIdx.x < C) cluster.map_shared_rank(&f, threadIdx.x)->kmaxes[w.rank] = f.kmax;
    const auto give = [&](int row, uint64_t best, uint32_t next) {
        const int at = 0xffff - int(uint32_t(best) & 0xffffu);
        for (int c = 0; c < C; ++c) {
            List *l = cluster.map_shared_rank(&lists[w.rank * p.score_rows + row], c);
            l->key[lane] = uint32_t(best >> 32);
            l->id[lane] = uint16_t(b0 + at);
            if (lane == 0) l->next = next;
        }
    };
    for (int task = warp; task < srows * p.segs; task += W) {
        const int row = task / p.segs, seg = task - row * p.segs;
        const int per = (n + p.segs - 1) / p.segs;
        const int i0 = min(n, seg * per), m = min(n, i0 + per) - i0;
        uint32_t next;
        uint64_t best = top32(sc + row * p.nloc + i0, m, kk, f.cand[warp], next, lane);
        if (best != 0) best -= uint64_t(i0);            // the row's index
        if (p.segs == 1) {
            give(row, best, next);
        } else {
            f.seg[task][lane] = best;
            if (lane == 0) f.seg_next[task] = next;
        }
    }
    if (p.segs > 1) {
        __syncthreads();
        for (int row = warp; row < srows; row += W) {
            uint64_t x[8], low = 0;
            uint32_t next = 0;
#pragma unroll
            for (int s = 0; s < 8; ++s) x[s] = s < p.segs ? f.seg[row * p.segs + s][lane] : 0;
            if (lane < p.segs) next = f.seg_next[row * p.segs + lane];
            if (p.segs > 4) merge32<uint64_t, 8, 4>(x, low, lane);
            if (p.segs > 2) merge32<uint64_t, 8, 2>(x, low, lane);
            merge32<uint64_t, 8, 1>(x, low, lane);
            next = __reduce_max_sync(kFull, max(next, uint32_t(low >> 32)));
            give(row, x[0], next);
        }
    }
    if (C > 1)
        cluster.sync();
    else
        __syncthreads();
    for (int row = warp; row < srows; row += W) {
        // t, the kk-th best of the whole row
        uint32_t key[kMaxCluster], x[kMaxCluster], low = 0, kmax = 0, next = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
            x[c] = key[c] = c < C ? lists[c * p.score_rows + row].key[lane] : 0u;
        if (lane < C) {
            next = lists[lane * p.score_rows + row].next;
            kmax = f.kmaxes[lane];
        }
        kmax = __reduce_max_sync(kFull, kmax);
        if (C > 4) merge32<uint32_t, 8, 4>(x, low, lane);
        if (C > 2) merge32<uint32_t, 8, 2>(x, low, lane);
        if (C > 1) merge32<uint32_t, 8, 1>(x, low, lane);
        const uint32_t t = __shfl_sync(kFull, x[0], kk - 1);
        // |computed - true| <= e: at most 4 + 5 roundings on a path of the
        // sum, 2^-24 each of sum |q||mean|, which is at most sum |q| times
        // the largest |mean|; a shared row's q is itself a sum of `group`
        // terms.  16 + group leaves room for this bound's own roundings.
        float qa = 0.f;
        const int h0 = w.head * p.group + (a.share ? 0 : w.row0 + row);
        const uint16_t *q = a.q + int64_t(w.token) * a.q_stride + int64_t(h0) * D;
#pragma unroll 4
        for (int e = lane; e < (a.share ? p.group : 1) * (D / 8); e += 32) {
            const uint4 u = *reinterpret_cast<const uint4 *>(q + e * 8);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qa += fabsf(bf16_low_half(v[i])) + fabsf(bf16_high_half(v[i]));
        }
        qa = warp_sum(qa);
        const float e = (qa * __uint_as_float(kmax)) * (float(16 + p.group) * 5.9604645e-8f) + 1e-36f;
        const float tv = key_value(t);
        uint32_t lo = 0u, hi = kFull;           // unknown: every block is open
        if (e < -kNegInf) {
            lo = key_of(tv - 2.f * e);
            hi = key_of(tv + 2.f * e);
        }
        // the blocks at or above t - 2e, if the lists hold them all
        int total = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
            if (c < C) {
                const bool in = key[c] >= lo && key[c] != 0u;
                const uint32_t b = __ballot_sync(kFull, in);
                const int at = total + __popc(b & ((1u << lane) - 1));
                if (in && at < kMaxK) f.fin[row][at] = lists[c * p.score_rows + row].id[lane];
                total += __popc(b);
            }
        const bool slow = total != kk || __any_sync(kFull, next >= lo && next != 0u);
        __syncwarp();
        // ascending ids
        const int mine = lane < kk ? f.fin[row][lane] : 0x7fffffff;
        int before = 0;
#pragma unroll 8
        for (int j = 0; j < kk; ++j) before += __shfl_sync(kFull, mine, j) < mine;
        __syncwarp();
        if (lane < kk && !slow) f.fin[row][before] = mine;
        if (lane == 0) {
            f.slow[row] = slow;
            f.lo[row] = lo;
            f.hi[row] = hi;
            if (slow) atomicOr(&f.any_slow, 1);
        }
    }
    __syncthreads();
    // made from the same lists in every CTA of the cluster, so this is the
    // same everywhere
    if (f.any_slow == 0) return;
    for (int row = warp; row < srows; row += W) {
        if (!f.slow[row]) continue;
        const uint32_t lo = f.lo[row], hi = f.hi[row];
        int ndef = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const bool sure = i0 + lane < n && sc[row * p.nloc + i0 + lane] > hi;
            const uint32_t d = __ballot_sync(kFull, sure);
            const int at = ndef + __popc(d & ((1u << lane) - 1));
            if (sure && at < kMaxK) f.def[row][at] = b0 + i0 + lane;
            ndef += __popc(d);
        }
        if (lane == 0) f.ndef[row] = ndef;
        double q[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) q[e] = 0.0;
        const int h0 = w.head * p.group + (a.share ? 0 : w.row0 + row);
        for (int g = 0; g < (a.share ? p.group : 1); ++g) {
            const uint16_t *src =
                a.q + int64_t(w.token) * a.q_stride + int64_t(h0 + g) * D + lane * (D / 32);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) q[e] += double(__uint_as_float(uint32_t(src[e]) << 16));
        }
        // lane i holds the i-th best so far; ids come in ascending order, so
        // an equal score goes behind those that are there
        double best = 0.0;
        int id = 0, held = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const uint32_t x = i0 + lane < n ? sc[row * p.nloc + i0 + lane] : 0u;
            uint32_t open = __ballot_sync(kFull, i0 + lane < n && x >= lo && !(x > hi));
            while (open != 0) {
                const int b = b0 + i0 + __ffs(open) - 1;
                open &= open - 1;
                const double s = score_fp64<D>(a, w, b, q, lane);
                const int at = __popc(__ballot_sync(kFull, lane < held && best >= s));
                if (at < kk) {
                    const double bu = __shfl_up_sync(kFull, best, 1);
                    const int iu = __shfl_up_sync(kFull, id, 1);
                    if (lane > at) {
                        best = bu;
                        id = iu;
                    } else if (lane == at) {
                        best = s;
                        id = b;
                    }
                    held = min(held + 1, kk);
                }
            }
        }
        f.dscore[row][lane] = best;
        f.did[row][lane] = id;
        if (lane == 0) f.nd[row] = held;
    }
    cluster.sync();
    for (int row = warp; row < srows; row += W) {
        if (!f.slow[row]) continue;
        int have = 0;
        for (int c = 0; c < C; ++c) {
            const Fixed *peer = cluster.map_shared_rank(&f, c);
            const int m = peer->ndef[row];
            if (lane < m && have + lane < kMaxK) f.fin[row][have + lane] = peer->def[row][lane];
            have += m;
        }
        // merge the CTAs' lists; lane c walks over CTA c's, whose ids are
        // below those of CTA c + 1
        const Fixed *peer = cluster.map_shared_rank(&f, min(lane, C - 1));
        const int m = lane < C ? peer->nd[row] : 0;
        int at = 0;
        while (have < kk) {
            const bool there = at < m;
            const double s = there ? peer->dscore[row][at] : 0.0;
            const int b = there ? peer->did[row][at] : -1;
            double bs = s;
            int bc = there ? lane : 64;
            for (int o = 16; o > 0; o >>= 1) {
                const double os = __shfl_xor_sync(kFull, bs, o);
                const int oc = __shfl_xor_sync(kFull, bc, o);
                if (oc < 64 && (bc == 64 || os > bs || (os == bs && oc < bc))) {
                    bs = os;
                    bc = oc;
                }
            }
            if (bc == 64) break;
            if (lane == bc) {
                f.fin[row][have] = b;
                ++at;
            }
            ++have;
        }
        __syncwarp();
        // ascending ids
        const int mine = lane < kk ? f.fin[row][lane] : 0x7fffffff;
        int before = 0;
        for (int j = 0; j < kk; ++j) before += __shfl_sync(kFull, mine, j) < mine;
        __syncwarp();
        if (lane < kk) f.fin[row][before] = mine;
    }
    __syncthreads();
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
    const auto put = [&](int at, int id) {
        int pid = w.table[id];
        if (pid < 0 || pid >= a.c.num_pages) {
            report_status(a.status, kStatusBadIndex);
            pid = -1;
        }
        f.items[at] = uint16_t(id);
        f.pages[at] = pid;
    };
    if (all || a.share || w.rows == 1) {
        for (int i = tid; i < cnt; i += kThreads) {
            put(i, i == sel ? w.own : all ? i : f.fin[0][i]);
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
            // the first row to come looks the page up
            if (atomicOr(&f.masks[at], 1u << r) == 0u) put(at, id);
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

// Stage 3 and the merge.  `part` is where the cluster leaves this CTA's share
// of the outputs, [CTA][rows * D / C].
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
        uint32_t b0[NT], b1[NT];
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
            // P rounds to bf16 for the product (as in the block-major fine
            // stage); its sum l stays fp32
            b0[t] = transpose_8x8(pack_bf16x2(s[t][0], s[t][1]));
            b1[t] = transpose_8x8(pack_bf16x2(s[t][2], s[t][3]));
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
                for (int t = 0; t < NT; ++t) mma_bf16(o[t][g * 4 + j], a0, a1, a2, a3, b0[t], b1[t]);
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
    const int C = p.cluster, share = w.rows * D / C;     // C divides D
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
            const float inv = ls > 0.f || ls != ls ? __fdiv_rn(1.f, ls) : 0.f;
            *reinterpret_cast<uint32_t *>(out + i) = pack_bf16x2(x0 * inv, x1 * inv);
        } else {
            *reinterpret_cast<float2 *>(cluster.map_shared_rank(part, i / share) + w.rank * share +
                                        i % share) = make_float2(x0, x1);
            if (c < 2 * C) {            // one thread of the row for each CTA
                Fixed *peer = cluster.map_shared_rank(&f, c / 2);
                peer->pm[w.rank][r] = mx;
                peer->pl[w.rank][r] = ls;
            }
        }
    }
    if (C == 1) return;
    cluster.sync();
    for (int j = 2 * tid; j < share; j += 2 * kThreads) {
        const int i = w.rank * share + j, r = i / D;
        float mx = kNegInf;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < C) mx = fmaxf(mx, f.pm[k][r]);
        const float base = mx == kNegInf ? 0.f : mx;
        float x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < C) {
                const float2 y = *reinterpret_cast<const float2 *>(part + k * share + j);
                const float x = exp2_fast(f.pm[k][r] - base);
                x0 = fmaf(x, y.x, x0);
                x1 = fmaf(x, y.y, x1);
                ls = fmaf(x, f.pl[k][r], ls);
            }
        const float inv = ls > 0.f || ls != ls ? __fdiv_rn(1.f, ls) : 0.f;
        *reinterpret_cast<uint32_t *>(out + i) = pack_bf16x2(x0 * inv, x1 * inv);
    }
}

// CTAs per SM: three of four warps or one of twelve (eight with 16 rows,
// whose accumulators take twice the registers).
constexpr int kWarpsSmall = 4;
constexpr int warps_large(int nt) { return nt == 1 ? 12 : 8; }

template <int D, int RP, int NT, int W>
__global__ void __launch_bounds__(W * 32, W == kWarpsSmall ? (NT == 1 ? 3 : 2) : 1)
    decode_kernel(DecodeArgs a, Plan p) {
    extern __shared__ __align__(16) char smem[];
    constexpr int kThreads = W * 32;
    Fixed &f = *reinterpret_cast<Fixed *>(smem);
    List *lists = reinterpret_cast<List *>(smem + p.list_off);
    float *part = reinterpret_cast<float *>(smem + p.part_off);
    uint32_t *sc = reinterpret_cast<uint32_t *>(smem + p.main_off);
    cg::cluster_group cluster = cg::this_cluster();
    // peers may write to this CTA once all of the cluster have come this far
    auto arrived = cluster.barrier_arrive();
    const int tid = threadIdx.x;
    Job w;
    w.rank = int(blockIdx.x % unsigned(p.cluster));
    const int64_t item = blockIdx.x / unsigned(p.cluster);
    const int per = a.c.heads * p.parts;
    w.token = int32_t(item / per);
    const int hp = int(item - int64_t(w.token) * per);
    w.head = hp / p.parts;
    w.part = hp - w.head * p.parts;
    w.row0 = w.part * p.rows;
    w.rows = min(p.rows, p.group - w.row0);
    const int64_t seq = a.token_seq != nullptr ? a.token_seq[w.token] : w.token;
    w.len = a.lens[w.token];
    for (int i = tid; i < kDecodeMaxWidth / 32; i += kThreads) f.bits[i] = 0u;
    for (int i = tid; i < kMaxItems; i += kThreads) f.masks[i] = 0u;
    if (tid == 0) {
        f.kmax = 0u;
        f.any_slow = 0;
    }
    if (seq < 0 || seq >= a.seqs) {
        if (tid == 0) report_status(a.status, kStatusBadIndex);
        w.len = 0;
    }
    const int64_t most = int64_t(a.width) * a.c.page;
    if (w.len < 0 || w.len > most) {
        if (tid == 0) report_status(a.status, kStatusInvalidArg);
        w.len = w.len < 0 ? 0 : most;
    }
    w.nb = int((w.len + a.c.page - 1) / a.c.page);
    if (w.nb == 0) {                    // the same for the whole cluster
        cluster.barrier_wait(std::move(arrived));
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
    w.ne = w.nb - (a.local ? 1 : 0);
    w.kk = a.topk - (a.local ? 1 : 0);
    if (w.ne > w.kk && w.kk > 0) {
        __syncthreads();
        const int each = (w.ne + p.cluster - 1) / p.cluster;
        const int b0 = min(w.ne, w.rank * each), n = min(w.ne, b0 + each) - b0;
        score_blocks<D, RP, W>(a, p, w, f, sc, b0, n);
        __syncthreads();
        cluster.barrier_wait(std::move(arrived));
        select_blocks<D, W>(a, p, w, f, sc, lists, b0, n);
    } else {
        cluster.barrier_wait(std::move(arrived));
        __syncthreads();
    }
    make_items<W>(a, p, w, f);
    attend<D, NT, W>(a, p, w, f, part, reinterpret_cast<float *>(sc));
}

template <int D, int RP, int NT, int W>
cudaError_t launch(const DecodeArgs &a, const Plan &p, size_t smem, int64_t items, cudaStream_t st) {
    auto kernel = decode_kernel<D, RP, NT, W>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(smem));
    if (e != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, kernel, a, p);
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
    // Few items: large CTAs, clusters of up to eight of them.  Many: small
    // CTAs, three to an SM, so that some load while others select.
    const bool large = items * kMaxCluster < 3 * 152;
    const int64_t want = large ? 152 : 3 * 152;
    p.cluster = 1;
    while (p.cluster < kMaxCluster &&
           (items * p.cluster < want || (a.width + p.cluster - 1) / p.cluster > kMaxLocal))
        p.cluster *= 2;
    if (items * p.cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.nloc = (a.width + p.cluster - 1) / p.cluster;
    const int warps = large ? warps_large(p.rows > 8 ? 2 : 1) : kWarpsSmall;
    p.segs = p.score_rows >= warps ? 1 : warps / p.score_rows;
    if (p.segs > 8) p.segs = 8;
    const auto up = [](size_t x) { return (x + 15) / 16 * 16; };
    size_t off = up(sizeof(Fixed));
    p.list_off = int32_t(off);
    off = up(off + size_t(p.cluster) * p.score_rows * sizeof(List));
    p.part_off = int32_t(off);
    if (p.cluster > 1) off = up(off + size_t(p.rows) * a.c.d * 4);
    p.main_off = int32_t(off);
    const size_t scores = size_t(p.score_rows) * p.nloc * 4;
    const size_t merge = size_t(warps) * p.rows * (a.c.d + 1) * 4;
    const size_t smem = off + up(scores > merge ? scores : merge);
    return a.c.d == 64 ? dispatch<64>(a, p, large, smem, items, st)
                       : dispatch<128>(a, p, large, smem, items, st);
}

}  // namespace bsa
