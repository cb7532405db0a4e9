// New tokens over the paged cache, few query rows at a time: the last token of
// each sequence, or a handful of drafted ones.  out_i = sum_j softmax_j(scale
// q_i . k_j) v_j over the keys j that token i sees: all before it, or with a
// window the last W and the first few (sinks), or in a tree of drafted tokens
// the prefix and its ancestors.
//
// One thread-block cluster of C CTAs serves a tile of up to 16 query rows (the
// heads that share a cache head, times as many tokens of one sequence as fit).
// The 16-key tiles of the keys that some row sees are dealt to the cluster's
// warps, which keep an online softmax each (paged_tiles.cuh); only tiles at
// the edge of what is seen are masked.  The states are merged over the warps
// and, through shared memory, over the cluster: no workspace, so captured
// graphs share nothing.
//
// Bound: memory (each visible K and V row once).  mma.sync of 16 x 8 x 16
// carries it, as in paged_decode.cuh: the rows are far below a tcgen05 tile's.
// Measured: one token for each of 64 sequences, 32 heads over 8, d 128, a window of
// 4096 and four sinks: 196 us, 5.5 TB/s (82 % of a plain copy's rate); over
// 8-bit pages 125 us, 4.4 TB/s.
#pragma once

#include <algorithm>
#include <atomic>

#include "bsa_device.cuh"
#include "bsa_internal.h"
#include "paged_common.cuh"
#include "paged_tiles.cuh"

namespace bsa {
namespace {

constexpr int kMaxSmem = 227 * 1024;

struct RowsPlan {
    int64_t items_each;   // tiles of a sequence, where all have as many tokens
    int32_t cluster, takers;
    int32_t size;         // tokens of a tile
    int32_t rows_cap;     // size times the heads of a cache head
    int32_t part_off, main_off;
};

struct RowsFixed {
    Merge merge;
    Sight sight[kMaxRows];
};

// The warp's tiles of the keys that the rows may see.
struct Seen {
    struct Tile {
        int32_t key0;
        bool full;                    // every row sees all of it
    };
    const AttentionArgs &a;
    const Reach &r;
    const RowsFixed &f;
    const int32_t *table;
    int head, step, at, units, gap, sinks, shift;
    int32_t lo_max, hi_min;
    int ids = -1, count = 32;         // this lane's page of a batch of 32 tiles, tiles of it used
    int64_t row0 = 0;
    int32_t valid = 0, key0 = 0;
    __device__ __forceinline__ Seen(const AttentionArgs &args, const Reach &reach, const RowsFixed &fixed,
                                    int head_, int rows, int first, int step_)
        : a(args), r(reach), f(fixed), head(head_), step(step_), at(first) {
        table = a.table + r.seq * a.width;
        shift = 31 - __clz(a.c.page);
        // tiles [0, s) hold sinks, tiles [gap + s, ...) the window
        const int s = min((r.sinks_end + 15) / 16, r.first / 16);
        gap = r.first / 16 - s;
        sinks = s;
        units = (r.end + 15) / 16 - gap;
        lo_max = 0;
        hi_min = 0x7fffffff;
        for (int i = 0; i < rows; ++i) {
            lo_max = max(lo_max, f.sight[i].lo);
            hi_min = min(hi_min, f.sight[i].hi);
        }
    }
    __device__ __forceinline__ int tile_of(int u) const { return u < sinks ? u : u + gap; }
    // the next of the warp's tiles whose page is there
    __device__ __forceinline__ bool next() {
        for (;; ) {
            if (count == 32) {
                const int u = at + int(threadIdx.x & 31) * step;
                ids = -1;
                if (u < units) {
                    ids = table[tile_of(u) * 16 >> shift];
                    if (ids < 0 || ids >= a.c.num_pages) {
                        report_status(a.status, kStatusBadIndex);
                        ids = -1;
                    }
                }
                count = 0;
            }
            if (at >= units) return false;
            const int64_t pid = __shfl_sync(kFull, ids, count);
            key0 = tile_of(at) * 16;
            at += step;
            ++count;
            if (pid < 0) continue;
            valid = min(16, r.end - key0);
            row0 = (pid * a.c.heads + head) * a.c.page + (key0 & (a.c.page - 1));
            return true;
        }
    }
    __device__ __forceinline__ bool first() { return next(); }
    __device__ __forceinline__ Tile tile() const {
        return {key0, key0 >= lo_max && key0 <= hi_min - 16};
    }
    __device__ __forceinline__ bool sees(int row, int32_t key) const {
        const Sight &s = f.sight[row];
        if (key < s.hi && (key >= s.lo || key < a.sinks)) return true;
        const int64_t bit = key - r.start;
        return bit >= 0 && bit < 64 && ((s.tree >> bit) & 1u) != 0;
    }
    __device__ __forceinline__ bool admits(const Tile &t, int row, int key) const {
        return t.full || sees(row, t.key0 + key);
    }
};

template <int NT>
constexpr int rows_warps_large() { return NT == 1 ? 12 : 8; }
constexpr int kRowsWarpsSmall = 4;
// (8-bit pages at d 128 leave registers for a fourth: 131 us for 64 windows of
// 4096 keys where three take 151; 125 now)
constexpr int rows_ctas_per_sm(int d, int nt, bool q8) { return nt == 2 ? 2 : d == 64 || q8 ? 4 : 3; }

template <int D, int NT, int W, bool Q8>
__global__ void __launch_bounds__(W * 32, W == kRowsWarpsSmall ? rows_ctas_per_sm(D, NT, Q8) : 1)
    attention_rows_kernel(AttentionArgs a, RowsPlan p) {
    extern __shared__ __align__(16) char smem[];
    RowsFixed &f = *reinterpret_cast<RowsFixed *>(smem);
    float *part = reinterpret_cast<float *>(smem + p.part_off);
    float *po = reinterpret_cast<float *>(smem + p.main_off);
    const int tid = threadIdx.x;
    const int rank = int(blockIdx.x % unsigned(p.cluster));
    const unsigned cluster = blockIdx.x / unsigned(p.cluster);
    const int64_t number = cluster / unsigned(a.c.heads);
    const int head = int(cluster - unsigned(number) * unsigned(a.c.heads));
    const int group = a.q_heads / a.c.heads;
    check_bounds(a.cu, a.seqs, a.tokens, int64_t(blockIdx.x) * (W * 32) + tid, a.status);
    Reach r;
    // the whole cluster leaves together
    if (!find_reach(a, p.size, p.items_each, number, rank == 0 && tid == 0, &r)) return;
    const int rows = r.nt * group;
    if (tid < kMaxRows) {
        const int row = min(tid, rows - 1);                    // rows that are not there see what the last sees
        f.sight[tid] = sight_of(a, r.start, r.lo, r.n, r.t0 + row / group);
    }
    if (tid == 0) f.merge.redo = 0u;
    __syncthreads();
    const auto token_row = [&](int row, int64_t stride) {
        const int t = row / group;
        return (r.lo + r.t0 + t) * stride + int64_t(head * group + row - t * group) * D;
    };
    const auto q_row = [&](int row) { return a.q + token_row(row, a.q_stride); };
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    clear_state<D, NT>(o, m, l);
    const int first = rank * W + (tid >> 5), step = p.cluster * W;
    Seen src(a, r, f, head, rows, first, step);
    if constexpr (Q8)
        attend_keys8<D, NT>(a.c, a.ks, a.vs, a.scale_log2, rows, q_row, src, o, m, l);
    else
        attend_keys<D, NT>(a.c, a.scale_log2, rows, q_row, src, o, m, l);
    // peers may be written to once all have started
    if (p.cluster > 1) cg::this_cluster().sync();
    merge_states<D, NT, W, Q8>(
        Gang{p.cluster, p.takers, rank, rows, p.rows_cap}, f.merge, o, m, l, part, po,
        [&](int row) { return a.out + token_row(row, int64_t(a.q_heads) * D); },
        // A row whose output is not finite, again and alone: masked keys had
        // weight 0, which must not count where a value is infinite or NaN.
        [&](int row, float mx, float *sum) {
            constexpr int E = D / 32;
            const int lane = tid & 31, warp = tid >> 5;
            const uint16_t *qr = q_row(row) + lane * E;
            float q[E], acc[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                q[e] = __uint_as_float(uint32_t(qr[e]) << 16);
                acc[e] = 0.f;
            }
            Seen all(a, r, f, head, rows, warp, W);
            while (all.next())
                for (int j = 0; j < all.valid; ++j) {
                    if (!all.sees(row, all.key0 + j)) continue;
                    const int64_t at = (all.row0 + j) * D + lane * E;
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        s = fmaf(q[e], __uint_as_float(uint32_t(a.c.k[at + e]) << 16), s);
                    const float x = exp2_fast(warp_sum(s) * a.scale_log2 - (mx == kNegInf ? 0.f : mx));
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[e] = fmaf(x, __uint_as_float(uint32_t(a.c.v[at + e]) << 16), acc[e]);
                }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) sum[warp * D + lane * E + e] = acc[e];
            __syncthreads();
            for (int c = tid; c < D; c += W * 32) {
                float x = 0.f;
                for (int k = 0; k < W; ++k) x += sum[k * D + c];
                sum[W * D + c] = x;
            }
            __syncthreads();
        });
}

// Clusters of 5 to 16 CTAs that the card holds with one CTA to an SM (as for
// paged_decode.cuh's kernel).
constexpr int kRowsFewItems = 28;
constexpr int8_t kRowsClustersFit[kMaxCluster + 1] = {0, 0, 0, 0, 0, 28, 23, 15, 15, 15, 13, 8, 8, 7, 7, 7, 7};

template <int D, int NT, int W, bool Q8>
cudaError_t launch_rows(const AttentionArgs &a, const RowsPlan &p, size_t smem, int64_t items,
                        cudaStream_t st) {
    auto kernel = attention_rows_kernel<D, NT, W, Q8>;
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

template <bool Q8>
cudaError_t launch_rows_form(const AttentionArgs &a, cudaStream_t st) {
    const int group = a.q_heads / a.c.heads;                  // at most kMaxRows
    const int64_t mean = (a.tokens + a.seqs - 1) / a.seqs;
    RowsPlan p;
    p.size = int32_t(std::min<int64_t>(kMaxRows / group, mean));
    p.rows_cap = p.size * group;
    const int nt = p.rows_cap > 8 ? 2 : 1;
    p.items_each = (a.tokens / a.seqs + p.size - 1) / p.size;
    const int64_t tiles = a.cu != nullptr ? a.tokens / p.size + 2 * a.seqs : a.seqs * p.items_each;
    const int64_t items = tiles * a.c.heads;
    // Few items: large CTAs, one to an SM, in the largest clusters that fit the
    // card all at once, no more warps than have two 16-key tiles each.  Many:
    // small CTAs, several to an SM, in clusters of C.  A CTA costs what its
    // keys do and about as much as 600 keys besides.  With a window the keys
    // are much the same everywhere, and the turns that the card takes count;
    // without one lengths are ragged, of which the host knows only the table's
    // width, and what counts is the longest CTA and the sum of all.  (4096 keys,
    // 64 sequences over 8 heads: C 1, 2, 4, 8: 228, 197, 189, 228 us; 20: 98, 66,
    // 74, 85 us.  24 sequences of 4096 to 32768 keys over 8: 668, 386, 314, 303.)
    const bool large = items <= kRowsFewItems;
    const int warps = large ? (nt == 1 ? rows_warps_large<1>() : rows_warps_large<2>()) : kRowsWarpsSmall;
    int64_t keys = int64_t(a.width) * a.c.page;
    if (a.window > 0) keys = std::min<int64_t>(keys, int64_t(a.window) + a.sinks + p.size);
    p.cluster = 1;
    if (large) {
        const int64_t pairs = keys / 32;
        p.cluster = kMaxCluster;
        while (p.cluster > 5 && kRowsClustersFit[p.cluster] < items) --p.cluster;
        while (p.cluster > 1 && (p.cluster - 1) * warps >= pairs) --p.cluster;
    } else {
        const int64_t slots = 152 * rows_ctas_per_sm(a.c.d, nt, Q8), besides = 600;
        int64_t least = INT64_MAX;
        for (int c = 1; c <= 8; c *= 2) {
            const int64_t one = keys / c + besides;
            const int64_t cost = a.window > 0 ? (items * c + slots - 1) / slots * one
                                              : std::max(one, items * (keys * 3 / 5 + besides * c) / slots);
            if (cost < least) {
                least = cost;
                p.cluster = c;
            }
        }
    }
    if (items * p.cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.takers = p.cluster >= 8 ? 8 : p.cluster >= 4 ? 4 : p.cluster >= 2 ? 2 : 1;
    const auto up = [](size_t x) { return (x + 15) / 16 * 16; };
    size_t off = up(sizeof(RowsFixed));
    p.part_off = int32_t(off);
    if (p.cluster > 1) off = up(off + size_t(p.cluster) * p.rows_cap * (a.c.d / p.takers) * 4);
    p.main_off = int32_t(off);
    const size_t merge = size_t(warps) * p.rows_cap * (a.c.d + 1) * 4;
    const size_t alone = size_t(warps + 1) * a.c.d * 4;
    const size_t smem = off + up(std::max(merge, alone));
    if (a.c.d == 64) {
        if (nt == 1)
            return large ? launch_rows<64, 1, rows_warps_large<1>(), Q8>(a, p, smem, items, st)
                         : launch_rows<64, 1, kRowsWarpsSmall, Q8>(a, p, smem, items, st);
        return large ? launch_rows<64, 2, rows_warps_large<2>(), Q8>(a, p, smem, items, st)
                     : launch_rows<64, 2, kRowsWarpsSmall, Q8>(a, p, smem, items, st);
    }
    if (nt == 1)
        return large ? launch_rows<128, 1, rows_warps_large<1>(), Q8>(a, p, smem, items, st)
                     : launch_rows<128, 1, kRowsWarpsSmall, Q8>(a, p, smem, items, st);
    return large ? launch_rows<128, 2, rows_warps_large<2>(), Q8>(a, p, smem, items, st)
                 : launch_rows<128, 2, kRowsWarpsSmall, Q8>(a, p, smem, items, st);
}

}  // namespace
}  // namespace bsa
