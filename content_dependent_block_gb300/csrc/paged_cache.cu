// Paged key/value cache: appending tokens with the means of the blocks they
// fall in, and copying pages.  A page is one key block of the selection: its
// row of kbar is the mean of the keys it holds (page
// "sparse-attention-triton-bench", Two-stage block indexer, Stage 1).
#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 128;

// Pages a sequence's `n` new tokens can touch is at most floor(n / B) + 2, so
// sequence s owns the work items [c / B + 2 s, c' / B + 2 (s + 1)), c and c' the
// tokens before and after its own: no item list has to be made, and spare items
// return at once.
__device__ __forceinline__ int64_t first_item(const int32_t *cu, int64_t s, int32_t page) {
    return (int64_t(cu[s]) - cu[0]) / page + 2 * s;
}

// One CTA per (touched page, head).  The new rows are copied into the page
// (16 bytes per thread, 16 or 8 lanes a row), K's values are summed on the
// way, and the rows that were there before are read back, so the mean is
// always that of the page's rows [0, filled): a call can be repeated, and a
// sequence cut short and appended to again needs no correction.  Sums are
// fp32 in a fixed order.  HBM-bound: 65521 tokens, 8 heads of 128 in 84 us, 6.4
// TB/s; one token for each of 64 sequences takes the 6 us of a launch (reading
// back up to 63 rows a page and head, 16 KB, instead of keeping running sums).
template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a, int64_t n_each,
                                                          int32_t items_each) {
    constexpr int CH = D / 8;               // 16-byte chunks of a row
    constexpr int RG = kThreads / CH;       // rows per pass
    __shared__ float part[RG][D];
    const int32_t head = blockIdx.y, page = a.c.page;
    int64_t seq, lo, hi;                    // the sequence and its tokens [lo, hi)
    int64_t item;                           // which of its touched pages
    if (a.cu == nullptr) {
        seq = blockIdx.x / items_each;
        item = blockIdx.x - seq * items_each;
        lo = seq * n_each;
        hi = lo + n_each;
    } else {
        // Where cu falls, the search below may pass over sequences (and over the
        // pages of others), so each is looked at here; the grid has more
        // threads than there are sequences.
        const int64_t mine = int64_t(blockIdx.x) * kThreads + threadIdx.x;
        if (head == 0 && mine < a.seqs) {
            const int32_t c0 = a.cu[mine], c1 = a.cu[mine + 1];
            if (c0 < 0 || c1 < c0 || c1 > a.tokens) report_status(a.status, kStatusInvalidArg);
        }
        // the last sequence whose items start at or before this one: 32-way
        // search, every lane probing one sequence
        int64_t s0 = 0, s1 = a.seqs;        // in [s0, s1)
        const int lane = threadIdx.x & 31;
        while (s1 - s0 > 1) {
            const int64_t step = (s1 - s0 + 31) / 32;
            const int64_t s = s0 + lane * step;
            const bool at = s < s1 && first_item(a.cu, s, page) <= int64_t(blockIdx.x);
            const uint32_t m = __ballot_sync(0xffffffffu, at);
            const int last = m == 0 ? 0 : 31 - __clz(m);
            s0 += last * step;
            s1 = i64min(s1, s0 + step);
        }
        seq = s0;
        item = int64_t(blockIdx.x) - first_item(a.cu, seq, page);
        lo = a.cu[seq];
        hi = a.cu[seq + 1];
        if (lo < 0 || hi < lo || hi > a.tokens || item < 0) return;
    }
    if (hi == lo) return;
    const int64_t start = a.start[seq];
    const int64_t end = start + (hi - lo);  // length afterwards
    const int64_t block = int32_t(start) / page + item;
    if (start < 0 || end > int64_t(a.width) * page) {
        if (threadIdx.x == 0) report_status(a.status, kStatusInvalidArg);
        return;
    }
    if (block * page >= end) return;
    const int64_t pid = a.table[seq * a.width + block];
    if (pid < 0 || pid >= a.c.num_pages) {
        if (threadIdx.x == 0) report_status(a.status, kStatusBadIndex);
        return;
    }
    const int32_t r0 = int32_t(i64max(0, start - block * page));          // first new row
    const int32_t r1 = int32_t(i64min(page, end - block * page));         // rows filled
    const int64_t tok = lo + (block * page + r0 - start);                 // its token
    const int ch = threadIdx.x % CH, rg = threadIdx.x / CH;
    uint16_t *kp = a.c.k + ((pid * a.c.heads + head) * page) * D + ch * 8;
    uint16_t *vp = a.c.v + ((pid * a.c.heads + head) * page) * D + ch * 8;
    const uint16_t *kn = a.k + (tok - r0) * a.k_stride + int64_t(head) * D + ch * 8;
    const uint16_t *vn = a.v + (tok - r0) * a.v_stride + int64_t(head) * D + ch * 8;
    float acc[8] = {};
    constexpr int U = 4;
    for (int32_t base = rg; base < r1; base += U * RG) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = base + u * RG;
            if (r < r1) {
                x[u] = r < r0 ? *reinterpret_cast<const uint4 *>(kp + int64_t(r) * D)
                              : *reinterpret_cast<const uint4 *>(kn + r * a.k_stride);
                if (r >= r0) y[u] = *reinterpret_cast<const uint4 *>(vn + r * a.v_stride);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = base + u * RG;
            if (r < r1) {
                if (r >= r0) {
                    *reinterpret_cast<uint4 *>(kp + int64_t(r) * D) = x[u];
                    *reinterpret_cast<uint4 *>(vp + int64_t(r) * D) = y[u];
                }
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[2 * e] += bf16_low_half(w[e]);
                    acc[2 * e + 1] += bf16_high_half(w[e]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[rg][ch * 8 + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < RG; ++g) s += part[g][threadIdx.x];
        a.c.kbar[(pid * a.c.heads + head) * D + threadIdx.x] = __fdiv_rn(s, float(r1));
    }
}

// One CTA per (pair, 16 KB piece of a page's K, V and means): plain 16-byte
// copies, four in flight per thread; 2500 pages of 133 KB in 100 us, 6.6 TB/s.
constexpr int kCopyThreads = 256, kCopyVecs = 4, kCopyPiece = kCopyThreads * kCopyVecs;

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(CacheView c,
                                                                  const int32_t *pairs,
                                                                  int32_t kv_pieces,
                                                                  int32_t pieces, int32_t kv_vecs,
                                                                  int32_t mean_vecs,
                                                                  int32_t *status) {
    const int64_t pair = blockIdx.x / pieces;
    int32_t piece = blockIdx.x - int32_t(pair * pieces);
    const int64_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
    if (src < 0 || src >= c.num_pages || dst < 0 || dst >= c.num_pages) {
        if (threadIdx.x == 0) report_status(status, kStatusBadIndex);
        return;
    }
    uint4 *base;
    int32_t vecs;
    if (piece < 2 * kv_pieces) {
        base = reinterpret_cast<uint4 *>(piece < kv_pieces ? c.k : c.v);
        piece = piece < kv_pieces ? piece : piece - kv_pieces;
        vecs = kv_vecs;
    } else {
        base = reinterpret_cast<uint4 *>(c.kbar);
        piece -= 2 * kv_pieces;
        vecs = mean_vecs;
    }
    const uint4 *from = base + src * vecs;
    uint4 *to = base + dst * vecs;
    const int32_t i0 = piece * kCopyPiece + threadIdx.x;
    uint4 x[kCopyVecs];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
        if (i0 + u * kCopyThreads < vecs) x[u] = from[i0 + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
        if (i0 + u * kCopyThreads < vecs) to[i0 + u * kCopyThreads] = x[u];
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t st) {
    const int64_t n_each = a.tokens / a.seqs;
    const int64_t items_each = (n_each + a.c.page - 2) / a.c.page + 1;
    const int64_t items = a.cu != nullptr ? a.tokens / a.c.page + 2 * a.seqs
                                          : a.seqs * items_each;
    if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid{unsigned(items), unsigned(a.c.heads)};
    if (a.c.d == 64)
        append_kernel<64><<<grid, kThreads, 0, st>>>(a, n_each, int32_t(items_each));
    else
        append_kernel<128><<<grid, kThreads, 0, st>>>(a, n_each, int32_t(items_each));
    return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CacheView &c, const int32_t *pairs, int64_t count,
                              int32_t *status, cudaStream_t st) {
    const int64_t kv_vecs = int64_t(c.heads) * c.page * c.d / 8;
    const int64_t mean_vecs = int64_t(c.heads) * c.d / 4;
    const int64_t kv_pieces = (kv_vecs + kCopyPiece - 1) / kCopyPiece;
    const int64_t pieces = 2 * kv_pieces + (mean_vecs + kCopyPiece - 1) / kCopyPiece;
    if (count * pieces > 0x7fffffff) return cudaErrorInvalidConfiguration;
    copy_pages_kernel<<<dim3(unsigned(count * pieces)), kCopyThreads, 0, st>>>(
        c, pairs, int32_t(kv_pieces), int32_t(pieces), int32_t(kv_vecs), int32_t(mean_vecs),
        status);
    return cudaGetLastError();
}

}  // namespace bsa
