// The paged cache in 8 bits: appending tokens (quantised as they are written)
// with the means of the blocks they fall in, copying pages, and reading cached
// tokens back out of their pages (of either kind of cache).
//
// A row x (d channels of one token and head) becomes codes c_i = round(127 x_i
// / a), ties to even, with a = max |x_i|, and the scale a / 127 in fp32; it
// stands for c_i * scale.  Whole numbers of 8 bits with a scale for each row
// are off by a / 254 at most (Gaussian rows of 128 channels: 0.6 % of their
// size), where the 8-bit floating-point form e4m3 is off by 2^-4 of each value
// (2.6 %), for the same bytes; and they are exact in fp16, which the attention
// multiplies them in.
//
// The codes are those of the exact quotients.  127 x_i is exact in fp32 (8 + 7
// bits).  With x_i and a of 8 bits, the quotient is a half or at least 7.7e-6
// 2^(8 - e) away from one, e <= 8 the difference of their exponents, while its
// own last place there is below 2^-24 of 254 2^-e: the rounded quotient lies on
// a half only if the exact one does.  It is t r, r = 1 / a, with one correction
// by the residual t - y a (Markstein's), which reaches every quotient that is
// representable, a half among them.
//
// 65521 tokens of 8 heads of 128 are appended in 79 us, 5.1 TB/s (76 % of a plain
// copy's rate: over half of the issue slots go to the quantising), and read back
// in 68 us, 6.0 TB/s; 131072 tokens in the [heads][n][d] layout in 128 us, 6.3 TB/s.
#include "paged_common.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 128;

// Page, rows and first token of a work item that has some; false otherwise.
struct Span {
    int64_t pid, tok;         // the page, the token of row r0
    int32_t r0, r1;           // its rows in the page
};

__device__ __forceinline__ bool find_span(const int32_t *cu, int64_t seqs, int64_t tokens,
                                          int64_t items_each, const int32_t *start_of,
                                          const int32_t *table, int32_t width, int32_t page, int64_t num_pages,
                                          int32_t *status, Span *sp) {
    Item it;
    if (blockIdx.y == 0)
        check_bounds(cu, seqs, tokens, int64_t(blockIdx.x) * kThreads + threadIdx.x, status);
    if (!find_item(cu, seqs, tokens, page, items_each, blockIdx.x, &it) || it.hi == it.lo) return false;
    const int64_t start = start_of[it.seq];
    const int64_t end = start + (it.hi - it.lo);
    const int64_t block = int32_t(start) / page + it.item;
    if (start < 0 || end > int64_t(width) * page) {
        if (threadIdx.x == 0) report_status(status, kStatusInvalidArg);
        return false;
    }
    if (block * page >= end) return false;
    sp->pid = table[it.seq * width + block];
    if (sp->pid < 0 || sp->pid >= num_pages) {
        if (threadIdx.x == 0) report_status(status, kStatusBadIndex);
        return false;
    }
    sp->r0 = int32_t(i64max(0, start - block * page));
    sp->r1 = int32_t(i64min(page, end - block * page));
    sp->tok = it.lo + (block * page + sp->r0 - start);
    return true;
}

// Two numbers at a time.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    uint64_t a, b, c, r;
    float2 o;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(z.x), "f"(z.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    uint64_t a, b, r;
    float2 o;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t a, b, r;
    float2 o;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// Quantises a row of which each of the CH lanes of a group has twice 8 channels;
// every lane of the warp takes part.  Returns the row's scale, and the codes also
// as floats.
template <int CH>
__device__ __forceinline__ float quantise(const uint4 (&x)[2], uint2 (&codes)[2], float2 (&value)[8]) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_u16x2(m, w[e] & 0x7fff7fffu);
#pragma unroll
    for (int o = CH / 2; o > 0; o /= 2) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xffffu, m >> 16);
    const float a = __uint_as_float(m << 16);
    if (m == 0u || m >= 0x7f80u) {      // zeros; or an infinity or a NaN: all of the row is NaN
        codes[0] = codes[1] = make_uint2(0u, 0u);
#pragma unroll
        for (int e = 0; e < 8; ++e) value[e] = make_float2(0.f, 0.f);
        return m == 0u ? 0.f : __uint_as_float(0x7fc00000u);
    }
    // times 2^(120 - E), E the exponent's field: a comes to [2^-14, 2^-6), and
    // neither its reciprocal nor the residuals leave the normal range
    const int exponent = max(int(m >> 7), 1);
    const float factor = exponent <= 246 ? __uint_as_float(uint32_t(247 - exponent) << 23)
                                         : __uint_as_float(1u << (22 - (exponent - 247)));
    const float as = a * factor;
    float r;                            // within an ulp or two is enough for the correction
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(as));
    const float2 c2 = both(127.f * factor), r2 = both(r), n2 = both(-as);
    const float2 shift = both(12582912.f), back = both(-12582912.f);   // 1.5 * 2^23: the low byte is the code
    uint32_t q[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 t = mul2(make_float2(bf16_low_half(w[e]), bf16_high_half(w[e])), c2);
        const float2 y0 = mul2(t, r2);
        const float2 y = add2(fma2(fma2(y0, n2, t), r2, y0), shift);
        value[e] = add2(y, back);
        q[2 * e] = __float_as_uint(y.x);
        q[2 * e + 1] = __float_as_uint(y.y);
    }
    const auto bytes = [&](int e) {
        return __byte_perm(__byte_perm(q[e], q[e + 1], 0x0040), __byte_perm(q[e + 2], q[e + 3], 0x0040),
                           0x5410);
    };
    codes[0] = make_uint2(bytes(0), bytes(4));
    codes[1] = make_uint2(bytes(8), bytes(12));
    if (exponent < 32) return __fdiv_rn(a, 127.f);              // a scale that may be subnormal
    // a / 127, corrected the same way: 1 / 127 to the nearest, then the residual
    const float s0 = __fmul_rn(a, 1.f / 127.f);
    return __fmaf_rn(__fmaf_rn(s0, -127.f, a), 1.f / 127.f, s0);
}

// The i-th signed byte of eight, as a float.
__device__ __forceinline__ float code_value(const uint2 &u, int i) {
    const uint32_t w = i < 4 ? u.x : u.y;
    return float(int32_t(w << (24 - 8 * (i & 3))) >> 24);
}

// One CTA per (touched page, head): new rows are quantised into the page, and
// the mean of the page's filled rows is taken of the values that they (and the
// rows that were there, read back) stand for, in fp32 and a fixed order, so a
// call can be repeated.  A row is 4 or 8 lanes of twice 8 channels (of 8
// channels, 8 or 16 lanes share what a row costs: 97 us where this takes 79; the
// bound of six CTAs keeps the compiler from 120 registers: 89 us).
template <int D>
__global__ void __launch_bounds__(kThreads, 6) append8_kernel(Append8Args a, int64_t items_each) {
    constexpr int CH = D / 16;
    constexpr int RG = kThreads / CH;       // rows per pass
    constexpr int U = 2;
    __shared__ __align__(8) float part[RG][D];
    Span sp;
    if (!find_span(a.cu, a.seqs, a.tokens, items_each, a.start, a.table, a.width, a.c.page, a.c.num_pages,
                   a.status, &sp))
        return;
    const int32_t head = blockIdx.y, page = a.c.page;
    const int ch = threadIdx.x % CH * 8, rg = threadIdx.x / CH;  // channels ch and D / 2 + ch on
    const int64_t row0 = (sp.pid * a.c.heads + head) * page;     // of the page's scales
    const uint16_t *kn = a.k + (sp.tok - sp.r0) * a.k_stride + int64_t(head) * D + ch;
    const uint16_t *vn = a.v + (sp.tok - sp.r0) * a.v_stride + int64_t(head) * D + ch;
    int8_t *kp = a.c.k + row0 * D + ch, *vp = a.c.v + row0 * D + ch;
    float2 acc[8] = {};
    for (int32_t base = 0; base < sp.r1; base += U * RG) {       // the same passes for every warp
        uint4 x[U][2], y[U][2];
        float scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = base + u * RG + rg;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[u][i] = y[u][i] = make_uint4(0u, 0u, 0u, 0u);
                if (r >= sp.r0 && r < sp.r1) {
                    x[u][i] = *reinterpret_cast<const uint4 *>(kn + r * a.k_stride + i * (D / 2));
                    y[u][i] = *reinterpret_cast<const uint4 *>(vn + r * a.v_stride + i * (D / 2));
                } else if (r < sp.r0) {                          // codes, in y
                    const uint2 c = *reinterpret_cast<const uint2 *>(kp + r * D + i * (D / 2));
                    y[u][i].x = c.x;
                    y[u][i].y = c.y;
                    scale[u] = a.c.ks[row0 + r];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = base + u * RG + rg;
            if (base + u * RG >= sp.r1) break;                   // for the whole CTA
            uint2 kc[2], vc[2];
            float2 kv[8], vv[8];
            float ks = quantise<CH>(x[u], kc, kv);
            const uint4 old[2] = {y[u][0], y[u][1]};
            const float vs = quantise<CH>(y[u], vc, vv);
            if (r >= sp.r1) continue;
            if (r >= sp.r0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    *reinterpret_cast<uint2 *>(kp + r * D + i * (D / 2)) = kc[i];
                    *reinterpret_cast<uint2 *>(vp + r * D + i * (D / 2)) = vc[i];
                }
                if (ch == 0) {
                    a.c.ks[row0 + r] = ks;
                    a.c.vs[row0 + r] = vs;
                }
            } else {
                ks = scale[u];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint2 c = make_uint2(old[e / 4].x, old[e / 4].y);
                    kv[e] = make_float2(code_value(c, 2 * (e % 4)), code_value(c, 2 * (e % 4) + 1));
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fma2(kv[e], both(ks), acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        *reinterpret_cast<float2 *>(&part[rg][ch + e / 4 * (D / 2) + 2 * (e % 4)]) = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < RG; ++g) s += part[g][threadIdx.x];
        a.c.kbar[(sp.pid * a.c.heads + head) * D + threadIdx.x] = __fdiv_rn(s, float(sp.r1));
    }
}

// One CTA per (touched page, head): the page's rows of the sequence to their
// places in the output, 16 bytes of it per thread, codes times their scale in
// fp32 rounded once.
template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a, int64_t items_each) {
    constexpr int CH = D / 8;
    constexpr int RG = kThreads / CH;
    constexpr int U = 4;
    Span sp;
    if (!find_span(a.cu, a.seqs, a.tokens, items_each, a.start, a.table, a.width, a.page, a.num_pages, a.status,
                   &sp))
        return;
    const int32_t head = blockIdx.y;
    const int ch = threadIdx.x % CH, rg = threadIdx.x / CH;
    const int64_t row0 = (sp.pid * a.heads + head) * a.page;
    const int64_t to = (sp.tok - sp.r0) * a.token_stride + head * a.head_stride + ch * 8;
    for (int32_t base = sp.r0 + rg; base < sp.r1; base += U * RG) {
        uint4 x[2][U];
        float scale[2][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = base + u * RG;
            if (r < sp.r1) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const void *src = i == 0 ? a.k : a.v;
                    const int64_t at = (row0 + r) * D + ch * 8;
                    if (Q8) {
                        const uint2 c = *reinterpret_cast<const uint2 *>(static_cast<const int8_t *>(src) + at);
                        x[i][u].x = c.x;
                        x[i][u].y = c.y;
                        scale[i][u] = (i == 0 ? a.ks : a.vs)[row0 + r];
                    } else {
                        x[i][u] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = base + u * RG;
            if (r < sp.r1) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 y = x[i][u];
                    if (Q8) {
                        const uint2 c = make_uint2(y.x, y.y);
                        const float s = scale[i][u];
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16x2(code_value(c, 2 * e) * s, code_value(c, 2 * e + 1) * s);
                        y = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    *reinterpret_cast<uint4 *>((i == 0 ? a.k_out : a.v_out) + to + r * a.token_stride) = y;
                }
            }
        }
    }
}

// One CTA per (pair, 16 KB piece of one of a page's five parts).
constexpr int kCopyThreads = 256, kCopyVecs = 4, kCopyPiece = kCopyThreads * kCopyVecs;
struct CopyParts {
    uint4 *base[5];
    int32_t vecs[5], pieces[5];
};

__global__ void __launch_bounds__(kCopyThreads) copy_pages8_kernel(CopyParts p, int64_t num_pages,
                                                                   const int32_t *pairs,
                                                                   int32_t pieces, int32_t *status) {
    const int64_t pair = blockIdx.x / pieces;
    int32_t piece = blockIdx.x - int32_t(pair * pieces);
    const int64_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
    if (src < 0 || src >= num_pages || dst < 0 || dst >= num_pages) {
        if (threadIdx.x == 0) report_status(status, kStatusBadIndex);
        return;
    }
    uint4 *base = p.base[0];
    int32_t vecs = p.vecs[0];
#pragma unroll
    for (int i = 1; i < 5; ++i)
        if (piece >= p.pieces[i - 1]) {     // pieces[i]: those of parts 0 to i
            base = p.base[i];
            vecs = p.vecs[i];
        }
#pragma unroll
    for (int i = 3; i >= 0; --i)
        if (piece >= p.pieces[i]) {
            piece -= p.pieces[i];
            break;
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

// The grid of one CTA per (touched page, head), or false if it is too large.
bool page_grid(const int32_t *cu, int64_t tokens, int64_t seqs, int32_t page, int32_t heads, dim3 *grid,
               int64_t *items_each) {
    *items_each = (tokens / seqs + page - 2) / page + 1;
    const int64_t items = cu != nullptr ? tokens / page + 2 * seqs : seqs * *items_each;
    *grid = dim3{unsigned(items), unsigned(heads)};
    return items <= 0x7fffffff;
}

}  // namespace

cudaError_t launch_cache_append8(const Append8Args &a, cudaStream_t st) {
    dim3 grid;
    int64_t each;
    if (!page_grid(a.cu, a.tokens, a.seqs, a.c.page, a.c.heads, &grid, &each)) return cudaErrorInvalidConfiguration;
    if (a.c.d == 64)
        append8_kernel<64><<<grid, kThreads, 0, st>>>(a, each);
    else
        append8_kernel<128><<<grid, kThreads, 0, st>>>(a, each);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const ReadArgs &a, cudaStream_t st) {
    dim3 grid;
    int64_t each;
    if (!page_grid(a.cu, a.tokens, a.seqs, a.page, a.heads, &grid, &each)) return cudaErrorInvalidConfiguration;
    if (a.ks != nullptr)
        a.d == 64 ? read_kernel<64, true><<<grid, kThreads, 0, st>>>(a, each)
                  : read_kernel<128, true><<<grid, kThreads, 0, st>>>(a, each);
    else
        a.d == 64 ? read_kernel<64, false><<<grid, kThreads, 0, st>>>(a, each)
                  : read_kernel<128, false><<<grid, kThreads, 0, st>>>(a, each);
    return cudaGetLastError();
}

cudaError_t launch_copy_pages8(const Cache8View &c, const int32_t *pairs, int64_t count,
                               int32_t *status, cudaStream_t st) {
    const int64_t rows = int64_t(c.heads) * c.page, kv = rows * c.d / 16, scales = rows / 4;
    CopyParts p;
    void *const base[5] = {c.k, c.v, c.ks, c.vs, c.kbar};
    const int64_t vecs[5] = {kv, kv, scales, scales, int64_t(c.heads) * c.d / 4};
    int64_t pieces = 0;
    for (int i = 0; i < 5; ++i) {
        p.base[i] = static_cast<uint4 *>(base[i]);
        p.vecs[i] = int32_t(vecs[i]);
        pieces += (vecs[i] + kCopyPiece - 1) / kCopyPiece;
        p.pieces[i] = int32_t(pieces);
    }
    if (count * pieces > 0x7fffffff) return cudaErrorInvalidConfiguration;
    copy_pages8_kernel<<<dim3(unsigned(count * pieces)), kCopyThreads, 0, st>>>(
        p, c.num_pages, pairs, int32_t(pieces), status);
    return cudaGetLastError();
}

}  // namespace bsa
