// Attention of up to sixteen query rows to 16-key tiles of a paged cache, whose
// tiles and masks a `Source` gives, and the merge of the warps' and the
// cluster's states.  Used for single tokens that select blocks
// (paged_decode.cuh) and for few rows over whole or windowed prefixes
// (paged_attention.cu).
//
// A Source has row0 and valid, the tile's first row in the cache's [page][head]
// [row] order and its keys (1 to 16); first() and next(), which move to
// the warp's first or next tile and say whether there is one; Tile and tile(),
// what admits(tile, row, key) needs to say whether a query row sees the tile's
// key once the source has moved on.
#pragma once

#include <cooperative_groups.h>

#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace cg = cooperative_groups;

namespace bsa {
namespace {

constexpr int kMaxRows = 16;        // query rows of one cluster
constexpr int kMaxWarps = 12;
constexpr int kMaxCluster = 16;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Four codes of 8 bits as fp16 pairs: a byte plus 128 is the low byte of 1024 + it.
__device__ __forceinline__ uint32_t half_codes(uint32_t biased, uint32_t selector) {
    const uint32_t x = __byte_perm(biased, 0x64646464u, selector);
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void mma_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The power of two that brings a row of q to fp16: its largest |q| (bits of a
// bf16) to [2^14, 2^15).  Values down to 2^-31 of that keep their eight bits, and
// what is smaller is off by 2^-39 of the largest: below fp32's own rounding of the
// scores.
// `back` undoes it.
__device__ __forceinline__ float half_factor(uint32_t bits, float *back) {
    const int e = min(max(int(bits >> 7), 15), 254) - 127;
    *back = power_of_two(e - 14);
    return power_of_two(14 - e);
}

// A warp's share of the keys, 16-bit pages: lane (n8, kq) ends with the
// sums o[t][i][e] of query row t * 8 + 2 kq + (e & 1), channel n8 * 8 + (i / 4) *
// 64 + (i % 4) * 2 + (e >> 1), and the rows' m and (over its own keys) l.  K of
// the next tile is requested as soon as the scores of this one are done, V as
// soon as its product is.
template <int D, int NT, typename Source, typename QRow>
__device__ __forceinline__ void attend_keys(const CacheView &c, float scale_log2, int rows,
                                            const QRow &q_row, Source &src,
                                            float (&o)[NT][D / 16][4], float (&m)[NT][2],
                                            float (&l)[NT][2]) {
    const int lane = threadIdx.x & 31;
    const int n8 = lane >> 2, kq = lane & 3;
    uint4 q[NT][D / 32];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = t * 8 + n8;
        const uint16_t *at = q_row(min(r, rows - 1)) + kq * 8;
#pragma unroll
        for (int g = 0; g < D / 32; ++g)
            q[t][g] = r < rows ? *reinterpret_cast<const uint4 *>(at + g * 32)
                               : make_uint4(0u, 0u, 0u, 0u);
    }
    uint4 kr[2][D / 32], vr[4][D / 64];
    const auto load_k = [&] {
        const uint16_t *kp = c.k + (src.row0 + n8) * D + kq * 8;
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
            kr[0][g] = __ldg(reinterpret_cast<const uint4 *>(kp + g * 32));
            kr[1][g] = __ldg(reinterpret_cast<const uint4 *>(kp + 8 * D + g * 32));
        }
    };
    const auto load_v = [&](int64_t row) {
        const uint16_t *vp = c.v + (row + 2 * kq) * D + n8 * 8;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
            vr[0][g] = __ldg(reinterpret_cast<const uint4 *>(vp + g * 64));
            vr[1][g] = __ldg(reinterpret_cast<const uint4 *>(vp + D + g * 64));
            vr[2][g] = __ldg(reinterpret_cast<const uint4 *>(vp + 8 * D + g * 64));
            vr[3][g] = __ldg(reinterpret_cast<const uint4 *>(vp + 9 * D + g * 64));
        }
    };
    bool more = src.first();
    if (more) {
        load_k();
        load_v(src.row0);
    }
    while (more) {
        const int now_valid = src.valid;
        const typename Source::Tile tile = src.tile();
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
        more = src.next();
        if (more) load_k();             // in flight during the softmax and P V
        uint32_t b0[NT], b1[NT], r0[NT], r1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float corr[2];
            bool moved = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = t * 8 + 2 * kq + e;
                const bool in0 = n8 < now_valid && src.admits(tile, row, n8);
                const bool in1 = n8 + 8 < now_valid && src.admits(tile, row, n8 + 8);
                // s[e]: key n8, s[2 + e]: key n8 + 8
                s[t][e] = in0 ? s[t][e] * scale_log2 : kNegInf;
                s[t][2 + e] = in1 ? s[t][2 + e] * scale_log2 : kNegInf;
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
            // in bf16: off by 2^-17 of p at most (of one bf16 value, 2^-8)
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
        if (more) load_v(src.row0);
    }
}

// The same over 8-bit pages, in fp16: codes are exact there, q is after a power
// of two for each row, and a key's scales multiply its score and its weight
// in fp32.  Weights w = p vs 2^(12 - E) enter the product, E the exponent of
// the largest vs that the row has admitted so far (its sums follow when it
// grows): fp16 rounds them to 2^-11 of themselves, those below 2^-26 of the
// largest to 2^-37 of that.  Each row has its own E: a key that it does not admit
// may have any scale, also where other rows of the tile admit it.  Scales that
// are not finite do not count.  A masked key's weight is 0, and 0 times a code
// is 0.  E seldom grows, so a vote passes over the reduction that finds it.
// Lane (n8, kq) ends with channel n8 * D / 8 + 2 i + (e >> 1) in o[t][i][e].
template <int D, int NT, typename Source, typename QRow>
__device__ __forceinline__ void attend_keys8(const CacheView &c, const float *ks_ptr,
                                             const float *vs_ptr, float scale_log2, int rows,
                                             const QRow &q_row, Source &src,
                                             float (&o)[NT][D / 16][4], float (&m)[NT][2],
                                             float (&l)[NT][2]) {
    constexpr int KV = D / 64;          // 16-byte loads of a key's row by its four lanes
    constexpr int VW = D / 32;          // words of a key that a lane has of V
    const int8_t *const kc = reinterpret_cast<const int8_t *>(c.k);
    const int8_t *const vc = reinterpret_cast<const int8_t *>(c.v);
    const int lane = threadIdx.x & 31;
    const int n8 = lane >> 2, kq = lane & 3;
    uint32_t q[NT][KV][8];
    float back[NT][2];                  // times the rows' scores
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = t * 8 + n8;
        const uint16_t *at = q_row(min(r, rows - 1)) + kq * 16;
        uint4 x[KV][2];
        uint32_t top = 0u;
#pragma unroll
        for (int g = 0; g < KV; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[g][i] = r < rows ? *reinterpret_cast<const uint4 *>(at + g * 64 + i * 8)
                                   : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j) top = __vmaxu2(top, word(x[g][i], j) & 0x7fff7fffu);
            }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        float un;
        const float to = half_factor(top, &un);
        un *= scale_log2;
        back[t][0] = __shfl_sync(kFull, un, 8 * kq);
        back[t][1] = __shfl_sync(kFull, un, 8 * kq + 4);
#pragma unroll
        for (int g = 0; g < KV; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t y = word(x[g][j / 4], j % 4);
                q[t][g][j] = pack_half2(bf16_low_half(y) * to, bf16_high_half(y) * to);
            }
    }
    uint4 kr[2][KV];
    uint32_t vr[4][VW];
    float ks[2], vs[2];
    const auto load_k = [&] {
        const int8_t *kp = kc + (src.row0 + n8) * D + kq * 16;
#pragma unroll
        for (int g = 0; g < KV; ++g) {
            kr[0][g] = __ldg(reinterpret_cast<const uint4 *>(kp + g * 64));
            kr[1][g] = __ldg(reinterpret_cast<const uint4 *>(kp + 8 * D + g * 64));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ks[i] = __ldg(ks_ptr + src.row0 + n8 + 8 * i);
            vs[i] = __ldg(vs_ptr + src.row0 + n8 + 8 * i);
        }
    };
    const auto load_v = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int8_t *vp = vc + (row + 2 * kq + (i & 1) + 8 * (i >> 1)) * D + n8 * (D / 8);
            if (D == 64) {
                const uint2 x = __ldg(reinterpret_cast<const uint2 *>(vp));
                vr[i][0] = x.x;
                vr[i][1] = x.y;
            } else {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(vp));
#pragma unroll
                for (int j = 0; j < VW; ++j) vr[i][j] = word(x, j);
            }
        }
    };
    int big[NT][2];                     // E of the lane's rows
#pragma unroll
    for (int t = 0; t < NT; ++t) big[t][0] = big[t][1] = -110;
    bool more = src.first();
    if (more) {
        load_k();
        load_v(src.row0);
    }
    while (more) {
        const int now_valid = src.valid;
        const typename Source::Tile tile = src.tile();
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int g = 0; g < KV; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x0 = word(kr[0][g], j) ^ 0x80808080u, x1 = word(kr[1][g], j) ^ 0x80808080u;
                const uint32_t a0 = half_codes(x0, 0x4140), a2 = half_codes(x0, 0x4342);
                const uint32_t a1 = half_codes(x1, 0x4140), a3 = half_codes(x1, 0x4342);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    mma_half(s[t], a0, a1, a2, a3, q[t][g][2 * j], q[t][g][2 * j + 1]);
            }
        float kn[2], vn[2];
        int of[2];                      // exponents of vs, of which E is the largest
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kn[i] = ks[i];
            vn[i] = vs[i];
            of[i] = fabsf(vn[i]) < -kNegInf ? int(__float_as_uint(fabsf(vn[i])) >> 23) - 127 : -127;
        }
        more = src.next();
        if (more) load_k();             // in flight during the softmax and P V
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float corr[2], grow[2] = {1.f, 1.f}, x[4];
            bool in[2][2], moved = false, larger = false;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    in[e][i] = n8 + 8 * i < now_valid && src.admits(tile, t * 8 + 2 * kq + e, n8 + 8 * i);
                    larger |= in[e][i] && of[i] > big[t][e];
                }
            if (__any_sync(kFull, larger)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    int top = max(in[e][0] ? of[0] : -127, in[e][1] ? of[1] : -127);
                    top = max(top, __shfl_xor_sync(kFull, top, 4));
                    top = max(top, __shfl_xor_sync(kFull, top, 8));
                    top = max(top, __shfl_xor_sync(kFull, top, 16));
                    if (top > big[t][e]) {
                        grow[e] = power_of_two(max(big[t][e] - top, -126));
                        big[t][e] = top;
                        moved = true;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool in0 = in[e][0], in1 = in[e][1];
                const float vf = power_of_two(12 - big[t][e]);
                // s[e]: key n8, s[2 + e]: key n8 + 8; the product of the
                // factors first, which is nearer to 1 than either
                s[t][e] = in0 ? s[t][e] * (kn[0] * back[t][e]) : kNegInf;
                s[t][2 + e] = in1 ? s[t][2 + e] * (kn[1] * back[t][e]) : kNegInf;
                float y = fmaxf(s[t][e], s[t][2 + e]);
                y = fmaxf(y, __shfl_xor_sync(kFull, y, 4));
                y = fmaxf(y, __shfl_xor_sync(kFull, y, 8));
                y = fmaxf(y, __shfl_xor_sync(kFull, y, 16));
                const float mn = fmaxf(m[t][e], y);
                const float base = mn == kNegInf ? 0.f : mn;     // nothing admitted yet
                moved |= mn != m[t][e];
                corr[e] = exp2_fast(m[t][e] - base);
                m[t][e] = mn;
                s[t][e] = exp2_fast(s[t][e] - base);
                s[t][2 + e] = exp2_fast(s[t][2 + e] - base);
                l[t][e] = l[t][e] * corr[e] + (s[t][e] + s[t][2 + e]);
                corr[e] *= grow[e];
                x[e] = in0 ? s[t][e] * (vn[0] * vf) : 0.f;
                x[2 + e] = in1 ? s[t][2 + e] * (vn[1] * vf) : 0.f;
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
            b0[t] = transpose_8x8(pack_half2(x[0], x[1]));
            b1[t] = transpose_8x8(pack_half2(x[2], x[3]));
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            const uint32_t w0 = vr[0][j] ^ 0x80808080u, w1 = vr[1][j] ^ 0x80808080u;
            const uint32_t w2 = vr[2][j] ^ 0x80808080u, w3 = vr[3][j] ^ 0x80808080u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // bytes 2 h and 2 h + 1 of two keys each
                const uint32_t y0 = __byte_perm(w0, w1, h == 0 ? 0x5140 : 0x7362);
                const uint32_t y1 = __byte_perm(w2, w3, h == 0 ? 0x5140 : 0x7362);
                const uint32_t a0 = half_codes(y0, 0x4140), a1 = half_codes(y0, 0x4342);
                const uint32_t a2 = half_codes(y1, 0x4140), a3 = half_codes(y1, 0x4342);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_half(o[t][2 * j + h], a0, a1, a2, a3, b0[t], b1[t]);
            }
        }
        if (more) load_v(src.row0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float un[2] = {power_of_two(big[t][0] - 12), power_of_two(big[t][1] - 12)};
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][i][e] *= un[e & 1];
    }
}

// Scratch of the merge, in shared memory.
struct Merge {
    float wm[kMaxWarps][kMaxRows], wl[kMaxWarps][kMaxRows];
    float pm[kMaxCluster][kMaxRows], pl[kMaxCluster][kMaxRows];   // of every CTA
    uint32_t redo;                   // rows whose output is not finite; zero before
    float redo_m[kMaxRows], redo_inv[kMaxRows];
};

struct Gang {
    int32_t cluster, takers;         // CTAs, and those that write outputs (a power of two)
    int32_t rank, rows, rows_cap;    // this CTA's, its rows, room for rows
};

template <int D, int NT>
__device__ __forceinline__ void clear_state(float (&o)[NT][D / 16][4], float (&m)[NT][2],
                                            float (&l)[NT][2]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
        m[t][0] = m[t][1] = kNegInf;
        l[t][0] = l[t][1] = 0.f;
    }
}

// Merges the warps' states over the CTA and then over the cluster, and writes
// the rows that out_row(r) points to.  `part` is where the cluster leaves this
// CTA's share of the outputs, [CTA][rows][D / takers]; `po` holds the warps'
// outputs, [W][rows_cap][D + 1], or W + 1 rows of D.  alone(r, m, po) leaves the
// sums of row r, taken without products with masked keys, in po + W * D.
template <int D, int NT, int W, bool Q8, typename OutRow, typename Alone>
__device__ __forceinline__ void merge_states(const Gang &g, Merge &f, const float (&o)[NT][D / 16][4],
                                             const float (&m)[NT][2], const float (&l)[NT][2],
                                             float *part, float *po, const OutRow &out_row,
                                             const Alone &alone) {
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int kThreads = W * 32;
    constexpr int PS = D + 1;           // row stride of the warps' outputs
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n8 = lane >> 2, kq = lane & 3;
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
            if (r < g.rows) {
                if (n8 == 0) {
                    f.wm[warp][r] = m[t][e];
                    f.wl[warp][r] = x;
                }
                float *dst = po + (warp * g.rows_cap + r) * PS + n8 * (Q8 ? D / 8 : 8);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int c = Q8 ? 2 * i : (i / 4) * 64 + (i % 4) * 2;
                    dst[c] = o[t][i][e];
                    dst[c + 1] = o[t][i][2 + e];
                }
            }
        }
    __syncthreads();
    const int C = g.cluster, share = D / g.takers;      // channels of each that writes
    const int shift_c = 31 - __clz(share);
    // a row with no key to attend to is zero
    const auto put = [&](int c, int r, float mx, float ls, float x0, float x1) {
        const float inv = ls > 0.f || ls != ls ? __fdiv_rn(1.f, ls) : 0.f;
        x0 *= inv;
        x1 *= inv;
        *reinterpret_cast<uint32_t *>(out_row(r) + c) = pack_bf16x2(x0, x1);
        // a sum that is not a number comes from the row's own scores, and 8-bit
        // codes are finite
        if (!Q8 && ls == ls && !(fabsf(x0) < -kNegInf && fabsf(x1) < -kNegInf)) {
            f.redo_m[r] = mx;
            f.redo_inv[r] = inv;
            atomicOr(&f.redo, 1u << r);
        }
    };
    for (int i = 2 * tid; i < g.rows * D; i += 2 * kThreads) {
        const int r = i / D, c = i % D;
        float mx = kNegInf;
#pragma unroll
        for (int k = 0; k < W; ++k) mx = fmaxf(mx, f.wm[k][r]);
        const float base = mx == kNegInf ? 0.f : mx;
        float x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float x = exp2_fast(f.wm[k][r] - base);
            x0 = fmaf(x, po[(k * g.rows_cap + r) * PS + c], x0);
            x1 = fmaf(x, po[(k * g.rows_cap + r) * PS + c + 1], x1);
            ls = fmaf(x, f.wl[k][r], ls);
        }
        if (C == 1) {
            put(c, r, mx, ls, x0, x1);
        } else {
            float *dst = cluster.map_shared_rank(part, c >> shift_c);
            *reinterpret_cast<float2 *>(dst + ((g.rank * g.rows + r) << shift_c) + (c & (share - 1))) =
                make_float2(x0, x1);
            if (c < 2 * g.takers) {     // one thread of the row for each
                Merge *peer = cluster.map_shared_rank(&f, c / 2);
                peer->pm[g.rank][r] = mx;
                peer->pl[g.rank][r] = ls;
            }
        }
    }
    if (C > 1) {
        cluster.sync();
        if (g.rank >= g.takers) return;
        for (int j = 2 * tid; j < g.rows * share; j += 2 * kThreads) {
            const int r = j >> shift_c, c = g.rank * share + (j & (share - 1));
            float mx = kNegInf;
#pragma unroll 4
            for (int k = 0; k < C; ++k) mx = fmaxf(mx, f.pm[k][r]);
            const float base = mx == kNegInf ? 0.f : mx;
            float x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll 4
            for (int k = 0; k < C; ++k) {
                const float2 y = *reinterpret_cast<const float2 *>(part + k * g.rows * share + j);
                const float x = exp2_fast(f.pm[k][r] - base);
                x0 = fmaf(x, y.x, x0);
                x1 = fmaf(x, y.y, x1);
                ls = fmaf(x, f.pl[k][r], ls);
            }
            put(c, r, mx, ls, x0, x1);
        }
    }
    if constexpr (Q8) return;
    __syncthreads();
    if (f.redo == 0u) return;
    for (int r = 0; r < g.rows; ++r) {
        if (!(f.redo >> r & 1u)) continue;
        alone(r, f.redo_m[r], po);
        for (int c = tid; c < share; c += kThreads) {
            const float x = po[W * D + g.rank * share + c] * f.redo_inv[r];
            out_row(r)[g.rank * share + c] = f32_to_bf16_bits(x);
        }
    }
}


}  // namespace
}  // namespace bsa
