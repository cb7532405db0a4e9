// Rotary positions on the heads of q and k, forward and backward.
//
// Pair i of a token at position p turns by the angle t = p f_i:
//   x_a' = m (x_a cos t - x_b sin t),  x_b' = m (x_b cos t + x_a sin t),
// (a, b) = (i, i + rot/2) or, interleaved, (2i, 2i + 1); channels from rot on
// are copied.  The gradient is the same map with -t.
//
// Angles.  A position of 10^6 times an fp32 frequency is off by up to 0.06
// rad, and fp64 products and sines for every pair would cost more than the
// memory traffic.  So the plan holds each frequency as turns per position in
// 64-bit fixed point (units of 2^-64 turns): the integer product with the
// position wraps modulo 2^64, which is modulo one turn, exactly.  Its top 32
// bits are split into the nearest quarter turn and a rest of at most an eighth
// of a turn either way; sine and cosine of the rest are their Taylor series
// (to x^11 and x^10: the terms left out are below 2^-29 and 2^-28 of the
// result).  The angle is off by 2^-25 of the rest, by 2^-32 of a turn, and by the
// position times the rounding of the table, which comes from fp64 frequencies:
// at most 2^-52 of all the p f / 2 pi turns (f = 1: 2^-31 of a turn at position
// 2^23, 2^-23 at 2^31).
//
// HBM-bound: x is read once and out written once (2 x 32 heads x 32768 x 128
// bf16: 161 us, 6.7 TB/s, 98 % of a plain copy's rate).  A thread owns V pairs
// of one token (two 16-byte vectors) and walks over the heads with them, so
// the sines are computed once per token and pair and shared by its heads.
#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void turn(uint64_t freq, int64_t pos, float factor, float sign,
                                     float &c, float &s) {
    const uint32_t t = uint32_t((freq * uint64_t(pos)) >> 32);
    const uint32_t quarter = (t + (1u << 29)) >> 30;
    const float x = float(int32_t(t - (quarter << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float z = x * x;
    float u = fmaf(z, -2.5052108e-8f, 2.7557319e-6f);       // 1/11!, 1/9!
    u = fmaf(z, u, -1.9841270e-4f);
    u = fmaf(z, u, 8.3333333e-3f);
    u = fmaf(z, u, -0.16666667f);
    const float sn = fmaf(x * z, u, x);
    float v = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);       // 1/10!, 1/8!
    v = fmaf(z, v, -1.3888889e-3f);
    v = fmaf(z, v, 4.1666667e-2f);
    v = fmaf(z, v, -0.5f);
    const float cs = fmaf(z, v, 1.f);
    // quarter 1: (cos, sin) -> (-sin, cos), and so on
    c = quarter & 1u ? sn : cs;
    s = quarter & 1u ? cs : sn;
    c = __uint_as_float(__float_as_uint(c) ^ (((quarter + 1u) & 2u) << 30));
    s = __uint_as_float(__float_as_uint(s) ^ ((quarter & 2u) << 30));
    c *= factor;
    s *= factor * sign;
}

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {          // bf16: 8 channels in 16 bytes
    static constexpr int V = 8;
    static __device__ __forceinline__ void load(uint4 u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_low_half(w[i]);
            x[2 * i + 1] = bf16_high_half(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 store(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                          pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ float get(uint16_t u) {
        return __uint_as_float(uint32_t(u) << 16);
    }
    static __device__ __forceinline__ uint16_t put(float x) { return f32_to_bf16_bits(x); }
};
template <>
struct Vec<float> {             // fp32: 4 channels in 16 bytes
    static constexpr int V = 4;
    static __device__ __forceinline__ void load(uint4 u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 store(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float get(float u) { return u; }
    static __device__ __forceinline__ float put(float x) { return x; }
};

// x / d, and x becomes the remainder; 64-bit division is some 150 instructions,
// which only a tensor of more than 2^32 threads pays.
__device__ __forceinline__ int64_t divide(int64_t &x, int64_t d, bool small) {
    if (small) {
        const uint32_t q = uint32_t(x) / uint32_t(d);
        x = uint32_t(x) - q * uint32_t(d);
        return q;
    }
    const int64_t q = x / d;
    x -= q * d;
    return q;
}

// Where thread t works: index of its vector or task (fastest), batch, token
// and chunk of heads, the last two in the order of the output's layout.
struct Place {
    int32_t task, chunk;
    int64_t i, b;
};
__device__ __forceinline__ Place place_of(const RopeArgs &a, int64_t t, int32_t tasks,
                                          int32_t chunks, int64_t total) {
    const bool small = total < (int64_t(1) << 32);
    Place p;
    int64_t r = divide(t, tasks, small);
    p.task = int32_t(t);
    if (a.heads_inner) {
        const int64_t row = divide(r, chunks, small);
        p.chunk = int32_t(r);
        p.i = row;
        p.b = divide(p.i, a.n, small);
    } else {
        int64_t col = divide(r, a.n, small);
        p.i = r;
        p.b = divide(col, chunks, small);
        p.chunk = int32_t(col);
    }
    return p;
}

__device__ __forceinline__ int64_t position_of(const RopeArgs &a, int64_t b, int64_t i) {
    return a.positions != nullptr ? int64_t(a.positions[b * a.n + i]) : a.first + i;
}

// Thread = (batch, token, chunk of heads, task), task fastest; a task is two
// vectors: V pairs, or 2 V copied channels.  Halves: rot a multiple of 2 V.
// Interleaved: any rot, the pairs from rot / 2 on being copied.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(RopeArgs a, int32_t hpt,
                                                            int32_t chunks, int64_t total) {
    constexpr int V = Vec<T>::V;
    const int64_t t = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= total) return;
    const Place w = place_of(a, t, a.d / (2 * V), chunks, total);
    const int32_t task = w.task, chunk = w.chunk;
    const int64_t i = w.i, b = w.b;
    const bool copied = task * 2 * V >= a.rot;
    if (copied && a.in_place) return;
    int32_t o0, o1;
    if (kInterleaved || copied) {
        o0 = task * 2 * V;
        o1 = o0 + V;
    } else {
        o0 = task * V;
        o1 = o0 + a.rot / 2;
    }
    // copied pairs of the task (interleaved): from this one on
    const int stay = kInterleaved ? a.rot / 2 - task * V : V;
    const int32_t h0 = chunk * hpt, h1 = h0 + hpt < a.heads ? h0 + hpt : a.heads;
    const T *x = static_cast<const T *>(a.x) + b * a.xs_b + i * a.xs_n;
    T *out = static_cast<T *>(a.out) + b * a.os_b + i * a.os_n;
    constexpr int U = 4;        // heads in flight
    uint4 u0[U], u1[U];
    const auto load = [&](int32_t h) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {
                const T *row = x + int64_t(h + u) * a.xs_h;
                u0[u] = *reinterpret_cast<const uint4 *>(row + o0);
                u1[u] = *reinterpret_cast<const uint4 *>(row + o1);
            }
    };
    load(h0);                   // on their way during the trigonometry
    float c[V], s[V];
    if (!copied) {
        const int64_t pos = position_of(a, b, i);
        const uint64_t *f = a.table + task * V;         // 16-byte aligned
#pragma unroll
        for (int p = 0; p < V; p += 2) {
            // an odd number of pairs: the last one alone, the table ends there
            ulonglong2 u = make_ulonglong2(0, 0);
            if (task * V + p + 1 < a.rot / 2)
                u = __ldg(reinterpret_cast<const ulonglong2 *>(f + p));
            else if (task * V + p < a.rot / 2)
                u.x = __ldg(reinterpret_cast<const unsigned long long *>(f + p));
            turn(u.x, pos, a.factor, a.sign, c[p], s[p]);
            turn(u.y, pos, a.factor, a.sign, c[p + 1], s[p + 1]);
        }
    }
    for (int32_t h = h0; h < h1; h += U) {
        if (h > h0) load(h);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {
                if (!copied) {
                    float x0[V], x1[V];
                    Vec<T>::load(u0[u], x0);
                    Vec<T>::load(u1[u], x1);
                    if (kInterleaved) {
#pragma unroll
                        for (int p = 0; p < V; ++p) {
                            float(&y)[V] = p < V / 2 ? x0 : x1;
                            const int e = 2 * (p % (V / 2));
                            const float y0 = y[e], y1 = y[e + 1];
                            if (p < stay) {
                                y[e] = y0 * c[p] - y1 * s[p];
                                y[e + 1] = y1 * c[p] + y0 * s[p];
                            }
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < V; ++p) {
                            const float p0 = x0[p], q0 = x1[p];
                            x0[p] = p0 * c[p] - q0 * s[p];
                            x1[p] = q0 * c[p] + p0 * s[p];
                        }
                    }
                    u0[u] = Vec<T>::store(x0);
                    u1[u] = Vec<T>::store(x1);
                }
                T *row = out + int64_t(h + u) * a.os_h;
                *reinterpret_cast<uint4 *>(row + o0) = u0[u];
                *reinterpret_cast<uint4 *>(row + o1) = u1[u];
            }
    }
}

// Halves with any even rot: a channel's partner lies rot / 2 away, at no vector
// boundary, so rows pass through shared memory.  Thread = (batch, token, chunk
// of heads, vector), vector fastest: a row belongs to lanes of one warp, which
// has read all of it before it writes any (out may be x).  bf16 runs at 45 to
// 68 % of the copy rate, bound by the 2-byte reads of the partners.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_row_kernel(RopeArgs a, int32_t hpt, int32_t chunks,
                                                            int64_t total) {
    constexpr int V = Vec<T>::V, U = 4;
    __shared__ uint4 rows[kThreads / 32][U][32];
    const int64_t t = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int lane = threadIdx.x & 31;
    const int32_t vecs = a.d / V;
    // threads past the end go along with the last rows, writing nothing
    const bool live = t < total;
    const Place w = place_of(a, live ? t : total - vecs + threadIdx.x % vecs, vecs, chunks, total);
    const int32_t vec = w.task, chunk = w.chunk;
    const int64_t i = w.i, b = w.b;
    const int half = a.rot / 2, c0 = vec * V;
    const int32_t h0 = chunk * hpt;
    const T *x = static_cast<const T *>(a.x) + b * a.xs_b + i * a.xs_n + c0;
    T *out = static_cast<T *>(a.out) + b * a.os_b + i * a.os_n + c0;
    uint4(&buf)[U][32] = rows[threadIdx.x >> 5];
    uint4 own[U];
    const auto load = [&](int32_t k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + u < hpt && h0 + k + u < a.heads)
                own[u] = *reinterpret_cast<const uint4 *>(x + int64_t(h0 + k + u) * a.xs_h);
    };
    load(0);                    // on their way during the trigonometry
    float c[V], s[V];
    const int64_t pos = position_of(a, b, i);
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (c0 + e < a.rot) {
            const bool first = c0 + e < half;
            turn(__ldg(a.table + (first ? c0 + e : c0 + e - half)), pos, a.factor,
                 first ? -a.sign : a.sign, c[e], s[e]);
        }
    for (int32_t k = 0; k < hpt; k += U) {
        if (k > 0) load(k);
#pragma unroll
        for (int u = 0; u < U; ++u) buf[u][lane] = own[u];
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T *row = reinterpret_cast<const T *>(&buf[u][lane - vec]);
            float y[V];
            Vec<T>::load(own[u], y);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int ch = c0 + e;
                if (ch < a.rot) y[e] = y[e] * c[e] + Vec<T>::get(row[ch < half ? ch + half : ch - half]) * s[e];
            }
            if (live && k + u < hpt && h0 + k + u < a.heads)
                *reinterpret_cast<uint4 *>(out + int64_t(h0 + k + u) * a.os_h) = Vec<T>::store(y);
        }
        __syncwarp();
    }
}

template <typename T>
cudaError_t launch(const RopeArgs &a, bool interleaved, cudaStream_t st) {
    constexpr int V = Vec<T>::V;
    const bool vec = interleaved || a.rot % (2 * V) == 0;
    const int64_t per_row = vec ? a.d / (2 * V) : a.d / V;
    // heads per thread: eight (64 heads of 128 channels, 32768 tokens: 161 us;
    // 169 with four, 163 with sixteen), fewer where that leaves less than the
    // threads of half a card (64 tokens of 32 heads: the same 6 us either way)
    int32_t hpt = 8;
    while (hpt > 1 && (hpt >= 2 * a.heads ||
                       a.batch * a.n * per_row * ((a.heads + hpt - 1) / hpt) < int64_t(152) * 1024))
        hpt /= 2;
    const int32_t chunks = (a.heads + hpt - 1) / hpt;
    hpt = (a.heads + chunks - 1) / chunks;              // ten heads: five and five
    const int64_t total = a.batch * a.n * per_row * chunks;
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid{unsigned(blocks)};
    if (!vec)
        rope_row_kernel<T><<<grid, kThreads, 0, st>>>(a, hpt, chunks, total);
    else if (interleaved)
        rope_vec_kernel<T, true><<<grid, kThreads, 0, st>>>(a, hpt, chunks, total);
    else
        rope_vec_kernel<T, false><<<grid, kThreads, 0, st>>>(a, hpt, chunks, total);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int32_t dtype, bool interleaved, cudaStream_t st) {
    return dtype == 0 ? launch<uint16_t>(a, interleaved, st) : launch<float>(a, interleaved, st);
}

}  // namespace bsa
