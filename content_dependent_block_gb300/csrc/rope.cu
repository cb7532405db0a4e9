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
// bits, as a signed number of 2^-31 half turns, go to sincospif; the angle is
// off by at most 2^-25 of a half turn (the int -> float rounding) at any
// position.
//
// HBM-bound: x is read once and out written once.  A thread owns V pairs of
// one token (two 16-byte vectors) and walks over the heads with them, so the
// sines are computed once per token and pair and shared by its heads.
#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void turn(uint64_t freq, int64_t pos, float factor, float sign,
                                     float &c, float &s) {
    const int32_t half_turns = int32_t(uint32_t((freq * uint64_t(pos)) >> 32));
    sincospif(float(half_turns) * 4.656612873077393e-10f, &s, &c);   // 2^-31
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

__device__ __forceinline__ int64_t position_of(const RopeArgs &a, int64_t b, int64_t i) {
    return a.positions != nullptr ? int64_t(a.positions[b * a.n + i]) : a.first + i;
}

// rot a multiple of 2 V: thread = (batch, token, task, chunk of heads), task
// fastest; a task is two vectors, either V pairs or 2 V copied channels.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(RopeArgs a, int32_t hpt,
                                                            int32_t chunks, int64_t total) {
    constexpr int V = Vec<T>::V;
    const int64_t t = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= total) return;
    const int32_t tasks = a.d / (2 * V);
    int64_t r = t / tasks;
    const int32_t task = int32_t(t - r * tasks);
    // the walk over (token, chunk of heads) follows the output's layout
    int64_t i, b;
    int32_t chunk;
    if (a.heads_inner) {
        chunk = int32_t(r % chunks);
        r /= chunks;
        i = r % a.n;
        b = r / a.n;
    } else {
        i = r % a.n;
        r /= a.n;
        chunk = int32_t(r % chunks);
        b = r / chunks;
    }
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
    float c[V], s[V];
    if (!copied) {
        const int64_t pos = position_of(a, b, i);
        const uint64_t *f = a.table + task * V;
#pragma unroll
        for (int p = 0; p < V; ++p) turn(__ldg(f + p), pos, a.factor, a.sign, c[p], s[p]);
    }
    const int32_t h0 = chunk * hpt, h1 = h0 + hpt < a.heads ? h0 + hpt : a.heads;
    const T *x = static_cast<const T *>(a.x) + b * a.xs_b + i * a.xs_n;
    T *out = static_cast<T *>(a.out) + b * a.os_b + i * a.os_n;
    constexpr int U = 4;        // heads in flight
    for (int32_t h = h0; h < h1; h += U) {
        uint4 u0[U], u1[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {
                const T *row = x + int64_t(h + u) * a.xs_h;
                u0[u] = *reinterpret_cast<const uint4 *>(row + o0);
                u1[u] = *reinterpret_cast<const uint4 *>(row + o1);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {
                if (!copied) {
                    float x0[V], x1[V];
                    Vec<T>::load(u0[u], x0);
                    Vec<T>::load(u1[u], x1);
                    if (kInterleaved) {
#pragma unroll
                        for (int p = 0; p < V / 2; ++p) {
                            const float p0 = x0[2 * p], q0 = x0[2 * p + 1];
                            x0[2 * p] = p0 * c[p] - q0 * s[p];
                            x0[2 * p + 1] = q0 * c[p] + p0 * s[p];
                            const float p1 = x1[2 * p], q1 = x1[2 * p + 1];
                            x1[2 * p] = p1 * c[p + V / 2] - q1 * s[p + V / 2];
                            x1[2 * p + 1] = q1 * c[p + V / 2] + p1 * s[p + V / 2];
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

// Any even rot: thread = (batch, token, channel pair), all heads in a loop.
// Pairs i < rot/2 are rotated; the others are copied.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_pair_kernel(RopeArgs a, int32_t interleaved,
                                                             int32_t hpt, int32_t chunks,
                                                             int64_t total) {
    const int64_t t = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= total) return;
    const int32_t pairs = a.d / 2;
    int64_t r = t / pairs;
    const int32_t p = int32_t(t - r * pairs);
    const int64_t i = r % a.n;
    r /= a.n;
    const int32_t chunk = int32_t(r % chunks);
    const int64_t b = r / chunks;
    const bool copied = 2 * p >= a.rot;
    if (copied && a.in_place) return;
    const int32_t o0 = interleaved || copied ? 2 * p : p;
    const int32_t o1 = interleaved || copied ? 2 * p + 1 : p + a.rot / 2;
    float c = 1.f, s = 0.f;
    if (!copied) turn(__ldg(a.table + p), position_of(a, b, i), a.factor, a.sign, c, s);
    const int32_t h0 = chunk * hpt, h1 = h0 + hpt < a.heads ? h0 + hpt : a.heads;
    const T *x = static_cast<const T *>(a.x) + b * a.xs_b + i * a.xs_n;
    T *out = static_cast<T *>(a.out) + b * a.os_b + i * a.os_n;
    for (int32_t h = h0; h < h1; ++h) {
        const T *row = x + int64_t(h) * a.xs_h;
        T *dst = out + int64_t(h) * a.os_h;
        const T r0 = row[o0], r1 = row[o1];
        if (copied) {
            dst[o0] = r0;
            dst[o1] = r1;
        } else {
            const float x0 = Vec<T>::get(r0), x1 = Vec<T>::get(r1);
            dst[o0] = Vec<T>::put(x0 * c - x1 * s);
            dst[o1] = Vec<T>::put(x1 * c + x0 * s);
        }
    }
}

template <typename T>
cudaError_t launch(const RopeArgs &a, bool interleaved, cudaStream_t st) {
    constexpr int V = Vec<T>::V;
    const bool vec = a.rot % (2 * V) == 0;
    const int64_t per_row = vec ? a.d / (2 * V) : a.d / 2;
    // heads per thread: as many as still leave the threads of a full card
    int32_t hpt = 16;
    while (hpt > 1 && (hpt >= 2 * a.heads ||
                       a.batch * a.n * per_row * ((a.heads + hpt - 1) / hpt) < int64_t(152) * 1024))
        hpt /= 2;
    const int32_t chunks = (a.heads + hpt - 1) / hpt;
    const int64_t total = a.batch * a.n * per_row * chunks;
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid{unsigned(blocks)};
    if (!vec)
        rope_pair_kernel<T><<<grid, kThreads, 0, st>>>(a, interleaved, hpt, chunks, total);
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
