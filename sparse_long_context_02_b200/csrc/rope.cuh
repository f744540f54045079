// Rotary positions of queries and keys, forward and backward.
//
// A pair (a, b) of a head's elements is turned by th = p_t w_i, the token's
// position times the pair's angular frequency:
//     y_a = m (a cos th - b sin th),   y_b = m (b cos th + a sin th),
// pairs being i and i + rot/2 ("half") or 2i and 2i + 1 ("interleaved") of
// the rotated part [off, off + rot) of the head; the rest passes through.
// The map is m times an orthogonal matrix, so the gradient of its input is the
// same call with -th.
//
// Angles.  p * w in fp32 loses the turn itself at far positions (2^-24 of
// 262144 rad is 0.016 rad).  The table holds each frequency as a fraction of a
// turn in units of 2^-64, so the 64-bit product p * f wraps modulo whole turns by
// itself: the angle, reduced exactly at every position.  Its distance from the
// nearest quarter turn, at most pi / 4, goes into Taylor's series as a sum of
// two fp32 numbers, and the series' leading terms are added last, so that cos and
// sin, times rot_scale, come out with little more than their one rounding
// (2^-24; sincospif on the rounded angle was off by 2e-7).
//
// The step only moves bytes: every element is read and written once, 36 heads
// of 128 per token in the 32/4-head shape.  cos and sin of a token's pairs are
// computed once, into shared memory, and shared by the heads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace dsa {
namespace rope {

constexpr int kThreads = 256;

struct Params {
    const void* x[2];        // q and k (k may be null: H[1] = 0)
    void* y[2];
    int64_t xs[2], ys[2];    // elements from one token to the next
    int H[2];                // heads
    const int64_t* pos;      // [L]
    const uint64_t* freqs;   // [rot / 2], 2^-64 turns per position
    int64_t L;
    int d, off, rot;
    int tokens;              // tokens per CTA
    int interleaved, inverse;
    float rot_scale, out_scale;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
// One rounding to e4m3 (nearest even, saturating); infinities become NaN, so
// that they do not pass for 448.
template <>
__device__ __forceinline__ __nv_fp8_e4m3 from_f32<__nv_fp8_e4m3>(float v) {
    __nv_fp8_e4m3 r;
    r.__x = __nv_cvt_float_to_fp8(fabsf(v) == INFINITY ? NAN : v, __NV_SATFINITE, __NV_E4M3);
    return r;
}

// cos and sin (times m) of one pair of one token.
__device__ __forceinline__ float2 angle(const Params& p, int64_t t, int i) {
    const uint64_t turns = (uint64_t)p.pos[t] * p.freqs[i];
    const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));  // [-2^61, 2^61)
    // x + y = rest * 2 pi / 2^64
    constexpr float kTurn = 6.2831855f * 0x1p-64f, kTurnRest = -1.7484555e-7f * 0x1p-64f;
    const float f = (float)rest, g = (float)(rest - (int64_t)f);
    const float x = f * kTurn;
    const float y = fmaf(f, kTurn, -x) + fmaf(f, kTurnRest, g * kTurn);
    const float z = x * x;
    // sin = x + ds, cos = c + dc
    const float ds = fmaf(
        x * z,
        fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 39916800, 1.f / 362880), -1.f / 5040), 1.f / 120),
             -1.f / 6),
        y * fmaf(z, -0.5f, 1.f));
    const float c = fmaf(z, -0.5f, 1.f);
    const float zl = fmaf(x, x, -z) + 2.f * x * y;  // (x + y)^2 - z
    const float dc = fmaf(
        z * z,
        fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 479001600, -1.f / 3628800), 1.f / 40320), -1.f / 720),
             1.f / 24),
        fmaf(z, -0.5f, 1.f - c) - 0.5f * zl);
    const float m = p.rot_scale;
    const float si = fmaf(x, m, ds * m), co = fmaf(c, m, dc * m);
    float2 r = quarter & 1 ? make_float2(-si, co) : make_float2(co, si);
    if (quarter & 2) r = make_float2(-r.x, -r.y);
    if (p.inverse) r.y = -r.y;
    return r;
}

// Any alignment, any even sizes: one pair per thread and step, for what the form below
// cannot take.  Scalar loads and two divisions a pair make it four times as slow (32768
// tokens of 36 heads x 128: 383 us against 98); nothing in the sizes asks for that.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Params p) {
    extern __shared__ float2 cs[];  // [tokens][rot / 2]
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)(p.L - t0 < p.tokens ? p.L - t0 : p.tokens);
    const int half = p.rot / 2;
    for (int e = threadIdx.x; e < nt * half; e += kThreads)
        cs[e] = angle(p, t0 + e / half, e % half);
    __syncthreads();
    const int H = p.H[0] + p.H[1], per = p.d / 2;
    for (int e = threadIdx.x; e < nt * H * per; e += kThreads) {
        const int i = e % per, h = e / per % H, t = e / (per * H);
        const int w = h >= p.H[0];
        const int hh = w ? h - p.H[0] : h;
        const TI* x = static_cast<const TI*>(w ? p.x[1] : p.x[0]) +
                      (t0 + t) * (w ? p.xs[1] : p.xs[0]) + (int64_t)hh * p.d;
        TO* y = static_cast<TO*>(w ? p.y[1] : p.y[0]) + (t0 + t) * (w ? p.ys[1] : p.ys[0]) +
                (int64_t)hh * p.d;
        int a, b;
        if (i < half) {
            a = p.off + (p.interleaved ? 2 * i : i);
            b = p.interleaved ? a + 1 : a + half;
        } else {  // two elements of the part that passes through
            a = 2 * (i - half);
            if (a >= p.off) a += p.rot;
            b = a + 1;
        }
        float u = to_f32(x[a]), v = to_f32(x[b]);
        if (i < half) {
            const float2 c = cs[t * half + i];
            const float r = u * c.x - v * c.y;
            v = v * c.x + u * c.y;
            u = r;
        }
        y[a] = from_f32<TO>(u * p.out_scale);
        y[b] = from_f32<TO>(v * p.out_scale);
    }
}

// E elements of one 16-byte load: 8 of bf16, 4 of fp32.
template <typename T>
constexpr int kPiece = 16 / sizeof(T);

__device__ __forceinline__ void unpack(float (&v)[8], uint4 q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

__device__ __forceinline__ void unpack(float (&v)[4], uint4 q) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
}

template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[N]) {
    if constexpr (N == 4) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (N == 2) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    if constexpr (N == 1) *static_cast<uint32_t*>(p) = w[0];
}

template <int E>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[E]) {
    uint32_t w[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
    store_words(p, w);
}

template <int E>
__device__ __forceinline__ void store(float* p, const float (&v)[E]) {
#pragma unroll
    for (int j = 0; j < E / 4; ++j)
        reinterpret_cast<float4*>(p)[j] =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

template <int E>
__device__ __forceinline__ void store(__nv_fp8_e4m3* p, const float (&v)[E]) {
    uint32_t w[E / 4] = {};
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, fabsf(v[j]));
    if (top < INFINITY) {  // no infinity among them: two at a time
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            uint16_t r;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(r)
                : "f"(v[2 * j + 1]), "f"(v[2 * j]));
            w[j >> 1] |= (uint32_t)r << (16 * (j & 1));
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
            w[j >> 2] |= (uint32_t)from_f32<__nv_fp8_e4m3>(v[j]).__x << (8 * (j & 3));
    }
    store_words(p, w);
}

// Heads of units of 2 E elements (d, off and rot multiples of 2 E, 16-byte
// aligned rows): a thread keeps one unit u of the head, two pieces of E elements,
// and walks over (token, head) rows, the next row's two 16-byte loads under way
// while it computes.  Units [0, rot / 2 E) hold E pairs each (pieces at off + E u and
// off + rot / 2 + E u, or 2 E u and 2 E u + E), the others pass through.
// The (cos, sin) of a token's pairs lie as [2 pairs of the unit][unit], so that
// the 8 threads of a 128-byte shared access read neighbours.
// Bound by memory; what counts is how many loads a multiprocessor has in flight.
// 32768 tokens of 36 heads x 128 in bf16 take 98 us, 6.2 TB/s (94 % of a copy's rate);
// with two rows at a time and no prefetch 105.0, two and the next two under way (3
// CTAs per SM instead of 5) 105.2.  8191 tokens in fp32: 48 us, 6.3 TB/s (8 elements
// per unit; 16, with twice the registers, 60).  16385 x 65 heads to e4m3: 75 us, 5.5 TB/s.
template <typename TI, typename TO, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(const Params p) {
    constexpr int E = kPiece<TI>;
    extern __shared__ float4 cs4[];  // [tokens][E / 2][rot / 2 E]
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)(p.L - t0 < p.tokens ? p.L - t0 : p.tokens);
    const int half = p.rot / 2, ru = half / E;
    for (int e = threadIdx.x; e < nt * half; e += kThreads) {
        const int t = e / half, i = e % half;
        reinterpret_cast<float2*>(cs4)[((t * (E / 2) + i % E / 2) * ru + i / E) * 2 + (i & 1)] =
            angle(p, t0 + t, i);
    }
    __syncthreads();
    const int units = p.d / (2 * E), per = kThreads / units, H = p.H[0] + p.H[1];
    const int u = threadIdx.x % units;
    if ((int)threadIdx.x >= per * units) return;
    int ea, eb;
    if (u < ru) {
        ea = p.off + (INTER ? 2 * E * u : E * u);
        eb = ea + (INTER ? E : half);
    } else {
        ea = 2 * E * (u - ru);
        if (ea >= p.off) ea += p.rot;
        eb = ea + E;
    }
    struct Row {
        uint4 a, b;
        int t, h;
    };
    int t = 0, h = threadIdx.x / units - per;
    auto fetch = [&](Row& r) {
        h += per;
        while (h >= H) {
            h -= H;
            ++t;
        }
        r.t = t;
        r.h = h;
        if (t < nt) {
            const bool w = h >= p.H[0];
            const TI* x = static_cast<const TI*>(w ? p.x[1] : p.x[0]) +
                          (t0 + t) * (w ? p.xs[1] : p.xs[0]) + (w ? h - p.H[0] : h) * p.d;
            r.a = __ldcs(reinterpret_cast<const uint4*>(x + ea));
            r.b = __ldcs(reinterpret_cast<const uint4*>(x + eb));
        }
    };
    Row r;
    fetch(r);
    while (r.t < nt) {
        Row next;
        fetch(next);
        float a[E], b[E];
        unpack(a, r.a);
        unpack(b, r.b);
        if (u < ru) {
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float4 c = cs4[(r.t * (E / 2) + j) * ru + u];
                float& a0 = INTER ? (4 * j < E ? a[4 * j % E] : b[4 * j % E]) : a[2 * j];
                float& b0 = INTER ? (4 * j < E ? a[4 * j % E + 1] : b[4 * j % E + 1]) : b[2 * j];
                float& a1 = INTER ? (4 * j < E ? a[4 * j % E + 2] : b[4 * j % E + 2]) : a[2 * j + 1];
                float& b1 = INTER ? (4 * j < E ? a[4 * j % E + 3] : b[4 * j % E + 3]) : b[2 * j + 1];
                const float r0 = a0 * c.x - b0 * c.y, r1 = a1 * c.z - b1 * c.w;
                b0 = b0 * c.x + a0 * c.y;
                b1 = b1 * c.z + a1 * c.w;
                a0 = r0;
                a1 = r1;
            }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
            a[j] *= p.out_scale;
            b[j] *= p.out_scale;
        }
        const bool w = r.h >= p.H[0];
        TO* y = static_cast<TO*>(w ? p.y[1] : p.y[0]) + (t0 + r.t) * (w ? p.ys[1] : p.ys[0]) +
                (w ? r.h - p.H[0] : r.h) * p.d;
        store(y + ea, a);
        store(y + eb, b);
        r = next;
    }
}

}  // namespace rope
}  // namespace dsa
