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
// turn in units of 2^-64, so the 64-bit product p * f wraps modulo whole turns
// by itself and its upper 32 bits, read as a signed number, are the angle in
// units of 2^-31 half turns, good to 2^-32 turns at any position.  It goes to
// sincospif, whose argument is in half turns, with fp32's rounding (2^-25 half
// turns, 9e-8 rad) as the only loss.
//
// The step only moves bytes: every element is read and written once, 36 heads
// of 128 per token in the 32/4-head shape.  The angles (one sincospif per pair
// and token) are computed once per token in shared memory and shared by the
// heads.
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
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    return make_float2(c * p.rot_scale, p.inverse ? -s * p.rot_scale : s * p.rot_scale);
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Params p) {
    extern __shared__ float2 cs[];  // [tokens][rot / 2]
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
        const TI* x = static_cast<const TI*>(p.x[w]) + (t0 + t) * p.xs[w] + (int64_t)hh * p.d;
        TO* y = static_cast<TO*>(p.y[w]) + (t0 + t) * p.ys[w] + (int64_t)hh * p.d;
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

}  // namespace rope
}  // namespace dsa
