// A paged K/V cache in 8 bits: appending to it and attending over it.
//
// Layout.  K8, V8 [pages][page][Hkv][d] hold e4m3 codes, k_scale and v_scale
// [pages][Hkv] one fp32 factor per page and head; a stored element is
// code * scale.  Position s of sequence b lies in page block_table[b][s / page],
// slot s % page.
//
// Half the bytes of the bf16 rows: one key costs 2 * Hkv * d bytes.  e4m3 is a
// floating-point format, so the scale only has to place the block's largest
// element inside the format's 17 binades; appending uses powers of two, by
// which codes are exact multiples and a later, larger scale shifts the older
// codes without a second rounding unless they fall into the subnormals.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace dsa {
namespace kv8 {

// Where a launch's rows (new tokens, or query rows) belong: rows
// [off[b], off[b + 1]) are sequence b's, rows outside all of them nobody's;
// without off, row b is sequence b's.
struct Rows {
    const int32_t* off;  // [B + 1] or null
    int B;
    int64_t n;           // rows of the arrays
};

// ------------------------------------------------------------------ append

struct AppendParams {
    const __nv_bfloat16* x[2];   // new K and V rows
    int64_t xs[2];               // elements from one row to the next
    uint8_t* code[2];            // K8, V8
    float* scale[2];
    const int32_t* table;        // [B][M]
    const int32_t* lens;         // [B] lengths before the call
    Rows rows;
    int M, Hkv;
    int64_t pages;
    int* err;
};

constexpr int kMinExp = -120;    // the smallest scale is 2^-120

// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), as an
// exponent; amax is finite and >= 0.
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e > kMinExp ? e : kMinExp;
}

// One rounding to e4m3 of x / s (nearest even); x / s is at most 448 by the
// choice of s.  NaN and infinities become the NaN code.
__device__ __forceinline__ uint32_t code_of(float q) {
    return __nv_cvt_float_to_fp8(fabsf(q) == INFINITY ? NAN : q, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float value_of(uint32_t code) {
    return __half2float(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3));
}

// Units of work: (sequence, touched page).  A sequence's n new tokens touch at
// most n / page + 2 pages, and off[b + 1] / page - off[b] / page >= n / page, so the
// unit ranges starting at off[b] / page + 2 b never overlap, and T / page + 2 B
// units cover all without knowing the lengths on the host.  Returns false for
// a unit that has nothing to do.
template <int PAGE>
__device__ __forceinline__ bool find_unit(const AppendParams& p, int u, int& b, int64_t& r0,
                                          int64_t& n, int& col) {
    const Rows& rw = p.rows;
    if (rw.off == nullptr) {
        b = u;
        r0 = u;
        n = 1;
        col = p.lens[b] >= 0 ? p.lens[b] / PAGE : 0;
        return p.lens[b] >= 0;
    }
    auto base = [&](int i) { return max(rw.off[i], 0) / PAGE + 2 * i; };
    int lo = 0, hi = rw.B - 1;  // the last b with base(b) <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base(mid) <= u) lo = mid;
        else hi = mid - 1;
    }
    b = lo;
    r0 = rw.off[b];
    const int64_t r1 = rw.off[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > rw.n) {
        if (threadIdx.x == 0) record_error_to(p.err, 2);
        return false;
    }
    n = r1 - r0;
    const int len = p.lens[b];
    if (len < 0 || n == 0) return false;
    const int64_t c = len / PAGE + (u - base(b));
    if (u < base(b) || c > (len + n - 1) / PAGE) return false;
    if (c >= p.M) {
        if (threadIdx.x == 0) record_error_to(p.err, 2);
        return false;
    }
    col = (int)c;
    return true;
}

template <int PAGE, int D>
struct AppendCfg {
    static constexpr int VECS = PAGE * D / 8;  // 8-element pieces of a (page, head)
    static constexpr int THREADS = VECS < 256 ? 128 : 256;
    static constexpr int VPT = VECS / THREADS;
    static constexpr int PER_ROW = D / 8;
};

// One CTA per (unit, head, K or V): the page's new elements stay in registers
// between the maximum and the rounding, so they are read once.
template <int PAGE, int D>
__global__ void __launch_bounds__(AppendCfg<PAGE, D>::THREADS) append_kernel(const AppendParams p) {
    using C = AppendCfg<PAGE, D>;
    const int h = blockIdx.x % p.Hkv, w = blockIdx.y;
    int b, col;
    int64_t r0, n;
    if (!find_unit<PAGE>(p, blockIdx.x / p.Hkv, b, r0, n, col)) return;
    const int32_t pg = col < p.M ? p.table[(int64_t)b * p.M + col] : -1;
    if (pg < 0 || pg >= p.pages) {
        if (threadIdx.x == 0) record_error_to(p.err, 2);
        return;
    }
    const int len = p.lens[b];
    // slot i of the page is the sequence's position col * PAGE + i
    const int64_t at = (int64_t)col * PAGE;
    const int first = len > at ? (int)(len - at) : 0;
    const int last = len + n < at + PAGE ? (int)(len + n - at) : PAGE;

    uint4 v[C::VPT];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < C::VPT; ++i) {
        const int e = i * C::THREADS + threadIdx.x;
        const int slot = e / C::PER_ROW, c = e % C::PER_ROW * 8;
        if (slot >= first && slot < last)
            v[i] = *reinterpret_cast<const uint4*>(p.x[w] + (r0 + at + slot - len) * p.xs[w] +
                                                   (int64_t)h * D + c);
        else
            v[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < C::VPT; ++i) {
        const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float((q[j] & 0x7fffu) << 16);
            const float hi = __uint_as_float(q[j] & 0x7fff0000u);
            if (lo < INFINITY) amax = fmaxf(amax, lo);
            if (hi < INFINITY) amax = fmaxf(amax, hi);
        }
    }
    __shared__ uint32_t top_s;
    if (threadIdx.x == 0) top_s = 0;
    __syncthreads();
    // non-negative floats order as their bits
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
    if ((threadIdx.x & 31) == 0) atomicMax(&top_s, m);
    float* sp = p.scale[w] + (int64_t)pg * p.Hkv + h;
    const float was = *sp;
    __syncthreads();
    const float need = __uint_as_float((uint32_t)(scale_exp(__uint_as_float(top_s)) + 127) << 23);
    const float now = first > 0 ? fmaxf(was, need) : need;
    if (threadIdx.x == 0) *sp = now;
    uint8_t* page = p.code[w] + ((int64_t)pg * PAGE * p.Hkv + h) * D;
    const int64_t row = (int64_t)p.Hkv * D;
    if (first > 0 && now != was) {  // the older codes under the larger scale
        const float f = __fdiv_rn(was, now);
        for (int e = threadIdx.x; e < first * C::PER_ROW; e += C::THREADS) {
            uint2* q = reinterpret_cast<uint2*>(page + e / C::PER_ROW * row + e % C::PER_ROW * 8);
            const uint2 old = *q;
            uint32_t o[2] = {old.x, old.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t r = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    r |= code_of(value_of(o[j] >> (8 * k) & 0xffu) * f) << (8 * k);
                o[j] = r;
            }
            *q = make_uint2(o[0], o[1]);
        }
    }
#pragma unroll
    for (int i = 0; i < C::VPT; ++i) {
        const int e = i * C::THREADS + threadIdx.x;
        const int slot = e / C::PER_ROW, c = e % C::PER_ROW * 8;
        if (slot < first || slot >= last) continue;
        const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            o[j] = code_of(__fdiv_rn(__uint_as_float(q[2 * j] << 16), now)) |
                   code_of(__fdiv_rn(__uint_as_float(q[2 * j] & 0xffff0000u), now)) << 8 |
                   code_of(__fdiv_rn(__uint_as_float(q[2 * j + 1] << 16), now)) << 16 |
                   code_of(__fdiv_rn(__uint_as_float(q[2 * j + 1] & 0xffff0000u), now)) << 24;
        *reinterpret_cast<uint2*>(page + slot * row + c) = make_uint2(o[0], o[1]);
    }
}

}  // namespace kv8
}  // namespace dsa
