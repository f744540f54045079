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

// ------------------------------------------------------------------ attention

struct AttnParams {
    const __nv_bfloat16* Q;      // [T][Hq][d]
    const uint8_t* code[2];      // K8, V8
    const float* scale[2];
    const int32_t* table;        // [B][M]
    const int32_t* lens;         // [B]
    const int32_t* idx;          // [T][k], or null: every key
    Rows rows;
    int M, Hkv, G, k, page_log2;
    int64_t pages;
    float scale_log2;            // softmax scale * log2(e)
    int nsplit;                  // slices of a row's keys
    __nv_bfloat16* O;            // [T][Hq][d]
    float* lse;                  // [T][Hq] or null
    // With nsplit > 1, per (row, slice, head): sums of 2^(y - My) V, and
    // (Mx, My, l), see attn_kernel.
    float* part_o;               // [T][nsplit][Hq][d]
    float* part_m;               // [T][nsplit][Hq][4]
    int* err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kWarps = 4;
constexpr float kWeightLog2 = 15.f;  // the largest fp16 weight is 2^15
constexpr float kWeightScale = 3.0517578125e-05f;  // 2^-15
constexpr int kChunk = 512;      // keys whose places and scales are staged at once

// The sequence of row t and the number of keys it sees; false: the row belongs
// to no sequence (it lies behind the last one).
__device__ __forceinline__ bool find_row(const AttnParams& p, int64_t t, int& b, int64_t& n) {
    const Rows& rw = p.rows;
    if (rw.off == nullptr) {
        b = (int)t;
        n = p.lens[b];
    } else {
        if (t < rw.off[0] || t >= rw.off[rw.B]) return false;
        int lo = 0, hi = rw.B - 1;  // the last b with off[b] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (rw.off[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        n = p.lens[b];
        const int64_t later = (int64_t)rw.off[b + 1] - 1 - t;
        if (later < 0 || rw.off[b + 1] > rw.n) {  // offsets that do not ascend
            if (threadIdx.x == 0) record_error_to(p.err, 2);
            n = 0;
        }
        // rows of a sequence are its last tokens; over every key they are causal
        if (p.idx == nullptr) n -= later;
    }
    const int64_t cap = (int64_t)p.M << p.page_log2;
    if (n > cap) {
        if (threadIdx.x == 0) record_error_to(p.err, 2);
        n = cap;
    }
    if (n < 0) n = 0;
    return true;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes to two fp16 values, exactly (every e4m3 value is one of fp16).
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <int N>
__device__ __forceinline__ void load_codes(uint32_t (&r)[N], const uint8_t* q, bool ok) {
    static_assert(N == 4 || N == 2, "");
    if constexpr (N == 4) {
        const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(q)) : make_uint4(0, 0, 0, 0);
        r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
    } else {
        const uint2 v = ok ? __ldg(reinterpret_cast<const uint2*>(q)) : make_uint2(0, 0);
        r[0] = v.x; r[1] = v.y;
    }
}

// One CTA per (KV head, slice, row).  Each warp takes every kWarps-th tile of 16
// keys by itself: no barrier inside a chunk, one merge at the end.
//
// S^T = K Q^T: the 16 keys are the rows of an m16n8k16 product, the head
// group's queries (up to 8) its columns.  The sum over d may run in any order,
// so thread (g, t) of the quad layout takes d = 16 t .. 16 t + 15 of keys g and
// g + 8 straight from global memory as one 16-byte load, which feeds four
// products; Q is laid out to match, once.  K is exact in fp16; Q's bf16 is made
// exact in fp16 by a power of two per head that puts its largest element at
// 2^14 (what falls below 2^-24 there is under 2^-38 of that element).
//
// O^T += V^T P: the rows are d, the columns heads, the depth the 16 keys.
// Thread (g, t) needs keys 2t, 2t+1, 2t+8, 2t+9 at its d, again 16 contiguous
// bytes of each key; byte permutes pair two keys' codes before widening.  The
// score tile's (key, head) fragment becomes the (head, key) operand by an 8x8
// transpose in registers.
//
// Softmax in log2 units: x = score, y = x + log2(v_scale[key]).  Two running
// maxima are kept: Mx for l = sum 2^(x - Mx), My for the weights 2^(y - My) that
// multiply the V codes, so the weights are at most 1 whatever the scales are:
// O = (sum 2^(y - My) code) * 2^(My - Mx) / l.  They are held times 2^15 in fp16:
// rounding them costs 2^-11 each, an eighth of the output's own bf16 rounding,
// down to 2^-29 of the largest, and 2^-40 of it below, so that a long tail of
// small weights (2^18 keys and more) still counts.
template <int D, bool DENSE>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const AttnParams p) {
    constexpr int NL = D / 64;       // 16-byte loads per key row and quad thread
    constexpr int MT = D / 16;       // m16 tiles of d
    constexpr int VW = D / 32;       // 32-bit words of one key's V row per thread
    const int h = blockIdx.x % p.Hkv, sp = blockIdx.y;
    const int64_t t = blockIdx.x / p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const int PAGE = 1 << p.page_log2;

    __shared__ int32_t row_s[kChunk];      // page * PAGE + slot, -1: no key
    __shared__ float ks_s[kChunk];         // k scale
    __shared__ float lv_s[kChunk];         // log2 of the v scale
    __shared__ float o_s[kWarps][8][D + 4];
    __shared__ float m_s[kWarps][8][3];    // Mx, My, l

    int b;
    int64_t n;
    if (!find_row(p, t, b, n)) return;
    // this slice's entries (list positions, or keys)
    const int64_t total = DENSE ? n : p.k;
    const int64_t per = ((total + p.nsplit - 1) / p.nsplit + 15) / 16 * 16;
    const int64_t e0 = sp * per < total ? sp * per : total;
    const int64_t e1 = e0 + per < total ? e0 + per : total;

    // Q, scaled by 2^qe
    uint32_t qf[NL][4][2];
    float qs[2];                           // for heads 2 t4, 2 t4 + 1
    {
        const __nv_bfloat16* q = p.Q + (t * p.Hkv * p.G + (int64_t)h * p.G + g) * D;
        uint32_t raw[NL][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            uint4 a = make_uint4(0, 0, 0, 0), c = a;
            if (g < p.G) {
                a = *reinterpret_cast<const uint4*>(q + 64 * i + 16 * t4);
                c = *reinterpret_cast<const uint4*>(q + 64 * i + 16 * t4 + 8);
            }
            raw[i][0] = a.x; raw[i][1] = a.y; raw[i][2] = a.z; raw[i][3] = a.w;
            raw[i][4] = c.x; raw[i][5] = c.y; raw[i][6] = c.z; raw[i][7] = c.w;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, max(raw[i][j] & 0x7fffu, raw[i][j] >> 16 & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the exponent that brings the largest element to [2^14, 2^15)
        int qe = top == 0 || top >= 0x7f80u ? 0 : 14 + 127 - (int)max(top >> 7, 1u);
        qe = min(qe, 126);
        const float up = __uint_as_float((uint32_t)(qe + 127) << 23);
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __half2 v = __floats2half2_rn(__uint_as_float(raw[i][j] << 16) * up,
                                                    __uint_as_float(raw[i][j] & 0xffff0000u) * up);
                qf[i][j >> 1][j & 1] = *reinterpret_cast<const uint32_t*>(&v);
            }
        const float back = p.scale_log2 * __uint_as_float((uint32_t)(127 - qe) << 23);
        qs[0] = __shfl_sync(0xffffffffu, back, 8 * t4);
        qs[1] = __shfl_sync(0xffffffffu, back, 8 * t4 + 4);
    }

    float o[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, my[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int64_t c0 = e0; c0 < e1; c0 += kChunk) {
        const int cn = (int)(e1 - c0 < kChunk ? e1 - c0 : kChunk);
        __syncthreads();
        for (int e = threadIdx.x; e < (cn + 15) / 16 * 16; e += kWarps * 32) {
            int64_t key = -1;
            if (e < cn) key = DENSE ? c0 + e : (int64_t)p.idx[t * p.k + c0 + e];
            int32_t row = -1;
            float ks = 0.f, lv = -INFINITY;
            if (key >= 0) {
                const int32_t pg = key < n ? p.table[(int64_t)b * p.M + (key >> p.page_log2)] : -1;
                if (pg >= 0 && pg < p.pages) {
                    row = (int32_t)(((int64_t)pg << p.page_log2) + (key & (PAGE - 1)));
                    ks = p.scale[0][(int64_t)pg * p.Hkv + h];
                    lv = log2f(p.scale[1][(int64_t)pg * p.Hkv + h]);
                } else {
                    record_error_to(p.err, 2);
                }
            }
            row_s[e] = row;
            ks_s[e] = ks;
            lv_s[e] = lv;
        }
        __syncthreads();
        for (int e = warp * 16; e < cn; e += kWarps * 16) {
            const int64_t rb = (int64_t)p.Hkv * D;
            const int32_t rk[2] = {row_s[e + g], row_s[e + g + 8]};
            uint32_t kr[2][NL][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    load_codes<4>(kr[j][i], p.code[0] + rk[j] * rb + h * D + 64 * i + 16 * t4,
                                  rk[j] >= 0);
            uint32_t vr[4][VW];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t rv = row_s[e + 2 * t4 + (j & 1) + (j >> 1) * 8];
                load_codes<VW>(vr[j], p.code[1] + rv * rb + h * D + VW * 4 * g, rv >= 0);
            }
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a[4] = {widen(kr[0][i][j]), widen(kr[1][i][j]),
                                           widen(kr[0][i][j] >> 16), widen(kr[1][i][j] >> 16)};
                    mma_f16(s, a, qf[i][j][0], qf[i][j][1]);
                }
            // x, y of keys g and g + 8, heads 2 t4 and 2 t4 + 1
            float x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kk = e + g + (j >> 1) * 8;
                x[j] = rk[j >> 1] >= 0 ? s[j] * (ks_s[kk] * qs[j & 1]) : -INFINITY;
                y[j] = x[j] + lv_s[kk];
            }
            float wgt[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float ax = fmaxf(x[c], x[c + 2]), ay = fmaxf(y[c], y[c + 2]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    ax = fmaxf(ax, __shfl_xor_sync(0xffffffffu, ax, d));
                    ay = fmaxf(ay, __shfl_xor_sync(0xffffffffu, ay, d));
                }
                const float nx = fmaxf(mx[c], ax), ny = fmaxf(my[c], ay);
                const float ux = nx == -INFINITY ? 0.f : nx, uy = ny == -INFINITY ? 0.f : ny;
                const float fx = ex2(mx[c] - ux), fy = ex2(my[c] - uy);
                const float ry = uy - kWeightLog2;
                mx[c] = nx;
                my[c] = ny;
                l[c] = l[c] * fx + ex2(x[c] - ux) + ex2(x[c + 2] - ux);
                wgt[c] = ex2(y[c] - ry);
                wgt[c + 2] = ex2(y[c + 2] - ry);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[i][c] *= fy;
                    o[i][c + 2] *= fy;
                }
            }
            uint32_t pf[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const __half2 v = __floats2half2_rn(wgt[2 * j], wgt[2 * j + 1]);
                pf[j] = transpose8x8(*reinterpret_cast<const uint32_t*>(&v));
            }
#pragma unroll
            for (int i = 0; i < VW; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t sel = j ? 0x7362u : 0x5140u;
                    const uint32_t lo = __byte_perm(vr[0][i], vr[1][i], sel);
                    const uint32_t hi = __byte_perm(vr[2][i], vr[3][i], sel);
                    const uint32_t a[4] = {widen(lo), widen(lo >> 16), widen(hi), widen(hi >> 16)};
                    mma_f16(o[2 * i + j], a, pf[0], pf[1]);
                }
        }
    }

    // ---- the warps' partial results
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int hh = 2 * t4 + c;
#pragma unroll
        for (int i = 0; i < MT; ++i) {  // m tile i, rows g and g + 8: d = MT * 2 * g + 2 i, + 1
            o_s[warp][hh][2 * MT * g + 2 * i] = o[i][c];
            o_s[warp][hh][2 * MT * g + 2 * i + 1] = o[i][c + 2];
        }
        if (g == 0) {
            m_s[warp][hh][0] = mx[c];
            m_s[warp][hh][1] = my[c];
            m_s[warp][hh][2] = l[c];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.G * D; e += kWarps * 32) {
        const int hh = e / D, d = e % D;
        float Mx = -INFINITY, My = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            Mx = fmaxf(Mx, m_s[w][hh][0]);
            My = fmaxf(My, m_s[w][hh][1]);
        }
        const float ux = Mx == -INFINITY ? 0.f : Mx, uy = My == -INFINITY ? 0.f : My;
        float ls = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            ls += m_s[w][hh][2] * ex2(m_s[w][hh][0] - ux);
            acc += o_s[w][hh][d] * ex2(m_s[w][hh][1] - uy);
        }
        const int64_t head = (int64_t)h * p.G + hh;
        const int64_t Hq = (int64_t)p.Hkv * p.G;
        if (p.nsplit == 1) {
            p.O[(t * Hq + head) * D + d] =
                __float2bfloat16_rn(ls == 0.f ? 0.f : acc / ls * kWeightScale * ex2(My - Mx));
            if (p.lse != nullptr && d == 0)
                p.lse[t * Hq + head] = ls == 0.f ? -INFINITY
                                                 : (Mx + log2f(ls)) * 0.6931471805599453f;
        } else {
            const int64_t at = (t * p.nsplit + sp) * Hq + head;
            p.part_o[at * D + d] = acc;
            if (d == 0)
                *reinterpret_cast<float4*>(p.part_m + at * 4) = make_float4(Mx, My, ls, 0.f);
        }
    }
}

// Merges the slices of one (row, head).
template <int D>
__global__ void __launch_bounds__(D) combine_kernel(const AttnParams p) {
    pdl_wait();
    const int64_t Hq = (int64_t)p.Hkv * p.G;
    const int64_t t = blockIdx.y, head = blockIdx.x;
    const int d = threadIdx.x;
    if (p.rows.off != nullptr && (t < p.rows.off[0] || t >= p.rows.off[p.rows.B])) return;
    auto at = [&](int j) { return (t * p.nsplit + j) * Hq + head; };
    float Mx = -INFINITY, My = -INFINITY;
    for (int j = 0; j < p.nsplit; ++j) {
        Mx = fmaxf(Mx, p.part_m[at(j) * 4]);
        My = fmaxf(My, p.part_m[at(j) * 4 + 1]);
    }
    const float ux = Mx == -INFINITY ? 0.f : Mx, uy = My == -INFINITY ? 0.f : My;
    float ls = 0.f, acc = 0.f;
    for (int j = 0; j < p.nsplit; ++j) {
        const float4 m = *reinterpret_cast<const float4*>(p.part_m + at(j) * 4);
        ls += m.z * ex2(m.x - ux);
        acc += p.part_o[at(j) * D + d] * ex2(m.y - uy);
    }
    p.O[(t * Hq + head) * D + d] = __float2bfloat16_rn(ls == 0.f ? 0.f : acc / ls * kWeightScale * ex2(My - Mx));
    if (p.lse != nullptr && d == 0)
        p.lse[t * Hq + head] = ls == 0.f ? -INFINITY : (Mx + log2f(ls)) * 0.6931471805599453f;
}

}  // namespace kv8
}  // namespace dsa
