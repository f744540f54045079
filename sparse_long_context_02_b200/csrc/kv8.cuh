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
//
// Every kernel here is launched by programmatic dependence and waits for the ones
// before it first thing: 2 us less between two calls (a token to each of 64
// sequences 4.1 -> 2.9 us a call, three short rows 8.2 -> 6.5).  So a kernel may be
// resident while the one before it still writes the index rows, tables or elements that
// it will read: those are plain loads after the wait, never the read-only path, whose
// data nobody may write while the kernel lives.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

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

// Records offsets of sequence b that do not ascend or lead past the arrays.  The lookups
// check the pair that they find, but where offsets run backwards a search need not come to
// every pair, so a launch looks at all of them.
__device__ __forceinline__ void check_offsets(const Rows& rw, int* err, int b) {
    const int32_t first = rw.off[b], end = rw.off[b + 1];
    if (first < 0 || end < first || end > rw.n) record_error_to(err, 2);
}

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

// Units of work of a call with offsets: (sequence, touched page).  A sequence's n
// new tokens touch at most n / page + 2 pages, and off[b + 1] / page - off[b] / page >=
// n / page, so the unit ranges starting at off[b] / page + 2 b never overlap, and
// T / page + 2 B units cover all without knowing the lengths on the host.
// Returns false for a unit that has nothing to do.
template <int PAGE>
__device__ __forceinline__ bool find_unit(const AppendParams& p, int u, bool report, int& b,
                                          int64_t& r0, int64_t& n, int& len, int& col) {
    const Rows& rw = p.rows;
    auto base = [&](int i) { return max(rw.off[i], 0) / PAGE + 2 * i; };
    int lo = 0, hi = rw.B - 1;  // the last b with base(b) <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base(mid) <= u) lo = mid;
        else hi = mid - 1;
    }
    b = lo;
    len = p.lens[b];
    r0 = rw.off[b];
    const int64_t r1 = rw.off[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > rw.n) {
        if (report) record_error_to(p.err, 2);
        return false;
    }
    n = r1 - r0;
    const int first = max((int)r0, 0) / PAGE + 2 * b;
    if (len < 0 || n == 0 || u < first) return false;
    const int64_t c = len / PAGE + (u - first);
    if (c > (len + n - 1) / PAGE) return false;
    if (c >= p.M) {
        if (report) record_error_to(p.err, 2);
        return false;
    }
    col = (int)c;
    return true;
}

// The page's scale under new elements whose largest has the bf16 bits `top`.
__device__ __forceinline__ float scale_for(uint32_t top) {
    return __uint_as_float((uint32_t)(scale_exp(__uint_as_float(top << 16)) + 127) << 23);
}

// 1 / s where that is exact (powers of two, all that this file stores), else 0.
__device__ __forceinline__ float exact_inverse(float s) {
    const uint32_t u = __float_as_uint(s), e = u >> 23;
    return (u & 0x7fffffu) == 0 && e >= 1 && e <= 253 ? __uint_as_float((254 - e) << 23) : 0.f;
}

// Codes of two finite bf16 elements under a scale with an exact inverse ...
__device__ __forceinline__ uint32_t codes_of(uint32_t two, float inv) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r)
        : "f"(__uint_as_float(two & 0xffff0000u) * inv), "f"(__uint_as_float(two << 16) * inv));
    return r;
}

// ... and of any two under any scale.
__device__ __forceinline__ uint32_t any_codes_of(uint32_t two, float s) {
    return code_of(__fdiv_rn(__uint_as_float(two << 16), s)) |
           code_of(__fdiv_rn(__uint_as_float(two & 0xffff0000u), s)) << 8;
}

// Rounds `count` 8-code pieces again under a scale that grew by 1 / f; piece e lies
// at row e / PER_ROW of the page.
template <int PER_ROW>
__device__ __forceinline__ void round_again(uint8_t* page, int64_t row, int count, float f, int at,
                                            int step) {
    for (int e = at; e < count; e += step) {
        uint2* q = reinterpret_cast<uint2*>(page + e / PER_ROW * row + e % PER_ROW * 8);
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

constexpr int kAppendThreads = 256;

template <int PAGE, int D>
struct AppendCfg {
    static constexpr int VECS = PAGE * D / 8;          // 8-element pieces of a (page, head)
    static constexpr int TEAM = VECS / 256 < 1 ? 1 : VECS / 256;  // warps that share one
    static constexpr int TEAMS = kAppendThreads / 32 / TEAM;
    static constexpr int VPT = VECS / (32 * TEAM);     // 8, or 4 for the smallest page
    static constexpr int PER_ROW = D / 8;
    static constexpr int ROWS = 32 * TEAM / PER_ROW;   // rows that a team takes at once
};

// Pieces of prompts: a team of warps per (unit, K or V, head), neighbouring
// heads side by side.  The page's new elements stay in registers between the
// maximum and the rounding, so they are read once; their loads go out before the
// page is looked up, eight (four) of 16 bytes per thread.  A chunk of 32768 rows of
// 4 x 128 takes 20.1 us (5.0 TB/s), with teams twice as large 20.9; issue slots are
// 60 % and the ALU pipe 56 % busy (maxima, conversions) in three and a half waves of
// four CTAs per SM.
template <int PAGE, int D>
__global__ void __launch_bounds__(kAppendThreads, AppendCfg<PAGE, D>::VPT == 4 ? 6 : 4)
append_kernel(const AppendParams p, int units) {
    using C = AppendCfg<PAGE, D>;
    __shared__ uint32_t top_s[kAppendThreads / 32];
    pdl_wait();
    // a thread for every sequence: the grid covers 2 B units, 2 tensors and the heads
    if (blockIdx.x <= p.rows.B / kAppendThreads) {
        const int b = blockIdx.x * kAppendThreads + threadIdx.x;
        if (b < p.rows.B) check_offsets(p.rows, p.err, b);
    }
    const int warp = threadIdx.x >> 5, team = warp / C::TEAM;
    const int me = threadIdx.x - team * C::TEAM * 32;  // thread of the team
    const uint32_t item = blockIdx.x * C::TEAMS + team, hkv = p.Hkv;  // below 2^31 + 8
    const uint32_t u = item / (2 * hkv), uh = item - u * 2 * hkv;
    const int w = uh >= hkv, h = uh - (w ? hkv : 0);
    int b = 0, len = 0, col = 0;
    int64_t r0 = 0, n = 0;
    bool live = u < (uint32_t)units && find_unit<PAGE>(p, (int)u, me == 0, b, r0, n, len, col);
    // slot i of the page is the sequence's position col * PAGE + i
    const int64_t at = (int64_t)col * PAGE;
    const int first = len > at ? (int)(len - at) : 0;
    const int last = !live ? 0 : len + n < at + PAGE ? (int)(len + n - at) : PAGE;

    const int slot = me / C::PER_ROW, c = me % C::PER_ROW * 8;  // + ROWS i: this thread's pieces
    uint4 v[C::VPT];
    {
        const int64_t xs = w ? p.xs[1] : p.xs[0], step = C::ROWS * xs;
        const __nv_bfloat16* x =
            (w ? p.x[1] : p.x[0]) + (r0 + at + slot - len) * xs + h * D + c;
#pragma unroll
        for (int i = 0; i < C::VPT; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (slot + C::ROWS * i >= first && slot + C::ROWS * i < last)
                v[i] = __ldcs(reinterpret_cast<const uint4*>(x + i * step));
        }
    }
    const int32_t pg = live ? p.table[(int64_t)b * p.M + col] : 0;
    if (pg < 0 || pg >= p.pages) {
        if (me == 0) record_error_to(p.err, 2);
        live = false;
    }
    float* sp = (w ? p.scale[1] : p.scale[0]) + (int64_t)(live ? pg : 0) * p.Hkv + h;
    const float was = *sp;
    uint32_t two = 0;  // bf16 magnitudes order as their bits
#pragma unroll
    for (int i = 0; i < C::VPT; ++i) {
        two = __vmaxu2(two, __vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu));
        two = __vmaxu2(two, __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
    }
    auto team_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if (C::TEAM > 1) {
            if ((threadIdx.x & 31) == 0) top_s[warp] = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < C::TEAM; ++i) m = max(m, top_s[team * C::TEAM + i]);
        }
        return m;
    };
    uint32_t top = team_max(max(two & 0xffffu, two >> 16));
    const bool odd = top >= 0x7f80u;
    const bool again = C::TEAM > 1 ? __syncthreads_or(odd) : odd;
    if (again) {  // infinities or NaN among them: the largest of the others
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < C::VPT; ++i) {
            const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = q[j] & 0x7fffu, hi = q[j] >> 16 & 0x7fffu;
                if (lo < 0x7f80u) m = max(m, lo);
                if (hi < 0x7f80u) m = max(m, hi);
            }
        }
        top = team_max(m);
    }
    if (!live) return;
    const float need = scale_for(top);
    const float now = first > 0 ? fmaxf(was, need) : need;
    if (me == 0) *sp = now;
    uint8_t* page = (w ? p.code[1] : p.code[0]) + ((int64_t)pg * PAGE * p.Hkv + h) * D;
    const int64_t row = (int64_t)p.Hkv * D;
    if (first > 0 && now != was)  // the older codes under the larger scale
        round_again<C::PER_ROW>(page, row, first * C::PER_ROW, __fdiv_rn(was, now), me,
                                32 * C::TEAM);
    const float inv = exact_inverse(now);
    auto store = [&](auto exact) {
#pragma unroll
        for (int i = 0; i < C::VPT; ++i) {
            if (slot + C::ROWS * i < first || slot + C::ROWS * i >= last) continue;
            auto codes = [&](uint32_t q) {
                return decltype(exact)::value ? codes_of(q, inv) : any_codes_of(q, now);
            };
            *reinterpret_cast<uint2*>(page + (slot + C::ROWS * i) * row + c) =
                make_uint2(codes(v[i].x) | codes(v[i].y) << 16,
                           codes(v[i].z) | codes(v[i].w) << 16);
        }
    };
    if (inv != 0.f && !odd) store(std::true_type{});
    else store(std::false_type{});
}

// One new token for each sequence: a warp per (sequence, K or V, head), so that no
// barrier stands in the chain of loads (length, page, scale) that is its time: 2.1 us for
// 64 sequences of 4 x 128, against 5.9 with a block per page and head.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_one_kernel(const AppendParams p,
                                                                    int page_log2) {
    constexpr int W = D / 64;  // 32-bit words of a lane
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5), hkv = p.Hkv;
    const int64_t b = item / (2 * hkv);
    const uint32_t uh = item - (uint32_t)b * 2 * hkv;
    const int w = uh >= hkv, h = uh - (w ? hkv : 0);
    if (b >= p.rows.B) return;
    const int len = p.lens[b];
    uint32_t v[W];
    const __nv_bfloat16* head = (w ? p.x[1] : p.x[0]) + b * (w ? p.xs[1] : p.xs[0]) + h * D;
    const uint32_t* x = reinterpret_cast<const uint32_t*>(head) + W * lane;
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = x[i];
    if (len < 0) return;
    const int col = len >> page_log2, first = len & ((1 << page_log2) - 1);
    const int32_t pg = col < p.M ? p.table[b * p.M + col] : -1;
    if (pg < 0 || pg >= p.pages) {
        if (lane == 0) record_error_to(p.err, 2);
        return;
    }
    float* sp = (w ? p.scale[1] : p.scale[0]) + (int64_t)pg * p.Hkv + h;
    const float was = *sp;
    uint32_t raw = 0, top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const uint32_t lo = v[i] & 0x7fffu, hi = v[i] >> 16 & 0x7fffu;
        raw = max(raw, max(lo, hi));
        if (lo < 0x7f80u) top = max(top, lo);
        if (hi < 0x7f80u) top = max(top, hi);
    }
    raw = __reduce_max_sync(0xffffffffu, raw);
    const float need = scale_for(__reduce_max_sync(0xffffffffu, top));
    const float now = first > 0 ? fmaxf(was, need) : need;
    if (lane == 0) *sp = now;
    uint8_t* page = (w ? p.code[1] : p.code[0]) + (((int64_t)pg << page_log2) * p.Hkv + h) * D;
    const int64_t row = (int64_t)p.Hkv * D;
    if (first > 0 && now != was)
        round_again<D / 8>(page, row, first * (D / 8), __fdiv_rn(was, now), lane, 32);
    const float inv = exact_inverse(now);
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < W; ++i)
        o |= (inv != 0.f && raw < 0x7f80u ? codes_of(v[i], inv) : any_codes_of(v[i], now))
             << (16 * i);
    uint8_t* out = page + first * row + 2 * W * lane;
    if (W == 2) *reinterpret_cast<uint32_t*>(out) = o;
    else *reinterpret_cast<uint16_t*>(out) = (uint16_t)o;
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
    int vec_scales;              // a group's scales may be read as one vector
    int64_t pages;
    float scale_log2;            // softmax scale * log2(e)
    int whole_rows;              // every key: rows are dealt out whole
    int cluster;                 // > 0: a row is a cluster's, of that many CTAs
    __nv_bfloat16* O;            // [T][Hq][d]
    float* lse;                  // [T][Hq] or null
    // Rows that several CTAs share, per (CTA, its first or its last row, head): sums of
    // 2^(y - My + 15) V, and (Mx, My, l), see attn_kernel; per CTA which rows these are.
    float* part_o;               // [C][2][Hq][d]
    float* part_m;               // [C][2][Hq][4]
    int4* part_row;              // [min(T, C)], null: no row is shared
    int* err;
};

constexpr int kConsumers = 8;    // consumer warps
constexpr int kKeys = 32;        // keys of one unit: a stage of the ring
constexpr int kMaxScan = 512;    // rows whose lengths a CTA adds up itself
constexpr float kWeightLog2 = 15.f;                // the largest fp16 weight is 2^15
constexpr float kWeightScale = 3.0517578125e-05f;  // 2^-15

template <int D, int HG>
struct AttnCfg {
    static constexpr int NSUB = kConsumers / HG;        // warps that take turns at a head's units
    static constexpr int BOX = kKeys * D;               // one head's K (or V) codes of a unit
    static constexpr int STAGE = 2 * HG * BOX;
    static constexpr int FIT = 4 * 32768 / STAGE;
    static constexpr int STAGES = FIT == 4 ? 6 : FIT < 16 ? FIT : 16;
    static constexpr int PRODUCERS = FIT == 4 ? 3 : 4;  // producer warps
    static constexpr int THREADS = (kConsumers + PRODUCERS) * 32;
    // A stage always belongs to the same producer warp and the same consumers: a barrier's
    // parity only tells neighbouring phases apart, so whoever waits for a phase has to have
    // waited for (or caused) the one before it.
    static_assert(STAGES % PRODUCERS == 0 && STAGES % NSUB == 0, "");
    static_assert(NSUB > 1, "the warps of a head join their sums behind a barrier");
    static constexpr int OROW = D + 4;
    static constexpr int O_AT = STAGES * STAGE;
    static constexpr int SC_AT = O_AT + (kConsumers - HG) * 8 * OROW * 4;
    static constexpr int M_AT = SC_AT + STAGES * HG * kKeys * 8;
    static constexpr int SCAN_AT = M_AT + (kConsumers + HG) * 8 * 16;
    static constexpr int BAR_AT = SCAN_AT + (kMaxScan + 2) * 8;
    static constexpr int SMEM = BAR_AT + STAGES * 20;
};

// What a producer warp waits for before it leaves, whose units are every PRODUCERS-th up to
// `issued` (-1: none): those whose stage it has not taken again, so whose copies may be in
// flight.  It depends on what was issued alone, not on how many units were still to come.
template <int STAGES, int PRODUCERS, typename Wait>
__host__ __device__ __forceinline__ void drain(int issued, Wait&& wait) {
    for (int j = issued; j >= 0 && j + STAGES > issued; j -= PRODUCERS) wait(j);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The sequence of row t and the number of keys it sees; false: the row belongs
// to no sequence (it lies behind the last one).
__device__ __forceinline__ bool find_row(const AttnParams& p, int64_t t, bool report, int& b,
                                         int64_t& n) {
    const Rows& rw = p.rows;
    b = 0;
    n = 0;
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
            if (report) record_error_to(p.err, 2);
            n = 0;
        }
        // rows of a sequence are its last tokens; over every key they are causal
        if (p.idx == nullptr) n -= later;
    }
    const int64_t cap = (int64_t)p.M << p.page_log2;
    if (n > cap) {
        if (report) record_error_to(p.err, 2);
        n = cap;
    }
    if (n < 0) n = 0;
    return true;
}

__device__ __forceinline__ int64_t row_units(const AttnParams& p, int64_t t) {
    int b;
    int64_t n;
    find_row(p, t, false, b, n);
    return n <= kKeys ? 1 : (n + kKeys - 1) / kKeys;  // a row without keys has a unit, too
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
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

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// The rows and units of one CTA, in order.  The units of all rows, laid end to
// end, are cut into equal ranges, one per CTA (whole_rows: CTA c takes the rows
// c, c + C, ...; cluster: the CTAs of a cluster share one row).  Every warp walks
// by itself.
struct Walk {
    int64_t t;           // row
    int64_t a, b, all;   // this CTA's units [a, b) of the row's [0, all)
    int64_t left;        // units of later rows
    int64_t U, C;        // all units, and the CTAs that share them

    template <bool DENSE>
    __device__ __forceinline__ void open(const AttnParams& p, const int64_t* scan) {
        left = 0;
        if (p.cluster > 0) {
            t = blockIdx.x / p.cluster;
            const int64_t r = blockIdx.x % p.cluster;
            all = DENSE ? row_units(p, t) : (p.k + kKeys - 1) / kKeys;
            a = all * r / p.cluster;
            b = all * (r + 1) / p.cluster;
            return;
        }
        if (DENSE && p.whole_rows) {
            t = blockIdx.x;
            a = 0;
            b = all = t < p.rows.n ? row_units(p, t) : 0;
            return;
        }
        const int64_t per = (p.k + kKeys - 1) / kKeys;
        U = DENSE ? scan[p.rows.n] : p.rows.n * per;
        C = U < gridDim.x ? U : gridDim.x;  // CTAs behind the last unit have none
        const int64_t c = blockIdx.x < C ? blockIdx.x : C;
        const int64_t u0 = U * c / C, u1 = c < C ? U * (c + 1) / C : U;
        if (DENSE) {
            int lo = 0, hi = (int)p.rows.n - 1;  // the last row that starts at u0 or before
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (scan[mid] <= u0) lo = mid;
                else hi = mid - 1;
            }
            t = lo;
            all = scan[lo + 1] - scan[lo];
            a = u0 - scan[lo];
        } else {
            t = u0 / per;
            all = per;
            a = u0 - t * per;
        }
        left = u1 - u0;
        b = a + left < all ? a + left : all;
        left -= b - a;
    }

    __device__ __forceinline__ bool done() const { return a >= b; }

    template <bool DENSE>
    __device__ __forceinline__ void next(const AttnParams& p, const int64_t* scan) {
        a = 0;
        if (DENSE && p.whole_rows) {
            t += gridDim.x;
            b = all = t < p.rows.n ? row_units(p, t) : 0;
            return;
        }
        ++t;
        if (left == 0) {
            b = 0;
            return;
        }
        if (DENSE) all = scan[t + 1] - scan[t];
        b = left < all ? left : all;
        left -= b;
    }
};

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// Joins the row of a cluster: every CTA's sums lie in its shared memory, [HG][8][D]
// at its start and (Mx, My, l) in row_s; CTA r writes every cluster-th piece.  Saves the
// second kernel: one row of 2048 keys 9.3 -> 8.1 us, three rows of up to 300 keys 7.8 -> 6.2.
template <int D, int HG>
__device__ __forceinline__ void merge_cluster(const AttnParams& p, const uint8_t* smem,
                                              const float4* row_s, int h0) {
    cluster_sync();
    const int n = p.cluster, rank = blockIdx.x % n;
    const int64_t t = blockIdx.x / n, Hq = (int64_t)p.Hkv * p.G;
    const bool write =
        p.rows.off == nullptr || (t >= p.rows.off[0] && t < p.rows.off[p.rows.B]);
    auto remote = [&](const void* q, int r) {
        uint32_t a;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(q)), "r"(r));
        float4 v;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(a)
                     : "memory");
        return v;
    };
    const int pieces = HG * p.G * (D / 4);
    for (int e = threadIdx.x * n + rank; write && e < pieces; e += kConsumers * 32 * n) {
        const int hq = e / (D / 4), c = e % (D / 4);
        const int at = hq / p.G * 8 + hq % p.G;
        float4 m[8], v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < n) {
                m[r] = remote(row_s + at, r);
                v[r] = remote(smem + (at * (D / 4) + c) * 16, r);
            }
        float Mx = -INFINITY, My = -INFINITY;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < n) {
                Mx = fmaxf(Mx, m[r].x);
                My = fmaxf(My, m[r].y);
            }
        const float ux = Mx == -INFINITY ? 0.f : Mx, uy = My == -INFINITY ? 0.f : My;
        float ls = 0.f, acc[4] = {};
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < n && m[r].z != 0.f) {  // a CTA without units left no sums
                ls += m[r].z * ex2(m[r].x - ux);
                const float f = ex2(m[r].y - uy);
                acc[0] += v[r].x * f;
                acc[1] += v[r].y * f;
                acc[2] += v[r].z * f;
                acc[3] += v[r].w * f;
            }
        const float f = ls == 0.f ? 0.f : kWeightScale / ls, s = ex2(My - Mx);
        uint32_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(ls == 0.f ? 0.f : acc[2 * j] * f * s,
                                                           ls == 0.f ? 0.f : acc[2 * j + 1] * f * s);
            o[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        const int64_t head = (int64_t)h0 * p.G + hq;
        *reinterpret_cast<uint2*>(p.O + (t * Hq + head) * D + 4 * c) = make_uint2(o[0], o[1]);
        if (p.lse != nullptr && c == 0)
            p.lse[t * Hq + head] = ls == 0.f ? -INFINITY : (Mx + log2f(ls)) * 0.6931471805599453f;
    }
    // nobody leaves while its sums are read
    cluster_sync();
}

// Attention of rows over cached keys.  A CTA serves HG neighbouring KV heads of
// its range of units (32 keys of one row): three or four producer warps bring
// units into a ring of shared-memory stages, eight consumer warps compute, HG of
// them, one per head, at each unit, the others at the units between.
//
// Measured on 32/4 heads of 128 (device time).  Over every key, 8 rows of 16K to
// 128K keys: 95.8 us, 6.0 TB/s of codes (92 % of a copy's rate), bound by HBM.  64 rows
// of 2048 selected keys: 31.0 us, 4.4 TB/s: the keys at HBM's rate for 512-byte pieces
// (24 us at the 5.6 TB/s that 300 rows and 600 rows reach) behind a single row's chain of
// dependent loads (index row, table, codes).  1000 rows of one chunk over a cache that fits
// L2: 285 us, 7.4 TB/s of gathered codes; issue slots are 54 % and the ALU pipe 49 % busy
// (widening codes takes half of it) with 11 warps per SM (a twelfth would fit 168
// registers, but six stages of 32 KB do not divide among four producers); the copies alone
// take 234 us with four producers.  One row of 2048: 7.8 us, latency.  Loads straight to
// registers, 16 warps per SM without a ring, took 242.6, 63.9, 444.9 and 11.5.
// Tried and slower: e4m3 operands on mma.sync, which converts inside (24 cycles against
// 8.4 for fp16's with fresh operands); V read transposed by ldmatrix b8 instead of byte
// permutes (305 us on the chunk against 295, for want of registers); 16 consumer warps
// (408, spills); the next unit's scores beside this one's softmax (354, holds stages).
//
// Copies.  Selected keys are gathered with 16-byte cp.async, a warp taking a
// key's HG * d bytes at once (one bulk copy for each row this short keeps the copy
// engine from the rate that the load path reaches).  Over every key a unit comes as
// one TMA box per head, or as two where it covers two pages of 16.  Either way a
// head's 32 rows of d bytes lie with their 16-byte pieces exclusive-or'ed by the
// row, as TMA's swizzle does.
//
// S^T = K Q^T: 16 keys are the rows of an m16n8k16 product, the head group's
// queries (up to 8) its columns.  The sum over d may run in any order, so thread
// (g, t) of the quad layout takes d = 16 t .. 16 t + 15 of its two keys as one
// 16-byte read, which feeds four products; Q is laid out to match, once per row.
// K is exact in fp16; Q's bf16 is made exact in fp16 by a power of two per head
// that puts its largest element at 2^14 (what falls below 2^-24 there is under
// 2^-38 of that element).
//
// O^T += V^T P: the rows are d, the columns heads, the depth the 16 keys.
// Thread (g, t) needs four keys at its d, again 16 contiguous bytes of each key;
// byte permutes pair two keys' codes before widening.  The score tile's (key,
// head) fragment becomes the (head, key) operand by an 8x8 transpose in
// registers.  Which key stands at which place of a tile is free: `place` orders
// them so that the eight threads of a shared access meet eight different
// 16-byte columns, for K (two keys x 64 bytes) and for V (four keys x 32).
//
// Softmax in log2 units: x = score, y = x + log2(v_scale[key]).  Two running
// maxima are kept: Mx for l = sum 2^(x - Mx), My for the weights 2^(y - My) that
// multiply the V codes, so the weights are at most 1 whatever the scales are:
// O = (sum 2^(y - My) code) * 2^(My - Mx) / l.  They are held times 2^15 in fp16:
// rounding them costs 2^-11 each, an eighth of the output's own bf16 rounding, down
// to 2^-29 of the largest, and 2^-40 of it below, so that a long tail of
// small weights (2^18 keys and more) still counts.
template <int D, int HG, bool DENSE>
__global__ void __launch_bounds__(AttnCfg<D, HG>::THREADS, 1)
attn_kernel(const AttnParams p, const __grid_constant__ CUtensorMap mk,
            const __grid_constant__ CUtensorMap mv) {
    using C = AttnCfg<D, HG>;
    constexpr int NL = D / 64;       // 16-byte reads per key row and quad thread
    constexpr int MT = D / 16;       // m16 tiles of d
    constexpr int VW = D / 32;       // 32-bit words of one key's V row per thread
    extern __shared__ __align__(1024) uint8_t smem[];
    float* o_s = reinterpret_cast<float*>(smem + C::O_AT);       // [warp][8][OROW]
    float2* sc_s = reinterpret_cast<float2*>(smem + C::SC_AT);   // [stage][HG][32]: k scale, log2 v
    float4* m_s = reinterpret_cast<float4*>(smem + C::M_AT);     // [warp][8]: Mx, My, l
    float4* row_s = m_s + kConsumers * 8;                        // [HG][8]: the same of the row
    int64_t* scan = reinterpret_cast<int64_t*>(smem + C::SCAN_AT);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_AT);
    uint64_t* empty = full + C::STAGES;
    uint32_t* mask_s = reinterpret_cast<uint32_t*>(empty + C::STAGES);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h0 = blockIdx.y * HG;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), DENSE ? 1 : 33);
            mbar_init(smem_u32(&empty[s]), HG);
        }
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (DENSE && !p.whole_rows && p.cluster == 0) {
        for (int t = threadIdx.x; t < p.rows.n; t += C::THREADS) scan[t + 1] = row_units(p, t);
        __syncthreads();
        if (warp == 0) {
            int64_t base = 0;
            for (int t0 = 0; t0 < p.rows.n; t0 += 32) {
                int64_t v = t0 + lane < p.rows.n ? scan[t0 + lane + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int64_t w = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += w;
                }
                if (t0 + lane < p.rows.n) scan[t0 + lane + 1] = base + v;
                base += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) scan[0] = 0;
        }
    }
    __syncthreads();

    Walk w{};
    w.open<DENSE>(p, scan);

    if (warp >= kConsumers) {
        // ------------------------------------------------ producers
        const int pw = warp - kConsumers;
        const int rb = p.Hkv * D;
        int i = pw;                    // this warp's units: pw, pw + PRODUCERS, ...
        int64_t u = w.a + pw;          // the unit to look at next, inside row w.t
        int issued = -1;
        bool ok = true;
        int64_t tb = -1, n = 0;        // row of the cached lookup, its sequence and keys
        int b = 0;
        bool owned = false;
        // Moves on to a unit of this warp; false at the end.
        auto settle = [&] {
            while (!w.done() && u >= w.b) {
                u -= w.b;
                w.next<DENSE>(p, scan);
            }
            return !w.done();
        };
        bool more = settle();
        // A unit on its way: this lane's key, then its page, then the scales.  Each is asked
        // for one turn before it is used, so that a turn waits for none of these loads (from
        // DRAM 1 us each and dependent on each other).
        struct Unit {
            bool some;
            int b;
            int64_t n;
            int32_t key, pg;
            float ks[HG], vs[HG];
        };
        auto take = [&](Unit& x) {
            x.some = more;
            x.key = -1;
            if (!more) return;
            if (tb != w.t) {
                tb = w.t;
                owned = find_row(p, w.t, lane == 0, b, n);
            }
            x.b = b;
            x.n = n;
            const int64_t e = u * kKeys + lane;
            if (DENSE) {
                if (e < n) x.key = (int32_t)e;
            } else if (e < p.k && owned) {  // does not wait for the sequence's length
                x.key = p.idx[w.t * p.k + e];
            }
            u += C::PRODUCERS;
            more = settle();
        };
        auto ask_page = [&](Unit& x) {
            x.pg = -1;
            if (x.key >= 0 && x.key < x.n)
                x.pg = p.table[(int64_t)x.b * p.M + (x.key >> p.page_log2)];
        };
        auto ask_scales = [&](Unit& x) {
            if (x.pg < 0 || x.pg >= p.pages) {
                if (x.key >= 0) record_error_to(p.err, 2);
                x.pg = -1;
            }
            const int64_t at = (int64_t)max(x.pg, 0) * p.Hkv + h0;
            const float *a = p.scale[0] + at, *c = p.scale[1] + at;
            if (HG == 4 && p.vec_scales) {
                const float4 k = *reinterpret_cast<const float4*>(a);
                const float4 v = *reinterpret_cast<const float4*>(c);
                x.ks[0] = k.x; x.ks[1 % HG] = k.y; x.ks[2 % HG] = k.z; x.ks[3 % HG] = k.w;
                x.vs[0] = v.x; x.vs[1 % HG] = v.y; x.vs[2 % HG] = v.z; x.vs[3 % HG] = v.w;
            } else {
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    x.ks[h] = a[h];
                    x.vs[h] = c[h];
                }
            }
        };
        Unit now, next, after;
        take(now);
        take(next);
        ask_page(now);
        take(after);
        ask_page(next);
        ask_scales(now);
        while (now.some && ok) {
            Unit last;
            ask_scales(next);
            ask_page(after);
            take(last);

            const int s = i % C::STAGES;
            if (i >= C::STAGES) {
                bool got = false;
                if (lane == 0)
                    got = mbar_wait_to(p.err, smem_u32(&empty[s]), ((i / C::STAGES) - 1) & 1);
                ok = __shfl_sync(0xffffffffu, got, 0);
                if (!ok) break;
            }
            const bool valid = now.pg >= 0;
            const int32_t row = (int32_t)((uint32_t)now.pg << p.page_log2) +
                                (now.key & ((1 << p.page_log2) - 1));  // below 2^31
            const uint32_t bal = __ballot_sync(0xffffffffu, valid);
            const uint32_t base = smem_u32(smem + s * C::STAGE), fb = smem_u32(&full[s]);
            if constexpr (!DENSE) {
                if (bal) {
                    constexpr int CPR = HG * D / 16;   // 16-byte pieces of a key's row
                    constexpr int RPI = 32 / CPR;      // rows per instruction
                    const int c = lane % CPR, r0 = lane / CPR;
                    const int hh = c / (D / 16), cc = c % (D / 16);
                    const uint8_t* kp = p.code[0] + h0 * D + c * 16;
                    const uint8_t* vp = p.code[1] + h0 * D + c * 16;
                    const uint32_t dst = base + hh * C::BOX;
#pragma unroll
                    for (int q = 0; q < kKeys / RPI; ++q) {
                        const int r = r0 + q * RPI;
                        const int64_t src = (int64_t)__shfl_sync(0xffffffffu, row, r) * rb;
                        const int sw = D == 128 ? cc ^ (r & 7) : cc ^ (r >> 1 & 3);
                        if (bal >> r & 1u) {
                            cp_async16(dst + r * D + sw * 16, kp + src);
                            cp_async16(dst + HG * C::BOX + r * D + sw * 16, vp + src);
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < HG; ++h)
                sc_s[(s * HG + h) * kKeys + lane] =
                    make_float2(now.ks[h], valid ? __log2f(now.vs[h]) : 0.f);
            if (lane == 0) mask_s[s] = bal;
            __syncwarp();
            if constexpr (DENSE) {
                // one box per head and tensor, two where a page is half a unit
                const int boxes = p.page_log2 < 5 ? 2 : 1, rows = kKeys / boxes;
                const int32_t r1 = __shfl_sync(0xffffffffu, row, 16);
                if (lane == 0) {
                    const bool have[2] = {(bal & 1u) != 0, boxes == 2 && (bal >> 16 & 1u)};
                    mbar_arrive_expect_tx(fb, (have[0] + have[1]) * 2 * HG * rows * D);
                    for (int q = 0; q < boxes; ++q)
                        if (have[q])
#pragma unroll
                            for (int h = 0; h < HG; ++h) {
                                const uint32_t dst = base + h * C::BOX + q * rows * D;
                                const int32_t z = q ? r1 : row;
                                tma_load_3d(dst, &mk, fb, 0, h0 + h, z);
                                tma_load_3d(dst + HG * C::BOX, &mv, fb, 0, h0 + h, z);
                            }
                }
            } else {
                cp_async_arrive(fb);
                if (lane == 0) mbar_arrive(fb);
            }
            issued = i;
            i += C::PRODUCERS;
            now = next;
            next = after;
            after = last;
        }
        if (pw == 0 && blockIdx.y == 0 && p.rows.off != nullptr)
            // here, as the consumers have no registers to spare and are not done yet
#pragma unroll 1
            for (int seq = blockIdx.x * 32 + lane; seq < p.rows.B; seq += gridDim.x * 32)
                check_offsets(p.rows, p.err, seq);
        // copies in flight end before the CTA does, also where a wait gave up above
        if (lane == 0)
            drain<C::STAGES, C::PRODUCERS>(issued, [&](int j) {
                mbar_wait_to(p.err, smem_u32(&full[j % C::STAGES]), (j / C::STAGES) & 1);
            });
        return;
    }

    // ---------------------------------------------------- consumers
    const int h = warp % HG, sub = warp / HG;
    const int g = lane >> 2, t4 = lane & 3;
    auto place = [](int m) { return (int)((D == 128 ? 0x37156240u : 0x65742130u) >> (4 * m) & 7u); };
    const int pk = place(g);
    const uint8_t* mine = smem + h * C::BOX;
    uint32_t koff[NL], voff[2];
#pragma unroll
    for (int i = 0; i < NL; ++i)
        koff[i] = pk * D + (D == 128 ? (4 * i + t4) ^ pk : t4 ^ (pk >> 1)) * 16;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = place(2 * t4 + e);
        voff[e] = HG * C::BOX + r * D +
                  (D == 128 ? (g ^ r) * 16 : ((g >> 1) ^ (r >> 1)) * 16 + (g & 1) * 8);
    }

    int done = 0;  // units before this one
    bool ok = true;
    int2 last = make_int2(-1, -1);
    const bool none = w.done();
    for (; !w.done(); w.next<DENSE>(p, scan)) {
        // Q, scaled by 2^qe
        uint32_t qf[NL][4][2];
        float qs[2];                           // for heads 2 t4, 2 t4 + 1
        {
            const __nv_bfloat16* q = p.Q + (w.t * p.Hkv * p.G + (int64_t)(h0 + h) * p.G + g) * D;
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
            // an infinity makes every score infinite or NaN, so the softmax NaN: said here, as
            // scores that are all -inf would pass for a row without keys
            const float back = top >= 0x7f80u
                                   ? NAN
                                   : p.scale_log2 * __uint_as_float((uint32_t)(127 - qe) << 23);
            qs[0] = __shfl_sync(0xffffffffu, back, 8 * t4);
            qs[1] = __shfl_sync(0xffffffffu, back, 8 * t4 + 4);
        }

        float o[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        float mx[2] = {-INFINITY, -INFINITY}, my[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int64_t u = w.a; u < w.b; ++u, ++done) {
            if (done % C::NSUB != sub) continue;
            const int st = done % C::STAGES;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_to(p.err, smem_u32(&full[st]),
                                                              (done / C::STAGES) & 1));
            const uint32_t msk = ok ? mask_s[st] : 0u;
            if (msk) {
                const uint8_t* at = mine + st * C::STAGE;
                const float2* sc = sc_s + (st * HG + h) * kKeys + pk;
                float x[2][4], y[2][4];
                float s[2][4] = {};
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    uint4 kr[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            kr[j][r] = *reinterpret_cast<const uint4*>(at + koff[i] +
                                                                       (16 * j + 8 * r) * D);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t k0 = word(kr[j][0], q), k1 = word(kr[j][1], q);
                            const uint32_t a[4] = {widen(k0), widen(k1), widen(k0 >> 16),
                                                   widen(k1 >> 16)};
                            mma_f16(s[j], a, qf[i][q][0], qf[i][q][1]);
                        }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 f = sc[16 * j + 8 * r];
                        const bool in = msk >> (16 * j + 8 * r + pk) & 1u;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            x[j][2 * r + c] = in ? s[j][2 * r + c] * (f.x * qs[c]) : -INFINITY;
                            y[j][2 * r + c] = x[j][2 * r + c] + f.y;
                        }
                    }
                }
                float wgt[2][4], fy[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float ax = fmaxf(fmaxf(x[0][c], x[0][c + 2]), fmaxf(x[1][c], x[1][c + 2]));
                    float ay = fmaxf(fmaxf(y[0][c], y[0][c + 2]), fmaxf(y[1][c], y[1][c + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        ax = fmaxf(ax, __shfl_xor_sync(0xffffffffu, ax, d));
                        ay = fmaxf(ay, __shfl_xor_sync(0xffffffffu, ay, d));
                    }
                    const float nx = fmaxf(mx[c], ax), ny = fmaxf(my[c], ay);
                    const float ux = nx == -INFINITY ? 0.f : nx, uy = ny == -INFINITY ? 0.f : ny;
                    const float fx = ex2(mx[c] - ux);
                    fy[c] = ex2(my[c] - uy);
                    const float ry = uy - kWeightLog2;
                    mx[c] = nx;
                    my[c] = ny;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            sum += ex2(x[j][2 * r + c] - ux);
                            wgt[j][2 * r + c] = ex2(y[j][2 * r + c] - ry);
                        }
                    l[c] = l[c] * fx + sum;
                }
                if (__any_sync(0xffffffffu, fy[0] != 1.f || fy[1] != 1.f)) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[i][c] *= fy[c & 1];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t vr[4][VW];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint8_t* q = at + voff[e & 1] + (16 * j + (e >> 1) * 8) * D;
                        if constexpr (VW == 4) {
                            const uint4 v = *reinterpret_cast<const uint4*>(q);
                            vr[e][0] = v.x; vr[e][1] = v.y; vr[e][2 % VW] = v.z; vr[e][3 % VW] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(q);
                            vr[e][0] = v.x; vr[e][1] = v.y;
                        }
                    }
                    if (msk != 0xffffffffu) {  // what lies in an absent key's place may be NaN
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(msk >> (16 * j + (e >> 1) * 8 + place(2 * t4 + (e & 1))) & 1u))
#pragma unroll
                                for (int q = 0; q < VW; ++q) vr[e][q] = 0;
                    }
                    uint32_t pf[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const __half2 v = __floats2half2_rn(wgt[j][2 * r], wgt[j][2 * r + 1]);
                        pf[r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&v));
                    }
#pragma unroll
                    for (int i = 0; i < VW; ++i)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t sel = q ? 0x7362u : 0x5140u;
                            const uint32_t lo = __byte_perm(vr[0][i], vr[1][i], sel);
                            const uint32_t hi = __byte_perm(vr[2][i], vr[3][i], sel);
                            const uint32_t a[4] = {widen(lo), widen(lo >> 16), widen(hi),
                                                   widen(hi >> 16)};
                            mma_f16(o[2 * i + q], a, pf[0], pf[1]);
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
        }

        // ---- the warps' sums of this row
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
        constexpr int DT = 2 * MT;  // d of a thread: DT g .. DT g + DT - 1, o[i][c] and o[i][c + 2]
        named_bar_sync(1, kConsumers * 32);  // the row before has been read
        if (sub > 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float* q = o_s + ((warp - HG) * 8 + 2 * t4 + c) * C::OROW + DT * g;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    q[2 * i] = o[i][c];
                    q[2 * i + 1] = o[i][c + 2];
                }
                if (g == 0) m_s[warp * 8 + 2 * t4 + c] = make_float4(mx[c], my[c], l[c], 0.f);
            }
        }
        // the others' sums are there; nobody reads the ring for this row any more, where a
        // cluster's go below
        named_bar_sync(1, kConsumers * 32);
        const bool whole = w.a == 0 && w.b == w.all;
        if (p.part_row != nullptr && threadIdx.x == 0 && blockIdx.y == 0 && w.a == 0) {
            // for the merge: the CTAs of this row, named by the one that has its first unit
            int2 r = make_int2(-1, -1);
            if (!whole) {
                const int64_t end = w.all + (DENSE ? scan[w.t] : w.t * w.all);
                r = make_int2((int)w.t, (int)((end * w.C + w.U - 1) / w.U - 1));
            }
            if (p.rows.n <= gridDim.x)
                p.part_row[w.t] = make_int4(r.x, r.x < 0 ? 0 : (int)blockIdx.x, r.y, 0);
            else
                last = r;
        }
        if (sub > 0) continue;
        bool write = true;
        if (whole && p.rows.off != nullptr)
            write = w.t >= p.rows.off[0] && w.t < p.rows.off[p.rows.B];
        const int64_t Hq = (int64_t)p.Hkv * p.G;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int hh = 2 * t4 + c;
            if (!write || hh >= p.G) continue;
            float Mx = mx[c], My = my[c];
#pragma unroll
            for (int v = 1; v < C::NSUB; ++v) {
                const float4 m = m_s[(v * HG + h) * 8 + hh];
                Mx = fmaxf(Mx, m.x);
                My = fmaxf(My, m.y);
            }
            const float ux = Mx == -INFINITY ? 0.f : Mx, uy = My == -INFINITY ? 0.f : My;
            float ls = l[c] * ex2(mx[c] - ux);
            const float f0 = ex2(my[c] - uy);
            float acc[DT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                acc[2 * i] = o[i][c] * f0;
                acc[2 * i + 1] = o[i][c + 2] * f0;
            }
#pragma unroll
            for (int v = 1; v < C::NSUB; ++v) {
                const float4 m = m_s[(v * HG + h) * 8 + hh];
                ls += m.z * ex2(m.x - ux);
                const float f = ex2(m.y - uy);
                const float4* q = reinterpret_cast<const float4*>(
                    o_s + (((v - 1) * HG + h) * 8 + hh) * C::OROW + DT * g);
#pragma unroll
                for (int i = 0; i < DT / 4; ++i) {
                    const float4 a = q[i];
                    acc[4 * i] += a.x * f;
                    acc[4 * i + 1] += a.y * f;
                    acc[4 * i + 2] += a.z * f;
                    acc[4 * i + 3] += a.w * f;
                }
            }
            const int64_t head = (int64_t)(h0 + h) * p.G + hh;
            if (p.cluster > 1) {
                float4* out = reinterpret_cast<float4*>(smem) + ((h * 8 + hh) * D + DT * g) / 4;
#pragma unroll
                for (int i = 0; i < DT / 4; ++i)
                    out[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                if (g == 0) row_s[h * 8 + hh] = make_float4(Mx, My, ls, 0.f);
            } else if (whole) {
                const float f = ls == 0.f ? 0.f : kWeightScale / ls, e = ex2(My - Mx);
                uint4* out = reinterpret_cast<uint4*>(p.O + (w.t * Hq + head) * D + DT * g);
#pragma unroll
                for (int i = 0; i < DT / 8; ++i) {
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(
                            ls == 0.f ? 0.f : acc[8 * i + 2 * j] * f * e,
                            ls == 0.f ? 0.f : acc[8 * i + 2 * j + 1] * f * e);
                        v[j] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    out[i] = make_uint4(v[0], v[1], v[2], v[3]);
                }
                if (p.lse != nullptr && g == 0)
                    p.lse[w.t * Hq + head] = ls == 0.f ? -INFINITY
                                                       : (Mx + log2f(ls)) * 0.6931471805599453f;
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + (w.a > 0 ? 0 : 1)) * Hq + head;
                float4* out = reinterpret_cast<float4*>(p.part_o + at * D + DT * g);
#pragma unroll
                for (int i = 0; i < DT / 4; ++i)
                    out[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                if (g == 0)
                    *reinterpret_cast<float4*>(p.part_m + at * 4) = make_float4(Mx, My, ls, 0.f);
            }
        }
    }
    if (p.cluster > 1) {
        if (none && threadIdx.x < HG * 8)
            row_s[threadIdx.x] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        merge_cluster<D, HG>(p, smem, row_s, h0);
    }
    if (p.part_row != nullptr && threadIdx.x == 0 && blockIdx.y == 0 && p.rows.n > gridDim.x)
        p.part_row[blockIdx.x] = make_int4(last.x, (int)blockIdx.x, last.y, 0);
}

// Merges one head of a row that several CTAs shared.  part_row has an entry (row,
// first CTA, last CTA) or -1 per row, or per CTA where rows are more.
// Latency decides it (a row of 148 parts is 78 KB): all maxima are loaded at
// once, then D / 4 threads take a part, four loads in flight each.  One row of 32 parts
// went from 19.3 to 11.7 us in all against a thread per element walking the parts.
constexpr int kCombineThreads = 256;
constexpr int kMaxParts = 512;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const AttnParams p) {
    constexpr int LP = D / 4, NG = kCombineThreads / LP;
    __shared__ float f_s[kMaxParts];      // 2^(My of a part - My)
    __shared__ float red_s[3][kCombineThreads / 32];
    __shared__ float4 o_s[NG][LP];
    pdl_wait();
    const int4 r = p.part_row[blockIdx.x];
    if (r.x < 0) return;
    const int64_t t = r.x;
    if (p.rows.off != nullptr && (t < p.rows.off[0] || t >= p.rows.off[p.rows.B])) return;
    const int64_t Hq = (int64_t)p.Hkv * p.G, head = blockIdx.y;
    const int n = r.z - r.y + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto at = [&](int j) { return ((int64_t)(r.y + j) * 2 + (j == 0 ? 1 : 0)) * Hq + head; };
    float4 m[kMaxParts / kCombineThreads];
    float Mx = -INFINITY, My = -INFINITY;
#pragma unroll
    for (int q = 0; q < kMaxParts / kCombineThreads; ++q) {
        const int j = q * kCombineThreads + threadIdx.x;
        m[q] = j < n ? *reinterpret_cast<const float4*>(p.part_m + at(j) * 4)
                     : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        Mx = fmaxf(Mx, m[q].x);
        My = fmaxf(My, m[q].y);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, d));
        My = fmaxf(My, __shfl_xor_sync(0xffffffffu, My, d));
    }
    if (lane == 0) {
        red_s[0][warp] = Mx;
        red_s[1][warp] = My;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kCombineThreads / 32; ++q) {
        Mx = fmaxf(Mx, red_s[0][q]);
        My = fmaxf(My, red_s[1][q]);
    }
    const float ux = Mx == -INFINITY ? 0.f : Mx, uy = My == -INFINITY ? 0.f : My;
    float ls = 0.f;
#pragma unroll
    for (int q = 0; q < kMaxParts / kCombineThreads; ++q) {
        const int j = q * kCombineThreads + threadIdx.x;
        ls += m[q].z * ex2(m[q].x - ux);
        if (j < n) f_s[j] = ex2(m[q].y - uy);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
    if (lane == 0) red_s[2][warp] = ls;
    __syncthreads();
    ls = 0.f;
#pragma unroll
    for (int q = 0; q < kCombineThreads / 32; ++q) ls += red_s[2][q];
    const int g = threadIdx.x / LP, c = threadIdx.x % LP;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = g; j < n; j += NG) {
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + at(j) * D + 4 * c);
        const float f = f_s[j];
        acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
    }
    o_s[g][c] = acc;
    __syncthreads();
    if (threadIdx.x < D) {
        float a = 0.f;
        const int groups = n < NG ? n : NG;
        for (int q = 0; q < groups; ++q) a += reinterpret_cast<const float*>(o_s[q])[threadIdx.x];
        p.O[(t * Hq + head) * D + threadIdx.x] =
            __float2bfloat16_rn(ls == 0.f ? 0.f : a / ls * kWeightScale * ex2(My - Mx));
        if (p.lse != nullptr && threadIdx.x == 0)
            p.lse[t * Hq + head] = ls == 0.f ? -INFINITY : (Mx + log2f(ls)) * 0.6931471805599453f;
    }
}

// The same for rows of few parts, as many rows leave: a warp per head, which walks over
// them.  The chunk of 1000 rows 294 -> 285 us.
template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_few_kernel(const AttnParams p) {
    constexpr int E = D / 32;  // elements of a lane
    pdl_wait();
    const int4 r = p.part_row[blockIdx.x];
    const int64_t Hq = (int64_t)p.Hkv * p.G;
    const int64_t head = blockIdx.y * (kCombineThreads / 32) + (threadIdx.x >> 5);
    if (r.x < 0 || head >= Hq) return;
    const int64_t t = r.x;
    if (p.rows.off != nullptr && (t < p.rows.off[0] || t >= p.rows.off[p.rows.B])) return;
    const int n = r.z - r.y + 1, lane = threadIdx.x & 31;
    auto at = [&](int j) { return ((int64_t)(r.y + j) * 2 + (j == 0 ? 1 : 0)) * Hq + head; };
    // a part's maxima per lane
    float Mx = -INFINITY, My = -INFINITY;
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
        const float4 m = *reinterpret_cast<const float4*>(p.part_m + at(j) * 4);
        Mx = fmaxf(Mx, m.x);
        My = fmaxf(My, m.y);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, d));
        My = fmaxf(My, __shfl_xor_sync(0xffffffffu, My, d));
    }
    const float ux = Mx == -INFINITY ? 0.f : Mx, uy = My == -INFINITY ? 0.f : My;
    float ls = 0.f, acc[E] = {};
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int some = n - j0 < 32 ? n - j0 : 32;
        float g = 0.f;
        if (lane < some) {
            const float4 m = *reinterpret_cast<const float4*>(p.part_m + at(j0 + lane) * 4);
            ls += m.z * ex2(m.x - ux);
            g = ex2(m.y - uy);
        }
#pragma unroll 16
        for (int j = 0; j < some; ++j) {
            const float* q = p.part_o + at(j0 + j) * D + E * lane;
            const float f = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2*>(q + e);
                acc[e] += v.x * f;
                acc[e + 1] += v.y * f;
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
    const float f = ls == 0.f ? 0.f : kWeightScale / ls, s = ex2(My - Mx);
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(p.O + (t * Hq + head) * D + E * lane + e) =
            __floats2bfloat162_rn(ls == 0.f ? 0.f : acc[e] * f * s,
                                  ls == 0.f ? 0.f : acc[e + 1] * f * s);
    if (p.lse != nullptr && lane == 0)
        p.lse[t * Hq + head] = ls == 0.f ? -INFINITY : (Mx + log2f(ls)) * 0.6931471805599453f;
}

}  // namespace kv8
}  // namespace dsa
