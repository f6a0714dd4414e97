// linear_act.cuh - the activations of the linear layers and their slopes, the bound that decides relu's sign, and
// the value of an 8-bit activation's scale.
//
// exp(-p) and 1 / (1 + exp(-p)) come from the hardware's ex2 and rcp (relative errors about
// 2^-22), far under the half step 2^-8 of the bf16 result. Those run at 16 a clock and SM, and at
// two for each value they and the arithmetic around them, not memory, bound a wide layer's epilogue
// (589824 x 128 -> 512 with silu: 226 us, without activation 137). So four values share one
// reciprocal: of a b c d, times c d and then b it is 1 / a, and so on; 1.25 for each, and fewer
// instructions too: 162 us (short runs at full clock, here and below). The product stays finite while
// all four p are over -21; where one of the values a thread has in hand is not, or is NaN, each takes
// its own (at p of size 11, where most threads have such a value, the same call takes 273 us).
#pragma once

#include "kernels.h"

namespace trimul {

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float min3_nan(float a, float b, float c) {
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Whether these may share reciprocals (false with a NaN among them). Asked once for all the
// values a thread has in hand: a test and branch for every eight kept the two warps of a scheduler
// from having enough exponentials in flight (286 us in the case above).
template <int N>
__device__ __forceinline__ bool can_share(const float2 (&p)[N]) {
    float m[2] = {p[0].x, p[0].y};
#pragma unroll
    for (int t = 1; t < N; ++t) m[t & 1] = min3_nan(m[t & 1], p[t].x, p[t].y);
    return min_nan(m[0], m[1]) >= -21.f;
}

// 1 / (1 + exp(-p)) of four values over -21; e receives the exponentials.
__device__ __forceinline__ void sigmoid_shared(const float2 (&p)[2], float2 (&s)[2], float2 (&e)[2]) {
    const float2 l = make_float2(-1.4426950408889634f, -1.4426950408889634f), one = make_float2(1.f, 1.f);
    const float2 y = __fmul2_rn(p[0], l), z = __fmul2_rn(p[1], l);
    e[0] = make_float2(ex2f(y.x), ex2f(y.y));
    e[1] = make_float2(ex2f(z.x), ex2f(z.y));
    const float2 a = __fadd2_rn(e[0], one), c = __fadd2_rn(e[1], one), ac = __fmul2_rn(a, c);
    const float r = rcpf(ac.x * ac.y);
    const float2 t = make_float2(r * ac.y, r * ac.x);  // 1 / (a.x c.x), 1 / (a.y c.y)
    s[0] = __fmul2_rn(t, c);
    s[1] = __fmul2_rn(t, a);
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float p) {
    const float s = rcpf(1.f + ex2f(p * -1.4426950408889634f));  // 0 where exp(-p) is infinite
    return ACT == LIN_SIGMOID ? s : p * s;
}

// act'(p) d. 1 - s is taken as s exp(-p), which keeps its digits where s is next to 1. p stops at
// -88: exp(-p) is finite there, and s, under the smallest normal number, is 0, and with it the slope, of
// -infinity too.
template <int ACT>
__device__ __forceinline__ float act_grad(float p, float d) {
    p = max_nan(p, -88.f);
    const float e = ex2f(p * -1.4426950408889634f), s = rcpf(1.f + e), c = s * e;
    return ACT == LIN_SIGMOID ? d * (s * c) : d * fmaf(p * s, c, s);
}

// Four values: p = act(p), and p = act'(p) d (not relu's, whose sign may need more than fp32: see its
// own code). kShare: can_share holds.
template <int ACT, bool kShare>
__device__ __forceinline__ void act_fwd4(float2 (&p)[2]) {
    if (ACT == LIN_NONE) return;
    float2 s[2], e[2];
    if (ACT != LIN_RELU && kShare) sigmoid_shared(p, s, e);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (ACT == LIN_RELU) p[t] = make_float2(max_nan(p[t].x, 0.f), max_nan(p[t].y, 0.f));
        else if (!kShare) p[t] = make_float2(act_fwd<ACT>(p[t].x), act_fwd<ACT>(p[t].y));
        else p[t] = ACT == LIN_SIGMOID ? s[t] : __fmul2_rn(p[t], s[t]);
    }
}

template <int ACT, bool kShare>
__device__ __forceinline__ void act_grad4(float2 (&p)[2], const float2 (&d)[2]) {
    float2 s[2], e[2];
    if (ACT != LIN_NONE && kShare) sigmoid_shared(p, s, e);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (ACT == LIN_NONE) {
            p[t] = d[t];
        } else if (!kShare) {
            p[t] = make_float2(act_grad<ACT>(p[t].x, d[t].x), act_grad<ACT>(p[t].y, d[t].y));
        } else {
            const float2 c = __fmul2_rn(s[t], e[t]);
            p[t] = __fmul2_rn(d[t], ACT == LIN_SIGMOID ? __fmul2_rn(s[t], c) : __ffma2_rn(__fmul2_rn(p[t], s[t]), c, s[t]));
        }
    }
}

// A scale byte's value: 2^(s - 127), at s = 0 a subnormal number; 255, which packing never writes, is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7FC00000u : s << 23);
}

// ---- the sign of relu's p -------------------------------------------------------------------------
// The accumulator's rounding decides the sign of a p next to 0, and a wrong one is not a small error of
// the gradient but the whole of dy. A step of 16 products cuts its 17 terms at 2^-25 of the largest and
// their sum at 2^-23 (measured: 1 and n terms of 2^-24, 2^-25, 2^-26 in one step give 1 + [n/2], [n/4], 0 steps
// of 2^-23, the lost parts towards 0): 17/4 + 1 steps of 2^-23, here 6, of a size that |x| |w| bounds (the
// norms: neither a term nor a partial sum is larger, by Cauchy and Schwarz). Where |p| is under
// the sum of these over the steps of the contraction, the kernels take p again in 64 bits. A row of zeros of
// x or W has bound 0, and is never asked for. At normal inputs about 5 in 10^5 places for 128
// products, 1 in 10^3 for 1024, 7 in 100 for 16384. The backward with relu, against a bound from the sums
// themselves, which missed signs where they cancel: 147456 x 128 -> 128 39 -> 44 us, x in 8 bits 45 -> 50, -> 512
// 125 -> 128; 147456 x 512 -> 128 138 -> 155; 28000 x 1024 -> 1024 243 -> 281; 3605 x 328 -> 200 26.6 -> 28.7; 3000 x
// 16384 -> 256 296 -> 1130 (inputs cold in L2; with a fifth of the rows 0 the first is 44 us as well, and was 758).
__device__ __forceinline__ float sign_bound(int k) { return (float)((k + 15) / 16) * (6.f * 1.1920929e-7f) * 1.0625f; }

// A row's norm from its sum of squares. Squares under 2^-126 may be lost, and products in p too: any norm but 0
// counts as 2^-50 at least, far over what is lost of it, and the bound of two such rows is over what p loses.
__device__ __forceinline__ float norm_of(float squares) { return squares > 0.f ? fmaxf(sqrtf(squares), 8.8817842e-16f) : 0.f; }

// s + the squares of two bf16, over 0 where one of them is not 0.
__device__ __forceinline__ float add_squares(float s, uint32_t w) {
    const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
    s = fmaf(a, a, fmaf(b, b, s));
    return (w & 0x7FFF7FFFu) ? fmaxf(s, 1.1754944e-38f) : s;
}

// Sums over the lanes of eight values each: lane l returns that of value l >> 2.
__device__ __forceinline__ float sums_of_8(const float (&v)[8], int lane) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = v[i];
#pragma unroll
    for (int w = 16, n = 4; n >= 1; w >>= 1, n >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? s[i + n] : s[i], give = up ? s[i] : s[i + n];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
    return s[0] + __shfl_xor_sync(0xffffffffu, s[0], 1);
}

}  // namespace trimul
