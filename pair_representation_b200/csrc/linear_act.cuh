// linear_act.cuh - the activations of the linear layers and their slopes.
//
// exp(-p) and 1 / (1 + exp(-p)) come from the hardware's ex2 and rcp (relative errors about
// 2^-22), far under the half step 2^-8 of the bf16 result. Those run at 16 a clock and SM, and at
// two for each value they, not memory, bound a wide layer's epilogue (589824 x 128 -> 512 with
// silu: 226 us, without activation 128). So two values share one reciprocal,
//   1 / a = b / (a b),  1 / b = a / (a b),
// which takes 1.5 for each. The product stays finite while both p are over -43; where one of the
// them is not, or is NaN, each takes its own.
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

// Whether pairs of these may share a reciprocal (false with a NaN among them). Asked once for all the
// values a thread has in hand: a test and branch for every eight kept the two warps of a scheduler
// from having enough exponentials in flight (286 us in the case above).
template <int N>
__device__ __forceinline__ bool can_share(const float2 (&p)[N]) {
    float m[4] = {p[0].x, p[0].y, p[1].x, p[1].y};
#pragma unroll
    for (int t = 2; t < N; ++t) {
        m[(2 * t) & 3] = min_nan(m[(2 * t) & 3], p[t].x);
        m[(2 * t + 1) & 3] = min_nan(m[(2 * t + 1) & 3], p[t].y);
    }
    return min_nan(min_nan(m[0], m[1]), min_nan(m[2], m[3])) >= -43.f;
}

// e = exp(-p) and 1 / (1 + e) of two values over -43.
__device__ __forceinline__ float2 sigmoid_shared(float2 p, float2 &e) {
    const float2 z = __fmul2_rn(p, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    e = make_float2(ex2f(z.x), ex2f(z.y));
    const float2 a = __fadd2_rn(e, make_float2(1.f, 1.f));
    const float r = rcpf(a.x * a.y);
    return __fmul2_rn(make_float2(r, r), make_float2(a.y, a.x));
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float p) {
    const float s = rcpf(1.f + ex2f(p * -1.4426950408889634f));  // 0 where exp(-p) is infinite
    return ACT == LIN_SIGMOID ? s : p * s;
}

// act'(p) d. 1 - s is taken as s exp(-p), which keeps its digits where s is next to 1. p stops at
// -87, where both factors are still finite and every slope is under 2e-36.
template <int ACT>
__device__ __forceinline__ float act_grad(float p, float d) {
    p = max_nan(p, -87.f);
    const float e = ex2f(p * -1.4426950408889634f), s = rcpf(1.f + e), c = s * e;
    return ACT == LIN_SIGMOID ? d * (s * c) : d * fmaf(p * s, c, s);
}

// Two values: act(p), and act'(p) d (not relu's, whose sign may need more than fp32: see its own
// code). kShare: can_share holds.
template <int ACT, bool kShare>
__device__ __forceinline__ float2 act_fwd2(float2 p) {
    if (ACT == LIN_NONE) return p;
    if (ACT == LIN_RELU) return make_float2(max_nan(p.x, 0.f), max_nan(p.y, 0.f));
    if (!kShare) return make_float2(act_fwd<ACT>(p.x), act_fwd<ACT>(p.y));
    float2 e;
    const float2 s = sigmoid_shared(p, e);
    return ACT == LIN_SIGMOID ? s : __fmul2_rn(p, s);
}

template <int ACT, bool kShare>
__device__ __forceinline__ float2 act_grad2(float2 p, float2 d) {
    if (ACT == LIN_NONE) return d;
    if (!kShare) return make_float2(act_grad<ACT>(p.x, d.x), act_grad<ACT>(p.y, d.y));
    float2 e;
    const float2 s = sigmoid_shared(p, e), c = __fmul2_rn(s, e);
    return __fmul2_rn(d, ACT == LIN_SIGMOID ? __fmul2_rn(s, c) : __ffma2_rn(__fmul2_rn(p, s), c, s));
}

}  // namespace trimul
