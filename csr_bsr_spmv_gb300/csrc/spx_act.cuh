// spx_act.cuh -- the activations of the experts' gate and their derivatives, in
// fp32.
#pragma once

#include <type_traits>

#include "spx_experts.cuh"

namespace spx_exp {

// What a product's sums pass through before they are stored.
enum Epilogue : int { kNone = 0, kGate = 1, kGateGrad = 2 };

// The gate of a product: kGate C = act(G) U, and H = G beside U where it is
// wanted; kGateGrad the sums are dC, and dH and (where wanted) C come from H.
struct Gate {
    Epilogue epi = kNone;
    int act = 0;
    void* H = nullptr;  // kGate: written, NULL: not; kGateGrad: read
    long long ldh = 0;
    void* dH = nullptr;
    long long lddh = 0;
};

// act(x) and act'(x).  All three are x p(x) with p in [0, 1], which keeps the
// small values far left of zero; the tanh form's p is the logistic function of
// z = 2 sqrt(2 / pi) (x + 0.044715 x^3), since (1 + tanh(z / 2)) / 2 is that.
// NaN passes; infinities give the limits: x is cut far out, where p is 0 or 1
// and the slope's other term 0 in fp32, before either could meet an infinity.
__device__ __forceinline__ float at_least(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float at_most(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 cut(float2 x, float most) {
    return make_float2(at_most(at_least(x.x, -most), most), at_most(at_least(x.y, -most), most));
}

// 1 / (1 + exp(-z)), z within +-88, where the exponential is finite, from the
// hardware's 2^t and 1 / y (off by two and one units in the last place): the
// rounding of t = -z log2(e), which is -(z log2(e) + t), is put back to first
// order, 2^(t + r) = 2^t (1 + r ln 2).  Off by less than 2^-21 of itself, and 0
// below 1e-38.  Two values at a time, as everything here: most of it is one
// instruction for both.
__device__ __forceinline__ float2 logistic(float2 z) {
    constexpr double log2e = 1.4426950408889634;
    constexpr float L = static_cast<float>(log2e), rest = static_cast<float>(log2e - static_cast<double>(L));
    const float2 t = __fmul2_rn(z, both(-L)), d = __ffma2_rn(z, both(rest), __ffma2_rn(z, both(L), t));
    float2 e, p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __fadd2_rn(__ffma2_rn(e, __fmul2_rn(d, both(-0.693147181f)), e), both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(e.y));
    return p;
}

// Phi(-|x|), |x| at most 100, and e = exp(-x^2 / 2).  Their quotient is smooth and falls like 1 / |x|: t P(t) with t = 1 / (1 +
// 0.35 |x|), P of degree 8 fitted in 40 digits to |x| up to 13.5, where Phi leaves fp32 (reweighted least squares, off by
// 2^-24.9 of itself); the exponential as above, with the rounding of x^2 put back as well.  Off by less than 2^-20.5 of itself;
// the activation of every 16-bit value comes out within 2^-20.9.  32768 x 2048 of 2048 bf16: the gate's gradient 245 us, with
// CUDA's normcdff and expf 301 (SiLU 235); the gated product 381 and 416 (SiLU 364).
__device__ __forceinline__ float2 normal_tail(float2 x, float2& e) {
    constexpr double half_log2e = 1.4426950408889634 / 2;
    constexpr float L = static_cast<float>(half_log2e), rest = static_cast<float>(half_log2e - static_cast<double>(L));
    constexpr float P[9] = {0.1396215697f, 0.1398590851f, 0.1198524147f, 0.1054330339f, -0.0229373839f, 0.1589296681f, -0.2555049107f, 0.1438724097f, -0.0291259024f};
    const float2 h = __fmul2_rn(x, x), low = __ffma2_rn(x, x, make_float2(-h.x, -h.y)), z = __fmul2_rn(h, both(-L));
    const float2 d = __ffma2_rn(low, both(L), __ffma2_rn(h, both(rest), __ffma2_rn(h, both(L), z)));
    const float2 y = __ffma2_rn(make_float2(fabsf(x.x), fabsf(x.y)), both(0.35f), both(1.f));
    float2 t, s = both(P[8]);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(y.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(y.y));
    e = __ffma2_rn(e, __fmul2_rn(d, both(-0.693147181f)), e);
#pragma unroll
    for (int i = 7; i >= 0; --i) s = __ffma2_rn(s, t, both(P[i]));
    return __fmul2_rn(__fmul2_rn(e, t), s);
}

constexpr float kTanh1 = 1.5957691216f, kTanh3 = 0.07135481628f;  // 2 sqrt(2 / pi), and that times 0.044715

template <int kind>
__device__ __forceinline__ float2 act_of(float2 x, float2& slope) {
    constexpr float most = kind == SPX_ACT_SILU ? 88.f : 100.f;
    const float2 low = make_float2(at_least(x.x, -most), at_least(x.y, -most)), near = make_float2(at_most(low.x, most), at_most(low.y, most));
    float2 z = near, dz = both(1.f), p;
    if (kind == SPX_ACT_GELU) {
        float2 e;
        const float2 q = normal_tail(near, e);
        p = make_float2(x.x > 0.f ? 1.f - q.x : q.x, x.y > 0.f ? 1.f - q.y : q.y);
        slope = __ffma2_rn(__fmul2_rn(near, both(0.3989422804f)), e, p);
        return __fmul2_rn(low, p);
    }
    if (kind == SPX_ACT_GELU_TANH) {
        const float2 xx = __fmul2_rn(near, near);
        z = cut(__fmul2_rn(near, __ffma2_rn(both(kTanh3), xx, both(kTanh1))), 88.f);
        dz = __ffma2_rn(both(3.f * kTanh3), xx, both(kTanh1));
    }
    p = logistic(z);
    const float2 q = __ffma2_rn(p, both(-1.f), both(1.f));  // 1 - p
    slope = __fmul2_rn(p, __ffma2_rn(kind == SPX_ACT_SILU ? near : __fmul2_rn(near, dz), q, both(1.f)));
    return __fmul2_rn(low, p);
}
template <int kind>
__device__ __forceinline__ float2 act_of(float2 x) {
    float2 slope;  // not used: its instructions go
    return act_of<kind>(x, slope);
}

// f with the activation as a constant (a lambda over std::integral_constant): a chunk of values then runs one straight
// piece of code.
template <class F>
__device__ __forceinline__ void with_act(int kind, F f) {
    if (kind == SPX_ACT_SILU) f(std::integral_constant<int, SPX_ACT_SILU>{});
    else if (kind == SPX_ACT_GELU) f(std::integral_constant<int, SPX_ACT_GELU>{});
    else f(std::integral_constant<int, SPX_ACT_GELU_TANH>{});
}

}  // namespace spx_exp
