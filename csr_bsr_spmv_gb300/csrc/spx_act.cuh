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

// 1 / (1 + exp(-z)), z within +-88, where the exponential is finite, from the
// hardware's 2^t and 1 / y (off by two and one units in the last place): the
// rounding of t = z log2(e) is put back to first order, 2^(t + d) = 2^t (1 + d
// ln 2).  Off by less than 2^-21 of itself, and 0 below 1e-38.
__device__ __forceinline__ float logistic(float z) {
    constexpr float L = 1.44269502f, rest = 1.92596303e-8f;  // log2(e) = L + rest
    const float t = -z * L, d = fmaf(-z, rest, fmaf(-z, L, -t));
    float e, p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = fmaf(e, d * 0.693147181f, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.f + e));
    return p;
}

constexpr float kTanh1 = 1.5957691216f, kTanh3 = 0.07135481628f;  // 2 sqrt(2 / pi), and that times 0.044715

template <int kind>
__device__ __forceinline__ float act_of(float x) {
    if (kind == SPX_ACT_SILU) {
        const float cut = at_least(x, -88.f);
        return cut * logistic(at_most(cut, 88.f));
    }
    const float cut = at_least(x, -100.f);
    if (kind == SPX_ACT_GELU) return cut * normcdff(x);
    const float z = cut * fmaf(kTanh3, fminf(x * x, 1e4f), kTanh1);
    return cut * logistic(at_most(at_least(z, -88.f), 88.f));
}
template <int kind>
__device__ __forceinline__ float act_of(float x, float& slope) {
    if (kind == SPX_ACT_SILU) {
        const float cut = at_least(x, -88.f), z = at_most(cut, 88.f), p = logistic(z);
        slope = p * fmaf(z, 1.f - p, 1.f);
        return cut * p;
    }
    const float cut = at_least(x, -100.f), near = at_most(cut, 100.f), xx = near * near;
    if (kind == SPX_ACT_GELU) {
        const float p = normcdff(x);
        slope = fmaf(near * 0.3989422804f, expf(-0.5f * xx), p);
        return cut * p;
    }
    const float z = near * fmaf(kTanh3, xx, kTanh1), dz = fmaf(3.f * kTanh3, xx, kTanh1);
    const float p = logistic(at_most(at_least(z, -88.f), 88.f));
    slope = p * fmaf(near * dz, 1.f - p, 1.f);
    return cut * p;
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
