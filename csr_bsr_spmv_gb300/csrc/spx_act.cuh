// spx_act.cuh -- the activations of the experts' gate and their derivatives, in
// fp32 with CUDA's own functions.
#pragma once

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
// Beyond |x| = 100 p is 0 or 1 and the slope's other term 0 in fp32, so x is cut
// there (and far below in x p) where an infinity would meet that zero.  NaN
// passes through p.
__device__ __forceinline__ float act_of(int kind, float x) {
    const float cut = fmaxf(x, -1e30f);
    if (kind == SPX_ACT_GELU) return cut * normcdff(x);
    float z = x;
    if (kind == SPX_ACT_GELU_TANH) z = x * fmaf(0.07135481628f, fminf(x * x, 1e4f), 1.5957691216f);
    return cut / (1.f + expf(-z));
}
__device__ __forceinline__ float act_of(int kind, float x, float& slope) {
    const float cut = fmaxf(x, -1e30f), near = fminf(fmaxf(x, -100.f), 100.f);
    if (kind == SPX_ACT_GELU) {
        const float p = normcdff(x);
        slope = fmaf(near * 0.3989422804f, expf(-0.5f * x * x), p);
        return cut * p;
    }
    float z = x, dz = 1.f;
    if (kind == SPX_ACT_GELU_TANH) {
        const float xx = fminf(x * x, 1e4f);
        z = x * fmaf(0.07135481628f, xx, 1.5957691216f);
        dz = fmaf(3.f * 0.07135481628f, xx, 1.5957691216f);
    }
    const float p = 1.f / (1.f + expf(-z));
    slope = p * fmaf(near * dz, 1.f - p, 1.f);
    return cut * p;
}

}  // namespace spx_exp
