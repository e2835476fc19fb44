// spx_rows.cuh -- rows in pieces that a thread moves as one word: what the norm
// and the embedding kernels share.
#pragma once

#include "spx_experts.cuh"

namespace spx_rows {

using namespace spx_exp;

// N values of V, N * sizeof(V) a power of two up to 16.
template <class V, int N>
struct alignas(N * sizeof(V) >= 16 ? 16 : N * sizeof(V)) Pack {
    V v[N];
};

// A piece is written as one word of its size; `once`: it is not read again soon.
template <class P>
__device__ __forceinline__ void write_piece(P* p, const P& v) {
    using T = typename Word<sizeof(P)>::T;
    T w;
    memcpy(&w, &v, sizeof(P));
    *reinterpret_cast<T*>(p) = w;
}
template <class P>
__device__ __forceinline__ void write_once(P* p, const P& v) {
    using T = typename Word<sizeof(P)>::T;
    T w;
    memcpy(&w, &v, sizeof(P));
    __stcs(reinterpret_cast<T*>(p), w);
}

// N values of type V or (wide) fp32, as fp32.
template <class V, int N>
__device__ __forceinline__ void load_floats(const void* p, bool wide, long long at, float (&f)[N]) {
    if (wide) {
        constexpr int Q = N < 4 ? N : 4;
#pragma unroll
        for (int i = 0; i < N / Q; ++i) {
            const Pack<float, Q> x = load(reinterpret_cast<const Pack<float, Q>*>(static_cast<const float*>(p) + at) + i);
#pragma unroll
            for (int j = 0; j < Q; ++j) f[Q * i + j] = x.v[j];
        }
    } else {
        const Pack<V, N> x = load(reinterpret_cast<const Pack<V, N>*>(static_cast<const V*>(p) + at));
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f(x.v[i]);
    }
}

// Sum (or maximum, as unsigned numbers) over the G threads of a group, G a power of two; groups of several warps meet in
// `s` (a word a warp) and the whole block has to call.
__device__ __forceinline__ float group_sum(float v, int G, float* s) {
    for (int d = (G < 32 ? G : 32) >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (G <= 32) return v;
    const int w = threadIdx.x >> 5, per = G >> 5, w0 = w & -per;
    if ((threadIdx.x & 31) == 0) s[w] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < per; ++i) v += s[w0 + i];
    return v;
}
__device__ __forceinline__ uint32_t group_max(uint32_t v, int G, uint32_t* s) {
    for (int d = (G < 32 ? G : 32) >> 1; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
    if (G <= 32) return v;
    const int w = threadIdx.x >> 5, per = G >> 5, w0 = w & -per;
    if ((threadIdx.x & 31) == 0) s[w] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < per; ++i) v = max(v, s[w0 + i]);
    return v;
}

}  // namespace spx_rows
