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

// A piece is read (from shared memory) and written as one word of its size: its own copy would go value by value.
// `once`: it is not read again soon.
template <class P>
__device__ __forceinline__ P read_piece(const P* p) {
    const auto w = *reinterpret_cast<const typename Word<sizeof(P)>::T*>(p);
    P v;
    memcpy(&v, &w, sizeof(P));
    return v;
}
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

// A piece of 4, 8 or 16 bytes to shared memory, asynchronously.
template <class P>
__device__ __forceinline__ void copy_piece(P* to, const P* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (sizeof(P) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(sizeof(P) < 4 ? 4 : sizeof(P)) : "memory");
}

// The piece itself, loaded by now: the compiler would otherwise move a load down to where its value is used, and loads
// meant to be in flight together would wait for one another.
template <class P>
__device__ __forceinline__ P stay(P p) {
    if constexpr (sizeof(P) >= 4) {
        uint32_t w[sizeof(P) / 4];
        memcpy(w, &p, sizeof(P));
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(P) / 4); ++i) asm volatile("" : "+r"(w[i]));
        memcpy(&p, w, sizeof(P));
    } else {
        uint16_t w;
        memcpy(&w, &p, sizeof(P));
        asm volatile("" : "+h"(w));
        memcpy(&p, &w, sizeof(P));
    }
    return p;
}

// A piece's values as fp32 in pairs (N == 1: one value and a zero), and back.
template <int N>
struct Floats {
    float2 v[(N + 1) / 2];
};
template <class V, int N>
__device__ __forceinline__ Floats<N> floats(const Pack<V, N>& p) {
    Floats<N> f;
    if constexpr (N == 1) {
        f.v[0] = make_float2(to_f(p.v[0]), 0.f);
    } else if constexpr (sizeof(V) == 2) {
        uint32_t w[N / 2];
        memcpy(w, &p, sizeof(p));
#pragma unroll
        for (int i = 0; i < N / 2; ++i) f.v[i] = widen2<V>(w[i]);
    } else {
        memcpy(&f, &p, sizeof(p));
    }
    return f;
}
template <class V, int N>
__device__ __forceinline__ Pack<V, N> packed(const Floats<N>& f) {
    Pack<V, N> p;
    if constexpr (N == 1) {
        p.v[0] = from_f<V>(f.v[0].x);
    } else if constexpr (sizeof(V) == 2) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = narrow2<V>(f.v[i]);
        memcpy(&p, w, sizeof(p));
    } else {
        memcpy(&p, &f, sizeof(p));
    }
    return p;
}

// N values of type V or (wide) fp32, as fp32.
template <class V, int N>
__device__ __forceinline__ Floats<N> load_floats(const void* p, bool wide, long long at) {
    if constexpr (N * sizeof(V) <= 16)
        if (!wide) return floats(load(reinterpret_cast<const Pack<V, N>*>(static_cast<const V*>(p) + at)));
    constexpr int Q = N < 4 ? N : 4;
    Floats<N> f;
#pragma unroll
    for (int i = 0; i < N / Q; ++i) {
        const Floats<Q> x = floats(load(reinterpret_cast<const Pack<float, Q>*>(static_cast<const float*>(p) + at) + i));
#pragma unroll
        for (int j = 0; j < (Q + 1) / 2; ++j) f.v[(Q + 1) / 2 * i + j] = x.v[j];
    }
    return f;
}

// Sum (or maximum, as unsigned numbers) over the G threads of a group, G a power of two; groups of several warps meet in
// `s` (a word a warp, on a 16-byte boundary) and the whole block has to call.
__device__ __forceinline__ float group_sum(float v, int G, float* s) {
    for (int d = (G < 32 ? G : 32) >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (G <= 32) return v;
    const int w = threadIdx.x >> 5, per = G >> 5, w0 = w & -per;
    if ((threadIdx.x & 31) == 0) s[w] = v;
    __syncthreads();
    if (per < 4) return per == 1 ? v : s[w0] + s[w0 + 1];
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < per; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(s + w0 + i);
        t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    return (t.x + t.y) + (t.z + t.w);
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
