// spx_rows.cuh -- rows in pieces that a thread moves as one word: what the norm
// and the embedding kernels share.
#pragma once

#include "spx_experts.cuh"

namespace spx_rows {

using namespace spx_exp;

// N values of V, N * sizeof(V) a power of two up to 16, held as one word: as an array of values the compiler copies,
// loads and stores it value by value.
template <class V, int N>
struct Pack {
    typename Word<N * sizeof(V)>::T w;
    __device__ __forceinline__ void get(V (&v)[N]) const { memcpy(v, &w, sizeof(w)); }
    __device__ __forceinline__ void set(const V (&v)[N]) { memcpy(&w, v, sizeof(w)); }
};

template <class P>
__device__ __forceinline__ P read_piece(const P* p) {
    P v;
    v.w = *reinterpret_cast<const decltype(v.w)*>(p);
    return v;
}
template <class P>
__device__ __forceinline__ void write_piece(P* p, const P& v) {
    *reinterpret_cast<decltype(P::w)*>(p) = v.w;
}
// A piece of 4, 8 or 16 bytes to shared memory, asynchronously.
template <class P>
__device__ __forceinline__ void copy_piece(P* to, const P* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (sizeof(P) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(sizeof(P) < 4 ? 4 : sizeof(P)) : "memory");
}

// The same of 16 bytes that a neighbour copies too: through L1.
template <class P>
__device__ __forceinline__ void copy_near(P* to, const P* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
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
        V v[1];
        p.get(v);
        f.v[0] = make_float2(to_f(v[0]), 0.f);
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
        const V v[1] = {from_f<V>(f.v[0].x)};
        p.set(v);
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

// ---------------- pieces off their boundaries
//
// Rows of any width and base still move in whole aligned words: a piece is put together from the two words around it,
// which its neighbours read too, and a word that is written from a thread's piece and its left neighbour's.

// Bytes off to off + 4 W of the 8 W in t.
template <int W>
__device__ __forceinline__ void shift_words(const uint32_t (&t)[2 * W], int off, uint32_t (&o)[W]) {
    uint32_t u[W + 1];
    if constexpr (W == 4) {
        const bool two = off & 8, one = off & 4;
        uint32_t v[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = two ? t[i + 2] : t[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = one ? v[i + 1] : v[i];
    } else {
        static_assert(W == 2, "pieces of 8 and 16 bytes");
        const bool one = off & 4;
#pragma unroll
        for (int i = 0; i < 3; ++i) u[i] = one ? t[i + 1] : t[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = __funnelshift_r(u[i], u[i + 1], (off & 3) * 8);
}

// The n values at p (0 to N, the others are zeros), from an array in [lo, hi).
template <class V, int N>
__device__ __forceinline__ Pack<V, N> read_any(const V* p, int n, const void* lo, const void* hi) {
    using P = Pack<V, N>;
    constexpr int W = sizeof(P) / 4;
    const int m = static_cast<int>(reinterpret_cast<uintptr_t>(p) & (sizeof(P) - 1));
    const char* at = reinterpret_cast<const char*>(p) - m;
    P r;
    if (n == N && m == 0) return load(reinterpret_cast<const P*>(p));
    if (n == N && at >= static_cast<const char*>(lo) && at + 2 * sizeof(P) <= static_cast<const char*>(hi)) {
        const P x = load(reinterpret_cast<const P*>(at)), y = load(reinterpret_cast<const P*>(at) + 1);
        uint32_t t[2 * W], o[W];
        memcpy(t, &x, sizeof(P));
        memcpy(t + W, &y, sizeof(P));
        shift_words<W>(t, m, o);
        memcpy(&r, o, sizeof(P));
        return r;
    }
    V v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        memset(&v[i], 0, sizeof(V));
        if (i < n) v[i] = load(p + i);
    }
    r.set(v);
    return r;
}

// Writes the first n values of v to p.  A whole warp calls; `left`: the lane before holds the whole piece before this one.
template <class V, int N>
__device__ __forceinline__ void write_any(V* p, int n, const Pack<V, N>& v, bool left) {
    using P = Pack<V, N>;
    constexpr int W = sizeof(P) / 4, B = sizeof(P);
    const int m = static_cast<int>(reinterpret_cast<uintptr_t>(p) & (B - 1));
    uint32_t t[2 * W], o[W];
    memcpy(t + W, &v, B);
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = __shfl_up_sync(0xffffffffu, t[W + i], 1);
    const bool wide = n == N && (m == 0 || left);
    const bool covered = __shfl_down_sync(0xffffffffu, wide && m != 0, 1) && (threadIdx.x & 31) != 31;  // the next lane writes this one's end
    int from = 0, to = n;  // values left to write one by one
    if (wide) {
        shift_words<W>(t, m == 0 ? 0 : B - m, o);
        P c;
        memcpy(&c, m == 0 ? t + W : o, B);
        write_piece(reinterpret_cast<P*>(reinterpret_cast<char*>(p) - m), c);
        from = m == 0 ? N : (B - m) / static_cast<int>(sizeof(V));
    }
    if (covered && n == N && m != 0) to = (B - m) / static_cast<int>(sizeof(V));
    if (from < to) {
        V e[N];
        v.get(e);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= from && i < to) p[i] = e[i];
    }
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

// Rows in pieces of N values: all on boundaries of a piece and of whole pieces, or (ANY) of any base, pitch and width.
template <class V, int N, bool ANY>
struct Rows {
    static_assert(!ANY || N * sizeof(V) == 16, "shifted pieces are of 16 bytes");
    using Piece = Pack<V, N>;
    int H;
    __device__ __forceinline__ int pieces() const { return ANY ? (H + N - 1) / N : H / N; }
    __device__ __forceinline__ int values(int p) const { return max(0, min(N, H - p * N)); }
    // ANY: whether both words around each of the row's pieces lie in the array [base, end), as they do for all but its
    // first and last rows.  No branch then stands between the loads of a row's pieces, which would keep them from being in
    // flight together (16384 x 4095 bf16, norm: 170 us with one, 161 without).
    __device__ __forceinline__ bool inside(const V* row, const V* base, const V* end) const {
        const auto down = [](const V* p) { return reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15); };
        return !ANY || (down(row) >= reinterpret_cast<uintptr_t>(base) && down(row + (pieces() - 1) * N) + 32 <= reinterpret_cast<uintptr_t>(end));
    }
    // The piece out of its two words; values past the row's end are zeros.
    __device__ __forceinline__ Piece join(const Piece& x, const Piece& y, int m, int p) const {
        uint32_t t[8], o[4];
        memcpy(t, &x, 16);
        memcpy(t + 4, &y, 16);
        shift_words<4>(t, m, o);
        Piece r;
        const int n = values(p);
        if (n < N) {  // one lane of a row
            if constexpr (sizeof(V) == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = 2 * i + 1 < n ? o[i] : 2 * i < n ? o[i] & 0xffffu : 0u;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = i < n ? o[i] : 0u;
            }
        }
        memcpy(&r, o, 16);
        return r;
    }
    // Piece p, or the last one beyond it, of a row that is inside(); KEEP: it is read again soon.
    template <bool KEEP = false>
    __device__ __forceinline__ Piece read(const V* row, int p) const {
        p = min(p, pieces() - 1);
        if constexpr (!ANY) {
            const Piece* q = reinterpret_cast<const Piece*>(row) + p;
            return KEEP ? load(q) : load_once(q);
        } else {
            const int m = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
            const Piece* q = reinterpret_cast<const Piece*>(reinterpret_cast<const char*>(row) - m) + p;
            const Piece x = load(q), y = load(q + 1);
            return join(x, y, m, p);
        }
    }
    // The same of a row that is not inside().
    __device__ __forceinline__ Piece read_edge(const V* row, int p) const {
        Piece r;
        V v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            memset(&v[i], 0, sizeof(V));
            if (i < values(p)) v[i] = load(row + p * N + i);
        }
        r.set(v);
        return r;
    }
    __device__ __forceinline__ Floats<N> weights(const void* w, bool wide, int p) const {
        if constexpr (!ANY) {
            return load_floats<V, N>(w, wide, static_cast<long long>(p) * N);
        } else {
            if (!wide) {
                const V* v = static_cast<const V*>(w);
                return floats(read_any<V, N>(v + p * N, values(p), v, v + H));
            }
            const float* v = static_cast<const float*>(w);
            Floats<N> f;
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const Floats<4> x = floats(read_any<float, 4>(v + p * N + 4 * i, max(0, min(4, H - p * N - 4 * i)), v, v + H));
                f.v[2 * i] = x.v[0], f.v[2 * i + 1] = x.v[1];
            }
            return f;
        }
    }
    // A whole warp calls, also for pieces that are not there; `left`: the lane before holds the piece before.
    template <class O>
    __device__ __forceinline__ void write(O* row, int p, const Pack<O, N>& v, bool on, bool left) const {
        if constexpr (ANY) write_any<O, N>(row + p * N, on ? values(p) : 0, v, left);
        else if (on && p < pieces()) write_piece(reinterpret_cast<Pack<O, N>*>(row) + p, v);
    }
};

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
