// spx_route.cu -- routed experts: the tokens' slots sorted by expert, tokens
// gathered into that order, the experts' rows returned weighted, and the
// gradients of the return.
//
// The sort is a stable counting sort with E buckets.  Each warp owns a run of
// consecutive slots, whose ids its lanes hold in registers: the warp counts them
// per expert (match_any finds the lanes of one expert, one lane adds their
// number to the warp's own counters), which also gives every slot its rank in
// the run; the counters of all warps before it give the run's first places.
// Nothing is atomic but integer sums, so places do not depend on timing.  Up to
// 2048 slots are one CTA, up to 16384 a cluster of CTAs that read each other's
// counts in shared memory; more take a counting launch first.  (More slots a
// CTA take longer: their scattered writes to `slot` pass one SM.)  Bound by
// latency: 8 slots 2.1 us, 3711 5.4, 65536 7.6.
//
// Gather, return and gradient are bound by HBM: every row is one contiguous
// copy.  All three are driven by the token, not by the sorted place: a token's
// row (X, Y or dY) is then read or written exactly once and its k partners
// are whole rows at scattered places, which cost no more than ordered ones
// because a row is far longer than a DRAM burst.
#include <algorithm>

#include "spx_experts.cuh"

using namespace spx_exp;

namespace {

// ---------------------------------------------------------------- the sort

struct Ids {
    const void* p;
    long long lde;
    int k, bytes;
};

// Expert of flat slot i, -1 when it is none.
__device__ __forceinline__ int id_of(const Ids& x, int i, int E) {
    const long long at = x.lde == x.k ? i : static_cast<long long>(i / x.k) * x.lde + i % x.k;
    if (x.bytes == 4) {
        const int e = load(static_cast<const int*>(x.p) + at);
        return e >= 0 && e < E ? e : -1;
    }
    const long long e = load(static_cast<const long long*>(x.p) + at);
    return e >= 0 && e < E ? static_cast<int>(e) : -1;
}

constexpr int kHeld = 4;              // ids a lane holds
constexpr int kRun = 32 * kHeld;      // slots of a warp
constexpr int kMostWarps = 16, kMostCluster = 8, kMaxBlocks = 304;

// Ids of this warp's run, -1 past the end and for dropped slots; done[w][e] = slots of expert e in the run; rank[i] =
// those before this lane's i-th.  Slot i of a lane is w0 + 32 i + lane.
__device__ __forceinline__ void rank_run(const Ids& x, int E, int w0, int end, int (&id)[kHeld], int (&rank)[kHeld],
                                         int* done) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) id[i] = w0 + 32 * i + lane < end ? id_of(x, w0 + 32 * i + lane, E) : -1;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        if (w0 + 32 * i >= end) break;
        const unsigned same = __match_any_sync(0xffffffffu, id[i]);
        const unsigned before = same & ((1u << lane) - 1u);
        if (id[i] >= 0) rank[i] = done[id[i]] + __popc(before);
        __syncwarp();
        if (id[i] >= 0 && before == 0) done[id[i]] += __popc(same);
        __syncwarp();
    }
}

// The block's slots of each expert, for the sort of more slots than a cluster holds.
__global__ void __launch_bounds__(32 * kMostWarps)
    route_count_kernel(Ids x, int S, int E, int runs, int* hist) {
    extern __shared__ int sm[];
    let_next_start();
    wait_for_previous();
    x.p = behind_wait(x.p);
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm[e] = 0;
    __syncthreads();
    const int per = runs * blockDim.x * kHeld, b0 = blockIdx.x * per, b1 = min(S, b0 + per);
    for (int i = b0 + threadIdx.x; i < b1; i += blockDim.x) {
        const int e = id_of(x, i, E);
        if (e >= 0) atomicAdd(sm + e, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[blockIdx.x * E + e] = sm[e];
}

// A block places `runs` rounds of blockDim.x * kHeld consecutive slots.  The other blocks' counts come from `hist`
// (counted before, any number of blocks), or (hist NULL) from the other CTAs of the cluster that the grid is.
__global__ void __launch_bounds__(32 * kMostWarps)
    route_place_kernel(Ids x, int S, int E, int runs, const int* hist, int* offsets, int* slot, int* pos) {
    extern __shared__ int sm[];  // counters of each warp (ES apart), E + 1 totals, E places before this block, E counts of it
    const int nw = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31, nb = gridDim.x, b = blockIdx.x;
    const int ES = E | 1;  // odd: a column of the counters touches every bank
    int *tot = sm + nw * ES, *before = tot + E + 1, *own = before + E;
    let_next_start();
    for (int i = threadIdx.x; i < nw * ES + 3 * E + 1; i += blockDim.x) sm[i] = 0;
    wait_for_previous();
    x.p = behind_wait(x.p);
    hist = behind_wait(hist);
    __syncthreads();
    const int per = runs * blockDim.x * kHeld, b0 = b * per, b1 = min(S, b0 + per);
    int id[kHeld], rank[kHeld];
    // the warps' counters of a round become places within it; the round's counts go to `own`
    auto scan_warps = [&]() {
        __syncthreads();
        if (nw <= 4) {  // a thread an expert
            for (int e = threadIdx.x; e < E; e += blockDim.x) {
                int sum = 0;
                for (int v = 0; v < nw; ++v) {
                    const int n = sm[v * ES + e];
                    sm[v * ES + e] = sum;
                    sum += n;
                }
                own[e] = sum;
            }
            __syncthreads();
            return;
        }
        for (int e = w; e < E; e += nw) {  // a warp an expert
            const int n = lane < nw ? sm[lane * ES + e] : 0;
            int inc = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += up;
            }
            if (lane < nw) sm[lane * ES + e] = inc - n;
            if (lane == 31) own[e] = inc;
        }
        __syncthreads();
    };
    if (runs == 1) {
        rank_run(x, E, b0 + w * kRun, b1, id, rank, sm + w * ES);
        scan_warps();
    }
    if (hist) {  // all blocks' counts: thread i takes expert i % E of every (blockDim.x / E)-th block
        const int parts = max(1, static_cast<int>(blockDim.x) / E);
        for (int i = threadIdx.x; i < E * parts; i += blockDim.x) {
            const int e = i % E;
            int all = 0, lower = 0;
#pragma unroll 4
            for (int o = i / E; o < nb; o += parts) {
                const int n = load(hist + static_cast<long long>(o) * E + e);
                all += n;
                lower += o < b ? n : 0;
            }
            atomicAdd(tot + e, all);
            atomicAdd(before + e, lower);
        }
    } else {
        if (nb == 1) {
            for (int e = threadIdx.x; e < E; e += blockDim.x) tot[e] = own[e];
        } else {
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            for (int e = threadIdx.x; e < E; e += blockDim.x) {
                int all = 0, lower = 0;
                for (int o = 0; o < nb; ++o) {
                    uint32_t there;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                 : "=r"(there)
                                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(own + e))), "r"(o));
                    int n;
                    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(n) : "r"(there) : "memory");
                    all += n;
                    lower += o < b ? n : 0;
                }
                tot[e] = all;
                before[e] = lower;
            }
        }
    }
    __syncthreads();
    if (w == 0) {  // totals -> offsets
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int n = e0 + lane < E ? tot[e0 + lane] : 0;
            int inc = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += up;
            }
            if (e0 + lane < E) {
                before[e0 + lane] += carry + inc - n;
                if (b == 0) offsets[e0 + lane] = carry + inc - n;
            }
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            tot[E] = carry;
            if (b == 0) offsets[E] = carry;
        }
    }
    __syncthreads();
    for (int round = 0; round < runs; ++round) {
        const int w0 = b0 + (round * nw + w) * kRun;
        if (runs > 1) {
            for (int i = threadIdx.x; i < nw * ES; i += blockDim.x) sm[i] = 0;
            __syncthreads();
            rank_run(x, E, w0, b1, id, rank, sm + w * ES);
            scan_warps();
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int at = w0 + 32 * i + lane;
            if (at >= b1) break;
            const int p = id[i] >= 0 ? before[id[i]] + sm[w * ES + id[i]] + rank[i] : -1;
            pos[at] = p;
            if (p >= 0) slot[p] = at;
        }
        if (runs > 1) {
            __syncthreads();
            for (int e = threadIdx.x; e < E; e += blockDim.x) before[e] += own[e];
        }
    }
    for (int p = tot[E] + b * blockDim.x + threadIdx.x; p < S; p += nb * blockDim.x) slot[p] = -1;
    if (!hist && nb > 1)  // nobody leaves while its counts may be read
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Warps a CTA, CTAs and rounds for S slots: the warps' counters fit 48 KB.
struct SortShape {
    int warps, blocks, runs;
    bool counted;  // a counting launch comes first
    size_t smem;
};
SortShape sort_shape(long long S, int E) {
    SortShape r{};
    r.warps = 1;
    while (r.warps < kMostWarps && static_cast<long long>(r.warps) * kRun < S && (2 * r.warps + 3) * (E + 2) * 4 <= 48 * 1024)
        r.warps *= 2;
    const long long one = static_cast<long long>(r.warps) * kRun;
    const long long blocks = std::max(1LL, (S + one - 1) / one);
    r.counted = blocks > kMostCluster;
    r.runs = r.counted ? static_cast<int>((blocks + kMaxBlocks - 1) / kMaxBlocks) : 1;
    r.blocks = static_cast<int>((blocks + r.runs - 1) / r.runs);
    if (!r.counted)
        while (r.blocks & (r.blocks - 1)) ++r.blocks;  // a cluster of 1, 2, 4 or 8
    r.smem = sizeof(int) * (static_cast<size_t>(r.warps) * (E | 1) + 3 * static_cast<size_t>(E) + 1);
    return r;
}

// ---------------------------------------------------------------- rows in pieces of VB bytes

// The values of one piece as floats, and back (rounded once each).
template <class V, class P>
__device__ __forceinline__ void widen(const P& p, float (&f)[sizeof(P) / sizeof(V)]) {
    V v[sizeof(P) / sizeof(V)];
    memcpy(v, &p, sizeof(P));
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(P) / sizeof(V)); ++i) f[i] = to_f(v[i]);
}
template <class V, class P>
__device__ __forceinline__ P narrow(const float (&f)[sizeof(P) / sizeof(V)]) {
    V v[sizeof(P) / sizeof(V)];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(P) / sizeof(V)); ++i) v[i] = from_f<V>(f[i]);
    P p;
    memcpy(&p, v, sizeof(P));
    return p;
}

constexpr int kRowThreads = 256;

// A group of G threads (G divides 256) works on one token; grid.y splits the
// row among groups when there are few tokens.  Pieces are values in the gather.
struct RowShape {
    int T, k, np, G;           // tokens, slots a token, pieces a row, threads a group
    long long a, b;            // row pitch in pieces of the token-ordered and of the sorted array
};

__device__ __forceinline__ int place(const int* pos, long long i, int S) {
    const int p = load(pos + i);
    if (SPX_CHECKED && (p < -1 || p >= S)) check_fail();
    return p >= 0 && p < S ? p : -1;
}

// The first sorted row past the last expert's, offsets[E].
__device__ __forceinline__ int rows_end(const int* end, int S) {
    const int p = load(end);
    if (SPX_CHECKED && !(0 <= p && p <= S)) check_fail();
    return min(max(p, 0), S);
}

// Zeros in the sorted array's rows from offsets[E] on: token t's group takes every T-th of them.
template <class P>
__device__ __forceinline__ void zero_tail(const RowShape& r, const int* end, int t, int v0, int dv, P* out) {
    const int S = r.T * r.k;
    for (long long p = rows_end(end, S) + static_cast<long long>(t); p < S; p += r.T)
        for (int v = v0; v < r.np; v += dv) memset(out + p * r.b + v, 0, sizeof(P));
}

// The 16 bytes at p (aligned to the element) out of the two aligned pieces
// around them, or value by value where those would leave the array [lo, hi).
template <class V>
__device__ __forceinline__ uint4 read16(const char* p, const char* lo, const char* hi) {
    const int m = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    const char* at = p - m;
    if (m == 0) return load(reinterpret_cast<const uint4*>(p));
    if (at < lo || at + 32 > hi) {
        V v[16 / sizeof(V)];
#pragma unroll
        for (int i = 0; i < static_cast<int>(16 / sizeof(V)); ++i) v[i] = load(reinterpret_cast<const V*>(p) + i);
        uint4 w;
        memcpy(&w, v, 16);
        return w;
    }
    const uint4 x = load(reinterpret_cast<const uint4*>(at)), y = load(reinterpret_cast<const uint4*>(at) + 1);
    const bool two = m & 8, one = m & 4;
    const uint32_t t0 = two ? x.z : x.x, t1 = two ? x.w : x.y, t2 = two ? y.x : x.z, t3 = two ? y.y : x.w,
                   t4 = two ? y.z : y.x, t5 = two ? y.w : y.y;
    const uint32_t u0 = one ? t1 : t0, u1 = one ? t2 : t1, u2 = one ? t3 : t2, u3 = one ? t4 : t3, u4 = one ? t5 : t4;
    const int sh = (m & 3) * 8;
    return make_uint4(__funnelshift_r(u0, u1, sh), __funnelshift_r(u1, u2, sh), __funnelshift_r(u2, u3, sh),
                      __funnelshift_r(u3, u4, sh));
}

// V: the copied values' type, or any of their size.  VB: rows on boundaries of
// 16 or 8 bytes move in pieces of that; 0: each written row is cut at its own
// 16-byte boundaries -- a head of single values, aligned pieces, a tail -- so
// that wide stores fill whole sectors, and the token's row, which L1 holds, is
// read around them.  12001 tokens x 8 fp32: rows of 4095 285 us so, 438 with
// 4-byte stores where they fall; of 4094 286 so and 344 in 8-byte pieces; of 130
// 20 and 12: rows on 8-byte boundaries are cut from kCutRow bytes on.
constexpr long long kCutRow = 8192;

template <class V, int VB>
__global__ void __launch_bounds__(kRowThreads)
    route_gather_kernel(RowShape r, const int* pos, const int* end, const V* X, V* Xs) {
    let_next_start();
    wait_for_previous();
    pos = behind_wait(pos), end = behind_wait(end), X = behind_wait(X);
    const int t = blockIdx.x * (kRowThreads / r.G) + threadIdx.x / r.G;
    if (t >= r.T) return;
    const int S = r.T * r.k, v0 = blockIdx.y * r.G + threadIdx.x % r.G, dv = gridDim.y * r.G;
    const long long i0 = static_cast<long long>(t) * r.k;
    const V* x = X + t * r.a;
    if constexpr (VB > 0) {
        using P = typename Word<VB>::T;
        for (int v = v0; v < r.np / static_cast<int>(VB / sizeof(V)); v += dv) {
            const P piece = load(reinterpret_cast<const P*>(x) + v);
            for (int j = 0; j < r.k; ++j) {
                const int p = place(pos, i0 + j, S);
                if (p >= 0) __stcs(reinterpret_cast<P*>(Xs + p * r.b) + v, piece);
            }
        }
    } else {
        constexpr int N = 16 / sizeof(V);
        const char *lo = reinterpret_cast<const char*>(X), *hi = reinterpret_cast<const char*>(X + (r.T - 1) * r.a + r.np);
        for (int j = 0; j < r.k; ++j) {
            const int p = place(pos, i0 + j, S);
            if (p < 0) continue;
            V* q = Xs + p * r.b;
            const int head = min(r.np, static_cast<int>((-reinterpret_cast<intptr_t>(q) & 15) / sizeof(V)));
            const int pieces = (r.np - head) / N, rest = r.np - head - pieces * N;
            for (int v = v0; v < pieces; v += dv)
                __stcs(reinterpret_cast<uint4*>(q + head) + v, read16<V>(reinterpret_cast<const char*>(x + head) + 16LL * v, lo, hi));
            for (int i = v0; i < head + rest; i += dv) {
                const int at = i < head ? i : i + pieces * N;
                q[at] = load(x + at);
            }
        }
    }
    zero_tail(r, end, t, v0, dv, Xs);
}

constexpr int kSlotsAtOnce = 4;  // rows of one token in flight in a thread

// VB: the widest piece, of 16 bytes down to a value, that all rows are aligned
// to (12001 tokens x 8 x 4094 fp32: 278 us in 8-byte pieces, 385 in 4-byte ones;
// pieces put together from aligned neighbours, as the gather does, took 440).
// Narrow pieces are bound by the loads' number: 12001 tokens x 8 bf16, rows of 4096
// 133 us, of 4094 (4-byte pieces) 222, of 4095 (2-byte pieces) 393; the gradient 269,
// 350 and 465.
template <class V, int VB>
__global__ void __launch_bounds__(kRowThreads)
    route_combine_kernel(RowShape r, const int* pos, const float* weight, const typename Word<VB>::T* Ys,
                         typename Word<VB>::T* Y) {
    using P = typename Word<VB>::T;
    constexpr int N = VB / sizeof(V);
    let_next_start();
    wait_for_previous();
    pos = behind_wait(pos), weight = behind_wait(weight), Ys = behind_wait(Ys);
    const int t = blockIdx.x * (kRowThreads / r.G) + threadIdx.x / r.G;
    if (t >= r.T) return;
    const int S = r.T * r.k, v0 = blockIdx.y * r.G + threadIdx.x % r.G, dv = gridDim.y * r.G;
    const long long i0 = static_cast<long long>(t) * r.k;
    for (int v = v0; v < r.np; v += dv) {
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        for (int j0 = 0; j0 < r.k; j0 += kSlotsAtOnce) {
            P piece[kSlotsAtOnce];
            float w[kSlotsAtOnce];
            bool on[kSlotsAtOnce];
#pragma unroll
            for (int u = 0; u < kSlotsAtOnce; ++u) {
                const int p = j0 + u < r.k ? place(pos, i0 + j0 + u, S) : -1;
                on[u] = p >= 0;
                if (on[u]) {
                    piece[u] = load_once(Ys + p * r.b + v);
                    w[u] = weight ? load(weight + i0 + j0 + u) : 1.f;
                }
            }
#pragma unroll
            for (int u = 0; u < kSlotsAtOnce; ++u) {
                if (!on[u]) continue;
                float f[N];
                widen<V, P>(piece[u], f);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = fmaf(w[u], f[i], acc[i]);
            }
        }
        Y[t * r.a + v] = narrow<V, P>(acc);
    }
}

// dweight: a thread's products in pieces order, then a fixed tree over the
// group's lanes and warps.  Pitches in bytes.
template <class V, int VB>
__global__ void __launch_bounds__(kRowThreads)
    route_combine_grad_kernel(RowShape r, const int* pos, const int* end, const float* weight, const char* dY,
                              long long ldys, const char* Ys, char* dYs, float* dw) {
    using P = typename Word<VB>::T;
    constexpr int N = VB / sizeof(V);
    __shared__ float part[kRowThreads / 32][kSlotsAtOnce];
    let_next_start();
    wait_for_previous();
    pos = behind_wait(pos), end = behind_wait(end), weight = behind_wait(weight), dY = behind_wait(dY), Ys = behind_wait(Ys);
    const int t = blockIdx.x * (kRowThreads / r.G) + threadIdx.x / r.G;
    const bool live = t < r.T;
    const int S = r.T * r.k, v0 = threadIdx.x % r.G;
    const long long i0 = static_cast<long long>(t) * r.k;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const char* g = dY + t * r.a;
    for (int j0 = 0; j0 < r.k; j0 += kSlotsAtOnce) {
        float dot[kSlotsAtOnce], w[kSlotsAtOnce];
        int at[kSlotsAtOnce];
#pragma unroll
        for (int u = 0; u < kSlotsAtOnce; ++u) {
            dot[u] = 0.f;
            at[u] = live && j0 + u < r.k ? place(pos, i0 + j0 + u, S) : -1;
            w[u] = at[u] >= 0 && weight ? load(weight + i0 + j0 + u) : 1.f;
        }
        if (live) {
#pragma unroll 1  // 12001 tokens x 8 x 4095 fp32 679 us, 720 unrolled
            for (int v = v0; v < r.np; v += r.G) {
                const P gp = load(reinterpret_cast<const P*>(g) + v);
                P y[kSlotsAtOnce];
                if (dw) {
#pragma unroll
                    for (int u = 0; u < kSlotsAtOnce; ++u)
                        if (at[u] >= 0) y[u] = load_once(reinterpret_cast<const P*>(Ys + at[u] * ldys) + v);
                }
                float gf[N];
                widen<V, P>(gp, gf);
#pragma unroll
                for (int u = 0; u < kSlotsAtOnce; ++u) {
                    if (at[u] < 0) continue;
                    float f[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) f[i] = w[u] * gf[i];
                    __stcs(reinterpret_cast<P*>(dYs + at[u] * r.b) + v, narrow<V, P>(f));
                    if (dw) {
                        widen<V, P>(y[u], f);
#pragma unroll
                        for (int i = 0; i < N; ++i) dot[u] = fmaf(gf[i], f[i], dot[u]);
                    }
                }
            }
        }
        if (dw) {
#pragma unroll
            for (int u = 0; u < kSlotsAtOnce; ++u)
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], d);
            if (r.G > 32) {
                if (lane == 0)
#pragma unroll
                    for (int u = 0; u < kSlotsAtOnce; ++u) part[warp][u] = dot[u];
                __syncthreads();
            }
            if (live && v0 < kSlotsAtOnce && j0 + v0 < r.k) {
                float s = 0.f;
                if (r.G > 32) {
                    for (int x = 0; x < r.G / 32; ++x) s += part[warp + x][v0];
                } else {
#pragma unroll
                    for (int u = 0; u < kSlotsAtOnce; ++u)
                        if (u == v0) s = dot[u];
                }
                dw[i0 + j0 + v0] = place(pos, i0 + j0 + v0, S) >= 0 ? s : 0.f;
            }
            if (r.G > 32) __syncthreads();
        }
    }
    if (live) {
        for (long long p = rows_end(end, S) + static_cast<long long>(t); p < S; p += r.T)
            for (int v = v0; v < r.np; v += r.G) memset(dYs + p * r.b + v * static_cast<long long>(VB), 0, VB);
    }
}

// ---------------------------------------------------------------- host side

// Threads a group: enough that a row of `steps` pieces is one step, no more
// than a CTA; a warp at least (the weights' gradient reduces over warps).  The
// gradient's groups of several warps meet at a barrier for every four slots, so
// it takes one warp a token (`warps`: rows of wide pieces, or short ones) where
// the tokens fill the SMs: 12001 tokens x 8 x 130 fp32 18 us, 65 with a CTA
// each; 3001 x 3 x 1002 fp32, in 8-byte pieces, 24 and 19.
constexpr int kWarpTokens = 152 * 16;

RowShape row_shape(int T, int k, int64_t np, int64_t steps, bool warps) {
    RowShape r{};
    r.T = T;
    r.k = k;
    r.np = static_cast<int>(np);
    r.G = 32;
    while (r.G < kRowThreads && r.G < steps && !(warps && T >= kWarpTokens)) r.G <<= 1;
    return r;
}

dim3 row_grid(const RowShape& r, int64_t pieces, bool split) {
    const int bx = (r.T + kRowThreads / r.G - 1) / (kRowThreads / r.G);
    // few tokens: their rows are cut so that a thread has one piece
    const int steps = static_cast<int>((pieces + r.G - 1) / r.G);
    const int by = split && bx < 608 ? std::min(steps, 608 / bx + 1) : 1;
    return dim3(bx, by);
}

spx_status check_rows(int32_t T, int32_t k, int32_t H) {
    if (T < 0 || k <= 0 || H < 0) return SPX_ERR_ARG;
    if (static_cast<int64_t>(T) * k > kMostIndex || H > kMostIndex) return SPX_ERR_INDEX_RANGE;
    return SPX_OK;
}

template <class V>
int piece_bytes(uint64_t bits) {
    return copy_width(bits, static_cast<int>(sizeof(V)));
}

template <class V, int VB>
cudaError_t combine_launch(RowShape r, const int32_t* pos, const float* weight, const void* Ys, void* Y, cudaStream_t st) {
    using P = typename Word<VB>::T;
    return launch_early(route_combine_kernel<V, VB>, row_grid(r, r.np, true), kRowThreads, 0, 1, st, r, pos, weight,
                        static_cast<const P*>(Ys), static_cast<P*>(Y));
}

template <class V>
spx_status combine(int T, int k, int H, const int32_t* pos, const float* weight, const void* Ys, int64_t ldys, void* Y,
                   int64_t ldy, cudaStream_t st) {
    const uint64_t row = static_cast<uint64_t>(H) * sizeof(V), a = ldy * sizeof(V), b = ldys * sizeof(V);
    const int vb = piece_bytes<V>(addr(Ys) | addr(Y) | row | a | b);
    RowShape r = row_shape(T, k, static_cast<int64_t>(row / vb), static_cast<int64_t>(row / vb), false);
    r.a = static_cast<long long>(a / vb);
    r.b = static_cast<long long>(b / vb);
    spx_note_launches(1);
    return spx_cuda_status(vb == 16  ? combine_launch<V, 16>(r, pos, weight, Ys, Y, st)
                           : vb == 8 ? combine_launch<V, 8>(r, pos, weight, Ys, Y, st)
                           : vb == 4 ? combine_launch<V, 4>(r, pos, weight, Ys, Y, st)
                                     : combine_launch<V, sizeof(V)>(r, pos, weight, Ys, Y, st));
}

template <class V>
spx_status combine_grad(int T, int k, int H, const int32_t* pos, const int32_t* end, const float* weight,
                        const void* dY, int64_t lddy, const void* Ys, int64_t ldys, void* dYs, int64_t lddys,
                        float* dw, cudaStream_t st) {
    const uint64_t row = static_cast<uint64_t>(H) * sizeof(V), a = lddy * sizeof(V), b = lddys * sizeof(V);
    const uint64_t y = dw ? ldys * sizeof(V) : 0;
    const int vb = piece_bytes<V>(addr(dY) | addr(dYs) | (dw ? addr(Ys) : 0) | row | a | b | y);
    const int64_t np = static_cast<int64_t>(row / vb);
    RowShape r = row_shape(T, k, np, np, vb == 16 || row <= 2048);
    r.a = static_cast<long long>(a);
    r.b = static_cast<long long>(b);
    const long long ly = static_cast<long long>(y);
    const dim3 grid = row_grid(r, np, false);
    const char *dy = static_cast<const char*>(dY), *ys = static_cast<const char*>(Ys);
    char* out = static_cast<char*>(dYs);
    spx_note_launches(1);
    auto launch = [&](auto kernel) { return launch_early(kernel, grid, kRowThreads, 0, 1, st, r, pos, end, weight, dy, ly, ys, out, dw); };
    return spx_cuda_status(vb == 16  ? launch(route_combine_grad_kernel<V, 16>)
                           : vb == 8 ? launch(route_combine_grad_kernel<V, 8>)
                           : vb == 4 ? launch(route_combine_grad_kernel<V, 4>)
                                     : launch(route_combine_grad_kernel<V, sizeof(V)>));
}

template <class V>
spx_status gather(int T, int k, int H, const int32_t* pos, const int32_t* end, const void* X, int64_t ldx, void* Xs,
                  int64_t ldxs, cudaStream_t st) {
    const uint64_t bits = addr(X) | addr(Xs) | (static_cast<uint64_t>(H) | ldx | ldxs) * sizeof(V);
    const int vb = bits % 16 == 0 ? 16 : bits % 8 == 0 && H * static_cast<long long>(sizeof(V)) < kCutRow ? 8 : 0;
    const int64_t per = (vb ? vb : 16) / sizeof(V), pieces = (H + per - 1) / per;
    RowShape r = row_shape(T, k, H, pieces, false);
    r.a = ldx;
    r.b = ldxs;
    const V* x = static_cast<const V*>(X);
    V* xs = static_cast<V*>(Xs);
    spx_note_launches(1);
    return spx_cuda_status(launch_early(vb == 16  ? route_gather_kernel<V, 16>
                                        : vb == 8 ? route_gather_kernel<V, 8>
                                                  : route_gather_kernel<V, 0>,
                                        row_grid(r, pieces, true), kRowThreads, 0, 1, st, r, pos, end, x, xs));
}

}  // namespace

int spx_route_check_take() { return spx_check_take(g_experts_check); }

extern "C" {

size_t spx_route_scratch_bytes(int32_t T, int32_t k, int32_t E) {
    if (T < 0 || k <= 0 || E <= 0) return 0;
    const SortShape h = sort_shape(static_cast<int64_t>(T) * k, E);
    return h.counted ? sizeof(int32_t) * static_cast<size_t>(h.blocks) * static_cast<size_t>(E) : 0;
}

spx_status spx_route_build(int32_t T, int32_t k, int32_t E, const void* expert, int32_t id_bytes, int64_t lde,
                           int32_t* offsets, int32_t* slot, int32_t* pos, void* scratch, size_t scratch_bytes,
                           spx_stream_t stream) {
    if (T < 0 || k <= 0 || E <= 0 || (id_bytes != 4 && id_bytes != 8)) return SPX_ERR_ARG;
    if (E > SPX_MAX_EXPERTS) return SPX_ERR_UNSUPPORTED;
    const int64_t S64 = static_cast<int64_t>(T) * k;
    if (S64 > kMostIndex) return SPX_ERR_INDEX_RANGE;
    if (!offsets || (S64 > 0 && (!expert || !slot || !pos || lde < k))) return SPX_ERR_ARG;
    if (!spx_aligned(offsets, 4) || !spx_aligned(slot, 4) || !spx_aligned(pos, 4) ||
        !spx_aligned(expert, static_cast<size_t>(id_bytes)))
        return SPX_ERR_ALIGN;
    const int S = static_cast<int>(S64);
    const SortShape h = sort_shape(S64, E);
    const size_t need = spx_route_scratch_bytes(T, k, E);
    if (need > 0 && (!scratch || scratch_bytes < need)) return SPX_ERR_ARG;
    if (need > 0 && !spx_aligned(scratch, 4)) return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const Ids ids{expert, lde, k, id_bytes};
    int* hist = h.counted ? static_cast<int*>(scratch) : nullptr;
    spx_note_launches(h.counted ? 2 : 1);
    cudaError_t e = cudaSuccess;
    if (h.counted)
        e = launch_early(route_count_kernel, dim3(h.blocks), 32 * h.warps, sizeof(int) * E, 1, st, ids, S, E, h.runs, hist);
    if (e == cudaSuccess)
        e = launch_early(route_place_kernel, dim3(h.blocks), 32 * h.warps, h.smem, h.counted ? 1 : h.blocks, st, ids, S, E,
                         h.runs, hist, offsets, slot, pos);
    return spx_cuda_status(e);
}

spx_status spx_route_gather(int32_t T, int32_t k, int32_t H, spx_type type, const int32_t* pos,
                            const int32_t* offsets_end, const void* X, int64_t ldx, void* Xs, int64_t ldxs,
                            spx_stream_t stream) {
    const spx_status c = check_rows(T, k, H);
    if (c != SPX_OK) return c;
    if (!is_float_type(type) && type != SPX_I8) return SPX_ERR_ARG;
    if (T == 0 || H == 0) return SPX_OK;
    if (!pos || !offsets_end || !X || !Xs || ldx < H || ldxs < H) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type);
    if (!spx_aligned(pos, 4) || !spx_aligned(offsets_end, 4) || !spx_aligned(X, eb) || !spx_aligned(Xs, eb))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (eb == 4) return gather<uint32_t>(T, k, H, pos, offsets_end, X, ldx, Xs, ldxs, st);
    if (eb == 2) return gather<uint16_t>(T, k, H, pos, offsets_end, X, ldx, Xs, ldxs, st);
    return gather<uint8_t>(T, k, H, pos, offsets_end, X, ldx, Xs, ldxs, st);
}

spx_status spx_route_combine(int32_t T, int32_t k, int32_t H, spx_type type, const int32_t* pos, const float* weight,
                             const void* Ys, int64_t ldys, void* Y, int64_t ldy, spx_stream_t stream) {
    const spx_status c = check_rows(T, k, H);
    if (c != SPX_OK) return c;
    if (!is_float_type(type)) return SPX_ERR_ARG;
    if (T == 0 || H == 0) return SPX_OK;
    if (!pos || !Ys || !Y || ldys < H || ldy < H) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type);
    if (!spx_aligned(pos, 4) || !spx_aligned(weight, 4) || !spx_aligned(Ys, eb) || !spx_aligned(Y, eb))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (type == SPX_F32) return combine<float>(T, k, H, pos, weight, Ys, ldys, Y, ldy, st);
    if (type == SPX_BF16) return combine<__nv_bfloat16>(T, k, H, pos, weight, Ys, ldys, Y, ldy, st);
    return combine<__half>(T, k, H, pos, weight, Ys, ldys, Y, ldy, st);
}

spx_status spx_route_combine_grad(int32_t T, int32_t k, int32_t H, spx_type type, const int32_t* pos,
                                  const int32_t* offsets_end, const float* weight, const void* dY, int64_t lddy,
                                  const void* Ys, int64_t ldys, void* dYs, int64_t lddys, float* dweight,
                                  spx_stream_t stream) {
    const spx_status c = check_rows(T, k, H);
    if (c != SPX_OK) return c;
    if (!is_float_type(type)) return SPX_ERR_ARG;
    if (T == 0) return SPX_OK;
    if (!pos || !offsets_end) return SPX_ERR_ARG;
    if (H > 0 && (!dY || !dYs || lddy < H || lddys < H || (dweight && (!Ys || ldys < H)))) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type);
    if (!spx_aligned(pos, 4) || !spx_aligned(offsets_end, 4) || !spx_aligned(weight, 4) || !spx_aligned(dweight, 4) ||
        !spx_aligned(dY, eb) || !spx_aligned(dYs, eb) || (dweight && !spx_aligned(Ys, eb)))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (type == SPX_F32)
        return combine_grad<float>(T, k, H, pos, offsets_end, weight, dY, lddy, Ys, ldys, dYs, lddys, dweight, st);
    if (type == SPX_BF16)
        return combine_grad<__nv_bfloat16>(T, k, H, pos, offsets_end, weight, dY, lddy, Ys, ldys, dYs, lddys, dweight,
                                           st);
    return combine_grad<__half>(T, k, H, pos, offsets_end, weight, dY, lddy, Ys, ldys, dYs, lddys, dweight, st);
}

}  // extern "C"
