// spx_int8.cu -- rows quantised to 8 bits and the product of 8-bit integers
// with a scale for each row and output channel.
//
// This chip has no fast 8-bit integer matrix rate, but fp16 holds every code
// exactly and the fp16 tensor cores sum their products exactly in fp32 up to
// 2^24, so the product runs on the experts' tensor-core kernel with codes
// widened to fp16, and its integer sums stay exact (see kExact there): widened
// by a pass of their own where there are rows enough to pay for it, on their
// way through shared memory where the weights' bytes count.  A few rows
// (decoded tokens) stream the weights straight into matrix fragments.
#include <algorithm>
#include <type_traits>

#include "spx_experts.cuh"

using namespace spx_exp;

namespace {

// ---------------------------------------------------------------- quantisation

// A row's largest magnitude, then its codes.  Bound by HBM.  A group of G
// threads takes a row: a warp where there are rows enough to fill the SMs and
// they are short (16384 rows x 2048 bf16: 21 us, 24 with a CTA a row; x 4096 53
// and 37), a CTA otherwise.  Up to kQHeld pieces a thread stay in registers
// between the two, a longer row is read again from L2: more of them held cost
// more in resident warps (eight: 38 us) than the reads.  Rows that are not on
// 16-byte boundaries go value by value (16384 x 2047 bf16: 47 us).
constexpr int kQThreads = 128, kQHeld = 4;
constexpr int kQWarpRows = 1216;  // rows that fill the SMs with a warp each: eight an SM

template <class V, int N>
struct alignas(N * sizeof(V) >= 16 ? 16 : N * sizeof(V)) Pack {
    V v[N];
};

// A piece is written as one word of its size.
template <class P>
__device__ __forceinline__ void write_piece(P* p, const P& v) {
    using T = typename Word<sizeof(P)>::T;
    T w;
    memcpy(&w, &v, sizeof(P));
    *reinterpret_cast<T*>(p) = w;
}

// The largest magnitude seen, as fp32 bits: those of an infinity or NaN are
// above every number's, so one of them anywhere shows in the result.
template <class V, int N>
struct Largest {
    uint32_t m = 0;
    __device__ __forceinline__ void look(const Pack<V, N>& p) {
#pragma unroll
        for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(to_f(p.v[i])) & 0x7fffffffu);
    }
    __device__ __forceinline__ uint32_t bits() const { return m; }
};
// 16-bit values two at a time.
__device__ __forceinline__ __nv_bfloat162 max_abs(__nv_bfloat162 m, __nv_bfloat162 x) { return __hmax2_nan(m, __habs2(x)); }
__device__ __forceinline__ __half2 max_abs(__half2 m, __half2 x) { return __hmax2_nan(m, __habs2(x)); }
template <class V>
struct Largest<V, 8> {
    using V2 = typename std::conditional<std::is_same<V, __half>::value, __half2, __nv_bfloat162>::type;
    uint32_t m = 0;  // two zeros
    __device__ __forceinline__ void look(const Pack<V, 8>& p) {
        V2 x[4], y;
        memcpy(x, &p, 16);
        memcpy(&y, &m, 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) y = max_abs(y, x[i]);
        memcpy(&m, &y, 4);
    }
    __device__ __forceinline__ uint32_t bits() const {
        V v[2];
        memcpy(v, &m, 4);
        return max(__float_as_uint(to_f(v[0])) & 0x7fffffffu, __float_as_uint(to_f(v[1])) & 0x7fffffffu);
    }
};

// Low bytes of N words.
template <int N>
__device__ __forceinline__ void low_bytes(const uint32_t (&t)[N], Pack<int8_t, N>& b) {
    if constexpr (N == 1) {
        b.v[0] = static_cast<int8_t>(t[0]);
    } else {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x0040), __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040), 0x5410);
        memcpy(&b, w, N);
    }
}

// The codes of a piece by division; a call, so that this rare path costs the
// kernel no registers.
template <class V, int N>
__device__ __noinline__ Pack<int8_t, N> divided_codes(Pack<V, N> p, float s) {
    Pack<int8_t, N> b;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float v = s > 0.f ? rintf(to_f(p.v[i]) / s) : 0.f;
        b.v[i] = static_cast<int8_t>(fminf(fmaxf(v, -127.f), 127.f));
    }
    return b;
}

// N values a piece: 16 bytes of X where rows are aligned, else 1 value.
template <class V, int N, int G>
__global__ void __launch_bounds__(kQThreads, 10)
    quant_rows_kernel(int M, int K, const V* X, long long ldx, int8_t* Q, long long ldq, float* scale) {
    using P = Pack<V, N>;
    using B = Pack<int8_t, N>;
    __shared__ uint32_t s_max[kQThreads / 32];
    let_next_start();
    wait_for_previous();
    X = behind_wait(X);
    const int row = blockIdx.x * (kQThreads / G) + threadIdx.x / G, at = threadIdx.x % G;
    if (row >= M) return;  // a whole group; G == kQThreads: never
    const P* x = reinterpret_cast<const P*>(X + row * ldx);
    B* q = reinterpret_cast<B*>(Q + row * ldq);
    const int np = K / N;
    Largest<V, N> big;
    P held[kQHeld];
#pragma unroll
    for (int h = 0; h < kQHeld; ++h)
        if (at + h * G < np) held[h] = load_once(x + at + h * G);
#pragma unroll
    for (int h = 0; h < kQHeld; ++h)
        if (at + h * G < np) big.look(held[h]);
    for (int k = at + kQHeld * G; k < np; k += G) big.look(load_once(x + k));
    uint32_t m = big.bits();
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (G > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
        __syncthreads();
        m = s_max[0];
#pragma unroll
        for (int w = 1; w < kQThreads / 32; ++w) m = max(m, s_max[w]);
    }
    const bool fine = m < 0x7f800000u;
    const float s = __uint_as_float(m) / 127.f;
    if (at == 0) scale[row] = fine ? s : __int_as_float(0x7fffffff);
    // The quotient x / s from the rounded reciprocal: a first quotient, its exact remainder (one fused multiply-add),
    // and a correction, which rounds it correctly (Markstein, "Computation of elementary functions on the IBM RISC
    // System/6000 processor", 1990).  In bf16 rows quotients that lie exactly between two whole numbers are common
    // (0.2% of them), so nothing less exact than the division itself would give its codes.  Subnormal scales, whose
    // reciprocal may not exist, divide; they are coarse, so the quotient may pass 127.
    const bool plain = fine && s >= 1e-30f;
    const float inv = plain ? 1.f / s : 0.f;
    constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
    auto code = [&](const P& p) {
        if (!plain) return divided_codes<V, N>(p, fine ? s : 0.f);
        B b;
        uint32_t t[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = to_f(p.v[i]), q0 = x * inv;
            t[i] = __float_as_uint(fmaf(fmaf(-q0, s, x), inv, q0) + kWhole);
        }
        low_bytes<N>(t, b);
        return b;
    };
#pragma unroll
    for (int h = 0; h < kQHeld; ++h)
        if (at + h * G < np) write_piece(q + at + h * G, code(held[h]));
    for (int k = at + kQHeld * G; k < np; k += G) write_piece(q + k, code(load_once(x + k)));
}

template <class V, int N>
cudaError_t quant_grid(int M, int K, const V* x, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int per = kQThreads / 32;
    const bool warps = M >= kQWarpRows && K <= (N == 1 ? 2048 : 256 * N);
    return warps ? launch_early(quant_rows_kernel<V, N, 32>, dim3((M + per - 1) / per), kQThreads, 0, 1, st, M, K, x,
                                          ldx, Q, ldq, scale)
                           : launch_early(quant_rows_kernel<V, N, kQThreads>, dim3(M), kQThreads, 0, 1, st, M, K, x, ldx, Q,
                                          ldq, scale);
}

template <class V>
cudaError_t quant_launch(int M, int K, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int N = 16 / sizeof(V);
    const V* x = static_cast<const V*>(X);
    if (spx_aligned(X, 16) && spx_aligned(Q, N) && ldx % N == 0 && ldq % N == 0 && K % N == 0)
        return quant_grid<V, N>(M, K, x, ldx, Q, ldq, scale, st);
    return quant_grid<V, 1>(M, K, x, ldx, Q, ldq, scale, st);
}

// ---------------------------------------------------------------- few rows

// Up to 8 NB rows of one expert against its channels, bound by the weights'
// bytes: a warp owns 16 MT channels and streams their codes from memory
// straight into matrix fragments.  The order of the reduction is free, so a
// lane's 16 neighbouring codes of a channel and the same 16 of a row are the
// operands of four m16n8k16 products, widened to fp16 in registers; up to eight
// rows they are those of two integer m16n8k32 products as they are (which run
// at a quarter of the fp16 form's rate here, 151 against 601 Tops, but eight
// rows need no more, and there is nothing to widen).  a.ks warps of a CTA share
// a channel block's reduction, in turns of 64 terms, where there are few blocks;
// their sums meet in shared memory.  A warp's fp32 sums go to int32 every 1024 terms, so they are exact.

constexpr long long kFewEnough = 152 * 64;  // warps that keep the memory busy

struct FewArgs {
    const int* offsets;
    int E, S, N, K, ks;
    const int8_t* Q;
    long long ldq;
    const float* row_scale;
    const int8_t* W;
    long long ldw, stride_w;
    const float* col_scale;
    void* C;
    long long ldc;
    spx_type c_type;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void few_store(const FewArgs& a, long long i, float v) {
    if (a.c_type == SPX_F32) static_cast<float*>(a.C)[i] = v;
    else if (a.c_type == SPX_BF16) static_cast<__nv_bfloat16*>(a.C)[i] = from_f<__nv_bfloat16>(v);
    else static_cast<__half*>(a.C)[i] = from_f<__half>(v);
}

template <int NB, int MT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) i8_few_kernel(FewArgs a) {
    constexpr int TM = 8 * NB, CH = 16 * MT;
    __shared__ int part[WARPS][TM * CH];
    let_next_start();
    wait_for_previous();
    a.Q = behind_wait(a.Q), a.W = behind_wait(a.W), a.row_scale = behind_wait(a.row_scale), a.col_scale = behind_wait(a.col_scale);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int e = 0, r0 = blockIdx.y * TM, hi = a.S;
    if (a.offsets && !warp_find_tile(a.offsets, a.E, a.S, TM, blockIdx.y, e, r0, hi)) return;
    const int R = min(TM, hi - r0);
    const int n0 = (blockIdx.x * (WARPS / a.ks) + warp / a.ks) * CH, turn = warp % a.ks;
    const bool on = n0 < a.N && R > 0;  // the same for the warps that share a block
    int* mine = part[warp];
#pragma unroll
    for (int i = 0; i < TM * CH / 32; ++i) mine[lane + 32 * i] = 0;
    __syncwarp();
    if (on && e < a.E) {
        const int8_t* w[2 * MT];
        const int8_t* q[NB];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m)
            w[m] = a.W + e * a.stride_w + static_cast<long long>(min(n0 + 8 * m + g, a.N - 1)) * a.ldw + 16 * t;
#pragma unroll
        for (int b = 0; b < NB; ++b) q[b] = a.Q + static_cast<long long>(min(r0 + 8 * b + g, a.S - 1)) * a.ldq + 16 * t;
        constexpr bool INT = NB == 1;
        using Acc = typename std::conditional<INT, int, float>::type;
        Acc acc[MT][NB][4];
        auto clear = [&]() {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][b][i] = Acc(0);
        };
        // value i of (m, b) is channel 16 m + g + 8 (i / 2), row 8 b + 2 t + i % 2
        auto flush = [&]() {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mine[(8 * b + 2 * t + (i & 1)) * CH + 16 * m + g + 8 * (i >> 1)] += INT ? static_cast<int>(acc[m][b][i]) : __float2int_rn(static_cast<float>(acc[m][b][i]));
        };
        constexpr int U = MT * NB > 4 ? 2 : 4;  // chunks of 64 terms whose weights are in flight
        const int step = 64 * a.ks;
        int done = 0;
        clear();
        for (int k0 = 64 * turn; k0 < a.K; k0 += step * U) {
            int4 x[U][2 * MT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * step;
                const bool in = k + 16 * t < a.K;  // K is a multiple of 16
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m)
                    x[u][m] = in ? load_once(reinterpret_cast<const int4*>(w[m] + k)) : make_int4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * step;
                if (k >= a.K) break;
                const bool in = k + 16 * t < a.K;
                if constexpr (INT) {
                    const int4 y = in ? load(reinterpret_cast<const int4*>(q[0] + k)) : make_int4(0, 0, 0, 0);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int4 &lo = x[u][2 * m], &up = x[u][2 * m + 1];
                        mma16832(acc[m][0], lo.x, up.x, lo.y, up.y, y.x, y.y);
                        mma16832(acc[m][0], lo.z, up.z, lo.w, up.w, y.z, y.w);
                    }
                    continue;
                } else {
                    uint2 f[2 * MT][4];
#pragma unroll
                    for (int m = 0; m < 2 * MT; ++m) {
                        f[m][0] = widen_codes(x[u][m].x), f[m][1] = widen_codes(x[u][m].y);
                        f[m][2] = widen_codes(x[u][m].z), f[m][3] = widen_codes(x[u][m].w);
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int4 y = in ? load(reinterpret_cast<const int4*>(q[b] + k)) : make_int4(0, 0, 0, 0);
                        const uint2 h[4] = {widen_codes(y.x), widen_codes(y.y), widen_codes(y.z), widen_codes(y.w)};
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                mma16816(acc[m][b], f[2 * m][s].x, f[2 * m + 1][s].x, f[2 * m][s].y, f[2 * m + 1][s].y, h[s].x,
                                         h[s].y);
                    }
                }
            }
            done += 64 * U;
            if (!INT && done == 1024) {  // U divides 16
                flush();
                clear();
                done = 0;
            }
        }
        flush();
    }
    if (a.ks > 1) __syncthreads();
    else __syncwarp();
    if (!on) return;
    // the sharing warps' sums, each warp a part of the rows
    const int first = warp - turn;
    for (int i = 32 * turn + lane; i < TM * CH; i += 32 * a.ks) {
        const int r = i / CH, n = n0 + i % CH;
        if (r >= R || n >= a.N) continue;
        int sum = 0;
        for (int p = 0; p < a.ks; ++p) sum += part[first + p][i];
        const float v = e < a.E ? static_cast<float>(sum) * (load(a.row_scale + r0 + r) *
                                                             load(a.col_scale + static_cast<long long>(e) * a.N + n))
                                : 0.f;
        few_store(a, (r0 + r) * a.ldc + n, v);
    }
}

template <int NB, int MT, int WARPS>
cudaError_t few_grid(FewArgs a, long long blocks, long long row_tiles, cudaStream_t st) {
    const long long per = WARPS / a.ks;
    return launch_early(i8_few_kernel<NB, MT, WARPS>,
                        dim3(static_cast<unsigned>((blocks + per - 1) / per), static_cast<unsigned>(row_tiles)), 32 * WARPS, 0,
                        1, st, a);
}

// A block's reduction is shared among warps until there are warps enough for the memory's latency: by the four of a
// small CTA, or by MOST of a large one where even that leaves few (8 rows x 4096 x 4096: 7.0 us, 8.3 with four).
template <int NB, int MT, int MOST>
cudaError_t few_launch(FewArgs a, long long row_tiles, cudaStream_t st) {
    const long long blocks = (a.N + 16 * MT - 1) / (16 * MT);
    const long long tiles = a.E == 1 ? (a.S + 8 * NB - 1) / (8 * NB) : std::min(a.E, a.S);
    a.ks = 1;
    while (a.ks < 4 && blocks * tiles * a.ks < kFewEnough && 64 * 2 * a.ks < a.K) a.ks *= 2;
    while (a.ks >= 4 && a.ks < MOST && blocks * tiles * a.ks < kFewEnough / 4 && 64 * 2 * a.ks < a.K) a.ks *= 2;
    return a.ks <= 4 ? few_grid<NB, MT, 4>(a, blocks, row_tiles, st) : few_grid<NB, MT, MOST>(a, blocks, row_tiles, st);
}

// One row (blockIdx.y) against its expert's channels, on the CUDA cores' byte
// dot product: a warp takes kChan channels, its lanes 16 codes of each at a
// time, so the reduction is split over the lanes and needs no shared memory.
// One row x 4096 x 4096 4.4 us, 6.4 with matrix fragments; at four rows 8.5 and 7.0.
constexpr int kRowChan = 2, kRowThreads = 128, kRowMost = 2;

__global__ void __launch_bounds__(kRowThreads) i8_row_kernel(FewArgs a) {
    let_next_start();
    wait_for_previous();
    a.Q = behind_wait(a.Q), a.W = behind_wait(a.W), a.row_scale = behind_wait(a.row_scale), a.col_scale = behind_wait(a.col_scale);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int e = 0, p = blockIdx.y, hi = a.S;
    if (a.offsets && !warp_find_tile(a.offsets, a.E, a.S, 1, blockIdx.y, e, p, hi)) return;
    const int n0 = (blockIdx.x * (kRowThreads / 32) + warp) * kRowChan, np = a.K / 16;
    if (n0 >= a.N) return;
    int sum[kRowChan] = {};
    if (e < a.E) {
        const int4* w[kRowChan];
#pragma unroll
        for (int c = 0; c < kRowChan; ++c)
            w[c] = reinterpret_cast<const int4*>(a.W + e * a.stride_w + static_cast<long long>(min(n0 + c, a.N - 1)) * a.ldw);
        const int4* q = reinterpret_cast<const int4*>(a.Q + p * a.ldq);
        constexpr int U = 4;  // pieces in flight
        for (int p0 = lane; p0 < np; p0 += 32 * U) {
            int4 y[U][kRowChan];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < kRowChan; ++c)
                    y[u][c] = p0 + 32 * u < np ? load_once(w[c] + p0 + 32 * u) : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int4 x = p0 + 32 * u < np ? load(q + p0 + 32 * u) : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < kRowChan; ++c) {
                    sum[c] = __dp4a(x.x, y[u][c].x, sum[c]);
                    sum[c] = __dp4a(x.y, y[u][c].y, sum[c]);
                    sum[c] = __dp4a(x.z, y[u][c].z, sum[c]);
                    sum[c] = __dp4a(x.w, y[u][c].w, sum[c]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kRowChan; ++c) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], d);
        if (lane == c && n0 + c < a.N)
            few_store(a, p * a.ldc + n0 + c,
                      e < a.E ? static_cast<float>(sum[c]) *
                                    (load(a.row_scale + p) * load(a.col_scale + static_cast<long long>(e) * a.N + n0 + c))
                              : 0.f);
    }
}

// Row tiles of 8, 16 or 32 rows, by an expert's average (at most kFewRows): most experts are one tile.
spx_status few_product(const FewArgs& a, cudaStream_t st) {
    if (a.S <= kRowMost) {
        constexpr int per = kRowThreads / 32 * kRowChan;
        spx_note_launches(1);
        return spx_cuda_status(launch_early(i8_row_kernel, dim3((a.N + per - 1) / per, a.S), kRowThreads, 0, 1, st, a));
    }
    const long long avg = (a.S + a.E - 1) / a.E, most = a.E == 1 ? avg : 3 * avg / 2;
    const int nb = most <= 8 ? 1 : most <= 16 ? 2 : 4;
    const long long ty = a.offsets ? std::min<long long>(max_row_tiles(a.E, a.S, 8 * nb), static_cast<long long>(a.S) + 1)
                                   : (a.S + 8 * nb - 1) / (8 * nb);
    spx_note_launches(1);
    return spx_cuda_status(nb == 1   ? few_launch<1, 1, 16>(a, ty, st)
                           : nb == 2 ? few_launch<2, 1, 16>(a, ty, st)
                                     : few_launch<4, 2, 8>(a, ty, st));
}

// ---------------------------------------------------------------- codes to fp16

// The rows of Q and of every expert that has rows, as fp16 with a row pitch of
// Kp (a multiple of 8) values; what lies between K and Kp is never read.
// blockIdx.y: 0 for Q, 1 + e for W_e.
constexpr int kWidenThreads = 256;

template <bool ALIGNED>
__global__ void __launch_bounds__(kWidenThreads)
    widen_kernel(const int* offsets, int S, int N, int K, int Kp, const int8_t* Q, long long ldq, const int8_t* W,
                 long long ldw, long long stride_w, __half* Q16, __half* W16, bool same_w) {
    let_next_start();
    wait_for_previous();
    offsets = behind_wait(offsets), Q = behind_wait(Q), W = behind_wait(W);
    const int8_t* src = Q;
    __half* dst = Q16;
    long long ld = ldq;
    int rows = S;
    if (blockIdx.y > 0) {
        const int e = blockIdx.y - 1;
        if (offsets && !same_w) {
            int lo, hi;
            expert_rows(offsets, e, S, lo, hi);
            if (lo == hi) return;
        }
        src = W + e * stride_w, ld = ldw, rows = N;
        dst = W16 + static_cast<long long>(e) * N * Kp;
    }
    // eight codes a piece: a warp's loads and stores are both contiguous
    const int np = (K + 7) / 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int U = 4;  // pieces in flight
    for (int r = blockIdx.x * (kWidenThreads / 32) + warp; r < rows; r += gridDim.x * (kWidenThreads / 32)) {
        const int8_t* s = src + r * ld;
        __half* d = dst + static_cast<long long>(r) * Kp;
        for (int p0 = lane; p0 < np; p0 += 32 * U) {
            uint2 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = 8 * (p0 + 32 * u);
                w[u] = make_uint2(0u, 0u);
                if (ALIGNED && k + 8 <= K) {
                    w[u] = load_once(reinterpret_cast<const uint2*>(s + k));
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (k + c < K)
                            (c < 4 ? w[u].x : w[u].y) |= static_cast<uint32_t>(static_cast<uint8_t>(load(s + k + c))) << (8 * (c & 3));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = p0 + 32 * u;
                const uint2 lo = widen_codes(w[u].x), hi = widen_codes(w[u].y);
                if (p < np) reinterpret_cast<uint4*>(d)[p] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
}

// Which kernel, by an expert's average rows (us, few rows / widened on the way / through widened copies; unevenly routed):
//   64 experts of 2048 x 2048: 4 rows 50/103/206, 16 rows 104/118/215, 64 rows (evenly) 190/124/217
//   8 of 4096 x 2048: 8 rows 26/35/54, 32 rows 41/39/56, 128 rows 101/65/64
//   one of 4096 x 4096: 16 rows 10/13/15, 32 rows 13/14/16, 64 rows 14/15/16, 128 rows 26/18/18
constexpr int kFewRows = 16, kWidenRows = 128;

int64_t avg_rows(int E, int S) { return (static_cast<int64_t>(S) + E - 1) / E; }

int pitch16(int K) { return (K + 7) / 8 * 8; }

}  // namespace

int spx_int8_check_take() { return spx_check_take(g_experts_check); }

extern "C" {

spx_status spx_quant_rows_i8(int32_t M, int32_t K, spx_type type, const void* X, int64_t ldx, int8_t* Q, int64_t ldq,
                             float* scale, spx_stream_t stream) {
    if (M < 0 || K < 0 || !is_float_type(type)) return SPX_ERR_ARG;
    if (M > kMostIndex || K > kMostIndex) return SPX_ERR_INDEX_RANGE;
    if (M == 0) return SPX_OK;
    if (!scale || (K > 0 && (!X || !Q || ldx < K || ldq < K))) return SPX_ERR_ARG;
    if (!spx_aligned(X, type_bytes(type)) || !spx_aligned(scale, 4)) return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    spx_note_launches(1);
    return spx_cuda_status(type == SPX_F32    ? quant_launch<float>(M, K, X, ldx, Q, ldq, scale, st)
                           : type == SPX_BF16 ? quant_launch<__nv_bfloat16>(M, K, X, ldx, Q, ldq, scale, st)
                                              : quant_launch<__half>(M, K, X, ldx, Q, ldq, scale, st));
}

size_t spx_gemm_i8_scratch_bytes(int32_t E, int32_t S, int32_t N, int32_t K, int32_t wide) {
    if (E <= 0 || S <= 0 || N <= 0 || K <= 0 || (wide && avg_rows(E, S) <= kWidenRows)) return 0;
    const size_t row = 2 * static_cast<size_t>(pitch16(K));
    const size_t q = (row * S + 255) / 256 * 256;
    return q + row * N * static_cast<size_t>(E);
}

spx_status spx_gemm_i8(int32_t E, int32_t S, int32_t N, int32_t K, const int32_t* offsets, const int8_t* Q,
                       int64_t ldq, const float* row_scale, const int8_t* W, int64_t ldw, int64_t stride_w,
                       const float* w_scale, void* C, int64_t ldc, spx_type c_type, void* scratch,
                       size_t scratch_bytes, spx_stream_t stream) {
    if (E <= 0 || S < 0 || N < 0 || K < 0 || !is_float_type(c_type)) return SPX_ERR_ARG;
    if (!offsets && E != 1) return SPX_ERR_ARG;
    if (E > SPX_MAX_EXPERTS || K > SPX_I8_MAX_K) return SPX_ERR_UNSUPPORTED;
    if (S > kMostIndex || N > kMostIndex) return SPX_ERR_INDEX_RANGE;
    if (S == 0 || N == 0) return SPX_OK;
    if (!row_scale || !w_scale || !C || ldc < N || (K > 0 && (!Q || !W || ldq < K || ldw < K || stride_w < 0)))
        return SPX_ERR_ARG;
    if (!spx_aligned(offsets, 4) || !spx_aligned(row_scale, 4) || !spx_aligned(w_scale, 4) ||
        !spx_aligned(C, type_bytes(c_type)))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t cb = type_bytes(c_type);
    if (K == 0)
        return spx_cuda_status(cudaMemset2DAsync(C, static_cast<size_t>(ldc) * cb, 0, static_cast<size_t>(N) * cb,
                                                 static_cast<size_t>(S), st));
    const int64_t rows = avg_rows(E, S);
    const bool wide = tc_codes_fit(Q, ldq, W, ldw, stride_w);  // rows on 16-byte boundaries
    if (wide && K % 16 == 0 && rows <= kFewRows)
        return few_product(FewArgs{offsets, E, S, N, K, 1, Q, ldq, row_scale, W, ldw, stride_w, w_scale, C, ldc, c_type}, st);
    if (wide && rows <= kWidenRows)
        return tc_product_codes(E, S, N, K, offsets, Q, ldq, row_scale, W, ldw, stride_w, w_scale, C, ldc, c_type, st);
    const size_t need = spx_gemm_i8_scratch_bytes(E, S, N, K, wide);
    if (need > 0 && (!scratch || scratch_bytes < need)) return SPX_ERR_ARG;
    if (need > 0 && !spx_aligned(scratch, 256)) return SPX_ERR_ALIGN;
    const bool same_w = E == 1 || stride_w == 0;
    const int Kp = pitch16(K), mats = same_w ? 1 : E;
    __half* Q16 = static_cast<__half*>(scratch);
    __half* W16 = Q16 + (static_cast<size_t>(Kp) * S + 127) / 128 * 128;
    {
        const bool aligned = spx_aligned(Q, 8) && spx_aligned(W, 8) && ldq % 8 == 0 && ldw % 8 == 0 && stride_w % 8 == 0;
        constexpr int per = kWidenThreads / 32;  // a row a warp
        const dim3 grid(std::min((std::max(S, N) + per - 1) / per, 1216), 1 + mats);
        const cudaError_t e = launch_early(aligned ? widen_kernel<true> : widen_kernel<false>, grid, kWidenThreads, 0, 1, st,
                                           offsets, S, N, K, Kp, Q, ldq, W, ldw, stride_w, Q16, W16, same_w);
        if (e != cudaSuccess) return spx_cuda_status(e);
        spx_note_launches(1);
    }
    return tc_product_i8(E, S, N, K, offsets, Q16, Kp, row_scale, W16, Kp, mats, w_scale, C, ldc, c_type, st);
}

}  // extern "C"
