// spx_int8.cu -- rows quantised to 8 bits and the product of 8-bit integers
// with a scale for each row and output channel.
//
// This chip has no fast 8-bit integer matrix rate, but fp16 holds every code
// exactly and the fp16 tensor cores sum their products exactly in fp32 up to
// 2^24, so the product runs on the experts' tensor-core kernel with codes
// widened to fp16, and its integer sums stay exact (see kExact there).  A few
// rows (decoded tokens) are bound by the weights' bytes: they run on the CUDA
// cores' four-way byte dot product straight from the 8-bit weights.
#include <algorithm>
#include <type_traits>

#include "spx_experts.cuh"

using namespace spx_exp;

namespace {

// ---------------------------------------------------------------- quantisation

// A row's largest magnitude, then its codes.  Bound by HBM.  A group of G
// threads takes a row: a warp where there are rows enough to fill the SMs (16384
// rows x 2048 bf16: MEASURE us, a CTA a row 52), a CTA otherwise.  Up to kQHeld
// pieces a thread stay in registers between the two; a longer row is read again
// (from L2).
constexpr int kQThreads = 256, kQHeld = 8;
constexpr int kQWarpRows = 1216;  // rows from which a warp takes one: eight a CTA, one CTA an SM

template <class V, int N>
struct alignas(N * sizeof(V) >= 16 ? 16 : N * sizeof(V)) Pack {
    V v[N];
};

// A piece is read and written as one word of its size.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using T = uint4;
};
template <>
struct Word<8> {
    using T = uint2;
};
template <>
struct Word<4> {
    using T = uint32_t;
};
template <>
struct Word<2> {
    using T = uint16_t;
};
template <>
struct Word<1> {
    using T = uint8_t;
};
template <class P>
__device__ __forceinline__ P read_piece(const P* p) {
    using T = typename Word<sizeof(P)>::T;
    const T w = __ldcs(reinterpret_cast<const T*>(p));
    P r;
    memcpy(&r, &w, sizeof(P));
    return r;
}
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
__global__ void __launch_bounds__(kQThreads, 4)
    quant_rows_kernel(int M, int K, const V* __restrict__ X, long long ldx, int8_t* __restrict__ Q, long long ldq,
                      float* __restrict__ scale) {
    using P = Pack<V, N>;
    using B = Pack<int8_t, N>;
    __shared__ uint32_t s_max[kQThreads / 32];
    const int row = blockIdx.x * (kQThreads / G) + threadIdx.x / G, at = threadIdx.x % G;
    if (row >= M) return;  // a whole group; G == kQThreads: never
    const P* x = reinterpret_cast<const P*>(X + row * ldx);
    B* q = reinterpret_cast<B*>(Q + row * ldq);
    const int np = K / N;
    Largest<V, N> big;
    P held[kQHeld];
#pragma unroll
    for (int h = 0; h < kQHeld; ++h)
        if (at + h * G < np) held[h] = read_piece(x + at + h * G);
#pragma unroll
    for (int h = 0; h < kQHeld; ++h)
        if (at + h * G < np) big.look(held[h]);
    for (int k = at + kQHeld * G; k < np; k += G) big.look(read_piece(x + k));
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
    for (int k = at + kQHeld * G; k < np; k += G) write_piece(q + k, code(read_piece(x + k)));
}

template <class V, int N>
void quant_grid(int M, int K, const V* x, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int per = kQThreads / 32;
    if (M >= kQWarpRows) quant_rows_kernel<V, N, 32><<<(M + per - 1) / per, kQThreads, 0, st>>>(M, K, x, ldx, Q, ldq, scale);
    else quant_rows_kernel<V, N, kQThreads><<<M, kQThreads, 0, st>>>(M, K, x, ldx, Q, ldq, scale);
}

template <class V>
void quant_launch(int M, int K, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, cudaStream_t st) {
    constexpr int N = 16 / sizeof(V);
    const V* x = static_cast<const V*>(X);
    if (spx_aligned(X, 16) && spx_aligned(Q, N) && ldx % N == 0 && ldq % N == 0 && K % N == 0)
        quant_grid<V, N>(M, K, x, ldx, Q, ldq, scale, st);
    else
        quant_grid<V, 1>(M, K, x, ldx, Q, ldq, scale, st);
}

// ---------------------------------------------------------------- few rows

// Up to kFew rows of one expert against all its channels: a warp takes kChan
// channels, its lanes 16 codes of each at a time, so every weight is read
// once, in 16-byte pieces; the rows' codes come from L1.  Bound by the
// weights' bytes.
constexpr int kFew = 8, kChan = 2, kFewThreads = 128;

struct FewArgs {
    const int* offsets;
    int E, S, N, K;
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

template <int R>
__device__ __forceinline__ void few_rows(const FewArgs& a, int e, int r0, int n0, int (&sum)[kFew][kChan]) {
    const int lane = threadIdx.x & 31, np = a.K / 16;
    const int4* w[kChan];
#pragma unroll
    for (int c = 0; c < kChan; ++c)
        w[c] = reinterpret_cast<const int4*>(a.W + e * a.stride_w + static_cast<long long>(min(n0 + c, a.N - 1)) * a.ldw);
    const int4* q = reinterpret_cast<const int4*>(a.Q + r0 * a.ldq);
    const long long dq = a.ldq / 16;
    constexpr int U = R <= 2 ? 4 : 2;  // pieces in flight
    for (int p0 = 0; p0 < np; p0 += 32 * U) {
        int4 y[U][kChan];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < kChan; ++c) {
                const int p = p0 + 32 * u + lane;
                y[u][c] = p < np ? __ldcs(w[c] + p) : make_int4(0, 0, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + 32 * u + lane;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int4 x = p < np ? __ldg(q + r * dq + p) : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < kChan; ++c) {
                    sum[r][c] = __dp4a(x.x, y[u][c].x, sum[r][c]);
                    sum[r][c] = __dp4a(x.y, y[u][c].y, sum[r][c]);
                    sum[r][c] = __dp4a(x.z, y[u][c].z, sum[r][c]);
                    sum[r][c] = __dp4a(x.w, y[u][c].w, sum[r][c]);
                }
            }
        }
    }
}

template <class O>
__device__ __forceinline__ void few_store(const FewArgs& a, long long i, float v) {
    static_cast<O*>(a.C)[i] = from_f<O>(v);
}

__global__ void __launch_bounds__(kFewThreads) i8_few_kernel(FewArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int e = 0, r0 = 0, hi = a.S;
    if (a.offsets) {
        if (!warp_find_tile(a.offsets, a.E, a.S, kFew, blockIdx.y, e, r0, hi)) return;
    } else {
        r0 = blockIdx.y * kFew;
    }
    const int R = min(kFew, hi - r0);
    const int n0 = (blockIdx.x * (kFewThreads / 32) + warp) * kChan;
    if (n0 >= a.N || R <= 0) return;
    int sum[kFew][kChan];
#pragma unroll
    for (int r = 0; r < kFew; ++r)
#pragma unroll
        for (int c = 0; c < kChan; ++c) sum[r][c] = 0;
    if (e < a.E) {
        if (R == 1) few_rows<1>(a, e, r0, n0, sum);
        else if (R == 2) few_rows<2>(a, e, r0, n0, sum);
        else if (R <= 4) {
            if (R == 3) few_rows<3>(a, e, r0, n0, sum);
            else few_rows<4>(a, e, r0, n0, sum);
        } else {
            switch (R) {
                case 5: few_rows<5>(a, e, r0, n0, sum); break;
                case 6: few_rows<6>(a, e, r0, n0, sum); break;
                case 7: few_rows<7>(a, e, r0, n0, sum); break;
                default: few_rows<8>(a, e, r0, n0, sum);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
        if (r >= R) break;
#pragma unroll
        for (int c = 0; c < kChan; ++c)
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum[r][c] += __shfl_xor_sync(0xffffffffu, sum[r][c], d);
    }
    // lane r * kChan + c stores row r of channel n0 + c
#pragma unroll
    for (int r = 0; r < kFew; ++r)
#pragma unroll
        for (int c = 0; c < kChan; ++c) {
            if (lane != r * kChan + c || r >= R || n0 + c >= a.N) continue;
            const float v = e < a.E ? static_cast<float>(sum[r][c]) *
                                          (__ldg(a.row_scale + r0 + r) * __ldg(a.col_scale + static_cast<long long>(e) * a.N + n0 + c))
                                    : 0.f;
            const long long i = (r0 + r) * a.ldc + n0 + c;
            if (a.c_type == SPX_F32) few_store<float>(a, i, v);
            else if (a.c_type == SPX_BF16) few_store<__nv_bfloat16>(a, i, v);
            else few_store<__half>(a, i, v);
        }
}

// ---------------------------------------------------------------- codes to fp16

// Four codes (bytes of w) to fp16: 0x6400 | u is 1024 + u for a byte u, and
// u = code + 128 after flipping its top bit, so one subtraction is exact.
__device__ __forceinline__ uint2 widen_codes(uint32_t w) {
    w ^= 0x80808080u;
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The rows of Q and of every expert that has rows, as fp16 with a row pitch of
// Kp (a multiple of 8) values; what lies between K and Kp is never read.
// blockIdx.y: 0 for Q, 1 + e for W_e.
constexpr int kWidenThreads = 256;

template <bool ALIGNED>
__global__ void __launch_bounds__(kWidenThreads)
    widen_kernel(const int* __restrict__ offsets, int S, int N, int K, int Kp, const int8_t* __restrict__ Q,
                 long long ldq, const int8_t* __restrict__ W, long long ldw, long long stride_w,
                 __half* __restrict__ Q16, __half* __restrict__ W16, bool same_w) {
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
                    w[u] = __ldcs(reinterpret_cast<const uint2*>(s + k));
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (k + c < K)
                            (c < 4 ? w[u].x : w[u].y) |= static_cast<uint32_t>(static_cast<uint8_t>(s[k + c])) << (8 * (c & 3));
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

// The few-rows kernel is taken up to kFewEach rows an expert on average and
// kFewMore in all besides: 64 experts of 2048 x 2048, 64 rows 41 us (146 through
// 16-bit codes), 512 rows 141 (219), 1024 rows 244 (215); one of 4096 x 4096, 16
// rows 14 us (22), 32 rows 24 (22).
constexpr int kFewEach = 8, kFewMore = 8;

int pitch16(int K) { return (K + 7) / 8 * 8; }

bool few_fits(int E, int S, const int8_t* Q, int64_t ldq, const int8_t* W, int64_t ldw, int64_t stride_w, int K) {
    return S <= kFewEach * static_cast<int64_t>(E) + kFewMore && K % 16 == 0 && spx_aligned(Q, 16) && spx_aligned(W, 16) && ldq % 16 == 0 && ldw % 16 == 0 &&
           stride_w % 16 == 0;
}

}  // namespace

extern "C" {

spx_status spx_quant_rows_i8(int32_t M, int32_t K, spx_type type, const void* X, int64_t ldx, int8_t* Q, int64_t ldq,
                             float* scale, spx_stream_t stream) {
    if (M < 0 || K < 0 || !is_float_type(type)) return SPX_ERR_ARG;
    if (M == 0) return SPX_OK;
    if (!scale || (K > 0 && (!X || !Q || ldx < K || ldq < K))) return SPX_ERR_ARG;
    if (!spx_aligned(X, type_bytes(type)) || !spx_aligned(scale, 4)) return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (type == SPX_F32) quant_launch<float>(M, K, X, ldx, Q, ldq, scale, st);
    else if (type == SPX_BF16) quant_launch<__nv_bfloat16>(M, K, X, ldx, Q, ldq, scale, st);
    else quant_launch<__half>(M, K, X, ldx, Q, ldq, scale, st);
    spx_note_launches(1);
    return spx_cuda_status(cudaGetLastError());
}

size_t spx_gemm_i8_scratch_bytes(int32_t E, int32_t S, int32_t N, int32_t K) {
    if (E <= 0 || S <= 0 || N <= 0 || K <= 0) return 0;
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
    if (few_fits(E, S, Q, ldq, W, ldw, stride_w, K)) {
        const FewArgs a{offsets, E, S, N, K, Q, ldq, row_scale, W, ldw, stride_w, w_scale, C, ldc, c_type};
        const long long ty = offsets ? std::min<long long>(max_row_tiles(E, S, kFew), static_cast<long long>(S) + 1) : (S + kFew - 1) / kFew;
        i8_few_kernel<<<dim3((N + kFewThreads / 32 * kChan - 1) / (kFewThreads / 32 * kChan), static_cast<unsigned>(ty)),
                        kFewThreads, 0, st>>>(a);
        spx_note_launches(1);
        return spx_cuda_status(cudaGetLastError());
    }
    const size_t need = spx_gemm_i8_scratch_bytes(E, S, N, K);
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
        if (aligned)
            widen_kernel<true><<<grid, kWidenThreads, 0, st>>>(offsets, S, N, K, Kp, Q, ldq, W, ldw, stride_w, Q16, W16, same_w);
        else
            widen_kernel<false><<<grid, kWidenThreads, 0, st>>>(offsets, S, N, K, Kp, Q, ldq, W, ldw, stride_w, Q16, W16, same_w);
        spx_note_launches(1);
    }
    return tc_product_i8(E, S, N, K, offsets, Q16, Kp, row_scale, W16, Kp, mats, w_scale, C, ldc, c_type, st);
}

}  // extern "C"
