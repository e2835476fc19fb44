// spx_int8.cu -- rows quantised to 8 bits and the product of 8-bit integers
// with a scale for each row and output channel.
#include <algorithm>

#include "spx_experts.cuh"

using namespace spx_exp;

namespace {

// One CTA a row: its largest magnitude, then the codes.  Bound by HBM: the
// second read of the row comes from L1 / L2.
constexpr int kQThreads = 256;

template <class V>
__global__ void __launch_bounds__(kQThreads)
    quant_rows_kernel(int K, const V* __restrict__ X, long long ldx, int8_t* __restrict__ Q, long long ldq,
                      float* __restrict__ scale) {
    __shared__ float s_max[kQThreads / 32];
    const V* x = X + blockIdx.x * ldx;
    int8_t* q = Q + blockIdx.x * ldq;
    // a NaN or infinity anywhere makes `bad` NaN: v * 0 is 0 for every other value
    float m = 0.f, bad = 0.f;
    for (int k = threadIdx.x; k < K; k += kQThreads) {
        const float v = to_f(x[k]);
        m = fmaxf(m, fabsf(v));
        bad = fmaf(v, 0.f, bad);
    }
    if (bad != bad) m = __int_as_float(0x7f800000);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = s_max[0];
#pragma unroll
    for (int w = 1; w < kQThreads / 32; ++w) m = fmaxf(m, s_max[w]);
    const bool fine = m < __int_as_float(0x7f800000);
    const float s = m / 127.f;
    if (threadIdx.x == 0) scale[blockIdx.x] = fine ? s : __int_as_float(0x7fffffff);
    for (int k = threadIdx.x; k < K; k += kQThreads) {
        // a subnormal scale is coarse, so the quotient may pass 127
        const float v = fine && s > 0.f ? rintf(to_f(x[k]) / s) : 0.f;
        q[k] = static_cast<int8_t>(fminf(fmaxf(v, -127.f), 127.f));
    }
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
    if (type == SPX_F32)
        quant_rows_kernel<float><<<M, kQThreads, 0, st>>>(K, static_cast<const float*>(X), ldx, Q, ldq, scale);
    else if (type == SPX_BF16)
        quant_rows_kernel<__nv_bfloat16>
            <<<M, kQThreads, 0, st>>>(K, static_cast<const __nv_bfloat16*>(X), ldx, Q, ldq, scale);
    else
        quant_rows_kernel<__half><<<M, kQThreads, 0, st>>>(K, static_cast<const __half*>(X), ldx, Q, ldq, scale);
    spx_note_launches(1);
    return spx_cuda_status(cudaGetLastError());
}

size_t spx_gemm_i8_scratch_bytes(int32_t E, int32_t S, int32_t N, int32_t K) { return 0; }

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
    const size_t need = spx_gemm_i8_scratch_bytes(E, S, N, K);
    if (need > 0 && (!scratch || scratch_bytes < need)) return SPX_ERR_ARG;
    if (need > 0 && !spx_aligned(scratch, 256)) return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    SimtGemm g{};
    g.L = Q, g.li = ldq, g.lr = 1;
    g.R = W, g.rj = ldw, g.rr = 1, g.re = stride_w;
    g.C = C, g.ldc = ldc;
    g.row_scale = row_scale, g.col_scale = w_scale;
    g.offsets = offsets, g.E = E, g.S = S, g.NI = S, g.NJ = N, g.NR = K, g.by_rows = true;
    return simt_gemm(g, SPX_I8, c_type, st);
}

}  // extern "C"
