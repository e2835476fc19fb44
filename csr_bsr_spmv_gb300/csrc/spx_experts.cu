// spx_experts.cu -- the experts' products and their gradients: entry points.
#include <algorithm>

#include "spx_experts.cuh"

using namespace spx_exp;

namespace {

spx_status check_sizes(int32_t E, int32_t S, int32_t N, int32_t K) {
    if (E <= 0 || S < 0 || N < 0 || K < 0) return SPX_ERR_ARG;
    if (E > SPX_MAX_EXPERTS) return SPX_ERR_UNSUPPORTED;
    if (S > kMostIndex || N > kMostIndex || K > kMostIndex) return SPX_ERR_INDEX_RANGE;
    return SPX_OK;
}

}  // namespace

extern "C" {

spx_status spx_gemm_grouped(int32_t E, int32_t S, int32_t N, int32_t K, const int32_t* offsets, const void* A,
                            int64_t lda, const void* W, int64_t ldw, int64_t stride_w, spx_w_layout layout,
                            spx_type type, void* C, int64_t ldc, spx_type c_type, spx_stream_t stream) {
    const spx_status c = check_sizes(E, S, N, K);
    if (c != SPX_OK) return c;
    if (!is_half_type(type) || (c_type != type && c_type != SPX_F32)) return SPX_ERR_ARG;
    if (layout != SPX_W_NK && layout != SPX_W_KN) return SPX_ERR_ARG;
    if (S == 0 || N == 0) return SPX_OK;
    const bool nk = layout == SPX_W_NK;
    if (!offsets || !C || ldc < N || (K > 0 && (!A || !W || lda < K || ldw < (nk ? K : N) || stride_w < 0)))
        return SPX_ERR_ARG;
    if (!spx_aligned(offsets, 4) || !spx_aligned(A, 2) || !spx_aligned(W, 2) || !spx_aligned(C, type_bytes(c_type)))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (K > 0 && tc_product_fits(A, lda, W, ldw, stride_w, E))
        return tc_product(E, S, N, K, offsets, A, lda, W, ldw, stride_w, layout, type, C, ldc, c_type, st);
    SimtGemm g{};
    g.L = A, g.li = lda, g.lr = 1;
    g.R = W, g.rj = nk ? ldw : 1, g.rr = nk ? 1 : ldw, g.re = stride_w;
    g.C = C, g.ldc = ldc;
    g.offsets = offsets, g.E = E, g.S = S, g.NI = S, g.NJ = N, g.NR = K, g.by_rows = true;
    return simt_gemm(g, type, c_type, st);
}

spx_status spx_gemm_grouped_wgrad(int32_t E, int32_t S, int32_t N, int32_t K, const int32_t* offsets, const void* G,
                                  int64_t ldg, const void* A, int64_t lda, spx_type type, void* dW, int64_t ldw,
                                  int64_t stride_w, spx_type w_type, spx_stream_t stream) {
    const spx_status c = check_sizes(E, S, N, K);
    if (c != SPX_OK) return c;
    if (!is_half_type(type) || (w_type != type && w_type != SPX_F32)) return SPX_ERR_ARG;
    if (N == 0 || K == 0) return SPX_OK;
    if (!offsets || !dW || ldw < K || stride_w < 0 || (S > 0 && (!G || !A || ldg < N || lda < K))) return SPX_ERR_ARG;
    if (E > 1 && stride_w < (N - 1) * ldw + K) return SPX_ERR_ARG;  // the experts' gradients may not overlap
    if (!spx_aligned(offsets, 4) || !spx_aligned(G, 2) || !spx_aligned(A, 2) || !spx_aligned(dW, type_bytes(w_type)))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (S > 0 && tc_wgrad_fits(G, ldg, A, lda))
        return tc_wgrad(E, S, N, K, offsets, G, ldg, A, lda, type, dW, ldw, stride_w, w_type, st);
    SimtGemm g{};
    g.L = G, g.li = 1, g.lr = ldg;
    g.R = A, g.rj = 1, g.rr = lda;
    g.C = dW, g.ldc = ldw, g.ce = stride_w;
    g.offsets = offsets, g.E = E, g.S = S, g.NI = N, g.NJ = K, g.by_rows = false;
    return simt_gemm(g, type, w_type, st);
}

}  // extern "C"
