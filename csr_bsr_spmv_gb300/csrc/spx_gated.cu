// spx_gated.cu -- experts with a gate and their gradient: entry points.  Both
// run on the experts' product kernels with the gate between the sums and what
// is stored (spx_act.cuh), so neither the factors before the activation nor the
// gradient behind it pass through memory on their own.  Measured: 32768 rows over
// 16 experts, 2 x 2048 of 2048 bf16, 358 to 365 us replayed as a graph and 377 as
// calls, 1.46 to 1.53 PFLOP/s, at the power limit (326 in a single launch; a
// library product of as many operations 336 to 353 repeated); its gradient 228 to
// 237 us and 243 (a library product of that size 182); a few rows an expert are
// bound by the weights' bytes (35 us at 6.1 TB/s).  fp32 instead of bf16 output
// costs 3% without H, 1% with it, "nk" weights of the gradient nothing.
#include "spx_act.cuh"

using namespace spx_exp;

namespace {

spx_status check_sizes(int32_t E, int32_t S, int32_t F, int32_t R) {
    if (E <= 0 || S < 0 || F < 0 || R < 0) return SPX_ERR_ARG;
    if (E > SPX_MAX_EXPERTS) return SPX_ERR_UNSUPPORTED;
    if (S > kMostIndex || 2 * static_cast<int64_t>(F) > kMostIndex || R > kMostIndex) return SPX_ERR_INDEX_RANGE;
    return SPX_OK;
}

bool act_ok(spx_act act) { return act == SPX_ACT_SILU || act == SPX_ACT_GELU || act == SPX_ACT_GELU_TANH; }

}  // namespace

extern "C" {

spx_status spx_gemm_grouped_gated(int32_t E, int32_t S, int32_t F, int32_t K, const int32_t* offsets, const void* A,
                                  int64_t lda, const void* W, int64_t ldw, int64_t stride_w, spx_act act, spx_type type,
                                  void* H, int64_t ldh, void* C, int64_t ldc, spx_type c_type, spx_stream_t stream) {
    const spx_status c = check_sizes(E, S, F, K);
    if (c != SPX_OK) return c;
    if (!is_half_type(type) || (c_type != type && c_type != SPX_F32) || !act_ok(act) || (!offsets && E != 1)) return SPX_ERR_ARG;
    if (S == 0 || F == 0) return SPX_OK;
    if (!C || ldc < F || (H && ldh < 2 * static_cast<int64_t>(F)) || (K > 0 && (!A || !W || lda < K || ldw < K || stride_w < 0)))
        return SPX_ERR_ARG;
    if (!spx_aligned(offsets, 4) || !spx_aligned(A, 2) || !spx_aligned(W, 2) || !spx_aligned(H, 2) ||
        !spx_aligned(C, type_bytes(c_type)))
        return SPX_ERR_ALIGN;
    Gate gate;
    gate.epi = kGate, gate.act = act, gate.H = H, gate.ldh = ldh;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (K > 0 && tc_product_fits(A, lda, W, ldw, stride_w, E))
        return tc_gated(E, S, F, K, offsets, A, lda, W, ldw, stride_w, gate, type, C, ldc, c_type, st);
    SimtGemm g{};
    g.L = A, g.li = lda, g.lr = 1;
    g.R = W, g.rj = ldw, g.rr = 1, g.re = stride_w;
    g.C = C, g.ldc = ldc;
    g.offsets = offsets, g.E = E, g.S = S, g.NI = S, g.NJ = F, g.NR = K, g.by_rows = true;
    return simt_gated(g, gate, type, c_type, st);
}

spx_status spx_gemm_grouped_gated_grad(int32_t E, int32_t S, int32_t F, int32_t N, const int32_t* offsets, const void* dY,
                                       int64_t lddy, const void* W, int64_t ldw, int64_t stride_w, spx_w_layout layout,
                                       spx_act act, spx_type type, const void* H, int64_t ldh, void* dH, int64_t lddh,
                                       void* C, int64_t ldc, spx_stream_t stream) {
    const spx_status c = check_sizes(E, S, F, N);
    if (c != SPX_OK) return c;
    if (!is_half_type(type) || !act_ok(act) || (layout != SPX_W_NK && layout != SPX_W_KN) || (!offsets && E != 1)) return SPX_ERR_ARG;
    if (S == 0 || F == 0) return SPX_OK;
    const bool kn = layout == SPX_W_KN;
    const int64_t two = 2 * static_cast<int64_t>(F);
    if (!H || ldh < two || !dH || lddh < two || (C && ldc < F) ||
        (N > 0 && (!dY || !W || lddy < N || ldw < (kn ? F : N) || stride_w < 0)))
        return SPX_ERR_ARG;
    if (!spx_aligned(offsets, 4) || !spx_aligned(dY, 2) || !spx_aligned(W, 2) || !spx_aligned(H, 2) || !spx_aligned(dH, 2) ||
        !spx_aligned(C, 2))
        return SPX_ERR_ALIGN;
    Gate gate;
    gate.epi = kGateGrad, gate.act = act, gate.H = const_cast<void*>(H), gate.ldh = ldh, gate.dH = dH, gate.lddh = lddh;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N > 0 && tc_product_fits(dY, lddy, W, ldw, stride_w, E))
        return tc_gated_grad(E, S, F, N, offsets, dY, lddy, W, ldw, stride_w, layout, gate, type, C, ldc, st);
    SimtGemm g{};
    g.L = dY, g.li = lddy, g.lr = 1;
    g.R = W, g.rj = kn ? 1 : ldw, g.rr = kn ? ldw : 1, g.re = stride_w;
    g.C = C, g.ldc = ldc;
    g.offsets = offsets, g.E = E, g.S = S, g.NI = S, g.NJ = F, g.NR = N, g.by_rows = true;
    return simt_gated(g, gate, type, type, st);
}

}  // extern "C"
