// spx_experts_simt.cu -- the experts' products on the CUDA cores, for arrays
// the copy engine cannot read: rows or bases off 16-byte boundaries.
//
// One kernel for the product and its gradients: out[i, j] = sum_r L(i, r)
// R(j, r) with any strides.  A CTA owns a 64 x 64 tile of the output; 32 terms
// at a time go through shared memory, each thread holds 4 x 4 fp32 sums.
// Bound by the FMA rate and the shared-memory reads that feed it (8 words for
// 16 FMAs): 32768 x 2047 x 4095 in 23.5 ms, 23 TFLOP/s, against 0.29 ms of
// 32768 x 2048 x 4096 on the tensor cores and 21.5 ms of a plain fp32 product.
#include "spx_act.cuh"
#include "spx_experts.cuh"

using namespace spx_exp;

namespace {

constexpr int kT = 64, kR = 32, kThreads = 256;

// 64 x 32 elements (x, r) of M at base + x * sx + r * sr, zeros outside [0, nx) x [0, nr); neighbouring
// threads take neighbouring addresses.
template <class V>
__device__ __forceinline__ void stage(float (*s)[kT + 1], const V* M, long long sx, long long sr, int nx,
                                      int nr) {
    const bool along_r = sr == 1;
    for (int i = threadIdx.x; i < kT * kR; i += kThreads) {
        const int x = along_r ? i / kR : i % kT, r = along_r ? i % kR : i / kT;
        s[r][x] = x < nx && r < nr ? to_f(load(M + x * sx + r * sr)) : 0.f;
    }
}

// EPI: kGate sums both factors of the gated product, kGateGrad passes the sums through the gate's gradient.
template <class V, class O, int EPI>
__global__ void __launch_bounds__(kThreads) experts_simt_kernel(SimtGemm g, Gate gate) {
    __shared__ float sl[kR][kT + 1], sr[EPI == kGate ? 2 : 1][kR][kT + 1];
    __shared__ int s_e, s_lo, s_hi;
    let_next_start();
    wait_for_previous();
    const V *L = static_cast<const V*>(behind_wait(g.L)), *R = static_cast<const V*>(behind_wait(g.R));
    O* C = static_cast<O*>(g.C);
    const int j0 = blockIdx.y * kT;
    int e, i0, i1, r0 = 0, r1 = g.NR;
    if (g.by_rows) {
        if (threadIdx.x < 32) {
            int te = 0, lo = 0, hi = 0;
            if (!g.offsets) te = 0, lo = min(static_cast<int>(blockIdx.x) * kT, g.S), hi = g.S;
            else if (!warp_find_tile(g.offsets, g.E, g.S, kT, blockIdx.x, te, lo, hi)) lo = hi = 0;
            if (threadIdx.x == 0) s_e = te, s_lo = lo, s_hi = hi;
        }
        __syncthreads();
        e = s_e, i0 = s_lo, i1 = min(s_hi, s_lo + kT);
        if (i0 >= i1) return;
        if (e == g.E) r1 = 0;  // rows past the last expert's: zeros
    } else {
        e = blockIdx.z;
        expert_rows(g.offsets, e, g.S, r0, r1);
        i0 = blockIdx.x * kT, i1 = min(g.NI, i0 + kT);
    }
    const int nj = min(g.NJ - j0, kT);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4], up[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = up[a][b] = 0.f;
    const V* Re = R + (g.by_rows && e < g.E ? e * g.re : 0);
    for (int r = r0; r < r1; r += kR) {
        stage<V>(sl, L + i0 * g.li + r * g.lr, g.li, g.lr, i1 - i0, r1 - r);
        stage<V>(sr[0], Re + j0 * g.rj + r * g.rr, g.rj, g.rr, nj, r1 - r);
        if constexpr (EPI == kGate) stage<V>(sr[1], Re + (static_cast<long long>(g.NJ) + j0) * g.rj + r * g.rr, g.rj, g.rr, nj, r1 - r);
        __syncthreads();
#pragma unroll 8
        for (int q = 0; q < kR; ++q) {
            float x[4], y[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) x[a] = sl[q][ty + 16 * a], y[a] = sr[0][q][tx + 16 * a];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] += x[a] * y[b];
            if constexpr (EPI == kGate) {
#pragma unroll
                for (int a = 0; a < 4; ++a) y[a] = sr[1][q][tx + 16 * a];
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b) up[a][b] += x[a] * y[b];
            }
        }
        __syncthreads();
    }
    O* Ce = C + (g.by_rows ? 0 : e * g.ce);
    auto put = [&](auto kind) {
        constexpr int ACT = decltype(kind)::value;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int i = i0 + ty + 16 * a;
            if (i >= i1) continue;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int j = tx + 16 * b;
                if (j >= nj) continue;
                O* c = Ce + i * g.ldc + j0 + j;
                if constexpr (EPI == kNone) {
                    *c = from_f<O>(acc[a][b]);
                } else if constexpr (EPI == kGate) {
                    *c = from_f<O>(e < g.E ? act_of<ACT>(make_float2(acc[a][b], 0.f)).x * up[a][b] : 0.f);
                    if (gate.H) {
                        V* h = static_cast<V*>(gate.H) + i * gate.ldh + j0 + j;
                        h[0] = from_f<V>(acc[a][b]);
                        h[g.NJ] = from_f<V>(up[a][b]);
                    }
                } else {
                    const V* h = behind_wait(static_cast<const V*>(gate.H)) + i * gate.ldh + j0 + j;
                    float dg = 0.f, du = 0.f, out = 0.f;
                    if (e < g.E) {  // rows past the last expert's are zeros, whatever H holds there
                        const float u = to_f(load(h + g.NJ));
                        float2 slope;
                        const float act = act_of<ACT>(make_float2(to_f(load(h)), 0.f), slope).x;
                        dg = acc[a][b] * u * slope.x, du = acc[a][b] * act, out = act * u;
                    }
                    V* d = static_cast<V*>(gate.dH) + i * gate.lddh + j0 + j;
                    d[0] = from_f<V>(dg);
                    d[g.NJ] = from_f<V>(du);
                    if (g.C) *c = from_f<O>(out);
                }
            }
        }
    };
    if constexpr (EPI == kNone) put(std::integral_constant<int, 0>{});
    else with_act(gate.act, put);
}

template <class V, int EPI>
spx_status launch(const SimtGemm& g, const Gate& gate, spx_type c_type, cudaStream_t st) {
    dim3 grid;
    if (g.by_rows) {
        grid = dim3(static_cast<unsigned>(max_row_tiles(g.E, g.S, kT)), (g.NJ + kT - 1) / kT);
    } else {
        grid = dim3((g.NI + kT - 1) / kT, (g.NJ + kT - 1) / kT, g.E);
    }
    if (grid.y > 65535) return SPX_ERR_UNSUPPORTED;
    spx_note_launches(1);
    auto kernel = experts_simt_kernel<V, V, EPI>;  // what is stored has the factors' type or, but for the gate's gradient, fp32
    if constexpr (EPI != kGateGrad)
        if (c_type == SPX_F32) kernel = experts_simt_kernel<V, float, EPI>;
    return spx_cuda_status(launch_early(kernel, grid, kThreads, 0, 1, st, g, gate));
}

}  // namespace

int spx_experts_simt_check_take() { return spx_check_take(g_experts_check); }

namespace spx_exp {

spx_status simt_gemm(const SimtGemm& g, spx_type type, spx_type c_type, cudaStream_t st) {
    if (type == SPX_BF16) return launch<__nv_bfloat16, kNone>(g, Gate{}, c_type, st);
    return launch<__half, kNone>(g, Gate{}, c_type, st);
}

spx_status simt_gated(const SimtGemm& g, const Gate& gate, spx_type type, spx_type c_type, cudaStream_t st) {
    if (gate.epi == kGate) return type == SPX_BF16 ? launch<__nv_bfloat16, kGate>(g, gate, c_type, st) : launch<__half, kGate>(g, gate, c_type, st);
    return type == SPX_BF16 ? launch<__nv_bfloat16, kGateGrad>(g, gate, c_type, st) : launch<__half, kGateGrad>(g, gate, c_type, st);
}

}  // namespace spx_exp
