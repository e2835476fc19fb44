// spx_norm.cu -- root-mean-square norm of rows with the residual's addition, in
// the rows' type or as 8-bit codes with a scale a row, and its gradients.
//
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//   d s = rstd (dy w) - s rstd^3 mean(dy w s) + dS,  d w = sum over rows of dy s rstd
//
// Every row is read once and stays in registers, 16 values a thread, between
// the sum over it and what is written from it, so both kernels are bound by
// HBM.
#include <algorithm>
#include <type_traits>

#include "spx_rows.cuh"

using namespace spx_rows;

namespace {

// Values of a row that a thread holds; twice as many for rows longer than a CTA's threads hold so, at the cost of spills.
constexpr int kHeld = 16;

struct NormArgs {
    int M, H, log_g;  // rows, their length, log2 of the threads a row
    long long ldx, ldr, lds, ldy;
    const void *X, *R, *w;
    void *S, *Y;
    float *scale, *rstd;
    float eps;
    bool wide_w;  // the weights are fp32
};

// The row's quotients y / s as codes (ties to even); a row that holds an infinity or NaN has codes 0.
template <class V, class O, int N, int HELD, int MAXT>
__global__ void __launch_bounds__(MAXT, 1280 / MAXT) rms_norm_kernel(NormArgs a) {
    constexpr int P = HELD / N;
    using Piece = Pack<V, N>;
    __shared__ float s_sum[MAXT / 32];
    __shared__ uint32_t s_max[MAXT / 32];
    let_next_start();
    wait_for_previous();
    const int G = 1 << a.log_g, at = threadIdx.x & (G - 1), np = a.H / N;
    const int row = blockIdx.x * (blockDim.x >> a.log_g) + (threadIdx.x >> a.log_g);
    const bool live = row < a.M;
    const Piece* x = reinterpret_cast<const Piece*>(behind_wait(static_cast<const V*>(a.X)) + row * a.ldx);
    const Piece* r = reinterpret_cast<const Piece*>(behind_wait(static_cast<const V*>(a.R)) + row * a.ldr);
    const void* w = behind_wait(a.w);
    float s[P][N];
    {
        Piece px[P], pr[P];
#pragma unroll
        for (int h = 0; h < P; ++h)
            if (live && at + h * G < np) {
                px[h] = load_once(x + at + h * G);
                if (a.R) pr[h] = load_once(r + at + h * G);
            }
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const bool on = live && at + h * G < np;
#pragma unroll
            for (int i = 0; i < N; ++i) s[h][i] = !on ? 0.f : a.R ? to_f(px[h].v[i]) + to_f(pr[h].v[i]) : to_f(px[h].v[i]);
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < P; ++h)
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(s[h][i], s[h][i], sum);
    if (a.S && live) {
        Piece* out = reinterpret_cast<Piece*>(static_cast<V*>(a.S) + row * a.lds);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            Piece p;
#pragma unroll
            for (int i = 0; i < N; ++i) p.v[i] = from_f<V>(s[h][i]);
            write_piece(out + at + h * G, p);
        }
    }
    sum = group_sum(sum, G, s_sum);
    const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
    if (a.rstd && live && at == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int h = 0; h < P; ++h) {
        if (at + h * G >= np) break;
        float f[N];
        if (a.w) load_floats<V, N>(w, a.wide_w, static_cast<long long>(at + h * G) * N, f);
#pragma unroll
        for (int i = 0; i < N; ++i) s[h][i] = s[h][i] * rstd * (a.w ? f[i] : 1.f);
    }
    if constexpr (sizeof(O) == 1) {
        uint32_t m = 0;  // the bits of an infinity or NaN are above every number's
#pragma unroll
        for (int h = 0; h < P; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(s[h][i]) & 0x7fffffffu);
        m = group_max(m, G, s_max);
        const bool fine = m < 0x7f800000u;
        const float q = __uint_as_float(m) / 127.f;
        if (live && at == 0) a.scale[row] = fine ? q : __int_as_float(0x7fffffff);
        if (!live) return;
        Pack<O, N>* y = reinterpret_cast<Pack<O, N>*>(static_cast<O*>(a.Y) + row * a.ldy);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            Pack<O, N> p;
#pragma unroll
            for (int i = 0; i < N; ++i)  // subnormal scales are coarse: the quotient may pass 127
                p.v[i] = static_cast<int8_t>(fine && q > 0.f ? fminf(fmaxf(rintf(s[h][i] / q), -127.f), 127.f) : 0.f);
            write_piece(y + at + h * G, p);
        }
    } else {
        if (!live) return;
        Piece* y = reinterpret_cast<Piece*>(static_cast<V*>(a.Y) + row * a.ldy);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            Piece p;
#pragma unroll
            for (int i = 0; i < N; ++i) p.v[i] = from_f<V>(s[h][i]);
            write_piece(y + at + h * G, p);
        }
    }
}

struct GradArgs {
    int M, H, log_g;
    long long lddy, lds, lddr, lddx;
    const void *dY, *S, *w, *dR;
    const float* rstd;
    void* dX;
    float* part;  // [blocks][H] sums of the weights' gradient, or the gradient itself with one block; NULL: not wanted
    bool wide_w;
};

template <class V, int N, int HELD, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1) rms_norm_grad_kernel(GradArgs a) {
    constexpr int P = HELD / N;
    using Piece = Pack<V, N>;
    extern __shared__ float sm[];  // H sums, where a block has several groups
    __shared__ float s_sum[2][MAXT / 32];
    let_next_start();
    wait_for_previous();
    const int G = 1 << a.log_g, at = threadIdx.x & (G - 1), np = a.H / N;
    const int groups = blockDim.x >> a.log_g, mine = threadIdx.x >> a.log_g;
    const V *dY = behind_wait(static_cast<const V*>(a.dY)), *S = behind_wait(static_cast<const V*>(a.S));
    const V* dR = behind_wait(static_cast<const V*>(a.dR));
    const float* rs = behind_wait(a.rstd);
    const void* w = behind_wait(a.w);
    const float over = 1.f / static_cast<float>(a.H);
    float acc[P][N];
#pragma unroll
    for (int h = 0; h < P; ++h)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[h][i] = 0.f;
    int turn = 0;
    for (int r0 = blockIdx.x * groups; r0 < a.M; r0 += gridDim.x * groups, turn ^= 1) {
        const int row = r0 + mine;
        const bool live = row < a.M;
        const Piece *dy = reinterpret_cast<const Piece*>(dY + row * a.lddy), *s = reinterpret_cast<const Piece*>(S + row * a.lds);
        const Piece* dr = reinterpret_cast<const Piece*>(dR + row * a.lddr);
        Piece* dx = reinterpret_cast<Piece*>(static_cast<V*>(a.dX) + row * a.lddx);
        const float rstd = live ? load(rs + row) : 0.f;
        Piece pg[P], ps[P];
#pragma unroll
        for (int h = 0; h < P; ++h)
            if (live && at + h * G < np) {
                pg[h] = load_once(dy + at + h * G);
                ps[h] = load_once(s + at + h * G);
            }
        float dot = 0.f;
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (!live || at + h * G >= np) break;
            float f[N];
            if (a.w) load_floats<V, N>(w, a.wide_w, static_cast<long long>(at + h * G) * N, f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = to_f(pg[h].v[i]), n = to_f(ps[h].v[i]) * rstd;
                acc[h][i] = fmaf(g, n, acc[h][i]);
                dot = fmaf(a.w ? g * f[i] : g, n, dot);
            }
        }
        dot = group_sum(dot, G, s_sum[turn]) * over;
        if (!live) continue;
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            float f[N];
            if (a.w) load_floats<V, N>(w, a.wide_w, static_cast<long long>(at + h * G) * N, f);
            Piece pr, out;
            if (a.dR) pr = load_once(dr + at + h * G);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = to_f(pg[h].v[i]), n = to_f(ps[h].v[i]) * rstd;
                const float d = rstd * ((a.w ? g * f[i] : g) - n * dot);
                out.v[i] = from_f<V>(a.dR ? d + to_f(pr.v[i]) : d);
            }
            write_piece(dx + at + h * G, out);
        }
    }
    if (!a.part) return;
    float* part = a.part + static_cast<long long>(blockIdx.x) * a.H;
    if (groups == 1) {
#pragma unroll
        for (int h = 0; h < P; ++h)
            if (at + h * G < np)
#pragma unroll
                for (int i = 0; i < N; ++i) part[(at + h * G) * N + i] = acc[h][i];
        return;
    }
    for (int g = 0; g < groups; ++g) {  // in the groups' order
        if (mine == g)
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (at + h * G < np)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        float* to = sm + (at + h * G) * N + i;
                        *to = g == 0 ? acc[h][i] : *to + acc[h][i];
                    }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) part[c] = sm[c];
}

// dw[c] = the blocks' sums, in their order within each of eight shares.
constexpr int kAddThreads = 256;
__global__ void __launch_bounds__(kAddThreads) add_parts_kernel(int H, int blocks, const float* part, float* dw) {
    __shared__ float s[kAddThreads / 32][32];
    let_next_start();
    wait_for_previous();
    part = behind_wait(part);
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int b = w; b < blocks; b += kAddThreads / 32) sum += load(part + static_cast<long long>(b) * H + c);
    }
    s[w][threadIdx.x & 31] = sum;
    __syncthreads();
    if (w || c >= H) return;
#pragma unroll
    for (int i = 1; i < kAddThreads / 32; ++i) sum += s[i][threadIdx.x];
    dw[c] = sum;
}

// ---------------------------------------------------------------- host side

constexpr int kThreads = 256, kMostThreads = 1024, kMostBlocks = 608, kMostRows = 1 << 30;

// log2 of the threads a row: enough that its values fit their registers, and where there are few rows as many as it has
// pieces, since every thread then waits for one load instead of several.
int threads_log(int M, int H, int pieces) {
    int lg = 2;
    while ((kHeld << lg) < H && (1 << lg) < kMostThreads) ++lg;
    while ((1 << lg) < pieces && (1 << lg) < kThreads && (static_cast<long long>(M) << lg) < 152 * 1024) ++lg;
    return lg;
}

spx_status check(int32_t M, int32_t H, spx_type type, spx_type w_type) {
    if (M < 0 || H <= 0) return SPX_ERR_ARG;
    if (H > SPX_NORM_MAX_H) return SPX_ERR_UNSUPPORTED;
    if (M > kMostIndex) return SPX_ERR_INDEX_RANGE;
    if (!is_float_type(type) || (w_type != type && w_type != SPX_F32)) return SPX_ERR_ARG;
    return SPX_OK;
}

template <class V, class O, int N>
cudaError_t norm_launch(NormArgs a, cudaStream_t st) {
    a.log_g = threads_log(a.M, a.H, a.H / N);
    const int threads = std::max(kThreads, 1 << a.log_g), per = threads >> a.log_g;
    const dim3 grid((a.M + per - 1) / per);
    if (threads == kThreads) return launch_early(rms_norm_kernel<V, O, N, kHeld, kThreads>, grid, threads, 0, 1, st, a);
    return launch_early(a.H <= kHeld * kMostThreads ? rms_norm_kernel<V, O, N, kHeld, kMostThreads> : rms_norm_kernel<V, O, N, 2 * kHeld, kMostThreads>, grid,
                        threads, 0, 1, st, a);
}

// The widest pieces, up to 16 bytes, that every row is made of; an output in 8 bits takes as many bytes as a piece has values.
template <class V, class O>
spx_status norm_pieces(const NormArgs& a, cudaStream_t st) {
    constexpr bool codes = sizeof(O) == 1;
    uint64_t bits = addr(a.X) | (static_cast<uint64_t>(a.H) | a.ldx) * sizeof(V);
    if (a.R) bits |= addr(a.R) | a.ldr * sizeof(V);
    if (a.S) bits |= addr(a.S) | a.lds * sizeof(V);
    bits |= codes ? (addr(a.Y) | a.ldy) * sizeof(V) : addr(a.Y) | a.ldy * sizeof(V);
    if (a.w) bits |= a.wide_w && sizeof(V) == 2 ? (addr(a.w) % 16 ? addr(a.w) / 2 : 0) : addr(a.w);
    const int vb = copy_width(bits, sizeof(V));
    spx_note_launches(1);
    if (vb == 16) return spx_cuda_status(norm_launch<V, O, 16 / sizeof(V)>(a, st));
    if (sizeof(V) == 2 && vb >= 4) return spx_cuda_status(norm_launch<V, O, 4 / sizeof(V)>(a, st));
    return spx_cuda_status(norm_launch<V, O, 1>(a, st));
}

// Rows a block works on at once, its threads, and the blocks of the gradient.
struct GradShape {
    int log_g, threads, blocks;
};
GradShape grad_shape(int M, int H) {
    GradShape g{};
    g.log_g = threads_log(kMostRows, H, 0);
    g.threads = std::max(kThreads, 1 << g.log_g);
    const int per = g.threads >> g.log_g;
    g.blocks = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(M) + per - 1) / per, g.threads > kThreads ? kMostBlocks / 4 : kMostBlocks));
    return g;
}

template <class V, int N>
cudaError_t grad_launch(GradArgs a, float* dw, cudaStream_t st) {
    const GradShape g = grad_shape(a.M, a.H);
    a.log_g = g.log_g;
    if (a.part && g.blocks == 1) a.part = dw;
    const size_t smem = a.part && g.threads > 1 << g.log_g ? sizeof(float) * a.H : 0;
    cudaError_t e = launch_early(g.threads == kThreads                ? rms_norm_grad_kernel<V, N, kHeld, kThreads>
                                 : a.H <= kHeld * kMostThreads ? rms_norm_grad_kernel<V, N, kHeld, kMostThreads>
                                                               : rms_norm_grad_kernel<V, N, 2 * kHeld, kMostThreads>,
                                 dim3(g.blocks), g.threads, smem, 1, st, a);
    if (e == cudaSuccess && a.part && g.blocks > 1)
        e = launch_early(add_parts_kernel, dim3((a.H + 31) / 32), kAddThreads, 0, 1, st, a.H, g.blocks, static_cast<const float*>(a.part), dw);
    return e;
}

template <class V>
spx_status grad_pieces(const GradArgs& a, float* dw, cudaStream_t st) {
    uint64_t bits = addr(a.dY) | addr(a.S) | addr(a.dX) | (static_cast<uint64_t>(a.H) | a.lddy | a.lds | a.lddx) * sizeof(V);
    if (a.dR) bits |= addr(a.dR) | a.lddr * sizeof(V);
    if (a.w) bits |= a.wide_w && sizeof(V) == 2 ? (addr(a.w) % 16 ? addr(a.w) / 2 : 0) : addr(a.w);
    const int vb = copy_width(bits, sizeof(V));
    spx_note_launches(a.part && grad_shape(a.M, a.H).blocks > 1 ? 2 : 1);
    if (vb == 16) return spx_cuda_status(grad_launch<V, 16 / sizeof(V)>(a, dw, st));
    if (sizeof(V) == 2 && vb >= 4) return spx_cuda_status(grad_launch<V, 4 / sizeof(V)>(a, dw, st));
    return spx_cuda_status(grad_launch<V, 1>(a, dw, st));
}

template <class V, bool CODES>
using OutOf = typename std::conditional<CODES, int8_t, V>::type;

template <bool CODES>
spx_status norm_typed(spx_type type, const NormArgs& a, cudaStream_t st) {
    if (type == SPX_F32) return norm_pieces<float, OutOf<float, CODES>>(a, st);
    if (type == SPX_BF16) return norm_pieces<__nv_bfloat16, OutOf<__nv_bfloat16, CODES>>(a, st);
    return norm_pieces<__half, OutOf<__half, CODES>>(a, st);
}

}  // namespace

extern "C" {

spx_status spx_rms_norm(int32_t M, int32_t H, spx_type type, const void* X, int64_t ldx, const void* R, int64_t ldr,
                        const void* weight, spx_type w_type, float eps, void* S, int64_t lds, void* Y, int64_t ldy,
                        float* rstd, spx_stream_t stream) {
    const spx_status c = check(M, H, type, w_type);
    if (c != SPX_OK) return c;
    if (M == 0) return SPX_OK;
    if (!X || !Y || ldx < H || ldy < H || (R && ldr < H) || (S && lds < H) || !(eps >= 0.f)) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type);
    if (!spx_aligned(X, eb) || !spx_aligned(R, eb) || !spx_aligned(S, eb) || !spx_aligned(Y, eb) ||
        !spx_aligned(weight, type_bytes(w_type)) || !spx_aligned(rstd, 4))
        return SPX_ERR_ALIGN;
    NormArgs a{};
    a.M = M, a.H = H, a.ldx = ldx, a.ldr = ldr, a.lds = lds, a.ldy = ldy;
    a.X = X, a.R = R, a.w = weight, a.S = S, a.Y = Y, a.rstd = rstd, a.eps = eps, a.wide_w = w_type == SPX_F32;
    return norm_typed<false>(type, a, reinterpret_cast<cudaStream_t>(stream));
}

spx_status spx_rms_norm_i8(int32_t M, int32_t H, spx_type type, const void* X, int64_t ldx, const void* R, int64_t ldr,
                           const void* weight, spx_type w_type, float eps, void* S, int64_t lds, int8_t* Q, int64_t ldq,
                           float* scale, spx_stream_t stream) {
    const spx_status c = check(M, H, type, w_type);
    if (c != SPX_OK) return c;
    if (M == 0) return SPX_OK;
    if (!X || !Q || !scale || ldx < H || ldq < H || (R && ldr < H) || (S && lds < H) || !(eps >= 0.f)) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type);
    if (!spx_aligned(X, eb) || !spx_aligned(R, eb) || !spx_aligned(S, eb) || !spx_aligned(weight, type_bytes(w_type)) ||
        !spx_aligned(scale, 4))
        return SPX_ERR_ALIGN;
    NormArgs a{};
    a.M = M, a.H = H, a.ldx = ldx, a.ldr = ldr, a.lds = lds, a.ldy = ldq;
    a.X = X, a.R = R, a.w = weight, a.S = S, a.Y = Q, a.scale = scale, a.eps = eps, a.wide_w = w_type == SPX_F32;
    return norm_typed<true>(type, a, reinterpret_cast<cudaStream_t>(stream));
}

size_t spx_rms_norm_grad_scratch_bytes(int32_t M, int32_t H) {
    if (M <= 0 || H <= 0 || H > SPX_NORM_MAX_H || M > kMostIndex) return 0;
    const GradShape g = grad_shape(M, H);
    return g.blocks > 1 ? sizeof(float) * static_cast<size_t>(g.blocks) * static_cast<size_t>(H) : 0;
}

spx_status spx_rms_norm_grad(int32_t M, int32_t H, spx_type type, const void* dY, int64_t lddy, const void* S, int64_t lds,
                             const float* rstd, const void* weight, spx_type w_type, const void* dS, int64_t ldds, void* dX,
                             int64_t lddx, float* dweight, void* scratch, size_t scratch_bytes, spx_stream_t stream) {
    const spx_status c = check(M, H, type, w_type);
    if (c != SPX_OK) return c;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (!dweight) return SPX_OK;
        return spx_cuda_status(cudaMemsetAsync(dweight, 0, sizeof(float) * H, st));
    }
    if (!dY || !S || !rstd || !dX || lddy < H || lds < H || lddx < H || (dS && ldds < H)) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type), need = dweight ? spx_rms_norm_grad_scratch_bytes(M, H) : 0;
    if (need > 0 && (!scratch || scratch_bytes < need)) return SPX_ERR_ARG;
    if (!spx_aligned(dY, eb) || !spx_aligned(S, eb) || !spx_aligned(dS, eb) || !spx_aligned(dX, eb) ||
        !spx_aligned(rstd, 4) || !spx_aligned(weight, type_bytes(w_type)) || !spx_aligned(dweight, 4) ||
        (need > 0 && !spx_aligned(scratch, 4)))
        return SPX_ERR_ALIGN;
    GradArgs a{};
    a.M = M, a.H = H, a.lddy = lddy, a.lds = lds, a.lddr = ldds, a.lddx = lddx;
    a.dY = dY, a.S = S, a.rstd = rstd, a.w = weight, a.wide_w = w_type == SPX_F32, a.dR = dS, a.dX = dX;
    a.part = !dweight ? nullptr : need > 0 ? static_cast<float*>(scratch) : dweight;
    if (type == SPX_F32) return grad_pieces<float>(a, dweight, st);
    if (type == SPX_BF16) return grad_pieces<__nv_bfloat16>(a, dweight, st);
    return grad_pieces<__half>(a, dweight, st);
}

}  // extern "C"
