// spx_norm.cu -- root-mean-square norm of rows with the residual's addition, in
// the rows' type or as 8-bit codes with a scale a row, and its gradients.
//
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//   d s = rstd (dy w) - s rstd^3 mean(dy w s) + dS,  d w = sum over rows of dy s rstd
//
// Every row is read once and stays in registers (the gradient: in shared
// memory), 16 or 32 values a thread, between the sum over it and what is written
// from it, so both are bound by HBM: 16384 x 4096 bf16 with a residual 80 us, 6.7
// TB/s, the gradient 88 us, 6.1 TB/s (copies run at 6.8).  Few rows are bound by
// the latency of one load, one sum and one store: a row of 4096 2.2 us, its
// launch included.  Rows off 16-byte boundaries are bound by their instructions:
// 4-byte pieces of 4094 values 97 us (gradient 136), shifted words of 4095 161
// (186); fp32 rows go in 4-byte pieces, in the gradient those over 8192 values in
// shifted words.  The gradient of rows over 8192 values runs on 1024 threads of 64
// registers and spills 100 to 770 bytes a thread (4096 x 16384 bf16 142 us for 79
// of HBM), the norm over 16384 values 24 to 104, in fp32 pieces of one value 530.
#include <algorithm>
#include <type_traits>

#include "spx_rows.cuh"
#include "spx_tc.cuh"

using namespace spx_rows;

namespace {

// Values of a row that a thread holds; twice as many where that pays (norm_launch) and for rows longer than a CTA's threads
// hold so.
constexpr int kHeld = 16;
constexpr int kThreads = 256, kMostThreads = 1024;

struct NormArgs {
    int M, H, log_g;  // rows, their length, log2 of the threads a row
    long long ldx, ldr, lds, ldy;
    const void *X, *R, *w;
    void *S, *Y;
    float *scale, *rstd;
    float eps;
    bool wide_w;  // the weights are fp32
};

// 4 to 1024 threads take a row and keep 16 or 32 of its values each in registers; a sum over them crosses lanes
// by shuffles and warps by shared memory.  Sums of squares are fp32, at most 32 a thread in two chains, then pairwise.  8-bit
// output: the row's quotients y / scale as codes (ties to even); a row that holds an infinity or NaN has codes 0.  What is
// done for each code bounds it where there is no residual to read (16384 x 4096 bf16: 58 us for 30 of HBM; with one 79 for
// 69).
template <class V, class O, int N, bool ANY, int HELD, int MAXT>
__global__ void __launch_bounds__(MAXT, ANY || MAXT > kThreads || HELD > kHeld ? 1024 / MAXT : 5) rms_norm_kernel(NormArgs a) {
    constexpr int P = HELD / N, X = (N + 1) / 2;
    using Piece = Pack<V, N>;
    __shared__ __align__(16) float s_sum[MAXT / 32];
    __shared__ uint32_t s_max[MAXT / 32];
    let_next_start();
    wait_for_previous();
    const Rows<V, N, ANY> rows{a.H};
    const int G = 1 << a.log_g, at = threadIdx.x & (G - 1), np = rows.pieces();
    const int row = blockIdx.x * (blockDim.x >> a.log_g) + (threadIdx.x >> a.log_g);
    const bool live = row < a.M, left = at > 0 && (threadIdx.x & 31) > 0;
    const V *x = behind_wait(static_cast<const V*>(a.X)), *r = behind_wait(static_cast<const V*>(a.R));
    const void* w = behind_wait(a.w);
    Floats<N> s[P];
    {
        Piece px[P], pr[P];
        const V *xr = x + row * a.ldx, *rr = r + row * a.ldr;
        if (live && rows.inside(xr, x, x + (a.M - 1) * a.ldx + a.H) && (!a.R || rows.inside(rr, r, r + (a.M - 1) * a.ldr + a.H))) {
#pragma unroll
            for (int h = 0; h < P; ++h) {
                if (h * G >= np) break;
                px[h] = rows.read(xr, at + h * G);
                if (a.R) pr[h] = rows.read(rr, at + h * G);
            }
        } else if (ANY && live) {
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (at + h * G < np) {
                    px[h] = rows.read_edge(xr, at + h * G);
                    if (a.R) pr[h] = rows.read_edge(rr, at + h * G);
                }
        }
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const bool on = live && at + h * G < np;
            const Floats<N> f = floats(px[h]), g = floats(pr[h]);
#pragma unroll
            for (int i = 0; i < X; ++i) s[h].v[i] = !on ? make_float2(0.f, 0.f) : a.R ? __fadd2_rn(f.v[i], g.v[i]) : f.v[i];
        }
    }
    float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int h = 0; h < P; ++h)
#pragma unroll
        for (int i = 0; i < X; ++i) sum2 = __ffma2_rn(s[h].v[i], s[h].v[i], sum2);
    if (a.S) {
        V* out = static_cast<V*>(a.S) + row * a.lds;
#pragma unroll
        for (int h = 0; h < P; ++h) rows.write(out, at + h * G, packed<V, N>(s[h]), live, left);
    }
    const float sum = group_sum(sum2.x + sum2.y, G, s_sum);
    const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
    if (a.rstd && live && at == 0) a.rstd[row] = rstd;
    const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int h = 0; h < P; ++h) {
        if (at + h * G >= np) break;
        Floats<N> f;
        if (a.w) f = rows.weights(w, a.wide_w, at + h * G);
#pragma unroll
        for (int i = 0; i < X; ++i) {
            s[h].v[i] = __fmul2_rn(s[h].v[i], r2);
            if (a.w) s[h].v[i] = __fmul2_rn(s[h].v[i], f.v[i]);
        }
    }
    O* y = static_cast<O*>(a.Y) + row * a.ldy;
    if constexpr (sizeof(O) == 1) {
        uint32_t m = 0;  // the bits of an infinity or NaN are above every number's
#pragma unroll
        for (int h = 0; h < P; ++h)
#pragma unroll
            for (int i = 0; i < X; ++i) m = max(m, max(__float_as_uint(s[h].v[i].x) & 0x7fffffffu, __float_as_uint(s[h].v[i].y) & 0x7fffffffu));
        m = group_max(m, G, s_max);
        const bool fine = m < 0x7f800000u;
        const float q = __uint_as_float(m) / 127.f;
        if (live && at == 0) a.scale[row] = fine ? q : __int_as_float(0x7fffffff);
        // The quotient from the rounded reciprocal: a first one, its exact remainder, and a correction that rounds it
        // correctly (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
        // Subnormal scales, whose reciprocal may not exist, divide; they are coarse, so the quotient may pass 127.
        const bool plain = fine && q >= 1e-30f;
        const float inv = plain ? 1.f / q : 0.f;
        constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
        const float2 inv2 = make_float2(inv, inv), q2 = make_float2(-q, -q), whole = make_float2(kWhole, kWhole);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            uint32_t t[2 * X];
#pragma unroll
            for (int i = 0; i < X; ++i) {
                const float2 v = s[h].v[i], q0 = __fmul2_rn(v, inv2), c = __fadd2_rn(__ffma2_rn(__ffma2_rn(q0, q2, v), inv2, q0), whole);
                t[2 * i] = __float_as_uint(c.x), t[2 * i + 1] = __float_as_uint(c.y);
            }
            if (!plain) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float v = i & 1 ? s[h].v[i / 2].y : s[h].v[i / 2].x;
                    t[i] = fine && q > 0.f ? static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(v / q), -127.f), 127.f))) : 0u;
                }
            }
            Pack<O, N> p;
            if constexpr (N >= 4) {
                uint32_t word[N / 4];
#pragma unroll
                for (int i = 0; i < N / 4; ++i)
                    word[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x0040), __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040), 0x5410);
                memcpy(&p, word, N);
            } else {
                int8_t c[N];
#pragma unroll
                for (int i = 0; i < N; ++i) c[i] = static_cast<int8_t>(t[i]);
                p.set(c);
            }
            rows.write(y, at + h * G, p, live, left);
        }
    } else {
#pragma unroll
        for (int h = 0; h < P; ++h) rows.write(y, at + h * G, packed<V, N>(s[h]), live, left);
    }
}

// ---------------------------------------------------------------- gradient

// A group of threads takes a row, each with columns of its own whose d w it sums over its rows.  A thread copies the
// pieces it is going to need asynchronously into its own slots of shared memory, DEPTH rows ahead: it waits for nobody
// else's copies, and they hold no registers.  That is three rows deep for 16-bit rows that need no shifting (up to 8192
// values; two up to 16384), two for those that do and for fp32 rows over 4096 values.  fp32 rows up to 4096 have room for one, whose copies
// are in flight beside the other blocks' rows (8192 x 4096 fp32 88 us, 90% of the copy rate, as bf16); rows in 4-byte pieces
// spill 72 bytes a thread there.  Between the two looks at a row -- the sum of dy w s, then what is written --
// only that sum crosses threads.  As many blocks as the SMs hold at once, three an SM, so that few rows of sums are left to
// add (add_parts_kernel).  16384 x 4096 bf16: 94 us with a row's pieces in a thread's slots three deep (118 with tiles of
// rows that a block waits for together; 235 with nothing ahead), 88 with the sums written in whole lines.
struct GradArgs {
    int M, H, log_g;
    long long lddy, lds, lddr, lddx;
    const void *dY, *S, *w, *dR;
    const float* rstd;
    void* dX;
    float* part;  // [blocks][H] sums of the weights' gradient, or the gradient itself with one block; NULL: not wanted
    bool wide_w;  // the weights are fp32
};

// A block's sums leave through shared memory, in whole lines: each thread's own pieces straight to memory, N values in N
// stores, cost 4 us at 4096 values a row (1237 rows of bf16 15.5 us and 11.3).  The last piece of a row of any width may pass its
// end (kSlack).
constexpr int kSlack = 8;
template <int N>
__device__ __forceinline__ void keep_sums(float* to, const Floats<N>& f, bool add) {
    constexpr int Q = N < 4 ? N : 4, X = (Q + 1) / 2;
    Pack<float, Q>* q = reinterpret_cast<Pack<float, Q>*>(to);
#pragma unroll
    for (int i = 0; i < N / Q; ++i) {
        Floats<Q> v;
        if (add) v = floats(read_piece(q + i));
#pragma unroll
        for (int j = 0; j < X; ++j) v.v[j] = add ? __fadd2_rn(v.v[j], f.v[X * i + j]) : f.v[X * i + j];
        write_piece(q + i, packed<float, Q>(v));
    }
}
__device__ __forceinline__ void write_sums(const GradArgs& a, const float* sums) {
    float* part = a.part + static_cast<long long>(blockIdx.x) * a.H;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) part[c] = sums[c];
}

// Rows off 16-byte boundaries (ANY) bring both words around each piece.  DEPTH 0 (rows that leave no room): loaded where
// they are needed.
template <class V, int N, bool ANY, int MAXT, int DEPTH>
__global__ void __launch_bounds__(MAXT, MAXT > kThreads ? 1 : ANY ? 2 : 3) rms_norm_grad_kernel(GradArgs a) {
    constexpr int P = kHeld / N, X = (N + 1) / 2;
    using Piece = Pack<V, N>;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(16) float s_sum[2][MAXT / 32];
    let_next_start();
    wait_for_previous();
    const Rows<V, N, ANY> rows{a.H};
    const int G = 1 << a.log_g, at = threadIdx.x & (G - 1), np = rows.pieces();
    const bool left = at > 0 && (threadIdx.x & 31) > 0;
    const int groups = blockDim.x >> a.log_g, mine = threadIdx.x >> a.log_g, step = gridDim.x * groups;
    const V *dY = behind_wait(static_cast<const V*>(a.dY)), *S = behind_wait(static_cast<const V*>(a.S));
    const V* dR = behind_wait(static_cast<const V*>(a.dR));
    const float* rs = behind_wait(a.rstd);
    const void* w = behind_wait(a.w);
    const float over = -1.f / static_cast<float>(a.H);
    // slot h of array x of stage d: a piece a thread
    constexpr int E = ANY ? 2 : 1;  // words a piece
    Piece* slots = reinterpret_cast<Piece*>(sm) + threadIdx.x;
    auto slot = [&](int d, int x, int h) { return slots + ((d * 3 + x) * P + h) * E * static_cast<int>(DEPTH > 0 ? MAXT : 0); };
    const V *dY1 = dY + (a.M - 1) * a.lddy + a.H, *S1 = S + (a.M - 1) * a.lds + a.H, *dR1 = dR + (a.M - 1) * a.lddr + a.H;
    int row = blockIdx.x * groups + mine, ahead = row;
    const V *g = dY + row * a.lddy, *s = S + row * a.lds, *r = dR + row * a.lddr;  // row `ahead` of each
    const long long dg = step * a.lddy, ds = step * a.lds, dr = step * a.lddr;
    auto ahead_one = [&]() { ahead += step, g += dg, s += ds, r += dr; };
    auto copy = [&](int d, int x, const V* from, const V* lo, const V* hi) {
        if (rows.inside(from, lo, hi)) {
            const Piece* q = reinterpret_cast<const Piece*>(reinterpret_cast<uintptr_t>(from) & ~static_cast<uintptr_t>(15)) + at;
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (at + h * G < np) {
                    copy_near(slot(d, x, h), q + h * G);
                    copy_near(slot(d, x, h) + MAXT, q + h * G + 1);
                }
        } else {
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (at + h * G < np) write_piece(slot(d, x, h), rows.read_edge(from, at + h * G));
        }
    };
    auto take = [&](int d, int x, int h, int m) {  // m: bytes that the row lies off a boundary
        const Piece p = read_piece(slot(d, x, h));
        if constexpr (!ANY) return p;
        else return rows.join(p, m ? read_piece(slot(d, x, h) + MAXT) : p, m, at + h * G);
    };
    auto off = [&](int row, const V* base, long long ld, const V* hi) {
        const V* p = base + row * ld;
        return ANY && rows.inside(p, base, hi) ? static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) : 0;
    };
    auto fetch = [&](int d) {
        if (ahead < a.M) {
            if constexpr (!ANY) {
#pragma unroll
                for (int h = 0; h < P; ++h)
                    if (at + h * G < np) {
                        copy_piece(slot(d, 0, h), reinterpret_cast<const Piece*>(g) + at + h * G);
                        copy_piece(slot(d, 1, h), reinterpret_cast<const Piece*>(s) + at + h * G);
                        if (a.dR) copy_piece(slot(d, 2, h), reinterpret_cast<const Piece*>(r) + at + h * G);
                    }
            } else {
                copy(d, 0, g, dY, dY1);
                copy(d, 1, s, S, S1);
                if (a.dR) copy(d, 2, r, dR, dR1);
            }
        }
        ahead_one();
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (DEPTH > 0)
#pragma unroll
        for (int i = 0; i < DEPTH - 1; ++i) fetch(i);
    Floats<N> wf[P], acc[P];
#pragma unroll
    for (int h = 0; h < P; ++h) {
#pragma unroll
        for (int i = 0; i < X; ++i) acc[h].v[i] = make_float2(0.f, 0.f), wf[h].v[i] = make_float2(1.f, 1.f);
        if (a.w && at + h * G < np) wf[h] = rows.weights(w, a.wide_w, at + h * G);
    }
    V* dx = static_cast<V*>(a.dX) + row * a.lddx;
    int d = 0, turn = 0;
    for (int r0 = blockIdx.x * groups; r0 < a.M; r0 += step, row += step, turn ^= 1) {
        const bool live = row < a.M;
        const float rstd = live ? load(rs + row) : 0.f;
        const float2 r2 = make_float2(rstd, rstd);
        Piece pg[P], ps[P], pr[P];
        if constexpr (DEPTH > 0) {
            fetch(d == 0 ? DEPTH - 1 : d - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        } else if (live && rows.inside(g, dY, dY1) && rows.inside(s, S, S1) && (!a.dR || rows.inside(r, dR, dR1))) {
#pragma unroll
            for (int h = 0; h < P; ++h) {
                if (h * G >= np) break;
                pg[h] = rows.read(g, at + h * G), ps[h] = rows.read(s, at + h * G);
                if (a.dR) pr[h] = rows.read(r, at + h * G);
            }
        } else if (ANY && live) {
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (at + h * G < np) {
                    pg[h] = rows.read_edge(g, at + h * G), ps[h] = rows.read_edge(s, at + h * G);
                    if (a.dR) pr[h] = rows.read_edge(r, at + h * G);
                }
        }
        const int mg = DEPTH > 0 ? off(row, dY, a.lddy, dY1) : 0, ms = DEPTH > 0 ? off(row, S, a.lds, S1) : 0;
        float2 dot2 = make_float2(0.f, 0.f);
        if (live) {
#pragma unroll
            for (int h = 0; h < P; ++h) {
                if (at + h * G >= np) break;
                if constexpr (DEPTH > 0) pg[h] = take(d, 0, h, mg), ps[h] = take(d, 1, h, ms);
                const Floats<N> x = floats(pg[h]), y = floats(ps[h]);
#pragma unroll
                for (int i = 0; i < X; ++i) {
                    const float2 b = __fmul2_rn(x.v[i], __fmul2_rn(y.v[i], r2));
                    acc[h].v[i] = __fadd2_rn(acc[h].v[i], b);
                    dot2 = __ffma2_rn(b, wf[h].v[i], dot2);
                }
            }
        }
        const float dot = group_sum(dot2.x + dot2.y, G, s_sum[turn]) * over;
        const float2 c2 = make_float2(dot, dot);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const bool on = live && at + h * G < np;
            if (!ANY && !on) continue;
            if constexpr (DEPTH > 0) {  // once more, sooner than held across the sum
                pg[h] = take(d, 0, h, mg), ps[h] = take(d, 1, h, ms);
                if (a.dR) pr[h] = take(d, 2, h, off(row, dR, a.lddr, dR1));
            }
            const Floats<N> x = floats(pg[h]), y = floats(ps[h]);
            Floats<N> z, o;
            if (a.dR) z = floats(pr[h]);
#pragma unroll
            for (int i = 0; i < X; ++i) {
                const float2 v = __ffma2_rn(__fmul2_rn(y.v[i], r2), c2, __fmul2_rn(x.v[i], wf[h].v[i]));
                o.v[i] = a.dR ? __ffma2_rn(v, r2, z.v[i]) : __fmul2_rn(v, r2);
            }
            rows.write(dx, at + h * G, packed<V, N>(o), on, left);
        }
        dx += step * a.lddx;
        if constexpr (DEPTH > 0) d = d == DEPTH - 1 ? 0 : d + 1;
        else ahead_one();
    }
    if (DEPTH > 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.part) return;
    float* sums = reinterpret_cast<float*>(sm);  // where the pieces were
    __syncthreads();
    for (int m = 0; m < groups; ++m) {  // in the groups' order
        if (mine == m)
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (at + h * G < np) keep_sums(sums + (at + h * G) * N, acc[h], m > 0);
        __syncthreads();
    }
    write_sums(a, sums);
}

// Rows longer than a block's threads hold so: a block a row, read twice, the second time from L2.  One row an SM in flight,
// nothing ahead, and the running sums spill (352 bytes of bf16, 548 off boundaries): 2048 x 20000 bf16 130 us for 48 of HBM.
constexpr int kLongValues = 32;
template <class V, int N, bool ANY>
__global__ void __launch_bounds__(kMostThreads, 1) rms_norm_grad_long_kernel(GradArgs a) {
    constexpr int K = kLongValues / N, X = (N + 1) / 2;
    extern __shared__ __align__(16) float sums[];
    __shared__ __align__(16) float s_sum[2][kMostThreads / 32];
    let_next_start();
    wait_for_previous();
    const Rows<V, N, ANY> rows{a.H};
    const int np = rows.pieces();
    const V *dY = behind_wait(static_cast<const V*>(a.dY)), *S = behind_wait(static_cast<const V*>(a.S));
    const V* dR = behind_wait(static_cast<const V*>(a.dR));
    const float* rs = behind_wait(a.rstd);
    const void* w = behind_wait(a.w);
    const V *dY1 = dY + (a.M - 1) * a.lddy + a.H, *S1 = S + (a.M - 1) * a.lds + a.H, *dR1 = dR + (a.M - 1) * a.lddr + a.H;
    Floats<N> acc[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < X; ++i) acc[k].v[i] = make_float2(0.f, 0.f);
    int turn = 0;
    for (int row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const V *g = dY + row * a.lddy, *s = S + row * a.lds, *r = dR + row * a.lddr;
        V* out = static_cast<V*>(a.dX) + row * a.lddx;
        const bool in = rows.inside(g, dY, dY1) && rows.inside(s, S, S1) && (!a.dR || rows.inside(r, dR, dR1));
        const float rstd = load(rs + row);
        float2 dot2 = make_float2(0.f, 0.f);
        const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = threadIdx.x + k * kMostThreads;
            if (p >= np) break;
            const Floats<N> u = floats(in ? rows.read(g, p) : rows.read_edge(g, p)), v = floats(in ? rows.read(s, p) : rows.read_edge(s, p));
            Floats<N> f;
            if (a.w) f = rows.weights(w, a.wide_w, p);
#pragma unroll
            for (int i = 0; i < X; ++i) {
                const float2 n = __fmul2_rn(v.v[i], r2);
                acc[k].v[i] = __ffma2_rn(u.v[i], n, acc[k].v[i]);
                dot2 = __ffma2_rn(a.w ? __fmul2_rn(u.v[i], f.v[i]) : u.v[i], n, dot2);
            }
        }
        const float dot = group_sum(dot2.x + dot2.y, kMostThreads, s_sum[turn]) / -static_cast<float>(a.H);
#pragma unroll 2
        for (int p0 = 0; p0 < np; p0 += kMostThreads) {
            const int p = p0 + threadIdx.x;
            const bool on = p < np;
            Floats<N> u, v, z, f, o;
            if (on) {
                u = floats(in ? rows.read(g, p) : rows.read_edge(g, p)), v = floats(in ? rows.read(s, p) : rows.read_edge(s, p));
                if (a.dR) z = floats(in ? rows.read(r, p) : rows.read_edge(r, p));
                if (a.w) f = rows.weights(w, a.wide_w, p);
            }
#pragma unroll
            for (int i = 0; i < X; ++i) {
                const float2 e = __ffma2_rn(__fmul2_rn(v.v[i], r2), make_float2(dot, dot), a.w ? __fmul2_rn(u.v[i], f.v[i]) : u.v[i]);
                o.v[i] = a.dR ? __ffma2_rn(e, r2, z.v[i]) : __fmul2_rn(e, r2);
            }
            rows.write(out, p, packed<V, N>(o), on, (threadIdx.x & 31) > 0);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (threadIdx.x + k * kMostThreads < np) keep_sums(sums + (threadIdx.x + k * kMostThreads) * N, acc[k], false);
    __syncthreads();
    write_sums(a, sums);
}

// dw[c] = the blocks' sums, in their order within each of 32 shares.  Bound by two rounds of loads from L2 behind the first
// kernel's end: 456 rows of 4096 in about 3 us of the 88.
constexpr int kAddThreads = 1024;
__global__ void __launch_bounds__(kAddThreads) add_parts_kernel(int H, int blocks, const float* part, float* dw) {
    __shared__ float s[kAddThreads / 32][32];
    let_next_start();
    wait_for_previous();
    part = behind_wait(part);
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    constexpr int kAhead = 8;  // loads in flight, also where there are fewer left: past the end the last again, not added
    const float* q = part + min(c, H - 1);
    float sum = 0.f;
    for (int b0 = w; b0 < blocks; b0 += kAhead * (kAddThreads / 32)) {
        float x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = load(q + static_cast<long long>(min(b0 + i * (kAddThreads / 32), blocks - 1)) * H);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) sum += b0 + i * (kAddThreads / 32) < blocks ? x[i] : 0.f;
    }
    s[w][threadIdx.x & 31] = sum;
    __syncthreads();
    if (w || c >= H) return;
#pragma unroll
    for (int i = 1; i < kAddThreads / 32; ++i) sum += s[i][threadIdx.x];
    dw[c] = sum;
}

// ---------------------------------------------------------------- host side

// log2 of the threads a row: enough that its values fit their registers, and where there are few rows so many that a thread
// waits for at most two pieces (1 x 1002 bf16 3.4 us with as many as needed and 2.2, 512 x 1001 fp32 9.6 and 5.9; with one
// piece a thread 512 x 2048 bf16 takes 3.2 us for 2.9), of rows off their boundaries for one (1000 x 1001 bf16 5.9 and 5.0).
// Larger blocks only where every row has an SM (1 x 4095 fp32 7.9 and 5.1, but 512 x 1001 5.9 and 7.5).
int threads_log(int M, int H, int pieces, bool any) {
    int lg = 2;
    while ((kHeld << lg) < H && (1 << lg) < kMostThreads) ++lg;
    while ((any ? 1 : 2) << lg < pieces && (1 << lg) < (M <= 152 ? kMostThreads : kThreads) && (static_cast<long long>(M) << lg) < 152 * 1024) ++lg;
    return lg;
}

spx_status check(int32_t M, int32_t H, spx_type type, spx_type w_type) {
    if (M < 0 || H <= 0) return SPX_ERR_ARG;
    if (H > SPX_NORM_MAX_H) return SPX_ERR_UNSUPPORTED;
    if (M > kMostIndex) return SPX_ERR_INDEX_RANGE;
    if (!is_float_type(type) || (w_type != type && w_type != SPX_F32)) return SPX_ERR_ARG;
    return SPX_OK;
}

template <class V, class O, int N, bool ANY>
cudaError_t norm_launch(NormArgs a, cudaStream_t st) {
    if constexpr (sizeof(V) == 2 && N == 8 && !ANY) {
        // Where rows fill the SMs anyway, half the threads with twice the values each: what a thread does once a row weighs
        // less (16384 x 4096 bf16 to 8 bits 86 us and 79, without a residual 73 and 58, 8192 x 8192 bf16 87 and 81; fp32
        // and 4-byte pieces are faster with more threads).
        int lg = 2;
        while ((2 * kHeld << lg) < a.H) ++lg;
        if ((1 << lg) <= kThreads && static_cast<long long>(a.M) << lg >= 152 * 1024) {
            a.log_g = lg;
            const int per = kThreads >> lg;
            return launch_early(rms_norm_kernel<V, O, N, ANY, 2 * kHeld, kThreads>, dim3((a.M - 1) / per + 1), kThreads, 0, 1, st, a);
        }
    }
    a.log_g = threads_log(a.M, a.H, (a.H + N - 1) / N, ANY);
    const int threads = std::max(kThreads, 1 << a.log_g), per = threads >> a.log_g;
    const dim3 grid((a.M - 1) / per + 1);
    if (threads == kThreads) return launch_early(rms_norm_kernel<V, O, N, ANY, kHeld, kThreads>, grid, threads, 0, 1, st, a);
    return launch_early(a.H <= kHeld * kMostThreads ? rms_norm_kernel<V, O, N, ANY, kHeld, kMostThreads> : rms_norm_kernel<V, O, N, ANY, 2 * kHeld, kMostThreads>, grid,
                        threads, 0, 1, st, a);
}

// Rows of 16-byte pieces in every array (of codes: of as many bytes as a piece has values), else of 4-byte ones (fp32 rows
// always), else, 16-bit rows of odd widths or bases, shifted ones.  16384 x 4096 bf16 80 us, rows of 4094 96, of 4095 161.
template <class V, class O>
spx_status norm_pieces(const NormArgs& a, cudaStream_t st) {
    uint64_t bits = addr(a.X) | (static_cast<uint64_t>(a.H) | a.ldx) * sizeof(V);
    if (a.R) bits |= addr(a.R) | a.ldr * sizeof(V);
    if (a.S) bits |= addr(a.S) | a.lds * sizeof(V);
    bits |= (addr(a.Y) | a.ldy * sizeof(O)) * (sizeof(V) / sizeof(O));
    if (a.w) bits |= a.wide_w && sizeof(V) == 2 ? (addr(a.w) % 16 ? addr(a.w) / 2 : 0) : addr(a.w);
    spx_note_launches(1);
    if (bits % 16 == 0) return spx_cuda_status(norm_launch<V, O, 16 / sizeof(V), false>(a, st));
    if (bits % 4 == 0) return spx_cuda_status(norm_launch<V, O, 4 / sizeof(V), false>(a, st));
    if constexpr (sizeof(V) == 2) return spx_cuda_status(norm_launch<V, O, 8, true>(a, st));
    return SPX_ERR_ALIGN;
}

// Threads a row (log2), a block's threads, and the blocks of the gradient: as many as the SMs hold at once.
struct GradShape {
    int log_g, threads, blocks;
};
constexpr int kGradBlocks = 456, kLongRow = kHeld * kMostThreads;

GradShape grad_shape(int M, int H, bool any) {
    GradShape g{};
    g.log_g = 2;
    while ((kHeld << g.log_g) < H && (1 << g.log_g) < kMostThreads) ++g.log_g;
    g.threads = std::max(kThreads, 1 << g.log_g);
    const int per = g.threads >> g.log_g;
    g.blocks = std::min((M - 1) / per + 1, g.threads > kThreads ? kGradBlocks / 3 : any ? kGradBlocks / 3 * 2 : kGradBlocks);
    return g;
}

size_t sums_bytes(const GradArgs& a) { return a.part ? sizeof(float) * (static_cast<size_t>(a.H) + kSlack) : 0; }

template <class V, int N, bool ANY, int MAXT, int DEPTH>
cudaError_t grad_kernel(const GradArgs& a, const GradShape& g, cudaStream_t st) {
    constexpr size_t ring = static_cast<size_t>(DEPTH) * 3 * kHeld * sizeof(V) * MAXT * (ANY ? 2 : 1);
    const size_t smem = std::max(ring, sums_bytes(a));
    const cudaError_t e = spx_tc::set_smem_limit(rms_norm_grad_kernel<V, N, ANY, MAXT, DEPTH>, std::max(ring, sizeof(float) * (kHeld * MAXT + kSlack)));
    return e != cudaSuccess ? e : launch_early(rms_norm_grad_kernel<V, N, ANY, MAXT, DEPTH>, dim3(g.blocks), g.threads, smem, 1, st, a);
}

template <class V, int N, bool ANY>
spx_status grad_launch(GradArgs a, float* dw, cudaStream_t st) {
    const GradShape g = grad_shape(a.M, a.H, ANY);
    a.log_g = g.log_g;
    if (a.part && g.blocks == 1) a.part = dw;
    spx_note_launches(a.part && g.blocks > 1 ? 2 : 1);
    constexpr bool half = sizeof(V) == 2, shorter = half || !ANY, longer = half || N == 4;  // what grad_pieces gives these pieces
    cudaError_t e = cudaErrorInvalidValue;
    if (g.threads < kMostThreads) {
        if constexpr (shorter) {
            if (g.threads == kThreads) e = grad_kernel<V, N, ANY, kThreads, half ? (ANY ? 2 : 3) : 1>(a, g, st);
            else e = grad_kernel<V, N, ANY, 512, half && !ANY ? 3 : 2>(a, g, st);
        }
    } else if constexpr (longer) {
        if (a.H <= kLongRow) e = grad_kernel<V, N, ANY, kMostThreads, half && !ANY ? 2 : 0>(a, g, st);
        else if ((e = spx_tc::set_smem_limit(rms_norm_grad_long_kernel<V, N, ANY>, sizeof(float) * (SPX_NORM_MAX_H + kSlack))) == cudaSuccess)
            e = launch_early(rms_norm_grad_long_kernel<V, N, ANY>, dim3(g.blocks), kMostThreads, sums_bytes(a), 1, st, a);
    }
    if (e == cudaSuccess && a.part && g.blocks > 1)
        e = launch_early(add_parts_kernel, dim3((a.H + 31) / 32), kAddThreads, 0, 1, st, a.H, g.blocks, static_cast<const float*>(a.part), dw);
    return spx_cuda_status(e);
}

template <class V>
spx_status grad_pieces(const GradArgs& a, float* dw, cudaStream_t st) {
    uint64_t bits = addr(a.dY) | addr(a.S) | addr(a.dX) | (static_cast<uint64_t>(a.H) | a.lddy | a.lds | a.lddx) * sizeof(V);
    if (a.dR) bits |= addr(a.dR) | a.lddr * sizeof(V);
    if (a.w) bits |= a.wide_w && sizeof(V) == 2 ? (addr(a.w) % 16 ? addr(a.w) / 2 : 0) : addr(a.w);
    if (bits % 16 == 0) return grad_launch<V, 16 / sizeof(V), false>(a, dw, st);
    // fp32 rows longer than 512 threads hold: shifted 16-byte pieces (2000 x 16383 409 us in 4-byte pieces and 245; of 8191
    // values 128 and 175)
    if (sizeof(V) == 4 && a.H > kHeld * 512) return grad_launch<V, 16 / sizeof(V), true>(a, dw, st);
    if (bits % 4 == 0) return grad_launch<V, 4 / sizeof(V), false>(a, dw, st);
    if constexpr (sizeof(V) == 2) return grad_launch<V, 8, true>(a, dw, st);
    return SPX_ERR_ALIGN;
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
    return M > 1 ? sizeof(float) * static_cast<size_t>(grad_shape(M, H, false).blocks) * static_cast<size_t>(H) : 0;
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
