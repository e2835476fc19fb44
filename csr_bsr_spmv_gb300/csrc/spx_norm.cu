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
#include "spx_tc.cuh"

using namespace spx_rows;

namespace {

// Values of a row that a thread holds; twice as many for rows longer than a CTA's threads hold so, at the cost of spills.
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
    constexpr int X = (N + 1) / 2;
    Floats<N> s[P];
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
    if (a.S && live) {
        Piece* out = reinterpret_cast<Piece*>(static_cast<V*>(a.S) + row * a.lds);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            write_piece(out + at + h * G, packed<V, N>(s[h]));
        }
    }
    const float sum = group_sum(sum2.x + sum2.y, G, s_sum);
    const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
    if (a.rstd && live && at == 0) a.rstd[row] = rstd;
    const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int h = 0; h < P; ++h) {
        if (at + h * G >= np) break;
        Floats<N> f;
        if (a.w) f = load_floats<V, N>(w, a.wide_w, static_cast<long long>(at + h * G) * N);
#pragma unroll
        for (int i = 0; i < X; ++i) {
            s[h].v[i] = __fmul2_rn(s[h].v[i], r2);
            if (a.w) s[h].v[i] = __fmul2_rn(s[h].v[i], f.v[i]);
        }
    }
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
        if (!live) return;
        auto code = [&](float v) {  // subnormal scales are coarse: the quotient may pass 127
            return static_cast<int8_t>(fine && q > 0.f ? fminf(fmaxf(rintf(v / q), -127.f), 127.f) : 0.f);
        };
        Pack<O, N>* y = reinterpret_cast<Pack<O, N>*>(static_cast<O*>(a.Y) + row * a.ldy);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            Pack<O, N> p;
#pragma unroll
            for (int i = 0; i < N; ++i) p.v[i] = code(i & 1 ? s[h].v[i / 2].y : s[h].v[i / 2].x);
            write_piece(y + at + h * G, p);
        }
    } else {
        if (!live) return;
        Piece* y = reinterpret_cast<Piece*>(static_cast<V*>(a.Y) + row * a.ldy);
#pragma unroll
        for (int h = 0; h < P; ++h) {
            if (at + h * G >= np) break;
            write_piece(y + at + h * G, packed<V, N>(s[h]));
        }
    }
}

// ---------------------------------------------------------------- gradient

// A block takes a tile of R rows at a time into shared memory, the next tile's copies in flight beside it.  First each
// warp sums dy w s over stretches of rows, 16 values a lane; then each thread goes over the tile with columns of its own,
// writes d s and adds to its columns' d w.  The two ways through a tile keep what is done once a row -- the sums'
// shuffles, the barriers, the addresses -- small beside what is done once a value, which at eight values a load is what
// would bound it (a thread with its own columns for both, a row at a time: 48 instructions a value, 225 us for 16384 x
// 4096 bf16).
struct GradArgs {
    int M, H, R, tiles;
    int log_c;       // log2 of the columns of threads, kGradThreads at most: the others take other rows of the tile
    int log_l;       // log2 of the lanes that sum a stretch
    int segs, dots;  // stretches a row, and that rounded up to a multiple of four
    int pitch;       // bytes of a row in shared memory
    long long lddy, lds, lddr, lddx;
    const void *dY, *S, *w, *dR;
    const float* rstd;
    void* dX;
    float* part;  // [blocks][H] sums of the weights' gradient, or the gradient itself with one block; NULL: not wanted
    bool wide_w;  // the weights are fp32
};

constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32, kGradBlocks = 304, kStageBytes = 49152, kMostRows = 64;
constexpr int kLaneValues = 32;  // values a lane sums

// A piece from memory to shared memory, asynchronously where there is a copy of its size.
template <class P>
__device__ __forceinline__ void copy_piece(P* to, const P* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (sizeof(P) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else if constexpr (sizeof(P) >= 4) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(sizeof(P)) : "memory");
    else *to = load_once(from);
}

// HELD: values of a row that a thread holds sums for.
template <class V, int N, int HELD>
__global__ void __launch_bounds__(kGradThreads, 2) rms_norm_grad_kernel(GradArgs a) {
    constexpr int K = HELD / N, X = (N + 1) / 2;
    using Piece = Pack<V, N>;
    using Two = Floats<N>;
    extern __shared__ __align__(16) uint8_t sm[];
    let_next_start();
    wait_for_previous();
    const int np = a.H / N, arrays = a.dR ? 3 : 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const V *dY = behind_wait(static_cast<const V*>(a.dY)), *S = behind_wait(static_cast<const V*>(a.S));
    const V* dR = behind_wait(static_cast<const V*>(a.dR));
    const float* rs = behind_wait(a.rstd);
    const void* w = behind_wait(a.w);
    // two stages of R rows of each array, the weights as fp32, the stretches' sums of a tile, rstd of two tiles
    const int bytes = a.R * a.pitch, stage = arrays * bytes;
    float* sw = reinterpret_cast<float*>(sm + 2 * stage);
    float* dots = sw + (a.H + 3) / 4 * 4;
    float* srs = dots + a.R * a.dots;
    // the copies: a warp a row, or several a row where a tile has few
    const int wpr = max(1, kGradWarps / a.R), first = warp / wpr, by = kGradWarps / wpr, piece = 32 * (warp % wpr) + lane;
    const Piece *pg = reinterpret_cast<const Piece*>(dY + (static_cast<long long>(blockIdx.x) * a.R + first) * a.lddy) + piece,
                *ps = reinterpret_cast<const Piece*>(S + (static_cast<long long>(blockIdx.x) * a.R + first) * a.lds) + piece,
                *pr = reinterpret_cast<const Piece*>(dR + (static_cast<long long>(blockIdx.x) * a.R + first) * a.lddr) + piece;
    auto copy = [&](const Piece* from, long long ld, uint8_t* to, int rows) {
        Piece* q = reinterpret_cast<Piece*>(to + first * a.pitch) + piece;
        for (int r = first; r < rows; r += by) {
#pragma unroll 4
            for (int i = 0; i < np - piece; i += 32 * wpr) copy_piece(q + i, from + i);
            q = reinterpret_cast<Piece*>(reinterpret_cast<uint8_t*>(q) + by * a.pitch);
            from = reinterpret_cast<const Piece*>(reinterpret_cast<const V*>(from) + by * ld);
        }
    };
    int next = blockIdx.x;  // tile
    auto fetch = [&](int b) {
        if (next < a.tiles) {
            const int row0 = next * a.R, rows = min(a.R, a.M - row0);
            uint8_t* to = sm + b * stage;
            copy(pg, a.lddy, to, rows);
            copy(ps, a.lds, to + bytes, rows);
            if (a.dR) copy(pr, a.lddr, to + 2 * bytes, rows);
            if (static_cast<int>(threadIdx.x) < rows) srs[b * a.R + threadIdx.x] = load(rs + row0 + threadIdx.x);
            next += gridDim.x;
            const long long step = static_cast<long long>(gridDim.x) * a.R;
            pg = reinterpret_cast<const Piece*>(reinterpret_cast<const V*>(pg) + step * a.lddy);
            ps = reinterpret_cast<const Piece*>(reinterpret_cast<const V*>(ps) + step * a.lds);
            pr = reinterpret_cast<const Piece*>(reinterpret_cast<const V*>(pr) + step * a.lddr);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    // the weights: pair j of piece p at 2 (j np + p), so that a warp's reads share no banks
    for (int i = threadIdx.x; i < a.H; i += kGradThreads)
        sw[N == 1 ? i : 2 * ((i % N) / 2 * np + i / N) + (i & 1)] =
            !a.w ? 1.f : a.wide_w ? load(static_cast<const float*>(w) + i) : to_f(load(static_cast<const V*>(w) + i));
    for (int i = threadIdx.x; i < a.R * a.dots; i += kGradThreads) dots[i] = 0.f;
    const int C = 1 << a.log_c, col = threadIdx.x & (C - 1), mine = threadIdx.x >> a.log_c, others = kGradThreads >> a.log_c;
    const int L = 1 << a.log_l, at = lane & (L - 1);
    // this warp's first stretch (of a row, or one a group of lanes) and the way to its next
    const int u = L < 32 ? (warp << (5 - a.log_l)) + (lane >> a.log_l) : warp, du = L < 32 ? kGradWarps << (5 - a.log_l) : kGradWarps;
    const int r_first = u / a.segs, s_first = u % a.segs, r_step = du / a.segs, s_step = du % a.segs;
    Two acc[K], wk[K];
    __syncthreads();
    auto weight = [&](int p) {
        Two f;
        if constexpr (N == 1) {
            f.v[0] = make_float2(sw[p], 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < X; ++i) f.v[i] = reinterpret_cast<const float2*>(sw)[i * np + p];
        }
        return f;
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int i = 0; i < X; ++i) acc[k].v[i] = make_float2(0.f, 0.f);
        if (col + k * C < np) wk[k] = weight(col + k * C);
    }
    const float over = -1.f / static_cast<float>(a.H);
    V* out0 = static_cast<V*>(a.dX) + (static_cast<long long>(blockIdx.x) * a.R + mine) * a.lddx;
    int b = 0;
    for (int t = blockIdx.x; t < a.tiles; t += gridDim.x, b ^= 1) {
        fetch(b ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const int rows = min(a.R, a.M - t * a.R);
        const uint8_t* tile = sm + b * stage;
        // the stretches' sums, L lanes each; every lane of a warp goes round as often as its first
        for (int r = r_first, seg = s_first; __any_sync(0xffffffffu, r < rows); r += r_step, seg += s_step) {
            if (seg >= a.segs) seg -= a.segs, ++r;
            float2 dot = make_float2(0.f, 0.f);
            if (r < rows) {
                const int p0 = seg * (kLaneValues / N) * L + at;
                const Piece *g = reinterpret_cast<const Piece*>(tile + r * a.pitch), *s = reinterpret_cast<const Piece*>(tile + bytes + r * a.pitch);
#pragma unroll
                for (int i = 0; i < kLaneValues / N; ++i) {
                    const int p = p0 + i * L;
                    if (p < np) {
                        const Two x = floats(read_piece(g + p)), y = floats(read_piece(s + p)), f = weight(p);
#pragma unroll
                        for (int j = 0; j < X; ++j) dot = __ffma2_rn(__fmul2_rn(x.v[j], f.v[j]), y.v[j], dot);
                    }
                }
            }
            float d = dot.x + dot.y;
            if (L == 32) {
#pragma unroll
                for (int e = 16; e > 0; e >>= 1) d += __shfl_xor_sync(0xffffffffu, d, e);
            } else {
                for (int e = L >> 1; e > 0; e >>= 1) d += __shfl_xor_sync(0xffffffffu, d, e);
            }
            if (r < rows && at == 0) dots[r * a.dots + seg] = d;
        }
        __syncthreads();
        // the tile by columns
        V* out = out0;
        for (int r = mine; r < rows; r += others, out += others * a.lddx) {
            const float rstd = srs[b * a.R + r];
            float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < a.dots; i += 4) {
                const float4 e = *reinterpret_cast<const float4*>(dots + r * a.dots + i);
                d.x += e.x, d.y += e.y, d.z += e.z, d.w += e.w;
            }
            const float c = ((d.x + d.y) + (d.z + d.w)) * rstd * over;
            const float2 r2 = make_float2(rstd, rstd), c2 = make_float2(c, c);
            const Piece *g = reinterpret_cast<const Piece*>(tile + r * a.pitch), *s = reinterpret_cast<const Piece*>(tile + bytes + r * a.pitch),
                        *q = reinterpret_cast<const Piece*>(tile + 2 * bytes + r * a.pitch);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int p = col + k * C;
                if (p >= np) break;
                const Two x = floats(read_piece(g + p)), y = floats(read_piece(s + p));
                Two z, o;
                if (a.dR) z = floats(read_piece(q + p));
#pragma unroll
                for (int j = 0; j < X; ++j) {
                    const float2 n = __fmul2_rn(y.v[j], r2);
                    acc[k].v[j] = __ffma2_rn(x.v[j], n, acc[k].v[j]);
                    const float2 v = __ffma2_rn(n, c2, __fmul2_rn(x.v[j], wk[k].v[j]));
                    o.v[j] = a.dR ? __ffma2_rn(v, r2, z.v[j]) : __fmul2_rn(v, r2);
                }
                write_piece(reinterpret_cast<Piece*>(out) + p, packed<V, N>(o));
            }
        }
        out0 += static_cast<long long>(gridDim.x) * a.R * a.lddx;
        __syncthreads();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.part) return;
    float* part = a.part + static_cast<long long>(blockIdx.x) * a.H;
    float* sums = others == 1 ? part : sw;  // the weights are not needed any more
    for (int m = 0; m < others; ++m) {  // in the rows' order
        if (mine == m)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int p = col + k * C;
                if (p >= np) break;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float* to = sums + p * N + i;
                    const float v = i & 1 ? acc[k].v[i / 2].y : acc[k].v[i / 2].x;
                    *to = m == 0 ? v : *to + v;
                }
            }
        if (others > 1) __syncthreads();
    }
    if (others > 1)
        for (int c = threadIdx.x; c < a.H; c += kGradThreads) part[c] = sw[c];
}

// Rows whose tile has no room in shared memory: a block a row, read twice, the second time from L2.
constexpr int kLongValues = 32;
template <class V, int N>
__global__ void __launch_bounds__(kMostThreads, 1) rms_norm_grad_long_kernel(GradArgs a) {
    constexpr int K = kLongValues / N;
    using Piece = Pack<V, N>;
    __shared__ float s_sum[2][kMostThreads / 32];
    let_next_start();
    wait_for_previous();
    const int np = a.H / N;
    const V *dY = behind_wait(static_cast<const V*>(a.dY)), *S = behind_wait(static_cast<const V*>(a.S));
    const V* dR = behind_wait(static_cast<const V*>(a.dR));
    const float* rs = behind_wait(a.rstd);
    const void* w = behind_wait(a.w);
    constexpr int X = (N + 1) / 2;
    Floats<N> acc[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < X; ++i) acc[k].v[i] = make_float2(0.f, 0.f);
    int turn = 0;
    for (int row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const Piece *g = reinterpret_cast<const Piece*>(dY + row * a.lddy), *s = reinterpret_cast<const Piece*>(S + row * a.lds);
        const Piece* r = reinterpret_cast<const Piece*>(dR + row * a.lddr);
        Piece* out = reinterpret_cast<Piece*>(static_cast<V*>(a.dX) + row * a.lddx);
        const float rstd = load(rs + row);
        float2 dot2 = make_float2(0.f, 0.f);
        const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = threadIdx.x + k * kMostThreads;
            if (p >= np) break;
            const Piece x = load(g + p), y = load(s + p);
            const Floats<N> u = floats(x), v = floats(y);
            Floats<N> f;
            if (a.w) f = load_floats<V, N>(w, a.wide_w, static_cast<long long>(p) * N);
#pragma unroll
            for (int i = 0; i < X; ++i) {
                const float2 n = __fmul2_rn(v.v[i], r2);
                acc[k].v[i] = __ffma2_rn(u.v[i], n, acc[k].v[i]);
                dot2 = __ffma2_rn(a.w ? __fmul2_rn(u.v[i], f.v[i]) : u.v[i], n, dot2);
            }
        }
        const float dot = group_sum(dot2.x + dot2.y, kMostThreads, s_sum[turn]) / -static_cast<float>(a.H);
#pragma unroll 2
        for (int p = threadIdx.x; p < np; p += kMostThreads) {
            const Piece x = load(g + p), y = load(s + p);
            const Floats<N> u = floats(x), v = floats(y);
            Floats<N> z, f, o;
            if (a.dR) z = floats(load_once(r + p));
            if (a.w) f = load_floats<V, N>(w, a.wide_w, static_cast<long long>(p) * N);
#pragma unroll
            for (int i = 0; i < X; ++i) {
                const float2 e = __ffma2_rn(__fmul2_rn(v.v[i], r2), make_float2(dot, dot), a.w ? __fmul2_rn(u.v[i], f.v[i]) : u.v[i]);
                o.v[i] = a.dR ? __ffma2_rn(e, r2, z.v[i]) : __fmul2_rn(e, r2);
            }
            write_piece(out + p, packed<V, N>(o));
        }
    }
    if (!a.part) return;
    float* part = a.part + static_cast<long long>(blockIdx.x) * a.H;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int p = threadIdx.x + k * kMostThreads;
        if (p >= np) break;
#pragma unroll
        for (int i = 0; i < N; ++i) part[p * N + i] = i & 1 ? acc[k].v[i / 2].y : acc[k].v[i / 2].x;
    }
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

// Rows of a tile and the blocks of the gradient: as many rows as a stage holds, fewer where every block then has one tile.
struct GradShape {
    int R, tiles, blocks;
};
constexpr int kLongRow = 32 * kGradThreads;  // longer ones go to the other kernel

GradShape grad_shape(int M, int H, int row_bytes) {
    GradShape g{};
    g.R = H > kLongRow ? 1 : std::max(1, std::min({kMostRows, kStageBytes / row_bytes, (M + kGradBlocks - 1) / kGradBlocks}));
    g.tiles = (M - 1) / g.R + 1;
    g.blocks = std::min(g.tiles, H > kLongRow ? kGradBlocks / 2 : kGradBlocks);
    return g;
}

template <class V, int N, int HELD>
cudaError_t grad_kernel(GradArgs a, int blocks, cudaStream_t st) {
    const int np = a.H / N;
    a.log_c = 0;
    while ((1 << a.log_c) < np && (1 << a.log_c) < kGradThreads) ++a.log_c;
    a.log_l = 0;
    while ((kLaneValues << a.log_l) < a.H && a.log_l < 5) ++a.log_l;
    a.segs = (a.H + (kLaneValues << a.log_l) - 1) / (kLaneValues << a.log_l);
    a.dots = (a.segs + 3) / 4 * 4;
    const size_t smem = 2 * static_cast<size_t>(a.dR ? 3 : 2) * a.R * a.pitch + sizeof(float) * ((a.H + 3) / 4 * 4 + a.R * (a.dots + 2));
    const cudaError_t e = spx_tc::set_smem_limit(rms_norm_grad_kernel<V, N, HELD>, 227 * 1024);
    if (e != cudaSuccess) return e;
    return launch_early(rms_norm_grad_kernel<V, N, HELD>, dim3(blocks), kGradThreads, smem, 1, st, a);
}

template <class V, int N>
cudaError_t grad_launch(GradArgs a, float* dw, cudaStream_t st) {
    a.pitch = static_cast<int>((a.H * sizeof(V) + 15) / 16 * 16);
    const GradShape g = grad_shape(a.M, a.H, (a.dR ? 3 : 2) * a.pitch);
    a.R = g.R, a.tiles = g.tiles;
    if (a.part && g.blocks == 1) a.part = dw;
    spx_note_launches(a.part && g.blocks > 1 ? 2 : 1);
    cudaError_t e = a.H > kLongRow            ? launch_early(rms_norm_grad_long_kernel<V, N>, dim3(g.blocks), kMostThreads, 0, 1, st, a)
                    : a.H <= 16 * kGradThreads ? grad_kernel<V, N, 16>(a, g.blocks, st)
                                               : grad_kernel<V, N, 32>(a, g.blocks, st);
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
    return M > 1 ? sizeof(float) * static_cast<size_t>(std::min(M, kGradBlocks)) * static_cast<size_t>(H) : 0;
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
