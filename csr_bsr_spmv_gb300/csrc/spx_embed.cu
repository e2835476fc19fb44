// spx_embed.cu -- rows of a table by token id, and the table's gradient.
//
// The lookup is a product with a sparse matrix that has one entry a row; bound
// by HBM.  Its gradient is the product with the transpose, which needs the
// entries by column: the tokens sorted by id, stable, so that the sums' order
// does not depend on timing.  Three launches:
//   1 embed_order_kernel  each block owns a range of ids.  It counts the tokens
//     of each and those of lower ranges, places its tokens, and writes zeros to
//     its rows that have none, which is most of the bytes.
//   2 embed_sum_kernel    chunks of consecutive sorted tokens, whatever their
//     ids, so that popular ones do not hold up a block.  Ids that lie within a
//     chunk are written, the sums of those that cross its ends kept.
//   3 embed_join_kernel   the kept sums of each such id, in chunk order.
#include <algorithm>

#include "spx_rows.cuh"

using namespace spx_rows;

namespace {

constexpr int kThreads = 256;

// Token t's id, -1 outside [0, V).
struct Ids {
    const void* p;
    int bytes, V;
};
__device__ __forceinline__ int id_of(const Ids& x, int t) {
    if (x.bytes == 4) {
        const int v = load(static_cast<const int*>(x.p) + t);
        return v >= 0 && v < x.V ? v : -1;
    }
    const long long v = load(static_cast<const long long*>(x.p) + t);
    return v >= 0 && v < x.V ? static_cast<int>(v) : -1;
}

// ---------------------------------------------------------------- lookup

constexpr int kTokens = 4;  // a group's tokens: their rows are in flight together

// Groups of G threads, G a power of two; grid.y splits the rows.
template <class V, int N>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(Ids x, int T, int np, int log_g, const V* W, long long ldw, float scale, V* Y, long long ldy) {
    using Piece = Pack<V, N>;
    let_next_start();
    wait_for_previous();
    x.p = behind_wait(x.p);
    W = behind_wait(W);
    const int G = 1 << log_g, t0 = (blockIdx.x * (kThreads >> log_g) + (threadIdx.x >> log_g)) * kTokens;
    int id[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) id[u] = t0 + u < T ? id_of(x, t0 + u) : -1;
    for (int v = blockIdx.y * G + (threadIdx.x & (G - 1)); v < np; v += gridDim.y * G) {
        Piece p[kTokens];
#pragma unroll
        for (int u = 0; u < kTokens; ++u)
            if (id[u] >= 0) p[u] = load(reinterpret_cast<const Piece*>(W + id[u] * ldw) + v);
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            if (t0 + u >= T) break;
            Floats<N> f = floats(p[u]);
#pragma unroll
            for (int i = 0; i < (N + 1) / 2; ++i) f.v[i] = id[u] >= 0 ? __fmul2_rn(f.v[i], make_float2(scale, scale)) : make_float2(0.f, 0.f);
            write_once(reinterpret_cast<Piece*>(Y + (t0 + u) * ldy) + v, packed<V, N>(f));
        }
    }
}

// ---------------------------------------------------------------- tokens by id

constexpr int kOrderThreads = 512, kOrderWarps = kOrderThreads / 32;
constexpr int kMostIds = 4096;   // ids a block owns
constexpr int kList = 2048;      // tokens of its ids that a block holds in shared memory

struct OrderArgs {
    Ids x;
    int T, per, padding;       // ids a block
    int *order, *sid, *list;   // sorted tokens and their ids; a block's tokens before they are sorted, where they do not fit
    int* kept;                 // tokens in all that have a row
    void* dW;                  // NULL: no zeros are written
    long long ldw;             // bytes
    long long row;             // bytes a row
};

// Z: the widest word that rows are made of.
template <class Z>
__global__ void __launch_bounds__(kOrderThreads, 2) embed_order_kernel(OrderArgs a) {
    __shared__ int s_at[kMostIds + 1];  // counts, then first places
    __shared__ int s_list[kList], s_lid[kList];
    __shared__ int s_warp[kOrderWarps], s_below[kOrderWarps], s_next;
    let_next_start();
    wait_for_previous();
    a.x.p = behind_wait(a.x.p);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long first = static_cast<long long>(blockIdx.x) * a.per;
    const int v0 = static_cast<int>(min(first, static_cast<long long>(a.x.V))), nv = min(a.per, a.x.V - v0);
    for (int i = threadIdx.x; i <= nv; i += kOrderThreads) s_at[i] = 0;
    if (threadIdx.x == 0) s_next = 0;
    __syncthreads();
    // each warp looks at a run of consecutive tokens
    const int run = ((a.T + kOrderThreads - 1) / kOrderThreads) * 32, t0 = min(w * static_cast<long long>(run), static_cast<long long>(a.T)), t1 = min(static_cast<long long>(t0) + run, static_cast<long long>(a.T));
    auto local = [&](int t) {  // the token's id in this block's range, -1: another's (lower: below the range), or none
        const int id = t < t1 ? id_of(a.x, t) : -1;
        return id == a.padding ? -1 : id;
    };
    int below = 0, mine = 0;
    for (int t = t0; t < t1; t += 128) {
        int id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) id[u] = local(t + 32 * u + lane);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool in = id[u] >= v0 && id[u] < v0 + nv;
            if (in) atomicAdd(s_at + id[u] - v0, 1);
            mine += in;
            below += id[u] >= 0 && id[u] < v0;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        mine += __shfl_xor_sync(0xffffffffu, mine, d);
        below += __shfl_xor_sync(0xffffffffu, below, d);
    }
    if (lane == 0) s_warp[w] = mine, s_below[w] = below;
    __syncthreads();
    int all = 0, before = 0;
    below = 0;
#pragma unroll
    for (int i = 0; i < kOrderWarps; ++i) {
        before += i < w ? s_warp[i] : 0;
        all += s_warp[i];
        below += s_below[i];
    }
    const bool held = all <= kList;
    if (mine) {  // this warp's tokens to the block's list, in order
        int at = before;
        for (int t = t0; t < t1; t += 32) {
            const int id = local(t + lane);
            const bool in = id >= v0 && id < v0 + nv;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            const int to = at + __popc(who & ((1u << lane) - 1u));
            if (in) {
                if (held) s_list[to] = t + lane, s_lid[to] = id - v0;
                else a.list[below + to] = t + lane;
            }
            at += __popc(who);
        }
    }
    // counts to first places, by the first warp
    __syncthreads();
    if (w == 0) {
        int carry = 0;
        for (int i0 = 0; i0 <= nv; i0 += 32) {
            const int n = i0 + lane < nv ? s_at[i0 + lane] : 0;
            int inc = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += up;
            }
            if (i0 + lane <= nv) s_at[i0 + lane] = carry + inc - n;
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0 && blockIdx.x == gridDim.x - 1) *a.kept = below + all;
    }
    __syncthreads();
    if (a.dW) {  // zeros, a warp a row
        char* dW = static_cast<char*>(a.dW) + v0 * a.ldw;
        for (int i = w; i < nv; i += kOrderWarps) {
            if (s_at[i] != s_at[i + 1]) continue;
            Z* q = reinterpret_cast<Z*>(dW + i * a.ldw);
            Z zero;
            memset(&zero, 0, sizeof(Z));
            for (int c = lane; c < a.row / static_cast<int>(sizeof(Z)); c += 32) q[c] = zero;
        }
        __syncthreads();
    }
    if (w != 0) return;
    for (int i0 = 0; i0 < all; i0 += 32) {
        const int i = i0 + lane;
        int t = 0, l = -1 - lane;
        if (i < all) {
            if (held) t = s_list[i], l = s_lid[i];
            else t = a.list[below + i], l = id_of(a.x, t) - v0;
        }
        const unsigned same = __match_any_sync(0xffffffffu, l), lower = same & ((1u << lane) - 1u);
        int to = 0;
        if (i < all) to = s_at[l] + __popc(lower);
        __syncwarp();
        if (i < all) {
            if (lower == 0) s_at[l] += __popc(same);
            a.order[below + to] = t;
            a.sid[below + to] = l + v0;
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- sums

struct SumArgs {
    int np, T, chunk;          // pieces a row, tokens, sorted tokens a chunk
    const int *order, *sid, *kept;
    const void* dY;
    long long lddy;
    void* dW;
    long long ldw;
    float* part;               // two rows of ldp values a chunk: the sums of an id that began before it, and of its last, open one
    long long ldp;
    float scale;
    bool add;
};

template <class O, int N>
__device__ __forceinline__ void write_sum(const SumArgs& a, int id, int v, const Floats<N>& acc) {
    constexpr int Q = N * sizeof(O) > 16 ? 16 / sizeof(O) : N, X = (Q + 1) / 2;
    Pack<O, Q>* q = reinterpret_cast<Pack<O, Q>*>(static_cast<O*>(a.dW) + id * a.ldw + static_cast<long long>(v) * N);
    const float2 c = make_float2(a.scale, a.scale);
#pragma unroll
    for (int i = 0; i < N / Q; ++i) {
        Floats<Q> f;
        if (a.add) f = floats(load(q + i));
#pragma unroll
        for (int j = 0; j < X; ++j) f.v[j] = a.add ? __ffma2_rn(acc.v[X * i + j], c, f.v[j]) : __fmul2_rn(acc.v[X * i + j], c);
        write_piece(q + i, packed<O, Q>(f));
    }
}

constexpr int kRows = 8;  // rows in flight

// A warp's lanes hold the tokens and ids of 32 sorted places, the next 32 on their way.
template <class V, class O, int N>
__global__ void __launch_bounds__(kThreads, 3) embed_sum_kernel(SumArgs a) {
    constexpr int X = (N + 1) / 2;
    using Piece = Pack<V, N>;
    let_next_start();
    wait_for_previous();
    const int *order = behind_wait(a.order), *sid = behind_wait(a.sid);
    const int lane = threadIdx.x & 31, v = min(static_cast<int>(blockIdx.y * kThreads + threadIdx.x), a.np - 1);
    const bool mine = static_cast<int>(blockIdx.y * kThreads + threadIdx.x) < a.np;
    const long long first = static_cast<long long>(blockIdx.x) * a.chunk;
    const int p0 = static_cast<int>(first), most = static_cast<int>(min(first + a.chunk, static_cast<long long>(a.T)));
    // places past the last token's hold anything: they are looked at with the number of tokens in hand
    int next_id = p0 + lane < most ? load(sid + p0 + lane) : -1, next_at = p0 + lane < most ? load(order + p0 + lane) : 0;
    const int left = p0 > 0 ? load(sid + p0 - 1) : -1, right = most < a.T ? load(sid + most) : -1;
    const int n = load(behind_wait(a.kept));
    if (p0 >= n) return;
    const int p1 = min(most, n);
    const V* dY = behind_wait(static_cast<const V*>(a.dY)) + static_cast<long long>(v) * N;
    int id = __shfl_sync(0xffffffffu, next_id, 0);
    bool open = p0 > 0 && left == id;  // the current id began before the chunk
    Floats<N> acc;
#pragma unroll
    for (int i = 0; i < X; ++i) acc.v[i] = make_float2(0.f, 0.f);
    auto keep = [&](int which) {
        if (!mine) return;
        constexpr int Q = N < 4 ? N : 4;
        Pack<float, Q>* q = reinterpret_cast<Pack<float, Q>*>(a.part + (2LL * blockIdx.x + which) * a.ldp + static_cast<long long>(v) * N);
#pragma unroll
        for (int i = 0; i < N / Q; ++i) {
            Floats<Q> f;
#pragma unroll
            for (int j = 0; j < (Q + 1) / 2; ++j) f.v[j] = acc.v[(Q + 1) / 2 * i + j];
            write_piece(q + i, packed<float, Q>(f));
        }
    };
    for (int base = p0; base < p1; base += 32) {
        const int my_id = next_id, my_at = next_at;
        if (base + 32 + lane < p1) next_id = load(sid + base + 32 + lane), next_at = load(order + base + 32 + lane);
        for (int u0 = 0; u0 < 32 && base + u0 < p1; u0 += kRows) {
            Piece x[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int t = __shfl_sync(0xffffffffu, my_at, u0 + u);
                if (base + u0 + u < p1) x[u] = load_once(reinterpret_cast<const Piece*>(dY + t * a.lddy));
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int next = __shfl_sync(0xffffffffu, my_id, u0 + u);
                if (base + u0 + u >= p1) continue;
                if (next != id) {
                    if (open) keep(0);
                    else if (mine) write_sum<O, N>(a, id, v, acc);
                    open = false;
                    id = next;
#pragma unroll
                    for (int i = 0; i < X; ++i) acc.v[i] = make_float2(0.f, 0.f);
                }
                const Floats<N> f = floats(x[u]);
#pragma unroll
                for (int i = 0; i < X; ++i) acc.v[i] = __fadd2_rn(acc.v[i], f.v[i]);
            }
        }
    }
    if (open) keep(0);
    else if (p1 < n && right == id) keep(1);
    else if (mine) write_sum<O, N>(a, id, v, acc);
}

// One block for each chunk whose last id began in it and goes on after it.
template <class O, int N>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(SumArgs a) {
    constexpr int X = (N + 1) / 2;
    let_next_start();
    wait_for_previous();
    const int* sid = behind_wait(a.sid);
    const float* part = behind_wait(static_cast<const float*>(a.part));
    const int v = blockIdx.y * kThreads + threadIdx.x;
    const long long p0 = static_cast<long long>(blockIdx.x) * a.chunk, p1 = p0 + a.chunk;
    if (p1 >= a.T) return;
    // places past the last token's hold anything
    const int n = load(behind_wait(a.kept)), id = load(sid + p1 - 1), after = load(sid + p1), before = p0 > 0 ? load(sid + p0 - 1) : -1;
    if (p1 >= n || after != id || (p0 > 0 && before == id)) return;
    // the chunks that the id goes on in, a thread a chunk
    int chunks = 0;
    for (;;) {
        const long long p = p1 + (chunks + static_cast<long long>(threadIdx.x)) * a.chunk;
        const int more = __syncthreads_count(p < n && load(sid + p) == id);
        chunks += more;
        if (more < kThreads) break;
    }
    if (v >= a.np) return;
    Floats<N> acc;
    part += 2LL * blockIdx.x * a.ldp + static_cast<long long>(v) * N;
    auto row = [&](const float* p) { return load_floats<float, N>(p, true, 0); };
    acc = row(part + a.ldp);
#pragma unroll 8
    for (int c = 1; c <= chunks; ++c) {
        const Floats<N> f = row(part + 2LL * c * a.ldp);
#pragma unroll
        for (int i = 0; i < X; ++i) acc.v[i] = __fadd2_rn(acc.v[i], f.v[i]);
    }
    write_sum<O, N>(a, id, v, acc);
}

// ---------------------------------------------------------------- host side

spx_status check(int32_t T, int32_t H, int32_t V, spx_type type, int32_t id_bytes) {
    if (T < 0 || H < 0 || V < 0 || !is_float_type(type) || (id_bytes != 4 && id_bytes != 8)) return SPX_ERR_ARG;
    if (T > kMostIndex || H > kMostIndex || V > kMostIndex) return SPX_ERR_INDEX_RANGE;
    return SPX_OK;
}

template <class V, int N>
cudaError_t embed_launch(int T, int H, Ids x, const void* W, int64_t ldw, float scale, void* Y, int64_t ldy, cudaStream_t st) {
    const int np = H / N;
    int lg = 3;
    while (lg < 8 && (1 << lg) < np) ++lg;
    const int per = (kThreads >> lg) * kTokens, bx = (T + per - 1) / per;
    const int steps = (np + (1 << lg) - 1) >> lg, by = std::min(steps, std::max(1, 1216 / bx));
    return launch_early(embed_kernel<V, N>, dim3(bx, by), kThreads, 0, 1, st, x, T, np, lg, static_cast<const V*>(W), static_cast<long long>(ldw), scale,
                        static_cast<V*>(Y), static_cast<long long>(ldy));
}

template <class V>
spx_status embed(int T, int H, Ids x, const void* W, int64_t ldw, float scale, void* Y, int64_t ldy, cudaStream_t st) {
    const int vb = copy_width(addr(W) | addr(Y) | (static_cast<uint64_t>(H) | ldw | ldy) * sizeof(V), sizeof(V));
    spx_note_launches(1);
    if (vb == 16) return spx_cuda_status(embed_launch<V, 16 / sizeof(V)>(T, H, x, W, ldw, scale, Y, ldy, st));
    if (sizeof(V) == 2 && vb >= 4) return spx_cuda_status(embed_launch<V, 4 / sizeof(V)>(T, H, x, W, ldw, scale, Y, ldy, st));
    return spx_cuda_status(embed_launch<V, 1>(T, H, x, W, ldw, scale, Y, ldy, st));
}

// Sorted tokens a chunk: 8 to 32, so that the chunks fill the SMs, more where there would be over 4096 of them.
int chunk_of(int T) { return std::max(std::min(32, (T / 512 + 7) / 8 * 8 + 8), (T + 4095) / 4096); }

struct Scratch {
    size_t order, sid, list, kept, part, bytes;
    long long ldp;
};
Scratch scratch_of(int T, int H) {
    Scratch s{};
    const size_t ints = (static_cast<size_t>(T) * 4 + 15) / 16 * 16;
    s.order = 0, s.sid = ints, s.list = 2 * ints, s.kept = 3 * ints, s.part = 3 * ints + 16;
    s.ldp = (static_cast<long long>(H) + 3) / 4 * 4;
    const size_t chunks = (static_cast<size_t>(T) + chunk_of(T) - 1) / chunk_of(T);
    s.bytes = s.part + chunks * 2 * static_cast<size_t>(s.ldp) * sizeof(float);
    return s;
}

template <class V, class O, int N>
cudaError_t sums(const SumArgs& a, int T, cudaStream_t st) {
    const dim3 grid((T + a.chunk - 1) / a.chunk, (a.np + kThreads - 1) / kThreads);
    if (grid.y > 65535) return cudaErrorInvalidValue;
    const cudaError_t e = launch_early(embed_sum_kernel<V, O, N>, grid, kThreads, 0, 1, st, a);
    return e != cudaSuccess ? e : launch_early(embed_join_kernel<O, N>, grid, kThreads, 0, 1, st, a);
}

template <class V, class O>
cudaError_t sums_in_pieces(SumArgs a, int T, int H, cudaStream_t st) {
    // pieces of dY of up to 16 bytes; dW's as many values, in words of up to 16 bytes
    uint64_t bits = addr(a.dY) | (static_cast<uint64_t>(H) | a.lddy) * sizeof(V);
    const uint64_t w = addr(a.dW) | (static_cast<uint64_t>(H) | a.ldw) * sizeof(O);
    const int N = copy_width(bits, sizeof(V)) / sizeof(V), M = copy_width(w, sizeof(O)) / sizeof(O);
    constexpr int N16 = 16 / sizeof(V), M16 = 16 / sizeof(O);
    if (N == N16 && M >= std::min(N16, M16)) {
        a.np = H / N16;
        return sums<V, O, N16>(a, T, st);
    }
    if (sizeof(V) == 2 && N >= 2 && M >= 2) {
        a.np = H / 2;
        return sums<V, O, 2>(a, T, st);
    }
    a.np = H;
    return sums<V, O, 1>(a, T, st);
}

}  // namespace

extern "C" {

spx_status spx_embed(int32_t T, int32_t H, int32_t V, spx_type type, const void* ids, int32_t id_bytes, const void* W,
                     int64_t ldw, float scale, void* Y, int64_t ldy, spx_stream_t stream) {
    const spx_status c = check(T, H, V, type, id_bytes);
    if (c != SPX_OK) return c;
    if (T == 0 || H == 0) return SPX_OK;
    if (!ids || !Y || ldy < H || (V > 0 && (!W || ldw < H))) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type);
    if (!spx_aligned(ids, static_cast<size_t>(id_bytes)) || !spx_aligned(W, eb) || !spx_aligned(Y, eb)) return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const Ids x{ids, id_bytes, V};
    if (type == SPX_F32) return embed<float>(T, H, x, W, ldw, scale, Y, ldy, st);
    if (type == SPX_BF16) return embed<__nv_bfloat16>(T, H, x, W, ldw, scale, Y, ldy, st);
    return embed<__half>(T, H, x, W, ldw, scale, Y, ldy, st);
}

size_t spx_embed_grad_scratch_bytes(int32_t T, int32_t H) {
    if (T < 0 || H < 0 || T > kMostIndex || H > kMostIndex) return 0;
    return scratch_of(T, H).bytes;
}

spx_status spx_embed_grad(int32_t T, int32_t H, int32_t V, spx_type type, const void* ids, int32_t id_bytes, int32_t padding,
                          float scale, const void* dY, int64_t lddy, void* dW, int64_t lddw, spx_type w_type,
                          int32_t accumulate, void* scratch, size_t scratch_bytes, spx_stream_t stream) {
    const spx_status c = check(T, H, V, type, id_bytes);
    if (c != SPX_OK) return c;
    if (w_type != type && w_type != SPX_F32) return SPX_ERR_ARG;
    if (H == 0 || V == 0 || (T == 0 && accumulate)) return SPX_OK;
    if (!dW || lddw < H || (T > 0 && (!ids || !dY || lddy < H))) return SPX_ERR_ARG;
    if (!scratch || scratch_bytes < spx_embed_grad_scratch_bytes(T, H)) return SPX_ERR_ARG;
    const size_t eb = type_bytes(type), wb = type_bytes(w_type);
    if (!spx_aligned(ids, static_cast<size_t>(id_bytes)) || !spx_aligned(dY, eb) || !spx_aligned(dW, wb) || !spx_aligned(scratch, 16))
        return SPX_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const Scratch s = scratch_of(T, H);
    char* base = static_cast<char*>(scratch);
    OrderArgs o{};
    o.x = Ids{ids, id_bytes, V};
    o.T = T, o.padding = padding;
    o.order = reinterpret_cast<int*>(base + s.order), o.sid = reinterpret_cast<int*>(base + s.sid);
    o.list = reinterpret_cast<int*>(base + s.list), o.kept = reinterpret_cast<int*>(base + s.kept);
    o.dW = accumulate ? nullptr : dW;
    o.ldw = static_cast<long long>(lddw * wb), o.row = static_cast<long long>(H * wb);
    const int blocks = std::max(304, (V + kMostIds - 1) / kMostIds);
    o.per = (V + blocks - 1) / blocks;
    const dim3 grid((V + o.per - 1) / o.per);
    const int zb = copy_width(addr(dW) | o.ldw | o.row, static_cast<int>(wb));
    spx_note_launches(3);
    cudaError_t e = zb == 16  ? launch_early(embed_order_kernel<uint4>, grid, kOrderThreads, 0, 1, st, o)
                    : zb == 8 ? launch_early(embed_order_kernel<uint2>, grid, kOrderThreads, 0, 1, st, o)
                    : zb == 4 ? launch_early(embed_order_kernel<uint32_t>, grid, kOrderThreads, 0, 1, st, o)
                              : launch_early(embed_order_kernel<uint16_t>, grid, kOrderThreads, 0, 1, st, o);
    if (e != cudaSuccess || T == 0) return spx_cuda_status(e);
    SumArgs a{};
    a.chunk = chunk_of(T), a.T = T;
    a.order = o.order, a.sid = o.sid, a.kept = o.kept;
    a.dY = dY, a.lddy = lddy, a.dW = dW, a.ldw = lddw;
    a.part = reinterpret_cast<float*>(base + s.part), a.ldp = s.ldp;
    a.scale = scale, a.add = accumulate != 0;
    if (type == SPX_F32) e = sums_in_pieces<float, float>(a, T, H, st);
    else if (type == SPX_BF16) e = w_type == SPX_F32 ? sums_in_pieces<__nv_bfloat16, float>(a, T, H, st) : sums_in_pieces<__nv_bfloat16, __nv_bfloat16>(a, T, H, st);
    else e = w_type == SPX_F32 ? sums_in_pieces<__half, float>(a, T, H, st) : sums_in_pieces<__half, __half>(a, T, H, st);
    return spx_cuda_status(e);
}

}  // extern "C"
