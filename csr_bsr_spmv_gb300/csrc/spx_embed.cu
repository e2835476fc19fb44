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
//
// Measured: 16384 rows of 4096 bf16 of 65536 looked up in 33 us, 5.7 TB/s of what
// has to move (rows that occur twice are read once); 301 of 1002 fp16 1.9 us.
// The gradient of 16384 tokens of 2048 bf16 over 65536 rows 61 us for 49 of HBM:
// about 40 the sort and the zeros, 20 the sums, whose launches follow one
// another; 7 for the sort alone where no token is left.  Writing the zeros
// beside the sums instead was not faster.
#include <algorithm>

#include "spx_rows.cuh"
#include "spx_tc.cuh"

using namespace spx_rows;

namespace {

constexpr int kThreads = 256, kMostGridY = 65535;

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

// Bound by HBM, with four rows of a group in flight.  Rows of 4094 values take 44 us where 4096 take 33, of 4095 67: pieces of 4
// bytes, or of 16 put together from two words.
constexpr int kTokens = 4;

// Groups of G threads, G a power of two; grid.y splits the rows.
template <class V, int N, bool ANY>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(Ids x, int T, int H, int log_g, const V* W, long long ldw, float scale, V* Y, long long ldy) {
    let_next_start();
    wait_for_previous();
    x.p = behind_wait(x.p);
    W = behind_wait(W);
    const Rows<V, N, ANY> rows{H};
    const int G = 1 << log_g, np = rows.pieces(), at = threadIdx.x & (G - 1), t0 = (blockIdx.x * (kThreads >> log_g) + (threadIdx.x >> log_g)) * kTokens;
    const bool left = at > 0 && (threadIdx.x & 31) > 0;
    const V* end = W + (x.V - 1LL) * ldw + H;
    int id[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) id[u] = t0 + u < T ? id_of(x, t0 + u) : -1;
    bool in = x.V > 0;  // all rows inside the table; of no token row 0 is read, and not used
#pragma unroll
    for (int u = 0; u < kTokens; ++u) in = in && rows.inside(W + max(id[u], 0) * ldw, W, end);
    for (int v0 = blockIdx.y * G; v0 < np; v0 += gridDim.y * G) {
        const int v = v0 + at;
        Pack<V, N> p[kTokens];
        if (in) {
#pragma unroll
            for (int u = 0; u < kTokens; ++u) p[u] = rows.template read<true>(W + max(id[u], 0) * ldw, v);
        } else {
#pragma unroll
            for (int u = 0; u < kTokens; ++u)
                if (id[u] >= 0 && v < np) p[u] = rows.read_edge(W + id[u] * ldw, v);
        }
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            Floats<N> f = floats(p[u]);
#pragma unroll
            for (int i = 0; i < (N + 1) / 2; ++i) f.v[i] = id[u] >= 0 ? __fmul2_rn(f.v[i], make_float2(scale, scale)) : make_float2(0.f, 0.f);
            rows.write(Y + (t0 + u) * ldy, v, packed<V, N>(f), t0 + u < T, left);
        }
    }
}

// ---------------------------------------------------------------- tokens by id

// A block owns `per` ids and looks at 16384 tokens at a time, 512 consecutive ones a warp, of which it takes those of its
// ids: a warp's go to a list of its own, in order.  Of one id among 32 neighbours of that list match_any finds the lanes;
// with counters per id of its own the warp so knows each token's rank in its list, and the counters of the warps before it
// and the counts of lower ids give the place.  Of more than 16384 tokens the block's go to a list of the block first, in
// order (65536 tokens over 65536 rows of 128 values 48 us without the list and 40); where they do not fit it, all are read
// once more.  The work so grows with tokens times blocks, of which there are 152 or one for every 1024 ids.  No floating-point and no order that depends on timing: the atomics are whole sums.  Nearly all of a block's
// work is passing over other blocks' tokens, so that is what is kept short; the other loops stay loops, since unrolled the kernel took longer to fetch its code than to run it.
constexpr int kOrderThreads = 1024, kOrderWarps = kOrderThreads / 32, kSlots = 16, kRun = 32 * kSlots, kBatch = kOrderWarps * kRun;
constexpr int kMostIds = 1024, kList = 4096;  // a warp's word: 10 bits of the id, 9 of the place in its run, 9 of the rank

struct OrderArgs {
    Ids x;
    int T, per, padding;
    int *order, *sid;   // sorted tokens and their ids
    int* kept;          // tokens in all that have a row
    void* dW;           // NULL: no zeros are written
    long long ldw, row; // bytes
};

// Zeros in a block's rows without tokens, a warp a row: whole aligned words, and 2-byte values before and after them.  Bit
// i of empty[j]: row 32 j + i.
__device__ __forceinline__ void fill_rows(const OrderArgs& a, long long v0, int nv, const uint32_t* empty) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < nv; i += kOrderWarps) {
        if (!(empty[i >> 5] >> (i & 31) & 1u)) continue;
        char* q = static_cast<char*>(a.dW) + (v0 + i) * a.ldw;
        const int head = static_cast<int>(min(a.row, static_cast<long long>(-reinterpret_cast<intptr_t>(q) & 15)));
        const int words = static_cast<int>((a.row - head) / 16), tail = static_cast<int>((a.row - head) % 16);
        for (int c = lane; c < words; c += 32) __stcs(reinterpret_cast<uint4*>(q + head) + c, make_uint4(0, 0, 0, 0));
        const int at = lane < 8 ? 2 * lane : head + 16 * words + 2 * (lane - 8);  // lanes 0 to 7: the head, 8 to 15: the tail
        if (lane < 8 ? 2 * lane < head : 2 * (lane - 8) < tail) *reinterpret_cast<uint16_t*>(q + at) = 0;
    }
}

// Sums of the warps before warp w and of all 32, from a word a warp.
__device__ __forceinline__ int2 warps_before(const int* s, int w) {
    const int own = s[threadIdx.x & 31];
    int up = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, up, d);
        if (static_cast<int>(threadIdx.x & 31) >= d) up += o;
    }
    return make_int2(__shfl_sync(0xffffffffu, up - own, w), __shfl_sync(0xffffffffu, up, 31));
}

__global__ void __launch_bounds__(kOrderThreads, 1) embed_order_kernel(OrderArgs a) {
    // the warps' lists (kRun each), the block's list (tokens, then ids), places of the block's ids (per), a counter for each
    // warp and id (16 bits, pitch odd)
    extern __shared__ int sm[];
    __shared__ int s_below[kOrderWarps], s_carry[kOrderWarps], s_found[2][kOrderWarps];
    __shared__ uint32_t s_empty[kOrderWarps];
    let_next_start();
    wait_for_previous();
    a.x.p = behind_wait(a.x.p);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned lower = (1u << lane) - 1u;
    const int v0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * a.per, static_cast<long long>(a.x.V))), nv = min(a.per, a.x.V - v0);
    int *own = sm + w * kRun, *list = sm + kBatch, *place = list + 2 * kList;
    uint16_t* counters = reinterpret_cast<uint16_t*>(place + a.per);
    const int pitch = (a.per + 1) | 1;
    uint16_t* mine = counters + w * pitch;
    int below = 0;  // this lane's tokens of lower ids
    // the warp's tokens of this block's ids: the id, and above it the place in the run; how many
    auto read = [&](int base, bool count) {
        const long long t0 = static_cast<long long>(base) + w * kRun + lane;
        constexpr int kAhead = 8;  // loads in flight; past the end the last token again: no branch between them
        int taken = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < kSlots; i0 += kAhead) {
            long long v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const long long t = min(t0 + 32 * (i0 + i), a.T - 1LL);
                v[i] = a.x.bytes == 4 ? load(static_cast<const int*>(a.x.p) + t) : load(static_cast<const long long*>(a.x.p) + t);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) asm volatile("" : "+l"(v[i]));
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const bool on = static_cast<unsigned long long>(v[i]) < static_cast<unsigned>(a.x.V) && static_cast<int>(v[i]) != a.padding &&
                                t0 + 32 * (i0 + i) < a.T;
                const int id = static_cast<int>(v[i]) - v0;
                const bool in = on && static_cast<unsigned>(id) < static_cast<unsigned>(nv);
                below += on && id < 0 && count;
                const unsigned who = __ballot_sync(0xffffffffu, in);
                if (!who) continue;
                if (in) {
                    own[taken + __popc(who & lower)] = id | (32 * (i0 + i) + lane) << 16;
                    if (count) atomicAdd(place + id, 1);
                }
                taken += __popc(who);
            }
        }
        __syncwarp();
        return taken;
    };
    if (static_cast<int>(threadIdx.x) < nv) place[threadIdx.x] = 0;
    __syncthreads();
    const bool once = a.T <= kBatch;
    int taken = 0, found = 0, turn = 0;  // found: tokens of this block in the batches so far
    for (int base = 0; a.T > 0; turn ^= 1) {
        taken = read(base, true);
        if (!once) {
            if (lane == 0) s_found[turn][w] = taken;
            __syncthreads();
            const int2 f = warps_before(s_found[turn], w);
            for (int i = lane; i < taken; i += 32) {
                const int to = found + f.x + i;
                if (to < kList) list[to] = base + w * kRun + (own[i] >> 16), list[kList + to] = own[i] & 0xffff;
            }
            __syncwarp();
            found += f.y;
        }
        if (a.T - base <= kBatch) break;
        base += kBatch;
    }
    const bool listed = !once && found <= kList;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
    if (lane == 0) s_below[w] = below;
    for (int i = threadIdx.x; i < (kOrderWarps * pitch + 1) / 2; i += kOrderThreads) reinterpret_cast<int*>(counters)[i] = 0;
    __syncthreads();
    // counts to first places: a warp's 32 ids, then the warps before it
    const int n = static_cast<int>(threadIdx.x) < nv ? place[threadIdx.x] : 0;
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 31) s_carry[w] = inc;
    const uint32_t none = __ballot_sync(0xffffffffu, n == 0);
    if (lane == 0) s_empty[w] = none;
    __syncthreads();
    below = warps_before(s_below, 0).y;
    const int2 carry = warps_before(s_carry, w);
    if (static_cast<int>(threadIdx.x) < nv) place[threadIdx.x] = below + carry.x + inc - n;
    if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) *a.kept = below + carry.y;
    for (int base = 0; a.T > 0;) {
        if (listed) {  // the block's list in runs
            taken = max(0, min(kRun, found - w * kRun));
            for (int i = lane; i < taken; i += 32) own[i] = list[kList + w * kRun + i] | i << 16;
            __syncwarp();
        } else if (!once) {
            taken = read(base, false);
        }
        // the ranks among the warp's tokens of an id, above the place in the run
#pragma unroll 1
        for (int i0 = 0; i0 < taken; i0 += 32) {
            const bool on = i0 + lane < taken;
            const int word = on ? own[i0 + lane] : 0, id = on ? word & 0x3ff : -1;
            const unsigned same = __match_any_sync(0xffffffffu, id), before = same & lower;
            if (on) own[i0 + lane] = word >> 16 << 10 | id | (mine[id] + __popc(before)) << 19;
            __syncwarp();
            if (on && before == 0) mine[id] += static_cast<uint16_t>(__popc(same));
            __syncwarp();
        }
        __syncthreads();
        int sum = 0;  // an id's tokens in this batch
        if (n > 0) {
            uint16_t* c = counters + threadIdx.x;
#pragma unroll 1
            for (int i = 0; i < kOrderWarps; i += 8) {
                int k[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) k[j] = c[(i + j) * pitch];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    c[(i + j) * pitch] = static_cast<uint16_t>(sum);
                    sum += k[j];
                }
            }
        }
        __syncthreads();
        for (int i = lane; i < taken; i += 32) {
            const int word = own[i], id = word & 0x3ff, at = word >> 10 & 0x1ff, to = place[id] + mine[id] + (word >> 19);
            a.order[to] = listed ? list[w * kRun + at] : base + w * kRun + at;
            a.sid[to] = id + v0;
        }
        if (listed || a.T - base <= kBatch) break;
        base += kBatch;
        __syncthreads();
        if (n > 0) place[threadIdx.x] += sum;
        for (int i = threadIdx.x; i < (kOrderWarps * pitch + 1) / 2; i += kOrderThreads) reinterpret_cast<int*>(counters)[i] = 0;
        __syncthreads();
    }
    if (a.dW) fill_rows(a, v0, nv, s_empty);
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

constexpr int kRows = 8, kSets = 3, kMostChunk = 1024;

// A thread's pieces of eight rows are a set: one set is added while two are on their way into the thread's own slots of
// shared memory (pieces of 2 bytes, which no asynchronous copy takes, through registers).  Bound by the latency of these
// reads and, at its ends, by filling and emptying the ring: 64 MB of 16384 x 2048 bf16 in 20 us.  The loop over a set stays
// a loop: with the sets in registers and the end of an id unrolled into each of their rows, the kernel fetched code for
// longer than it added.
template <class V, class O, int N>
__global__ void __launch_bounds__(kThreads, 2) embed_sum_kernel(SumArgs a) {
    constexpr int X = (N + 1) / 2;
    using Piece = Pack<V, N>;
    // the threads' slots; the tokens of the chunk's places; the ids of them, of the one before and the one after
    extern __shared__ __align__(16) uint8_t ring[];
    const int threads = blockDim.x;
    int *s_at = reinterpret_cast<int*>(ring + sizeof(Piece) * kSets * kRows * threads), *s_id = s_at + a.chunk;
    let_next_start();
    wait_for_previous();
    const int *order = behind_wait(a.order), *sid = behind_wait(a.sid);
    const long long first = static_cast<long long>(blockIdx.x) * a.chunk;
    const int p0 = static_cast<int>(first), most = static_cast<int>(min(first + a.chunk, static_cast<long long>(a.T)));
    // places past the last token's hold anything: they are looked at with the number of tokens in hand
    for (int i = threadIdx.x; i < most - p0 + 2; i += threads) {
        const int p = p0 - 1 + i;
        s_id[i] = p >= 0 && p < a.T ? load(sid + p) : -1;
        if (i < most - p0) s_at[i] = load(order + p0 + i);
    }
    const int kept = load(behind_wait(a.kept)), n = min(most, kept) - p0;  // n: places of this chunk
    const int v = blockIdx.y * threads + threadIdx.x;
    __syncthreads();
    if (n <= 0 || v >= a.np) return;
    const V* dY = behind_wait(static_cast<const V*>(a.dY)) + static_cast<long long>(v) * N;
    O* dW = static_cast<O*>(a.dW) + static_cast<long long>(v) * N;
    Piece* slots = reinterpret_cast<Piece*>(ring) + threadIdx.x;
    auto fetch = [&](int p, int set) {
        const int rows = min(kRows, n - p);
        if constexpr (sizeof(Piece) >= 4) {
#pragma unroll 4
            for (int u = 0; u < rows; ++u) copy_piece(slots + (set * kRows + u) * threads, reinterpret_cast<const Piece*>(dY + s_at[p + u] * a.lddy));
        } else {
            Piece x[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) x[u] = load(reinterpret_cast<const Piece*>(dY + s_at[max(0, min(p + u, n - 1))] * a.lddy));
#pragma unroll
            for (int u = 0; u < kRows; ++u) write_piece(slots + (set * kRows + u) * threads, stay(x[u]));
        }
        // what the sums will be added to, once for each id: those of one line by all blocks queue (16384 tokens of one id, 2048
        // bf16, 87 us with one for each token and 42)
        if (a.add)
            for (int u = 0; u < rows; ++u)
                if (s_id[p + u + 1] != s_id[p + u]) asm volatile("prefetch.global.L2 [%0];" ::"l"(dW + s_id[p + u + 1] * a.ldw));
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    bool open = p0 > 0 && s_id[0] == s_id[1];  // the current id began before the chunk
    Floats<N> acc;
#pragma unroll
    for (int i = 0; i < X; ++i) acc.v[i] = make_float2(0.f, 0.f);
    for (int i = 0; i < kSets - 1; ++i) fetch(i * kRows, i);
    int set = 0;
    for (int p = 0; p < n; p += kRows) {
        fetch(p + (kSets - 1) * kRows, set == 0 ? kSets - 1 : set - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kSets - 1) : "memory");
        const Piece* x = slots + set * kRows * threads;
#pragma unroll 1
        for (int u = 0; u < min(kRows, n - p); ++u, x += threads) {
            const Floats<N> f = floats(read_piece(x));
#pragma unroll
            for (int i = 0; i < X; ++i) acc.v[i] = __fadd2_rn(acc.v[i], f.v[i]);
            const int id = s_id[p + u + 1], end = p + u + 1 == n;
            if (!end && s_id[p + u + 2] == id) continue;
            // the id ends here, or the chunk does
            const bool on = end && p0 + n < kept && s_id[n + 1] == id;
            if (open || on) {
                constexpr int Q = N < 4 ? N : 4;
                Pack<float, Q>* q = reinterpret_cast<Pack<float, Q>*>(a.part + (2LL * blockIdx.x + !open) * a.ldp + static_cast<long long>(v) * N);
#pragma unroll
                for (int i = 0; i < N / Q; ++i) {
                    Floats<Q> part;
#pragma unroll
                    for (int j = 0; j < (Q + 1) / 2; ++j) part.v[j] = acc.v[(Q + 1) / 2 * i + j];
                    write_piece(q + i, packed<float, Q>(part));
                }
            } else {
                write_sum<O, N>(a, id, v, acc);
            }
            open = false;
#pragma unroll
            for (int i = 0; i < X; ++i) acc.v[i] = make_float2(0.f, 0.f);
        }
        set = set == kSets - 1 ? 0 : set + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// One block for each chunk whose last id began in it and goes on after it.  Groups of 2^log_g threads hold the row; where
// that is less than a block, each takes every so many of the chunks, and they are added in the groups' order.  Most blocks end at once; an id
// of many chunks is bound by the latency of its reads, eight at a time.
template <class O, int N>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(SumArgs a, int log_g) {
    constexpr int X = (N + 1) / 2;
    __shared__ Floats<N> s_sum[kThreads];
    let_next_start();
    wait_for_previous();
    const int* sid = behind_wait(a.sid);
    const float* part = behind_wait(static_cast<const float*>(a.part));
    const int G = 1 << log_g, groups = kThreads >> log_g, mine = threadIdx.x >> log_g, v = blockIdx.y * G + (threadIdx.x & (G - 1));
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
    Floats<N> acc;
#pragma unroll
    for (int i = 0; i < X; ++i) acc.v[i] = make_float2(0.f, 0.f);
    if (v < a.np) {
        part += 2LL * blockIdx.x * a.ldp + static_cast<long long>(v) * N;
        auto row = [&](const float* p) { return load_floats<float, N>(p, true, 0); };
        if (mine == 0) acc = row(part + a.ldp);
        constexpr int kAhead = 8;  // rows in flight, also where there are fewer left: past the end the last again, not added
        for (int c0 = 1 + mine; c0 <= chunks; c0 += kAhead * groups) {
            Floats<N> f[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) f[u] = row(part + 2LL * min(c0 + u * groups, chunks) * a.ldp);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int i = 0; i < X; ++i) acc.v[i] = c0 + u * groups <= chunks ? __fadd2_rn(acc.v[i], f[u].v[i]) : acc.v[i];
        }
    }
    if (groups > 1) {
        s_sum[threadIdx.x] = acc;
        __syncthreads();
        for (int g = 1; g < groups && mine == 0; ++g)
#pragma unroll
            for (int i = 0; i < X; ++i) acc.v[i] = __fadd2_rn(acc.v[i], s_sum[threadIdx.x + (g << log_g)].v[i]);
    }
    if (mine == 0 && v < a.np) write_sum<O, N>(a, id, v, acc);
}

// ---------------------------------------------------------------- host side

spx_status check(int32_t T, int32_t H, int32_t V, spx_type type, int32_t id_bytes) {
    if (T < 0 || H < 0 || V < 0 || !is_float_type(type) || (id_bytes != 4 && id_bytes != 8)) return SPX_ERR_ARG;
    if (T > kMostIndex || H > kMostIndex || V > kMostIndex) return SPX_ERR_INDEX_RANGE;
    return SPX_OK;
}

template <class V, int N, bool ANY>
cudaError_t embed_launch(int T, int H, Ids x, const void* W, int64_t ldw, float scale, void* Y, int64_t ldy, cudaStream_t st) {
    const int np = (H + N - 1) / N;
    int lg = 3;
    while (lg < 8 && (1 << lg) < np) ++lg;
    const int per = (kThreads >> lg) * kTokens, bx = (T - 1) / per + 1;
    const int steps = (np + (1 << lg) - 1) >> lg, by = std::min(steps, std::max(1, 1216 / bx));
    return launch_early(embed_kernel<V, N, ANY>, dim3(bx, by), kThreads, 0, 1, st, x, T, H, lg, static_cast<const V*>(W), static_cast<long long>(ldw), scale,
                        static_cast<V*>(Y), static_cast<long long>(ldy));
}

template <class V>
spx_status embed(int T, int H, Ids x, const void* W, int64_t ldw, float scale, void* Y, int64_t ldy, cudaStream_t st) {
    const uint64_t bits = addr(W) | addr(Y) | (static_cast<uint64_t>(H) | ldw | ldy) * sizeof(V);
    spx_note_launches(1);
    if (bits % 16 == 0) return spx_cuda_status(embed_launch<V, 16 / sizeof(V), false>(T, H, x, W, ldw, scale, Y, ldy, st));
    if (bits % 4 == 0) return spx_cuda_status(embed_launch<V, 4 / sizeof(V), false>(T, H, x, W, ldw, scale, Y, ldy, st));
    if constexpr (sizeof(V) == 2) return spx_cuda_status(embed_launch<V, 8, true>(T, H, x, W, ldw, scale, Y, ldy, st));
    return SPX_ERR_ALIGN;
}

// A block's threads for rows of np pieces.
int sum_threads(long long np) { return static_cast<int>(std::min<long long>(kThreads, std::max(1LL, (np + 31) / 32) * 32)); }

// Sorted tokens a chunk, 8 to 1024: as many chunks as run at once, of 16-byte pieces of two-byte values.  Short rows take
// smaller blocks and so more of them (16384 tokens of 512 bf16 of 30000 ids, added: 31 us with blocks of 256, 18 so; of 1024 values 33 and 24).
constexpr int kSumBlocks = 304;
int chunk_of(int T, int H) {
    const long long np = (H + 7LL) / 8, tiles = (np + kThreads - 1) / kThreads, blocks = kSumBlocks * kThreads / sum_threads(np);
    return static_cast<int>(std::min<long long>(kMostChunk, std::max(8LL, (T * tiles + blocks - 1) / blocks)));
}

struct Scratch {
    size_t order, sid, kept, part, bytes;
    long long ldp;
};
Scratch scratch_of(int T, int H) {
    Scratch s{};
    const size_t ints = (static_cast<size_t>(T) * 4 + 15) / 16 * 16;
    s.order = 0, s.sid = ints, s.kept = 2 * ints, s.part = 2 * ints + 16;
    s.ldp = (static_cast<long long>(H) + 3) / 4 * 4;
    const size_t chunk = chunk_of(T, H), chunks = (T + chunk - 1) / chunk;
    s.bytes = s.part + chunks * 2 * static_cast<size_t>(s.ldp) * sizeof(float);
    return s;
}

template <class V, class O, int N>
cudaError_t sums(SumArgs a, int T, cudaStream_t st) {
    const unsigned chunks = (T + a.chunk - 1) / a.chunk;
    const int threads = sum_threads(a.np);
    constexpr size_t piece = sizeof(V) * N * kSets * kRows;
    cudaError_t e = spx_tc::set_smem_limit(embed_sum_kernel<V, O, N>, piece * kThreads + sizeof(int) * (2 * kMostChunk + 2));
    if (e == cudaSuccess)
        e = launch_early(embed_sum_kernel<V, O, N>, dim3(chunks, (a.np + threads - 1) / threads), threads, piece * threads + sizeof(int) * (2 * a.chunk + 2), 1, st, a);
    if (e != cudaSuccess || chunks < 2) return e;
    // the kept sums in pieces of four: more threads, each with more of them in flight
    constexpr int J = N < 4 ? N : 4;
    a.np = a.np * (N / J);
    // two shares of the chunks at least (16384 tokens of one id, 2048 bf16, 18 us less than one; four shares 8 less again, but
    // with ordinary ids 1 us more)
    int log_g = 5;
    while ((1 << log_g) < std::min(a.np, kThreads / 2)) ++log_g;
    while (((a.np - 1) >> log_g) >= kMostGridY) ++log_g;  // rows past 8388480 values in pieces of one: one share
    return launch_early(embed_join_kernel<O, J>, dim3(chunks, ((a.np - 1) >> log_g) + 1), kThreads, 0, 1, st, a, log_g);
}

template <class V, class O>
cudaError_t sums_in_pieces(SumArgs a, int T, int H, cudaStream_t st) {
    // pieces of dY of up to 16 bytes; dW's as many values, in words of up to 16 bytes.  Rows off 16-byte boundaries go in
    // pieces of two 16-bit values or of one value (16384 tokens of 2048 bf16 61 us, of 2046 78, of 2047 113).
    uint64_t bits = addr(a.dY) | (static_cast<uint64_t>(H) | a.lddy) * sizeof(V);
    const uint64_t w = addr(a.dW) | (static_cast<uint64_t>(H) | a.ldw) * sizeof(O);
    const int N = copy_width(bits, sizeof(V)) / sizeof(V), M = copy_width(w, sizeof(O)) / sizeof(O);
    constexpr int N16 = 16 / sizeof(V), M16 = 16 / sizeof(O);
    if (N == N16 && M >= std::min(N16, M16)) {
        a.np = H / N16;
        return sums<V, O, N16>(a, T, st);
    }
    if constexpr (sizeof(V) == 2) {
        if (N >= 2 && M >= 2) {
            a.np = H / 2;
            return sums<V, O, 2>(a, T, st);
        }
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
    if (H > kMostGridY * kThreads) return SPX_ERR_UNSUPPORTED;
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
    o.kept = reinterpret_cast<int*>(base + s.kept);
    o.dW = accumulate ? nullptr : dW;
    o.ldw = static_cast<long long>(lddw * wb), o.row = static_cast<long long>(H * wb);
    const int blocks = std::max(152, (V + kMostIds - 1) / kMostIds);
    o.per = (V + blocks - 1) / blocks;
    const dim3 grid((V + o.per - 1) / o.per);
    const bool joins = T > chunk_of(T, H);
    spx_note_launches(T == 0 ? 1 : joins ? 3 : 2);
    const size_t smem = sizeof(int) * (kBatch + 2 * kList + o.per) + sizeof(uint16_t) * (kOrderWarps * ((o.per + 1) | 1) + 2);
    cudaError_t e = spx_tc::set_smem_limit(embed_order_kernel, 200 * 1024);
    if (e == cudaSuccess) e = launch_early(embed_order_kernel, grid, kOrderThreads, smem, 1, st, o);
    if (e != cudaSuccess || T == 0) return spx_cuda_status(e);
    SumArgs a{};
    a.chunk = chunk_of(T, H), a.T = T;
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
