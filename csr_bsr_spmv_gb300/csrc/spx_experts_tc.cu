// spx_experts_tc.cu -- the experts' products and their weight gradients on the
// sm_103a tensor cores (tcgen05 + TMEM, TMA-fed), 16-bit factors, fp32 sums.
//
// One kernel body, three ways the factors lie in memory:
//   kNK  C[p, n] = sum_k A[p, k] W_e[n, k]      both with k contiguous (K-major)
//   kKN  C[p, n] = sum_k A[p, k] W_e[k, n]      the weights with n contiguous (MN-major)
//   kWG  dW_e[n, k] = sum_p G[p, n] A[p, k]     both MN-major, the reduction runs over the expert's rows
// and three that the sums are stored: as they are, through the experts' gate,
// or through its gradient (Epilogue in spx_act.cuh).
// The MMA computes the transposed tile: its 128 lanes (256 for a CTA pair)
// run along the output's contiguous axis -- n, or k for kWG -- and its columns
// along the output's rows -- tokens, or n for kWG.  So each TMEM lane is one
// output column; and the ragged number of an expert's rows is the MMA's N, which
// comes in steps of 16, so a short last tile costs the time of its own rows, not
// of a whole tile, and a handful of decoded tokens runs on the same kernel as a
// prefill batch.
//
// Persistent: each CTA (pair) walks a static list of tiles; two TMA warps keep
// a ring of 64-deep stages filled across tiles, one thread issues the MMAs into
// one of two TMEM accumulators, eight warps store the other one.  The tile list
// comes from the offsets on the device: nothing waits for the host.
//
// What bounds it, measured: whole 256 x 256 tiles of a CTA pair run at the
// tensor rate (32768 rows x 2048 x 4096 over 16 experts, even: 286 us, 1922
// TFLOP/s; tensor pipe 85 to 88% active in ncu, uneven, 298 us), repeated for
// tens of milliseconds at the power limit (335 us, 8192^3 566 rested and 650 to
// 680 repeated).  Few rows are bound by the weights' bytes (32 rows, 23 experts
// of 2048 x 2048 hit: 34 us, 5.6 TB/s), the smallest by a fixed cost (16 rows x
// 128 x 64: 4.6 us), a weight gradient over few rows by its stores (64 experts of
// 2048 x 2048, 16 or 32 rows each: 537 MB of gradients in 107 us; filling that
// memory takes 132), or by clearing what a last step of 16 rows does not hold (12
// rows each 111, 8 130, 1 155).  The gate costs the product little (358 to 365 us
// repeated for 32768 rows x 2 x 2048 of 2048 over 16 experts; tensor pipe 83% active).  The
// gate's gradient is bound by what its storing warps do for each sum, beside
// MMAs of only 2048 terms: 228 to 237 us for 32768 x 2048 of 2048 (tensor pipe 64%
// active, DRAM 54%), 183 with the sums stored as they are;
// 349 with 8 storing warps that read H when a chunk's turn came.
//
// Every mbarrier wait is bounded; on expiry the CTA records an error word
// (read by spx_last_device_error), stops, waits (bounded) for its copies and
// MMAs in flight, frees its TMEM and exits.
#include <algorithm>
#include <tuple>

#include "spx_act.cuh"
#include "spx_experts.cuh"
#include "spx_experts_tile.h"
#include "spx_tc.cuh"

using namespace spx_exp;
using namespace spx_tc;

namespace {

enum Mode : int { kNK = 0, kKN = 1, kWG = 2 };

// Warps: 8 that store (two for each quarter of the lanes, taking turns at the
// tile's rows), one for the lane factor's copies, one for the MMAs, one for
// the column factor's copies.  The gate's gradient, which reads two values and
// writes three for every sum, takes 16 storing warps to hide their latency.
constexpr int kWidenWarps = 8;  // FUSE
template <bool SPLIT, int EPI>
constexpr int kStoreWarpsOf = EPI == kGateGrad && !SPLIT ? 16 : 8;
template <bool SPLIT, bool FUSE, int EPI>
constexpr int kThreadsOf = 32 * (kStoreWarpsOf<SPLIT, EPI> + 3 + (FUSE ? kWidenWarps : 0));
constexpr uint32_t kLaneBytes = 128 * kDepth * 2;  // a stage's lane factor: 128 lanes a CTA, 16 KB
constexpr uint32_t kBox = 64 * kDepth * 2;      // an MN-major box: 64 long, 64 deep, 8 KB
constexpr int kMaxStages = 12;
// 8-bit codes are held as fp16, exactly; a product is at most 2^14 and an fp32
// sum of 1024 of them at most 2^24, so every partial sum up to there is an
// exact whole number.  Longer sums go to int32 every 1024 terms, in
// registers or, with a shared reduction, in shared memory.
constexpr int kExact = 1024;
constexpr int kBand = 8;                        // row tiles that run side by side before the next lane tile
constexpr size_t kSmemMax = 224 * 1024;         // dynamic shared memory of a CTA
template <bool SPLIT, int EPI>
constexpr size_t kSmemOf = EPI == kGateGrad && !SPLIT ? 226 * 1024 : kSmemMax;  // leaves the gate's gradient six stages of pairs
// Cycles of a wait, about a second; and as some waits last as long as a tile's
// reduction (the storing warps', a pair's second CTA's for the last stage, those
// of CTAs that share a reduction for each other), so many more for each of its
// stages, which take 350 to 1165.  Only a broken pipeline reaches the sum.
constexpr long long kSpinLimit = 2000000000LL, kStageLimit = 8192;

enum : int { kErrFull = 1, kErrEmpty = 2, kErrAcc = 3, kErrDrain = 4 };

__device__ int g_experts_error;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_experts_error, 0, code); }

// Division of 0 <= n < 2^31 by a number known at the launch: a multiply, an
// add and a shift (m = 2^32 (2^s - d) / d + 1 rounded down, s = ceil(log2 d)).
struct Divisor {
    uint32_t d = 1, m = 1, s = 0;
    Divisor() = default;
    explicit Divisor(uint32_t v) : d(v) {
        while ((1ull << s) < v) ++s;
        m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - v)) / v + 1);
    }
    __device__ __forceinline__ int of(int n) const {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
    }
};

struct TcArgs {
    const int* offsets;
    int E, S;
    int NL;           // output columns: the lanes' axis
    int NC;           // kWG: output rows
    int NR;           // kNK, kKN: reduction length
    int TN, log_tn;   // output rows a tile: 32 to 256, a power of two
    int max_tiles;    // kWG: the tiles; else no fewer than sound offsets give
    int stages;
    int raw_stages;   // FUSE
    uint32_t raw_bytes;
    uint32_t stage_bytes, idesc, part_off;  // part_off: the shared partial tile, behind the tile list
    int split, split_red;  // CTAs that share a tile's reduction, and the length of a share (a multiple of kDepth)
    int same_w;       // 1: every expert reads W_0
    long long spin_limit;  // cycles of a wait
    Divisor by_lane, by_group;  // lane tiles; kNK, kKN: tiles of a full band, kWG: tiles of an expert
    void* C;
    long long ldc, ce;
    spx_type c_type;
    bool wide_f;      // fp32 output with rows on 16-byte boundaries, NL a multiple of 4
    bool wide_c;      // 16-bit output with rows on 16-byte boundaries, NL a multiple of 8
    const float *row_scale, *col_scale;  // 8-bit integers: [S], [E * NL]
    Gate gate;        // kGate, kGateGrad
    spx_type h_type;
    bool wide_h;      // H and dH with rows and halves on 16-byte boundaries
    bool by16;        // kGate: F a multiple of 16, one copy a stage
};

struct Item {
    int e;            // expert (its weights' coordinate)
    int lane0;        // first output column of the tile
    int row0, rows;   // output rows [row0, row0 + rows)
    int red0, red;    // reduction range [red0, red0 + red): k, or the expert's rows
};

// The tile list in shared memory, E + 1 entries each: an expert's first row and
// the row after its last, and (kNK, kKN) its first tile; the last entry stands
// for the rows past the last expert's, and one more first tile is the count.
struct List {
    int *lo, *hi, *first;
};
inline size_t list_bytes(int E) { return sizeof(int) * (3 * static_cast<size_t>(E) + 4); }

// Tile t of the list.  kNK, kKN: an expert's tiles go in bands of kBand row
// tiles, lane tiles within a band, row tiles fastest, so that tiles that run
// together share both factors in L2.  No global read, and no division but the
// one in an expert's last, shorter band: the thread that issues the MMAs does
// this between tiles.
template <int MODE, int CG>
__device__ __forceinline__ Item tile_item(const TcArgs& a, const List& list, int t) {
    Item it;
    if (MODE == kWG) {
        it.e = a.by_group.of(t);
        const int in = t - it.e * static_cast<int>(a.by_group.d), c = a.by_lane.of(in);
        it.lane0 = (in - c * static_cast<int>(a.by_lane.d)) * 128 * CG;
        it.row0 = c * a.TN;
        it.rows = min(a.TN, a.NC - it.row0);
        it.red0 = list.lo[it.e];
        it.red = list.hi[it.e] - it.red0;
        return it;
    }
    int lo = 0, up = a.E;  // the last expert whose first tile is <= t
    while (lo < up) {
        const int mid = (lo + up + 1) >> 1;
        if (list.first[mid] <= t) lo = mid;
        else up = mid - 1;
    }
    const int r0 = list.lo[lo], r1 = list.hi[lo];
    const int in = t - list.first[lo], mt = (r1 - r0 + a.TN - 1) >> a.log_tn;
    const int band = a.by_group.of(in), inb = in - band * static_cast<int>(a.by_group.d);
    const int high = min(kBand, mt - band * kBand);
    const int nt = high == kBand ? inb / kBand : inb / high;
    it.e = lo;
    it.lane0 = nt * 128 * CG;
    it.row0 = r0 + (band * kBand + inb - nt * high) * a.TN;
    it.rows = min(a.TN, r1 - it.row0);
    it.red0 = 0;
    it.red = lo < a.E ? a.NR : 0;  // the rows past the last expert's: zeros
    return it;
}

template <int CG>
__device__ __forceinline__ uint32_t leader_addr(uint32_t local) {
    if (CG == 1) return local;
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(local));
    return r;
}

template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
            "%4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// The gate's weights (kGate): 16 rows of the gate and the same 16 of the other factor, in turn.
__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar, bool pair) {
    if (!pair)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
            "%5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void load_5d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, int v, uint32_t bar, bool pair) {
    if (!pair)
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
            "%5, %6}], [%7];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// The ring position of a role: stage and phase, stepped without a division.
// The warps that issue copies and MMAs run their loops with all lanes and
// elect one for the instruction itself: what they compute then stays in
// uniform registers, where those instructions take their operands from.  (A
// stage's MMAs take 512 cycles on a whole tile.  With the ring's stage from a
// remainder a stage cost the issuing thread about 1000 cycles, with a single
// lane's loop about 650.)
struct Ring {
    uint32_t n, s = 0, ph = 0;
    __device__ __forceinline__ explicit Ring(uint32_t stages) : n(stages) {}
    __device__ __forceinline__ void next() {
        if (++s == n) s = 0, ph ^= 1u;
    }
};

// Arrives on `bar` (of both CTAs of a pair) when the MMAs issued so far have completed.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}

// The columns an MMA takes for `rows` output rows: steps of 16, of 32 for a pair.
template <int CG>
__device__ __forceinline__ int mma_cols(int rows) {
    return (rows + 16 * CG - 1) / (16 * CG) * (16 * CG);
}

// Bounded wait for arrivals that may come from the other CTA of the pair.
template <int CG>
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, long long limit) {
    if (CG == 1) return mbar_wait(bar, parity, limit);
    long long t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (t0 == 0) t0 = clock64();
        else if (clock64() - t0 > limit) return false;
    }
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Two floats as a pair of 16-bit values, `lo` in the low half.
template <class O>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    return narrow2<O>(make_float2(lo, hi));
}

// 32 accumulator columns (output rows) of a warp's 32 lanes (output columns)
// as matrix fragments: thread t's value (h, q, i) -- v[16 h + 4 q + i] -- is
// lane 16 h + t / 4 + 8 (i / 2), column 8 q + 2 (t % 4) + i % 2.
__device__ __forceinline__ void load_frag(uint32_t taddr, uint32_t (&v)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t* r = v + 16 * h;
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16)));
    }
}

// Row pitch of a warp's transpose buffer: 64 bytes of a row and 16 of slack,
// so that neither the matrices' rows nor the reads of whole rows share banks.
constexpr uint32_t kPatchPitch = 80, kPatchBytes = 32 * kPatchPitch;

// Stores 32 output rows from it.row0 + c0 on of the output columns x .. x + 31.
// 16-bit rows on 16-byte boundaries (`wide`) go through the warp's patch of
// shared memory: stmatrix transposes 8 x 8 blocks, and each store then covers
// eight rows of 64 bytes (weight gradients of 64 experts of 2048 x 2048: 170 us,
// 182 with each value stored by itself).
template <class O>
__device__ __forceinline__ void store_rows(const TcArgs& a, const Item& it, O* C, int x, int lane, bool wide,
                                           uint32_t patch, int c0, const float (&v)[32]) {
    C += static_cast<long long>(it.row0 + c0) * a.ldc + x;
    const int rows = it.rows - c0, cols = a.NL - x;
    if constexpr (sizeof(O) == 2) {
        if (wide) {
#pragma unroll
            for (int hg = 0; hg < 4; ++hg) {
                const float* f = v + 16 * (hg >> 1) + 2 * (hg & 1);
                asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                                 patch + lane * kPatchPitch + 16 * hg),
                             "r"(pack<O>(f[0], f[1])), "r"(pack<O>(f[4], f[5])), "r"(pack<O>(f[8], f[9])),
                             "r"(pack<O>(f[12], f[13]))
                             : "memory");
            }
            __syncwarp();
            const int r = lane >> 2, p = lane & 3;
            O* q = C + r * a.ldc + 8 * p;
#pragma unroll
            for (int u = 0; u < 4; ++u, q += 8 * a.ldc) {
                uint4 w;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                             : "r"(patch + (r + 8 * u) * kPatchPitch + 16 * p)
                             : "memory");
                if (r + 8 * u < rows && 8 * p < cols) *reinterpret_cast<uint4*>(q) = w;
            }
            __syncwarp();
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int n = 16 * (i >> 4) + (lane >> 2) + 8 * ((i >> 1) & 1), r = 8 * ((i >> 2) & 3) + 2 * (lane & 3) + (i & 1);
        if (n < cols && r < rows) C[r * a.ldc + n] = from_f<O>(v[i]);
    }
}

// ---------------- the gate between the sums and what is stored
//
// Forward (kGate), a warp's 32 lanes hold 16 columns of the gate and then the
// same 16 of the other factor, so that a thread's fragments have both sums of
// an output: v[i] and v[16 + i].  A tile of 128 lanes then gives 64 columns.

// Column group hg (eight columns of a row's 32) of a warp's 32 rows to its patch, transposed.
__device__ __forceinline__ void patch_in(uint32_t patch, int lane, int hg, uint32_t q0, uint32_t q1, uint32_t q2, uint32_t q3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(patch + lane * kPatchPitch + 16 * hg),
                 "r"(q0), "r"(q1), "r"(q2), "r"(q3)
                 : "memory");
}
__device__ __forceinline__ uint4 patch_row(uint32_t patch, int r, int p) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(patch + r * kPatchPitch + 16 * p)
                 : "memory");
    return w;
}

// 32 rows from it.row0 + c0 on of the 16 columns from x on: H, and C in its type.
template <class V>
__device__ __forceinline__ void store_factors(const TcArgs& a, const Item& it, int x, int lane, uint32_t patch, int c0, const float (&v)[32]) {
    const int rows = it.rows - c0, cols = a.NL - x;
    V* H = static_cast<V*>(a.gate.H) + (it.row0 + c0) * a.gate.ldh + x;
    if (a.wide_h) {
#pragma unroll
        for (int hg = 0; hg < 4; ++hg) {
            const float* f = v + 16 * (hg >> 1) + 2 * (hg & 1);
            patch_in(patch, lane, hg, pack<V>(f[0], f[1]), pack<V>(f[4], f[5]), pack<V>(f[8], f[9]), pack<V>(f[12], f[13]));
        }
        __syncwarp();
        const int r = lane >> 2, p = lane & 3, c = 8 * (p & 1);
        V* q = H + r * a.gate.ldh + c + (p >> 1) * static_cast<long long>(a.NL);
#pragma unroll
        for (int u = 0; u < 4; ++u, q += 8 * a.gate.ldh) {
            const uint4 w = patch_row(patch, r + 8 * u, p);
            if (r + 8 * u < rows && c < cols) *reinterpret_cast<uint4*>(q) = w;
        }
        __syncwarp();
        return;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int n = (lane >> 2) + 8 * ((i >> 1) & 1), r = 8 * ((i >> 2) & 3) + 2 * (lane & 3) + (i & 1);
        if (n < cols && r < rows) H[r * a.gate.ldh + n + (i >> 4) * static_cast<long long>(a.NL)] = from_f<V>(v[i]);
    }
}

template <class O>
__device__ __forceinline__ void store_gated(const TcArgs& a, const Item& it, int x, int lane, uint32_t patch, int c0, const float (&v)[32]) {
    const int rows = it.rows - c0, cols = a.NL - x;
    O* C = static_cast<O*>(a.C) + (it.row0 + c0) * a.ldc + x;
    float f[16];
    with_act(a.gate.act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float2 c = __fmul2_rn(act_of<decltype(kind)::value>(make_float2(v[i], v[i + 1])), make_float2(v[16 + i], v[17 + i]));
            f[i] = c.x, f[i + 1] = c.y;
        }
    });
    if constexpr (sizeof(O) == 2) {
        if (a.wide_c) {
#pragma unroll
            for (int hg = 0; hg < 2; ++hg) {
                const float* g = f + 2 * hg;
                patch_in(patch, lane, hg, pack<O>(g[0], g[1]), pack<O>(g[4], g[5]), pack<O>(g[8], g[9]), pack<O>(g[12], g[13]));
            }
            __syncwarp();
            const int r = lane >> 1, p = lane & 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint4 w = patch_row(patch, r + 16 * u, p);
                if (r + 16 * u < rows && 8 * p < cols) *reinterpret_cast<uint4*>(C + (r + 16 * u) * a.ldc + 8 * p) = w;
            }
            __syncwarp();
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int n = (lane >> 2) + 8 * ((i >> 1) & 1), r = 8 * ((i >> 2) & 3) + 2 * (lane & 3) + (i & 1);
        if (n < cols && r < rows) C[r * a.ldc + n] = from_f<O>(f[i]);
    }
}

__device__ __forceinline__ void store_gate(const TcArgs& a, const Item& it, int x, int lane, uint32_t patch, int c0, const float (&v)[32]) {
    if (a.gate.H) {
        if (a.h_type == SPX_BF16) store_factors<__nv_bfloat16>(a, it, x, lane, patch, c0, v);
        else store_factors<__half>(a, it, x, lane, patch, c0, v);
    }
    if (a.c_type == SPX_F32) store_gated<float>(a, it, x, lane, patch, c0, v);
    else if (a.c_type == SPX_BF16) store_gated<__nv_bfloat16>(a, it, x, lane, patch, c0, v);
    else store_gated<__half>(a, it, x, lane, patch, c0, v);
}

// Gradient (kGateGrad): the sums are dC; both factors come from H, dH and C go
// out.  A warp takes 16 rows of its 32 columns at a time.  On wide rows both
// factors are copied ahead of the sums into the warp's two patches of shared
// memory, reach the fragments' order by ldmatrix, and what goes out takes the
// same way back.
// A patch is 16 rows of 64 bytes; piece p of row r lies at p ^ (r / 2 % 4), so that neither eight rows of one piece nor
// whole rows share banks.
constexpr uint32_t kFactorPitch = 64, kFactorBytes = 16 * kFactorPitch;
__device__ __forceinline__ uint32_t factor_at(int r, int p) { return r * kFactorPitch + 16 * (p ^ (r >> 1 & 3)); }

// Where a thread reads and writes whole pieces (r = lane / 4, p = lane % 4: rows r and r + 8, columns 8 p to 8 p + 7 of
// a warp's chunk), stepped from chunk to chunk.
struct Pieces {
    const uint16_t* h;
    uint16_t *d, *c;
    int left;    // rows of the tile from r on; none where the columns end before these
    bool live;   // rows of an expert
    __device__ __forceinline__ void start(const TcArgs& a, const Item& it, int x, int lane, int c0) {
        const int r = c0 + (lane >> 2), p = 8 * (lane & 3);
        const long long row = it.row0 + r;
        h = behind_wait(static_cast<const uint16_t*>(a.gate.H)) + row * a.gate.ldh + x + p;
        d = static_cast<uint16_t*>(a.gate.dH) + row * a.gate.lddh + x + p;
        c = static_cast<uint16_t*>(a.C) + row * a.ldc + x + p;
        left = p < a.NL - x ? it.rows - r : 0;
        live = it.e < a.E;
    }
    __device__ __forceinline__ void step(const TcArgs& a, int by) {
        h += by * a.gate.ldh, d += by * a.gate.lddh, c += by * a.ldc, left -= by;
    }
    // both factors to the warp's patches; what lies outside is not read
    __device__ __forceinline__ void fetch(const TcArgs& a, uint32_t to) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (live && 8 * i < left) {
                const uint16_t* q = h + i * 8 * a.gate.ldh;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 8 * kFactorPitch), "l"(q) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 8 * kFactorPitch + kFactorBytes), "l"(q + a.NL) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // a patch's rows to memory
    __device__ __forceinline__ void put(uint32_t from, uint16_t* to, long long ld) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(from + i * 8 * kFactorPitch) : "memory");
            if (8 * i < left) __stcs(reinterpret_cast<uint4*>(to + i * 8 * ld), w);
        }
    }
};

// 16 rows of a warp's 32 lanes: thread t's v[8 h + 4 q + i] is lane 16 h + t / 4 + 8 (i / 2), row 8 q + 2 (t % 4) + i % 2.
__device__ __forceinline__ void load_frag16(uint32_t taddr, uint32_t (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t* r = v + 8 * h;
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16)));
    }
}

// Columns 16 h to 16 h + 15 of a patch's 16 rows as fragments, and back: q[m] holds rows 8 (m % 2) + 2 (t % 4) and the
// next of column 16 h + 8 (m / 2) + t / 4.
__device__ __forceinline__ uint32_t frag_addr(uint32_t patch, int lane, int h) {
    return patch + factor_at((lane >> 3 & 1) * 8 + (lane & 7), 2 * h + (lane >> 4));
}
__device__ __forceinline__ void frag_out(uint32_t at, uint32_t (&q)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void frag_in(uint32_t at, const uint32_t (&q)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3])
                 : "memory");
}
// dG, dU and C of two outputs.
template <int ACT>
__device__ __forceinline__ void gate_grad(float2 dc, float2 g, float2 u, float2& dg, float2& du, float2& c) {
    float2 slope;
    const float2 act = act_of<ACT>(g, slope);
    dg = __fmul2_rn(__fmul2_rn(dc, u), slope);
    du = __fmul2_rn(dc, act);
    c = __fmul2_rn(act, u);
}

// 16 rows on wide rows.  The rows past the last expert's are zeros: their sums are, and so is what stands for H.
template <class V, int ACT>
__device__ __forceinline__ void store_gate_grad(const TcArgs& a, const Pieces& at, int lane, uint32_t patch, const uint32_t (&v)[16]) {
    const uint32_t piece = patch + factor_at(lane >> 2, lane & 3);  // rows r and r + 8 have the same place
    uint32_t c[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t g[4], u[4];
        const uint32_t to = frag_addr(patch, lane, h);
        frag_out(to, g);
        frag_out(to + kFactorBytes, u);
        if (!at.live) g[0] = g[1] = g[2] = g[3] = u[0] = u[1] = u[2] = u[3] = 0;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = 8 * h + 4 * (m & 1) + 2 * (m >> 1);
            float2 a0, a1, a2;
            gate_grad<ACT>(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), widen2<V>(g[m]), widen2<V>(u[m]), a0, a1, a2);
            g[m] = pack<V>(a0.x, a0.y), u[m] = pack<V>(a1.x, a1.y), c[h][m] = pack<V>(a2.x, a2.y);
        }
        __syncwarp();
        frag_in(to, g);
        frag_in(to + kFactorBytes, u);
    }
    __syncwarp();
    at.put(piece, at.d, a.gate.lddh);
    at.put(piece + kFactorBytes, at.d + a.NL, a.gate.lddh);
    __syncwarp();
    if (a.C) {
#pragma unroll
        for (int h = 0; h < 2; ++h) frag_in(frag_addr(patch, lane, h), c[h]);
        __syncwarp();
        at.put(piece, at.c, a.ldc);
        __syncwarp();
    }
}

// The same value by value.
template <class V, int ACT>
__device__ __forceinline__ void store_gate_grad_narrow(const TcArgs& a, const Item& it, int x, int lane, int c0, const uint32_t (&v)[16]) {
    const int rows = it.rows - c0, cols = a.NL - x;
    const bool live = it.e < a.E;
    const long long row = it.row0 + c0;
    V* dH = static_cast<V*>(a.gate.dH) + row * a.gate.lddh + x;
    V* C = static_cast<V*>(a.C) + row * a.ldc + x;
    const V* H = behind_wait(static_cast<const V*>(a.gate.H)) + row * a.gate.ldh + x;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int n = 16 * (i >> 3) + (lane >> 2) + 8 * ((i >> 1) & 1), r = 8 * ((i >> 2) & 1) + 2 * (lane & 3) + (i & 1);
        if (n >= cols || r >= rows) continue;
        float2 dg, du, c;
        const V* p = H + r * a.gate.ldh + n;
        gate_grad<ACT>(make_float2(__uint_as_float(v[i]), 0.f), make_float2(live ? to_f(load(p)) : 0.f, 0.f),
                       make_float2(live ? to_f(load(p + a.NL)) : 0.f, 0.f), dg, du, c);
        V* d = dH + r * a.gate.lddh + n;
        d[0] = from_f<V>(dg.x);
        d[a.NL] = from_f<V>(du.x);
        if (a.C) C[r * a.ldc + n] = from_f<V>(c.x);
    }
}

// Pitch of a shared partial tile: a row of 128 sums and four words of slack,
// so that a fragment's stores touch every bank once.
constexpr uint32_t kPartPitch = 132 * 4;

// Four values of neighbouring columns, `left` of them inside the row.
template <class O>
__device__ __forceinline__ void put_four(O* q, int left, bool wide, const float (&f)[4]) {
    if (wide) {
        if (left < 4) return;
        if constexpr (sizeof(O) == 2) *reinterpret_cast<uint2*>(q) = make_uint2(pack<O>(f[0], f[1]), pack<O>(f[2], f[3]));
        else *reinterpret_cast<float4*>(q) = make_float4(f[0], f[1], f[2], f[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) q[i] = from_f<O>(f[i]);
}

// Four sums of this lane's columns of one output row (shared reductions).
template <class O>
__device__ __forceinline__ void store_four(const TcArgs& a, long long row, int x, const float (&f)[4]) {
    put_four(static_cast<O*>(a.C) + row * a.ldc + x, a.NL - x, a.wide_c || (sizeof(O) == 4 && a.wide_f), f);
}

// The same through the gate: lanes 8 i to 8 i + 3 of a warp hold 16 columns of the gate, the next four those of the other factor.
__device__ __forceinline__ void gate_four(const TcArgs& a, const Item& it, int r, int lane, const float (&f)[4]) {
    const long long row = it.row0 + r;
    const int x = it.lane0 / 2 + 16 * (lane >> 3) + 4 * (lane & 3);
    const bool up = lane & 4;
    float c[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __shfl_xor_sync(0xffffffffu, f[i], 4);
    with_act(a.gate.act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float2 r = __fmul2_rn(act_of<decltype(kind)::value>(make_float2(f[i], f[i + 1])), make_float2(u[i], u[i + 1]));
            c[i] = r.x, c[i + 1] = r.y;
        }
    });
    if (a.gate.H) {
        const long long at = row * a.gate.ldh + x + (up ? a.NL : 0);
        if (a.h_type == SPX_BF16) put_four(static_cast<__nv_bfloat16*>(a.gate.H) + at, a.NL - x, a.wide_h, f);
        else put_four(static_cast<__half*>(a.gate.H) + at, a.NL - x, a.wide_h, f);
    }
    if (up) return;
    if (a.c_type == SPX_F32) store_four<float>(a, row, x, c);
    else if (a.c_type == SPX_BF16) store_four<__nv_bfloat16>(a, row, x, c);
    else store_four<__half>(a, row, x, c);
}

template <class V>
__device__ __forceinline__ void gate_grad_four(const TcArgs& a, const Item& it, int r, int lane, const float (&f)[4]) {
    const long long row = it.row0 + r;
    const int x = it.lane0 + 4 * lane, left = a.NL - x;
    const V* H = behind_wait(static_cast<const V*>(a.gate.H)) + row * a.gate.ldh + x;
    float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f}, dg[4], du[4], c[4];
    const bool live = it.e < a.E;
    if (live && a.wide_h && left >= 4) {
        const uint2 wg = load(reinterpret_cast<const uint2*>(H)), wu = load(reinterpret_cast<const uint2*>(H + a.NL));
        const float2 g0 = widen2<V>(wg.x), g1 = widen2<V>(wg.y), u0 = widen2<V>(wu.x), u1 = widen2<V>(wu.y);
        g[0] = g0.x, g[1] = g0.y, g[2] = g1.x, g[3] = g1.y, u[0] = u0.x, u[1] = u0.y, u[2] = u1.x, u[3] = u1.y;
    } else if (live) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) g[i] = to_f(load(H + i)), u[i] = to_f(load(H + a.NL + i));
    }
    with_act(a.gate.act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            float2 a0, a1, a2;
            gate_grad<decltype(kind)::value>(make_float2(f[i], f[i + 1]), make_float2(g[i], g[i + 1]), make_float2(u[i], u[i + 1]), a0, a1, a2);
            dg[i] = a0.x, dg[i + 1] = a0.y, du[i] = a1.x, du[i + 1] = a1.y, c[i] = a2.x, c[i + 1] = a2.y;
        }
    });
    V* d = static_cast<V*>(a.gate.dH) + row * a.gate.lddh + x;
    put_four(d, left, a.wide_h, dg);
    put_four(d + a.NL, left, a.wide_h, du);
    if (a.C) put_four(static_cast<V*>(a.C) + row * a.ldc + x, left, a.wide_c, c);
}

__device__ __forceinline__ void store_chunk(const TcArgs& a, const Item& it, long long off, int x, int lane,
                                            uint32_t patch, int c0, const float (&v)[32]) {
    if (a.c_type == SPX_F32) store_rows(a, it, static_cast<float*>(a.C) + off, x, lane, false, patch, c0, v);
    else if (a.c_type == SPX_BF16)
        store_rows(a, it, static_cast<__nv_bfloat16*>(a.C) + off, x, lane, a.wide_c, patch, c0, v);
    else store_rows(a, it, static_cast<__half*>(a.C) + off, x, lane, a.wide_c, patch, c0, v);
}

// FUSE: the factors are 8-bit codes.  Their bytes arrive in a ring of raw
// stages, and eight more warps widen them to fp16 into the ring the MMAs read.
// The weights then cost one byte each wherever they come from, against five
// through a widened copy in memory; but the widening bounds a stage: 900 cycles
// with 32 rows, 985 with 64, 1165 with 128 (from the time's slope over K).
// SPLIT: a cluster of a.split CTAs shares each tile, every one the products of
// its part of the reduction; the partial tiles meet in shared memory, where
// CTA r adds the parts of its share of the rows in rank order.
template <int MODE, int CG, bool I8, bool SPLIT, bool FUSE, int EPI>
__global__ void __launch_bounds__(kThreadsOf<SPLIT, FUSE, EPI>, 1)
    experts_tc_kernel(const __grid_constant__ CUtensorMap tm_lane, const __grid_constant__ CUtensorMap tm_col,
                      const __grid_constant__ TcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ uint32_t s_issued, s_issued_col, s_consumed, s_tails_in, s_tails_done;
    __shared__ __align__(8) uint64_t s_bars[6 * kMaxStages + 7];

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bars = smem_u32(s_bars);
    auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bars + 8u * (kMaxStages + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (2 * kMaxStages + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (2 * kMaxStages + 2 + b); };
    const uint32_t fin_bar = bars + 8u * (2 * kMaxStages + 4);
    // kWG: a last stage that ends inside a step of 16 rows lands on its own CTA's tail_bar; both CTAs clear the
    // rows past the expert's and arrive on the first one's clear_bar.  One of each a ring stage: several short
    // reductions can be in the ring at once, but a stage is not filled again before it was consumed.
    auto tail_bar = [&](uint32_t s) { return bars + 8u * (2 * kMaxStages + 5 + s); };
    auto clear_bar = [&](uint32_t s) { return bars + 8u * (3 * kMaxStages + 5 + s); };
    // SPLIT: every part of a tile is in place; everybody has read this CTA's
    const uint32_t ready_bar = bars + 8u * (4 * kMaxStages + 5), done_bar = bars + 8u * (4 * kMaxStages + 6);
    // FUSE: a raw stage has arrived, has been read
    auto raw_full = [&](uint32_t s) { return bars + 8u * (4 * kMaxStages + 7 + s); };
    auto raw_empty = [&](uint32_t s) { return bars + 8u * (5 * kMaxStages + 7 + s); };
    const uint32_t NS = a.stages, NR = a.raw_stages;
    constexpr int SW = kStoreWarpsOf<SPLIT, EPI>;
    constexpr uint32_t PATCH = EPI == kGateGrad ? 2 * kFactorBytes : kPatchBytes;  // a storing warp's
    // the storing warps' patches, then the tile list, behind the ring
    List list;
    const uint32_t raw0 = base + NS * a.stage_bytes;  // FUSE: the raw ring
    const uint32_t behind = raw0 + (FUSE ? NR * a.raw_bytes : 0);
    list.lo = reinterpret_cast<int*>(smem_raw + (behind - smem_u32(smem_raw)) + (SPLIT ? 0 : SW * PATCH));
    list.hi = list.lo + a.E + 1;
    list.first = list.hi + a.E + 1;

    constexpr int LOAD = SW, MMA = SW + 1, LOAD2 = SW + 2;  // the roles' warps
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    int rank = 0, part = 0;  // place in the pair, share of the reduction
    if (CG == 2) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (SPLIT) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(part));
    const int team = SPLIT ? a.split : CG;
    const int G = static_cast<int>(gridDim.x) / team, me = static_cast<int>(blockIdx.x) / team;
    // Bounded wait by a whole warp, with one answer for all lanes.
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.spin_limit)) != 0;
    };
    // The same, that also ends when another warp gave up.  The flag is part of the vote: lanes may look at it at
    // different times, and a warp that left its loop in part would hang at the next vote or election.
    auto warp_wait_live = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.spin_limit) && !s_abort) != 0;
    };
    // this CTA's part of a tile's reduction
    auto share = [&](Item it) {
        if (SPLIT) {
            it.red0 = part * a.split_red;
            it.red = max(0, min(it.red - it.red0, a.split_red));
        }
        return it;
    };
    const uint32_t tmem_cols = 2u * a.TN;  // two accumulators

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < NS; ++s) {
            mbar_init(full_bar(s), FUSE ? kWidenWarps / 2 : 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), SW * CG);  // one arrive per storing warp of the pair
        }
        mbar_init(fin_bar, 1);
        if (SPLIT) {
            mbar_init(ready_bar, SW * a.split);
            mbar_init(done_bar, SW * a.split);
        }
        if (FUSE)
            for (uint32_t s = 0; s < NR; ++s) {
                mbar_init(raw_full(s), 1);
                mbar_init(raw_empty(s), kWidenWarps);
            }
        if (MODE == kWG)
            for (uint32_t s = 0; s < NS; ++s) {
                mbar_init(tail_bar(s), 1);
                mbar_init(clear_bar(s), CG);
            }
        s_abort = 0;
        s_issued = s_issued_col = s_consumed = s_tails_in = s_tails_done = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == MMA) {
        if (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                         "r"(tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                         "r"(tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    // (The next kernel is not let in early: its blocks beside this one's cost more than its launch, 224 us for the 8-bit
    // prefill product against 215.)
    wait_for_previous();
    int ntiles = a.max_tiles;  // kWG: every expert's tiles, rows or not
    for (int e = threadIdx.x; e <= a.E; e += kThreadsOf<SPLIT, FUSE, EPI>) {
        int lo = 0, hi = a.S;
        if (a.offsets) {
            if (e < a.E) expert_rows(a.offsets, e, a.S, lo, hi);
            else lo = min(max(load(behind_wait(a.offsets) + a.E), 0), a.S);
        } else if (e == a.E) {
            lo = hi;
        }
        list.lo[e] = lo;
        list.hi[e] = hi;
    }
    if (MODE != kWG) {
        __syncthreads();
        if (warp == 0) {
            long long carry = 0;
            for (int e0 = 0; e0 <= a.E; e0 += 32) {
                const int e = e0 + lane;
                const long long n = e <= a.E ? ((list.hi[e] - list.lo[e] + a.TN - 1) >> a.log_tn) * static_cast<long long>(a.by_lane.d) : 0;
                long long inc = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const long long up = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += up;
                }
                if (e <= a.E) list.first[e] = static_cast<int>(carry + inc - n);
                carry += __shfl_sync(0xffffffffu, inc, 31);
            }
            // offsets out of order can overlap and give more tiles than rows: then none is run
            if (lane == 0) list.first[a.E + 1] = carry <= a.max_tiles ? static_cast<int>(carry) : 0;
        }
    }
    tc_fence_before();
    if (CG == 2 || SPLIT) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    const uint32_t full0 = leader_addr<CG>(full_bar(0));
    if (MODE != kWG) ntiles = uniform(list.first[a.E + 1]);
    const uint32_t buf_cols = tmem_cols / 2;

    if (warp == LOAD || warp == LOAD2) {
        // ---------------- producers: this CTA's part of every stage, one thread for each factor (a thread takes
        // about 250 cycles from one copy to the next, so one alone would hold up the MMAs)
        const bool lanes = warp == LOAD;
        Ring ring(FUSE ? NR : NS);
        uint32_t issued = 0, tails = 0;
        bool ok = true;
        constexpr int depth = FUSE ? kRawDepth : kDepth;
        for (int t = me; t < ntiles && ok; t += G) {
            const Item it = share(tile_item<MODE, CG>(a, list, t));
            const int cols = MODE == kWG ? a.TN : mma_cols<CG>(it.rows);  // a pair's CTA holds half of them
            const int lane0 = uniform(it.lane0) + 128 * rank, col0 = uniform(it.row0 + rank * cols / 2);
            const int z = a.same_w ? 0 : uniform(it.e), r0 = uniform(it.red0), end = r0 + uniform(it.red);
            for (int r = r0; r < end; r += depth, ring.next(), ++issued) {
                const uint32_t s8 = 8u * ring.s, sl = FUSE ? raw0 + ring.s * a.raw_bytes : base + ring.s * a.stage_bytes;
                const uint32_t sc = sl + (FUSE ? 128 * kRawDepth : kLaneBytes);
                ok = warp_wait_live((FUSE ? raw_empty(0) : empty_bar(0)) + s8, ring.ph ^ 1u);
                if (!ok) break;
                if (FUSE) {
                    if (!elect()) continue;
                    if (lanes) {
                        mbar_expect_tx(raw_full(0) + s8, a.raw_bytes);
                        load_3d<CG>(sl, &tm_lane, r, lane0, z, raw_full(0) + s8);
                    } else {
                        load_2d<CG>(sc, &tm_col, r, col0, raw_full(0) + s8);
                    }
                    continue;
                }
                uint32_t bar = full0 + s8;
                const bool ragged = MODE == kWG && end - r < kDepth && (end - r) % 16;
                if (ragged) {
                    bar = tail_bar(ring.s);
                    tails ^= 1u << ring.s;
                }
                if (!elect()) continue;
                if (lanes) {
                    if (ragged) {
                        if (rank == 0) mbar_arrive(full_bar(0) + s8);
                        mbar_expect_tx(bar, a.stage_bytes);
                    } else if (rank == 0) {
                        mbar_expect_tx(full_bar(0) + s8, CG * a.stage_bytes);
                    }
                    if (EPI == kGate) {
                        const int f0 = lane0 / 2;  // lane0 counts both factors
                        if (a.by16) {
                            load_5d(sl, &tm_lane, r, 0, 0, f0 / 16, z, bar, CG == 2);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) load_4d(sl + i * (kLaneBytes / 4), &tm_lane, r, f0 + 16 * i, 0, z, bar, CG == 2);
                        }
                    } else if (MODE == kNK) {
                        load_3d<CG>(sl, &tm_lane, r, lane0, z, bar);
                    } else if (MODE == kKN) {
                        load_3d<CG>(sl, &tm_lane, lane0, r, z, bar);
                        load_3d<CG>(sl + kBox, &tm_lane, lane0 + 64, r, z, bar);
                    } else {
                        load_2d<CG>(sl, &tm_lane, lane0, r, bar);
                        load_2d<CG>(sl + kBox, &tm_lane, lane0 + 64, r, bar);
                    }
                } else if (MODE == kWG) {
                    for (int c = 0; c < a.TN / CG; c += 64) load_2d<CG>(sc + c / 64 * kBox, &tm_col, col0 + c, r, bar);
                } else {
                    load_2d<CG>(sc, &tm_col, r, col0, bar);
                }
            }
        }
        if (lane == 0) {
            if (!ok) {
                record_error(kErrEmpty);
                s_abort = 1;
            }
            (lanes ? s_issued : s_issued_col) = issued;
            if (lanes) s_tails_in = tails;
        }
    } else if (FUSE && warp > LOAD2) {
        // ---------------- widening: raw bytes to the swizzled fp16 stages
        // four warps take the first half of every raw stage, four the second: two stages are in the making at once
        const int h = (warp - LOAD2 - 1) >> 2, w = (warp - LOAD2 - 1) & 3;
        Ring raw(NR), ring(NS);
        uint32_t taken = 0;
        bool ok = true;
        // eight rows of four 16-byte pieces a step; a quarter of a warp takes rows q and q + 4, and the two rows' halves
        // are stored in opposite order, so that neither the reads nor the stores of the swizzled rows share banks
        const int piece = lane & 3, odd = lane >> 2 & 1, row8 = odd * 4 + (lane >> 3);
        for (int t = me; t < ntiles && ok; t += G) {
            const Item it = share(tile_item<MODE, CG>(a, list, t));
            const int rows = 128 + uniform(mma_cols<CG>(it.rows));  // the lanes' rows, then the columns'
            for (int left = uniform(it.red); left > 0; left -= kRawDepth, raw.next(), ++taken) {
                ok = warp_wait(raw_full(raw.s), raw.ph);
                if (!ok) break;
                const int halves = left > 64 ? 2 : 1;
                if (h < halves) {
                    const uint32_t src = raw0 + raw.s * a.raw_bytes;
                    Ring mine = ring;
                    if (h) mine.next();
                    const uint32_t dst = base + mine.s * a.stage_bytes;
                    for (int i0 = 0; 8 * (w + 4 * i0) < rows; i0 += 4) {
                        uint4 c[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * (w + 4 * (i0 + i)) + row8;
                            if (r < rows)
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(c[i].x), "=r"(c[i].y), "=r"(c[i].z), "=r"(c[i].w)
                                             : "r"(src + 128 * r + 16 * ((4 * h + piece) ^ (r & 7)))
                                             : "memory");
                        }
                        if (i0 == 0) {
                            ok = warp_wait_live(empty_bar(mine.s), mine.ph ^ 1u);
                            if (!ok) break;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * (w + 4 * (i0 + i)) + row8;
                            if (r >= rows) break;
                            const uint2 h0 = widen_codes(c[i].x), h1 = widen_codes(c[i].y), h2 = widen_codes(c[i].z),
                                        h3 = widen_codes(c[i].w);
                            const uint4 lo = make_uint4(h0.x, h0.y, h1.x, h1.y), hi = make_uint4(h2.x, h2.y, h3.x, h3.y);
                            const uint4 a1 = odd ? hi : lo, a2 = odd ? lo : hi;
                            const uint32_t q = dst + 128 * r, i1 = (2 * piece + odd) ^ (r & 7), i2 = i1 ^ 1;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q + 16 * i1), "r"(a1.x),
                                         "r"(a1.y), "r"(a1.z), "r"(a1.w)
                                         : "memory");
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q + 16 * i2), "r"(a2.x),
                                         "r"(a2.y), "r"(a2.z), "r"(a2.w)
                                         : "memory");
                        }
                    }
                    if (!ok) break;
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full_bar(mine.s));
                }
                if (lane == 0) mbar_arrive(raw_empty(raw.s));
                ring.next();
                if (halves == 2) ring.next();
            }
        }
        if (lane == 0) {
            if (!ok) {
                record_error(kErrFull);
                s_abort = 1;
            }
            if (w == 0 && h == 0) s_consumed = taken;
        }
    } else if (warp == MMA) {
        // ---------------- MMA issuer (the pair's first CTA)
        uint32_t tails = 0;  // bit s: the phase of tail_bar(s) and clear_bar(s)
        // The rows of the next expert inside the last step of 16 of ring stage s: zeros in both factors.  Both are
        // cleared because a NaN or infinity there would survive a product with zero.
        auto clear_tail = [&](uint32_t s, int tail) {
            if (!warp_wait(tail_bar(s), (tails >> s) & 1u)) return false;
            tails ^= 1u << s;
            const uint32_t sl = base + s * a.stage_bytes;
            const int bad = (-tail) & 15, boxes = 2 + a.TN / CG / 64;
            for (int q = lane; q < bad * 8 * boxes; q += 32) {
                const uint32_t at = sl + (q / (bad * 8)) * kBox + (tail + q / 8 % bad) * 128 + q % 8 * 16;
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                 leader_addr<CG>(clear_bar(s)))
                             : "memory");
            return true;
        };
        if (rank == 0) {
            // descriptors of stage 0; a stage or a step of 16 adds to their low words (16-byte units)
            const uint64_t ad0 = MODE == kNK ? sw128_desc(base, 16u, 1024u) : sw128_desc(base, kBox, 1024u);
            const uint64_t bd0 = MODE == kWG ? sw128_desc(base + kLaneBytes, kBox, 1024u)
                                             : sw128_desc(base + kLaneBytes, 16u, 1024u);
            constexpr uint32_t a_step = (MODE == kNK ? 32u : 2048u) >> 4, b_step = (MODE == kWG ? 2048u : 32u) >> 4;
            const uint32_t stage_step = a.stage_bytes >> 4;
            Ring ring(NS);
            uint32_t consumed = 0, d = tmem, tph = 1;
            int buf = 0;
            bool ok = true;
            for (int t = me; t < ntiles && ok; t += G) {
                const Item it = share(tile_item<MODE, CG>(a, list, t));
                const uint32_t idesc = a.idesc | (uniform(MODE == kWG ? a.TN : mma_cols<CG>(it.rows)) >> 3 << 17);
                int left = uniform(it.red);
                do {  // one accumulator's worth: the whole reduction, or kExact terms of it
                    const int now = I8 ? min(left, kExact) : left;
                    left -= now;
                    ok = warp_wait_live(tempty_bar(buf), tph);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t acc = 0;
                    for (int k = now; k > 0; k -= kDepth) {
                        if (MODE == kWG && k < kDepth && (k & 15)) {
                            ok = clear_tail(ring.s, k) &&
                                 __all_sync(0xffffffffu, pair_wait<CG>(clear_bar(ring.s), ((tails >> ring.s) & 1u) ^ 1u, a.spin_limit));
                            if (!ok) break;
                        }
                        ok = warp_wait(full_bar(0) + 8u * ring.s, ring.ph);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = ad0 + ring.s * stage_step, bd = bd0 + ring.s * stage_step;
                        if (elect()) {
                            mma<CG>(d, ad, bd, idesc, acc);
                            if (k > kDepth - 16) {
#pragma unroll
                                for (uint32_t ks = 1; ks < kDepth / 16; ++ks)
                                    mma<CG>(d, ad + ks * a_step, bd + ks * b_step, idesc, 1u);
                            } else {  // the reduction's last stage: the steps that hold something
                                for (uint32_t ks = 1; 16 * static_cast<int>(ks) < k; ++ks)
                                    mma<CG>(d, ad + ks * a_step, bd + ks * b_step, idesc, 1u);
                            }
                            commit<CG>(empty_bar(0) + 8u * ring.s);
                        }
                        acc = 1;
                        ring.next();
                        ++consumed;
                    }
                    if (!ok) break;
                    if (elect()) commit<CG>(tfull_bar(buf));
                    buf ^= 1;
                    d = tmem + buf * buf_cols;
                    if (buf == 0) tph ^= 1u;
                } while (I8 && left > 0);
            }
            if (!ok && lane == 0) {
                record_error(kErrFull);
                s_abort = 1;
            }
            if (lane == 0 && !FUSE) s_consumed = consumed;
        } else if (MODE == kWG) {
            // the pair's second CTA: only its part of clearing the tails
            uint32_t at = 0;
            for (int t = me; t < ntiles && __all_sync(0xffffffffu, !s_abort); t += G) {
                const int red = tile_item<MODE, CG>(a, list, t).red;
                if ((red & 15) && !clear_tail((at + red / kDepth) % NS, red % kDepth)) {
                    if (lane == 0) {
                        record_error(kErrFull);
                        s_abort = 1;
                    }
                    break;
                }
                at = (at + (red + kDepth - 1) / kDepth) % NS;
            }
        }
        if (lane == 0) s_tails_done = tails;
    } else if (warp < SW) {
        // ---------------- storing warps: TMEM lane quarter = warp % 4
        int buf = 0;
        uint32_t tph = 0;
        auto acc_wait = [&]() {
            const bool ok = warp_wait_live(tfull_bar(buf), tph);
            if (!ok && lane == 0) {
                record_error(kErrAcc);
                s_abort = 1;
            }
            tc_fence_after();
            return ok;
        };
        auto acc_free = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1) mbar_arrive(tempty_bar(buf));
                else
                    // relaxed: a release would wait for this warp's stores to the output (1200 cycles and more);
                    // all that has to come before it are the accumulator's loads, which are complete
                    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                     leader_addr<CG>(tempty_bar(buf)))
                                 : "memory");
            }
            buf ^= 1;
            if (buf == 0) tph ^= 1u;
        };
        const uint32_t patch = behind + warp * PATCH;
        const uint32_t quarter = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        // A tile whose reduction the cluster shares: this CTA's sums to its shared partial tile, then its rows of all.
        uint32_t pph = 0;  // tiles so far, mod 2
        auto tell_all = [&](uint32_t bar) {
            __syncwarp();
            if (lane < a.split) {
                uint32_t there;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(bar), "r"(lane));
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(there) : "memory");
            }
        };
        auto meet = [&](uint32_t bar, uint32_t parity) {
            const bool ok = __all_sync(0xffffffffu, pair_wait<2>(bar, parity, a.spin_limit) && !s_abort) != 0;
            if (!ok && lane == 0) {
                record_error(kErrAcc);
                s_abort = 1;
            }
            return ok;
        };
        auto shared_tile = [&](const Item& it) {
            const Item mine = share(it);
            const uint32_t part0 = behind + a.part_off;
            if (!meet(done_bar, pph ^ 1u)) return false;
            int left = mine.red;
            bool fresh = true;
            do {
                left -= I8 ? min(left, kExact) : left;
                if (!acc_wait()) return false;
                const uint32_t src = tmem + buf * buf_cols + quarter;
#pragma unroll 1
                for (int c0 = 32 * (warp >> 2); c0 < it.rows; c0 += 64) {
                    uint32_t v[32];
                    if (mine.red > 0) {
                        load_frag(src + c0, v);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int n = 32 * (warp & 3) + 16 * (i >> 4) + (lane >> 2) + 8 * ((i >> 1) & 1);
                        const int r = c0 + 8 * ((i >> 2) & 3) + 2 * (lane & 3) + (i & 1);
                        const uint32_t at = part0 + r * kPartPitch + 4 * n;
                        uint32_t w = v[i];
                        if (I8) {
                            int whole = __float2int_rn(__uint_as_float(v[i]));
                            if (!fresh) {
                                int before;
                                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(before) : "r"(at) : "memory");
                                whole += before;
                            }
                            w = static_cast<uint32_t>(whole);
                        }
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
                    }
                }
                acc_free();
                fresh = false;
            } while (left > 0);
            tell_all(ready_bar);
            if (!meet(ready_bar, pph)) return false;
            const int per = a.TN / a.split, col = it.lane0 + 4 * lane;
            float cs[4] = {0.f, 0.f, 0.f, 0.f};
            if (I8 && it.e < a.E)
                for (int i = 0; i < 4; ++i)
                    if (col + i < a.NL) cs[i] = load(behind_wait(a.col_scale) + static_cast<long long>(it.e) * a.NL + col + i);
            for (int r = part * per + warp; r < min((part + 1) * per, it.rows); r += SW) {
                uint32_t v[4], sum[4] = {0u, 0u, 0u, 0u};
                for (int p = 0; p < a.split; ++p) {
                    uint32_t there;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(part0 + r * kPartPitch + 16 * lane), "r"(p));
                    asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                 : "r"(there)
                                 : "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum[i] = I8 ? sum[i] + v[i] : __float_as_uint(__uint_as_float(sum[i]) + __uint_as_float(v[i]));
                }
                float f[4];
                const float rs = I8 ? load(behind_wait(a.row_scale) + it.row0 + r) : 1.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[i] = !I8 ? __uint_as_float(sum[i])
                               : it.e < a.E ? static_cast<float>(static_cast<int>(sum[i])) * (rs * cs[i]) : 0.f;
                if constexpr (EPI == kGate) gate_four(a, it, r, lane, f);
                else if constexpr (EPI == kGateGrad) {
                    if (a.h_type == SPX_BF16) gate_grad_four<__nv_bfloat16>(a, it, r, lane, f);
                    else gate_grad_four<__half>(a, it, r, lane, f);
                }
                else if (a.c_type == SPX_F32) store_four<float>(a, it.row0 + r, col, f);
                else if (a.c_type == SPX_BF16) store_four<__nv_bfloat16>(a, it.row0 + r, col, f);
                else store_four<__half>(a, it.row0 + r, col, f);
            }
            tell_all(done_bar);
            pph ^= 1u;
            return true;
        };
        if constexpr (EPI == kGateGrad && !SPLIT) {
            const int first = 16 * (warp >> 2), x0 = 128 * rank + 32 * (warp & 3);
            const uint32_t piece = patch + factor_at(lane >> 2, lane & 3);  // rows r and r + 8 have the same place
            Item it{};
            Pieces at{};
            // the first rows' factors of the next tile, while this warp has none to wait for (its other rows' fetched to L2 as
            // well: 249 us for 242)
            auto begin = [&](int t) {
                if (t >= ntiles) return;
                it = tile_item<MODE, CG>(a, list, t);
                if (!a.wide_h || first >= it.rows) return;
                at.start(a, it, it.lane0 + x0, lane, first);
                at.fetch(a, piece);
            };
            begin(me);
            for (int t = me; t < ntiles; t += G) {
                if (!acc_wait()) break;
                const uint32_t src = tmem + buf * buf_cols + quarter;
                const int x = it.lane0 + x0;
                bool held = true;
#pragma unroll 1
                for (int c0 = first; c0 < it.rows; c0 += 4 * SW) {
                    uint32_t v[16];
                    if (it.red > 0) {
                        load_frag16(src + c0, v);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0u;
                    }
                    if (c0 + 4 * SW >= it.rows) {  // this warp's last look at the accumulator
                        acc_free();
                        held = false;
                    }
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();
                    with_act(a.gate.act, [&](auto kind) {
                        constexpr int ACT = decltype(kind)::value;
                        if (a.wide_h) {
                            if (a.h_type == SPX_BF16) store_gate_grad<__nv_bfloat16, ACT>(a, at, lane, patch, v);
                            else store_gate_grad<__half, ACT>(a, at, lane, patch, v);
                        } else {
                            if (a.h_type == SPX_BF16) store_gate_grad_narrow<__nv_bfloat16, ACT>(a, it, x, lane, c0, v);
                            else store_gate_grad_narrow<__half, ACT>(a, it, x, lane, c0, v);
                        }
                    });
                    if (a.wide_h && c0 + 4 * SW < it.rows) {
                        at.step(a, 4 * SW);
                        at.fetch(a, piece);
                    }
                }
                if (held) acc_free();
                begin(t + G);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else
        for (int t = me; t < ntiles; t += G) {
            const Item it = tile_item<MODE, CG>(a, list, t);
            const int x = it.lane0 + 128 * rank + 32 * (warp & 3);
            const long long off = MODE == kWG ? it.e * a.ce : 0;
            if constexpr (SPLIT) {
                if (!shared_tile(it)) break;
                continue;
            }
            if (!I8) {
                if (!acc_wait()) break;
                const uint32_t src = tmem + buf * buf_cols + quarter;
                bool held = true;
#pragma unroll 1
                for (int c0 = 32 * (warp >> 2); c0 < it.rows; c0 += 64) {
                    uint32_t v[32];
                    if (it.red > 0) {
                        load_frag(src + c0, v);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
                    if (c0 + 64 >= it.rows) {  // this warp's last look at the accumulator
                        acc_free();
                        held = false;
                    }
                    float f[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
                    if constexpr (EPI == kGate) store_gate(a, it, (it.lane0 + 128 * rank) / 2 + 16 * (warp & 3), lane, patch, c0, f);
                    else store_chunk(a, it, off, x, lane, patch, c0, f);
                }
                if (held) acc_free();
                continue;
            }
            // 8-bit integers: the exact partial sums are added in int32, scaled at the end
            const int half = warp >> 2;  // this warp's rows: every other 32 of the tile
            int sum[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[q][j] = 0;
            bool ok = true;
            int left = it.red;
            do {
                left -= min(left, kExact);
                ok = acc_wait();
                if (!ok) break;
                const uint32_t src = tmem + buf * buf_cols + quarter;
                if (it.red > 0) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c0 = 64 * q + 32 * half;
                        if (c0 >= it.rows) break;
                        uint32_t v[32];
                        load_frag(src + c0, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[q][j] += __float2int_rn(__uint_as_float(v[j]));
                    }
                }
                acc_free();
            } while (left > 0);
            if (!ok) break;
            float cs[4];  // of this thread's four lanes
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int n = x + 8 * g + (lane >> 2);
                cs[g] = it.e < a.E && n < a.NL ? load(behind_wait(a.col_scale) + static_cast<long long>(it.e) * a.NL + n) : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c0 = 64 * q + 32 * half;
                if (c0 >= it.rows) break;
                float f[32];
#pragma unroll
                for (int r = 0; r < 8; ++r) {  // this thread's eight rows of the 32
                    const int row = 8 * (r >> 1) + 2 * (lane & 3) + (r & 1);
                    const float rs = load(behind_wait(a.row_scale) + min(it.row0 + c0 + row, a.S - 1));
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int i = 16 * (g >> 1) + 4 * (r >> 1) + 2 * (g & 1) + (r & 1);
                        f[i] = it.e < a.E ? static_cast<float>(sum[q][i]) * (rs * cs[g]) : 0.f;
                    }
                }
                store_chunk(a, it, off, x, lane, patch, c0, f);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (CG == 2 || SPLIT) cluster_sync();  // the peer's waits are over too
    else __syncthreads();
    if (MODE == kWG && s_abort && warp == LOAD && lane == 0)
        for (uint32_t s = 0; s < NS; ++s)
            if (((s_tails_in ^ s_tails_done) >> s & 1u) && !mbar_wait(tail_bar(s), (s_tails_done >> s) & 1u, kSpinLimit))
                record_error(kErrDrain);
    if (s_abort && rank == 0) {
        if (warp == LOAD && lane == 0) {
            // copies issued but never consumed: wait (bounded) until each has landed (a stage that only one factor's
            // copies were issued for runs into the limit, by which time they have)
            for (uint32_t g = s_consumed; g < max(s_issued, s_issued_col); ++g)
                if (!mbar_wait(FUSE ? raw_full(g % NR) : full_bar(g % NS), (g / (FUSE ? NR : NS)) & 1u, kSpinLimit)) {
                    record_error(kErrDrain);
                    break;
                }
        } else if (warp == MMA && lane == 0) {
            // MMAs in flight: one more commit, then wait (bounded) for it
            commit<CG>(fin_bar);
            if (!mbar_wait(fin_bar, 0, kSpinLimit)) record_error(kErrDrain);
        }
    }
    __syncwarp();
    if (CG == 2 || SPLIT) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == MMA) {
        if (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols) : "memory");
    }
}

// ------------------------------------------------------------ host side

// Tensor map of up to three axes, 128-byte swizzle, a box of 128 bytes x rows (x 1).
bool make_map3(CUtensorMap* m, const void* base, spx_type type, uint64_t inner, uint64_t rows, uint64_t ld, uint64_t mats,
               uint64_t stride, uint32_t box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const uint32_t size = static_cast<uint32_t>(type_bytes(type));
    cuuint64_t dims[3] = {inner, rows, mats};
    cuuint64_t strides[2] = {ld * size, stride * size};
    cuuint32_t box[3] = {128 / size, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m,
               type == SPX_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
               : type == SPX_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
               mats ? 3 : 2,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The gate's weights, F rows of each factor: (K, 16 rows, factor, groups of 16 rows, matrix), or, where F is no multiple
// of 16, (K, F rows, factor, matrix), whose groups end with the factor.  A box is 16 rows of each factor, or four such.
bool make_gate_map(CUtensorMap* m, const void* base, spx_type type, uint64_t K, uint64_t F, uint64_t ld, uint64_t mats, uint64_t stride,
                   bool by16) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[5] = {K, by16 ? 16 : F, 2, by16 ? F / 16 : mats, mats};
    cuuint64_t strides[4] = {ld * 2, F * ld * 2, by16 ? 16 * ld * 2 : stride * 2, stride * 2};
    cuuint32_t box[5] = {kDepth, 16, 2, by16 ? 4u : 1u, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, type == SPX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, by16 ? 5 : 4,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static std::mutex mu;
    static std::map<int, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(dev);
    if (it != cache.end()) return it->second;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return cache[dev] = n;
}

// Clusters of `team` CTAs of `kernel` the device holds at once, asked once per (kernel, size, device).
int resident_teams(const void* kernel, int team, const cudaLaunchConfig_t& cfg) {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, int>, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(kernel, team, dev);
    auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    cudaLaunchConfig_t most = cfg;
    most.dynamicSmemBytes = kSmemMax;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &most) != cudaSuccess) return 0;
    return cache[key] = n;
}

// Takes the tile for a's sizes; returns the CTAs of a tile, 1 or 2.
int take_tile(TcArgs& a, Kind kind, int lanes) {
    const Tile t = choose_tile(kind, a.E, a.S, lanes, a.NC, a.NR, sm_count());
    a.TN = t.tn;
    a.split = t.split;
    a.split_red = t.split_red;
    return t.cg;
}

bool rows_aligned(const void* p, int64_t ld) { return spx_aligned(p, 16) && ld % 8 == 0; }

template <int MODE, int CG, bool I8 = false, bool SPLIT = false, bool FUSE = false, int EPI = kNone>
spx_status launch(const CUtensorMap& tl, const CUtensorMap& tc, TcArgs a, long long max_tiles, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return SPX_ERR_CUDA;
    a.wide_c = spx_aligned(a.C, 16) && a.ldc % 8 == 0 && a.ce % 8 == 0 && a.NL % 8 == 0;
    a.spin_limit = kSpinLimit + kStageLimit * ((MODE == kWG ? a.S : a.NR) / kDepth + 1);
    a.log_tn = 0;
    while ((1 << a.log_tn) < a.TN) ++a.log_tn;
    a.wide_f = spx_aligned(a.C, 16) && a.ldc % 4 == 0 && a.NL % 4 == 0;
    const int team = SPLIT ? a.split : CG;  // CTAs that work on one tile
    a.part_off = static_cast<uint32_t>((list_bytes(a.E) + 15) / 16 * 16);
    const size_t list = a.part_off + (SPLIT ? a.TN * kPartPitch : kStoreWarpsOf<SPLIT, EPI> * (EPI == kGateGrad ? 2 * kFactorBytes : kPatchBytes));
    size_t room = kSmemOf<SPLIT, EPI> - 1024 - list;
    if (FUSE) {  // stages for the MMAs, more than the widening warps fill at once where there is room, and raw ones
        a.stages = a.TN > 64 ? 2 : 4;
        room -= a.stages * a.stage_bytes;
        a.raw_stages = static_cast<int>(std::min<size_t>(kMaxStages, room / a.raw_bytes));
        room = a.raw_stages * a.raw_bytes;
    } else {
        a.stages = static_cast<int>(std::min<size_t>(kMaxStages, room / a.stage_bytes));
        room = 0;
    }
    const size_t smem = 1024 + static_cast<size_t>(a.stages) * a.stage_bytes + room + list;
    if (set_smem_limit(experts_tc_kernel<MODE, CG, I8, SPLIT, FUSE, EPI>, kSmemOf<SPLIT, EPI>) != cudaSuccess) return SPX_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreadsOf<SPLIT, FUSE, EPI>);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = team;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;  // for the question below
    cfg.numAttrs = 1;
    // as many CTAs as run at once: one an SM; teams only where a GPC has the SMs left for them
    int groups = sms;
    if (team > 1) {
        cfg.gridDim = dim3(sms / team * team);
        groups = resident_teams(reinterpret_cast<const void*>(experts_tc_kernel<MODE, CG, I8, SPLIT, FUSE, EPI>), team, cfg);
        if (groups <= 0) return SPX_ERR_CUDA;
    }
    spx_note_launches(1);
    return spx_cuda_status(launch_early(experts_tc_kernel<MODE, CG, I8, SPLIT, FUSE, EPI>,
                                        dim3(static_cast<unsigned>(std::min<long long>(max_tiles, groups)) * team),
                                        kThreadsOf<SPLIT, FUSE, EPI>, smem, team, st, tl, tc, a));
}

uint32_t idesc_of(spx_type type, int mode, int cg) {
    uint32_t d = 1u << 4;                                 // fp32 sums
    if (type == SPX_BF16) d |= (1u << 7) | (1u << 10);    // both factors bf16 (else fp16)
    if (mode != kNK) d |= 1u << 15;                       // lane factor MN-major
    if (mode == kWG) d |= 1u << 16;                       // column factor MN-major
    return d | ((128u * cg >> 4) << 24);
}

}  // namespace

int spx_experts_error_take() {
    int h = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_experts_error, sizeof(int)) != cudaSuccess) return SPX_ERR_CUDA;
    if (h != 0 && cudaMemcpyToSymbol(g_experts_error, &zero, sizeof(int)) != cudaSuccess) return SPX_ERR_CUDA;
    return h ? static_cast<int>(SPX_ERR_TIMEOUT) : 0;
}

int spx_experts_check_take() { return spx_check_take(g_experts_check); }

namespace spx_exp {

bool tc_product_fits(const void* A, int64_t lda, const void* W, int64_t ldw, int64_t stride_w, int E) {
    return rows_aligned(A, lda) && rows_aligned(W, ldw) && (E == 1 || stride_w % 8 == 0);
}

spx_status tc_product(int E, int S, int N, int K, const int* offsets, const void* A, int64_t lda, const void* W,
                      int64_t ldw, int64_t stride_w, spx_w_layout layout, spx_type type, void* C, int64_t ldc,
                      spx_type c_type, cudaStream_t st) {
    const bool nk = layout == SPX_W_NK;
    TcArgs a{};
    a.offsets = offsets, a.E = E, a.S = S, a.NL = N, a.NR = K;
    a.C = C, a.ldc = ldc, a.c_type = c_type;
    a.same_w = E == 1 || stride_w == 0;
    const int cg = take_tile(a, kProduct, N);
    a.stage_bytes = kLaneBytes + static_cast<uint32_t>(a.TN / cg) * kDepth * 2;
    a.idesc = idesc_of(type, nk ? kNK : kKN, cg);
    CUtensorMap tl, tc;
    const uint64_t mats = a.same_w ? 1 : E, sw = a.same_w ? static_cast<uint64_t>(ldw) * (nk ? N : K) : stride_w;
    const bool ok = nk ? make_map3(&tl, W, type, K, N, ldw, mats, sw, 128) : make_map3(&tl, W, type, N, K, ldw, mats, sw, 64);
    if (!ok || !make_map3(&tc, A, type, K, S, lda, 0, 0, a.TN / cg)) return SPX_ERR_CUDA;
    const long long nlt = (N + 128 * cg - 1) / (128 * cg), tiles = max_row_tiles(E, S, a.TN) * nlt;
    if (tiles > kI32Max - 4096) return SPX_ERR_INDEX_RANGE;  // the list's walk steps past its end by a grid
    a.max_tiles = static_cast<int>(tiles);
    a.by_lane = Divisor(static_cast<uint32_t>(nlt));
    a.by_group = Divisor(static_cast<uint32_t>(kBand * nlt));
    if (a.split > 1)
        return nk ? launch<kNK, 1, false, true>(tl, tc, a, tiles, st) : launch<kKN, 1, false, true>(tl, tc, a, tiles, st);
    if (cg == 2) return nk ? launch<kNK, 2>(tl, tc, a, tiles, st) : launch<kKN, 2>(tl, tc, a, tiles, st);
    return nk ? launch<kNK, 1>(tl, tc, a, tiles, st) : launch<kKN, 1>(tl, tc, a, tiles, st);
}

spx_status tc_gated(int E, int S, int F, int K, const int* offsets, const void* A, int64_t lda, const void* W, int64_t ldw, int64_t stride_w,
                    const Gate& gate, spx_type type, void* C, int64_t ldc, spx_type c_type, cudaStream_t st) {
    TcArgs a{};
    a.offsets = offsets, a.E = E, a.S = S, a.NL = F, a.NR = K;
    a.C = C, a.ldc = ldc, a.c_type = c_type;
    a.gate = gate, a.h_type = type;
    a.wide_h = gate.H && rows_aligned(gate.H, gate.ldh) && F % 8 == 0;
    a.by16 = F % 16 == 0;
    a.same_w = E == 1 || stride_w == 0;
    const int cg = take_tile(a, kProduct, 2 * F);
    a.stage_bytes = kLaneBytes + static_cast<uint32_t>(a.TN / cg) * kDepth * 2;
    a.idesc = idesc_of(type, kNK, cg);
    CUtensorMap tl, tc;
    const uint64_t mats = a.same_w ? 1 : E, sw = a.same_w ? 2 * static_cast<uint64_t>(ldw) * F : stride_w;
    if (!make_gate_map(&tl, W, type, K, F, ldw, mats, sw, a.by16) || !make_map3(&tc, A, type, K, S, lda, 0, 0, a.TN / cg)) return SPX_ERR_CUDA;
    const long long nlt = (F + 64 * cg - 1) / (64 * cg), tiles = max_row_tiles(E, S, a.TN) * nlt;
    if (tiles > kI32Max - 4096) return SPX_ERR_INDEX_RANGE;
    a.max_tiles = static_cast<int>(tiles);
    a.by_lane = Divisor(static_cast<uint32_t>(nlt));
    a.by_group = Divisor(static_cast<uint32_t>(kBand * nlt));
    if (a.split > 1) return launch<kNK, 1, false, true, false, kGate>(tl, tc, a, tiles, st);
    return cg == 2 ? launch<kNK, 2, false, false, false, kGate>(tl, tc, a, tiles, st) : launch<kNK, 1, false, false, false, kGate>(tl, tc, a, tiles, st);
}

spx_status tc_gated_grad(int E, int S, int F, int N, const int* offsets, const void* dY, int64_t lddy, const void* W, int64_t ldw,
                         int64_t stride_w, spx_w_layout layout, const Gate& gate, spx_type type, void* C, int64_t ldc, cudaStream_t st) {
    const bool nk = layout == SPX_W_NK;
    TcArgs a{};
    a.offsets = offsets, a.E = E, a.S = S, a.NL = F, a.NR = N;
    a.C = C, a.ldc = ldc, a.c_type = type;
    a.gate = gate, a.h_type = type;
    a.wide_h = rows_aligned(gate.H, gate.ldh) && rows_aligned(gate.dH, gate.lddh) && F % 8 == 0 && (!C || rows_aligned(C, ldc));
    a.same_w = E == 1 || stride_w == 0;
    const int cg = take_tile(a, kGateBack, F);
    a.stage_bytes = kLaneBytes + static_cast<uint32_t>(a.TN / cg) * kDepth * 2;
    a.idesc = idesc_of(type, nk ? kNK : kKN, cg);
    CUtensorMap tl, tc;
    const uint64_t mats = a.same_w ? 1 : E, sw = a.same_w ? static_cast<uint64_t>(ldw) * (nk ? F : N) : stride_w;
    const bool ok = nk ? make_map3(&tl, W, type, N, F, ldw, mats, sw, 128) : make_map3(&tl, W, type, F, N, ldw, mats, sw, 64);
    if (!ok || !make_map3(&tc, dY, type, N, S, lddy, 0, 0, a.TN / cg)) return SPX_ERR_CUDA;
    const long long nlt = (F + 128 * cg - 1) / (128 * cg), tiles = max_row_tiles(E, S, a.TN) * nlt;
    if (tiles > kI32Max - 4096) return SPX_ERR_INDEX_RANGE;
    a.max_tiles = static_cast<int>(tiles);
    a.by_lane = Divisor(static_cast<uint32_t>(nlt));
    a.by_group = Divisor(static_cast<uint32_t>(kBand * nlt));
    if (a.split > 1)
        return nk ? launch<kNK, 1, false, true, false, kGateGrad>(tl, tc, a, tiles, st) : launch<kKN, 1, false, true, false, kGateGrad>(tl, tc, a, tiles, st);
    if (cg == 2)
        return nk ? launch<kNK, 2, false, false, false, kGateGrad>(tl, tc, a, tiles, st) : launch<kKN, 2, false, false, false, kGateGrad>(tl, tc, a, tiles, st);
    return nk ? launch<kNK, 1, false, false, false, kGateGrad>(tl, tc, a, tiles, st) : launch<kKN, 1, false, false, false, kGateGrad>(tl, tc, a, tiles, st);
}

// The 8-bit product on codes held as fp16: Q is S x K (lda), W is mats x N x K
// (ldw rows, N * ldw apart), both 16-byte aligned.
spx_status tc_product_i8(int E, int S, int N, int K, const int* offsets, const void* Q, int64_t ldq,
                         const float* row_scale, const void* W, int64_t ldw, int64_t mats, const float* col_scale,
                         void* C, int64_t ldc, spx_type c_type, cudaStream_t st) {
    TcArgs a{};
    a.offsets = offsets, a.E = E, a.S = S, a.NL = N, a.NR = K;
    a.C = C, a.ldc = ldc, a.c_type = c_type;
    a.row_scale = row_scale, a.col_scale = col_scale;
    a.same_w = mats == 1;
    const int cg = take_tile(a, kProduct, N);
    a.stage_bytes = kLaneBytes + static_cast<uint32_t>(a.TN / cg) * kDepth * 2;
    a.idesc = idesc_of(SPX_F16, kNK, cg);
    CUtensorMap tl, tc;
    if (!make_map3(&tl, W, SPX_F16, K, N, ldw, mats, ldw * N, 128) || !make_map3(&tc, Q, SPX_F16, K, S, ldq, 0, 0, a.TN / cg))
        return SPX_ERR_CUDA;
    const long long nlt = (N + 128 * cg - 1) / (128 * cg), tiles = max_row_tiles(E, S, a.TN) * nlt;
    if (tiles > kI32Max - 4096) return SPX_ERR_INDEX_RANGE;
    a.max_tiles = static_cast<int>(tiles);
    a.by_lane = Divisor(static_cast<uint32_t>(nlt));
    a.by_group = Divisor(static_cast<uint32_t>(kBand * nlt));
    if (a.split > 1) return launch<kNK, 1, true, true>(tl, tc, a, tiles, st);
    return cg == 2 ? launch<kNK, 2, true>(tl, tc, a, tiles, st) : launch<kNK, 1, true>(tl, tc, a, tiles, st);
}

bool tc_codes_fit(const int8_t* Q, int64_t ldq, const int8_t* W, int64_t ldw, int64_t stride_w) {
    return spx_aligned(Q, 16) && spx_aligned(W, 16) && ldq % 16 == 0 && ldw % 16 == 0 && stride_w % 16 == 0;
}

spx_status tc_product_codes(int E, int S, int N, int K, const int* offsets, const int8_t* Q, int64_t ldq,
                            const float* row_scale, const int8_t* W, int64_t ldw, int64_t stride_w,
                            const float* col_scale, void* C, int64_t ldc, spx_type c_type, cudaStream_t st) {
    TcArgs a{};
    a.offsets = offsets, a.E = E, a.S = S, a.NL = N, a.NR = K;
    a.C = C, a.ldc = ldc, a.c_type = c_type;
    a.row_scale = row_scale, a.col_scale = col_scale;
    a.same_w = E == 1 || stride_w == 0;
    take_tile(a, kCodes, N);
    a.stage_bytes = kLaneBytes + static_cast<uint32_t>(a.TN) * kDepth * 2;
    a.raw_bytes = static_cast<uint32_t>(128 + a.TN) * kRawDepth;
    a.idesc = idesc_of(SPX_F16, kNK, 1);
    const uint64_t mats = a.same_w ? 1 : E, sw = a.same_w ? static_cast<uint64_t>(ldw) * N : stride_w;
    CUtensorMap tl, tc;
    if (!make_map3(&tl, W, SPX_I8, K, N, ldw, mats, sw, 128) || !make_map3(&tc, Q, SPX_I8, K, S, ldq, 0, 0, a.TN))
        return SPX_ERR_CUDA;
    const long long nlt = (N + 127) / 128, tiles = max_row_tiles(E, S, a.TN) * nlt;
    if (tiles > kI32Max - 4096) return SPX_ERR_INDEX_RANGE;
    a.max_tiles = static_cast<int>(tiles);
    a.by_lane = Divisor(static_cast<uint32_t>(nlt));
    a.by_group = Divisor(static_cast<uint32_t>(kBand * nlt));
    return launch<kNK, 1, true, true, true>(tl, tc, a, tiles, st);
}

bool tc_wgrad_fits(const void* G, int64_t ldg, const void* A, int64_t lda) {
    return rows_aligned(G, ldg) && rows_aligned(A, lda);
}

spx_status tc_wgrad(int E, int S, int N, int K, const int* offsets, const void* G, int64_t ldg, const void* A,
                    int64_t lda, spx_type type, void* dW, int64_t ldw, int64_t stride_w, spx_type w_type,
                    cudaStream_t st) {
    TcArgs a{};
    a.offsets = offsets, a.E = E, a.S = S, a.NL = K, a.NC = N;
    a.C = dW, a.ldc = ldw, a.ce = stride_w, a.c_type = w_type;
    const int cg = take_tile(a, kGradient, K);
    a.stage_bytes = kLaneBytes + static_cast<uint32_t>(a.TN / cg) * kDepth * 2;
    a.idesc = idesc_of(type, kWG, cg);
    CUtensorMap tl, tc;
    if (!make_map3(&tl, A, type, K, S, lda, 0, 0, 64) || !make_map3(&tc, G, type, N, S, ldg, 0, 0, 64))
        return SPX_ERR_CUDA;
    const long long nlt = (K + 128 * cg - 1) / (128 * cg), per = nlt * ((N + a.TN - 1) / a.TN), tiles = E * per;
    if (tiles > kI32Max - 4096) return SPX_ERR_INDEX_RANGE;
    a.max_tiles = static_cast<int>(tiles);
    a.by_lane = Divisor(static_cast<uint32_t>(nlt));
    a.by_group = Divisor(static_cast<uint32_t>(per));
    return cg == 2 ? launch<kWG, 2>(tl, tc, a, tiles, st) : launch<kWG, 1>(tl, tc, a, tiles, st);
}

}  // namespace spx_exp
