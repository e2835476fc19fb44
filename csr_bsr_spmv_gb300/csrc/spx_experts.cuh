// spx_experts.cuh -- what the routed-expert kernels share: element types and
// their conversions, the tested row range of an expert, the alignment of rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "spx_check.cuh"
#include "spx_internal.h"

namespace spx_exp {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

template <class V>
__device__ __forceinline__ V from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
    return __float2half_rn(v);
}

// Four 8-bit codes (bytes of w) as fp16: 0x6400 | u is 1024 + u for a byte u,
// and u = code + 128 after flipping its top bit, so one subtraction is exact.
__device__ __forceinline__ uint2 widen_codes(uint32_t w) {
    w ^= 0x80808080u;
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The calls of a layer follow one another on a stream and run for a few
// microseconds each, so every kernel waits for the one before -- all of it --
// only when it is about to touch global memory, and the short ones let the next
// be scheduled early (programmatic dependent launch): the launch and the set-up
// overlap the kernel before (sort, gather and return of 16384 x 4 x 2048 bf16
// 125 -> 118 us).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Such a kernel is on its SM while the calls before it still write what it is
// going to read.  The read-only path (__ldg, const __restrict__) is for memory
// that nobody writes during the kernel's life, so every read of an array is a
// coherent load, from an address that passed behind_wait() after
// wait_for_previous(): the compiler cannot know that address sooner, and may
// still batch and move the loads (volatile ones took 55 us for 36 in the
// quantisation of 16384 x 4096 bf16, 8.9 for 6.1 in the 8-bit product of 8 rows
// x 4096 x 4096).
template <class T>
__device__ __forceinline__ T* behind_wait(T* p) {
    asm volatile("" : "+l"(p));
    return p;
}

// Words of a size that a load or store moves as one.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using T = uint4;
};
template <>
struct Word<8> {
    using T = uint2;
};
template <>
struct Word<4> {
    using T = uint32_t;
};
template <>
struct Word<2> {
    using T = uint16_t;
};
template <>
struct Word<1> {
    using T = uint8_t;
};

template <class T>
__device__ __forceinline__ T load(const T* p) {
    const auto w = __ldca(reinterpret_cast<const typename Word<sizeof(T)>::T*>(p));
    T v;
    memcpy(&v, &w, sizeof(T));
    return v;
}
// The same for data that is not read again.
template <class T>
__device__ __forceinline__ T load_once(const T* p) {
    const auto w = __ldcs(reinterpret_cast<const typename Word<sizeof(T)>::T*>(p));
    T v;
    memcpy(&v, &w, sizeof(T));
    return v;
}

// The checked build's error word, one in every translation unit with kernels.
static __device__ int g_experts_check;
static __device__ __forceinline__ void check_fail() { atomicExch(&g_experts_check, 1); }

// Rows [lo, hi) of expert e, whatever the offsets hold: inside [0, S], lo <= hi.
__device__ __forceinline__ void expert_rows(const int* offsets, int e, int S, int& lo, int& hi) {
    const int* o = behind_wait(offsets);
    const int a = load(o + e), b = load(o + e + 1);
    if (SPX_CHECKED && !(0 <= a && a <= b && b <= S)) check_fail();
    lo = min(max(a, 0), S);
    hi = min(max(b, lo), S);
}

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st,
                         A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Slots, rows and row lengths stay below 2^31 by more than a grid's threads or
// a CTA's slots, so that an int index that steps past its end does not wrap.
constexpr int64_t kMostIndex = kI32Max - (1 << 23);

inline size_t type_bytes(spx_type t) { return t == SPX_F32 ? 4 : t == SPX_I8 ? 1 : 2; }
inline bool is_float_type(spx_type t) { return t == SPX_F32 || t == SPX_BF16 || t == SPX_F16; }
inline bool is_half_type(spx_type t) { return t == SPX_BF16 || t == SPX_F16; }

// Largest of 16, 8, ..., `least` bytes that divides all of them.
inline int copy_width(uint64_t bits, int least) {
    int v = 16;
    while (v > least && bits % v) v >>= 1;
    return v;
}
inline uint64_t addr(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }

}  // namespace spx_exp

namespace spx_exp {

// Row tile `tile` of height TM over the experts' rows, experts in order, the
// rows from offsets[E] on as one more "expert" E: which expert, its rows
// [r0, hi).  False when there is no such tile.  One full warp.
__device__ __forceinline__ bool warp_find_tile(const int* offsets, int E, int S, int TM, int tile, int& e,
                                               int& r0, int& hi) {
    const int lane = threadIdx.x & 31;
    constexpr int P = 4;  // experts a lane looks at in a round, their offsets read side by side
    int base = 0;
    for (int e0 = 0; e0 <= E; e0 += 32 * P) {
        int lo[P], up[P], n = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int x = e0 + lane * P + i;
            lo[i] = up[i] = 0;
            if (x < E) expert_rows(offsets, x, S, lo[i], up[i]);
            else if (x == E) lo[i] = min(max(load(behind_wait(offsets) + E), 0), S), up[i] = S;
            n += (up[i] - lo[i] + TM - 1) / TM;
        }
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const unsigned at = __ballot_sync(0xffffffffu, tile < base + inc);
        if (at) {
            const int src = __ffs(at) - 1;
            int first = base + inc - n, x = e0 + lane * P, r = 0, h = 0;  // the answer is that of lane src
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int m = (up[i] - lo[i] + TM - 1) / TM;
                if (h == 0 && tile < first + m) {
                    r = lo[i] + (tile - first) * TM;
                    h = up[i];
                    x = e0 + lane * P + i;
                    if (tile < first) r = h = 0;  // only sums of wrong offsets that passed int32
                }
                first += m;
            }
            e = __shfl_sync(0xffffffffu, x, src);
            r0 = __shfl_sync(0xffffffffu, r, src);
            hi = __shfl_sync(0xffffffffu, h, src);
            return r0 < hi;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// No more row tiles than this, whatever the offsets.
inline long long max_row_tiles(int E, int S, int TM) { return (S + TM - 1) / TM + static_cast<long long>(E) + 1; }

// Sums in plain CUDA-core arithmetic, for arrays the copy engine cannot read
// (rows or bases off 16-byte boundaries): spx_experts_simt.cu.
struct SimtGemm {
    const void *L, *R;             // the factors: out[i, j] = sum_r L(i, r) * R(j, r)
    long long li, lr, rj, rr, re;  // element strides; re: of R between experts
    void* C;
    long long ldc, ce;             // row pitch of C, and its stride between experts
    const int* offsets;
    int E, S, NI, NJ, NR;          // rows of experts run over i (by_rows) or over r
    bool by_rows;
};
spx_status simt_gemm(const SimtGemm& g, spx_type type, spx_type c_type, cudaStream_t st);

// The tensor-core form (spx_experts_tc.cu) of the product and of the weights'
// gradient, for rows the copy engine can read: 16-byte aligned bases, row
// pitches and expert strides that are multiples of 8 values.
bool tc_product_fits(const void* A, int64_t lda, const void* W, int64_t ldw, int64_t stride_w, int E);
spx_status tc_product(int E, int S, int N, int K, const int* offsets, const void* A, int64_t lda, const void* W,
                      int64_t ldw, int64_t stride_w, spx_w_layout layout, spx_type type, void* C, int64_t ldc,
                      spx_type c_type, cudaStream_t st);
spx_status tc_product_i8(int E, int S, int N, int K, const int* offsets, const void* Q, int64_t ldq,
                         const float* row_scale, const void* W, int64_t ldw, int64_t mats, const float* col_scale,
                         void* C, int64_t ldc, spx_type c_type, cudaStream_t st);
// The same from the 8-bit codes themselves, for rows on 16-byte boundaries.
bool tc_codes_fit(const int8_t* Q, int64_t ldq, const int8_t* W, int64_t ldw, int64_t stride_w);
spx_status tc_product_codes(int E, int S, int N, int K, const int* offsets, const int8_t* Q, int64_t ldq,
                            const float* row_scale, const int8_t* W, int64_t ldw, int64_t stride_w,
                            const float* col_scale, void* C, int64_t ldc, spx_type c_type, cudaStream_t st);
bool tc_wgrad_fits(const void* G, int64_t ldg, const void* A, int64_t lda);
spx_status tc_wgrad(int E, int S, int N, int K, const int* offsets, const void* G, int64_t ldg, const void* A,
                    int64_t lda, spx_type type, void* dW, int64_t ldw, int64_t stride_w, spx_type w_type,
                    cudaStream_t st);

}  // namespace spx_exp
