// Shared pieces of the 4-bit weight and gated feed-forward operators (sm_100a): element types,
// activations with their derivatives, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "externd.h"

namespace externd_llm {

constexpr unsigned FULL = 0xffffffffu;

// ---- element types -------------------------------------------------------------------------------

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// two fp32 values -> one register of two 16-bit values (lo in the low half)
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// ---- activations ---------------------------------------------------------------------------------
//
// silu       g s(g),                     s(g) = 1 / (1 + e^-g);     derivative s + g s (1 - s)
// gelu       g P(g),                     P the normal distribution; derivative P + g e^{-g^2/2} / sqrt(2 pi)
// gelu_tanh  g s(2y), y = sqrt(2/pi) (g + 0.044715 g^3);            derivative s + g s (1 - s) 2 y'
// relu2      max(g, 0)^2;                                           derivative 2 max(g, 0)
// e^-g overflows to +inf for g < -88: s is then 0 and g s is -0, the limit.
//
// PRECISE takes the full-precision exponential and division (fp32 results); the others are rounded to
// 16 bits, which hides the few ulp (growing with |g|) of the hardware exponential.  P is taken as
// erfc(-g / sqrt 2) / 2, which keeps its relative accuracy where P is small.

template <bool PRECISE>
__device__ __forceinline__ float sigmoid(float v) {
    if constexpr (PRECISE) return 1.0f / (1.0f + expf(-v));
    // 1 / y as computed here is 0 for y in 2^126..2^128 too (v below -87): the value there is below 1e-37
    return __fdividef(1.0f, 1.0f + __expf(-v));
}

// -inf (a sum below the fp32 range) -> the least finite value, where the activations are at their limit 0; NaN stays
__device__ __forceinline__ float not_minus_inf(float g) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(g), "f"(-FLT_MAX));
    return r;
}

template <int ACT, bool PRECISE>
__device__ __forceinline__ float act_fn(float g) {
    g = not_minus_inf(g);
    if constexpr (ACT == EXTERND_ACT_SILU) {
        return g * sigmoid<PRECISE>(g);
    } else if constexpr (ACT == EXTERND_ACT_GELU) {
        return 0.5f * g * erfcf(-0.70710678118654752f * g);
    } else if constexpr (ACT == EXTERND_ACT_GELU_TANH) {
        return g * sigmoid<PRECISE>(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f));
    } else {
        const float r = g <= 0.0f ? 0.0f : g;      // NaN stays
        return r * r;
    }
}

// activation and derivative together
template <int ACT, bool PRECISE>
__device__ __forceinline__ float2 act_both(float g) {
    if constexpr (ACT == EXTERND_ACT_SILU) {
        const float s = sigmoid<PRECISE>(g), a = g * s;
        return make_float2(a, fmaf(a, 1.0f - s, s));
    } else if constexpr (ACT == EXTERND_ACT_GELU) {
        const float p = 0.5f * erfcf(-0.70710678118654752f * g);
        return make_float2(g * p, fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p));
    } else if constexpr (ACT == EXTERND_ACT_GELU_TANH) {
        const float c = fminf(0.044715f * g * g, 1e4f);   // far past the sigmoid's end: keeps 0 * inf away
        const float s = sigmoid<PRECISE>(1.5957691216057308f * g * (1.0f + c)), a = g * s;
        return make_float2(a, fmaf(a * (1.0f - s), 1.5957691216057308f * fmaf(3.0f, c, 1.0f), s));
    } else {
        // finite where the square leaves the fp32 range, so that a gradient of 0 stays 0
        const float r = g <= 0.0f ? 0.0f : g, a = r * r, d = 2.0f * r;
        return make_float2(a > FLT_MAX ? FLT_MAX : a, d > FLT_MAX ? FLT_MAX : d);
    }
}

template <bool PRECISE>
__device__ __forceinline__ float act_rt(int act, float g) {
    switch (act) {   // uniform over the launch
        case EXTERND_ACT_SILU: return act_fn<EXTERND_ACT_SILU, PRECISE>(g);
        case EXTERND_ACT_GELU: return act_fn<EXTERND_ACT_GELU, PRECISE>(g);
        case EXTERND_ACT_GELU_TANH: return act_fn<EXTERND_ACT_GELU_TANH, PRECISE>(g);
        default: return act_fn<EXTERND_ACT_RELU2, PRECISE>(g);
    }
}

// ---- argument checks -----------------------------------------------------------------------------

inline bool valid_dtype(int t) { return t == EXTERND_F32 || t == EXTERND_F16 || t == EXTERND_BF16; }
inline size_t dtype_bytes(int t) { return t == EXTERND_F32 ? 4 : 2; }
inline bool valid_act(int a) { return a >= EXTERND_ACT_SILU && a <= EXTERND_ACT_RELU2; }
inline bool valid_group(int g) { return g == 32 || g == 64 || g == 128; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// the current device, and whether its kernels may use a pointer
struct Device {
    int id = -1;
    Device() { if (cudaGetDevice(&id) != cudaSuccess) { cudaGetLastError(); id = -1; } }
    bool holds(const void* p) const {
        cudaPointerAttributes a;
        if (id < 0 || cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == id);
    }
};

inline int sm_count() {
    int dev = 0, v = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    cudaGetLastError();
    return v;
}

// Dynamic shared memory of a kernel, set once per device of the process.  Several host threads may be the first.
using PerDevice = std::atomic<bool>[64];
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, PerDevice& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
    const bool known = dev >= 0 && dev < 64;
    if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_release);
    return e;
}

// ---- waits -----------------------------------------------------------------------------------------

constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;   // per wait, as for the factorizations

// The limit of the tile kernels' waits, and the worker whose products are withheld (counted from 1; 0: none), so that
// the waits for them run out: externd_debug_wait_fault sets both for the calls of its thread.
struct WaitFault { uint64_t limit_ns = WAIT_LIMIT_NS; int withhold = 0; };
WaitFault& wait_fault();                            // gated.cu

// ---- warp-level matrix product ---------------------------------------------------------------------
//
// d += a b for a 16 x 16 and b 16 x 8, fp32 accumulation.  Lane 4 r + c holds a's rows r and r + 8 and b's
// column r; the order of the 16 inner indices is free as long as a and b agree, so a lane takes
// consecutive elements of its row.
template <typename T> __device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                               uint32_t a3, uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- vectors as product operands -------------------------------------------------------------------

// x = hi + mid + lo with bf16 terms; infinities and NaN stay in hi
__device__ __forceinline__ void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const uint32_t u = __float_as_uint(x);
    hi = u >> 16;
    const bool special = (u & 0x7f800000u) == 0x7f800000u;
    if (special && (u & 0x007fffffu)) hi |= 0x0040u;          // a NaN whose payload sits in the low half
    const float r = special ? 0.0f : x - __uint_as_float(u & 0xffff0000u);
    mid = __float_as_uint(r) >> 16;
    const float r2 = r - __uint_as_float(__float_as_uint(r) & 0xffff0000u);
    lo = __float_as_uint(r2) >> 16;
}

// Eight consecutive 16-bit entries k .. k + 7 (k a multiple of 8) of a row; entries from n on are 0.  vec: rows
// start on 16-byte boundaries.  Otherwise, away from the row's ends, the two aligned 16-byte pieces that hold the
// entries are shifted into place.
__device__ __forceinline__ uint4 load8(const unsigned short* __restrict__ x, int64_t k, int64_t n, bool vec) {
    const unsigned short* const p = x + k;
    if (vec && k + 8 <= n) return __ldg(reinterpret_cast<const uint4*>(p));
    if (k >= 8 && k + 16 <= n) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const uint32_t off = (uint32_t)(at & 15);                        // even
        const uint4* const q = reinterpret_cast<const uint4*>(at - off);
        const uint4 a = __ldg(q), b = __ldg(q + 1);
        uint32_t w[5];                                                   // the five words from word off / 4 on
        const uint32_t word = off >> 2;
        w[0] = word == 0 ? a.x : word == 1 ? a.y : word == 2 ? a.z : a.w;
        w[1] = word == 0 ? a.y : word == 1 ? a.z : word == 2 ? a.w : b.x;
        w[2] = word == 0 ? a.z : word == 1 ? a.w : word == 2 ? b.x : b.y;
        w[3] = word == 0 ? a.w : word == 1 ? b.x : word == 2 ? b.y : b.z;
        w[4] = word == 0 ? b.x : word == 1 ? b.y : word == 2 ? b.z : b.w;
        const uint32_t sh = (off & 2) * 8;
        return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                          __funnelshift_r(w[3], w[4], sh));
    }
    uint32_t v[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = k + 2 * i < n ? __ldg(p + 2 * i) : 0;
        const uint32_t b = k + 2 * i + 1 < n ? __ldg(p + 2 * i + 1) : 0;
        v[i] = a | (b << 16);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

struct F8 { float4 a, b; };
__device__ __forceinline__ F8 load8(const float* __restrict__ x, int64_t k, int64_t n, bool vec) {
    if (vec && k + 8 <= n) return {__ldg(reinterpret_cast<const float4*>(x + k)), __ldg(reinterpret_cast<const float4*>(x + k) + 1)};
    float v[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < n ? __ldg(x + k + i) : 0.0f;
    return {make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
}

// ... as product operands: one plane of 16-bit pairs, or the three bf16 planes of fp32 entries
template <typename X> struct Raw8;
template <> struct Raw8<float> { using type = F8; static constexpr int PLANES = 3; };
template <> struct Raw8<__half> { using type = uint4; static constexpr int PLANES = 1; };
template <> struct Raw8<__nv_bfloat16> { using type = uint4; static constexpr int PLANES = 1; };

__device__ __forceinline__ void planes8(const uint4& r, uint32_t (&v)[1][4]) {
    v[0][0] = r.x; v[0][1] = r.y; v[0][2] = r.z; v[0][3] = r.w;
}
__device__ __forceinline__ void planes8(const F8& r, uint32_t (&v)[3][4]) {
    const float e[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h0, m0, l0, h1, m1, l1;
        split3(e[2 * i], h0, m0, l0);
        split3(e[2 * i + 1], h1, m1, l1);
        v[0][i] = h0 | (h1 << 16);
        v[1][i] = m0 | (m1 << 16);
        v[2][i] = l0 | (l1 << 16);
    }
}

// ---- operands whose rows do not start on 16-byte boundaries ---------------------------------------------

// Up to three matrices are laid out in rows that do, in one launch, 16 bytes a lane.  TMA needs that,
// and wide loads; such operands are odd-sized ones, a model's own sizes hardly ever come here.
// Elements count as 16-bit ones (an fp32 as two).
struct AlignJob { const unsigned short* src; int64_t lds; unsigned short* dst; int64_t ldd; int64_t rows, cols; };
struct AlignJobs { AlignJob j[3]; int count; };

// a block of 256 threads, `block` of `count`: a warp takes 256 columns of a row at a time
__device__ __forceinline__ void align_rows(const AlignJob& j, int64_t block, int64_t count) {
    const int lane = threadIdx.x & 31;
    const int64_t per = (j.cols + 255) / 256;
    for (int64_t i = block * 8 + (threadIdx.x >> 5); i < j.rows * per; i += count * 8) {
        const int64_t r = i / per, k = 256 * (i - r * per) + 8 * lane;
        if (k < j.cols) *reinterpret_cast<uint4*>(j.dst + r * j.ldd + k) = load8(j.src + r * j.lds, k, j.cols, false);
    }
}
static __global__ void __launch_bounds__(256) align_rows_kernel(const AlignJobs jobs) { align_rows(jobs.j[blockIdx.y], blockIdx.x, gridDim.x); }

inline int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
inline bool row_aligned(const void* p, int64_t rows, int64_t ld, size_t bytes) { return aligned(p, 16) && (rows < 2 || ld * bytes % 16 == 0); }
// bytes of rows x cols elements laid out in aligned rows
inline size_t plane_bytes(int64_t rows, int64_t cols, size_t bytes) {
    return ((size_t)rows * (size_t)round8(cols * (int64_t)(bytes / 2)) * 2 + 255) / 256 * 256;
}

// Where p (rows x cols elements of `bytes` bytes) has misaligned rows: give it a place at the start of the workspace
// and note the job.  false: the workspace is too small.
inline bool place_rows(AlignJobs& jobs, const void*& p, int64_t& ld, int64_t rows, int64_t cols, size_t bytes, unsigned char*& work,
                       size_t& work_bytes) {
    const int64_t wide = round8(cols * (int64_t)(bytes / 2));           // in 16-bit elements
    if (row_aligned(p, rows, ld, bytes)) {
        if (rows < 2) ld = wide / (int64_t)(bytes / 2);                 // one row: any leading dimension serves
        return true;
    }
    const size_t need = plane_bytes(rows, cols, bytes);
    if (!work || work_bytes < need) return false;
    jobs.j[jobs.count++] = {(const unsigned short*)p, ld * (int64_t)(bytes / 2), (unsigned short*)work, wide, rows, cols * (int64_t)(bytes / 2)};
    p = work;
    ld = wide / (int64_t)(bytes / 2);
    work += need;
    work_bytes -= need;
    return true;
}

inline cudaError_t launch_align(const AlignJobs& jobs, cudaStream_t stream) {
    if (jobs.count == 0) return cudaSuccess;
    int64_t items = 1;
    for (int i = 0; i < jobs.count; ++i) {
        const int64_t n = jobs.j[i].rows * ((jobs.j[i].cols + 255) / 256);
        items = items > n ? items : n;
    }
    const int64_t want = (items + 7) / 8, cap = (int64_t)sm_count() * 8;
    align_rows_kernel<<<dim3((unsigned)(want < cap ? want : cap), (unsigned)jobs.count), 256, 0, stream>>>(jobs);
    return cudaGetLastError();
}

// ---- clusters ------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// a shared-memory address of this CTA -> the same place in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

}  // namespace externd_llm
