// 4-bit weights with group scales (sm_100a): quantiser, dequantiser and the products Y = X W^T and, gated,
// H = act(X Wg^T) * (X Wu^T).
//
// Format: w = s (q - 8) + b, q in 0..15, s and b fp16 per row and group of 32, 64 or 128 columns.  A row of
// codes is blocks of 128 columns in 64 bytes; column 128 B + 32 i + 8 c + t is nibble 4 (t % 2) + t / 2 of
// word 4 c + i of block B.  A lane c of four that loads 16 bytes of a block thus holds, word by word, 8
// consecutive columns of each of the block's four 32-column spans: the four lanes together cover one span
// (one group at most) per word, and (word >> 4 p) & 0x000f000f is a pair of neighbouring columns, ready to
// become two 16-bit floats.
#include <type_traits>

#include "sm100.cuh"

namespace externd_int4 {

using namespace externd_llm;

__host__ __device__ __forceinline__ int64_t row_bytes(int64_t n) { return (n + 127) / 128 * 64; }

// ---------------------------------------------------------------------------------------------------
// quantise: a warp per row and pair of blocks, 8 columns (one word of codes) a lane
// ---------------------------------------------------------------------------------------------------
//
// One pass over A: the group's extremes stay in registers.  The format's fp64 decisions are taken in fp64 only next
// to a border (1e-5-wide bands around the rounding borders of codes, 2^-8 of the scales), where the fp32 value
// cannot decide.  Bound by instructions, 247 a warp for 256 columns: 2560 x 6912 bf16 in 28 us, 45 MB at 1.6 TB/s.
// (4 columns a lane, 267 instructions for 128 columns: 48 us.)

// says whether the fp32 estimate e (relative error below 2^-20) of a value leaves open to which fp16 it rounds
__device__ __forceinline__ bool near_half_border(float e) {
    const uint32_t u = __float_as_uint(e) & 0x7fffffffu;
    const uint32_t low = u & 0x1fffu;                       // bits below the fp16 mantissa
    return u < 0x38800000u + 64u || u >= 0x477fe000u || (low > 0x1000u - 16u && low < 0x1000u + 16u);   // subnormal or top fp16s too
}

// Greatest entry and greatest negated entry of a lane's eight, then of the LANES lanes of its group.  16-bit
// entries travel as a pair in one register.  `bad` becomes NaN where an entry is not finite.
template <int LANES>
__device__ __forceinline__ float2 group_extremes(const float (&w)[8], float& bad) {
    float mx = w[0], mn = w[0];
    #pragma unroll
    for (int t = 0; t < 8; ++t) {
        bad = fmaf(w[t], 0.0f, bad);
        mx = fmaxf(mx, w[t]);
        mn = fminf(mn, w[t]);
    }
    #pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        mn = fminf(mn, __shfl_xor_sync(FULL, mn, o));
    }
    return make_float2(mx, -mn);
}
template <int LANES, typename T, typename T2>
__device__ __forceinline__ float2 pair_extremes(const T (&w)[8], float& bad) {
    const T2* const v = reinterpret_cast<const T2*>(w);
    const T zero = from_f32<T>(0.0f);
    T2 z;
    z.x = z.y = zero;
    const T2 zz = z;
    #pragma unroll
    for (int t = 0; t < 4; ++t) z = __hfma2(v[t], zz, z);
    bad += to_f32(z.x) + to_f32(z.y);
    const T2 hi = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3])), lo = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
    T2 e;
    e.x = __hmax(hi.x, hi.y);
    e.y = __hneg(__hmin(lo.x, lo.y));
    #pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        const uint32_t u = __shfl_xor_sync(FULL, *reinterpret_cast<const uint32_t*>(&e), o);
        e = __hmax2(e, *reinterpret_cast<const T2*>(&u));
    }
    return make_float2(to_f32(e.x), to_f32(e.y));
}
template <int LANES> __device__ __forceinline__ float2 group_extremes(const __half (&w)[8], float& bad) {
    return pair_extremes<LANES, __half, __half2>(w, bad);
}
template <int LANES> __device__ __forceinline__ float2 group_extremes(const __nv_bfloat16 (&w)[8], float& bad) {
    return pair_extremes<LANES, __nv_bfloat16, __nv_bfloat162>(w, bad);
}

constexpr int QPAIRS = 4;                               // pairs of blocks a warp works on at once

// LG = log2(group).  A warp takes QPAIRS pairs of blocks of its row at once: the loads are in flight together, and
// of the lanes that share a group each quarter computes the scale of another pair (they would all compute the same).
template <typename T, bool AFFINE, bool VEC, int LG>
__global__ void __launch_bounds__(256, 4) quantize_kernel(const T* __restrict__ A, int64_t m, int64_t n, int64_t lda,
                                                       uint32_t* __restrict__ q, __half* __restrict__ scale,
                                                       __half* __restrict__ offset, int* __restrict__ status) {
    constexpr int LANES = 1 << (LG - 3), QUARTER = LANES / QPAIRS;      // lanes of a group
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);   // neighbouring warps, neighbouring rows: their scales share a sector
    if (row >= m) return;
    const int blocks = (int)((n + 127) / 128), pairs = (blocks + 1) / 2, sub = lane >> 4, l = lane & 15;
    const T* const arow = A + row * lda;
    uint32_t* const qrow = q + row * blocks * 16 + 16 * sub + 4 * (l & 3) + (l >> 2);    // word 4 c + i of a block
    const int mine = (lane % LANES) / QUARTER;              // the pair whose scale this lane computes
    const int head = lane & ~(LANES - 1);                   // the group's first lane
    for (int p0 = blockIdx.y * QPAIRS; p0 < pairs; p0 += gridDim.y * QPAIRS) {
        __align__(16) T w[QPAIRS][8];
        #pragma unroll
        for (int u = 0; u < QPAIRS; ++u) {
            const int64_t j0 = (int64_t)(p0 + u) * 256 + 8 * lane;
            if (VEC && j0 + 8 <= n) {
                #pragma unroll
                for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                    reinterpret_cast<uint4*>(w[u])[h] = __ldcs(reinterpret_cast<const uint4*>(arow + j0) + h);
            } else if (j0 + 8 <= n) {
                using E = typename std::conditional<sizeof(T) == 4, float, unsigned short>::type;
                const auto v = load8(reinterpret_cast<const E*>(arow), j0, n, false);
                static_assert(sizeof(v) == sizeof(w[u]), "eight entries");
                memcpy(w[u], &v, sizeof(v));
            } else {
                // columns past the last one repeat the group's first: they change no extreme
                const int64_t g0 = j0 >> LG << LG;
                #pragma unroll
                for (int t = 0; t < 8; ++t) w[u][t] = g0 < n ? arow[j0 + t < n ? j0 + t : g0] : from_f32<T>(0.0f);
            }
        }
        float2 ext = make_float2(0.0f, 0.0f);               // greatest, greatest negated: of this lane's pair
        float bad = 0.0f;
        #pragma unroll
        for (int u = 0; u < QPAIRS; ++u) {
            const float2 e = group_extremes<LANES>(w[u], bad);
            if (u == mine) ext = e;
        }
        const float mx = ext.x, mn = -ext.y;
        const float range = AFFINE ? mx - mn : fmaxf(mx, ext.y);
        float e = range * (AFFINE ? 1.0f / 15.0f : 1.0f / 7.0f);
        if (near_half_border(e)) e = (float)(AFFINE ? ((double)mx - (double)mn) / 15.0 : (double)range / 7.0);
        const __half sh = __float2half_rn(e);
        const float s1 = __half2float(sh);
        float b1 = 0.0f;
        if (AFFINE) {
            float f = fmaf(8.0f, s1, mn);
            if (near_half_border(f)) f = (float)((double)mn + 8.0 * (double)s1);
            b1 = __half2float(__float2half_rn(f));
        }
        const float inv1 = s1 > 0.0f ? __fdividef(1.0f, s1) : 0.0f;
        // a group with NaN or Inf reports that, whatever other groups report
        if (!(bad == 0.0f)) atomicExch(status, EXTERND_ENONFINITE);
        else if (fmaxf(mx, ext.y) <= FLT_MAX && (isinf(s1) || isinf(b1))) atomicCAS(status, EXTERND_OK, EXTERND_ELIMIT);
        #pragma unroll
        for (int u = 0; u < QPAIRS; ++u) {
            if (p0 + u >= pairs) break;
            const int from = head + u * QUARTER;
            const float s = __shfl_sync(FULL, s1, from), inv = __shfl_sync(FULL, inv1, from);
            const float b = AFFINE ? __shfl_sync(FULL, b1, from) : 0.0f;
            const int64_t j0 = (int64_t)(p0 + u) * 256 + 8 * lane;
            uint32_t code = 0;
            float off = 0.0f;                               // distance from an integer, the largest of the eight
            #pragma unroll
            for (int t = 0; t < 8; ++t) {
                // c in -8 .. 7 plus 1.5 2^23 + 8: rounded to an integer, ties to even, whose low bits are the code.
                // The error of c stays below 3e-6: three roundings of 2^-24 and a reciprocal of 2^-22 at |c| <= 8.
                const float v = to_f32(w[u][t]);
                const float c = fminf(fmaxf((AFFINE ? v - b : v) * inv, -8.0f), 7.0f);
                const float k = c + 12582920.0f;
                off = fmaxf(off, fabsf(c - (k - 12582920.0f)));
                code |= (__float_as_uint(k) & 15u) << (4 * (4 * (t & 1) + (t >> 1)));
            }
            if (off > 0.49999f || j0 + 8 > n) {
                code = 0;
                #pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const double c = s > 0.0f ? rint(((double)to_f32(w[u][t]) - (double)b) / (double)s) : 0.0;
                    const uint32_t d = j0 + t < n ? (uint32_t)((int)fmin(fmax(c, -8.0), 7.0) + 8) : 8u;
                    code |= d << (4 * (4 * (t & 1) + (t >> 1)));
                }
            }
            if (2 * (p0 + u) + sub < blocks) qrow[(int64_t)(p0 + u) * 32] = code;
        }
        // the lane at the head of a pair's quarter stores its scale
        if (lane % QUARTER == 0) {
            const int64_t j = (int64_t)(p0 + mine) * 256 + 8 * head;
            if (j < n) {
                const int64_t at = (j >> LG) * m + row;
                scale[at] = sh;
                if (AFFINE) offset[at] = __float2half_rn(b1);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// codes -> 16-bit floats
// ---------------------------------------------------------------------------------------------------

// (w & mask) | magic in one instruction (two immediates would make it two)
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}

// the four pairs of codes of a word -> pairs of floats q - 8
template <typename T> __device__ __forceinline__ void codes8(uint32_t w, uint32_t (&a)[4]);
template <> __device__ __forceinline__ void codes8<__half>(uint32_t w, uint32_t (&a)[4]) {
    // 0x6400 | q = 1024 + q, 0x6400 | 16 q = 1024 + 16 q (exact); subtract 1032, or scale by 1/16 and subtract 72
    const __half2 k1032 = __half2half2(__ushort_as_half(0x6408)), sixteenth = __half2half2(__ushort_as_half(0x2c00)),
                  m72 = __half2half2(__ushort_as_half(0xd480));
    const uint32_t w8 = w >> 8;
    const uint32_t u0 = pick(w, 0x000f000fu, 0x64006400u), u1 = pick(w, 0x00f000f0u, 0x64006400u);
    const uint32_t u2 = pick(w8, 0x000f000fu, 0x64006400u), u3 = pick(w8, 0x00f000f0u, 0x64006400u);
    const __half2 v0 = __hsub2(*reinterpret_cast<const __half2*>(&u0), k1032);
    const __half2 v1 = __hfma2(*reinterpret_cast<const __half2*>(&u1), sixteenth, m72);
    const __half2 v2 = __hsub2(*reinterpret_cast<const __half2*>(&u2), k1032);
    const __half2 v3 = __hfma2(*reinterpret_cast<const __half2*>(&u3), sixteenth, m72);
    a[0] = *reinterpret_cast<const uint32_t*>(&v0);
    a[1] = *reinterpret_cast<const uint32_t*>(&v1);
    a[2] = *reinterpret_cast<const uint32_t*>(&v2);
    a[3] = *reinterpret_cast<const uint32_t*>(&v3);
}
template <> __device__ __forceinline__ void codes8<__nv_bfloat16>(uint32_t w, uint32_t (&a)[4]) {
    // 0x4300 | q = 128 + q; subtract 136
    const __nv_bfloat162 k136 = __bfloat162bfloat162(__ushort_as_bfloat16(0x4308));
    #pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t u = pick(w >> (4 * p), 0x000f000fu, 0x43004300u);
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), k136);
        a[p] = *reinterpret_cast<const uint32_t*>(&v);
    }
}

// ---------------------------------------------------------------------------------------------------
// dequantise: a warp per row and pair of blocks, 8 columns a lane
// ---------------------------------------------------------------------------------------------------

// VEC: rows of 16-bit values start on 16-byte boundaries.  Otherwise a warp's 256 values pass through shared memory, so
// that neighbouring lanes store neighbouring columns (5196 x 3405 bf16: 13 us, 52 without).  2560 x 6912: bf16 9.4 us,
// 4.8 TB/s; fp32 13.9 us, 5.8 TB/s.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint32_t* __restrict__ q, const __half* __restrict__ scale,
                                                         const __half* __restrict__ offset, int64_t m, int64_t n, int lg,
                                                         T* __restrict__ out, int64_t ldo) {
    __shared__ __align__(16) T stage[VEC ? 1 : 8][256];
    const int lane = threadIdx.x & 31, l = lane & 15, sub = lane >> 4;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= m) return;
    const int blocks = (int)((n + 127) / 128), pairs = (blocks + 1) / 2;
    const uint32_t* const qrow = q + row * blocks * 16 + 16 * sub + 4 * (l & 3) + (l >> 2);
    const int64_t jump = (256 >> lg) * m;               // a pair of blocks on in the scales
    constexpr int UB = 4;                               // pairs of blocks in flight
    T* const orow = out + row * ldo;
    T* const mine = stage[VEC ? 0 : threadIdx.x >> 5];
    for (int p0 = UB * blockIdx.y; p0 < pairs; p0 += UB * gridDim.y) {
        uint32_t w[UB];
        __half s[UB], b[UB];
        const int64_t at = ((int64_t)p0 * 256 + 8 * lane >> lg) * m + row;
        #pragma unroll
        for (int u = 0; u < UB; ++u) {
            const bool in = (int64_t)(p0 + u) * 256 + 8 * lane < n;
            w[u] = in ? __ldg(qrow + (p0 + u) * 32ll) : 0;
            s[u] = in ? __ldg(scale + at + u * jump) : __ushort_as_half(0);
            b[u] = in && offset ? __ldg(offset + at + u * jump) : __ushort_as_half(0);
        }
        #pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int64_t c0 = (int64_t)(p0 + u) * 256, j0 = c0 + 8 * lane;
            if (c0 >= n) break;                         // the whole warp
            const float sf = __half2float(s[u]), bf = __half2float(b[u]);
            uint32_t c4[4];
            codes8<__half>(w[u], c4);                    // q - 8, exactly
            __align__(16) T v[8];
            #pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 f = unpack2<__half>(c4[t]);
                v[2 * t] = from_f32<T>(fmaf(sf, f.x, bf));
                v[2 * t + 1] = from_f32<T>(fmaf(sf, f.y, bf));
            }
            constexpr int PARTS = sizeof(T) / 2;         // 16-byte pieces of the eight
            if (VEC && j0 + 8 <= n) {
                #pragma unroll
                for (int h = 0; h < PARTS; ++h) __stcs(reinterpret_cast<uint4*>(orow + j0) + h, reinterpret_cast<const uint4*>(v)[h]);
            } else if (VEC) {
                #pragma unroll
                for (int t = 0; t < 8; ++t)
                    if (j0 + t < n) orow[j0 + t] = v[t];
            } else {
                #pragma unroll
                for (int h = 0; h < PARTS; ++h) reinterpret_cast<uint4*>(mine + 8 * lane)[h] = reinterpret_cast<const uint4*>(v)[h];
                __syncwarp();
                #pragma unroll
                for (int t = 0; t < 8; ++t)
                    if (c0 + 32 * t + lane < n) orow[c0 + 32 * t + lane] = mine[32 * t + lane];
                __syncwarp();
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------------------------------
//
// Codes become exact 16-bit floats q - 8 two at a time, the tensor cores sum each group's products in fp32, and
// the group's sum is scaled once.  fp32 vectors enter as three bf16 terms x = hi + mid + lo cut off from the
// top (8 + 8 + 8 bits: no loss), three products into one sum.

struct Mat4 {                       // one 4-bit matrix
    const uint8_t* q;
    const __half* scale;
    const __half* offset;           // nullptr: symmetric
};

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ uint32_t word_of(const uint4& q, int i) { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }

// (16 rows' codes of one word span) x (8 vectors' entries): the most significant plane into hi, the others into lo,
// whose roundings are then 2^-8 as large
template <typename T, int PLANES>
__device__ __forceinline__ void span_mma(float (&hi)[4], float (&lo)[4], const uint32_t (&a)[4], const uint32_t (&b)[4], const uint32_t (&x)[PLANES][4]) {
    #pragma unroll
    for (int p = PLANES - 1; p >= 0; --p) {
        float(&d)[4] = p == 0 ? hi : lo;
        mma16816<T>(d, a[0], b[0], a[1], b[1], x[p][0], x[p][1]);
        mma16816<T>(d, a[2], b[2], a[3], b[3], x[p][2], x[p][3]);
    }
}

// ---- up to 8 vectors ----------------------------------------------------------------------------------
//
// A CTA takes 16 rows (of both matrices when gated); its warps take the 128-column blocks in turn and add
// their sums in shared memory in a fixed order.  The warp-level products carry the arithmetic: a warp's 16 rows
// by eight vectors in one instruction, straight from registers.  (The tile-level products read their operands
// from shared memory: the codes would cross it as 16-bit floats, and of a tile's columns 16 at least.)
// Every lane keeps the codes of its next VEC_DEPTH blocks in flight to shared memory (its own 16 bytes of each row:
// no barrier, no registers); the scales, whose way from memory is as long, come four blocks ahead through
// registers; the vectors' entries come from the first-level cache.  163 instructions a block of 128
// columns and 16 rows, 72 of them to unpack the codes.  8192 x 28672, one fp16 vector: 34 us, 3.5 TB/s (0.54 of
// the measured copy rate); issue slots are 62 % busy, no pipe above 48 %.  Its 512 equal CTAs are four on 68 SMs and
// three on 80: the last end 1.16 times later than the average, and an SM with three has few warps to hide its waits.
// Where an SM has one CTA (2560 rows: 160) the blocks' latency is the time.  Measured and not taken: bulk copies (a warp issues them one lane at a time: 271
// instructions), the entries through the ring too (183), 32 rows a warp (the same time), 6 blocks ahead (slower).
// The offsets' part b sum(x) takes sum(x) from the lanes that hold x (products with ones would double the work of
// the warp-level products).
// X element type, T product type (bf16 for fp32 X), NM matrices, WORDS = group / 32.
constexpr int VEC_DEPTH = 4, VEC_WARPS = 8, VEC_BATCH = 8;

__device__ __forceinline__ float sum8(const uint4& r, __half*) {
    const float2 a = unpack2<__half>(r.x), b = unpack2<__half>(r.y), c = unpack2<__half>(r.z), d = unpack2<__half>(r.w);
    return ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (d.x + d.y));
}
__device__ __forceinline__ float sum8(const uint4& r, __nv_bfloat16*) {
    const float2 a = unpack2<__nv_bfloat16>(r.x), b = unpack2<__nv_bfloat16>(r.y), c = unpack2<__nv_bfloat16>(r.z),
                 d = unpack2<__nv_bfloat16>(r.w);
    return ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (d.x + d.y));
}
__device__ __forceinline__ float sum8(const F8& r, __nv_bfloat16*) {
    return ((r.a.x + r.a.y) + (r.a.z + r.a.w)) + ((r.b.x + r.b.y) + (r.b.z + r.b.w));
}

template <typename X, typename T, int NM, int WORDS, bool AFFINE>
__global__ void __launch_bounds__(VEC_WARPS * 32) vec4_kernel(Mat4 w0, Mat4 w1, int64_t m, int64_t n, int act, const X* __restrict__ x,
                                                             int64_t ldx, int vec, int batch, X* __restrict__ y, int64_t ldy) {
    using Raw = typename Raw8<X>::type;
    constexpr int PLANES = Raw8<X>::PLANES;
    using XE = typename std::conditional<PLANES == 3, float, unsigned short>::type;
    constexpr int GROUPS = 4 / WORDS;                   // groups of a block
    constexpr int FAR = 4;                              // blocks whose scales are fetched at a time
    constexpr int KINDS = NM * (AFFINE ? 2 : 1), HALVES = FAR * GROUPS / 2;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __half side[VEC_WARPS][KINDS][FAR * GROUPS][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int blocks = (int)((n + 127) / 128), groups = (int)((n + 32 * WORDS - 1) / (32 * WORDS));
    const int whole = vec ? (int)(n / 128) : 0;         // blocks whose entries load 16 bytes at a time, unchecked

    // this lane's codes: rows r and r + 8.  Rows past the last one repeat it (their sums are not stored)
    const uint8_t* q[NM][2];
    #pragma unroll
    for (int j = 0; j < NM; ++j)
        #pragma unroll
        for (int h = 0; h < 2; ++h)
            q[j][h] = (NM == 2 && j == 1 ? w1.q : w0.q) + (min(row0 + r + 8 * h, m - 1) * blocks + warp) * 64 + 16 * c;
    const uint32_t mine = smem_u32(ring) + (warp * (VEC_DEPTH * NM * 2) * 32 + lane) * 16;     // 512 bytes a row half
    const auto issue = [&](bool on, uint32_t slot) {
        #pragma unroll
        for (int j = 0; j < NM; ++j)
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (on) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + slot + (2 * j + h) * 512), "l"(q[j][h]) : "memory");
                q[j][h] += VEC_WARPS * 64;
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // scales (and offsets) of the warp's next FAR blocks: 16 rows, a lane two groups at a time, fetched while the
    // FAR blocks before them are worked on and then laid down in the warp's own shared memory
    __half ahead[KINDS][HALVES];
    const int srow = lane & 15, sgroup = lane >> 4;
    const auto fetch = [&](int blk0) {                   // blk0: the warp's first block of the FAR
        #pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const int e = 2 * h + sgroup, g = (blk0 + e / GROUPS * VEC_WARPS) * GROUPS + e % GROUPS;
            #pragma unroll
            for (int k = 0; k < KINDS; ++k) {
                const int j = k % NM;
                const Mat4& w = NM == 2 && j == 1 ? w1 : w0;
                const __half* const p = k < NM ? w.scale : w.offset;
                const int64_t sr = min(row0 + srow, m - 1);
                ahead[k][h] = p && g < groups ? __ldg(p + g * m + sr) : __ushort_as_half(0);   // past the last group: entries are 0
            }
        }
    };
    #pragma unroll
    for (int d = 0; d < VEC_DEPTH; ++d) issue(warp + d * VEC_WARPS < blocks, d * (NM * 1024));
    fetch(warp);
    // columns of the products past the last vector repeat it (they are not stored)
    const XE* const xr = reinterpret_cast<const XE*>(x + min(r, batch - 1) * ldx);
    const XE* xp = xr + warp * 128 + 8 * c;
    float out[NM][4] = {};
    uint32_t slot = 0;
    int step = 0;                                        // block within the FAR
    #pragma unroll 1
    for (int blk = warp; blk < blocks; blk += VEC_WARPS) {
        Raw xs[4];
        if (blk < whole) {
            #pragma unroll
            for (int i = 0; i < 4; ++i) xs[i] = *reinterpret_cast<const Raw*>(xp + 32 * i);
        } else {
            #pragma unroll
            for (int i = 0; i < 4; ++i) xs[i] = load8(xr, (int64_t)blk * 128 + 32 * i + 8 * c, n, vec);
        }
        xp += VEC_WARPS * 128;
        if (step == 0) {
            __syncwarp();
            #pragma unroll
            for (int h = 0; h < HALVES; ++h)
                #pragma unroll
                for (int k = 0; k < KINDS; ++k) side[warp][k][2 * h + sgroup][srow] = ahead[k][h];
            __syncwarp();
            fetch(blk + FAR * VEC_WARPS);
        }
        const __half* const sp = &side[warp][0][step * GROUPS][r];
        step = (step + 1) & (FAR - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(VEC_DEPTH - 1) : "memory");
        uint4 code[NM][2];
        #pragma unroll
        for (int j = 0; j < NM; ++j)
            #pragma unroll
            for (int h = 0; h < 2; ++h)
                code[j][h] = lds128(mine + slot + (2 * j + h) * 512);
        float acc[NM][4] = {}, low[NM][4] = {}, sum = 0.0f;      // low: planes 1 and 2 of fp32 entries
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t xv[PLANES][4];
            planes8(xs[i], xv);
            #pragma unroll
            for (int j = 0; j < NM; ++j) {
                uint32_t a[4], b[4];
                codes8<T>(word_of(code[j][0], i), a);
                codes8<T>(word_of(code[j][1], i), b);
                span_mma<T, PLANES>(acc[j], low[j], a, b, xv);
            }
            if (AFFINE) sum += sum8(xs[i], (T*)nullptr);
            if ((i + 1) % WORDS == 0) {                  // the group ends here
                const __half* const sg = sp + i / WORDS * 16;
                float s0 = 0.0f, s1 = 0.0f;              // the group's sums of this lane's two output vectors, 2 c and 2 c + 1
                if (AFFINE) {
                    sum += __shfl_xor_sync(FULL, sum, 1);
                    sum += __shfl_xor_sync(FULL, sum, 2);
                    s0 = __shfl_sync(FULL, sum, 8 * c);
                    s1 = __shfl_sync(FULL, sum, 8 * c + 4);
                    sum = 0.0f;
                }
                #pragma unroll
                for (int j = 0; j < NM; ++j) {
                    const float sa = __half2float(sg[j * FAR * GROUPS * 16]), sb = __half2float(sg[j * FAR * GROUPS * 16 + 8]);
                    if (PLANES > 1) {
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            acc[j][e] += low[j][e];
                            low[j][e] = 0.0f;
                        }
                    }
                    out[j][0] = fmaf(sa, acc[j][0], out[j][0]);
                    out[j][1] = fmaf(sa, acc[j][1], out[j][1]);
                    out[j][2] = fmaf(sb, acc[j][2], out[j][2]);
                    out[j][3] = fmaf(sb, acc[j][3], out[j][3]);
                    if (AFFINE) {
                        const float oa = __half2float(sg[(NM + j) * FAR * GROUPS * 16]), ob = __half2float(sg[(NM + j) * FAR * GROUPS * 16 + 8]);
                        out[j][0] = fmaf(oa, s0, out[j][0]);
                        out[j][1] = fmaf(oa, s1, out[j][1]);
                        out[j][2] = fmaf(ob, s0, out[j][2]);
                        out[j][3] = fmaf(ob, s1, out[j][3]);
                    }
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
                }
            }
        }
        issue(blk + VEC_DEPTH * VEC_WARPS < blocks, slot);   // the slot's codes have been used
        slot = slot == (VEC_DEPTH - 1) * (NM * 1024) ? 0 : slot + NM * 1024;
    }
    // the ring becomes the warps' sums
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* const part = reinterpret_cast<float*>(ring);  // [matrix][warp][row][9]
    #pragma unroll
    for (int j = 0; j < NM; ++j) {
        float* const p = part + ((j * VEC_WARPS + warp) * 16 + r) * 9 + 2 * c;
        p[0] = out[j][0];
        p[1] = out[j][1];
        p[72] = out[j][2];
        p[73] = out[j][3];
    }
    __syncthreads();
    const int e = threadIdx.x, rr = e & 15, cc = e >> 4;
    if (e < 128 && row0 + rr < m && cc < batch) {
        float v[NM] = {};
        #pragma unroll
        for (int j = 0; j < NM; ++j)
            #pragma unroll
            for (int p = 0; p < VEC_WARPS; ++p) v[j] += part[((j * VEC_WARPS + p) * 16 + rr) * 9 + cc];
        const float res = NM == 1 ? v[0] : act_rt<PLANES == 3>(act, v[0]) * v[NM - 1];
        y[cc * ldy + row0 + rr] = from_f32<X>(res);
    }
}

// ---- more vectors -------------------------------------------------------------------------------------
//
// A CTA takes 128 rows of one matrix (gated: 64 rows of both) and N = 16, 32 or 64 vectors on the 5th-generation
// tensor cores; a cluster of up to 8 CTAs one such tile, each a share of its columns.  Eight warps turn codes
// into 16-bit floats and stage them with the vectors' entries in swizzled shared memory, 128 columns a stage;
// one thread issues the products, every group of columns into an accumulator of its own; eight warps scale
// each group's accumulator into fp32 registers, a row and half of the vectors per thread, so that the row's scale
// is one register.
// The offsets' part comes from a second product of the same entries with ones, whose accumulator holds the
// group's sum of x in every row.  The CTAs' sums meet through distributed shared memory in a fixed order.
// (Weights scaled before the product would need no accumulator per group, but s (q - 8) + b does not fit 16
// bits: measured against 64 bits that costs bf16 results 1.4 times the error of their own rounding.)
// More than 64 vectors are tiles of 64 side by side, each of which unpacks its rows' codes again: 1537 vectors through
// 2560 x 6912 take 183 us (298 TFLOP/s), 512 take 81, 128 22.5; dequantising and a dense library product take 47, 27
// and 21.5.
// Bound by the latency of its stages: 64 vectors through 4096 x 4096 take 15.4 us, of which 4 until the first stage
// is full and 3 to add up; the tensor memory's pipe is 19 percent busy.  (The same tile with warp-level products took
// 43 us: those run at a ninth of this rate.)
constexpr int TC_EPI = 8, TC_PROD = 8, TC_THREADS = (TC_EPI + 1 + TC_PROD) * 32;
template <int N> __host__ __device__ constexpr int tc_bufs() { return N == 64 ? 4 : 8; }     // accumulators in flight
template <typename X> __host__ __device__ constexpr int tc_stages() { return Raw8<X>::PLANES == 3 ? 2 : 3; }
constexpr int TC_CODES = 6;                               // blocks of codes in flight, 32 bytes a thread each
template <typename X, int N> __host__ __device__ constexpr int tc_stage() { return 128 * 256 + Raw8<X>::PLANES * N * 256; }
template <typename X, int N> __host__ __device__ constexpr int tc_smem() {
    return tc_stages<X>() * tc_stage<X, N>() + 128 * 128 + TC_CODES * TC_PROD * 32 * 32 + 1024;   // stages, the ones, codes, alignment
}

template <typename X, typename T, int N, int NM, int WORDS, bool AFFINE>
__global__ void __launch_bounds__(TC_THREADS, 1) tile4_kernel(Mat4 w0, Mat4 w1, int64_t m, int64_t n, int act, const X* __restrict__ x,
                                                             int64_t ldx, int64_t batch, X* __restrict__ y, int64_t ldy,
                                                             int splits, const WaitFault fault) {
    using Raw = typename Raw8<X>::type;
    constexpr int PLANES = Raw8<X>::PLANES;
    using XE = typename std::conditional<PLANES == 3, float, unsigned short>::type;
    constexpr int GROUPS = 4 / WORDS, STAGES = tc_stages<X>(), STAGE = tc_stage<X, N>(), ROWS = 128 / NM;
    constexpr int TC_BUFS = tc_bufs<N>();
    constexpr uint32_t COLUMNS = TC_BUFS * N * 2;           // tensor memory: products and sums (256 or 512 columns)
    static_assert(128 * N * 4 <= STAGES * STAGE, "the tile of sums takes the stages' place");
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[2 * STAGES + 2 * TC_BUFS + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int quit_flag;
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    unsigned char* const smem = raw + (base - smem_u32(raw));
    const uint32_t ones = base + STAGES * STAGE;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, dfull0 = empty0 + 8 * STAGES, dempty0 = dfull0 + 8 * TC_BUFS,
                   drain = dempty0 + 8 * TC_BUFS;
    volatile int* const quit = &quit_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int split = blockIdx.x % splits;
    const int64_t row0 = (int64_t)(blockIdx.x / splits) * ROWS, col0 = (int64_t)blockIdx.y * N;
    const int blocks = (int)((n + 127) / 128), groups = (int)((n + 32 * WORDS - 1) / (32 * WORDS));
    const int first = (int)((int64_t)blocks * split / splits), last = (int)((int64_t)blocks * (split + 1) / splits);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full0 + 8 * i, TC_PROD * 32);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < TC_BUFS; ++i) {
            mbar_init(dfull0 + 8 * i, 1);
            mbar_init(dempty0 + 8 * i, TC_EPI);
        }
        mbar_init(drain, 1);
        quit_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == TC_EPI) tmem_alloc<1>(smem_u32(&tmem_slot), COLUMNS);
    if (AFFINE) {                                            // 128 rows of ones, 64 deep (every 16 of them serve)
        const uint32_t one = std::is_same<T, __half>::value ? 0x3c003c00u : 0x3f803f80u;
        for (int e = threadIdx.x; e < 128 * 8; e += TC_THREADS)
            *reinterpret_cast<uint4*>(smem + STAGES * STAGE + 16 * e) = make_uint4(one, one, one, one);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;

    constexpr int W = N / 2;                                 // vectors of a scaling warp
    float out[W];
    if (warp > TC_EPI) {
        // ---- codes and entries into shared memory: thread p unpacks half of row p % 128, and a share of the entries
        const int p = threadIdx.x - (TC_EPI + 1) * 32, r = p & 127, h = p >> 7;
        const Mat4 w = NM == 2 && r >= 64 ? w1 : w0;
        const int64_t row = min(row0 + (NM == 2 ? r & 63 : r), m - 1);    // rows past the last one repeat it
        const uint8_t* src = w.q + (row * blocks + first) * 64 + 32 * h;
        constexpr int PIECES = N * 16 / (TC_PROD * 32);      // pieces of 8 entries a thread: vectors col, col + 16, ..
        constexpr int AHEAD = PLANES == 3 ? 1 : 2;           // blocks of entries in flight
        const int whole = (int)(n / 128);          // blocks whose entries load 16 bytes at a time, unchecked
        const int col = p >> 4, piece = p & 15;
        Raw ent[AHEAD][PIECES];
        // vectors past the last one repeat it: their sums are not stored
        const XE* xp[PIECES];
        #pragma unroll
        for (int e = 0; e < PIECES; ++e) xp[e] = reinterpret_cast<const XE*>(x + min(col0 + col + 16 * e, batch - 1) * ldx) + (int64_t)first * 128 + 8 * piece;
        const auto load = [&](int u, int blk) {
            if (blk >= last) return;
            if (blk < whole) {
                #pragma unroll
                for (int e = 0; e < PIECES; ++e) ent[u][e] = *reinterpret_cast<const Raw*>(xp[e]);
            } else {
                const int64_t k = (int64_t)blk * 128 + 8 * piece;
                #pragma unroll
                for (int e = 0; e < PIECES; ++e) ent[u][e] = load8(xp[e] - k, k, n, true);
            }
            #pragma unroll
            for (int e = 0; e < PIECES; ++e) xp[e] += 128;
        };
        // codes ride a ring of their own, each thread copying what it will unpack: no barrier
        const uint32_t cring = ones + 128 * 128 + p * 16;    // halves of the 32 bytes TC_PROD * 512 bytes apart
        const auto issue = [&](int blk, uint32_t at) {
            if (blk < last) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(cring + at), "l"(src) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(cring + at + TC_PROD * 512), "l"(src + 16) : "memory");
                src += 64;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        #pragma unroll
        for (int d = 0; d < TC_CODES; ++d) issue(first + d, d * (TC_PROD * 1024));
        uint32_t slot = 0;
        // places within a stage: columns 32 i + 8 c (c = 2 h, 2 h + 1) of the block are 16-byte chunk 4 (i % 2) + c of half
        // i / 2, a row 128 bytes, chunks swizzled by the row; entries alike (vectors 16 apart share their swizzle)
        const uint32_t place = r * 128 + (((2 * h) ^ (r & 7)) << 4), xplace = 128 * 256 + (piece >> 3) * (N * 128) + col * 128 + (((piece & 7) ^ (col & 7)) << 4);
        const auto sts = [&](uint32_t at, const uint32_t (&v)[4]) {
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
        };
        #pragma unroll
        for (int u = 0; u < AHEAD; ++u) load(u, first + u);
        int s = 0, phase = 1;
        bool ok = true;
        for (int b0 = first; b0 < last && ok; b0 += AHEAD) {
            #pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int blk = b0 + u;
                if (blk >= last) break;
                if (!mbar_wait(empty0 + 8 * s, phase, quit, fault.limit_ns)) { ok = false; break; }
                const uint32_t st = base + s * STAGE, at = st + place;
                asm volatile("cp.async.wait_group %0;" ::"n"(TC_CODES - 1) : "memory");
                const uint4 code[2] = {lds128(cring + slot), lds128(cring + slot + TC_PROD * 512)};
                #pragma unroll
                for (int i = 0; i < 4; ++i)
                    #pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t v[4];
                        codes8<T>(word_of(code[cc], i), v);
                        sts(((at ^ (16u * cc)) ^ (64u * (i & 1))) + (i >> 1) * (128 * 128), v);
                    }
                #pragma unroll
                for (int e = 0; e < PIECES; ++e) {
                    uint32_t v[PLANES][4];
                    planes8(ent[u][e], v);
                    #pragma unroll
                    for (int q = 0; q < PLANES; ++q) sts(st + xplace + q * N * 256 + e * 2048, v[q]);
                }
                load(u, blk + AHEAD);
                issue(blk + TC_CODES, slot);                 // the slot's codes have been used
                slot = slot == (TC_CODES - 1) * (TC_PROD * 1024) ? 0 : slot + TC_PROD * 1024;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(full0 + 8 * s);
                if (++s == STAGES) { s = 0; phase ^= 1; }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();                                        // lanes that left the loop apart
    } else if (warp == TC_EPI) {
        // ---- products.  (Nothing in the loop needs the whole warp: where a wait runs out, lanes may leave it one by one)
        const bool leader = elect_one();
        constexpr uint32_t idesc = f16_idesc(std::is_same<T, __half>::value ? 0 : 1, false, false, 128, N);
        const uint64_t a0 = smem_desc(base, 16, 1024), one = smem_desc(ones, 16, 1024);
        int s = 0, phase = 0, d = 0, dphase = 1;
        bool ok = (int)blockIdx.x + 1 != fault.withhold;
        for (int blk = first; blk < last && ok; ++blk) {
            if (!mbar_wait(full0 + 8 * s, phase, quit, fault.limit_ns)) break;
            fence_after();
            const uint64_t da = a0 + (uint32_t)(s * (STAGE >> 4));   // the address field counts 16 bytes
            #pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                if (!mbar_wait(dempty0 + 8 * d, dphase, quit, fault.limit_ns)) { ok = false; break; }
                fence_after();
                const uint32_t acc = tmem + d * N;
                if (leader) {
                    // the least significant plane first: only the last one's sums are rounded at the result's magnitude
                    #pragma unroll
                    for (int q = PLANES - 1; q >= 0; --q)
                        #pragma unroll
                        for (int k = 0; k < 2 * WORDS; ++k) {
                            const int kk = g * 2 * WORDS + k;    // 16 columns of the block: half kk / 4, 32 bytes each
                            const uint64_t db = da + ((128 * 256 + q * N * 256 + (kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4);
                            const bool more = k > 0 || q < PLANES - 1;
                            mma_f16<1>(acc, da + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4), db, idesc, more);
                            if (AFFINE) mma_f16<1>(acc + TC_BUFS * N, one, db, idesc, more);
                        }
                    mma_commit<1>(dfull0 + 8 * d);
                    if (g == GROUPS - 1) mma_commit<1>(empty0 + 8 * s);
                }
                if (++d == TC_BUFS) { d = 0; dphase ^= 1; }
            }
            if (++s == STAGES) { s = 0; phase ^= 1; }
        }
        // the tensor memory is freed and the stages reused only when everything issued has ended
        if (leader) {
            mma_commit<1>(drain);
            const uint64_t t0 = timer_ns();
            while (!mbar_try(drain, 0) && timer_ns() - t0 < WAIT_LIMIT_NS) {}
        }
        __syncwarp();
    } else {
        // ---- scaling: warp w holds rows 32 (w % 4) .. + 31 of the tile and half w / 4 of the vectors
        const int r = 32 * (warp & 3) + lane;
        const Mat4 w = NM == 2 && r >= 64 ? w1 : w0;
        const int64_t row = min(row0 + (NM == 2 ? r & 63 : r), m - 1);
        const __half* ps = w.scale + (int64_t)first * GROUPS * m + row;
        const __half* po = AFFINE && w.offset ? w.offset + (int64_t)first * GROUPS * m + row : nullptr;
        const int count = min(last * GROUPS, groups) - first * GROUPS, all = (last - first) * GROUPS;
        #pragma unroll
        for (int t = 0; t < W; ++t) out[t] = 0.0f;
        // scales and offsets come from memory while seven groups are worked on: one group takes a fraction of the way
        constexpr int FAR = 8;
        __half sr[FAR], orr[FAR];
        #pragma unroll
        for (int i = 0; i < FAR; ++i) {
            sr[i] = i < count ? __ldg(ps + i * m) : __ushort_as_half(0);
            orr[i] = AFFINE && po && i < count ? __ldg(po + i * m) : __ushort_as_half(0);
        }
        ps += FAR * m;
        if (AFFINE && po) po += FAR * m;
        bool ok = true;
        for (int g0 = 0; g0 < all && ok; g0 += FAR) {
            #pragma unroll
            for (int i = 0; i < FAR; ++i) {
                const int g = g0 + i;
                if (g >= all) break;
                const float s = __half2float(sr[i]), o = __half2float(orr[i]);
                // past the last group the entries are 0
                sr[i] = g + FAR < count ? __ldg(ps) : __ushort_as_half(0);
                if (AFFINE) orr[i] = po && g + FAR < count ? __ldg(po) : __ushort_as_half(0);
                ps += m;
                if (AFFINE && po) po += m;
                const int d = i % TC_BUFS;
                if (!mbar_wait_warp(dfull0 + 8 * d, (g / TC_BUFS) & 1, quit, fault.limit_ns)) { ok = false; break; }
                fence_after();
                const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + d * N + (warp >> 2) * W;
                uint32_t v[W], x1[W];
                if constexpr (W == 32) tmem_ld32(at, v); else if constexpr (W == 16) tmem_ld16(at, v); else tmem_ld8(at, v);
                if constexpr (AFFINE) {
                    const uint32_t ax = at + TC_BUFS * N;
                    if constexpr (W == 32) tmem_ld32(ax, x1); else if constexpr (W == 16) tmem_ld16(ax, x1); else tmem_ld8(ax, x1);
                }
                tmem_wait_ld();
                #pragma unroll
                for (int e = 0; e < W; ++e) {
                    out[e] = fmaf(s, __uint_as_float(v[e]), out[e]);
                    if constexpr (AFFINE) out[e] = fmaf(o, __uint_as_float(x1[e]), out[e]);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dempty0 + 8 * d);
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    // the stages become the tile of sums (all products have ended)
    float* const red = reinterpret_cast<float*>(smem);
    if (warp < TC_EPI) {
        const bool bad = *quit != 0;                         // a wait gave up: NaN rather than a wrong number
        #pragma unroll
        for (int t = 0; t < W; ++t) red[((warp >> 2) * W + t) * 128 + 32 * (warp & 3) + lane] = bad ? __uint_as_float(0x7fffffffu) : out[t];
    }
    if (warp == TC_EPI) {
        __syncwarp();
        tmem_free<1>(tmem, COLUMNS);
    }
    if (splits > 1) cluster_sync();
    else __syncthreads();
    // each CTA of the cluster adds and stores a share of the rows, four at a time: neighbouring lanes, neighbouring rows,
    // so that a warp's read of a peer is one piece
    const int q0 = ROWS / 4 * split / splits, share = ROWS / 4 * (split + 1) / splits - q0;
    for (int e = threadIdx.x; e < share * N; e += TC_THREADS) {
        const int cc = e / share, rr = 4 * (q0 + e - cc * share);
        if (row0 + rr >= m || col0 + cc >= batch) continue;
        float v[NM][4] = {};
        #pragma unroll
        for (int j = 0; j < NM; ++j) {
            const uint32_t at = smem_u32(red + cc * 128 + 64 * j + rr);
            float4 part[8];
            #pragma unroll
            for (int q = 0; q < 8; ++q) part[q] = q < splits ? ld_cluster4(map_rank(at, q)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            #pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[j][0] += part[q].x; v[j][1] += part[q].y; v[j][2] += part[q].z; v[j][3] += part[q].w;
            }
        }
        X* const o = y + (col0 + cc) * ldy + row0 + rr;
        #pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float res = NM == 1 ? v[0][t] : act_rt<PLANES == 3>(act, v[0][t]) * v[NM - 1][t];
            if (row0 + rr + t < m) o[t] = from_f32<X>(res);
        }
    }
    if (splits > 1) cluster_sync();                          // peers may still read this CTA's sums
}

// one call's arguments
struct Product {
    Mat4 w0, w1;
    int64_t m, n;
    int group, act;
    const void* x; int64_t ldx;
    int64_t batch;
    void* y; int64_t ldy;
    cudaStream_t stream;
};

template <typename X, typename T, int NM, int WORDS, bool AFFINE>
cudaError_t launch_vec4(const Product& p) {
    const auto kernel = vec4_kernel<X, T, NM, WORDS, AFFINE>;
    constexpr int smem = VEC_WARPS * VEC_DEPTH * NM * 1024;
    static PerDevice done;
    const cudaError_t e = allow_smem(kernel, smem, done);
    if (e != cudaSuccess) return e;
    const bool vec = row_aligned(p.x, p.batch, p.ldx, sizeof(X));
    kernel<<<(unsigned)((p.m + 15) / 16), VEC_WARPS * 32, smem, p.stream>>>(p.w0, p.w1, p.m, p.n, p.act, (const X*)p.x, p.ldx, (int)vec,
                                                                           (int)p.batch, (X*)p.y, p.ldy);
    return cudaGetLastError();
}

template <typename X, typename T, int NM, int WORDS, bool AFFINE, int N>
cudaError_t launch_tile4(const Product& p) {
    const auto kernel = tile4_kernel<X, T, N, NM, WORDS, AFFINE>;
    constexpr int smem = tc_smem<X, N>();
    static PerDevice done;
    const cudaError_t e = allow_smem(kernel, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.m + 128 / NM - 1) / (128 / NM), cols = (p.batch + N - 1) / N, blocks = (p.n + 127) / 128;
    // Shares of the columns: the fewest rounds of CTAs times the blocks of a share, each CTA costing about
    // nine blocks' time (of 0.8 us) to start, fill its stages and add up.  A round is counted as one CTA an SM, whole clusters
    // or not.  Where the clusters of c CTAs do not fill the GPCs evenly that is too few: 2560 x 6912, 16 vectors, takes
    // 7 shares (20 clusters) for one round and 22.3 us, where 6 shares take 12.7, 5 13.4, 4 15.1 and 1 35.6 (64 vectors: 29.1,
    // 16.1, 17.2, 18.3, 45.2).  4096 x 4096, 64 vectors: 4 shares, 15.7 us, against 18.2 with 3 and 28.3 with 5.
    int splits = 1;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 8 && c <= blocks; ++c) {
        const int64_t cost = (tiles * cols * c + sm_count() - 1) / sm_count() * ((blocks + c - 1) / c + 9);
        if (cost < best) { best = cost; splits = c; }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * splits), (unsigned)cols);
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = p.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p.w0, p.w1, p.m, p.n, p.act, (const X*)p.x, p.ldx, p.batch, (X*)p.y, p.ldy, splits, wait_fault());
}

template <typename X, typename T, int NM, int WORDS, bool AFFINE>
cudaError_t run_kernel(const Product& p) {
    if (p.batch <= VEC_BATCH) return launch_vec4<X, T, NM, WORDS, AFFINE>(p);
    if (p.batch <= 16) return launch_tile4<X, T, NM, WORDS, AFFINE, 16>(p);
    if (p.batch <= 32) return launch_tile4<X, T, NM, WORDS, AFFINE, 32>(p);
    return launch_tile4<X, T, NM, WORDS, AFFINE, 64>(p);
}

template <typename X, typename T, int NM, int WORDS>
cudaError_t run_group(const Product& p) {
    return p.w0.offset || (NM == 2 && p.w1.offset) ? run_kernel<X, T, NM, WORDS, true>(p) : run_kernel<X, T, NM, WORDS, false>(p);
}

template <typename X, typename T, int NM>
cudaError_t run_product(const Product& p) {
    switch (p.group) {
        case 32: return run_group<X, T, NM, 1>(p);
        case 64: return run_group<X, T, NM, 2>(p);
        default: return run_group<X, T, NM, 4>(p);
    }
}

template <int NM>
int products(const Mat4& w0, const Mat4& w1, int64_t m, int64_t n, int group, int act, const void* X, int dtype, int64_t ldx,
             int64_t batch, void* Y, int64_t ldy, void* work, size_t work_bytes, void* stream) {
    if (m < 1 || n < 1 || batch < 0 || !valid_group(group) || !valid_dtype(dtype) || ldx < n || ldy < m) return EXTERND_EINVAL;
    if (NM == 2 && !valid_act(act)) return EXTERND_EINVAL;
    const Device dev;
    const Mat4* w[2] = {&w0, &w1};
    for (int j = 0; j < NM; ++j) {
        if (!w[j]->q || !w[j]->scale || !aligned(w[j]->q, 16) || !aligned(w[j]->scale, 2) || !aligned(w[j]->offset, 2)) return EXTERND_EINVAL;
        if (!dev.holds(w[j]->q) || !dev.holds(w[j]->scale) || (w[j]->offset && !dev.holds(w[j]->offset))) return EXTERND_EINVAL;
    }
    if (batch == 0) return EXTERND_OK;
    const size_t eb = dtype_bytes(dtype);
    if (!X || !Y || !aligned(X, eb) || !aligned(Y, eb) || !dev.holds(X) || !dev.holds(Y)) return EXTERND_EINVAL;
    // grid dimensions, 32-bit column blocks
    if ((m + 15) / 16 > 0x7fffffff / 8 || (batch + 63) / 64 > 65535 || n > 0x7fffffff - 128) return EXTERND_ELIMIT;
    if (work && (!aligned(work, 256) || !dev.holds(work))) return EXTERND_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    AlignJobs jobs = {};
    unsigned char* place = (unsigned char*)work;
    if (batch > VEC_BATCH && !place_rows(jobs, X, ldx, batch, n, eb, place, work_bytes)) return EXTERND_EINVAL;
    const Product p = {w0, w1, m, n, group, act, X, ldx, batch, Y, ldy, s};
    cudaError_t e = launch_align(jobs, s);
    if (e != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
    switch (dtype) {
        case EXTERND_F32: e = run_product<float, __nv_bfloat16, NM>(p); break;
        case EXTERND_F16: e = run_product<__half, __half, NM>(p); break;
        default: e = run_product<__nv_bfloat16, __nv_bfloat16, NM>(p); break;
    }
    if (e != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
    return EXTERND_OK;
}

// rows in x; y splits a row where the rows alone leave the SMs short of warps
dim3 row_grid(int64_t m, int64_t steps) {
    const int64_t x = (m + 7) / 8, want = (int64_t)sm_count() * 16;
    int64_t y = x >= want ? 1 : (want + x - 1) / x;
    y = y < steps ? y : steps;
    return dim3((unsigned)x, (unsigned)(y < 65535 ? y : 65535));
}

int log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

template <typename T, bool AFFINE, int LG>
cudaError_t run_quantize(const void* A, int64_t m, int64_t n, int64_t lda, uint8_t* q, void* scale, void* offset, int* status,
                         cudaStream_t s) {
    const dim3 grid = row_grid(m, ((n + 255) / 256 + QPAIRS - 1) / QPAIRS);
    const bool vec = aligned(A, 16) && lda * sizeof(T) % 16 == 0;
    const auto kernel = vec ? quantize_kernel<T, AFFINE, true, LG> : quantize_kernel<T, AFFINE, false, LG>;
    kernel<<<grid, 256, 0, s>>>((const T*)A, m, n, lda, (uint32_t*)q, (__half*)scale, (__half*)offset, status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_quantize(const void* A, int64_t m, int64_t n, int64_t lda, int group, uint8_t* q, void* scale, void* offset,
                         int* status, cudaStream_t s) {
    switch (log2_of(group) + (offset ? 8 : 0)) {
        case 5: return run_quantize<T, false, 5>(A, m, n, lda, q, scale, offset, status, s);
        case 6: return run_quantize<T, false, 6>(A, m, n, lda, q, scale, offset, status, s);
        case 7: return run_quantize<T, false, 7>(A, m, n, lda, q, scale, offset, status, s);
        case 13: return run_quantize<T, true, 5>(A, m, n, lda, q, scale, offset, status, s);
        case 14: return run_quantize<T, true, 6>(A, m, n, lda, q, scale, offset, status, s);
        default: return run_quantize<T, true, 7>(A, m, n, lda, q, scale, offset, status, s);
    }
}

template <typename T>
cudaError_t run_dequantize(const uint8_t* q, const void* scale, const void* offset, int64_t m, int64_t n, int group, void* out,
                           int64_t ldo, cudaStream_t s) {
    const dim3 grid = row_grid(m, ((n + 127) / 128 + 7) / 8);
    // fp32 rows always pass through shared memory: 16 bytes a lane, 32 apart, take 21.0 us for 2560 x 6912 where this
    // takes 13.9 (8192 x 28672: 245 and 185)
    auto kernel = dequantize_kernel<T, false>;
    if constexpr (sizeof(T) == 2)
        if (row_aligned(out, m, ldo, sizeof(T))) kernel = dequantize_kernel<T, true>;
    kernel<<<grid, 256, 0, s>>>((const uint32_t*)q, (const __half*)scale, (const __half*)offset, m, n, log2_of(group), (T*)out, ldo);
    return cudaGetLastError();
}

}  // namespace externd_int4

using namespace externd_int4;

extern "C" {

size_t externd_int4_row_bytes(int64_t n) { return n < 1 ? 0 : (size_t)row_bytes(n); }

int externd_int4_quantize(const void* A, int dtype, int64_t m, int64_t n, int64_t lda, int group, uint8_t* q_out, void* scale_out,
                          void* offset_out, int* async_status, void* stream) {
    if (!A || !q_out || !scale_out || m < 1 || n < 1 || lda < n || !valid_dtype(dtype) || !valid_group(group)) return EXTERND_EINVAL;
    if (!aligned(A, dtype_bytes(dtype)) || !aligned(q_out, 16) || !aligned(scale_out, 2) || !aligned(offset_out, 2) ||
        !aligned(async_status, 4))
        return EXTERND_EINVAL;
    if (m > 0x7fffffffll * 8 || n > 0x7fffffff - 128) return EXTERND_ELIMIT;
    const Device dev;
    if (!dev.holds(A) || !dev.holds(q_out) || !dev.holds(scale_out) || (offset_out && !dev.holds(offset_out)) ||
        (async_status && !dev.holds(async_status)))
        return EXTERND_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* status = async_status;
    if (!status && cudaMallocAsync((void**)&status, sizeof(int), s) != cudaSuccess) { cudaGetLastError(); return EXTERND_ENOMEM; }
    int rc = EXTERND_OK;
    cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int), s);
    if (e == cudaSuccess) {
        switch (dtype) {
            case EXTERND_F32: e = run_quantize<float>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s); break;
            case EXTERND_F16: e = run_quantize<__half>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s); break;
            default: e = run_quantize<__nv_bfloat16>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s); break;
        }
    }
    if (e != cudaSuccess) { cudaGetLastError(); rc = EXTERND_ECUDA; }
    if (!async_status) {
        int got = 0;
        if (cudaMemcpyAsync(&got, status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess) { cudaGetLastError(); rc = EXTERND_ECUDA; }
        cudaFreeAsync(status, s);
        cudaGetLastError();
        if (rc == EXTERND_OK) rc = got;
    }
    return rc;
}

int externd_int4_dequantize(const uint8_t* q, const void* scale, const void* offset, int64_t m, int64_t n, int group, void* out,
                            int dtype, int64_t ldo, void* stream) {
    if (!q || !scale || !out || m < 1 || n < 1 || ldo < n || !valid_dtype(dtype) || !valid_group(group)) return EXTERND_EINVAL;
    if (!aligned(q, 16) || !aligned(scale, 2) || !aligned(offset, 2) || !aligned(out, dtype_bytes(dtype))) return EXTERND_EINVAL;
    if (m > 0x7fffffffll * 8 || n > 0x7fffffff - 128) return EXTERND_ELIMIT;
    const Device dev;
    if (!dev.holds(q) || !dev.holds(scale) || (offset && !dev.holds(offset)) || !dev.holds(out)) return EXTERND_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case EXTERND_F32: e = run_dequantize<float>(q, scale, offset, m, n, group, out, ldo, s); break;
        case EXTERND_F16: e = run_dequantize<__half>(q, scale, offset, m, n, group, out, ldo, s); break;
        default: e = run_dequantize<__nv_bfloat16>(q, scale, offset, m, n, group, out, ldo, s); break;
    }
    if (e != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
    return EXTERND_OK;
}

int externd_int4_matvec(const uint8_t* q, const void* scale, const void* offset, int64_t m, int64_t n, int group, const void* X,
                        int dtype, int64_t ldx, int64_t batch, void* Y, int64_t ldy, void* work, size_t work_bytes, void* stream) {
    const Mat4 w = {q, (const __half*)scale, (const __half*)offset};
    return products<1>(w, Mat4{}, m, n, group, 0, X, dtype, ldx, batch, Y, ldy, work, work_bytes, stream);
}

int externd_int4_gated(const uint8_t* qg, const void* scale_g, const void* offset_g, const uint8_t* qu, const void* scale_u,
                       const void* offset_u, int64_t m, int64_t n, int group, int act, const void* X, int dtype, int64_t ldx,
                       int64_t batch, void* H, int64_t ldh, void* work, size_t work_bytes, void* stream) {
    const Mat4 wg = {qg, (const __half*)scale_g, (const __half*)offset_g}, wu = {qu, (const __half*)scale_u, (const __half*)offset_u};
    return products<2>(wg, wu, m, n, group, act, X, dtype, ldx, batch, H, ldh, work, work_bytes, stream);
}

}  // extern "C"
