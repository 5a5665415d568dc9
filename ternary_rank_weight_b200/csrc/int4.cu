// 4-bit weights with group scales (sm_100a): quantiser, dequantiser and the products that stream the
// weights once -- Y = X W^T and the gated H = act(X Wg^T) * (X Wu^T) for 4-bit and for dense 16-bit weights.
//
// Format: w = s (q - 8) + b, q in 0..15, s and b fp16 per row and group of 32, 64 or 128 columns.  A row of
// codes is blocks of 128 columns in 64 bytes; column 128 B + 32 i + 8 c + t is nibble 4 (t % 2) + t / 2 of
// word 4 c + i of block B.  A lane c of four that loads 16 bytes of a block thus holds, word by word, 8
// consecutive columns of each of the block's four 32-column spans: the four lanes together cover one span
// (one group at most) per word, and (word >> 4 p) & 0x000f000f is a pair of neighbouring columns, ready to
// become two 16-bit floats.
#include "llm_ops.cuh"

namespace externd_int4 {

using namespace externd_llm;

__host__ __device__ __forceinline__ int64_t row_bytes(int64_t n) { return (n + 127) / 128 * 64; }

// ---------------------------------------------------------------------------------------------------
// quantise: one warp per row and block of 128 columns; lane L holds columns 4 L .. 4 L + 3
// ---------------------------------------------------------------------------------------------------
//
// One pass over A: the group's extremes stay in registers.  Bound by memory when the arithmetic stays in
// fp32; the format's fp64 decisions are taken in fp64 only next to a border (1e-4-wide bands around the
// rounding borders of codes, 2^-10 of the scales), where the fp32 value cannot decide.

// fp16 of the fp64 value v (rounded to fp32 first), given its fp32 estimate e with relative error below
// 2^-21: `near` says that e does not decide it
__device__ __forceinline__ bool near_half_border(float e) {
    const uint32_t u = __float_as_uint(e) & 0x7fffffffu;
    const uint32_t low = u & 0x1fffu;                       // bits below the fp16 mantissa
    return u < 0x38800000u + 64u || (low > 0x1000u - 16u && low < 0x1000u + 16u);   // below 2^-14: fp16 subnormals
}

template <typename T, bool AFFINE, bool VEC>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ A, int64_t m, int64_t n, int64_t lda, int group,
                                                       uint32_t* __restrict__ q, __half* __restrict__ scale,
                                                       __half* __restrict__ offset, int* __restrict__ status) {
    const int lane = threadIdx.x & 31;
    const int64_t blocks = (n + 127) / 128;
    const int64_t items = m * blocks;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t item = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; item < items; item += warps) {
        // neighbouring warps take neighbouring rows of one block: their scales share a sector
        const int64_t blk = item / m, row = item - blk * m;
        const int64_t j0 = blk * 128 + 4 * lane;
        const T* a = A + row * lda + j0;
        float w[4];
        if (VEC && j0 + 4 <= n) {
            if constexpr (sizeof(T) == 4) {
                const float4 v = __ldcs(reinterpret_cast<const float4*>(a));
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
                const uint2 v = __ldcs(reinterpret_cast<const uint2*>(a));
                const float2 lo = unpack2<T>(v.x), hi = unpack2<T>(v.y);
                w[0] = lo.x; w[1] = lo.y; w[2] = hi.x; w[3] = hi.y;
            }
        } else {
            #pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = j0 + t < n ? to_f32(a[t]) : 0.0f;
        }
        float mn = INFINITY, mx = -INFINITY;
        bool finite = true;
        #pragma unroll
        for (int t = 0; t < 4; ++t)
            if (j0 + t < n) {
                finite = finite && fabsf(w[t]) <= FLT_MAX;
                mn = fminf(mn, w[t]);
                mx = fmaxf(mx, w[t]);
            }
        for (int o = 1; o < group / 4; o <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(FULL, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        }
        const bool any = j0 / group * group < n;   // the group has columns
        float s = 0.0f, b = 0.0f;
        if (any) {
            float e = AFFINE ? (mx - mn) / 15.0f : fmaxf(-mn, mx) / 7.0f;
            if (near_half_border(e) || e > 65000.0f)
                e = (float)(AFFINE ? ((double)mx - (double)mn) / 15.0 : (double)fmaxf(-mn, mx) / 7.0);
            s = __half2float(__float2half_rn(e));
            if (AFFINE) {
                float f = fmaf(8.0f, s, mn);
                if (near_half_border(f)) f = (float)((double)mn + 8.0 * (double)s);
                b = __half2float(__float2half_rn(f));
            }
        }
        // a group with NaN or Inf reports that, whatever other groups report
        if (!finite) atomicExch(status, EXTERND_ENONFINITE);
        else if (fmaxf(-mn, mx) <= FLT_MAX && (isinf(s) || isinf(b))) atomicCAS(status, EXTERND_OK, EXTERND_ELIMIT);
        const float inv = s > 0.0f ? 1.0f / s : 0.0f;
        uint32_t code = 0;
        #pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float d = AFFINE ? w[t] - b : w[t];
            float c = d * inv;
            float r = rintf(c);
            // |c| <= 16 wherever it is not clamped: its error is below 1e-5
            if (fabsf(fabsf(c - r) - 0.5f) < 1e-4f && fabsf(c) < 16.0f && s > 0.0f)
                r = (float)rint(((double)w[t] - (double)b) / (double)s);
            r = fminf(fmaxf(r, -8.0f), 7.0f);
            const int v = j0 + t < n ? (int)r + 8 : 8;
            code |= (uint32_t)v << (4 * (4 * (t & 1) + (t >> 1)));
        }
        if (lane & 1) code <<= 8;                              // t = 4..7 sit two nibbles above t = 0..3
        code |= __shfl_xor_sync(FULL, code, 1);
        if (!(lane & 1)) {
            const int word = 4 * ((lane % 8) / 2) + lane / 8;   // 4 c + i
            q[(row * blocks + blk) * 16 + word] = code;
        }
        if (any && (4 * lane) % group == 0) {
            const int64_t at = (j0 / group) * m + row;
            scale[at] = __float2half_rn(s);
            if (AFFINE) offset[at] = __float2half_rn(b);
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// dequantise: lane L of a half-warp holds the 8 columns 8 L .. 8 L + 7 of a block
// ---------------------------------------------------------------------------------------------------

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint32_t* __restrict__ q, const __half* __restrict__ scale,
                                                         const __half* __restrict__ offset, int64_t m, int64_t n, int group,
                                                         T* __restrict__ out, int64_t ldo) {
    const int64_t blocks = (n + 127) / 128;
    const int64_t items = m * blocks;
    const int l = threadIdx.x & 15;
    const int64_t halves = (int64_t)gridDim.x * (blockDim.x / 16);
    for (int64_t item = (int64_t)blockIdx.x * (blockDim.x / 16) + threadIdx.x / 16; item < items; item += halves) {
        const int64_t row = item / blocks, blk = item - row * blocks;
        const int64_t j0 = blk * 128 + 8 * l;
        if (j0 >= n) continue;
        const uint32_t w = q[item * 16 + 4 * (l & 3) + (l >> 2)];
        const int64_t at = (j0 / group) * m + row;
        const float s = __half2float(scale[at]), b = offset ? __half2float(offset[at]) : 0.0f;
        float v[8];
        #pragma unroll
        for (int t = 0; t < 8; ++t)
            v[t] = fmaf(s, (float)((int)((w >> (4 * (4 * (t & 1) + (t >> 1)))) & 15u) - 8), b);
        T* o = out + row * ldo + j0;
        if (VEC && j0 + 8 <= n) {
            if constexpr (sizeof(T) == 4) {
                __stcs(reinterpret_cast<float4*>(o), make_float4(v[0], v[1], v[2], v[3]));
                __stcs(reinterpret_cast<float4*>(o) + 1, make_float4(v[4], v[5], v[6], v[7]));
            } else {
                __stcs(reinterpret_cast<uint4*>(o), make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                               pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])));
            }
        } else {
            #pragma unroll
            for (int t = 0; t < 8; ++t)
                if (j0 + t < n) o[t] = from_f32<T>(v[t]);
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// products: a CTA of WARPS warps takes 16 rows of W (of both matrices when gated) and 8 NT vectors; its warps
// split the columns and add their partial sums in shared memory in a fixed order
// ---------------------------------------------------------------------------------------------------
//
// Bound by the weights' bytes for few vectors.  The tensor cores' warp-level product does the arithmetic:
// codes become exact 16-bit floats q - 8 two at a time, eight vectors ride in one instruction, and each
// group's fp32 sum is scaled once.  (The tile-level product of the tensor cores reads its operands from
// shared memory: the weights would cross it twice more, for arithmetic that does not bound here.)
// fp32 vectors enter as three bf16 terms x = hi + mid + lo cut off from the top (8 + 8 + 8 bits: no loss),
// three products into one sum.  The offsets' part b sum(x) takes sum(x) from a product with ones.

// a pair of codes -> a pair of floats q - 8; p = 0..3 selects the pair of the word
template <typename T> __device__ __forceinline__ void codes8(uint32_t w, uint32_t (&a)[4]);
template <> __device__ __forceinline__ void codes8<__half>(uint32_t w, uint32_t (&a)[4]) {
    // 0x6400 | q = 1024 + q, 0x6400 | 16 q = 1024 + 16 q (exact); subtract 1032, or scale by 1/16 and subtract 72
    const __half2 k1032 = __half2half2(__ushort_as_half(0x6408)), sixteenth = __half2half2(__ushort_as_half(0x2c00)),
                  m72 = __half2half2(__ushort_as_half(0xd480));
    const uint32_t w8 = w >> 8;
    const uint32_t u0 = (w & 0x000f000fu) | 0x64006400u, u1 = (w & 0x00f000f0u) | 0x64006400u;
    const uint32_t u2 = (w8 & 0x000f000fu) | 0x64006400u, u3 = (w8 & 0x00f000f0u) | 0x64006400u;
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
        const uint32_t u = ((w >> (4 * p)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), k136);
        a[p] = *reinterpret_cast<const uint32_t*>(&v);
    }
}

struct Mat4 {                       // one 4-bit matrix
    const uint8_t* q;
    const __half* scale;
    const __half* offset;           // nullptr: symmetric
};

template <typename T> __device__ constexpr uint32_t one2();
template <> __device__ constexpr uint32_t one2<__half>() { return 0x3c003c00u; }
template <> __device__ constexpr uint32_t one2<__nv_bfloat16>() { return 0x3f803f80u; }

// X element type, T product type (bf16 for fp32 X), NM matrices (1, or 2: gated)
template <typename X, typename T, int NT, int NM, int WARPS, bool VEC>
__global__ void __launch_bounds__(WARPS * 32) stream4_kernel(Mat4 w0, Mat4 w1, int64_t m, int64_t n, int group, int act,
                                                            const X* __restrict__ x, int64_t ldx, int64_t batch,
                                                            X* __restrict__ y, int64_t ldy) {
    constexpr int PLANES = sizeof(X) == 4 ? 3 : 1;
    constexpr int COLS = 8 * NT;
    __shared__ float part[NM][WARPS][16][COLS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int64_t col0 = (int64_t)blockIdx.y * COLS;
    const int64_t blocks = (n + 127) / 128;
    // rows past the last one repeat it (their sums are not stored)
    const int64_t ra = min(row0 + r, m - 1), rb = min(row0 + r + 8, m - 1);
    const Mat4 w[2] = {w0, w1};
    const bool affine = w0.offset != nullptr || (NM == 2 && w1.offset != nullptr);
    const int words = group / 32;                       // words of a block that share a group

    const X* xr[NT];
    #pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = col0 + 8 * t + r < batch ? x + (col0 + 8 * t + r) * ldx : nullptr;

    float out[NM][NT][4] = {};
    for (int64_t blk = warp; blk < blocks; blk += WARPS) {
        uint4 qa[NM], qb[NM];
        #pragma unroll
        for (int j = 0; j < NM; ++j) {
            qa[j] = __ldcs(reinterpret_cast<const uint4*>(w[j].q + (ra * blocks + blk) * 64 + 16 * c));
            qb[j] = __ldcs(reinterpret_cast<const uint4*>(w[j].q + (rb * blocks + blk) * 64 + 16 * c));
        }
        float acc[NM][NT][4] = {}, sum[NT][4] = {};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = blk * 128 + 32 * i + 8 * c;
            XFrag<T, PLANES> xf[NT];
            #pragma unroll
            for (int t = 0; t < NT; ++t) load_x<X, T, PLANES, VEC>(xr[t], k, n, xf[t]);
            #pragma unroll
            for (int j = 0; j < NM; ++j) {
                const uint32_t wa = i == 0 ? qa[j].x : i == 1 ? qa[j].y : i == 2 ? qa[j].z : qa[j].w;
                const uint32_t wb = i == 0 ? qb[j].x : i == 1 ? qb[j].y : i == 2 ? qb[j].z : qb[j].w;
                uint32_t a[4], b[4];
                codes8<T>(wa, a);
                codes8<T>(wb, b);
                #pragma unroll
                for (int t = 0; t < NT; ++t)
                    #pragma unroll
                    for (int p = PLANES - 1; p >= 0; --p) {
                        mma16816<T>(acc[j][t], a[0], b[0], a[1], b[1], xf[t].v[p][0], xf[t].v[p][1]);
                        mma16816<T>(acc[j][t], a[2], b[2], a[3], b[3], xf[t].v[p][2], xf[t].v[p][3]);
                    }
            }
            if (affine) {
                #pragma unroll
                for (int t = 0; t < NT; ++t)
                    #pragma unroll
                    for (int p = PLANES - 1; p >= 0; --p) {
                        mma16816<T>(sum[t], one2<T>(), one2<T>(), one2<T>(), one2<T>(), xf[t].v[p][0], xf[t].v[p][1]);
                        mma16816<T>(sum[t], one2<T>(), one2<T>(), one2<T>(), one2<T>(), xf[t].v[p][2], xf[t].v[p][3]);
                    }
            }
            if ((i + 1) % words == 0 && blk * 128 + 32 * (i + 1 - words) < n) {   // the group ends here
                const int64_t at = (blk * 128 + 32 * i) / group * m;
                #pragma unroll
                for (int j = 0; j < NM; ++j) {
                    const float sa = __half2float(__ldg(w[j].scale + at + ra)), sb = __half2float(__ldg(w[j].scale + at + rb));
                    float ba = 0.0f, bb = 0.0f;
                    if (w[j].offset) {
                        ba = __half2float(__ldg(w[j].offset + at + ra));
                        bb = __half2float(__ldg(w[j].offset + at + rb));
                    }
                    #pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        out[j][t][0] = fmaf(sa, acc[j][t][0], out[j][t][0]);
                        out[j][t][1] = fmaf(sa, acc[j][t][1], out[j][t][1]);
                        out[j][t][2] = fmaf(sb, acc[j][t][2], out[j][t][2]);
                        out[j][t][3] = fmaf(sb, acc[j][t][3], out[j][t][3]);
                        if (w[j].offset) {
                            out[j][t][0] = fmaf(ba, sum[t][0], out[j][t][0]);
                            out[j][t][1] = fmaf(ba, sum[t][1], out[j][t][1]);
                            out[j][t][2] = fmaf(bb, sum[t][2], out[j][t][2]);
                            out[j][t][3] = fmaf(bb, sum[t][3], out[j][t][3]);
                        }
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][t][e] = 0.0f;
                    }
                }
                #pragma unroll
                for (int t = 0; t < NT; ++t)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) sum[t][e] = 0.0f;
            }
        }
    }
    #pragma unroll
    for (int j = 0; j < NM; ++j)
        #pragma unroll
        for (int t = 0; t < NT; ++t) {
            part[j][warp][r][8 * t + 2 * c] = out[j][t][0];
            part[j][warp][r][8 * t + 2 * c + 1] = out[j][t][1];
            part[j][warp][r + 8][8 * t + 2 * c] = out[j][t][2];
            part[j][warp][r + 8][8 * t + 2 * c + 1] = out[j][t][3];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * COLS; e += WARPS * 32) {
        const int rr = e & 15, cc = e >> 4;
        if (row0 + rr >= m || col0 + cc >= batch) continue;
        float v[NM] = {};
        #pragma unroll
        for (int j = 0; j < NM; ++j)
            #pragma unroll
            for (int p = 0; p < WARPS; ++p) v[j] += part[j][p][rr][cc];
        const float res = NM == 1 ? v[0] : act_rt<sizeof(X) == 4>(act, v[0]) * v[NM - 1];
        y[(col0 + cc) * ldy + row0 + rr] = from_f32<X>(res);
    }
}

template <typename X, typename T, int NT, int NM, int WARPS>
cudaError_t launch_stream4(const Mat4& w0, const Mat4& w1, int64_t m, int64_t n, int group, int act, const void* x, int64_t ldx,
                           int64_t batch, void* y, int64_t ldy, cudaStream_t s) {
    const dim3 grid((unsigned)((m + 15) / 16), (unsigned)((batch + 8 * NT - 1) / (8 * NT)));
    const bool vec = aligned(x, 16) && ldx * sizeof(X) % 16 == 0;
    if (vec) stream4_kernel<X, T, NT, NM, WARPS, true><<<grid, WARPS * 32, 0, s>>>(w0, w1, m, n, group, act, (const X*)x, ldx, batch, (X*)y, ldy);
    else stream4_kernel<X, T, NT, NM, WARPS, false><<<grid, WARPS * 32, 0, s>>>(w0, w1, m, n, group, act, (const X*)x, ldx, batch, (X*)y, ldy);
    return cudaGetLastError();
}

template <typename X, typename T, int NM>
cudaError_t run_stream4(const Mat4& w0, const Mat4& w1, int64_t m, int64_t n, int group, int act, const void* x, int64_t ldx,
                        int64_t batch, void* y, int64_t ldy, cudaStream_t s) {
    if (batch <= 8) return launch_stream4<X, T, 1, NM, 8>(w0, w1, m, n, group, act, x, ldx, batch, y, ldy, s);
    return launch_stream4<X, T, 4, NM, 4>(w0, w1, m, n, group, act, x, ldx, batch, y, ldy, s);
}

template <int NM>
int products(const Mat4& w0, const Mat4& w1, int64_t m, int64_t n, int group, int act, const void* X, int dtype, int64_t ldx,
             int64_t batch, void* Y, int64_t ldy, void* stream) {
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
    if ((m + 15) / 16 > 0x7fffffff || (batch + 7) / 8 > 65535) return EXTERND_ELIMIT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case EXTERND_F32: e = run_stream4<float, __nv_bfloat16, NM>(w0, w1, m, n, group, act, X, ldx, batch, Y, ldy, s); break;
        case EXTERND_F16: e = run_stream4<__half, __half, NM>(w0, w1, m, n, group, act, X, ldx, batch, Y, ldy, s); break;
        default: e = run_stream4<__nv_bfloat16, __nv_bfloat16, NM>(w0, w1, m, n, group, act, X, ldx, batch, Y, ldy, s); break;
    }
    if (e != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
    return EXTERND_OK;
}

unsigned grid_for(int64_t items, int per_cta) {
    const int64_t want = (items + per_cta - 1) / per_cta, cap = (int64_t)sm_count() * 64;
    return (unsigned)(want < cap ? want : cap);
}

template <typename T, bool AFFINE>
cudaError_t run_quantize(const void* A, int64_t m, int64_t n, int64_t lda, int group, uint8_t* q, void* scale, void* offset,
                         int* status, cudaStream_t s) {
    const unsigned grid = grid_for(m * ((n + 127) / 128), 8);
    const bool vec = aligned(A, 4 * sizeof(T)) && lda % 4 == 0;
    if (vec) quantize_kernel<T, AFFINE, true><<<grid, 256, 0, s>>>((const T*)A, m, n, lda, group, (uint32_t*)q, (__half*)scale, (__half*)offset, status);
    else quantize_kernel<T, AFFINE, false><<<grid, 256, 0, s>>>((const T*)A, m, n, lda, group, (uint32_t*)q, (__half*)scale, (__half*)offset, status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_dequantize(const uint8_t* q, const void* scale, const void* offset, int64_t m, int64_t n, int group, void* out,
                           int64_t ldo, cudaStream_t s) {
    const unsigned grid = grid_for(m * ((n + 127) / 128), 16);
    const bool vec = aligned(out, 16) && ldo * sizeof(T) % 16 == 0;
    if (vec) dequantize_kernel<T, true><<<grid, 256, 0, s>>>((const uint32_t*)q, (const __half*)scale, (const __half*)offset, m, n, group, (T*)out, ldo);
    else dequantize_kernel<T, false><<<grid, 256, 0, s>>>((const uint32_t*)q, (const __half*)scale, (const __half*)offset, m, n, group, (T*)out, ldo);
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
        const bool aff = offset_out != nullptr;
        switch (dtype) {
            case EXTERND_F32:
                e = aff ? run_quantize<float, true>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s)
                        : run_quantize<float, false>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s);
                break;
            case EXTERND_F16:
                e = aff ? run_quantize<__half, true>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s)
                        : run_quantize<__half, false>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s);
                break;
            default:
                e = aff ? run_quantize<__nv_bfloat16, true>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s)
                        : run_quantize<__nv_bfloat16, false>(A, m, n, lda, group, q_out, scale_out, offset_out, status, s);
                break;
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
                        int dtype, int64_t ldx, int64_t batch, void* Y, int64_t ldy, void* stream) {
    const Mat4 w = {q, (const __half*)scale, (const __half*)offset};
    return products<1>(w, Mat4{}, m, n, group, 0, X, dtype, ldx, batch, Y, ldy, stream);
}

int externd_int4_gated(const uint8_t* qg, const void* scale_g, const void* offset_g, const uint8_t* qu, const void* scale_u,
                       const void* offset_u, int64_t m, int64_t n, int group, int act, const void* X, int dtype, int64_t ldx,
                       int64_t batch, void* H, int64_t ldh, void* stream) {
    const Mat4 wg = {qg, (const __half*)scale_g, (const __half*)offset_g}, wu = {qu, (const __half*)scale_u, (const __half*)offset_u};
    return products<2>(wg, wu, m, n, group, act, X, dtype, ldx, batch, H, ldh, stream);
}

}  // extern "C"
