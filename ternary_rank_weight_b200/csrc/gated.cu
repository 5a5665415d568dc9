// The dense gated feed-forward block (sm_100a): H = act(G) * U with G = X Wg^T, U = X Wu^T, and its gradients
//     dG = dH U act'(G),  dU = dH act(G),  dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
// for bf16 and fp16, fp32 sums.
//
// Few tokens: the weights stream once through the warp-level products (dense_stream_kernel).  Otherwise one
// persistent kernel on the 5th-generation tensor cores (gemm_kernel): TMA brings 64-deep operand slabs into
// a ring of swizzled shared-memory stages, one thread issues tcgen05.mma into tensor memory, four warps drain
// a finished accumulator while the next one fills.  It runs as
//   FWD  both projections of a tile in one 256-column accumulator, activation and product in the epilogue;
//   DX   dG Wg + dU Wu as one sum of 2 m terms (weights read along their columns, as stored);
//   DW   dG^T X and dU^T X as one list of tiles (both operands read along their columns, as stored).
#include <cuda.h>

#include "llm_ops.cuh"

namespace externd_gated {

using namespace externd_llm;

// ---------------------------------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ uint64_t timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// arrive on a barrier of any CTA of the cluster (shared::cluster address)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;   // per wait, as for the factorizations

// Wait for a phase.  Gives up after WAIT_LIMIT_NS, or when another warp of the CTA gave up: the CTA then
// leaves its loops and the launch reports EXTERND_ETIMEOUT.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
    if (mbar_try(bar, parity)) return true;
    uint64_t t0 = 0;
    for (;;) {
        #pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try(bar, parity)) return true;
        if (*abort) return false;
        const uint64_t t = timer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > WAIT_LIMIT_NS) { *abort = 1; return false; }
    }
}

// 2-D tiled load, box at (x, y); completes on `bar` (shared::cluster address)
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if constexpr (CG == 1)
        asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}

// arrive on `bar` (in both CTAs of a pair) when the MMAs issued so far have finished
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(bar), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
          "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------------------------------
// the tile kernel
// ---------------------------------------------------------------------------------------------------

enum Mode { FWD = 0, DX = 1, DW = 2 };

constexpr int BK = 64;                     // depth of one stage: 128 bytes, one swizzle span
constexpr int THREADS = 256;               // warp 0 TMA, warp 1 MMA, warps 4-7 epilogue
constexpr int ACC = 256;                   // accumulator columns; two accumulators fill tensor memory
constexpr int STG_ROW = 80;                // bytes of a staged row of 32 outputs (64 + 16: no bank conflicts)

template <int CG> struct Cfg {
    static constexpr int BM = 128 * CG;                    // tile rows (128 per CTA)
    static constexpr int BBYTES = 256 / CG * BK * 2;       // a CTA's share of the 256 B rows
    static constexpr int STAGE = 128 * BK * 2 + BBYTES;
    static constexpr int STAGES = CG == 1 ? 4 : 6;
    static constexpr int SMEM = STAGES * STAGE + 4 * 32 * STG_ROW + 1024 + 256;
};

struct GemmArgs {
    int rows, cols;          // outputs: FWD tokens x m; DX tokens x n; DW 2 x (m x n), rows = m
    int depth;               // FWD n; DX m (per half); DW tokens
    int tiles_r, tiles_c;    // tile grid (DW: tiles_r counts both matrices)
    int act;
    void* out0; int64_t ld0; // FWD H, DX dX, DW dWg
    void* out1; int64_t ld1; // FWD G, DW dWu (FWD: may be null)
    void* out2;              // FWD U, leading dimension ld1
    int* status;             // may be null
};

// shared-memory operand descriptor, 128-byte swizzle: start, leading and stride byte offsets
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// 32 columns of a warp's 32 rows, packed (16 registers a row), to global memory through the warp's staging
// buffer: four lanes write a row's 64 bytes
template <typename T>
__device__ __forceinline__ void store32(const uint32_t (&v)[16], uint32_t stg, const unsigned char* stg_ptr, T* out, int64_t ld,
                                        int row0, int rows, int col0, int cols, int lane) {
    #pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(stg + lane * STG_ROW + 16 * i), "r"(v[4 * i]), "r"(v[4 * i + 1]),
                     "r"(v[4 * i + 2]), "r"(v[4 * i + 3]) : "memory");
    __syncwarp();
    const bool vec = col0 + 32 <= cols && (ld & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    if (vec) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2), c = lane & 3;
            const uint4 w = *reinterpret_cast<const uint4*>(stg_ptr + r * STG_ROW + 16 * c);
            if (row0 + r < rows) *reinterpret_cast<uint4*>(out + (int64_t)(row0 + r) * ld + col0 + 8 * c) = w;
        }
    } else {
        #pragma unroll 4
        for (int r = 0; r < 32; ++r) {
            const T w = *reinterpret_cast<const T*>(stg_ptr + r * STG_ROW + 2 * lane);
            if (row0 + r < rows && col0 + lane < cols) out[(int64_t)(row0 + r) * ld + col0 + lane] = w;
        }
    }
    __syncwarp();
}

template <typename T, int ACT>
__device__ __forceinline__ void gate_chunk(const uint32_t (&g)[32], const uint32_t (&u)[32], uint32_t (&h)[16]) {
    #pragma unroll
    for (int i = 0; i < 16; ++i)
        h[i] = pack2<T>(act_fn<ACT, false>(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                        act_fn<ACT, false>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
}

template <typename T>
__device__ __forceinline__ void pack_chunk(const uint32_t (&v)[32], uint32_t (&h)[16]) {
    #pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = pack2<T>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// tile t -> (row tile, column tile): bands of 8 row tiles walked column by column, so the tiles in flight
// share operands in L2
__device__ __forceinline__ void tile_at(int t, int tiles_r, int tiles_c, int& r, int& c) {
    const int band = t / (8 * tiles_c), first = band * 8;
    const int h = min(8, tiles_r - first), in = t - band * 8 * tiles_c;
    c = in / h;
    r = first + in - c * h;
}

template <typename T, int MODE, int CG>
__global__ void __launch_bounds__(THREADS, 1) gemm_kernel(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap a1,
                                                          const __grid_constant__ CUtensorMap b0, const __grid_constant__ CUtensorMap b1,
                                                          const GemmArgs g) {
    using C = Cfg<CG>;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[2 * C::STAGES + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;          // swizzle atoms are 1024-byte aligned
    unsigned char* const stg_base = raw + (base - smem_u32(raw)) + C::STAGES * C::STAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0 : cluster_rank();
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES, tfull0 = empty0 + 8 * C::STAGES, tempty0 = tfull0 + 16,
                   drain = tempty0 + 16;
    volatile int* const abort = &abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, 4 * CG);                      // one arrival per epilogue warp of the pair
        }
        mbar_init(drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;

    const int kb_half = (g.depth + BK - 1) / BK;
    const int kbs = MODE == DX ? 2 * kb_half : kb_half;
    const int tiles = g.tiles_r * g.tiles_c;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int half_r = g.tiles_r / 2;                                  // DW: row tiles of one matrix

    if (warp == 0 && lane == 0) {
        // ---- loads: each CTA fetches its 128 rows of A and its share of B; both complete on the leader's barrier
        int it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            int tr, tc;
            tile_at(t, g.tiles_r, g.tiles_c, tr, tc);
            const CUtensorMap *ma = &a0, *mb = MODE == FWD && CG == 2 && rank == 1 ? &b1 : &b0;
            int rr = tr;
            if (MODE == DW && tr >= half_r) { ma = &a1; rr -= half_r; }
            const int ar = rr * C::BM + 128 * (int)rank;               // first A row (FWD, DX: token; DW: row of the matrix)
            for (int kb = 0; kb < kbs; ++kb, ++it) {
                const int s = it % C::STAGES;
                if (!mbar_wait(empty0 + 8 * s, ((it / C::STAGES) & 1) ^ 1, abort)) { ok = false; break; }
                const uint32_t sa = base + s * C::STAGE, sb = sa + 128 * BK * 2;
                uint32_t bar = full0 + 8 * s;
                if (rank == 0) mbar_expect(bar, CG * C::STAGE);
                if constexpr (CG == 2) bar = map_rank(bar, 0);
                if constexpr (MODE == FWD) {
                    tma_load<CG>(sa, ma, kb * BK, ar, bar);
                    tma_load<CG>(sb, mb, kb * BK, tc * 128, bar);       // CG 1: Wg, then Wu; CG 2: Wg in CTA 0, Wu in CTA 1
                    if constexpr (CG == 1) tma_load<CG>(sb + 128 * BK * 2, &b1, kb * BK, tc * 128, bar);
                } else if constexpr (MODE == DX) {
                    const bool second = kb >= kb_half;
                    const int k = (second ? kb - kb_half : kb) * BK;
                    tma_load<CG>(sa, second ? &a1 : &a0, k, ar, bar);
                    const CUtensorMap* m = second ? &b1 : &b0;
                    const int x = tc * 256 + 128 * (int)rank;
                    #pragma unroll
                    for (int i = 0; i < 4 / CG; ++i) tma_load<CG>(sb + i * 64 * BK * 2, m, x + 64 * i, k, bar);
                } else {
                    #pragma unroll
                    for (int i = 0; i < 2; ++i) tma_load<CG>(sa + i * 64 * BK * 2, ma, ar + 64 * i, kb * BK, bar);
                    const int x = tc * 256 + 128 * (int)rank;
                    #pragma unroll
                    for (int i = 0; i < 4 / CG; ++i) tma_load<CG>(sb + i * 64 * BK * 2, &b0, x + 64 * i, kb * BK, bar);
                }
            }
        }
        if (rank == 0) {
            // leave only when every issued load has landed (with a limit each)
            const int last = it < C::STAGES ? it : C::STAGES;
            for (int i = it - last; i < it; ++i) {
                const uint64_t t0 = timer_ns();
                while (!mbar_try(full0 + 8 * (i % C::STAGES), (i / C::STAGES) & 1) && timer_ns() - t0 < WAIT_LIMIT_NS) {}
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- products
        constexpr bool A_MN = MODE == DW, B_MN = MODE != FWD;
        constexpr uint32_t fmt = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
        constexpr uint32_t idesc = 1u << 4 | fmt << 7 | fmt << 10 | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) |
                                   (uint32_t)(ACC >> 3) << 17 | (uint32_t)(C::BM >> 4) << 24;
        // along K: 8-row groups 1024 bytes apart, 32 bytes per 16 elements of depth.  Along M or N: 64-element
        // boxes BK * 128 bytes apart, 8-deep groups 1024 bytes apart, 2048 bytes per 16 elements of depth.
        constexpr uint32_t box = 64 * BK * 2;
        int it = 0, n = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step, ++n) {
            const uint32_t acc = tmem + (n & 1) * ACC;
            if (!mbar_wait(tempty0 + 8 * (n & 1), ((n >> 1) & 1) ^ 1, abort)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (int kb = 0; kb < kbs; ++kb, ++it) {
                const int s = it % C::STAGES;
                if (!mbar_wait(full0 + 8 * s, (it / C::STAGES) & 1, abort)) { ok = false; break; }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sa = base + s * C::STAGE, sb = sa + 128 * BK * 2;
                const uint64_t da = A_MN ? smem_desc(sa, box, 1024) : smem_desc(sa, 16, 1024);
                const uint64_t db = B_MN ? smem_desc(sb, box, 1024) : smem_desc(sb, 16, 1024);
                #pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    mma_f16<CG>(acc, da + (uint64_t)(k * ((A_MN ? 2048 : 32) >> 4)), db + (uint64_t)(k * ((B_MN ? 2048 : 32) >> 4)),
                                idesc, kb > 0 || k > 0);
                mma_commit<CG>(empty0 + 8 * s);
            }
            if (ok) mma_commit<CG>(tfull0 + 8 * (n & 1));
        }
        if (*abort) {
            // issued products end before the tensor memory is freed
            mma_commit<CG>(drain);
            const uint64_t t0 = timer_ns();
            while (!mbar_try(drain, 0) && timer_ns() - t0 < WAIT_LIMIT_NS) {}
        }
    } else if (warp >= 4) {
        // ---- epilogue: warp w reads lanes 32 (w % 4) .. + 31 of the accumulator, a row per thread
        const int w = warp - 4;
        const uint32_t stg = smem_u32(stg_base) + w * 32 * STG_ROW;
        const unsigned char* stg_ptr = stg_base + w * 32 * STG_ROW;
        int n = 0;
        for (int t = first; t < tiles; t += step, ++n) {
            int tr, tc;
            tile_at(t, g.tiles_r, g.tiles_c, tr, tc);
            if (!mbar_wait(tfull0 + 8 * (n & 1), (n >> 1) & 1, abort)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (n & 1) * ACC + ((uint32_t)(32 * w) << 16);
            T* out = (T*)g.out0;
            int64_t ld = g.ld0;
            int rr = tr;
            if (MODE == DW && tr >= half_r) { out = (T*)g.out1; ld = g.ld1; rr -= half_r; }
            const int row0 = rr * C::BM + 128 * (int)rank + 32 * w;
            if constexpr (MODE == FWD) {
                #pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t vg[32], vu[32], h[16];
                    tmem_ld32(acc + c, vg);
                    tmem_ld32(acc + 128 + c, vu);
                    tmem_wait_ld();
                    const int col0 = tc * 128 + c;
                    if (col0 >= g.cols || row0 >= g.rows) continue;     // the whole warp
                    switch (g.act) {
                        case EXTERND_ACT_SILU: gate_chunk<T, EXTERND_ACT_SILU>(vg, vu, h); break;
                        case EXTERND_ACT_GELU: gate_chunk<T, EXTERND_ACT_GELU>(vg, vu, h); break;
                        case EXTERND_ACT_GELU_TANH: gate_chunk<T, EXTERND_ACT_GELU_TANH>(vg, vu, h); break;
                        default: gate_chunk<T, EXTERND_ACT_RELU2>(vg, vu, h); break;
                    }
                    store32<T>(h, stg, stg_ptr, out, ld, row0, g.rows, col0, g.cols, lane);
                    if (g.out1) {
                        pack_chunk<T>(vg, h);
                        store32<T>(h, stg, stg_ptr, (T*)g.out1, g.ld1, row0, g.rows, col0, g.cols, lane);
                        pack_chunk<T>(vu, h);
                        store32<T>(h, stg, stg_ptr, (T*)g.out2, g.ld1, row0, g.rows, col0, g.cols, lane);
                    }
                }
            } else {
                #pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t v[32], h[16];
                    tmem_ld32(acc + c, v);
                    tmem_wait_ld();
                    const int col0 = tc * 256 + c;
                    if (col0 >= g.cols || row0 >= g.rows) continue;
                    pack_chunk<T>(v, h);
                    store32<T>(h, stg, stg_ptr, out, ld, row0, g.rows, col0, g.cols, lane);
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                uint32_t bar = tempty0 + 8 * (n & 1);
                bar = map_rank(bar, 0);
                mbar_arrive_cluster(bar);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && abort_flag && g.status) atomicExch(g.status, EXTERND_ETIMEOUT);
    if constexpr (CG == 2) cluster_sync();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (CG == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}
