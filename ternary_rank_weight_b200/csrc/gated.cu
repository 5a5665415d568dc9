// The dense gated feed-forward block (sm_100a): H = act(G) * U with G = X Wg^T, U = X Wu^T, and its gradients
//     dG = dH U act'(G),  dU = dH act(G),  dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
// for bf16 and fp16, fp32 sums.
//
// Few tokens: the weights stream once through the warp-level products (dense_stream_kernel).  Otherwise one
// persistent kernel on the 5th-generation tensor cores (gemm_kernel): TMA brings 64-deep operand slabs into
// a ring of swizzled shared-memory stages, one thread issues tcgen05.mma into tensor memory, eight warps drain
// a finished accumulator while the next one fills.  It runs as
//   FWD  both projections of a tile in one accumulator, activation and product in the epilogue;
//   BWD  two lists of tiles: dX = dG Wg + dU Wu as one sum of 2 m terms (weights read along their columns, as
//        stored), then dG^T X and dU^T X (both operands read along their columns, as stored).
#include <cuda.h>

#include <type_traits>

#include "sm100.cuh"

namespace externd_ffn {

using namespace externd_llm;

// ---------------------------------------------------------------------------------------------------
// the tile kernel
// ---------------------------------------------------------------------------------------------------

enum Mode { FWD = 0, BWD = 1 };

constexpr int BK = 64;                     // depth of one stage: 128 bytes, one swizzle span
constexpr int EPI = 8;                     // epilogue warps: two for each quarter of the accumulator's rows
constexpr int THREADS = 128 + 32 * EPI;    // warp 0 TMA, warp 1 MMA, warps 4-11 epilogue
constexpr int ACC = 256;                   // accumulator columns; two accumulators fill tensor memory
constexpr int STG_ROW = 64;                // bytes of a staged row of outputs; its 16-byte pieces swizzled by the row: no bank conflicts

// CG = 2: a pair of CTAs works on one tile of 256 rows, each fetching its 128 rows of A and half of B, so that B
// crosses shared memory once for two SMs.  4096 tokens through 6912 x 2560: forward 183 us against 207 with CG = 1.
template <int CG> struct Cfg {
    static constexpr int BM = 128 * CG;                    // tile rows (128 per CTA)
    static constexpr int BBYTES = 256 / CG * BK * 2;       // a CTA's share of at most 256 B rows
    static constexpr int STAGE = 128 * BK * 2 + BBYTES;
    static constexpr int STAGES = CG == 1 ? 4 : 6;
    static constexpr int SMEM = STAGES * STAGE + EPI * 32 * STG_ROW + 1024 + 256;
};

// one list of output tiles
struct TileList {
    int tiles_r, tiles_c;    // tile grid
    int rows, cols;          // outputs
    int blocks;              // stages of depth BK of a tile
    int splits;              // shares of the depth, each a tile of its own
};

struct GemmArgs {
    TileList main;           // FWD: H (tokens x m); BWD: dX (tokens x n), possibly no tiles
    TileList grad;           // BWD: dWg, dWu (m x n each; tiles_r counts both), possibly no tiles
    int half_r;              // row tiles of one of the two
    int width;               // accumulator columns of a tile: FWD twice the output columns; BWD the output columns
    int skip;                // BWD: rounds of grad that workers with one main tile more sit out
    int act;
    void* h; int64_t ldh;    // FWD H, BWD dX
    void* s[2]; int64_t lds; // FWD G and U (or null), BWD dWg and dWu
    int save32;              // FWD: G and U in fp32 (otherwise in the operands' type)
    float* part;             // BWD, main.splits > 1: the shares' sums (splits x tokens x ldp) instead of dX
    int64_t ldp;
    int* status;             // may be null
    WaitFault fault;
};

struct Tile { bool grad; int r, c, split, first, last; };    // stages first .. last - 1

// tile t of a list: bands of 8 row tiles walked column by column, so the tiles in flight share operands in L2
__device__ __forceinline__ void tile_at(int t, const TileList& l, Tile& o) {
    o.split = t % l.splits;
    t /= l.splits;
    o.first = (int)((int64_t)l.blocks * o.split / l.splits);
    o.last = (int)((int64_t)l.blocks * (o.split + 1) / l.splits);
    const int band = t / (8 * l.tiles_c), first = band * 8;
    const int h = min(8, l.tiles_r - first), in = t - band * 8 * l.tiles_c;
    o.c = in / h;
    o.r = first + in - o.c * h;
}

// The i-th tile of a worker (a CTA or a pair): the main list in turn, then the grad list in rounds, of which the
// workers that got one main tile more (the first `more`) sit out the first `skip`: dX tiles are longer than dW
// tiles, and so all end at about the same time.
__device__ __forceinline__ bool tile_of(const GemmArgs& g, int worker, int workers, int i, Tile& o) {
    const int nm = g.main.tiles_r * g.main.tiles_c * g.main.splits, ng = g.grad.tiles_r * g.grad.tiles_c;
    const int mine = nm > worker ? (nm - worker + workers - 1) / workers : 0;
    if (i < mine) {
        o.grad = false;
        tile_at(worker + i * workers, g.main, o);
        return true;
    }
    const int more = nm % workers, few = workers - more;
    const int64_t round = (int64_t)i - mine + (worker < more ? g.skip : 0);
    const int64_t t = round < g.skip ? round * few + worker - more : (int64_t)g.skip * few + (round - g.skip) * workers + worker;
    if (t >= ng) return false;
    o.grad = true;
    tile_at((int)t, g.grad, o);
    return true;
}

// piece i of a staged row r sits at piece i ^ (r / 2 % 4)
__device__ __forceinline__ int staged(int r, int i) { return r * STG_ROW + ((i ^ (r >> 1 & 3)) << 4); }

// the warp's staged rows to global memory, as units of U: neighbouring lanes write neighbouring units
template <typename U, typename T>
__device__ __forceinline__ void store_units(const unsigned char* stg_ptr, T* out, int64_t ld, int rows, int cols, int lane) {
    constexpr int LANES = 64 / sizeof(U), STEP = 32 / LANES;       // lanes of a row, rows at a time
    const int r0 = lane / LANES, byte = lane % LANES * (int)sizeof(U);
    const int last = byte < cols * (int)sizeof(T) ? rows : 0;      // units lie inside the columns: all of them, or units of one
    unsigned char* o = reinterpret_cast<unsigned char*>(out + r0 * ld) + byte;
    #pragma unroll 8
    for (int r = r0; r < 32; r += STEP, o += STEP * ld * sizeof(T))
        if (r < last) *reinterpret_cast<U*>(o) = *reinterpret_cast<const U*>(stg_ptr + staged(r, byte >> 4) + (byte & 15));
}

// 64 bytes of each of a warp's 32 rows (a row per lane, 16 registers) to global memory through the warp's staging
// buffer, in the widest units that the rows' starts allow
template <typename T>
__device__ __forceinline__ void store64(const uint32_t* v, uint32_t stg, const unsigned char* stg_ptr, T* out, int64_t ld, int row0, int rows,
                                        int col0, int cols, int lane) {
    #pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(stg + staged(lane, i)), "r"(v[4 * i]), "r"(v[4 * i + 1]), "r"(v[4 * i + 2]),
                     "r"(v[4 * i + 3]) : "memory");
    __syncwarp();
    T* const o = out + (int64_t)row0 * ld + col0;
    const int nr = min(32, rows - row0), nc = min((int)(64 / sizeof(T)), cols - col0);
    const uint32_t starts = (uint32_t)(reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ld * sizeof(T)));
    if (nc < (int)(64 / sizeof(T))) store_units<T>(stg_ptr, o, ld, nr, nc, lane);
    else if ((starts & 15) == 0) store_units<uint4>(stg_ptr, o, ld, nr, nc, lane);
    else if ((starts & 7) == 0) store_units<uint2>(stg_ptr, o, ld, nr, nc, lane);
    else if ((starts & 3) == 0) store_units<uint32_t>(stg_ptr, o, ld, nr, nc, lane);
    else store_units<T>(stg_ptr, o, ld, nr, nc, lane);
    __syncwarp();
}

// NaN in a warp's share of a tile: 32 rows, every other 32 of the columns col0 + turn .. end - 1
template <typename T>
__device__ __noinline__ void store_nan(uint32_t stg, const unsigned char* stg_ptr, T* out, int64_t ld, int row0, int rows, int col0, int turn,
                                       int end, int cols, int lane) {
    uint32_t v[16];
    for (int i = 0; i < 16; ++i) v[i] = 0x7fff7fffu;                    // NaN in fp32, fp16 and bf16
    if (row0 >= rows) return;
    for (int c = turn; c < end; c += 64)
        for (int e = c; e < c + 32; e += 64 / (int)sizeof(T))
            if (col0 + e < cols) store64<T>(v, stg, stg_ptr, out, ld, row0, rows, col0 + e, cols, lane);
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

struct Maps { CUtensorMap a[2], b[2], d[2], x; };    // FWD X, Wg, Wu; BWD dG, dU by rows, Wg, Wu, dG, dU by columns, X

template <typename T, int MODE, int CG>
__global__ void __launch_bounds__(THREADS, 1) gemm_kernel(const __grid_constant__ Maps maps, const GemmArgs g) {
    using C = Cfg<CG>;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[2 * C::STAGES + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int quit_flag;
    __shared__ uint32_t issued[2];                                  // stages that each CTA of the pair sent loads for
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;          // swizzle atoms are 1024-byte aligned
    unsigned char* const stg_base = raw + (base - smem_u32(raw)) + C::STAGES * C::STAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0 : cluster_rank();
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES, tfull0 = empty0 + 8 * C::STAGES, tempty0 = tfull0 + 16,
                   drain = tempty0 + 16;
    volatile int* const quit = &quit_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, EPI * CG);                      // one arrival per epilogue warp of the pair
        }
        mbar_init(drain, 1);
        quit_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(&tmem_slot), 512);
    }
    fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    fence_after();
    const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;

    const int worker = blockIdx.x / CG, workers = gridDim.x / CG;
    const uint32_t b_bytes = (uint32_t)(g.width / CG) * (BK * 2);     // a CTA's share of a stage's B

    // wait until the loads of stage i have landed
    const auto land = [&](int i) {
        const uint64_t t0 = timer_ns();
        while (!mbar_try(full0 + 8 * (i % C::STAGES), (i / C::STAGES) & 1) && timer_ns() - t0 < WAIT_LIMIT_NS) {}
    };
    if (warp == 0 && lane == 0) {
        // ---- loads: each CTA fetches its 128 rows of A and its share of B; both complete on the leader's barrier
        int it = 0;
        bool ok = true;
        Tile t;
        for (int i = 0; ok && tile_of(g, worker, workers, i, t); ++i) {
            for (int kb = t.first; kb < t.last; ++kb, ++it) {
                const int s = it % C::STAGES;
                if (!mbar_wait(empty0 + 8 * s, ((it / C::STAGES) & 1) ^ 1, quit, g.fault.limit_ns)) { ok = false; break; }
                const uint32_t sa = base + s * C::STAGE, sb = sa + 128 * BK * 2;
                uint32_t bar = full0 + 8 * s;
                if (rank == 0) mbar_expect(bar, CG * (128 * BK * 2 + b_bytes));
                if constexpr (CG == 2) bar = map_rank(bar, 0);
                if constexpr (MODE == FWD) {
                    const int x = kb * BK, y = t.c * (g.width / 2);
                    tma_load<CG>(sa, &maps.a[0], x, t.r * C::BM + 128 * (int)rank, bar);
                    if constexpr (CG == 1) {                             // Wg's rows, then Wu's
                        tma_load<CG>(sb, &maps.b[0], x, y, bar);
                        tma_load<CG>(sb + b_bytes / 2, &maps.b[1], x, y, bar);
                    } else {                                             // Wg's rows in CTA 0, Wu's in CTA 1
                        tma_load<CG>(sb, &maps.b[rank], x, y, bar);
                    }
                } else {
                    const int x = t.c * g.width + (int)(g.width / CG * rank);
                    if (!t.grad) {
                        const int half = g.main.blocks / 2, which = kb >= half, k = (which ? kb - half : kb) * BK;
                        tma_load<CG>(sa, &maps.a[which], k, t.r * C::BM + 128 * (int)rank, bar);
                        for (int i = 0; i < g.width / CG; i += 64) tma_load<CG>(sb + i * (BK * 2), &maps.b[which], x + i, k, bar);
                    } else {
                        const int which = t.r >= g.half_r, row = (t.r - (which ? g.half_r : 0)) * C::BM + 128 * (int)rank, k = kb * BK;
                        tma_load<CG>(sa, &maps.d[which], row, k, bar);
                        tma_load<CG>(sa + 64 * BK * 2, &maps.d[which], row + 64, k, bar);
                        for (int i = 0; i < g.width / CG; i += 64) tma_load<CG>(sb + i * (BK * 2), &maps.x, x + i, k, bar);
                    }
                }
            }
        }
        if (rank == 0) {
            // leave only when every issued load has landed (with a limit each)
            for (int i = max(0, it - C::STAGES); i < it; ++i) land(i);
        }
        if constexpr (CG == 2) {
            issued[rank] = it;
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(smem_u32(&issued[rank]), rank ^ 1)), "r"(it) : "memory");
        }
    } else if (warp == 1 && rank == 0) {
        // ---- products.  (Nothing in the loop needs the whole warp: where a wait runs out, lanes may leave it one by one)
        const bool leader = elect_one();
        constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
        // along K: 8-row groups 1024 bytes apart, 32 bytes per 16 elements of depth.  Along M or N: 64-element
        // boxes BK * 128 bytes apart, 8-deep groups 1024 bytes apart, 2048 bytes per 16 elements of depth.
        constexpr uint32_t box = 64 * BK * 2;
        int s = 0, phase = 0, n = 0;
        bool ok = worker + 1 != g.fault.withhold;
        Tile t;
        for (; ok && tile_of(g, worker, workers, n, t); ++n) {
            const bool a_mn = MODE == BWD && t.grad, b_mn = MODE == BWD;
            const uint32_t idesc = f16_idesc(fmt, a_mn, b_mn, C::BM, g.width);
            const uint32_t a_lbo = a_mn ? box : 16, b_lbo = b_mn ? box : 16, a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
            const int kbs = t.last - t.first;
            const uint32_t acc = tmem + (n & 1) * ACC;
            if (!mbar_wait(tempty0 + 8 * (n & 1), ((n >> 1) & 1) ^ 1, quit, g.fault.limit_ns)) break;
            fence_after();
            for (int kb = 0; kb < kbs; ++kb) {
                if (!mbar_wait(full0 + 8 * s, phase, quit, g.fault.limit_ns)) { ok = false; break; }
                fence_after();
                const uint32_t sa = base + s * C::STAGE, sb = sa + 128 * BK * 2;
                const uint64_t da = smem_desc(sa, a_lbo, 1024), db = smem_desc(sb, b_lbo, 1024);
                if (leader) {
                    #pragma unroll
                    for (int k = 0; k < BK / 16; ++k) mma_f16<CG>(acc, da + k * a_step, db + k * b_step, idesc, kb > 0 || k > 0);
                    mma_commit<CG>(empty0 + 8 * s);
                    if (kb == kbs - 1) mma_commit<CG>(tfull0 + 8 * (n & 1));
                }
                if (++s == C::STAGES) { s = 0; phase ^= 1; }
            }
        }
        if (leader) {
            // issued products end before the tensor memory is freed
            mma_commit<CG>(drain, 1);
            const uint64_t t0 = timer_ns();
            while (!mbar_try(drain, 0) && timer_ns() - t0 < WAIT_LIMIT_NS) {}
        }
        __syncwarp();                                          // lanes that left the loop apart
    } else if (warp >= 4) {
        // ---- epilogue: warp w reads lanes 32 (w % 4) .. + 31 of the accumulator, a row per thread, and every other
        // 32 columns
        const int w = warp & 3, turn = 32 * ((warp >> 2) - 1);
        const uint32_t stg = smem_u32(stg_base) + (warp - 4) * 32 * STG_ROW;
        const unsigned char* stg_ptr = stg_base + (warp - 4) * 32 * STG_ROW;
        Tile t;
        int n = 0;
        bool late = false;
        for (; tile_of(g, worker, workers, n, t); ++n) {
            if (!mbar_wait_warp(tfull0 + 8 * (n & 1), (n >> 1) & 1, quit, g.fault.limit_ns)) { late = true; break; }
            fence_after();
            const uint32_t acc = tmem + (n & 1) * ACC + ((uint32_t)(32 * w) << 16);
            if constexpr (MODE == FWD) {
                const int row0 = t.r * C::BM + 128 * (int)rank + 32 * w, half = g.width / 2;
                #pragma unroll 1
                for (int c = turn; c < half; c += 64) {
                    const int col0 = t.c * half + c;
                    if (col0 >= g.main.cols || row0 >= g.main.rows) break;     // the whole warp
                    uint32_t vg[32], vu[32], h[16];
                    tmem_ld32(acc + c, vg);
                    tmem_ld32(acc + half + c, vu);
                    tmem_wait_ld();
                    switch (g.act) {
                        case EXTERND_ACT_SILU: gate_chunk<T, EXTERND_ACT_SILU>(vg, vu, h); break;
                        case EXTERND_ACT_GELU: gate_chunk<T, EXTERND_ACT_GELU>(vg, vu, h); break;
                        case EXTERND_ACT_GELU_TANH: gate_chunk<T, EXTERND_ACT_GELU_TANH>(vg, vu, h); break;
                        default: gate_chunk<T, EXTERND_ACT_RELU2>(vg, vu, h); break;
                    }
                    store64<T>(h, stg, stg_ptr, (T*)g.h, g.ldh, row0, g.main.rows, col0, g.main.cols, lane);
                    if (g.s[0] && g.save32) {
                        #pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            if (col0 + e >= g.main.cols) break;
                            store64<float>(vg + e, stg, stg_ptr, (float*)g.s[0], g.lds, row0, g.main.rows, col0 + e, g.main.cols, lane);
                            store64<float>(vu + e, stg, stg_ptr, (float*)g.s[1], g.lds, row0, g.main.rows, col0 + e, g.main.cols, lane);
                        }
                    } else if (g.s[0]) {
                        pack_chunk<T>(vg, h);
                        store64<T>(h, stg, stg_ptr, (T*)g.s[0], g.lds, row0, g.main.rows, col0, g.main.cols, lane);
                        pack_chunk<T>(vu, h);
                        store64<T>(h, stg, stg_ptr, (T*)g.s[1], g.lds, row0, g.main.rows, col0, g.main.cols, lane);
                    }
                }
            } else {
                const TileList& l = t.grad ? g.grad : g.main;
                const int which = t.grad && t.r >= g.half_r;
                T* const out = (T*)(t.grad ? g.s[which] : g.h);
                const int64_t ld = t.grad ? g.lds : g.ldh;
                const int row0 = (t.r - (which ? g.half_r : 0)) * C::BM + 128 * (int)rank + 32 * w;
                #pragma unroll 1
                for (int c = turn; c < g.width; c += 64) {
                    const int col0 = t.c * g.width + c;
                    if (col0 >= l.cols || row0 >= l.rows) break;
                    uint32_t v[32], h[16];
                    tmem_ld32(acc + c, v);
                    tmem_wait_ld();
                    if (!t.grad && g.part) {
                        #pragma unroll
                        for (int e = 0; e < 32; e += 16)
                            if (col0 + e < l.cols)
                                store64<float>(v + e, stg, stg_ptr, g.part + (int64_t)t.split * l.rows * g.ldp, g.ldp, row0, l.rows, col0 + e, l.cols, lane);
                        continue;
                    }
                    pack_chunk<T>(v, h);
                    store64<T>(h, stg, stg_ptr, out, ld, row0, l.rows, col0, l.cols, lane);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                uint32_t bar = tempty0 + 8 * (n & 1);
                bar = map_rank(bar, 0);
                mbar_arrive_cluster(bar);
            }
        }
        // a wait gave up: NaN instead of what the outputs' memory held, whether or not the caller looks at a status
        for (; late && tile_of(g, worker, workers, n, t); ++n) {
            const int which = MODE == BWD && t.grad && t.r >= g.half_r;
            const int row0 = (t.r - (which ? g.half_r : 0)) * C::BM + 128 * (int)rank + 32 * w;
            const TileList& l = MODE == BWD && t.grad ? g.grad : g.main;
            const int wide = MODE == FWD ? g.width / 2 : g.width, col0 = t.c * wide;
            if (MODE == BWD && !t.grad && g.part) {
                store_nan<float>(stg, stg_ptr, g.part + (int64_t)t.split * l.rows * g.ldp, g.ldp, row0, l.rows, col0, turn, wide, l.cols, lane);
            } else if (MODE == BWD && t.grad) {
                store_nan<T>(stg, stg_ptr, (T*)g.s[which], g.lds, row0, l.rows, col0, turn, wide, l.cols, lane);
            } else {
                store_nan<T>(stg, stg_ptr, (T*)g.h, g.ldh, row0, l.rows, col0, turn, wide, l.cols, lane);
                for (int i = 0; MODE == FWD && g.s[0] && i < 2; ++i) {
                    if (g.save32) store_nan<float>(stg, stg_ptr, (float*)g.s[i], g.lds, row0, l.rows, col0, turn, wide, l.cols, lane);
                    else store_nan<T>(stg, stg_ptr, (T*)g.s[i], g.lds, row0, l.rows, col0, turn, wide, l.cols, lane);
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && quit_flag && g.status) atomicExch(g.status, EXTERND_ETIMEOUT);
    if constexpr (CG == 2) {
        cluster_sync();
        if (issued[0] != issued[1]) {
            // The CTAs gave up at different stages.  Loads complete on CTA 0's barriers, which do not yet expect what CTA 1
            // alone sent: its own 128 rows of A and share of B
            if (rank == 0 && threadIdx.x == 0)
                for (int i = (int)issued[0]; i < (int)issued[1]; ++i) {
                    mbar_expect(full0 + 8 * (i % C::STAGES), 128 * BK * 2 + b_bytes);
                    land(i);
                }
            cluster_sync();
        }
    }
    if (warp == 1) {
        __syncwarp();
        fence_after();
        tmem_free<CG>(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------------------
// dG and dU from the saved projections
// ---------------------------------------------------------------------------------------------------

// Bound by memory: reads dH, G, U and writes dG, dU; 4096 tokens x 6912 with G, U in fp32: 396 MB in 54 us, 7.4 TB/s
// (gelu: bound by erfc, 80 us).  dG and dU are rounded to the operands' type, which the
// tensor cores need.  Against a step that keeps everything in 32 bits this rounding makes the gradients' error
// 1.4 times theirs (the output's rounding alone); G and U saved in 16 bits make it 1.8 times, with
// relu2, which doubles their relative error, 2.5 times.
template <typename T> __device__ __forceinline__ float2 pair_of(const uint4& v, int e) {
    return unpack2<T>(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
}
template <typename T> __device__ __forceinline__ float2 pair_of(const F8& v, int e) {
    return e == 0 ? make_float2(v.a.x, v.a.y) : e == 1 ? make_float2(v.a.z, v.a.w) : e == 2 ? make_float2(v.b.x, v.b.y) : make_float2(v.b.z, v.b.w);
}

// A projection that was saved as infinite (fp16: past 65504) counts as the type's largest value: act and act' are at their
// limits there (silu, gelu, gelu_tanh: 0 or g, and 0 or 1), where infinity itself would meet them as 0 * inf.  NaN stays.
template <typename S> struct Largest { static constexpr float value = FLT_MAX; };
template <> struct Largest<__half> { static constexpr float value = 65504.0f; };
template <> struct Largest<__nv_bfloat16> { static constexpr float value = 3.38953139e38f; };
template <typename S> __device__ __forceinline__ float finite(float v) { return fabsf(v) > Largest<S>::value ? copysignf(Largest<S>::value, v) : v; }

// 8 columns a thread; hvec, svec: dH's rows, G's and U's, start on 16-byte boundaries.  S: float, or the operands' 16 bits.
template <typename T, typename S, int ACT>
__global__ void __launch_bounds__(256) gate_grad_kernel(const T* __restrict__ dh, int64_t lddh, int hvec, const S* __restrict__ gs,
                                                        const S* __restrict__ us, int64_t ldgu, int svec, int64_t rows, int64_t m,
                                                        T* __restrict__ dg, T* __restrict__ du, int64_t ldw, const AlignJobs jobs) {
    if (blockIdx.y > 0) {                                  // copies of operands with misaligned rows ride along
        align_rows(jobs.j[blockIdx.y - 1], blockIdx.x, gridDim.x);
        return;
    }
    const int64_t per = ldw / 8;                           // ldw: m rounded up to 8
    using Saved = typename std::conditional<std::is_same<S, float>::value, float, T>::type;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, k = 8 * (i - r * per);
        const uint4 h8 = load8(reinterpret_cast<const unsigned short*>(dh + r * lddh), k, m, hvec);
        const auto g8 = load8(gs + r * ldgu, k, m, svec), u8 = load8(us + r * ldgu, k, m, svec);
        uint32_t og[4], ou[4];
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 h = pair_of<T>(h8, e), g = pair_of<T>(g8, e), u = pair_of<T>(u8, e);
            const float2 a = act_both<ACT, false>(finite<Saved>(g.x)), b = act_both<ACT, false>(finite<Saved>(g.y));
            // dH act' first: a derivative of 0 makes 0 of any U, where dH U may be past the fp32 range
            og[e] = pack2<T>(h.x * a.y * finite<Saved>(u.x), h.y * b.y * finite<Saved>(u.y));
            ou[e] = pack2<T>(h.x * a.x, h.y * b.x);
        }
        *reinterpret_cast<uint4*>(dg + r * ldw + k) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(du + r * ldw + k) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    }
}

// dX from the shares' sums, in their order
template <typename T>
__global__ void __launch_bounds__(256) add_shares_kernel(const float* __restrict__ part, int64_t ldp, int splits, int64_t rows, int64_t cols,
                                                         T* __restrict__ out, int64_t ld) {
    const int64_t per = ldp / 4;                             // ldp: cols rounded up to 8
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = 4 * (i - r * per);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < splits; ++s) {
            const float4 p = __ldg(reinterpret_cast<const float4*>(part + (s * rows + r) * ldp + c));
            v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
        }
        const float e[4] = {v.x, v.y, v.z, v.w};
        #pragma unroll
        for (int t = 0; t < 4; ++t)
            if (c + t < cols) out[r * ld + c + t] = from_f32<T>(e[t]);
    }
}

// ---------------------------------------------------------------------------------------------------
// few tokens: stream the weights once
// ---------------------------------------------------------------------------------------------------

// A CTA takes 16 rows of both matrices and 8 NT tokens; its warps split the columns and meet in shared memory
// in a fixed order.  Bound by the weights' bytes: one token, 6912 x 2560 bf16, 14 us, 5.1 TB/s.  A tile of the
// tile kernel would leave most of its 128 token rows empty, and half of the SMs without a tile.
template <typename T, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) dense_stream_kernel(const T* __restrict__ wg, int64_t ldg, const T* __restrict__ wu,
                                                                 int64_t ldu, int64_t m, int64_t n, int act,
                                                                 const T* __restrict__ x, int64_t ldx, int64_t tokens,
                                                                 T* __restrict__ hout, int64_t ldh, void* __restrict__ gout,
                                                                 void* __restrict__ uout, int64_t ldgu, int save32) {
    constexpr int COLS = 8 * NT;
    __shared__ float part[2][WARPS][16][COLS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int64_t ra = min(row0 + r, m - 1), rb = min(row0 + r + 8, m - 1);
    using S16 = unsigned short;
    const S16* rows[4] = {(const S16*)(wg + ra * ldg), (const S16*)(wg + rb * ldg), (const S16*)(wu + ra * ldu), (const S16*)(wu + rb * ldu)};
    const S16* xr[NT];
    #pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = 8 * t + r < tokens ? (const S16*)(x + (8 * t + r) * ldx) : nullptr;
    float acc[2][NT][4] = {};
    const int64_t blocks = (n + 63) / 64;
    for (int64_t blk = warp; blk < blocks; blk += WARPS) {
        uint4 w[2][4], xf[2][NT];
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t k = blk * 64 + 32 * i + 8 * c;
            #pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = load8(rows[j], k, n, true);
            #pragma unroll
            for (int t = 0; t < NT; ++t) xf[i][t] = xr[t] ? load8(xr[t], k, n, true) : make_uint4(0, 0, 0, 0);
        }
        #pragma unroll
        for (int i = 0; i < 2; ++i)
            #pragma unroll
            for (int j = 0; j < 2; ++j)
                #pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 a = w[i][2 * j], b = w[i][2 * j + 1], v = xf[i][t];
                    mma16816<T>(acc[j][t], a.x, b.x, a.y, b.y, v.x, v.y);
                    mma16816<T>(acc[j][t], a.z, b.z, a.w, b.w, v.z, v.w);
                }
    }
    #pragma unroll
    for (int j = 0; j < 2; ++j)
        #pragma unroll
        for (int t = 0; t < NT; ++t) {
            part[j][warp][r][8 * t + 2 * c] = acc[j][t][0];
            part[j][warp][r][8 * t + 2 * c + 1] = acc[j][t][1];
            part[j][warp][r + 8][8 * t + 2 * c] = acc[j][t][2];
            part[j][warp][r + 8][8 * t + 2 * c + 1] = acc[j][t][3];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * COLS; e += WARPS * 32) {
        const int rr = e & 15, cc = e >> 4;
        if (row0 + rr >= m || cc >= tokens) continue;
        float g = 0.0f, u = 0.0f;
        #pragma unroll
        for (int p = 0; p < WARPS; ++p) {
            g += part[0][p][rr][cc];
            u += part[1][p][rr][cc];
        }
        hout[cc * ldh + row0 + rr] = from_f32<T>(act_rt<false>(act, g) * u);
        const int64_t at = cc * ldgu + row0 + rr;
        if (gout && save32) {
            ((float*)gout)[at] = g;
            ((float*)uout)[at] = u;
        } else if (gout) {
            ((T*)gout)[at] = from_f32<T>(g);
            ((T*)uout)[at] = from_f32<T>(u);
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------------

constexpr int64_t STREAM_TOKENS = 16;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return (EncodeFn)p;
    }();
    return fn;
}

// rows x cols matrix, boxes of 64 columns (128 bytes) x box_rows; reads past the edges give 0
bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows, int dtype) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return fn(map, dtype == EXTERND_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p),
              dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int MODE, int CG>
cudaError_t launch_gemm(const Maps& maps, const GemmArgs& g, cudaStream_t s) {
    static PerDevice done;
    const cudaError_t e = allow_smem(gemm_kernel<T, MODE, CG>, Cfg<CG>::SMEM, done);
    if (e != cudaSuccess) return e;
    const int tiles = g.main.tiles_r * g.main.tiles_c * g.main.splits + g.grad.tiles_r * g.grad.tiles_c, slots = sm_count() / CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < slots ? tiles : slots) * CG));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Cfg<CG>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CG > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, gemm_kernel<T, MODE, CG>, maps, g);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// one call's arguments, with the operands' final places
struct Call {
    const void* X; int64_t ldx;
    const void* W[2]; int64_t ldw[2];
    int dtype;
    int64_t m, n, tokens;
    int act;
    void* H; int64_t ldh;
    void* S[2]; int save_dtype; int64_t lds;          // G and U
    const void* dH; int64_t lddh;
    void* dX; int64_t lddx;
    void* dW[2]; int64_t lddw;
    unsigned char* work; size_t work_bytes;
    int* status;
    cudaStream_t stream;
};

// Give the operands that need it a place in `work` (consumed from its start).  false: it is too small.
bool place_operands(Call& c, bool x, bool w, AlignJobs& jobs) {
    if (x && !place_rows(jobs, c.X, c.ldx, c.tokens, c.n, 2, c.work, c.work_bytes)) return false;
    if (w)
        for (int i = 0; i < 2; ++i)
            if (!place_rows(jobs, c.W[i], c.ldw[i], c.m, c.n, 2, c.work, c.work_bytes)) return false;
    return true;
}

template <typename T, int CG>
int forward_tiles(const Call& c, int width) {
    Maps maps = {};
    if (!make_map(&maps.a[0], c.X, c.tokens, c.n, c.ldx, 128, c.dtype) || !make_map(&maps.b[0], c.W[0], c.m, c.n, c.ldw[0], width / 2, c.dtype) ||
        !make_map(&maps.b[1], c.W[1], c.m, c.n, c.ldw[1], width / 2, c.dtype))
        return EXTERND_ECUDA;
    GemmArgs g = {};
    g.main = {ceil_div(c.tokens, Cfg<CG>::BM), ceil_div(c.m, width / 2), (int)c.tokens, (int)c.m, ceil_div(c.n, BK), 1};
    g.grad.splits = 1;
    g.width = width;
    g.act = c.act;
    g.fault = wait_fault();
    g.h = c.H; g.ldh = c.ldh; g.s[0] = c.S[0]; g.s[1] = c.S[1]; g.lds = c.lds; g.save32 = c.save_dtype == EXTERND_F32;
    g.status = c.status;
    return launch_gemm<T, FWD, CG>(maps, g, c.stream) == cudaSuccess ? EXTERND_OK : EXTERND_ECUDA;
}

// Pairs of CTAs or single ones, and how wide the tiles: the fewest weighted rounds.  Narrow tiles save little of a round:
// shared memory writes and reads of both operands bound it, and a narrower tile still moves all of A.  4096 tokens x 6912 x
// 2560, us a round: pairs 15.3 / 12.3 / 10.5 at 256 / 192 / 128 columns, single CTAs 17.3 / 14.9 / 13.0.  The weights are not
// those ratios (1, 0.80, 0.69; 1.13, 0.97, 0.85): calls of one or two rounds, where the choice matters most, have their
// start and end besides.  Over 120 shapes (32 to 2048 tokens, 2048 to 11008 rows, depths 768 and 2560) the plan they
// pick takes 2.0 % longer than the best of the six on average (at worst 22 %, at depth 768); the bare ratios' 2.8 % (32 %).
template <typename T>
int forward_tiles(const Call& c) {
    constexpr double ROUND[2][3] = {{1.22, 1.03, 0.91}, {1.00, 0.93, 0.85}};
    int best_cg = 1, best_width = 256;
    double best = 1e300;
    for (int cg = 1; cg <= 2; ++cg)
        for (int i = 0; i < 3; ++i) {
            const int width = 256 - 64 * i;
            const double cost = ceil_div((int64_t)ceil_div(c.tokens, 128 * cg) * ceil_div(c.m, width / 2), sm_count() / cg) * ROUND[cg - 1][i];
            if (cost < best) { best = cost; best_cg = cg; best_width = width; }
        }
    return best_cg == 1 ? forward_tiles<T, 1>(c, best_width) : forward_tiles<T, 2>(c, best_width);
}

template <typename T, int NT>
int forward_stream(const Call& c) {
    dense_stream_kernel<T, NT, 8><<<(unsigned)((c.m + 15) / 16), 256, 0, c.stream>>>(
        (const T*)c.W[0], c.ldw[0], (const T*)c.W[1], c.ldw[1], c.m, c.n, c.act, (const T*)c.X, c.ldx, c.tokens, (T*)c.H, c.ldh, c.S[0],
        c.S[1], c.lds, c.save_dtype == EXTERND_F32);
    return cudaGetLastError() == cudaSuccess ? EXTERND_OK : EXTERND_ECUDA;
}

template <typename T>
int forward(const Call& c) {
    if (c.tokens <= 8) return forward_stream<T, 1>(c);
    if (c.tokens <= STREAM_TOKENS) return forward_stream<T, 2>(c);
    return forward_tiles<T>(c);
}

template <typename T, typename S, int ACT>
void launch_gate_grad(const Call& c, T* dg, T* du, int64_t ldd, const AlignJobs& jobs) {
    const int64_t items = c.tokens * (ldd / 8), cap = (int64_t)sm_count() * 32;
    int64_t want = (items + 255) / 256;
    for (int i = 0; i < jobs.count; ++i) {
        const int64_t n = (jobs.j[i].rows * ((jobs.j[i].cols + 255) / 256) + 7) / 8;
        want = want > n ? want : n;
    }
    const dim3 grid((unsigned)(want < cap ? want : cap), 1 + jobs.count);
    gate_grad_kernel<T, S, ACT><<<grid, 256, 0, c.stream>>>(
        (const T*)c.dH, c.lddh, row_aligned(c.dH, c.tokens, c.lddh, 2), (const S*)c.S[0], (const S*)c.S[1], c.lds,
        row_aligned(c.S[0], c.tokens, c.lds, sizeof(S)) && row_aligned(c.S[1], c.tokens, c.lds, sizeof(S)), c.tokens, c.m, dg, du, ldd, jobs);
}

template <typename T, typename S>
cudaError_t gate_grad(const Call& c, T* dg, T* du, int64_t ldd, const AlignJobs& jobs) {
    switch (c.act) {
        case EXTERND_ACT_SILU: launch_gate_grad<T, S, EXTERND_ACT_SILU>(c, dg, du, ldd, jobs); break;
        case EXTERND_ACT_GELU: launch_gate_grad<T, S, EXTERND_ACT_GELU>(c, dg, du, ldd, jobs); break;
        case EXTERND_ACT_GELU_TANH: launch_gate_grad<T, S, EXTERND_ACT_GELU_TANH>(c, dg, du, ldd, jobs); break;
        default: launch_gate_grad<T, S, EXTERND_ACT_RELU2>(c, dg, du, ldd, jobs); break;
    }
    return cudaGetLastError();
}

// Shares of the depth of dX's 2 m terms: with few tokens its tiles are few and long, and a tile is left to as many
// workers as there are for each (the backward pass of 64 tokens x 6912 x 2560 took 88 us without).  Below 64 stages (24 us)
// the launch that adds the shares up would take back what they save.  For the widest tiles; narrower ones have no
// fewer workers each.
constexpr int MAX_SPLITS = 16;
int dx_splits(int64_t m, int64_t n, int64_t tokens) {
    const int64_t tiles = (int64_t)ceil_div(tokens, 128) * ceil_div(n, 256), stages = 2 * (int64_t)ceil_div(m, BK);
    if (stages < 64) return 1;
    int64_t s = sm_count() / tiles;
    s = s < MAX_SPLITS ? s : MAX_SPLITS;
    s = s < stages / 8 ? s : stages / 8;
    return s < 1 ? 1 : (int)s;
}
size_t share_bytes(int64_t m, int64_t n, int64_t tokens) {
    const int s = dx_splits(m, n, tokens);
    return s == 1 ? 0 : ((size_t)s * (size_t)tokens * (size_t)round8(n) * 4 + 255) / 256 * 256;
}

template <typename T, int CG>
int backward_tiles(const Call& c, const T* dg, const T* du, int64_t ldd, float* part, int splits, int width) {
    constexpr int BM = Cfg<CG>::BM;
    GemmArgs g = {};
    Maps maps = {};
    g.width = width;
    g.status = c.status;
    g.fault = wait_fault();
    g.main.splits = g.grad.splits = 1;
    if (c.dX) {
        if (!make_map(&maps.a[0], dg, c.tokens, c.m, ldd, 128, c.dtype) || !make_map(&maps.a[1], du, c.tokens, c.m, ldd, 128, c.dtype) ||
            !make_map(&maps.b[0], c.W[0], c.m, c.n, c.ldw[0], BK, c.dtype) || !make_map(&maps.b[1], c.W[1], c.m, c.n, c.ldw[1], BK, c.dtype))
            return EXTERND_ECUDA;
        g.main = {ceil_div(c.tokens, BM), ceil_div(c.n, width), (int)c.tokens, (int)c.n, 2 * ceil_div(c.m, BK), splits};
        g.h = c.dX; g.ldh = c.lddx;
        if (splits > 1) { g.part = part; g.ldp = round8(c.n); }
    }
    if (c.dW[0] || c.dW[1]) {
        // the list holds the wanted matrices one after the other
        const T* const one[2] = {c.dW[0] ? dg : du, du};
        void* const out[2] = {c.dW[0] ? c.dW[0] : c.dW[1], c.dW[1]};
        for (int i = 0; i < 2; ++i) {
            if (!make_map(&maps.d[i], one[i], c.tokens, c.m, ldd, BK, c.dtype)) return EXTERND_ECUDA;
            g.s[i] = out[i];
        }
        if (!make_map(&maps.x, c.X, c.tokens, c.n, c.ldx, BK, c.dtype)) return EXTERND_ECUDA;
        g.half_r = ceil_div(c.m, BM);
        g.grad = {(c.dW[0] && c.dW[1] ? 2 : 1) * g.half_r, ceil_div(c.n, width), (int)c.m, (int)c.n, ceil_div(c.tokens, BK), 1};
        g.lds = c.lddw;
        g.skip = g.main.tiles_r ? (g.main.blocks / splits + g.grad.blocks / 2) / g.grad.blocks : 0;
    }
    return launch_gemm<T, BWD, CG>(maps, g, c.stream) == cudaSuccess ? EXTERND_OK : EXTERND_ECUDA;
}

template <typename T>
int backward(const Call& c, const AlignJobs& jobs) {
    const int64_t ldd = round8(c.m);
    const size_t plane = plane_bytes(c.tokens, c.m, 2);
    const int splits = c.dX ? dx_splits(c.m, c.n, c.tokens) : 1;
    if (!c.work || c.work_bytes < 2 * plane + share_bytes(c.m, c.n, c.tokens)) return EXTERND_EINVAL;
    T* const dg = (T*)c.work;
    T* const du = (T*)(c.work + plane);
    float* const part = (float*)(c.work + 2 * plane);
    const cudaError_t e = c.save_dtype == EXTERND_F32 ? gate_grad<T, float>(c, dg, du, ldd, jobs) : gate_grad<T, unsigned short>(c, dg, du, ldd, jobs);
    if (e != cudaSuccess) return EXTERND_ECUDA;
    // as for the forward pass: the stages the busiest worker goes through, weighted.  4096 x 6912 x 2560, whole pass: pairs
    // 455 us, single CTAs 513, half as wide 756 with twice the stages; 1184 tokens: 158, 180, 257.  The second weight leans
    // further to pairs than these times (1.13, 1.14): over 120 shapes (32 to 4096 tokens, 300 to 6912 rows, depths 300 to
    // 2560) the plan taken is 2.8 % slower than the best of the three on average, at worst 45 % (32 tokens x 5504 x 768: 30.7 us,
    // single CTAs 21.1), and with a weight of 1.14 it would be 0.9 % and 20 %.
    struct { int cg, width; double stage; } const shapes[3] = {{2, 256, 1.00}, {1, 256, 1.20}, {1, 128, 0.85}};
    int best_i = 0;
    double best = 1e300;
    for (int i = 0; i < 3; ++i) {
        const int cg = shapes[i].cg, workers = sm_count() / cg, cols = ceil_div(c.n, shapes[i].width);
        const double nx = c.dX ? (double)ceil_div(c.tokens, 128 * cg) * cols * splits : 0, lx = 2.0 * ceil_div(c.m, BK) / splits;
        const double nw = ((c.dW[0] ? 1.0 : 0.0) + (c.dW[1] ? 1.0 : 0.0)) * ceil_div(c.m, 128 * cg) * cols, lw = ceil_div(c.tokens, BK) > 8 ? ceil_div(c.tokens, BK) : 8;   // storing a tile takes 8 stages' time
        const double even = (nx * lx + nw * lw) / workers + (nw > 0 ? lw / 2 : 0), longest = ceil_div((int64_t)nx, workers) * lx;
        const double cost = (even > longest ? even : longest) * shapes[i].stage;
        if (cost < best) { best = cost; best_i = i; }
    }
    const int rc = best_i == 0   ? backward_tiles<T, 2>(c, dg, du, ldd, part, splits, 256)
                   : best_i == 1 ? backward_tiles<T, 1>(c, dg, du, ldd, part, splits, 256)
                                 : backward_tiles<T, 1>(c, dg, du, ldd, part, splits, 128);
    if (rc != EXTERND_OK || splits == 1) return rc;
    const int64_t items = c.tokens * (round8(c.n) / 4), cap = (int64_t)sm_count() * 16;
    add_shares_kernel<T><<<(unsigned)((items + 255) / 256 < cap ? (items + 255) / 256 : cap), 256, 0, c.stream>>>(
        part, round8(c.n), splits, c.tokens, c.n, (T*)c.dX, c.lddx);
    return cudaGetLastError() == cudaSuccess ? EXTERND_OK : EXTERND_ECUDA;
}

bool too_large(int64_t m, int64_t n, int64_t tokens) {
    const int64_t lim = 0x7fffffff - 1024;
    if (m > lim || n > lim || tokens > lim) return true;
    return (tokens / 128 + 1) * (m / 128 + 1) > lim || (tokens / 128 + 1) * (n / 128 + 1) > lim || 2 * (m / 128 + 1) * (n / 128 + 1) > lim;
}

// a matrix of elements of `bytes` bytes with at least `cols` columns of its leading dimension
bool good(const Device& dev, const void* p, size_t bytes, int64_t ld, int64_t cols) {
    return p && aligned(p, bytes) && ld >= cols && dev.holds(p);
}

bool good_common(const Device& dev, const Call& c) {
    if (c.m < 1 || c.n < 1 || c.tokens < 0 || (c.dtype != EXTERND_F16 && c.dtype != EXTERND_BF16) || !valid_act(c.act)) return false;
    if (c.work_bytes && !c.work) return false;
    if (c.work && (!aligned(c.work, 256) || !dev.holds(c.work))) return false;
    return !c.status || (aligned(c.status, 4) && dev.holds(c.status));
}

bool good_saved(const Device& dev, const Call& c) {
    if (c.save_dtype != EXTERND_F32 && c.save_dtype != c.dtype) return false;
    const size_t b = dtype_bytes(c.save_dtype);
    return good(dev, c.S[0], b, c.lds, c.m) && good(dev, c.S[1], b, c.lds, c.m);
}

}  // namespace externd_ffn

namespace externd_llm {

WaitFault& wait_fault() {
    thread_local WaitFault f;
    return f;
}

}  // namespace externd_llm

using namespace externd_ffn;

extern "C" {

int externd_debug_wait_fault(double wait_limit_s, int withhold) {
    if (!(wait_limit_s == 0.0 || (wait_limit_s >= 0.001 && wait_limit_s <= 2.0)) || withhold < 0) return EXTERND_EINVAL;
    wait_fault().limit_ns = wait_limit_s == 0.0 ? WAIT_LIMIT_NS : (uint64_t)(wait_limit_s * 1e9);
    wait_fault().withhold = withhold;
    return EXTERND_OK;
}

size_t externd_aligned_bytes(int dtype, int64_t rows, int64_t n) {
    return rows < 1 || n < 1 || !valid_dtype(dtype) ? 0 : plane_bytes(rows, n, dtype_bytes(dtype));
}

int externd_gated(const void* X, int64_t ldx, const void* Wg, int64_t ldg, const void* Wu, int64_t ldu, int dtype, int64_t m, int64_t n,
                  int64_t tokens, int act, void* H, int64_t ldh, void* G, void* U, int save_dtype, int64_t ldgu, void* work,
                  size_t work_bytes, int* async_status, void* stream) {
    Call c = {};
    c.X = X; c.ldx = ldx; c.W[0] = Wg; c.ldw[0] = ldg; c.W[1] = Wu; c.ldw[1] = ldu;
    c.dtype = dtype; c.m = m; c.n = n; c.tokens = tokens; c.act = act;
    c.H = H; c.ldh = ldh; c.S[0] = G; c.S[1] = U; c.save_dtype = save_dtype; c.lds = ldgu;
    c.work = (unsigned char*)work; c.work_bytes = work_bytes; c.status = async_status;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    const Device dev;
    if (!good_common(dev, c) || !G != !U) return EXTERND_EINVAL;
    if (!good(dev, Wg, 2, ldg, n) || !good(dev, Wu, 2, ldu, n)) return EXTERND_EINVAL;
    if (tokens > 0) {
        if (!good(dev, X, 2, ldx, n) || !good(dev, H, 2, ldh, m) || (G && !good_saved(dev, c))) return EXTERND_EINVAL;
        if (too_large(m, n, tokens)) return EXTERND_ELIMIT;
    }
    if (async_status && cudaMemsetAsync(async_status, 0, sizeof(int), c.stream) != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
    if (tokens == 0) return EXTERND_OK;
    AlignJobs jobs = {};
    int rc = !place_operands(c, true, true, jobs) ? EXTERND_EINVAL : launch_align(jobs, c.stream) != cudaSuccess ? EXTERND_ECUDA : EXTERND_OK;
    if (rc == EXTERND_OK) rc = dtype == EXTERND_F16 ? forward<__half>(c) : forward<__nv_bfloat16>(c);
    if (rc != EXTERND_OK) cudaGetLastError();
    return rc;
}

size_t externd_gated_backward_work(int64_t m, int64_t n, int64_t tokens) {
    return m < 1 || n < 1 || tokens < 1 || too_large(m, n, tokens) ? 0 : 2 * plane_bytes(tokens, m, 2) + share_bytes(m, n, tokens);
}

int externd_gated_backward(const void* dH, int64_t lddh, const void* X, int64_t ldx, const void* Wg, int64_t ldg, const void* Wu,
                           int64_t ldu, const void* G, const void* U, int save_dtype, int64_t ldgu, int dtype, int64_t m, int64_t n,
                           int64_t tokens, int act, void* dX, int64_t lddx, void* dWg, void* dWu, int64_t lddw, void* work,
                           size_t work_bytes, int* async_status, void* stream) {
    Call c = {};
    c.X = X; c.ldx = ldx; c.W[0] = Wg; c.ldw[0] = ldg; c.W[1] = Wu; c.ldw[1] = ldu;
    c.dtype = dtype; c.m = m; c.n = n; c.tokens = tokens; c.act = act;
    c.S[0] = const_cast<void*>(G); c.S[1] = const_cast<void*>(U); c.save_dtype = save_dtype; c.lds = ldgu;
    c.dH = dH; c.lddh = lddh; c.dX = dX; c.lddx = lddx; c.dW[0] = dWg; c.dW[1] = dWu; c.lddw = lddw;
    c.work = (unsigned char*)work; c.work_bytes = work_bytes; c.status = async_status;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    const Device dev;
    const bool dw = dWg || dWu;
    if (!good_common(dev, c)) return EXTERND_EINVAL;
    for (void* p : c.dW)
        if (p && !good(dev, p, 2, lddw, n)) return EXTERND_EINVAL;
    if (tokens > 0 && (dX || dw)) {
        if (!good(dev, dH, 2, lddh, m) || !good_saved(dev, c)) return EXTERND_EINVAL;
        if (dX && (!good(dev, dX, 2, lddx, n) || !good(dev, Wg, 2, ldg, n) || !good(dev, Wu, 2, ldu, n))) return EXTERND_EINVAL;
        if (dw && !good(dev, X, 2, ldx, n)) return EXTERND_EINVAL;
        if (too_large(m, n, tokens)) return EXTERND_ELIMIT;
        size_t need = externd_gated_backward_work(m, n, tokens);
        if (dX)
            for (int i = 0; i < 2; ++i) need += row_aligned(c.W[i], m, c.ldw[i], 2) ? 0 : plane_bytes(m, n, 2);
        if (dw) need += row_aligned(X, tokens, ldx, 2) ? 0 : plane_bytes(tokens, n, 2);
        if (!work || work_bytes < need) return EXTERND_EINVAL;
    }
    if (async_status && cudaMemsetAsync(async_status, 0, sizeof(int), c.stream) != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
    if (tokens == 0) {
        for (void* p : c.dW)   // a sum of no terms
            if (p && cudaMemset2DAsync(p, (size_t)lddw * 2, 0, (size_t)n * 2, (size_t)m, c.stream) != cudaSuccess) { cudaGetLastError(); return EXTERND_ECUDA; }
        return EXTERND_OK;
    }
    if (!dX && !dw) return EXTERND_OK;
    AlignJobs jobs = {};
    int rc = place_operands(c, dw, dX != nullptr, jobs) ? EXTERND_OK : EXTERND_EINVAL;
    if (rc == EXTERND_OK) rc = dtype == EXTERND_F16 ? backward<__half>(c, jobs) : backward<__nv_bfloat16>(c, jobs);
    if (rc != EXTERND_OK) cudaGetLastError();
    return rc;
}

}  // extern "C"
