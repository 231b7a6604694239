// The product of two microscaled 4-bit matrices on the 5th-generation tensor
// cores (zs_mx4_matmul): out[m][n] = sum over k of A[m][k] * B[n][k].
//
// tcgen05.mma kind::mxf4 multiplies e2m1 codes, applies both scales and adds
// in float32 in tensor memory, 64 elements of k an instruction.  256 elements
// of k are 128 bytes a row, one 128-byte swizzled tensor copy an operand, and
// two scale atoms a 128 rows, which tcgen05.cp moves to tensor memory; a stage
// holds them once or twice.  One warp loads, one issues the products, the
// others store.
//
// Two kernels, by the work there is:
//  - products that give every pair of SMs about a 256 x 256 tile or more:
//    mx4_matmul_pair_kernel.  8192 x 14336 x 4096 bf16: 139 us, 6.9 PFLOP/s in
//    short runs, 156 us, 6.2 PFLOP/s in long ones, which run at the board's
//    power limit; 8192 x 8192 x 8192 147 us, 7.5 PFLOP/s, and 163 us.
//  - smaller ones: mx4_matmul_kernel, tiles of 128 rows, k shared out over a
//    cluster when the tiles are few.  One token through 4096 x 14336: 8.0 us
//    from HBM, 3.9 TB/s of weight bytes, 6.0 from L2; 16 through 14336 x 4096:
//    7.3 and 5.1 us; 256 x 4096 x 4096 from L2: 8.3 us.  What is left there is
//    the latency of a chain of few stages and the 2.1 us of a launch that
//    computes nothing.
#include <atomic>

#include "zs_launch.h"
#include "zs_mx4.cuh"

namespace zsk {

constexpr int MM_P = 128;                 // rows of P a tile: lanes of tensor memory
constexpr int MM_KB = 128;                // bytes of a row a stage: 256 elements
constexpr int MM_THREADS = 192;           // 4 warps store, 1 loads, 1 multiplies
constexpr uint64_t MM_WAIT_NS = 1000000000ull;   // one wait gives up after 1 s

__device__ int g_mx4_wait_timeouts;       // waits that gave up

// The least shared memory of a CTA that allocates `cols` columns of an SM's
// 512 of tensor memory: the CTAs that fit an SM by their shared memory then
// never want more columns than it has, whichever calls they are of.  (128
// columns are one of four shares, and five do not fit.)  A CTA of a split
// keeps its columns until its cluster's others have their sums, and
// tcgen05.alloc waits without a bound: without this, clusters of several
// streams that share SMs could each wait for columns that another one keeps.
constexpr int SM_SHARED = 228 * 1024;
constexpr int tmem_share(int cols) { return cols / 128 * ((SM_SHARED / 5 + 1024) / 1024 * 1024); }
static_assert(5 * tmem_share(128) > SM_SHARED, "more than 512 columns would fit an SM");

// P holds the tile's 128 rows, Q its BN; D[p][q].
template <int BN>
struct MmShape {
    static constexpr int P_BYTES = MM_P * MM_KB, Q_BYTES = BN * MM_KB;
    static constexpr int SP_BYTES = 2 * MX4_ATOM, SQ_BYTES = 2 * MX4_ATOM;
    static constexpr int SUB = P_BYTES + Q_BYTES + SP_BYTES + SQ_BYTES;      // 256 elements of k, a multiple of 1024
    // Of them a stage.  Waiting for a stage and releasing it costs the issuing
    // warp about as much as its products, so two where enough fit: 16 x 14336
    // x 4096 from L2 takes 6.46 us with four stages of one, 5.32 with two of
    // two; for 128 columns two of two lost to three of one, 128 x 4096 x 4096
    // 7.9 us against 7.6.
    static constexpr int KS = BN == 128 ? 1 : 2;
    static constexpr int STAGE = KS * SUB;
    // At most; a launch takes no more than its parts of k fill, so that two
    // CTAs share an SM where parts are short and the next kernel's begin
    // early (1 x 4096 x 4096 3.9 us, with four always 4.2).  Bytes in flight
    // count where the matrix is not in L2: 1 x 4096 x 14336 9.6, 8.5, 8.1 and
    // 8.3 us with 2, 3, 4 and 5 of two; 256 x 4096 x 14336 16.8, 15.0 and 13.7
    // with 3, 4 and 6 of one (from L2, 256 x 4096 x 4096 8.0, 8.2 and 8.4).
    static constexpr int STAGES = BN == 128 ? 6 : 4;
    // tensor memory: accumulator, then two sets of scales
    static constexpr int SP_COL = BN < 32 ? 32 : BN, SQ_COL = SP_COL + 16 * KS;
    static constexpr int USED = SQ_COL + 16 * KS;
    static constexpr int COLS = USED <= 128 ? 128 : 256;                     // two CTAs of an SM fit
    static constexpr int RED = BN * MM_P * 4 + 16 * (BN > MM_P ? BN : MM_P);   // the tile, rows 16 bytes apart
    static constexpr int need(int stages) { return (stages * STAGE > RED ? stages * STAGE : RED) + 1024; }   // with room to align
    static constexpr int smem(int stages) { return need(stages) > tmem_share(COLS) ? need(stages) : tmem_share(COLS); }
    static constexpr int SMEM = smem(STAGES);
    static_assert(COLS % 128 == 0 && smem(1) >= tmem_share(COLS), "CTAs that share an SM have to find their columns");
};

struct MmArgs {
    const uint8_t *p_scales, *q_scales;
    void *out;
    int64_t ldo;
    int32_t np, nq;           // rows of P and Q
    int32_t k_tiles, atoms;   // stages along k, scale atoms a row tile
    int32_t p_tiles, q_tiles;
    int32_t split;            // CTAs of the cluster that share the tile's k
    int32_t stages;           // of the ring
    int32_t dtype;
    int32_t vec;              // rows of out are aligned to 4 elements
    int32_t give_up;          // for tests: the stage of the last part whose wait runs out, or -1
};

__device__ __forceinline__ uint64_t mm_desc(uint32_t addr, uint32_t sbo, uint64_t layout) {
    // shared-memory operand: start address, leading and stride byte offsets
    // (16-byte units), version 1, swizzle
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(sbo >> 4) << 32) |
           ((uint64_t)1 << 46) | (layout << 61);
}

__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :
                 : "r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" : : "r"(bar) : "memory");
}

__device__ __forceinline__ void tc_ld32_nowait(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}

__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t *v) {
    tc_ld32_nowait(addr, v);
    asm volatile("tcgen05.wait::ld.sync.aligned;" : : : "memory");
}

__device__ __forceinline__ uint32_t mm_cast(float x, int dtype) {
    return dtype == ZS_DTYPE_FP16 ? FP16T::from_f32(x) : BF16T::from_f32(x);
}

// Tiles of 128 rows of P by BN of Q.  FLIP: P are the rows of B (features) and
// Q those of A (tokens), for up to 64 tokens: out[q][p]; the tensor cores'
// 128 rows are then filled by features, and a product over few tokens reads
// the weight's bytes and little else.  Otherwise out[p][q].  split > 1: the
// CTAs of a cluster take parts of k and add their tiles through distributed
// shared memory, in the order of the parts, so that a result has the same bits
// every time.
template <int BN, bool FLIP>
__global__ void __launch_bounds__(MM_THREADS)
mx4_matmul_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, MmArgs a) {
    using S = MmShape<BN>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::STAGES + 1];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int failed;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(bars), done = bar0 + 16 * S::STAGES;
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (S::STAGES + s); };
    const int stages = a.stages;
    const int part = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    const int tile = (int)(blockIdx.x / a.split);
    const int pt = tile % a.p_tiles, qt = tile / a.p_tiles;
    const int k0 = (int)((int64_t)a.k_tiles * part / a.split), k1 = (int)((int64_t)a.k_tiles * (part + 1) / a.split);
    // the loading warp sets up the barriers and begins; the others join it
    // behind the __syncthreads below
    const uint8_t *sp = a.p_scales + ((int64_t)pt * a.atoms) * MX4_ATOM;
    const int steps = (k1 - k0 + S::KS - 1) / S::KS;
    const int give_up = part == a.split - 1 ? a.give_up : -1;
    auto load = [&](int i, int s) {
        if (elect_one()) {
            const int n = min(S::KS, k1 - k0 - i * S::KS);
            // (give_up: 16 bytes that never come)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" : : "r"(full(s)), "r"(n * S::SUB + (i == give_up ? 16 : 0)) : "memory");
#pragma unroll
            for (int h = 0; h < S::KS; ++h) {
                if (h >= n) break;
                const int k = k0 + i * S::KS + h;
                const uint32_t p = base + s * S::STAGE + h * S::SUB, q = p + S::P_BYTES, scp = q + S::Q_BYTES, scq = scp + S::SP_BYTES;
                tma2d(p, &map_p, k * MM_KB, pt * MM_P, full(s));
                tma2d(q, &map_q, k * MM_KB, qt * BN, full(s));
                bulk(scp, sp + (int64_t)k * S::SP_BYTES, S::SP_BYTES, full(s));
                bulk(scq, a.q_scales + ((int64_t)(BN == 128 ? qt : 0) * a.atoms + 2 * k) * MX4_ATOM, S::SQ_BYTES, full(s));
            }
        }
        __syncwarp();
    };
    int issued = 0, slot = 0;              // stages that warp 4 issued loads for; the next one's place
    if (warp == 4) {
        if (elect_one()) {
            failed = 0;
            for (int i = 0; i < 2 * S::STAGES + 1; ++i)
                asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" : : "r"(bar0 + 8 * i) : "memory");
            asm volatile("fence.mbarrier_init.release.cluster;" : : : "memory");
            asm volatile("fence.proxy.async.shared::cta;" : : : "memory");
        }
        __syncwarp();
        pdl_wait();
        for (; issued < stages && issued < steps; ++issued) load(issued, issued);
    }
    if (warp == 5 && elect_one()) {
        asm volatile("prefetch.tensormap [%0];" : : "l"(&map_p) : "memory");
        asm volatile("prefetch.tensormap [%0];" : : "l"(&map_q) : "memory");
    }
    __syncwarp();
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :
                     : "r"(smem_u32(&tmem_base)), "n"(S::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" : : : "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
    const uint32_t tmem = tmem_base;
    pdl_trigger();                         // tensor memory is allocated: the next kernel may wait for its own

    if (warp == 4) {
        uint32_t phase = 0;
        for (; issued < steps; ++issued) {
            if (!warp_wait(empty(slot), phase, MM_WAIT_NS)) {
                failed = 1;
                break;
            }
            load(issued, slot);
            if (++slot == stages) {
                slot = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 5) {
        // kind::mxf4: e2m1 x e2m1, ue8m0 scales, M = 128, N = BN
        const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(BN / 8) << 17) | (1u << 23) | (8u << 24);
        int s = 0;
        uint32_t phase = 0;
        for (int i = 0; i < steps; ++i) {
            if (!warp_wait(full(s), phase, MM_WAIT_NS)) {
                // the storing warps are to know it, and to find no load in
                // flight to where they write, when they see `done`
                for (int j = i + 1; j < steps && j < i + stages; ++j)
                    if (!warp_wait(full(j % stages), (uint32_t)((j / stages) & 1), MM_WAIT_NS)) break;
                failed = 1;
                __threadfence_block();
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
            const int n = min(S::KS, k1 - k0 - i * S::KS);
            if (elect_one()) {
#pragma unroll
                for (int h = 0; h < S::KS; ++h) {
                    if (h >= n) break;
                    const uint32_t p = base + s * S::STAGE + h * S::SUB, q = p + S::P_BYTES, scp = q + S::Q_BYTES, scq = scp + S::SP_BYTES;
                    const uint32_t tp = tmem + S::SP_COL + 8 * (S::KS * (i & 1) + h), tq = tmem + S::SQ_COL + 8 * (S::KS * (i & 1) + h);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;"
                                     :
                                     : "r"(tp + 4 * j), "l"(mm_desc(scp + j * MX4_ATOM, 128, 0))
                                     : "memory");
                        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;"
                                     :
                                     : "r"(tq + 4 * j), "l"(mm_desc(scq + j * MX4_ATOM, 128, 0))
                                     : "memory");
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t id = (uint32_t)(2 * (j & 1));        // scale bytes 0-1 or 2-3 of an atom
                        const uint32_t d = idesc | (id << 4) | (id << 29);
                        asm volatile(
                            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
                            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                            :
                            : "r"(tmem), "l"(mm_desc(p + 32 * j, 1024, 2)), "l"(mm_desc(q + 32 * j, 1024, 2)), "r"(d),
                              "r"(tp + 4 * (j >> 1)), "r"(tq + 4 * (j >> 1)), "r"((uint32_t)(i > 0 || h > 0 || j > 0))
                            : "memory");
                    }
                }
                tc_commit(empty(s));
            }
            __syncwarp();
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
        __syncwarp();
        if (elect_one()) tc_commit(done);
        __syncwarp();
    }
    // everyone waits until the products of this CTA are in tensor memory
    if (!mbar_wait_quick(done, 0, 4 * MM_WAIT_NS + 4000ull * (uint64_t)(k1 - k0))) failed = 1;
    __syncwarp();
    // an unfinished sum is NaN, for the other parts of a split too
    const bool unfinished = failed;
    asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
    // The tile goes to shared memory as rows of out (the loads and products
    // that used it are done), then the CTAs of a split share it out, each
    // element summed over the parts in order, and store neighbouring columns.
    constexpr int ROWS = FLIP ? BN : MM_P, COLS = FLIP ? MM_P : BN, PITCH = 4 * COLS + 16;
    const int row0 = FLIP ? qt * BN : pt * MM_P, col0 = FLIP ? pt * MM_P : qt * BN;
    const int rows = min(ROWS, (FLIP ? a.nq : a.np) - row0), cols = min(COLS, (FLIP ? a.np : a.nq) - col0);
    if (warp < 4) {
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
            if (FLIP && c >= rows) break;
            uint32_t v[32];
            tc_ld32(tmem + ((uint32_t)warp << 21) + c, v);
            if (unfinished) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0x7FC00000u;
            }
            if (FLIP) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i < ROWS)
                        asm volatile("st.shared.b32 [%0], %1;" : : "r"(base + PITCH * (c + i) + 4 * (32 * warp + lane)), "r"(v[i]) : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 :
                                 : "r"(base + PITCH * (32 * warp + lane) + 4 * c + 16 * i), "r"(v[4 * i]), "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                                 : "memory");
            }
        }
    }
    __syncwarp();
    if (a.split > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" : : : "memory");
    else __syncthreads();
    {
        const int es = a.dtype == ZS_DTYPE_FP32 ? 4 : 2;
        const int units = rows * (COLS / 4), step = a.split * MM_THREADS;      // runs of 4 columns
        auto store = [&](int u, const float (&f)[4]) {
            const int r = u / (COLS / 4), c = 4 * (u % (COLS / 4));
            if (c >= cols) return;
            char *o = static_cast<char *>(a.out) + ((int64_t)(row0 + r) * a.ldo + col0 + c) * es;
            if (a.vec && c + 4 <= cols) {
                if (es == 4) *reinterpret_cast<float4 *>(o) = make_float4(f[0], f[1], f[2], f[3]);
                else
                    *reinterpret_cast<uint2 *>(o) = make_uint2(mm_cast(f[0], a.dtype) | (mm_cast(f[1], a.dtype) << 16),
                                                               mm_cast(f[2], a.dtype) | (mm_cast(f[3], a.dtype) << 16));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < cols) {
                        if (es == 4) reinterpret_cast<float *>(o)[e] = f[e];
                        else reinterpret_cast<uint16_t *>(o)[e] = (uint16_t)mm_cast(f[e], a.dtype);
                    }
            }
        };
        auto place = [&](int u) { return base + PITCH * (u / (COLS / 4)) + 16 * (u % (COLS / 4)); };
        if (a.split == 1) {
            for (int u = threadIdx.x; u < units; u += MM_THREADS) {
                float f[4];
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(place(u)) : "memory");
                store(u, f);
            }
        } else {
            // several runs and parts at a time, so that the reads of the other
            // CTAs' shared memory overlap
            constexpr int RUNS = BN == 128 ? 4 : 1, PARTS = BN == 128 ? 2 : 4;
            for (int u0 = part * MM_THREADS + (int)threadIdx.x; u0 < units; u0 += RUNS * step) {
                float f[RUNS][4];
#pragma unroll
                for (int i = 0; i < RUNS; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[i][e] = 0.0f;
                for (int h = 0; h < a.split; h += PARTS) {
                    float x[PARTS][RUNS][4];
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int i = 0; i < RUNS; ++i)
                            if (u0 + i * step < units && h + p < a.split)
                                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                             : "=f"(x[p][i][0]), "=f"(x[p][i][1]), "=f"(x[p][i][2]), "=f"(x[p][i][3])
                                             : "r"(map_to(place(u0 + i * step), (uint32_t)(h + p)))
                                             : "memory");
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
                        if (h + p < a.split)
#pragma unroll
                            for (int i = 0; i < RUNS; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) f[i][e] = __fadd_rn(f[i][e], x[p][i][e]);
                }
#pragma unroll
                for (int i = 0; i < RUNS; ++i)
                    if (u0 + i * step < units) store(u0 + i * step, f[i]);
            }
        }
    }
    // no CTA leaves while another reads its part
    __syncwarp();
    if (a.split > 1) asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" : : : "memory");
    if (warp == 4 && lane == 0 && failed) {
        // let the loads already issued land before the shared memory goes away
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
            mbar_wait_quick(full(i % stages), (uint32_t)((i / stages) & 1), MM_WAIT_NS);
        atomicAdd(&g_mx4_wait_timeouts, 1);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory");
    __syncthreads();
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" : : "r"(tmem), "n"(S::COLS));
    }
}

// ------------------------------------------------------ two-SM products --
// For products with enough work: a cluster of two CTAs (two SMs) works on a
// 256 x 256 tile of out, each holding half of the rows of A and half of
// those of B in its shared memory, so that a byte of B is read once for
// 256 rows.  Persistent: a pair walks tiles, the loads running ahead over
// the tile boundary, while 8 warps of each CTA empty the accumulator of the
// previous tile into registers, release it, and store.  (Two accumulators of
// 256 columns would leave no tensor memory for the scales.)
// A stage takes the tensor cores 512 cycles (four instructions of K = 64; the
// PTX ISA lists K = 96 for sm_103a too, whose 48-byte steps would cross the
// 128-byte rows of a stage: not tried) and brings 35 KB to each SM.  With 6
// in flight 8192 x 8192 x 8192 takes 620 cycles a stage all in all, with 5 630,
// with 4 650, with 3 760: the way from a product's end over its barrier and the loads to the
// next product is what remains, besides 400 cycles a tile between its last
// product and the next one's first.  (Loads beside the products do not slow
// them, and the same loads from a few hot lines gained 4 %.)  Then power: the
// SMs run at 1.86 GHz in short runs, at 1.62 to 1.67 in long ones, at 1.36 kW.
// Clusters of two pairs that share B by multicast took as long (144 of the 152
// SMs fit such clusters); scales placed by tcgen05.st in the place of
// tcgen05.cp took 8192 x 8192 x 8192 387 us and more, where this form took 246
// at the time.
constexpr int PAIR_ROWS = 256, PAIR_COLS = 256;
constexpr int PAIR_THREADS = 320;         // 8 warps store, 1 loads, 1 multiplies (leader only)
constexpr int PAIR_P = 128 * MM_KB, PAIR_Q = 128 * MM_KB;
constexpr int PAIR_SP = 2 * MX4_ATOM, PAIR_SQ = 4 * MX4_ATOM;
constexpr int PAIR_STAGE = PAIR_P + PAIR_Q + PAIR_SP + PAIR_SQ;
constexpr int PAIR_SP_COL = 256, PAIR_SQ_COL = PAIR_SP_COL + 16;   // scales, two sets of each

// A ring of 5 stages leaves every storing warp a slab of 32 rows of 128 bytes,
// one of 6 rows of 64.
template <int STAGES>
struct PairShape {
    static constexpr int ROW = STAGES == 6 ? 64 : 128;
    static constexpr int SLAB = 32 * ROW;
    static constexpr int BARS = STAGES * PAIR_STAGE + 8 * SLAB;      // the barriers are after them
    static constexpr int SMEM = BARS + 256;
    static_assert(SMEM >= tmem_share(512), "nothing else of tensor memory shares the SM");
    // the 16-byte pieces of a row are turned by this: no bank conflicts
    static __device__ __forceinline__ int turn(int row) { return ROW == 128 ? row & 7 : (row >> 1) & 3; }
};

__device__ __forceinline__ void tma2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        :
        : "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :
        : "r"(bar), "h"((uint16_t)3)
        : "memory");
}

struct PairArgs {
    void *out;
    int64_t ldo;
    int32_t m, n;
    int32_t k_tiles, p_tiles, tiles;
    int32_t dtype;
    int32_t vec;              // rows of out are 16-byte aligned
    int32_t give_up;          // for tests: the stage (of a pair's) whose wait runs out, or -1
};

template <int STAGES>
__global__ void __launch_bounds__(PAIR_THREADS)
mx4_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_sp, const __grid_constant__ CUtensorMap map_sq, PairArgs a) {
    using S = PairShape<STAGES>;
    // the swizzle wants 1024-byte alignment; nothing static, so that none of it is lost
    extern __shared__ __align__(1024) uint8_t pair_raw[];
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(pair_raw), bar0 = base + S::BARS;
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(pair_raw + S::BARS + 8 * (2 * STAGES + 2));
    volatile int &failed = *reinterpret_cast<volatile int *>(pair_raw + S::BARS + 8 * (2 * STAGES + 3));
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (STAGES + s); };
    const uint32_t acc_full = bar0 + 16 * STAGES, acc_empty = acc_full + 8;
    const int rank = (int)(blockIdx.x & 1);
    const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        failed = 0;
        for (int i = 0; i < 2 * STAGES + 1; ++i)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" : : "r"(bar0 + 8 * i) : "memory");
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 16;" : : "r"(acc_empty) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" : : : "memory");
        asm volatile("fence.proxy.async.shared::cta;" : : : "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" : : "r"(smem_u32(&tmem_base)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" : : : "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" : : : "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
    const uint32_t tmem = tmem_base;
    pdl_trigger();                         // tensor memory is allocated: the next kernel may wait for its own
    // every role: the limits of the waits below begin when the loads can, not
    // while the previous kernel still works
    pdl_wait();

    int issued = 0;
    if (warp == 8) {
        // loads of this CTA: its half of the rows of A and of B, the scales
        // of its rows of A, and all the tile's scales of B
        bool ok = true;
        for (int t = first; t < a.tiles && ok; t += stride) {
            const int pt = t % a.p_tiles, qt = t / a.p_tiles;
            for (int k = 0; k < a.k_tiles; ++k, ++issued) {
                const int s = issued % STAGES;
                if (issued >= STAGES && !warp_wait(empty(s), (uint32_t)((issued / STAGES - 1) & 1), MM_WAIT_NS)) {
                    failed = 1;
                    ok = false;
                    break;
                }
                const uint32_t p = base + s * PAIR_STAGE, q = p + PAIR_P, sp = q + PAIR_Q, sq = sp + PAIR_SP;
                if (elect_one()) {
                    const uint32_t bar = map_to(full(s), 0);       // the leader multiplies for both
                    if (rank == 0)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" : : "r"(full(s)), "r"(2 * PAIR_STAGE + (issued == a.give_up ? 16 : 0)) : "memory");
                    tma2d_pair(p, &map_p, k * MM_KB, pt * PAIR_ROWS + rank * 128, bar);
                    tma2d_pair(q, &map_q, k * MM_KB, qt * PAIR_COLS + rank * 128, bar);
                    tma2d_pair(sp, &map_sp, k * (PAIR_SP / 4), pt * 2 + rank, bar);
                    tma2d_pair(sq, &map_sq, k * (PAIR_SP / 4), qt * 2, bar);
                }
                __syncwarp();
            }
        }
        // every signal to this CTA's barriers has come before it leaves
        for (int i = issued > STAGES ? issued - STAGES : 0; ok && i < issued; ++i)
            ok = warp_wait(empty(i % STAGES), (uint32_t)((i / STAGES) & 1), MM_WAIT_NS);
        if (!ok) failed = 1;
    } else if (warp == 9 && rank == 0) {
        const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(PAIR_COLS / 8) << 17) | (1u << 23) | (16u << 24);
        int i = 0, n = 0;
        bool ok = true;
        for (int t = first; t < a.tiles && ok; t += stride, ++n) {
            if (n > 0 && !warp_wait(acc_empty, (uint32_t)((n - 1) & 1), MM_WAIT_NS)) {
                failed = 1;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
            for (int k = 0; k < a.k_tiles; ++k, ++i) {
                const int s = i % STAGES;
                if (!warp_wait(full(s), (uint32_t)((i / STAGES) & 1), MM_WAIT_NS)) {
                    failed = 1;
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
                const uint32_t p = base + s * PAIR_STAGE, q = p + PAIR_P, sp = q + PAIR_Q, sq = sp + PAIR_SP;
                const uint32_t tp = tmem + PAIR_SP_COL + 8 * (i & 1), tq = tmem + PAIR_SQ_COL + 16 * (i & 1);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;"
                                     : : "r"(tp + 4 * j), "l"(mm_desc(sp + j * MX4_ATOM, 128, 0)) : "memory");
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;"
                                         : : "r"(tq + 4 * (2 * j + h)), "l"(mm_desc(sq + h * PAIR_SP + j * MX4_ATOM, 128, 0)) : "memory");
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t id = (uint32_t)(2 * (j & 1));
                        const uint32_t d = idesc | (id << 4) | (id << 29);
                        asm volatile(
                            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
                            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                            :
                            : "r"(tmem), "l"(mm_desc(p + 32 * j, 1024, 2)), "l"(mm_desc(q + 32 * j, 1024, 2)), "r"(d),
                              "r"(tp + 4 * (j >> 1)), "r"(tq + 8 * (j >> 1)), "r"((uint32_t)(k > 0 || j > 0))
                            : "memory");
                    }
                    tc_commit_pair(empty(s));
                }
                __syncwarp();
            }
            // an unfinished sum is never signalled: the storing warps of both
            // CTAs give up in their turn and leave the tile as it was
            if (ok && elect_one()) tc_commit_pair(acc_full);
            __syncwarp();
        }
    } else if (warp < 8) {
        const uint32_t slab = base + STAGES * PAIR_STAGE + warp * S::SLAB;
        const uint32_t release = map_to(acc_empty, 0);
        const int sub = warp & 3, c0 = 128 * (warp >> 2);
        int n = 0;
        for (int t = first; t < a.tiles; t += stride, ++n) {
            const int pt = t % a.p_tiles, qt = t / a.p_tiles;
            if (!warp_wait(acc_full, (uint32_t)(n & 1), 2 * MM_WAIT_NS + 4000ull * (uint64_t)a.k_tiles) ||
                __any_sync(0xFFFFFFFFu, failed)) {
                failed = 1;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
            uint32_t v[128];
#pragma unroll
            for (int j = 0; j < 4; ++j) tc_ld32_nowait(tmem + ((uint32_t)sub << 21) + c0 + 32 * j, v + 32 * j);
            asm volatile("tcgen05.wait::ld.sync.aligned;" : : : "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory");
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" : : "r"(release) : "memory");
            const int row0 = pt * PAIR_ROWS + rank * 128 + 32 * sub, col0 = qt * PAIR_COLS + c0;
            const bool fp32 = a.dtype == ZS_DTYPE_FP32;
            if (!fp32) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    v[i] = mm_cast(__uint_as_float(v[2 * i]), a.dtype) | (mm_cast(__uint_as_float(v[2 * i + 1]), a.dtype) << 16);
            }
            // 32 rows of ROW bytes at a time through this warp's slab; then
            // lanes store neighbouring elements
            constexpr int PER = S::ROW / 16;          // pieces of a row
            const int times = (fp32 ? 512 : 256) / S::ROW, width = S::ROW / (fp32 ? 4 : 2);
#pragma unroll
            for (int j = 0; j < 512 / S::ROW; ++j) {
                if (j >= times) break;
                const int col = col0 + j * width;
                if (row0 >= a.m || col >= a.n) break;
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 :
                                 : "r"(slab + S::ROW * lane + 16 * (c ^ S::turn(lane))), "r"(v[4 * PER * j + 4 * c]), "r"(v[4 * PER * j + 4 * c + 1]),
                                   "r"(v[4 * PER * j + 4 * c + 2]), "r"(v[4 * PER * j + 4 * c + 3])
                                 : "memory");
                __syncwarp();
                if (a.vec && col + width <= a.n) {
                    // whole lines (or their halves) of several rows a store
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int row = 32 / PER * i + lane / PER;
                        uint32_t x[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                     : "r"(slab + S::ROW * row + 16 * (lane % PER ^ S::turn(row)))
                                     : "memory");
                        if (row0 + row < a.m)
                            *reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + ((int64_t)(row0 + row) * a.ldo + col) * (fp32 ? 4 : 2) + 16 * (lane % PER)) =
                                make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    __syncwarp();
                    continue;
                }
                const int rows = min(32, a.m - row0);
                // 8 reads, then their stores: a row of fp32 slabs is 16 or 32
                // elements, of 16-bit ones 32 or 64
                auto element = [&](int row, int byte) { return slab + S::ROW * row + (byte ^ (16 * S::turn(row))); };
                if (fp32) {
                    constexpr int WIDTH = S::ROW / 4, SKIP = 32 / WIDTH;         // rows a read
                    const int c = lane % WIDTH;
#pragma unroll 1
                    for (int i = lane / WIDTH; i < rows; i += 8 * SKIP) {
                        uint32_t x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[e]) : "r"(element(i + SKIP * e, 4 * c)) : "memory");
                        float *o = static_cast<float *>(a.out) + (int64_t)(row0 + i) * a.ldo + col + c;
                        if (col + c < a.n) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (i + SKIP * e < rows) o[SKIP * e * a.ldo] = __uint_as_float(x[e]);
                        }
                    }
                } else {
                    constexpr int TIMES = S::ROW / 64;                           // reads a row
                    uint16_t *o = static_cast<uint16_t *>(a.out) + (int64_t)row0 * a.ldo + col + lane;
#pragma unroll 1
                    for (int i = 0; i < rows; i += 8 / TIMES, o += 8 / TIMES * a.ldo) {
                        uint32_t x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            asm volatile("ld.shared.u16 %0, [%1];"
                                         : "=r"(x[e])
                                         : "r"(element(i + e / TIMES, 2 * (32 * (e % TIMES) + lane)))
                                         : "memory");
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (i + e / TIMES < rows && col + 32 * (e % TIMES) + lane < a.n)
                                o[(e / TIMES) * a.ldo + 32 * (e % TIMES)] = (uint16_t)x[e];
                    }
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory");
    __syncthreads();                       // every role has said whether it gave up
    if (warp == 8 && lane == 0 && failed) {
        if (rank == 0)   // the leader's barriers count the loads of both CTAs
            for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                mbar_wait_quick(full(i % STAGES), (uint32_t)((i / STAGES) & 1), MM_WAIT_NS);
        atomicAdd(&g_mx4_wait_timeouts, 1);
    }
    __syncwarp();
    // neither CTA leaves while the other may still write to its barriers
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" : : : "memory");
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" : : "r"(tmem));
    }
}

// out = 0, for a product over no elements
__global__ void mx4_zero_kernel(void *out, int64_t m, int64_t n, int64_t ldo, int fp32) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < m * n; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / n * ldo + i % n;
        if (fp32) static_cast<float *>(out)[at] = 0.0f;
        else static_cast<uint16_t *>(out)[at] = 0;
    }
}

// Codes as bytes [rows][row_bytes]: boxes of 128 bytes (256 elements) by
// `box` rows; zero (value 0) outside.
static bool code_map(CUtensorMap *m, const void *codes, int64_t rows, int64_t row_bytes, int box) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t boxes[2] = {MM_KB, (cuuint32_t)box}, ones[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(codes), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale atoms as 32-bit words [row tiles][atoms * 128]: boxes of two atoms
// (256 elements of k) by `box` row tiles; zero outside.
static bool scale_map(CUtensorMap *m, const void *scales, int64_t rows, int64_t cols, int box) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t words = (cuuint64_t)mx4_atoms(cols) * (MX4_ATOM / 4);
    const cuuint64_t dims[2] = {words, (cuuint64_t)mx4_row_tiles(rows)}, strides[1] = {4 * words};
    const cuuint32_t boxes[2] = {2 * MX4_ATOM / 4, (cuuint32_t)box}, ones[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(scales), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The device's SM count, once its kernel attributes are set (`set`, the same
// from every host thread).
static cudaError_t device_sms(std::atomic<int> (&known)[64], cudaError_t (*set)(), int *sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    *sms = known[dev].load(std::memory_order_relaxed);
    if (*sms > 0) return cudaSuccess;
    if ((e = set()) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    known[dev].store(*sms, std::memory_order_relaxed);
    return cudaSuccess;
}

template <int STAGES>
static cudaError_t pair_launch(const CUtensorMap (&map)[4], const PairArgs &a, cudaStream_t s) {
    static std::atomic<int> known[64];
    int sms = 0;
    const cudaError_t e = device_sms(known, [] {
        return cudaFuncSetAttribute(mx4_matmul_pair_kernel<STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, PairShape<STAGES>::SMEM);
    }, &sms);
    if (e != cudaSuccess) return e;
    const int pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
    return launch_dependent(mx4_matmul_pair_kernel<STAGES>, (unsigned)(2 * pairs), PAIR_THREADS, PairShape<STAGES>::SMEM, 2, s, map[0], map[1], map[2], map[3], a);
}

// What zs_mx4_matmul launches for a product.
struct MmPlan {
    bool pair, flip;
    int bn, split, stages;
    int smem, columns;        // of a CTA: shared memory, tensor memory
    int64_t p_tiles, q_tiles;
};

template <int BN>
static void mm_ring(MmPlan &r, int k_tiles) {
    using S = MmShape<BN>;
    const int steps = ((k_tiles + r.split - 1) / r.split + S::KS - 1) / S::KS;     // of the longest part
    r.stages = steps < S::STAGES ? steps : S::STAGES;
    r.smem = S::smem(r.stages);
    r.columns = S::COLS;
}

static MmPlan mm_plan(int64_t m, int64_t n, int64_t k) {
    MmPlan r = {};
    const int k_tiles = (int)((k + 255) / 256);
    // The pair kernel from half a tile a pair on: 640 x 4096 x 4096 (48 tiles)
    // takes it 10.4 us, the other kernel 11.2; 1024 x 4096 x 14336 (64 tiles)
    // 21.3 and 25.1; 512 x 4096 x 4096 and 2048 x 1024 x 4096 (32 tiles) 9.6
    // and 8.5.
    r.p_tiles = (m + PAIR_ROWS - 1) / PAIR_ROWS;
    r.q_tiles = (n + PAIR_COLS - 1) / PAIR_COLS;
    if (m > 128 && r.p_tiles * r.q_tiles >= 38 && r.p_tiles * r.q_tiles < 0x7FFF0000) {
        r.pair = true;
        r.bn = PAIR_COLS;
        r.split = 1;
        // Every pair of the 76 has (tiles / 76) k_tiles stages.  When they are
        // many, 6 in flight: 8192 x 8192 x 8192 154 -> 148 us (fp32 out 169 ->
        // 160), 4096 x 4096 x 11008 59.6 -> 58.7; when few, the store after the
        // last tile counts, and slabs of whole lines: 1024 x 4096 x 4096 10.6 us
        // against 11.4, 4097 x 4100 x 4096 (64 stages) 28.6 against 29.1.
        r.stages = (r.p_tiles * r.q_tiles + 75) / 76 * k_tiles >= 128 ? 6 : 5;
        r.smem = r.stages == 6 ? PairShape<6>::SMEM : PairShape<5>::SMEM;
        r.columns = 512;
        return r;
    }
    // 128 features a tile for up to 64 tokens: 64 x 4096 x 4096 5.2 us, 5.8 with
    // 128 tokens a tile; 48 x 1024 x 4096 4.3 us against 5.0.
    r.flip = m <= 64;
    r.bn = !r.flip ? 128 : m <= 16 ? 16 : m <= 32 ? 32 : 64;   // flipped, one tile of Q: scale addresses are whole atoms
    r.p_tiles = ((r.flip ? n : m) + MM_P - 1) / MM_P;
    r.q_tiles = ((r.flip ? m : n) + r.bn - 1) / r.bn;
    // k is shared out while that leaves an SM to every CTA and each enough
    // stages to hide its part of the sum.  One token through 4096 x 4096 (32
    // tiles) took 5.8, 4.9, 4.2 and 4.5 us in 1, 2, 4 and 8 parts, 256 x 4096 x
    // 14336 (64 tiles) 17.3, 12.5 and 14.4 us in 1, 2 and 4; more CTAs than SMs
    // lose: 16 x 14336 x 4096 (112 tiles) 6.2 us in one part, 9.7 in four.
    r.split = 1;
    while (r.split < 8 && r.p_tiles * r.q_tiles * r.split * 2 <= 152 && k_tiles >= (r.bn == 128 ? 8 : 4) * r.split) r.split *= 2;
    if (r.bn == 16) mm_ring<16>(r, k_tiles);
    else if (r.bn == 32) mm_ring<32>(r, k_tiles);
    else if (r.bn == 64) mm_ring<64>(r, k_tiles);
    else mm_ring<128>(r, k_tiles);
    return r;
}

template <int BN, bool FLIP>
static cudaError_t mm_launch(const MmPlan &r, const CUtensorMap &p, const CUtensorMap &q, const MmArgs &a, cudaStream_t s) {
    static std::atomic<int> known[64];
    int sms = 0;
    cudaError_t e = device_sms(known, [] {
        return cudaFuncSetAttribute(mx4_matmul_kernel<BN, FLIP>, cudaFuncAttributeMaxDynamicSharedMemorySize, MmShape<BN>::SMEM);
    }, &sms);
    if (e != cudaSuccess) return e;
    return launch_dependent(mx4_matmul_kernel<BN, FLIP>, (unsigned)(r.p_tiles * r.q_tiles * r.split), MM_THREADS, r.smem,
                            (unsigned)r.split, s, p, q, a);
}

}  // namespace zsk

cudaError_t zsl_mx4_wait_timeouts(int *count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, zsk::g_mx4_wait_timeouts, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(zsk::g_mx4_wait_timeouts, &zero, sizeof(int));
    }
    return e;
}

extern "C" zs_status zs_mx4_matmul(int64_t m, int64_t n, int64_t k, const void *a_codes, const void *a_scales,
                                   const void *b_codes, const void *b_scales, void *out, int64_t ldo, int32_t dtype,
                                   void *stream) {
    const char *fn = "zs_mx4_matmul";
    constexpr int64_t MOST = (int64_t)1 << 31;
    if (m < 0 || n < 0 || k < 0 || m >= MOST || n >= MOST || k >= MOST)
        return zs_fail(ZS_EINVAL, "%s: m %lld, n %lld, k %lld out of range", fn, (long long)m, (long long)n, (long long)k);
    if (dtype < ZS_DTYPE_BF16 || dtype > ZS_DTYPE_FP32) return zs_fail(ZS_EINVAL, "%s: dtype %d", fn, dtype);
    if (ldo < n) return zs_fail(ZS_EINVAL, "%s: row stride %lld < n = %lld", fn, (long long)ldo, (long long)n);
    if (m == 0 || n == 0) {
        zs_clear_error();
        return ZS_OK;
    }
    const int size = dtype == ZS_DTYPE_FP32 ? 4 : 2;
    if (!out || reinterpret_cast<uintptr_t>(out) % size)
        return zs_fail(ZS_EINVAL, "%s: out NULL or not aligned to its elements", fn);
    const cudaStream_t s = (cudaStream_t)stream;
    if (k == 0) {
        const int64_t grid = (m * n + 255) / 256;
        zsk::mx4_zero_kernel<<<(unsigned)(grid < 4096 ? grid : 4096), 256, 0, s>>>(out, m, n, ldo, dtype == ZS_DTYPE_FP32);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
        zs_clear_error();
        return ZS_OK;
    }
    const void *four[4] = {a_codes, a_scales, b_codes, b_scales};
    for (const void *p : four)
        if (!p || (reinterpret_cast<uintptr_t>(p) & 15))
            return zs_fail(ZS_EINVAL, "%s: codes or scales NULL or not 16-byte aligned", fn);
    using namespace zsk;
    const MmPlan r = mm_plan(m, n, k);
    cudaError_t e;
    if (r.pair) {
        CUtensorMap map[4];
        if (!code_map(&map[0], a_codes, m, mx4_row_bytes(k), 128) || !code_map(&map[1], b_codes, n, mx4_row_bytes(k), 128) ||
            !scale_map(&map[2], a_scales, m, k, 1) || !scale_map(&map[3], b_scales, n, k, 2))
            return zs_fail(ZS_ECUDA, "%s: cuTensorMapEncodeTiled failed", fn);
        PairArgs a;
        a.out = out;
        a.ldo = ldo;
        a.m = (int32_t)m;
        a.n = (int32_t)n;
        a.k_tiles = (int32_t)((k + 255) / 256);
        a.p_tiles = (int32_t)r.p_tiles;
        a.tiles = (int32_t)(r.p_tiles * r.q_tiles);
        a.dtype = dtype;
        a.vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ldo * size % 16 == 0;
        a.give_up = zsl_test_give_up();
        e = r.stages == 6 ? pair_launch<6>(map, a, s) : pair_launch<5>(map, a, s);
        if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
        zs_clear_error();
        return ZS_OK;
    }
    if (r.p_tiles * r.q_tiles * r.split > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: too many tiles", fn);
    const int64_t np = r.flip ? n : m, nq = r.flip ? m : n;
    MmArgs a;
    a.p_scales = static_cast<const uint8_t *>(r.flip ? b_scales : a_scales);
    a.q_scales = static_cast<const uint8_t *>(r.flip ? a_scales : b_scales);
    a.out = out;
    a.ldo = ldo;
    a.np = (int32_t)np;
    a.nq = (int32_t)nq;
    a.k_tiles = (int32_t)((k + 255) / 256);
    a.atoms = (int32_t)mx4_atoms(k);
    a.p_tiles = (int32_t)r.p_tiles;
    a.q_tiles = (int32_t)r.q_tiles;
    a.split = r.split;
    a.stages = r.stages;
    a.dtype = dtype;
    a.vec = reinterpret_cast<uintptr_t>(out) % (4 * size) == 0 && ldo % 4 == 0;
    a.give_up = zsl_test_give_up();
    CUtensorMap mp, mq;
    if (!code_map(&mp, r.flip ? b_codes : a_codes, np, mx4_row_bytes(k), MM_P) ||
        !code_map(&mq, r.flip ? a_codes : b_codes, nq, mx4_row_bytes(k), r.bn))
        return zs_fail(ZS_ECUDA, "%s: cuTensorMapEncodeTiled failed", fn);
    if (r.flip)
        e = r.bn == 16 ? mm_launch<16, true>(r, mp, mq, a, s) : r.bn == 32 ? mm_launch<32, true>(r, mp, mq, a, s) : mm_launch<64, true>(r, mp, mq, a, s);
    else
        e = mm_launch<128, false>(r, mp, mq, a, s);
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

extern "C" zs_status zs_test_mx4_launch(int64_t m, int64_t n, int64_t k, zs_mx4_launch *out) {
    constexpr int64_t MOST = (int64_t)1 << 31;
    if (!out || m < 1 || n < 1 || k < 1 || m >= MOST || n >= MOST || k >= MOST)
        return zs_fail(ZS_EINVAL, "zs_test_mx4_launch: NULL result or m, n, k out of range");
    const zsk::MmPlan r = zsk::mm_plan(m, n, k);
    *out = {r.pair ? 2 : r.split, r.split, r.stages, r.smem, r.columns, 0};
    zs_clear_error();
    return ZS_OK;
}
