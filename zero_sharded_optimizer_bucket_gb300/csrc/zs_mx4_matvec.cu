// A few tokens of 16 or 32 bits through a weight held in 4 bits
// (zs_mx4_matvec): out[m][n] = sum over k of x[m][k] w[n][k].
//
// The weight's 0.53 bytes an element are read once, and each is decoded once
// for 8, 16 or 32 tokens.  Products go to the tensor cores in fp16 (mma
// m16n8k16): a code is exact there, and so are a token's values, 32 of them
// (those that meet a group of the weight) times a power of two of their own;
// fp32 ones are two numbers of 11 bits each.  The 32 products' sum in fp32 is
// multiplied by both powers of two and added to the row's.
#include <atomic>
#include <cooperative_groups.h>

#include "zs_launch.h"
#include "zs_mx4.cuh"

namespace zsk {

namespace cg = cooperative_groups;

struct MatvecArgs {
    const void *x;
    const uint8_t *codes, *scales;
    void *out;
    int64_t m, n, k, ldx, ldo;
    int32_t out_kind;
    int32_t warps_n, warps_k;        // warps of a CTA along the rows and along k
    int32_t stage;                   // chunks of k whose tokens lie in shared memory at a time
    int32_t columns;                 // of shared memory: tokens, two each for fp32
    uint32_t per_token, per_row;     // 2^32 over the pieces of a token's stage, over the rows of a CTA
    bool vec;                        // 16-byte aligned rows of x
};

constexpr int MV_THREADS = 512, MV_WARPS = MV_THREADS / 32;
constexpr int MV_CHUNK = 128;        // k of one atom of scales: 4 groups
constexpr int MV_ROW = 80;           // bytes from row to row of 64 bytes of codes: 8 rows' words meet 32 banks
constexpr int MV_PIECES = 5;         // pieces of 8 values of x that a thread holds for the next stage
// NB: tiles of 8 columns of tokens; a warp takes mv_tiles(NB) tiles of 16 rows
// (so that a token's values, once loaded, meet as many rows as registers hold),
// with MV_DEPTH chunks in flight.
__host__ __device__ constexpr int mv_tiles(int nb) { return nb == 1 ? 1 : 2; }
constexpr int MV_DEPTH = 3;
__host__ __device__ constexpr int mv_chunk_bytes(int nb) { return mv_tiles(nb) * (16 * MV_ROW + 64); }
__host__ __device__ constexpr int mv_ring_bytes(int nb) { return MV_WARPS * MV_DEPTH * mv_chunk_bytes(nb); }
__host__ __device__ constexpr int mv_most_stage(int nb) { return nb == 1 ? 16 : nb == 2 ? 10 : 5; }
// columns are 64 bytes past a multiple of 128 apart: two of them side by side in the banks
__host__ __device__ constexpr int mv_pitch(int stage) { return stage * MV_CHUNK + 32; }      // halves
// a stage's powers of two, one a group and column, and its columns
__host__ __device__ constexpr int mv_powers(int columns) { return (columns + 1) & ~1; }
__host__ __device__ constexpr int mv_stage_bytes(int stage, int columns) { return ((16 * stage * mv_powers(columns) + 15) & ~15) + columns * mv_pitch(stage) * 2; }

// the values of 8 codes as four pairs of halves
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t o[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// four scale bytes as floats (0: 2^-127, 255: NaN)
__device__ __forceinline__ void scales4(uint32_t w, float o[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    o[0] = __uint_as_float(lo << 16);
    o[1] = __uint_as_float(lo & 0xFFFF0000u);
    o[2] = __uint_as_float(hi << 16);
    o[3] = __uint_as_float(hi & 0xFFFF0000u);
}

// the products of 16 rows, 32 of k and 8 columns
__device__ __forceinline__ void mma_group(float d[4], const uint32_t lo[4], const uint32_t hi[4], const uint4 &v) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]), "r"(v.x), "r"(v.y), "f"(0.0f));
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]), "r"(v.z), "r"(v.w));
}

// 16 or 4 bytes to shared memory, zeros where there is nothing
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" : : "r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" : : "r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}

__device__ __forceinline__ float mv_power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }     // 2^e, normal

// 8 values of a token as they lie in memory
template <int KIND>
struct Piece {
    uint4 a;
};
template <>
struct Piece<ZS_DTYPE_FP32> {
    uint4 a, b;
};
template <int KIND>
__device__ __forceinline__ Piece<KIND> mv_load(const void *x, int64_t at, int n, bool vec) {
    Piece<KIND> p;
    if constexpr (KIND == ZS_DTYPE_FP32) {
        const uint32_t *q = static_cast<const uint32_t *>(x) + at;
        if (vec && n >= 8) {
            p.a = *reinterpret_cast<const uint4 *>(q);
            p.b = *reinterpret_cast<const uint4 *>(q + 4);
        } else {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? q[i] : 0u;
            p.a = make_uint4(v[0], v[1], v[2], v[3]);
            p.b = make_uint4(v[4], v[5], v[6], v[7]);
        }
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(x) + at;
        if (vec && n >= 8) {
            p.a = *reinterpret_cast<const uint4 *>(q);
        } else {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? (uint32_t)q[i] : 0u;
            p.a = pack8(v);
        }
    }
    return p;
}
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A CTA takes 16 * mv_tiles * warps_n rows of the weight and, of a cluster of
// S, one S-th of k, whose chunks its warps_k warps of the same rows take in
// turn.  A warp copies its chunks' codes and scales ahead into a ring of its
// own; all share the tokens, which lie in shared memory as halves: of all the
// CTA's k where there is room, otherwise for a stage of chunks at a time while
// the next stage's are on their way to registers.
// Sums go from the warps to the CTA and from there to the cluster in a fixed
// order.
template <int KIND, int NB>
__global__ void __launch_bounds__(MV_THREADS, NB == 1 ? 2 : 1)
mx4_matvec_kernel(MatvecArgs a) {
    constexpr bool HALVES = KIND == ZS_DTYPE_FP16;
    constexpr int PER = KIND == ZS_DTYPE_FP32 ? 2 : 1, TOKENS = 8 * NB / PER, TILES = mv_tiles(NB), DEPTH = MV_DEPTH, CHUNK = mv_chunk_bytes(NB);
    constexpr int HOLD = KIND == ZS_DTYPE_FP32 ? (MV_PIECES + 1) / 2 : MV_PIECES;
    extern __shared__ __align__(16) uint8_t raw[];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = lane >> 2, t = lane & 3;
    const int wn = warp / a.warps_k, wk = warp % a.warps_k;
    const bool works = wn < a.warps_n;
    const int64_t row0 = ((int64_t)(blockIdx.x / ranks) * a.warps_n + wn) * (16 * TILES), token0 = (int64_t)blockIdx.y * TOKENS;
    const int tokens = (int)min((int64_t)TOKENS, a.m - token0);
    const int groups = (int)mx4_groups(a.k), chunks = (groups + 3) / 4, atoms = (int)mx4_atoms(a.k);
    const int64_t row_bytes = mx4_row_bytes(a.k);
    const int first = (int)((int64_t)chunks * rank / ranks), last = (int)((int64_t)chunks * (rank + 1) / ranks);
    const int stage = a.stage, pitch = mv_pitch(stage);
    const uint32_t ring = smem_u32(raw) + warp * (DEPTH * CHUNK);
    uint8_t *area = raw + mv_ring_bytes(NB);                              // one or two stages of tokens
    const int powers = mv_powers(a.columns), area_bytes = mv_stage_bytes(stage, a.columns), xs_at = area_bytes - a.columns * pitch * 2;
    pdl_wait();
    pdl_trigger();
    // a warp's chunks: every warps_k-th (a stage is a multiple of them)
    int ahead = first + wk, slot = 0;                                     // the next chunk to be copied, and its place
    const int64_t row = row0 + q, scale_row = row0 + lane;                // of the copies: 4 lanes a row
    const uint8_t *codes = a.codes + row * row_bytes + 64 * (int64_t)ahead + 16 * t;
    const uint8_t *scales = a.scales + ((scale_row >> 7) * atoms + ahead) * MX4_ATOM + mx4_in_atom((int)(scale_row & 127), 0);
    const int codes_n = works ? (int)min((int64_t)(16 * TILES), max((int64_t)0, a.n - row0)) : 0;     // rows that there are
    auto copy = [&] {
        const uint32_t to = ring + slot * CHUNK;
        if (ahead < last && codes_n > 0) {
            const bool inside = 4 * ahead + t < groups;
#pragma unroll
            for (int i = 0; i < 2 * TILES; ++i) {
                const bool there = inside && q + 8 * i < codes_n;
                copy16(to + (8 * i + q) * MV_ROW + 16 * t, there ? codes + 8 * i * row_bytes : a.codes, there);
            }
            if (lane < 16 * TILES) copy4(to + 16 * TILES * MV_ROW + 4 * lane, lane < codes_n ? scales : a.scales, lane < codes_n);
        }
        ahead += a.warps_k;
        codes += 64 * (int64_t)a.warps_k;
        scales += (int64_t)MX4_ATOM * a.warps_k;
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
        asm volatile("cp.async.commit_group;" : : : "memory");
    };
#pragma unroll
    for (int u = 0; u < DEPTH - 1; ++u) copy();
    Piece<KIND> held[HOLD];
    const int pieces = 16 * stage;                                        // of a token
    // pieces j0, j0 + 1, .. of this thread in the stage from chunk c0 on
    auto load = [&](int c0, int j0) {
        const int64_t k0 = (int64_t)c0 * MV_CHUNK;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            if (MV_THREADS * (j0 + j) >= tokens * pieces) break;
            const int p = (int)threadIdx.x + MV_THREADS * (j0 + j), token = (int)__umulhi((uint32_t)p, a.per_token);
            const int64_t k = k0 + 8 * (p - token * pieces);
            const int n = token < tokens ? (int)max((int64_t)0, min((int64_t)8, a.k - k)) : 0;
            held[j] = mv_load<KIND>(a.x, (token0 + token) * a.ldx + k, n, a.vec);
        }
    };
    auto put = [&](int buffer, int j0) {
        float *fe = reinterpret_cast<float *>(area + buffer * area_bytes);
        uint8_t *xs = area + buffer * area_bytes + xs_at;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            if (MV_THREADS * (j0 + j) >= tokens * pieces) break;
            const int p = (int)threadIdx.x + MV_THREADS * (j0 + j), token = (int)__umulhi((uint32_t)p, a.per_token), at = p - token * pieces;
            if constexpr (HALVES) {
                if (token < tokens) *reinterpret_cast<uint4 *>(xs + token * pitch * 2 + 16 * at) = held[j].a;
            } else {
                float v[8];
                if constexpr (KIND == ZS_DTYPE_FP32) {
                    const uint32_t u[8] = {held[j].a.x, held[j].a.y, held[j].a.z, held[j].a.w, held[j].b.x, held[j].b.y, held[j].b.z, held[j].b.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = BF16T::to_f32(lane16(held[j].a, i));
                }
                uint32_t top = 0;                                         // of the finite ones
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
                    top = max(top, b < 0x7F800000u ? b : 0u);
                }
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // the largest to [2^14, 2^15), as far as the inverse is a normal number
                const int e = max((int)(top >> 23) - 127, PER == 2 ? -101 : -112);
                const float f = mv_power(14 - e);
                if (token < tokens) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = half_pair(__fmul_rn(v[2 * i], f), __fmul_rn(v[2 * i + 1], f));
                    *reinterpret_cast<uint4 *>(xs + PER * token * pitch * 2 + 16 * at) = make_uint4(h[0], h[1], h[2], h[3]);
                    if constexpr (PER == 2) {                             // what 11 bits left; nothing of an infinity or NaN
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 w = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                            const float l0 = __fmul_rn(__fsub_rn(__fmul_rn(v[2 * i], f), w.x), 2048.0f), l1 = __fmul_rn(__fsub_rn(__fmul_rn(v[2 * i + 1], f), w.y), 2048.0f);
                            h[i] = half_pair(fabsf(l0) < 65504.0f ? l0 : 0.0f, fabsf(l1) < 65504.0f ? l1 : 0.0f);
                        }
                        *reinterpret_cast<uint4 *>(xs + (PER * token + 1) * pitch * 2 + 16 * at) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    if ((lane & 3) == 0) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) fe[(at >> 2) * powers + PER * token + i] = mv_power(e - 14 - 11 * i);
                    }
                }
            }
        }
    };
    for (int j0 = 0; MV_THREADS * j0 < tokens * pieces; j0 += HOLD) {
        load(first, j0);
        put(0, j0);
    }
    __syncthreads();
    float acc[TILES][NB][4] = {};
    int place = 0;
    for (int c0 = first, s = 0; c0 < last; c0 += stage, ++s) {
        if (c0 + stage < last) load(c0 + stage, 0);
        const float *fe = reinterpret_cast<const float *>(area + (s & 1) * area_bytes);
        const uint8_t *xs = area + (s & 1) * area_bytes + xs_at;
        for (int c = wk; c < stage; c += a.warps_k) {                     // in the stage
            copy();
            asm volatile("cp.async.wait_group %0;" : : "n"(DEPTH - 1) : "memory");
            __syncwarp();
            if (codes_n > 0 && c0 + c < last) {
                const uint8_t *from = raw + warp * (DEPTH * CHUNK) + place * CHUNK;
                float fs[TILES][2][4];
#pragma unroll
                for (int r = 0; r < TILES; ++r) {
                    scales4(*reinterpret_cast<const uint32_t *>(from + 16 * TILES * MV_ROW + 4 * (16 * r + q)), fs[r][0]);
                    scales4(*reinterpret_cast<const uint32_t *>(from + 16 * TILES * MV_ROW + 4 * (16 * r + q + 8)), fs[r][1]);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t lo[TILES][4], hi[TILES][4];
#pragma unroll
                    for (int r = 0; r < TILES; ++r) {
                        uint32_t pa[4], pb[4];
                        code_pairs(*reinterpret_cast<const uint32_t *>(from + (16 * r + q) * MV_ROW + 16 * g + 4 * t), pa);
                        code_pairs(*reinterpret_cast<const uint32_t *>(from + (16 * r + q + 8) * MV_ROW + 16 * g + 4 * t), pb);
                        lo[r][0] = pa[0]; lo[r][1] = pb[0]; lo[r][2] = pa[1]; lo[r][3] = pb[1];
                        hi[r][0] = pa[2]; hi[r][1] = pb[2]; hi[r][2] = pa[3]; hi[r][3] = pb[3];
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (8 * b + q < PER * tokens) v = *reinterpret_cast<const uint4 *>(xs + (8 * b + q) * pitch * 2 + 2 * (c * MV_CHUNK + 32 * g + 8 * t));
                        float2 f = make_float2(1.0f, 1.0f);
                        if (!HALVES) f = *reinterpret_cast<const float2 *>(fe + (4 * c + g) * powers + 8 * b + 2 * t);
#pragma unroll
                        for (int r = 0; r < TILES; ++r) {
                            float d[4];
                            mma_group(d, lo[r], hi[r], v);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[r][b][j] = __fmaf_rn(HALVES ? d[j] : __fmul_rn(d[j], j & 1 ? f.y : f.x), fs[r][j >> 1][g], acc[r][b][j]);
                        }
                    }
                }
            }
            place = place + 1 == DEPTH ? 0 : place + 1;
            __syncwarp();                                                 // the chunk's place may be filled again
        }
        if (c0 + stage < last) put((s + 1) & 1, 0);
        __syncthreads();
    }
    asm volatile("cp.async.wait_all;" : : : "memory");
    __syncthreads();
    // the warps' sums: [warp][column][rows of a warp]
    constexpr int ROWS = 16 * TILES;
    float *red = reinterpret_cast<float *>(raw), *share = reinterpret_cast<float *>(area);
#pragma unroll
    for (int r = 0; r < TILES; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) red[(warp * 8 * NB + 8 * b + 2 * t + (j & 1)) * ROWS + 16 * r + q + 8 * (j >> 1)] = acc[r][b][j];
    __syncthreads();
    const int rows = ROWS * a.warps_n;
    for (int i = threadIdx.x; i < tokens * rows; i += MV_THREADS) {
        const int token = (int)__umulhi((uint32_t)i, a.per_row), r = i - token * rows;
        float s[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            s[p] = 0.0f;
            for (int w = 0; w < a.warps_k; ++w)
                s[p] = __fadd_rn(s[p], red[((r / ROWS * a.warps_k + w) * 8 * NB + PER * token + p) * ROWS + r % ROWS]);
        }
        share[i] = PER == 2 ? __fadd_rn(s[0], s[PER - 1]) : s[0];
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    const int64_t block0 = (int64_t)(blockIdx.x / ranks) * rows;
    for (int i = rank * MV_THREADS + threadIdx.x; i < tokens * rows; i += MV_THREADS * ranks) {
        float s = share[i];
        if (ranks > 1) {
            s = 0.0f;
            for (int r = 0; r < ranks; ++r) s = __fadd_rn(s, cluster.map_shared_rank(share, r)[i]);
        }
        const int token = (int)__umulhi((uint32_t)i, a.per_row);
        const int64_t o = block0 + i - token * rows, at = (token0 + token) * a.ldo + o;
        if (o >= a.n) continue;
        if (a.out_kind == ZS_DTYPE_FP32) static_cast<float *>(a.out)[at] = s;
        else static_cast<uint16_t *>(a.out)[at] = (uint16_t)(a.out_kind == ZS_DTYPE_FP16 ? FP16T::from_f32(s) : BF16T::from_f32(s));
    }
    if (ranks > 1) cluster.sync();   // the others may still read this CTA's sums
}

template <int KIND, int NB>
static cudaError_t matvec_launch(MatvecArgs a, cudaStream_t s) {
    static std::atomic<bool> set[64];
    constexpr int PER = KIND == ZS_DTYPE_FP32 ? 2 : 1, TOKENS = 8 * NB / PER;
    constexpr int ROOM = 227 * 1024 - mv_ring_bytes(NB);                 // of tokens, a CTA alone on its SM
    static_assert(2 * mv_stage_bytes(mv_most_stage(NB), 8 * NB) <= ROOM, "shared memory");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(mx4_matvec_kernel<KIND, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    const int64_t ty = (a.m + TOKENS - 1) / TOKENS, tiles = (a.n + 16 * mv_tiles(NB) - 1) / (16 * mv_tiles(NB));
    const int64_t chunks = (mx4_groups(a.k) + 3) / 4;
    // How warps and CTAs share rows and k.  In units of about 100 cycles: a step
    // of an SM's 16 warps 5 where instructions bound it, and 2 of latency; a
    // CTA's beginning and end 15 (tokens to halves, the sums), an exchange 4.
    int64_t best = -1;
    int split = 1;
    for (int wk = 1; wk <= mv_most_stage(NB); ++wk) {
        if (wk > 1 && wk > chunks) break;
        const int64_t wn = tiles < MV_WARPS / wk ? tiles : MV_WARPS / wk, blocks = (tiles + wn - 1) / wn * ty;
        for (int sp = 1; sp <= 8 && (sp == 1 || chunks >= (int64_t)sp * wk); ++sp) {
            const int64_t steps = ((chunks + sp - 1) / sp + wk - 1) / wk, cost = (blocks * sp + 151) / 152 * (5 * steps + 15) + 2 * steps + (sp > 1 ? 4 : 0);
            if (best >= 0 && cost >= best) continue;
            best = cost;
            a.warps_k = wk;
            a.warps_n = (int)wn;
            split = sp;
        }
    }
    a.columns = (int)(a.m < TOKENS ? a.m : TOKENS) * PER;
    const int64_t whole = ((chunks + split - 1) / split + a.warps_k - 1) / a.warps_k * a.warps_k;
    const bool fits = whole <= 1024 && mv_stage_bytes((int)whole, a.columns) <= (NB == 1 ? 113 * 1024 - mv_ring_bytes(NB) : ROOM);     // two CTAs an SM, one
    a.stage = fits ? (int)whole : mv_most_stage(NB) / a.warps_k * a.warps_k;
    // exact for the numbers below 2^16 that are divided
    a.per_token = (uint32_t)(((uint64_t)1 << 32) / (16 * a.stage) + 1);
    a.per_row = (uint32_t)(((uint64_t)1 << 32) / (16 * mv_tiles(NB) * a.warps_n) + 1);
    const int64_t grid = (tiles + a.warps_n - 1) / a.warps_n * split;
    if (grid > 0x7FFFFFFF || ty > 65535) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)ty);
    cfg.blockDim = dim3(MV_THREADS);
    cfg.dynamicSmemBytes = mv_ring_bytes(NB) + (fits ? 1 : 2) * mv_stage_bytes(a.stage, a.columns);
    const int share = 16 * mv_tiles(NB) * a.warps_n * (a.columns / PER) * 4;     // the CTA's sums, in the tokens' place
    if ((int)cfg.dynamicSmemBytes < mv_ring_bytes(NB) + share) cfg.dynamicSmemBytes = mv_ring_bytes(NB) + share;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, mx4_matvec_kernel<KIND, NB>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int KIND>
static cudaError_t matvec_of(const MatvecArgs &a, cudaStream_t s) {
    const int64_t cols = a.m * (KIND == ZS_DTYPE_FP32 ? 2 : 1);
    if (cols <= 8) return matvec_launch<KIND, 1>(a, s);
    if (cols <= 16) return matvec_launch<KIND, 2>(a, s);
    return matvec_launch<KIND, 4>(a, s);
}

}  // namespace zsk

extern "C" zs_status zs_mx4_matvec(int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, int32_t dtype, const void *w_codes,
                                   const void *w_scales, void *out, int64_t ldo, int32_t out_dtype, void *stream) {
    const char *fn = "zs_mx4_matvec";
    auto addr = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    auto size = [](int32_t t) { return t == ZS_DTYPE_FP32 ? 4u : 2u; };
    const int64_t most = (int64_t)1 << 31;
    if (m < 0 || n < 0 || k < 0 || n >= most || k >= most) return zs_fail(ZS_EINVAL, "%s: %lld x %lld x %lld out of range", fn, (long long)m, (long long)n, (long long)k);
    if (m > ZS_MATVEC_MAX_TOKENS) return zs_fail(ZS_EINVAL, "%s: %lld tokens, %d at most", fn, (long long)m, ZS_MATVEC_MAX_TOKENS);
    if (dtype < ZS_DTYPE_BF16 || dtype > ZS_DTYPE_FP32 || out_dtype < ZS_DTYPE_BF16 || out_dtype > ZS_DTYPE_FP32)
        return zs_fail(ZS_EINVAL, "%s: dtype %d, out_dtype %d", fn, dtype, out_dtype);
    if (ldx < k || ldo < n) return zs_fail(ZS_EINVAL, "%s: row stride %lld < %lld or %lld < %lld", fn, (long long)ldx, (long long)k, (long long)ldo, (long long)n);
    if (m > 0 && n > 0 && k > 0) {
        if (!x || addr(x) % size(dtype)) return zs_fail(ZS_EINVAL, "%s: x NULL or not aligned to its elements", fn);
        if (!w_codes || !w_scales || addr(w_codes) % 16 || addr(w_scales) % 16)
            return zs_fail(ZS_EINVAL, "%s: weight: codes or scales NULL or not 16-byte aligned", fn);
    }
    if (m > 0 && n > 0 && (!out || addr(out) % size(out_dtype))) return zs_fail(ZS_EINVAL, "%s: out NULL or not aligned to its elements", fn);
    cudaError_t e = cudaSuccess;
    const cudaStream_t s = (cudaStream_t)stream;
    if (m > 0 && n > 0 && k == 0) {
        e = cudaMemset2DAsync(out, (size_t)(ldo * size(out_dtype)), 0, (size_t)(n * size(out_dtype)), (size_t)m, s);
    } else if (m > 0 && n > 0) {
        zsk::MatvecArgs a;
        a.x = x; a.codes = static_cast<const uint8_t *>(w_codes); a.scales = static_cast<const uint8_t *>(w_scales); a.out = out;
        a.m = m; a.n = n; a.k = k; a.ldx = ldx; a.ldo = ldo; a.out_kind = out_dtype;
        a.vec = addr(x) % 16 == 0 && (m == 1 || ldx * size(dtype) % 16 == 0);
        e = dtype == ZS_DTYPE_FP32 ? zsk::matvec_of<ZS_DTYPE_FP32>(a, s)
          : dtype == ZS_DTYPE_FP16 ? zsk::matvec_of<ZS_DTYPE_FP16>(a, s) : zsk::matvec_of<ZS_DTYPE_BF16>(a, s);
    }
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}
