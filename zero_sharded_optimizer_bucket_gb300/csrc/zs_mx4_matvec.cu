// A few tokens of 16 or 32 bits through a weight held in 4 bits
// (zs_mx4_matvec): out[m][n] = sum over k of x[m][k] w[n][k].
//
// The weight's 0.53 bytes an element are read once, and each is decoded once
// for 8, 16 or 32 tokens.  Products go to the tensor cores in fp16 (mma
// m16n8k16): a code is exact there, and so are a token's values, 32 of them
// (those that meet a group of the weight) times a power of two of their own;
// fp32 ones are two numbers of 11 bits each.  The 32 products' sum in fp32 is
// multiplied by both powers of two and added to the row's.
//
// 1 x 4096 x 14336 bf16 takes 12 us where the weight's bytes at a copy's rate are
// 4.6: about 4.5 go before the first unit and behind the last one (launch, first
// loads, sums of warps and cluster), and in between latency bounds the six units or
// so that a warp has (issue slots 40 %, tensor pipe 16 %, DRAM 26 % busy).  32 x
// 14336 x 4096 fp16 takes 18 us, of which the products alone are 6.4 (mma m16n8k16:
// 2.07 cycles of an SM each; tensor pipe 36 % busy), the rest what a group's scale
// and its tokens' way cost 12 warps an SM.  Every 32 tokens read and decode the
// weight again: 128 x 14336 x 4096 bf16 takes 70 us.
// (tcgen05's 16-bit kinds would take the decoded weight from shared or tensor
// memory, written there and read again at four times its bytes, in tiles of 128
// rows, of which these sizes have few.  Not built.)  Codes decoded by bit
// operations and loaded as they were needed took 34 and 87 us; by the conversion
// instruction, from rings that copies fill ahead, 14 and 39; two tiles of rows a
// warp, k and rows shared out by measured costs, 12 and 18.
#include <atomic>
#include <cooperative_groups.h>
#include <type_traits>

#include "zs_launch.h"
#include "zs_mx4.cuh"

namespace zsk {

namespace cg = cooperative_groups;
typedef unsigned long long f2;

struct MatvecArgs {
    const void *x;
    const uint8_t *codes, *scales;
    void *out;
    int64_t m, n, k, ldx, ldo;
    int32_t out_kind;
    int32_t warps_n, warps_k;        // warps of a CTA along the rows and along k
    int32_t depth;                   // units of a warp's ring
    int32_t units;                   // of k, of each CTA of a cluster
    int32_t stage;                   // units of k whose tokens lie in shared memory at a time
    int32_t columns;                 // of shared memory: tokens, two each for fp32
    // 2^32 over the pieces of a token's stage, a quarter of a CTA's rows, warps_k, rounded up
    uint32_t per_token, per_row, per_warp;
    bool vec_out;                    // 16-byte aligned rows of out
    bool vec;                        // rows of x are 16-byte aligned and whole pieces of 8 values
};

// 16 warps at 128 registers, or for 32 columns, whose sums take 64, 12 at 168
// (24 warps at 80 registers for 8 columns: 15.2 us for 1 x 4096 x 14336, not 11.7).
__host__ __device__ constexpr int mv_warps(int nb) { return nb == 4 ? 12 : 16; }
constexpr int MV_PIECES = 5;         // pieces of 8 values of x that a thread holds for the next stage
// A warp's unit is 32 rows by 128 of k, one atom of scales wide: each token's
// values, once loaded, meet two tiles of 16 rows.
constexpr int MV_TILES = 2, MV_ROWS = 16 * MV_TILES, MV_SPAN = 128;
// bytes from row to row of a unit's codes: 16 past them, so that 8 rows' words meet 32 banks
constexpr int MV_ROW = MV_SPAN / 2 + 16, MV_UNIT = MV_ROWS * MV_ROW + 4 * MV_ROWS;
// NB: tiles of 8 columns of tokens
// units of a warp's ring: as many as the tokens leave room for
constexpr int MV_LEAST_DEPTH = 2, MV_MOST_DEPTH = 4;
__host__ __device__ constexpr int mv_ring_bytes(int nb, int depth) { return mv_warps(nb) * depth * MV_UNIT; }
__host__ __device__ constexpr int mv_most_stage(int nb) { return nb == 1 ? 16 : nb == 2 ? 10 : 3; }
// columns are 64 bytes past a multiple of 128 apart: two of them side by side in the banks
__host__ __device__ constexpr int mv_pitch(int stage) { return stage * MV_SPAN + 32; }      // halves
// a stage's powers of two, one a group and column, and its columns
__host__ __device__ constexpr int mv_powers(int columns) { return (columns + 1) & ~1; }
__host__ __device__ constexpr int mv_stage_bytes(int stage, int columns) {
    return ((16 * stage * mv_powers(columns) + 15) & ~15) + columns * mv_pitch(stage) * 2;
}

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

// 16 or 4 bytes to shared memory
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" : : "r"(to), "l"(from) : "memory");
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
__device__ __forceinline__ Piece<KIND> mv_load(const void *x, int64_t at) {
    if constexpr (KIND == ZS_DTYPE_FP32) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + at);
        return {q[0], q[1]};
    } else {
        return {*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at)};
    }
}
// n of them, at any address
template <int KIND>
__device__ __noinline__ Piece<KIND> mv_load_some(const void *x, int64_t at, int n) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i >= n ? 0u : KIND == ZS_DTYPE_FP32 ? static_cast<const uint32_t *>(x)[at + i] : (uint32_t)static_cast<const uint16_t *>(x)[at + i];
    if constexpr (KIND == ZS_DTYPE_FP32) return {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])};
    else return {pack8(v)};
}
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A CTA takes 32 * warps_n rows of the weight and, of a cluster of
// S, one S-th of k, whose units its warps_k warps of the same rows take in
// turn.  A warp copies its units' codes and scales ahead into a ring of its
// own; all share the tokens, which lie in shared memory as halves: of all the
// CTA's k where there is room, otherwise for a stage of units at a time while
// the next stage's are on their way to registers.  Sums go from the warps to
// the CTA and from there to the cluster in a fixed order.
template <int KIND, int NB>
__global__ void __launch_bounds__(32 * mv_warps(NB))
mx4_matvec_kernel(MatvecArgs a) {
    constexpr bool HALVES = KIND == ZS_DTYPE_FP16;
    constexpr int PER = KIND == ZS_DTYPE_FP32 ? 2 : 1, TOKENS = 8 * NB / PER, TILES = MV_TILES, UNIT = MV_UNIT;
    constexpr int THREADS = 32 * mv_warps(NB);
    constexpr int GROUPS = MV_SPAN / MX4_GROUP, SPAN = MV_SPAN, ROW = MV_ROW;
    constexpr int HOLD = KIND == ZS_DTYPE_FP32 ? (MV_PIECES + 1) / 2 : MV_PIECES;
    extern __shared__ __align__(16) uint8_t raw[];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = lane >> 2, t = lane & 3;
    const int wn = a.warps_k == 1 ? warp : (int)__umulhi((uint32_t)warp, a.per_warp), wk = warp - wn * a.warps_k;
    uint32_t block;                                                       // of rows: a cluster's
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(block));
    const int64_t row0 = ((int64_t)block * a.warps_n + wn) * MV_ROWS, token0 = (int64_t)blockIdx.y * TOKENS;
    const int tokens = (int)min((int64_t)TOKENS, a.m - token0);
    const int64_t row_bytes = mx4_row_bytes(a.k), atoms = mx4_atoms(a.k);
    const int first = rank * a.units, last = min(first + a.units, (int)((mx4_groups(a.k) + GROUPS - 1) / GROUPS));
    const int stage = a.stage, pitch = mv_pitch(stage);
    const int depth = a.depth, around = depth * UNIT;
    uint8_t *area = raw + mv_ring_bytes(NB, depth);                              // one or two stages of tokens
    const int powers = mv_powers(a.columns), area_bytes = mv_stage_bytes(stage, a.columns), xs_at = area_bytes - a.columns * pitch * 2;
    pdl_wait();
    pdl_trigger();
    // A warp's units: every warps_k-th (a stage is a multiple of them).  Rows
    // behind the last one are copies of it, whose sums nobody takes; groups
    // behind a row's last are copies of that one, and meet zeros of x and the
    // scales' padding, which is 2^-127.
    const uint32_t ring = smem_u32(raw) + warp * around, to_codes = ring + q * ROW + 16 * t;     // of the copies: 4 lanes a row
    int ahead = first + wk, slot = 0;                                     // the next unit to be copied, and its place
    const uint8_t *codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[i] = a.codes + min(row0 + q + 8 * i, a.n - 1) * row_bytes;
    const int64_t scale_row = min(row0 + lane, a.n - 1);
    const uint8_t *scales = a.scales + ((scale_row >> 7) * atoms + ahead) * MX4_ATOM + mx4_in_atom((int)(scale_row & 127), 0);
    const bool works = wn < a.warps_n && row0 < a.n;
    const int end = works ? last : 0;
    auto copy = [&] {
        if (ahead < end) {
            const uint32_t at = min(SPAN / 2 * (uint32_t)ahead + 16u * t, (uint32_t)row_bytes - 16u);
#pragma unroll
            for (int i = 0; i < 4; ++i) copy16(to_codes + slot + 8 * i * ROW, codes[i] + at);
            copy4(ring + slot + MV_ROWS * ROW + 4 * lane, scales);
        }
        ahead += a.warps_k;
        scales += MX4_ATOM * a.warps_k;
        slot = slot + UNIT == around ? 0 : slot + UNIT;
        asm volatile("cp.async.commit_group;" : : : "memory");
    };
    for (int u = 0; u < depth - 1; ++u) copy();
    Piece<KIND> held[HOLD];
    const int pieces = SPAN / 8 * stage;                                  // of a token
    // pieces j0, j0 + 1, .. of this thread in the stage from unit u0 on
    auto load = [&](int u0, int j0) {
        const int left = (int)min((int64_t)0x7FFFFFFF, a.k - (int64_t)u0 * SPAN);      // of k from there on
        const int64_t from = token0 * a.ldx + (int64_t)u0 * SPAN;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            if (THREADS * (j0 + j) >= tokens * pieces) break;
            const int p = (int)threadIdx.x + THREADS * (j0 + j), token = (int)__umulhi((uint32_t)p, a.per_token), at = 8 * (p - token * pieces);
            held[j] = {};
            if (token >= tokens || at >= left) continue;
            if (a.vec) held[j] = mv_load<KIND>(a.x, from + token * a.ldx + at);
            else held[j] = mv_load_some<KIND>(a.x, from + token * a.ldx + at, left - at);
        }
    };
    auto put = [&](int buffer, int j0) {
        float *fe = reinterpret_cast<float *>(area + buffer * area_bytes);
        uint8_t *xs = area + buffer * area_bytes + xs_at;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            if (THREADS * (j0 + j) >= tokens * pieces) break;
            const int p = (int)threadIdx.x + THREADS * (j0 + j), token = (int)__umulhi((uint32_t)p, a.per_token), at = p - token * pieces;
            uint8_t *to = xs + PER * token * pitch * 2 + 16 * at;
            if constexpr (HALVES) {
                if (token < tokens) *reinterpret_cast<uint4 *>(to) = held[j].a;
            } else {
                // the exponent of the largest of 4 lanes' values, bits of the
                // magnitude; infinities and NaN, which are rare, do not count
                float v[8];
                uint32_t top;
                if constexpr (KIND == ZS_DTYPE_FP32) {
                    const uint32_t u[8] = {held[j].a.x, held[j].a.y, held[j].a.z, held[j].a.w, held[j].b.x, held[j].b.y, held[j].b.z, held[j].b.w};
                    top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[i] = __uint_as_float(u[i]);
                        top = max(top, u[i] & 0x7FFFFFFFu);
                    }
                } else {
                    const uint32_t u[4] = {held[j].a.x, held[j].a.y, held[j].a.z, held[j].a.w};
                    uint32_t two = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] = __uint_as_float(u[i] << 16);
                        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                        two = __vmaxu2(two, u[i] & 0x7FFF7FFFu);
                    }
                    top = max(two << 16, two & 0xFFFF0000u);
                }
                if (__any_sync(0xFFFFFFFFu, top >= 0x7F800000u)) {
                    top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
                        top = max(top, b < 0x7F800000u ? b : 0u);
                    }
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
                    *reinterpret_cast<uint4 *>(to) = make_uint4(h[0], h[1], h[2], h[3]);
                    if constexpr (PER == 2) {                             // what 11 bits left; nothing of an infinity or NaN
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 w = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                            const float l0 = __fmul_rn(__fsub_rn(__fmul_rn(v[2 * i], f), w.x), 2048.0f), l1 = __fmul_rn(__fsub_rn(__fmul_rn(v[2 * i + 1], f), w.y), 2048.0f);
                            h[i] = half_pair(fabsf(l0) < 65504.0f ? l0 : 0.0f, fabsf(l1) < 65504.0f ? l1 : 0.0f);
                        }
                        *reinterpret_cast<uint4 *>(to + pitch * 2) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    if ((lane & 3) == 0) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) fe[(at >> 2) * powers + PER * token + i] = mv_power(e - 14 - 11 * i);
                    }
                }
            }
        }
    };
    if (HALVES && a.vec) {                                                // as they are: copied
        const int left = (int)min((int64_t)0x7FFFFFFF, a.k - (int64_t)first * SPAN);
        const uint16_t *from = static_cast<const uint16_t *>(a.x) + token0 * a.ldx + (int64_t)first * SPAN;
        // each cluster begins elsewhere: all of them read the same lines
        const int total = tokens * pieces, turn = (int)(block * (uint32_t)THREADS % (uint32_t)total);
        for (int i = threadIdx.x; i < total; i += THREADS) {
            const int p = i + turn < total ? i + turn : i + turn - total;
            const int token = (int)__umulhi((uint32_t)p, a.per_token), at = p - token * pieces;
            uint8_t *to = area + xs_at + token * pitch * 2 + 16 * at;
            if (8 * at < left) copy16(smem_u32(to), from + token * a.ldx + 8 * at);
            else *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("cp.async.wait_all;" : : : "memory");
    } else {
        for (int j0 = 0; THREADS * j0 < tokens * pieces; j0 += HOLD) {
            load(first, j0);
            put(0, j0);
        }
    }
    __syncthreads();
    f2 acc[TILES][NB][2];                                                 // pairs of neighbouring columns: rows q and q + 8
#pragma unroll
    for (int r = 0; r < TILES; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[r][b][0] = acc[r][b][1] = 0;
    // a lane's columns of tokens; where there is none another one, whose sums nobody takes
    uint32_t column[NB], power[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        column[b] = min(8 * b + q, a.columns - 1) * pitch * 2 + 16 * t;
        power[b] = 4 * min(8 * b + 2 * t, powers - 2);
    }
    const uint8_t *mine = raw + warp * around + q * ROW + 4 * t;  // of a unit's codes
    const uint8_t *mine_s = raw + warp * around + MV_ROWS * ROW + 4 * q;
    int place = 0;
    for (int u0 = first, s = 0; u0 < last; u0 += stage, ++s) {
        if (u0 + stage < last) load(u0 + stage, 0);
        const uint8_t *fe = area + (s & 1) * area_bytes, *xs = fe + xs_at;
        for (int u = wk; u < stage; u += a.warps_k) {                     // in the stage
            copy();
            if (depth == 4) asm volatile("cp.async.wait_group 3;" : : : "memory");
            else if (depth == 3) asm volatile("cp.async.wait_group 2;" : : : "memory");
            else asm volatile("cp.async.wait_group 1;" : : : "memory");
            __syncwarp();
            if (u0 + u < end) {
                float fs[TILES][2][4];
#pragma unroll
                for (int r = 0; r < TILES; ++r) {
                    scales4(*reinterpret_cast<const uint32_t *>(mine_s + place + 64 * r), fs[r][0]);
                    scales4(*reinterpret_cast<const uint32_t *>(mine_s + place + 64 * r + 32), fs[r][1]);
                }
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    uint32_t lo[TILES][4], hi[TILES][4];
#pragma unroll
                    for (int r = 0; r < TILES; ++r) {
                        uint32_t pa[4], pb[4];
                        code_pairs(*reinterpret_cast<const uint32_t *>(mine + place + 16 * r * ROW + 16 * g), pa);
                        code_pairs(*reinterpret_cast<const uint32_t *>(mine + place + (16 * r + 8) * ROW + 16 * g), pb);
                        lo[r][0] = pa[0]; lo[r][1] = pb[0]; lo[r][2] = pa[1]; lo[r][3] = pb[1];
                        hi[r][0] = pa[2]; hi[r][1] = pb[2]; hi[r][2] = pa[3]; hi[r][3] = pb[3];
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(xs + column[b] + 2 * (u * SPAN + 32 * g));
                        f2 f = 0;
                        if (!HALVES) f = *reinterpret_cast<const f2 *>(fe + power[b] + 4 * (GROUPS * u + g) * powers);
#pragma unroll
                        for (int r = 0; r < TILES; ++r) {
                            float d[4];
                            mma_group(d, lo[r], hi[r], v);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                f2 two = f2pack(d[2 * j], d[2 * j + 1]);
                                const f2 scale = f2pack(fs[r][j][g], fs[r][j][g]);
                                if (!HALVES) asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(two) : "l"(f));
                                asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[r][b][j]) : "l"(two), "l"(scale));
                            }
                        }
                    }
                }
            }
            place = place + UNIT == around ? 0 : place + UNIT;
            __syncwarp();                                                 // the unit's place may be filled again
        }
        if (u0 + stage < last) put((s + 1) & 1, 0);
        __syncthreads();
    }
    asm volatile("cp.async.wait_all;" : : : "memory");
    __syncthreads();
    // The warps' sums: [warp][column][rows of a warp], 36 apart so that a store's
    // lanes meet 32 banks; then four rows a thread.
    constexpr int APART = MV_ROWS + 4;
    float *red = reinterpret_cast<float *>(raw);
    float4 *share = reinterpret_cast<float4 *>(area);
#pragma unroll
    for (int r = 0; r < TILES; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float *to = red + (warp * 8 * NB + 8 * b + 2 * t) * APART + 16 * r + q + 8 * j;
                f2unpack(acc[r][b][j], to[0], to[APART]);
            }
    __syncthreads();
    const int rows4 = MV_ROWS / 4 * a.warps_n, values4 = tokens * rows4;
    const int64_t block0 = (int64_t)block * (4 * rows4);
    auto add = [](float4 x, float4 y) { return make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w)); };
    auto write = [&](int token, int r, float4 v) {
        const int64_t o = block0 + 4 * r, at = (token0 + token) * a.ldo + o;
        const float s[4] = {v.x, v.y, v.z, v.w};
        const bool all = a.vec_out && o + 4 <= a.n;
        if (a.out_kind == ZS_DTYPE_FP32) {
            float *to = static_cast<float *>(a.out) + at;
            if (all) *reinterpret_cast<float4 *>(to) = v;
            else
                for (int j = 0; j < 4; ++j) if (o + j < a.n) to[j] = s[j];
            return;
        }
        uint16_t *to = static_cast<uint16_t *>(a.out) + at;
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = a.out_kind == ZS_DTYPE_FP16 ? FP16T::from_f32(s[j]) : BF16T::from_f32(s[j]);
        if (all) *reinterpret_cast<uint2 *>(to) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        else
            for (int j = 0; j < 4; ++j) if (o + j < a.n) to[j] = (uint16_t)h[j];
    };
    for (int i = threadIdx.x; i < values4; i += THREADS) {
        const int token = (int)__umulhi((uint32_t)i, a.per_row), r = i - token * rows4;
        const float *from = red + ((r >> 3) * a.warps_k * 8 * NB + PER * token) * APART + 4 * (r & 7);
        float4 s[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) s[p] = *reinterpret_cast<const float4 *>(from + p * APART);
#pragma unroll 4
        for (int w = 1; w < a.warps_k; ++w)
#pragma unroll
            for (int p = 0; p < PER; ++p) s[p] = add(s[p], *reinterpret_cast<const float4 *>(from + (w * 8 * NB + p) * APART));
        const float4 v = PER == 2 ? add(s[0], s[PER - 1]) : s[0];
        if (ranks == 1) write(token, r, v);
        else share[i] = v;
    }
    if (ranks == 1) return;
    cluster.sync();
    for (int i = rank * THREADS + threadIdx.x; i < values4; i += THREADS * ranks) {
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r >= ranks) break;
            v[r] = cluster.map_shared_rank(share, r)[i];
        }
#pragma unroll
        for (int r = 1; r < 8; ++r) {
            if (r >= ranks) break;
            v[0] = add(v[0], v[r]);
        }
        const int token = (int)__umulhi((uint32_t)i, a.per_row);
        write(token, i - token * rows4, v[0]);
    }
    cluster.sync();                  // the others may still read this CTA's sums
}

struct MvLaunch {
    int tokens, split, ty, shared_bytes;
    int64_t grid;
};

// The fields of a that follow from its sizes, and the launch's.
template <int KIND, int NB>
static cudaError_t matvec_plan(MatvecArgs &a, MvLaunch &l) {
    constexpr int PER = KIND == ZS_DTYPE_FP32 ? 2 : 1, TOKENS = 8 * NB / PER;
    constexpr int ROOM = 227 * 1024 - mv_ring_bytes(NB, MV_LEAST_DEPTH), THREADS = 32 * mv_warps(NB);      // of tokens
    static_assert(2 * mv_stage_bytes(mv_most_stage(NB), 8 * NB) <= ROOM, "shared memory");
    static_assert(8 * NB * 16 * mv_most_stage(NB) <= MV_PIECES * THREADS, "pieces");
    static std::atomic<int> seats[64][9];        // CTAs in clusters of S that the device has room for at once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!seats[dev][8].load(std::memory_order_acquire)) {
        cudaLaunchConfig_t cfg = {};
        cfg.blockDim = dim3(THREADS);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        e = cudaFuncSetAttribute(mx4_matvec_kernel<KIND, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        for (int sp = 1; sp <= 8 && e == cudaSuccess; ++sp) {
            int clusters = 0;
            attr.val.clusterDim.x = (unsigned)sp;
            cfg.gridDim = dim3((unsigned)sp);
            cfg.dynamicSmemBytes = 227 * 1024;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&clusters, mx4_matvec_kernel<KIND, NB>, &cfg);
            seats[dev][sp].store(clusters > 0 ? clusters * sp : sp, std::memory_order_release);
        }
        if (e != cudaSuccess) return e;
    }
    const int ty = (int)((a.m + TOKENS - 1) / TOKENS), tiles = (int)((a.n + MV_ROWS - 1) / MV_ROWS), units = (int)((mx4_groups(a.k) + 3) / 4);
    a.columns = (int)(a.m < TOKENS ? a.m : TOKENS) * PER;
    auto fits = [&](int whole) { return whole <= 512 && mv_stage_bytes(whole, a.columns) <= ROOM; };
    // How warps and CTAs share rows and k, by the time that an SM takes, in ns as
    // measured (in a graph, with warps and split set by hand, and by a kernel whose
    // loop over the units was left out): a step (a unit of each warp) 54, 75 or 130
    // a warp, and 450 at least; a CTA's beginning and end 2000, with 280 for each 8
    // values of tokens a thread, an exchange 700.
    constexpr int STEP = NB == 1 ? 54 : NB == 2 ? 75 : 130, MOST_WARPS = mv_warps(NB);
    int64_t best = -1;
    int split = 1;
    for (const int wk : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (wk > MOST_WARPS || (wk > 1 && wk > units)) break;
        const int most_n = tiles < MOST_WARPS / wk ? tiles : MOST_WARPS / wk, blocks = (tiles + most_n - 1) / most_n, wn = (tiles + blocks - 1) / blocks;
        for (const int sp : {1, 2, 3, 4, 6, 8}) {
            if (sp > 1 && units < sp * wk) break;
            const int slice = (units + sp - 1) / sp, steps = (slice + wk - 1) / wk, room = seats[dev][sp].load(std::memory_order_relaxed);
            const bool once = fits(steps * wk);
            if (slice * (sp - 1) >= units || (!once && wk > mv_most_stage(NB))) continue;
            const int step = wn * wk * STEP;
            const int64_t pieces = (int64_t)(a.columns / PER) * steps * wk * 16 / THREADS;
            const int64_t one = 2000 + (int64_t)steps * (step > 450 ? step : 450) + 280 * pieces + (once ? 0 : 500) + (sp > 1 ? 700 : 0);
            const int64_t cost = ((int64_t)blocks * ty * sp + room - 1) / room * one;
            if (best >= 0 && cost >= best) continue;
            best = cost;
            a.warps_k = wk;
            a.warps_n = wn;
            split = sp;
        }
    }
    a.units = (units + split - 1) / split;
    const int whole = (a.units + a.warps_k - 1) / a.warps_k * a.warps_k;
    const bool once = fits(whole);
    a.stage = once ? whole : mv_most_stage(NB) / a.warps_k * a.warps_k;
    // exact for the numbers below 2^16 that are divided
    a.per_token = (uint32_t)(((uint64_t)1 << 32) / (16 * a.stage) + 1);
    a.per_row = (uint32_t)(((uint64_t)1 << 32) / (MV_ROWS / 4 * a.warps_n) + 1);
    a.per_warp = (uint32_t)(((uint64_t)1 << 32) / a.warps_k + 1);
    const int room = (once ? 1 : 2) * mv_stage_bytes(a.stage, a.columns);
    const int share = MV_ROWS * a.warps_n * (a.columns / PER) * 4;     // the CTA's sums, in the tokens' place
    const int left = 227 * 1024 - (room > share ? room : share);
    a.depth = left / mv_ring_bytes(NB, 1) < MV_MOST_DEPTH ? left / mv_ring_bytes(NB, 1) : MV_MOST_DEPTH;
    l = {TOKENS, split, ty, mv_ring_bytes(NB, a.depth) + (room > share ? room : share), (int64_t)((tiles + a.warps_n - 1) / a.warps_n) * split};
    return cudaSuccess;
}

template <int KIND, int NB>
static cudaError_t matvec_launch(MatvecArgs a, cudaStream_t s) {
    MvLaunch l;
    const cudaError_t e = matvec_plan<KIND, NB>(a, l);
    if (e != cudaSuccess) return e;
    if (l.grid > 0x7FFFFFFF || l.ty > 65535) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)l.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3((unsigned)l.grid, (unsigned)l.ty);
    cfg.blockDim = dim3(32 * mv_warps(NB));
    cfg.dynamicSmemBytes = l.shared_bytes;
    cfg.stream = s;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, mx4_matvec_kernel<KIND, NB>, a);
    return launched != cudaSuccess ? launched : cudaGetLastError();
}

// f with the kernel's tiles of 8 columns for m tokens
template <int KIND, class F>
static cudaError_t by_columns(int64_t m, F f) {
    const int64_t cols = m * (KIND == ZS_DTYPE_FP32 ? 2 : 1);
    if (cols <= 8) return f(std::integral_constant<int, 1>());
    if (cols <= 16) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 4>());
}
template <int KIND>
static cudaError_t matvec_of(const MatvecArgs &a, cudaStream_t s) {
    return by_columns<KIND>(a.m, [&](auto nb) { return matvec_launch<KIND, decltype(nb)::value>(a, s); });
}
template <int KIND>
static cudaError_t matvec_plan_of(MatvecArgs &a, MvLaunch &l) {
    return by_columns<KIND>(a.m, [&](auto nb) { return matvec_plan<KIND, decltype(nb)::value>(a, l); });
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
        a.vec_out = addr(out) % 16 == 0 && (m == 1 || ldo * size(out_dtype) % 16 == 0);
        a.vec = addr(x) % 16 == 0 && k % 8 == 0 && (m == 1 || ldx * size(dtype) % 16 == 0);
        e = dtype == ZS_DTYPE_FP32 ? zsk::matvec_of<ZS_DTYPE_FP32>(a, s)
          : dtype == ZS_DTYPE_FP16 ? zsk::matvec_of<ZS_DTYPE_FP16>(a, s) : zsk::matvec_of<ZS_DTYPE_BF16>(a, s);
    }
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

extern "C" zs_status zs_test_mx4_matvec_launch(int64_t m, int64_t n, int64_t k, int32_t dtype, zs_mx4_matvec_launch *out) {
    const char *fn = "zs_test_mx4_matvec_launch";
    const int64_t most = (int64_t)1 << 31;
    if (!out || m < 1 || m > ZS_MATVEC_MAX_TOKENS || n < 1 || n >= most || k < 1 || k >= most || dtype < ZS_DTYPE_BF16 || dtype > ZS_DTYPE_FP32)
        return zs_fail(ZS_EINVAL, "%s: NULL result, or m, n, k or dtype out of range", fn);
    zsk::MatvecArgs a = {};
    zsk::MvLaunch l = {};
    a.m = m; a.n = n; a.k = k;
    const cudaError_t e = dtype == ZS_DTYPE_FP32 ? zsk::matvec_plan_of<ZS_DTYPE_FP32>(a, l)
                        : dtype == ZS_DTYPE_FP16 ? zsk::matvec_plan_of<ZS_DTYPE_FP16>(a, l) : zsk::matvec_plan_of<ZS_DTYPE_BF16>(a, l);
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    *out = {l.tokens, a.warps_n, a.warps_k, l.split, a.units, a.stage, a.depth, l.shared_bytes};
    zs_clear_error();
    return ZS_OK;
}
