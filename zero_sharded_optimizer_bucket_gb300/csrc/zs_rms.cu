// Root-mean-square norm in front of a linear layer, with the residual's
// addition, its result whole and / or held in 4 bits along its rows and its
// columns, and its backward pass (zs_rms_norm, zs_rms_norm_backward).
//
// Forward, a row of `cols` values:
//   h = x + residual;  sum = rne(h);  rstd = 1 / sqrt(mean(h h) + eps)
//   y = (h rstd) w, rounded to the matrix's type
// Backward, with g = w dy and x the norm's input:
//   c = rstd^2 mean(g x);  dx = (g - x c) rstd + residual
//   dw = sum over rows of dy (x rstd)
// Results go straight to 4 bits, whose borders lie densely: a unit in the last
// place of rstd moves values across them.  So the sums over a row are made as
// float32 pairs, good to about 2^-44, and rstd is the float32 nearest to the
// formula's value but where that lies within 2^-40 of the middle of two.
//
// A result held along its columns needs 32 rows at a time, which no SM holds
// whole: a cluster shares them out by columns and exchanges the rows' sums
// through distributed shared memory.
#include <atomic>
#include <cooperative_groups.h>

#include "zs_launch.h"
#include "zs_mx4.cuh"

namespace zsk {

namespace cg = cooperative_groups;
typedef unsigned long long f2;

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// ------------------------------------------------------ 8 values a lane --

struct RowF32 {
    static constexpr int SIZE = 4;
    struct Raw { uint4 a, b; };
    static __device__ __forceinline__ Raw load(const void *p, int64_t at) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at);
        return {q[0], q[1]};
    }
    static __device__ __forceinline__ Raw some(const void *p, int64_t at, int n) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? static_cast<const uint32_t *>(p)[at + i] : 0u;
        return {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])};
    }
    static __device__ __forceinline__ void floats(const Raw &r, float o[8]) {
        const uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ Raw rounded(const float o[8]) {
        return {make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])),
                make_uint4(__float_as_uint(o[4]), __float_as_uint(o[5]), __float_as_uint(o[6]), __float_as_uint(o[7]))};
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, int n, bool vec, const Raw &r) {
        if (vec && n == 8) {
            uint4 *q = reinterpret_cast<uint4 *>(static_cast<float *>(p) + at);
            q[0] = r.a;
            q[1] = r.b;
            return;
        }
        const uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) if (i < n) static_cast<uint32_t *>(p)[at + i] = v[i];
    }
};
template <class T, bool FP16>
struct Row16 {
    static constexpr int SIZE = 2;
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw load(const void *p, int64_t at) {
        return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
    }
    static __device__ __forceinline__ Raw some(const void *p, int64_t at, int n) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? (uint32_t)static_cast<const uint16_t *>(p)[at + i] : 0u;
        return pack8(v);
    }
    static __device__ __forceinline__ void floats(const Raw &r, float o[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = T::to_f32(lane16(r, i));
    }
    static __device__ __forceinline__ Raw rounded(const float o[8]) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (FP16) {
                const __half2 h = __floats2half2_rn(o[2 * i], o[2 * i + 1]);
                r[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                r[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, int n, bool vec, const Raw &r) {
        uint16_t *q = static_cast<uint16_t *>(p) + at;
        if (vec && n == 8) {
            *reinterpret_cast<uint4 *>(q) = r;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) if (i < n) q[i] = (uint16_t)lane16(r, i);
    }
};
typedef Row16<BF16T, false> RowBF16;
typedef Row16<FP16T, true> RowFP16;

template <class R>
__device__ __forceinline__ typename R::Raw fetch8(const void *p, int64_t at, int n, bool vec) {
    return vec && n == 8 ? R::load(p, at) : R::some(p, at, n);
}

// n of 8 weights of any type
__device__ __forceinline__ void weights8(const void *w, int kind, int64_t at, int n, bool vec, float o[8]) {
    if (kind == ZS_DTYPE_FP32) RowF32::floats(fetch8<RowF32>(w, at, n, vec), o);
    else if (kind == ZS_DTYPE_FP16) RowFP16::floats(fetch8<RowFP16>(w, at, n, vec), o);
    else RowBF16::floats(fetch8<RowBF16>(w, at, n, vec), o);
}

__device__ __forceinline__ int part(int64_t cols, int64_t at) {      // of 8 columns from `at` on, how many there are
    return (int)max((int64_t)0, min((int64_t)8, cols - at));
}

// ------------------------------------------------------- sums of a row --

// A sum of products a b as hi + lo.  The accumulator begins at 3 * 2^m, 2^m
// above the sum of the magnitudes, and so stays in [2^(m+1), 2^(m+2)): then
//   s = a b + h;  d = h - s (exact);  e = a b + d (the rounding error of s)
// four paired instructions for two products.  m: from the largest magnitudes,
// at least -100 (products below 2^-126 are lost then).
struct Dot {
    f2 h, l;
    float start;
    // of at most 8 N pairs with |a| <= top_a, |b| <= top_b; false: too large
    template <int N>
    __device__ __forceinline__ bool begin(float top_a, float top_b) {
        const int ea = (int)(__float_as_uint(top_a) >> 23) - 127, eb = (int)(__float_as_uint(top_b) >> 23) - 127;
        constexpr int LOG = N <= 1 ? 2 : N <= 2 ? 3 : N <= 4 ? 4 : 5;      // of the products of one half
        const int m = max(ea + eb + 2 + LOG, -100);
        const bool ok = max(ea, eb) < 60;            // infinities and NaN have 128
        start = __uint_as_float(ok ? (uint32_t)(m + 1 + 127) << 23 | 0x400000u : 0x7F800000u);
        h = f2pack(start, start);
        l = 0;
        return ok;
    }
    __device__ __forceinline__ void add(f2 a, f2 b) {
        f2 s, d, e;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(s) : "l"(a), "l"(b), "l"(h));
        asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(h), "l"(s));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(a), "l"(b), "l"(d));
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(l) : "l"(l), "l"(e));
        h = s;
    }
    __device__ __forceinline__ void end(float &hi, float &lo) const {
        float h0, h1, l0, l1;
        f2unpack(h, h0, h1);
        f2unpack(l, l0, l1);
        hi = __fsub_rn(h0, start);
        lo = l0;
        add22(hi, lo, __fsub_rn(h1, start), l1);
    }
};

__device__ __forceinline__ void max_abs3(float &m, float a, float b) {
    asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, %0, t;\n\t}" : "+f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
}

// A row's pair over the lanes of a warp; the same in all of them.
__device__ __forceinline__ void warp_pair(float &hi, float &lo) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float h2 = __shfl_xor_sync(0xFFFFFFFFu, hi, off), l2 = __shfl_xor_sync(0xFFFFFFFFu, lo, off);
        add22(hi, lo, h2, l2);
    }
}
__device__ __forceinline__ double warp_double(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// 1 / cols as a pair
struct Mean {
    float hi, lo;
};
__device__ __forceinline__ void times(float &hi, float &lo, float bh, float bl) {
    const float p = __fmul_rn(hi, bh);
    const float e = __fmaf_rn(hi, bh, -p);
    lo = __fadd_rn(e, __fadd_rn(__fmul_rn(hi, bl), __fmul_rn(lo, bh)));
    hi = __fadd_rn(p, lo);
    lo = __fsub_rn(lo, __fsub_rn(hi, p));
}

// 1 / sqrt(s / cols + eps): an estimate r of the root's reciprocal and one
// Newton step r + r (1 - v r r) / 2, whose residual is formed to 2^-45 by fused
// products, after v was taken to [1, 4) by a power of four.
__device__ __forceinline__ float rstd_of(float hi, float lo, const Mean &mean, float eps) {
    times(hi, lo, mean.hi, mean.lo);
    add22(hi, lo, eps, 0.0f);
    const int e = ((int)(__float_as_uint(hi) >> 23) - 127) >> 1;           // floor
    if (!(hi >= 1.1754944e-38f) || hi > 3e38f) return __fdiv_rn(1.0f, __fsqrt_rn(hi));
    const float s = __uint_as_float((uint32_t)(127 - e) << 23);
    hi = __fmul_rn(__fmul_rn(hi, s), s);
    lo = __fmul_rn(__fmul_rn(lo, s), s);
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(hi));
    const float a = __fmul_rn(r, r), ae = __fmaf_rn(r, r, -a);
    const float p = __fmul_rn(hi, a), pe = __fmaf_rn(hi, a, -p);
    const float d = __fsub_rn(__fsub_rn(__fsub_rn(1.0f, p), pe), __fmaf_rn(hi, ae, __fmul_rn(lo, a)));
    return __fmul_rn(__fmaf_rn(__fmul_rn(0.5f, r), d, r), s);
}
__device__ __forceinline__ float rstd_of(double total, double cols, float eps) {
    return (float)__drcp_rn(__dsqrt_rn(__dadd_rn(__ddiv_rn(total, cols), (double)eps)));
}
// rstd^2 mean(g x)
__device__ __forceinline__ float slope_of(float hi, float lo, const Mean &mean, float rstd) {
    times(hi, lo, mean.hi, mean.lo);
    const float a = __fmul_rn(rstd, rstd), ae = __fmaf_rn(rstd, rstd, -a);
    times(hi, lo, a, ae);
    return hi;
}

// -------------------------------------------------------------- 4 bits --

struct NormHeld {
    uint8_t *r_codes, *r_scales, *c_codes, *c_scales;
    int64_t rows, cols;
};

// 8 values a lane, 4 neighbouring lanes a group along the row; y is 0 past the
// matrix.  `row` may lie past the matrix, in the tile of scales that holds it.
__device__ __forceinline__ void hold_rows(const NormHeld &h, int64_t row, int64_t col, const float v[8]) {
    float top = 0.0f, y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) max_abs3(top, v[i], v[i + 1]);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, top, off);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(o));
    }
    const uint32_t byte = mx4_scale_byte(__float_as_uint(top) >> 23);
    const float inv = byte == 255u ? 0.0f : mx4_inverse(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(v[i], inv);
    const uint32_t word = byte == 255u ? 0u : e2m1x8(y);
    const int64_t g = col / MX4_GROUP;
    if (row < h.rows && g < mx4_groups(h.cols))
        *reinterpret_cast<uint32_t *>(h.r_codes + row * mx4_row_bytes(h.cols) + col / 2) = word;
    if ((threadIdx.x & 3) == 0 && row < 128 * mx4_row_tiles(h.rows) && g < 4 * mx4_atoms(h.cols))
        h.r_scales[((row >> 7) * mx4_atoms(h.cols) + (g >> 2)) * MX4_ATOM + mx4_in_atom((int)(row & 127), (int)(g & 3))] = (uint8_t)byte;
}

// The 32 rows from 32 * g on of one column, in shared memory `pitch` floats apart.
__device__ __forceinline__ void hold_column(const NormHeld &h, int64_t g, int64_t col, const float *from, int pitch) {
    float v[32], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = from[i * pitch];
#pragma unroll
    for (int i = 0; i < 32; i += 2) max_abs3(top, v[i], v[i + 1]);
    const uint32_t byte = mx4_scale_byte(__float_as_uint(top) >> 23);
    const float inv = byte == 255u ? 0.0f : mx4_inverse(byte);
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(v[8 * j + i], inv);
        q[j] = byte == 255u ? 0u : e2m1x8(y);
    }
    if (col < h.cols && g < mx4_groups(h.rows))
        *reinterpret_cast<uint4 *>(h.c_codes + col * mx4_row_bytes(h.rows) + 16 * g) = make_uint4(q[0], q[1], q[2], q[3]);
    if (col < 128 * mx4_row_tiles(h.cols) && g < 4 * mx4_atoms(h.rows))
        h.c_scales[((col >> 7) * mx4_atoms(h.rows) + (g >> 2)) * MX4_ATOM + mx4_in_atom((int)(col & 127), (int)(g & 3))] = (uint8_t)byte;
}

// ------------------------------------------------------- forward, rows --

struct NormArgs {
    const void *x, *residual, *w;
    void *sum, *out;
    float *rstd;
    int64_t ldx, ldr, lds, ldo;
    int32_t w_kind;
    bool vec;                        // every matrix has 16-byte aligned rows
    float eps;
    Mean mean;
    NormHeld held;
};

// WPR warps take a row, 8 values a lane and block of 256 columns; a lane keeps
// its NB blocks (NB 0: more than registers hold, read again).  Bandwidth
// bounds many rows, the way through the sum's exchange a few.
template <class R, int WPR, int NB>
__global__ void __launch_bounds__(THREADS)
rms_rows_kernel(NormArgs a) {
    constexpr int ROWS = WARPS / WPR, KEEP = NB > 0 ? NB : 1;
    __shared__ float2 parts[WARPS];
    __shared__ double wides[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % WPR;
    const int64_t rows = a.held.rows, cols = a.held.cols, row = (int64_t)blockIdx.x * ROWS + warp / WPR;
    const int blocks = NB > 0 ? NB : (int)((cols + 256 * WPR - 1) / (256 * WPR));
    const bool there = row < rows;
    pdl_wait();
    pdl_trigger();
    auto input = [&](int b, float h[8]) {
        const int64_t c = 256 * (int64_t)(mine + WPR * b) + 8 * lane;
        const int n = there ? part(cols, c) : 0;
        R::floats(fetch8<R>(a.x, row * a.ldx + c, n, a.vec), h);
        if (!a.residual) return;
        float r[8];
        R::floats(fetch8<R>(a.residual, row * a.ldr + c, n, a.vec), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __fadd_rn(h[i], r[i]);
    };
    float h[KEEP][8];
    float hi = 0.0f, lo = 0.0f;
    auto square = [&](auto &v) {                     // of one or all blocks
        constexpr int N = sizeof(v) / 32;
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
            for (int i = 0; i < 8; i += 2) max_abs3(top, v[b][i], v[b][i + 1]);
        Dot d;
        const bool ok = d.begin<N>(top, top);
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const f2 p = f2pack(v[b][i], v[b][i + 1]);
                d.add(p, p);
            }
        float dh, dl;
        d.end(dh, dl);
        add22(hi, lo, ok ? dh : __uint_as_float(0x7F800000u), dl);
    };
    if constexpr (NB > 0) {
#pragma unroll
        for (int b = 0; b < NB; ++b) input(b, h[b]);
        square(h);
    } else {
        for (int b = 0; b < blocks; ++b) {
            input(b, h[0]);
            square(h);
        }
    }
    warp_pair(hi, lo);
    if (WPR > 1) {
        if (lane == 0) parts[warp] = make_float2(hi, lo);
        __syncthreads();
        const int first = warp - mine;
        hi = parts[first].x;
        lo = parts[first].y;
#pragma unroll
        for (int k = 1; k < WPR; ++k) add22(hi, lo, parts[first + k].x, parts[first + k].y);
    }
    float rstd = rstd_of(hi, lo, a.mean, a.eps);
    // too large for float32's squares (or not finite): in 64 bits
    if (__syncthreads_or(!finite_f32(hi))) {
        double s = 0.0;
        for (int b = 0; b < blocks; ++b) {
            float v[8];
            input(b, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __dadd_rn(s, __dmul_rn((double)v[i], (double)v[i]));
        }
        s = warp_double(s);
        if (lane == 0) wides[warp] = s;
        __syncthreads();
        s = 0.0;
        for (int k = 0; k < WPR; ++k) s = __dadd_rn(s, wides[warp - mine + k]);
        if (!finite_f32(hi)) rstd = rstd_of(s, (double)cols, a.eps);
    }
    if (there && mine == 0 && lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int b = 0; b < blocks; ++b) {
        const int64_t c = 256 * (int64_t)(mine + WPR * b) + 8 * lane;
        const int n = there ? part(cols, c) : 0;
        float v[8], w[8];
        if constexpr (NB > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h[b][i];
        } else {
            input(b, v);
        }
        if (a.sum) R::store(a.sum, row * a.lds + c, n, a.vec, R::rounded(v));
        weights8(a.w, a.w_kind, c, n, a.vec, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rstd), w[i]);
        const typename R::Raw y = R::rounded(v);
        if (a.out) R::store(a.out, row * a.ldo + c, n, a.vec, y);
        if (a.held.r_codes) {
            R::floats(y, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i >= n) v[i] = 0.0f;
            hold_rows(a.held, row, c, v);
        }
    }
}

// ---------------------------------------------- 32 rows, shared by columns --

constexpr int TILE_ROWS = 32;
constexpr int TILE_COLS = 512;       // of 8 warps; K times as many of a CTA
constexpr int tile_smem(int k) { return TILE_ROWS * TILE_COLS * k * 4; }
constexpr int64_t TILE_MOST = 8 * 3 * TILE_COLS;     // columns that a cluster holds

// Place of 8 columns from 8 * lane on in a block of 256 floats: pieces of four
// side by side over the lanes, so that no two lanes meet in a bank.
__device__ __forceinline__ float4 *piece(float *block, int lane, int half) { return reinterpret_cast<float4 *>(block + 128 * half + 4 * lane); }
__device__ __forceinline__ int column_at(int place) {        // the column of a place, in its block of 256
    return 8 * ((place & 127) >> 2) + 4 * ((place >> 7) & 1) + (place & 3);
}

// What a cluster's CTAs tell one another: a pair for each row and 8 warps.
struct Exchange {
    float2 pairs[2][TILE_ROWS][4];
    double wides[TILE_ROWS][4];
};

// A cluster of ceil(cols / (512 K)) CTAs takes 32 rows.  A warp takes 4 of
// them, 512 columns of each: loads, the rows' sums of squares, the inputs to
// shared memory as floats; the exchange; then the result, its form along the
// rows from registers (4 lanes a group), and through shared memory the one
// along the columns (a thread 32 rows of a column).
template <class R, int K>
__global__ void __launch_bounds__(THREADS *K, K == 1 ? 3 : 1)
rms_tile_kernel(NormArgs a) {
    extern __shared__ __align__(16) float tile[];
    __shared__ Exchange ex;
    __shared__ float rstds[TILE_ROWS];
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kk = warp / WARPS, rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int64_t rows = a.held.rows, cols = a.held.cols, rb = blockIdx.x / ranks, row0 = TILE_ROWS * rb;
    const int64_t col0 = (int64_t)rank * TILE_COLS * K + TILE_COLS * kk + 8 * lane;      // and 256 on
    constexpr int PITCH = TILE_COLS * K;
    pdl_wait();
    pdl_trigger();
#pragma unroll 2
    for (int i = 0; i < TILE_ROWS / WARPS; ++i) {
        const int r = warp % WARPS + WARPS * i;
        const int64_t row = row0 + r;
        float h[2][8], top = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int64_t c = col0 + 256 * b;
            const int n = row < rows ? part(cols, c) : 0;
            R::floats(fetch8<R>(a.x, row * a.ldx + c, n, a.vec), h[b]);
            if (a.residual) {
                float q[8];
                R::floats(fetch8<R>(a.residual, row * a.ldr + c, n, a.vec), q);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[b][j] = __fadd_rn(h[b][j], q[j]);
                R::store(a.sum, row * a.lds + c, n, a.vec, R::rounded(h[b]));
            }
            float *block = tile + r * PITCH + TILE_COLS * kk + 256 * b;
            *piece(block, lane, 0) = make_float4(h[b][0], h[b][1], h[b][2], h[b][3]);
            *piece(block, lane, 1) = make_float4(h[b][4], h[b][5], h[b][6], h[b][7]);
#pragma unroll
            for (int j = 0; j < 8; j += 2) max_abs3(top, h[b][j], h[b][j + 1]);
        }
        Dot d;
        const bool ok = d.begin<2>(top, top);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const f2 p = f2pack(h[b][j], h[b][j + 1]);
                d.add(p, p);
            }
        float hi, lo;
        d.end(hi, lo);
        if (!ok) hi = __uint_as_float(0x7F800000u);
        warp_pair(hi, lo);
        if (lane == 0) ex.pairs[0][r][kk] = make_float2(hi, lo);
    }
    cluster.sync();
    float hi = 0.0f, lo = 0.0f;
    if (threadIdx.x < TILE_ROWS) {
        for (int q = 0; q < ranks; ++q) {
            const Exchange *other = cluster.map_shared_rank(&ex, q);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float2 p = other->pairs[0][threadIdx.x][k];
                add22(hi, lo, p.x, p.y);
            }
        }
        rstds[threadIdx.x] = rstd_of(hi, lo, a.mean, a.eps);
    }
    // too large for float32's squares (or not finite): in 64 bits; every CTA of
    // the cluster has seen the same sums and comes here, or none does
    if (__syncthreads_or(!finite_f32(hi))) {
        for (int i = 0; i < TILE_ROWS / WARPS; ++i) {
            const int r = warp % WARPS + WARPS * i;
            double s = 0.0;
            for (int j = lane; j < TILE_COLS; j += 32) {
                const double v = tile[r * PITCH + TILE_COLS * kk + j];
                s = __dadd_rn(s, __dmul_rn(v, v));
            }
            s = warp_double(s);
            if (lane == 0) ex.wides[r][kk] = s;
        }
        cluster.sync();
        if (threadIdx.x < TILE_ROWS && !finite_f32(hi)) {
            double s = 0.0;
            for (int q = 0; q < ranks; ++q)
                for (int k = 0; k < K; ++k) s = __dadd_rn(s, cluster.map_shared_rank(&ex, q)->wides[threadIdx.x][k]);
            rstds[threadIdx.x] = rstd_of(s, (double)cols, a.eps);
        }
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x < TILE_ROWS && row0 + threadIdx.x < rows) a.rstd[row0 + threadIdx.x] = rstds[threadIdx.x];
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
        const int64_t c = col0 + 256 * b;
        const int nc = part(cols, c);
        float w[8];
        weights8(a.w, a.w_kind, c, nc, a.vec, w);
#pragma unroll 2
        for (int i = 0; i < TILE_ROWS / WARPS; ++i) {
            const int r = warp % WARPS + WARPS * i;
            const int64_t row = row0 + r;
            const int n = row < rows ? nc : 0;
            float *block = tile + r * PITCH + TILE_COLS * kk + 256 * b;
            const float4 p = *piece(block, lane, 0), q = *piece(block, lane, 1);
            float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
            const float rstd = rstds[r];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], rstd), w[j]);
            const typename R::Raw y = R::rounded(v);
            if (a.out) R::store(a.out, row * a.ldo + c, n, a.vec, y);
            R::floats(y, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) if (j >= n) v[j] = 0.0f;
            *piece(block, lane, 0) = make_float4(v[0], v[1], v[2], v[3]);
            *piece(block, lane, 1) = make_float4(v[4], v[5], v[6], v[7]);
            if (a.held.r_codes) hold_rows(a.held, row, c, v);
        }
    }
    __syncthreads();
    for (int place = threadIdx.x; place < PITCH; place += THREADS * K)
        hold_column(a.held, rb, (int64_t)rank * PITCH + (place & ~255) + column_at(place & 255), tile + place, PITCH);
    cluster.sync();                  // the others may still read this CTA's sums
}

// ------------------------------------------------------------- backward --

struct BackArgs {
    const void *dy, *x, *w, *residual;
    const float *rstd;
    void *dx;
    float *dw_parts;                 // [clusters][cols], or NULL
    int64_t lddy, ldx, ldr, ldd;
    int32_t w_kind;
    bool vec;
    Mean mean;
    NormHeld held;
    int64_t row_blocks;
};

// As rms_tile_kernel, a cluster taking row blocks b, b + clusters, ...: a lane
// adds up its columns' part of dw over all of them.  Shared memory keeps both
// inputs of 16 bits in the place of a float; of 32 bits x alone, and dy is read
// again.
template <class R, int K>
__global__ void __launch_bounds__(THREADS *K, K == 1 ? 2 : 1)
rms_back_kernel(BackArgs a) {
    extern __shared__ __align__(16) float tile[];
    __shared__ Exchange ex;
    __shared__ float slopes[TILE_ROWS], rstds[TILE_ROWS];
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kk = warp / WARPS, rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int64_t rows = a.held.rows, cols = a.held.cols;
    const int64_t col0 = (int64_t)rank * TILE_COLS * K + TILE_COLS * kk + 8 * lane;
    constexpr int PITCH = TILE_COLS * K;
    pdl_wait();
    pdl_trigger();
    float w[2][8], dw[2][8] = {};
#pragma unroll
    for (int b = 0; b < 2; ++b) weights8(a.w, a.w_kind, col0 + 256 * b, part(cols, col0 + 256 * b), a.vec, w[b]);
    int turn = 0;
    for (int64_t rb = blockIdx.x / ranks; rb < a.row_blocks; rb += gridDim.x / ranks, turn ^= 1) {
        const int64_t row0 = TILE_ROWS * rb;
#pragma unroll 1
        for (int i = 0; i < TILE_ROWS / WARPS; ++i) {
            const int r = warp % WARPS + WARPS * i;
            const int64_t row = row0 + r;
            const float rstd = row < rows ? a.rstd[row] : 0.0f;
            float g[2][8], x[2][8], tg = 0.0f, tx = 0.0f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int64_t c = col0 + 256 * b;
                const int n = row < rows ? part(cols, c) : 0;
                const typename R::Raw rd = fetch8<R>(a.dy, row * a.lddy + c, n, a.vec), rx = fetch8<R>(a.x, row * a.ldx + c, n, a.vec);
                float *block = tile + r * PITCH + TILE_COLS * kk + 256 * b;
                R::floats(rd, g[b]);
                R::floats(rx, x[b]);
                if constexpr (R::SIZE == 2) {
                    uint32_t u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] = lane16(rd, j) | lane16(rx, j) << 16;
                    *reinterpret_cast<uint4 *>(piece(block, lane, 0)) = make_uint4(u[0], u[1], u[2], u[3]);
                    *reinterpret_cast<uint4 *>(piece(block, lane, 1)) = make_uint4(u[4], u[5], u[6], u[7]);
                } else {
                    *piece(block, lane, 0) = make_float4(x[b][0], x[b][1], x[b][2], x[b][3]);
                    *piece(block, lane, 1) = make_float4(x[b][4], x[b][5], x[b][6], x[b][7]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[b][j] = __fmaf_rn(g[b][j], __fmul_rn(x[b][j], rstd), dw[b][j]);
                    g[b][j] = __fmul_rn(g[b][j], w[b][j]);
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    max_abs3(tg, g[b][j], g[b][j + 1]);
                    max_abs3(tx, x[b][j], x[b][j + 1]);
                }
            }
            Dot d;
            const bool ok = d.begin<2>(tg, tx);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 8; j += 2) d.add(f2pack(g[b][j], g[b][j + 1]), f2pack(x[b][j], x[b][j + 1]));
            float hi, lo;
            d.end(hi, lo);
            if (!ok) {                               // far outside of any gradient's range: in 64 bits
                double s = 0.0;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s = __dadd_rn(s, __dmul_rn((double)g[b][j], (double)x[b][j]));
                hi = (float)s;
                lo = finite_f32(hi) ? (float)(s - (double)hi) : 0.0f;
            }
            warp_pair(hi, lo);
            if (lane == 0) ex.pairs[turn][r][kk] = make_float2(hi, lo);
        }
        cluster.sync();
        if (threadIdx.x < TILE_ROWS) {
            float hi = 0.0f, lo = 0.0f;
            for (int q = 0; q < ranks; ++q) {
                const Exchange *other = cluster.map_shared_rank(&ex, q);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 p = other->pairs[turn][threadIdx.x][k];
                    add22(hi, lo, p.x, p.y);
                }
            }
            const float rstd = row0 + threadIdx.x < rows ? a.rstd[row0 + threadIdx.x] : 0.0f;
            rstds[threadIdx.x] = rstd;
            slopes[threadIdx.x] = slope_of(hi, lo, a.mean, rstd);
        }
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < TILE_ROWS / WARPS; ++i) {
            const int r = warp % WARPS + WARPS * i;
            const int64_t row = row0 + r;
            const float rstd = rstds[r], slope = slopes[r];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int64_t c = col0 + 256 * b;
                const int n = row < rows ? part(cols, c) : 0;
                float *block = tile + r * PITCH + TILE_COLS * kk + 256 * b;
                float v[8], x[8];
                if constexpr (R::SIZE == 2) {
                    const uint4 p = *reinterpret_cast<const uint4 *>(piece(block, lane, 0)), q = *reinterpret_cast<const uint4 *>(piece(block, lane, 1));
                    const uint32_t u[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                    uint32_t ud[8], ux[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ud[j] = u[j] & 0xFFFFu;
                        ux[j] = u[j] >> 16;
                    }
                    R::floats(pack8(ud), v);
                    R::floats(pack8(ux), x);
                } else {
                    const float4 p = *piece(block, lane, 0), q = *piece(block, lane, 1);
                    x[0] = p.x; x[1] = p.y; x[2] = p.z; x[3] = p.w;
                    x[4] = q.x; x[5] = q.y; x[6] = q.z; x[7] = q.w;
                    R::floats(fetch8<R>(a.dy, row * a.lddy + c, n, a.vec), v);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = __fmul_rn(__fsub_rn(__fmul_rn(v[j], w[b][j]), __fmul_rn(x[j], slope)), rstd);
                if (a.residual) {
                    float q[8];
                    R::floats(fetch8<R>(a.residual, row * a.ldr + c, n, a.vec), q);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], q[j]);
                }
                const typename R::Raw y = R::rounded(v);
                R::store(a.dx, row * a.ldd + c, n, a.vec, y);
                if (!a.held.r_codes && !a.held.c_codes) continue;
                R::floats(y, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) if (j >= n) v[j] = 0.0f;
                if (a.held.c_codes) {
                    *piece(block, lane, 0) = make_float4(v[0], v[1], v[2], v[3]);
                    *piece(block, lane, 1) = make_float4(v[4], v[5], v[6], v[7]);
                }
                if (a.held.r_codes) hold_rows(a.held, row, c, v);
            }
        }
        __syncthreads();
        if (a.held.c_codes) {
            for (int place = threadIdx.x; place < PITCH; place += THREADS * K)
                hold_column(a.held, rb, (int64_t)rank * PITCH + (place & ~255) + column_at(place & 255), tile + place, PITCH);
            __syncthreads();
        }
    }
    // the 8 warps' parts of dw, in their order
    if (a.dw_parts) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float *block = tile + (warp % WARPS) * PITCH + TILE_COLS * kk + 256 * b;
            *piece(block, lane, 0) = make_float4(dw[b][0], dw[b][1], dw[b][2], dw[b][3]);
            *piece(block, lane, 1) = make_float4(dw[b][4], dw[b][5], dw[b][6], dw[b][7]);
        }
        __syncthreads();
        for (int place = threadIdx.x; place < PITCH; place += THREADS * K) {
            float s = tile[place];
#pragma unroll
            for (int i = 1; i < WARPS; ++i) s = __fadd_rn(s, tile[i * PITCH + place]);
            const int64_t col = (int64_t)rank * PITCH + (place & ~255) + column_at(place & 255);
            if (col < cols) a.dw_parts[blockIdx.x / ranks * cols + col] = s;
        }
    }
    cluster.sync();                  // the others may still read this CTA's sums
}

// Rows longer than a cluster holds: a CTA a row, both inputs read twice.
template <class R>
__global__ void __launch_bounds__(THREADS)
rms_back_rows_kernel(BackArgs a) {
    __shared__ float2 parts[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x, cols = a.held.cols;
    pdl_wait();
    pdl_trigger();
    const float rstd = a.rstd[row];
    float hi = 0.0f, lo = 0.0f;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < cols; c += 8 * THREADS) {
        const int n = part(cols, c);
        float g[8], x[8], w[8], tg = 0.0f, tx = 0.0f;
        R::floats(fetch8<R>(a.dy, row * a.lddy + c, n, a.vec), g);
        R::floats(fetch8<R>(a.x, row * a.ldx + c, n, a.vec), x);
        weights8(a.w, a.w_kind, c, n, a.vec, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], w[j]);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            max_abs3(tg, g[j], g[j + 1]);
            max_abs3(tx, x[j], x[j + 1]);
        }
        Dot d;
        float dh, dl;
        if (d.begin<1>(tg, tx)) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) d.add(f2pack(g[j], g[j + 1]), f2pack(x[j], x[j + 1]));
            d.end(dh, dl);
        } else {
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = __dadd_rn(s, __dmul_rn((double)g[j], (double)x[j]));
            dh = (float)s;
            dl = finite_f32(dh) ? (float)(s - (double)dh) : 0.0f;
        }
        add22(hi, lo, dh, dl);
    }
    warp_pair(hi, lo);
    if (lane == 0) parts[warp] = make_float2(hi, lo);
    __syncthreads();
    hi = parts[0].x;
    lo = parts[0].y;
    for (int k = 1; k < WARPS; ++k) add22(hi, lo, parts[k].x, parts[k].y);
    const float slope = slope_of(hi, lo, a.mean, rstd);
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < cols; c += 8 * THREADS) {
        const int n = part(cols, c);
        float v[8], x[8], w[8];
        R::floats(fetch8<R>(a.dy, row * a.lddy + c, n, a.vec), v);
        R::floats(fetch8<R>(a.x, row * a.ldx + c, n, a.vec), x);
        weights8(a.w, a.w_kind, c, n, a.vec, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fsub_rn(__fmul_rn(v[j], w[j]), __fmul_rn(x[j], slope)), rstd);
        if (a.residual) {
            float q[8];
            R::floats(fetch8<R>(a.residual, row * a.ldr + c, n, a.vec), q);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], q[j]);
        }
        R::store(a.dx, row * a.ldd + c, n, a.vec, R::rounded(v));
    }
}
// Their part of dw: 2048 columns of the rows b, b + gridDim.y, ...
template <class R>
__global__ void __launch_bounds__(THREADS)
rms_back_weight_kernel(BackArgs a) {
    const int64_t cols = a.held.cols, c = 8 * ((int64_t)blockIdx.x * THREADS + threadIdx.x);
    const int n = part(cols, c);
    pdl_wait();
    pdl_trigger();
    float dw[8] = {};
    for (int64_t row = blockIdx.y; row < a.held.rows; row += gridDim.y) {
        const float rstd = a.rstd[row];
        float v[8], x[8];
        R::floats(fetch8<R>(a.dy, row * a.lddy + c, n, a.vec), v);
        R::floats(fetch8<R>(a.x, row * a.ldx + c, n, a.vec), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = __fmaf_rn(v[j], __fmul_rn(x[j], rstd), dw[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) if (j < n) a.dw_parts[blockIdx.y * cols + c + j] = dw[j];
}

// dw from its parts, in their order: 32 columns a CTA, 8 shares of the parts.
__global__ void __launch_bounds__(THREADS)
rms_weight_kernel(const float *parts, int n, int64_t cols, void *dw, int kind) {
    __shared__ float share[WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = 32 * (int64_t)blockIdx.x + lane;
    pdl_wait();
    pdl_trigger();
    float s = 0.0f;
    if (c < cols)
        for (int i = warp; i < n; i += WARPS) s = __fadd_rn(s, parts[i * cols + c]);
    share[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    for (int i = 1; i < WARPS; ++i) s = __fadd_rn(s, share[i][lane]);
    if (kind == ZS_DTYPE_FP32) static_cast<float *>(dw)[c] = s;
    else static_cast<uint16_t *>(dw)[c] = (uint16_t)(kind == ZS_DTYPE_FP16 ? FP16T::from_f32(s) : BF16T::from_f32(s));
}

// ------------------------------------------------------------- launches --

template <class R, int WPR, int NB>
static cudaError_t rows_launch(const NormArgs &a, int64_t grid_rows, cudaStream_t s) {
    const int64_t per = WARPS / WPR, grid = (grid_rows + per - 1) / per;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_dependent(rms_rows_kernel<R, WPR, NB>, (unsigned)grid, THREADS, 0, 1, s, a);
}
// As many warps a row as give each lane 16 values; past 8 warps more values.
template <class R>
static cudaError_t rows_of(const NormArgs &a, int64_t grid_rows, cudaStream_t s) {
    const int64_t cols = a.held.cols;
    if (cols <= 256) return rows_launch<R, 1, 1>(a, grid_rows, s);
    if (cols <= 512) return rows_launch<R, 1, 2>(a, grid_rows, s);
    if (cols <= 1024) return rows_launch<R, 2, 2>(a, grid_rows, s);
    if (cols <= 2048) return rows_launch<R, 4, 2>(a, grid_rows, s);
    if (cols <= 4096) return rows_launch<R, 8, 2>(a, grid_rows, s);
    if (cols <= 8192) return rows_launch<R, 8, 4>(a, grid_rows, s);
    if (cols <= 16384) return rows_launch<R, 8, 8>(a, grid_rows, s);
    return rows_launch<R, 8, 0>(a, grid_rows, s);
}

// CTAs of a cluster, and warps of a CTA by 8, for rows of these columns.
static void tile_shape(int64_t cols, unsigned &ctas, int &k) {
    k = cols <= 8 * TILE_COLS ? 1 : cols <= 16 * TILE_COLS ? 2 : 3;
    ctas = (unsigned)((cols + TILE_COLS * k - 1) / (TILE_COLS * k));
}

template <class... P>
static cudaError_t tile_launch(void (*kernel)(P...), std::atomic<bool> (&set)[64], int k, unsigned ctas, int64_t clusters, cudaStream_t s, const P &...args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem(k));
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    return launch_dependent(kernel, (unsigned)(ctas * clusters), THREADS * k, tile_smem(k), ctas, s, args...);
}

template <class R, int K>
static cudaError_t norm_tile(const NormArgs &a, unsigned ctas, cudaStream_t s) {
    static std::atomic<bool> set[64];
    return tile_launch(rms_tile_kernel<R, K>, set, K, ctas, 4 * mx4_atoms(a.held.rows), s, a);
}
template <class R, int K>
static cudaError_t back_tile(const BackArgs &a, unsigned ctas, int64_t clusters, cudaStream_t s) {
    static std::atomic<bool> set[64];
    return tile_launch(rms_back_kernel<R, K>, set, K, ctas, clusters, s, a);
}

// Parts of dw: clusters that are resident at once (a number of the sizes
// alone, so that a sum has the same bits whatever forms are asked for).
static int64_t back_parts(int64_t rows, int64_t cols) {
    const int64_t blocks = (rows + TILE_ROWS - 1) / TILE_ROWS;
    if (cols > TILE_MOST) return blocks < 64 ? blocks : 64;
    unsigned ctas;
    int k;
    tile_shape(cols, ctas, k);
    const int64_t most = (k == 1 ? 304 : 152) / (int64_t)ctas;
    return blocks < most ? blocks : most;
}

template <class F>
static cudaError_t by_type(int32_t dtype, F f) {
    if (dtype == ZS_DTYPE_FP32) return f(RowF32());
    if (dtype == ZS_DTYPE_FP16) return f(RowFP16());
    return f(RowBF16());
}

}  // namespace zsk

namespace {

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
bool dtype_ok(int32_t t) { return t >= ZS_DTYPE_BF16 && t <= ZS_DTYPE_FP32; }
int dtype_size(int32_t t) { return t == ZS_DTYPE_FP32 ? 4 : 2; }
constexpr int64_t MOST = (int64_t)1 << 31;           // rows, columns

zs_status cuda_status(cudaError_t e, const char *fn) {
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

struct Matrix {
    const void *p;
    int64_t ld;
    bool need;
    const char *name;
};

// Sizes and matrices; *vec: all that are there have 16-byte aligned rows.
template <int N>
zs_status check(const Matrix (&m)[N], int64_t rows, int64_t cols, int32_t dtype, bool *vec, const char *fn) {
    if (rows < 0 || cols < 0 || rows >= MOST || cols >= MOST)
        return zs_fail(ZS_EINVAL, "%s: %lld x %lld out of range", fn, (long long)rows, (long long)cols);
    if (!dtype_ok(dtype)) return zs_fail(ZS_EINVAL, "%s: dtype %d", fn, dtype);
    *vec = true;
    for (const Matrix &x : m) {
        if (!x.p) {
            if (x.need && rows > 0 && cols > 0) return zs_fail(ZS_EINVAL, "%s: %s NULL", fn, x.name);
            continue;
        }
        if (x.ld < cols) return zs_fail(ZS_EINVAL, "%s: %s: row stride %lld < %lld columns", fn, x.name, (long long)x.ld, (long long)cols);
        if (addr(x.p) % dtype_size(dtype)) return zs_fail(ZS_EINVAL, "%s: %s not aligned to its elements", fn, x.name);
        if (addr(x.p) % 16 || (rows > 1 && x.ld * dtype_size(dtype) % 16)) *vec = false;
    }
    return ZS_OK;
}

zs_status check_vector(const void *p, int32_t kind, bool need, bool *vec, const char *name, const char *fn) {
    if (!p) return need ? zs_fail(ZS_EINVAL, "%s: %s NULL", fn, name) : ZS_OK;
    if (!dtype_ok(kind)) return zs_fail(ZS_EINVAL, "%s: %s: dtype %d", fn, name, kind);
    if (addr(p) % dtype_size(kind)) return zs_fail(ZS_EINVAL, "%s: %s not aligned to its elements", fn, name);
    if (vec && addr(p) % 16) *vec = false;
    return ZS_OK;
}

zs_status check_held(const void *codes, const void *scales, const char *what, const char *fn) {
    if ((codes || scales) && (!codes || !scales || addr(codes) % 16 || addr(scales) % 16))
        return zs_fail(ZS_EINVAL, "%s: %s: codes or scales NULL or not 16-byte aligned", fn, what);
    return ZS_OK;
}

zsk::Mean mean_of(int64_t cols) {
    const double m = 1.0 / (double)cols;
    const float hi = (float)m;
    return {hi, (float)(m - (double)hi)};
}

}  // namespace

extern "C" {

zs_status zs_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, int32_t weight_dtype,
                      int64_t rows, int64_t cols, int32_t dtype, float eps, void *sum, int64_t lds, void *out, int64_t ldo,
                      float *rstd, void *r_codes, void *r_scales, void *c_codes, void *c_scales, void *stream) {
    const char *fn = "zs_rms_norm";
    const Matrix m[] = {{x, ldx, true, "x"}, {residual, ldr, false, "residual"}, {sum, lds, residual != nullptr, "sum"}, {out, ldo, false, "out"}};
    bool vec;
    zs_status r = check(m, rows, cols, dtype, &vec, fn);
    if (r) return r;
    if (sum && !residual) return zs_fail(ZS_EINVAL, "%s: sum without a residual is x itself", fn);
    if (!(eps >= 0.0f) || eps > 3e38f) return zs_fail(ZS_EINVAL, "%s: eps %g", fn, (double)eps);
    if ((r = check_held(r_codes, r_scales, "along rows", fn)) || (r = check_held(c_codes, c_scales, "along columns", fn))) return r;
    if (rows == 0 || cols == 0) {
        zs_clear_error();
        return ZS_OK;
    }
    if ((r = check_vector(weight, weight_dtype, true, &vec, "weight", fn)) || (r = check_vector(rstd, ZS_DTYPE_FP32, true, nullptr, "rstd", fn)))
        return r;
    if (!out && !r_codes && !c_codes) return zs_fail(ZS_EINVAL, "%s: no form of the result is asked for", fn);
    using namespace zsk;
    if (c_codes && cols > TILE_MOST && !out)
        return zs_fail(ZS_EINVAL, "%s: along the columns of more than %d columns needs out", fn, (int)TILE_MOST);
    NormArgs a;
    a.x = x; a.residual = residual; a.w = weight; a.sum = sum; a.out = out; a.rstd = rstd;
    a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldo = ldo;
    a.w_kind = weight_dtype; a.vec = vec; a.eps = eps; a.mean = mean_of(cols);
    const bool tiles = c_codes && cols <= TILE_MOST;
    a.held = {static_cast<uint8_t *>(r_codes), static_cast<uint8_t *>(r_scales), tiles ? static_cast<uint8_t *>(c_codes) : nullptr,
              tiles ? static_cast<uint8_t *>(c_scales) : nullptr, rows, cols};
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (tiles) {
        unsigned ctas;
        int k;
        tile_shape(cols, ctas, k);
        if (4 * mx4_atoms(rows) * ctas > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: %lld x %lld too large", fn, (long long)rows, (long long)cols);
        e = by_type(dtype, [&](auto t) {
            typedef decltype(t) R;
            return k == 1 ? norm_tile<R, 1>(a, ctas, s) : k == 2 ? norm_tile<R, 2>(a, ctas, s) : norm_tile<R, 3>(a, ctas, s);
        });
        return cuda_status(e, fn);
    }
    // the rows' tiles of scales have to be whole
    const int64_t grid_rows = r_codes ? 128 * mx4_row_tiles(rows) : rows;
    e = by_type(dtype, [&](auto t) { return rows_of<decltype(t)>(a, grid_rows, s); });
    if (e != cudaSuccess || !c_codes) return cuda_status(e, fn);
    return zs_mx4_quantize(out, rows, cols, ldo, dtype, nullptr, nullptr, c_codes, c_scales, stream);
}

zs_status zs_rms_norm_scratch(int64_t rows, int64_t cols, int64_t *bytes) {
    const char *fn = "zs_rms_norm_scratch";
    if (!bytes) return zs_fail(ZS_EINVAL, "%s: NULL result", fn);
    if (rows < 0 || cols < 0 || rows >= MOST || cols >= MOST)
        return zs_fail(ZS_EINVAL, "%s: %lld x %lld out of range", fn, (long long)rows, (long long)cols);
    *bytes = rows > 0 && cols > 0 ? zsk::back_parts(rows, cols) * cols * 4 : 0;
    zs_clear_error();
    return ZS_OK;
}

zs_status zs_rms_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *weight, int32_t weight_dtype,
                               const float *rstd, const void *residual, int64_t ldr, int64_t rows, int64_t cols, int32_t dtype,
                               void *dx, int64_t lddx, void *dw, int32_t dw_dtype, float *scratch, void *r_codes, void *r_scales,
                               void *c_codes, void *c_scales, void *stream) {
    const char *fn = "zs_rms_norm_backward";
    const Matrix m[] = {{dy, lddy, true, "dy"}, {x, ldx, true, "x"}, {residual, ldr, false, "residual"}, {dx, lddx, true, "dx"}};
    bool vec;
    zs_status r = check(m, rows, cols, dtype, &vec, fn);
    if (r) return r;
    if ((r = check_held(r_codes, r_scales, "along rows", fn)) || (r = check_held(c_codes, c_scales, "along columns", fn))) return r;
    if ((r = check_vector(dw, dw_dtype, false, nullptr, "dw", fn))) return r;
    const cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0 || cols == 0) {                    // dw of no rows is 0
        if (dw && cols > 0) return cuda_status(cudaMemsetAsync(dw, 0, (size_t)(cols * dtype_size(dw_dtype)), s), fn);
        zs_clear_error();
        return ZS_OK;
    }
    if ((r = check_vector(weight, weight_dtype, true, &vec, "weight", fn)) || (r = check_vector(rstd, ZS_DTYPE_FP32, true, nullptr, "rstd", fn)))
        return r;
    if (dw && (!scratch || addr(scratch) % 16)) return zs_fail(ZS_EINVAL, "%s: scratch NULL or not 16-byte aligned", fn);
    using namespace zsk;
    const bool tiles = cols <= TILE_MOST;
    BackArgs a;
    a.dy = dy; a.x = x; a.w = weight; a.residual = residual; a.rstd = rstd; a.dx = dx; a.dw_parts = dw ? scratch : nullptr;
    a.lddy = lddy; a.ldx = ldx; a.ldr = ldr; a.ldd = lddx;
    a.w_kind = weight_dtype; a.vec = vec; a.mean = mean_of(cols);
    a.held = {static_cast<uint8_t *>(r_codes), static_cast<uint8_t *>(r_scales), static_cast<uint8_t *>(c_codes),
              static_cast<uint8_t *>(c_scales), rows, cols};
    a.row_blocks = c_codes ? 4 * mx4_atoms(rows) : r_codes ? 4 * mx4_row_tiles(rows) : (rows + TILE_ROWS - 1) / TILE_ROWS;
    const int64_t parts = back_parts(rows, cols);
    cudaError_t e;
    if (tiles) {
        unsigned ctas;
        int k;
        tile_shape(cols, ctas, k);
        e = by_type(dtype, [&](auto t) {
            typedef decltype(t) R;
            return k == 1 ? back_tile<R, 1>(a, ctas, parts, s) : k == 2 ? back_tile<R, 2>(a, ctas, parts, s) : back_tile<R, 3>(a, ctas, parts, s);
        });
    } else {
        e = by_type(dtype, [&](auto t) {
            typedef decltype(t) R;
            cudaError_t f = cudaSuccess;
            if (dw) {                                // first: dx may be dy's memory
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)((cols + 8 * THREADS - 1) / (8 * THREADS)), (unsigned)parts);
                cfg.blockDim = dim3(THREADS);
                cfg.stream = s;
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
                attr[0].val.programmaticStreamSerializationAllowed = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                f = cudaLaunchKernelEx(&cfg, rms_back_weight_kernel<R>, a);
            }
            return f != cudaSuccess ? f : launch_dependent(rms_back_rows_kernel<R>, (unsigned)rows, THREADS, 0, 1, s, a);
        });
    }
    if (e == cudaSuccess && dw)
        e = launch_dependent(rms_weight_kernel, (unsigned)((cols + 31) / 32), THREADS, 0, 1, s, scratch, (int)parts, cols, dw, dw_dtype);
    if (e != cudaSuccess || tiles || (!r_codes && !c_codes)) return cuda_status(e, fn);
    return zs_mx4_quantize(dx, rows, cols, lddx, dtype, r_codes, r_scales, c_codes, c_scales, stream);
}

}  // extern "C"
