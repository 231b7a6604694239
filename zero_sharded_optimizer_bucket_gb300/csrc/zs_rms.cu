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

template <class T>
__device__ __forceinline__ void max_two(uint32_t &m, uint32_t w);        // the larger magnitudes of two pairs; a NaN stays
template <>
__device__ __forceinline__ void max_two<BF16T>(uint32_t &m, uint32_t w) {
    asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %1;\n\tmax.NaN.bf16x2 %0, %0, a;\n\t}" : "+r"(m) : "r"(w));
}
template <>
__device__ __forceinline__ void max_two<FP16T>(uint32_t &m, uint32_t w) {
    asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %1;\n\tmax.NaN.f16x2 %0, %0, a;\n\t}" : "+r"(m) : "r"(w));
}
__device__ __forceinline__ void max_abs3(float &m, float a, float b) {
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
}

// Raw: 8 elements of a lane as they lie in memory.
struct RowF32 {
    static constexpr int SIZE = 4;
    typedef uint32_t Elem;
    struct __align__(16) Raw { uint4 a, b; };
    static __device__ __forceinline__ Raw zero() { return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
    static __device__ __forceinline__ Raw of(const uint32_t v[8]) { return {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])}; }
    static __device__ __forceinline__ void floats(const Raw &r, float o[8]) {
        const uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ Raw rounded(const float o[8]) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(o[i]);
        return of(v);
    }
    static __device__ __forceinline__ Elem element(const Raw &r, int i) {
        const uint4 &q = i < 4 ? r.a : r.b;
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    }
    // the largest magnitude of the four neighbouring lanes' values
    static __device__ __forceinline__ float top4(const Raw &r) {
        float v[8], top = 0.0f;
        floats(r, v);
#pragma unroll
        for (int i = 0; i < 8; i += 2) max_abs3(top, v[i], v[i + 1]);
        max_abs3(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1), 0.0f);
        max_abs3(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2), 0.0f);
        return top;
    }
};
template <class T, bool FP16>
struct Row16 {
    static constexpr int SIZE = 2;
    typedef uint16_t Elem;
    typedef T Type;
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ Raw of(const uint32_t v[8]) { return pack8(v); }
    static __device__ __forceinline__ void floats(const Raw &r, float o[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (FP16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                o[2 * i] = f.x;
                o[2 * i + 1] = f.y;
            } else {
                o[2 * i] = __uint_as_float(w[i] << 16);
                o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
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
    static __device__ __forceinline__ Elem element(const Raw &r, int i) { return (Elem)lane16(r, i); }
    static __device__ __forceinline__ float top4(const Raw &r) {
        uint32_t m = 0;
        max_two<T>(m, r.x);
        max_two<T>(m, r.y);
        max_two<T>(m, r.z);
        max_two<T>(m, r.w);
        max_two<T>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        max_two<T>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        return T::to_f32(max(m & 0xFFFFu, m >> 16));
    }
};
typedef Row16<BF16T, false> RowBF16;
typedef Row16<FP16T, true> RowFP16;

// A lane's 8 of a block of 256 columns, `there` of which exist (any integer).
// vec: the row is 16-byte aligned.  Otherwise lanes load neighbouring elements,
// which turn (256 elements of the warp's shared memory) deals out: 8 loads of 2
// or 4 bytes a lane instead of 8 that each meet another sector.
template <class R>
__device__ __forceinline__ typename R::Raw block_load(const void *p, int64_t at, int there, bool vec, typename R::Elem *turn) {
    const int lane = threadIdx.x & 31, n = there - 8 * lane;
    const typename R::Elem *q = static_cast<const typename R::Elem *>(p) + at;
    if (vec && n >= 8) return *reinterpret_cast<const typename R::Raw *>(q + 8 * lane);
    if (vec) {
        if (n <= 0) return R::zero();
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? (uint32_t)q[8 * lane + i] : 0u;
        return R::of(v);
    }
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 32 * i + lane < there ? (uint32_t)q[32 * i + lane] : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) turn[32 * i + lane] = (typename R::Elem)v[i];
    __syncwarp();
    const typename R::Raw r = *reinterpret_cast<const typename R::Raw *>(turn + 8 * lane);
    __syncwarp();
    return r;
}
template <class R>
__device__ __forceinline__ void block_store(void *p, int64_t at, int there, bool vec, typename R::Elem *turn, const typename R::Raw &r) {
    const int lane = threadIdx.x & 31, n = there - 8 * lane;
    typename R::Elem *q = static_cast<typename R::Elem *>(p) + at;
    if (vec) {
        if (n >= 8) *reinterpret_cast<typename R::Raw *>(q + 8 * lane) = r;
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i < n) q[8 * lane + i] = R::element(r, i);
        return;
    }
    *reinterpret_cast<typename R::Raw *>(turn + 8 * lane) = r;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) if (32 * i + lane < there) q[32 * i + lane] = turn[32 * i + lane];
    __syncwarp();
}

// 8 weights of any type from column `at` on, n of which exist
__device__ __forceinline__ void weights8(const void *w, int kind, bool vec, int64_t at, int n, float o[8]) {
    if (kind == ZS_DTYPE_FP32) {
        const float *q = static_cast<const float *>(w) + at;
        if (vec && n >= 8) RowF32::floats(*reinterpret_cast<const RowF32::Raw *>(q), o);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = i < n ? q[i] : 0.0f;
        return;
    }
    const uint16_t *q = static_cast<const uint16_t *>(w) + at;
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0;
    uint4 r = make_uint4(0, 0, 0, 0);
    if (vec && n >= 8) r = *reinterpret_cast<const uint4 *>(q);
    else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? (uint32_t)q[i] : 0u;
        r = pack8(v);
    }
    if (kind == ZS_DTYPE_FP16) RowFP16::floats(r, o);
    else RowBF16::floats(r, o);
}

// of the 256 columns from `at` on, how many exist (0 and less: none)
__device__ __forceinline__ int part(int64_t cols, int64_t at) { return (int)max((int64_t)-1, min((int64_t)256, cols - at)); }

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

// Paired products and sums.  A paired sum of a paired product would be fused
// with it in spite of both roundings, so such a sum is written as a product with
// a 1 that the compiler does not know, plus the other.
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return f2pack(x, x); }

// A row's pair over the lanes of a warp; the same in all of them.
__device__ __forceinline__ void warp_pair(float &hi, float &lo) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float h2 = __shfl_xor_sync(0xFFFFFFFFu, hi, off), l2 = __shfl_xor_sync(0xFFFFFFFFu, lo, off);
        add22(hi, lo, h2, l2);
    }
}
// The pairs of four rows at once: halves of the warp keep two rows each, then
// quarters one; afterwards lane l has row l / 8.
__device__ __forceinline__ void warp_pair4(float (&hi)[4], float (&lo)[4]) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, odd = lane & 8;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float h = __shfl_xor_sync(0xFFFFFFFFu, up ? hi[k] : hi[2 + k], 16), l = __shfl_xor_sync(0xFFFFFFFFu, up ? lo[k] : lo[2 + k], 16);
        if (up) {
            hi[k] = hi[2 + k];
            lo[k] = lo[2 + k];
        }
        add22(hi[k], lo[k], h, l);
    }
    const float h = __shfl_xor_sync(0xFFFFFFFFu, odd ? hi[0] : hi[1], 8), l = __shfl_xor_sync(0xFFFFFFFFu, odd ? lo[0] : lo[1], 8);
    if (odd) {
        hi[0] = hi[1];
        lo[0] = lo[1];
    }
    add22(hi[0], lo[0], h, l);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
        const float h2 = __shfl_xor_sync(0xFFFFFFFFu, hi[0], off), l2 = __shfl_xor_sync(0xFFFFFFFFu, lo[0], off);
        add22(hi[0], lo[0], h2, l2);
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

// codes of 8 values times inv
__device__ __forceinline__ uint32_t encode8(const float v[8], float inv) {
    float y[8];
    const f2 two = both(inv);
#pragma unroll
    for (int i = 0; i < 8; i += 2) f2unpack(mul2(f2pack(v[i], v[i + 1]), two), y[i], y[i + 1]);
    return e2m1x8(y);
}

// 8 values a lane, 4 neighbouring lanes a group along the row; y is 0 past the
// matrix.  `row` may lie past the matrix, in the tile of scales that holds it.
template <class R>
__device__ __forceinline__ void hold_rows(const NormHeld &h, int64_t row, int64_t col, const typename R::Raw &y) {
    const uint32_t byte = mx4_scale_byte(__float_as_uint(R::top4(y)) >> 23);
    float v[8];
    R::floats(y, v);
    const uint32_t word = byte == 255u ? 0u : encode8(v, byte == 255u ? 0.0f : mx4_inverse(byte));
    const int64_t g = col / MX4_GROUP;
    if (row < h.rows && g < mx4_groups(h.cols))
        *reinterpret_cast<uint32_t *>(h.r_codes + row * mx4_row_bytes(h.cols) + col / 2) = word;
    // the scales of a row's four groups lie side by side: one lane writes them
    uint32_t four = byte << (8 * (g & 3));
    four |= __shfl_xor_sync(0xFFFFFFFFu, four, 4);
    four |= __shfl_xor_sync(0xFFFFFFFFu, four, 8);
    if ((threadIdx.x & 15) == 0 && row < 128 * mx4_row_tiles(h.rows) && g < 4 * mx4_atoms(h.cols))
        *reinterpret_cast<uint32_t *>(h.r_scales + ((row >> 7) * mx4_atoms(h.cols) + (g >> 2)) * MX4_ATOM + mx4_in_atom((int)(row & 127), 0)) = four;
}

// 32 values of one column: the rows from 32 g on
__device__ __forceinline__ void hold_column(const NormHeld &h, int64_t g, int64_t col, float top, const float v[32]) {
    const uint32_t byte = mx4_scale_byte(__float_as_uint(top) >> 23);
    const float inv = byte == 255u ? 0.0f : mx4_inverse(byte);
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = byte == 255u ? 0u : encode8(v + 8 * j, inv);
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
    bool vec, vec_w;                 // every matrix has 16-byte aligned rows; so does the weight
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
    __shared__ __align__(16) typename R::Elem turns[WARPS][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % WPR;
    const int64_t rows = a.held.rows, cols = a.held.cols, row = (int64_t)blockIdx.x * ROWS + warp / WPR;
    const int blocks = NB > 0 ? NB : (int)((cols + 256 * WPR - 1) / (256 * WPR));
    const bool there = row < rows;
    typename R::Elem *turn = turns[warp];
    pdl_wait();
    pdl_trigger();
    auto input = [&](int b, float h[8]) {
        const int64_t c = 256 * (int64_t)(mine + WPR * b);
        const int n = there ? part(cols, c) : 0;
        R::floats(block_load<R>(a.x, row * a.ldx + c, n, a.vec, turn), h);
        if (!a.residual) return;
        float r[8];
        R::floats(block_load<R>(a.residual, row * a.ldr + c, n, a.vec, turn), r);
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
        const int64_t c = 256 * (int64_t)(mine + WPR * b);
        const int n = there ? part(cols, c) : 0;
        float v[8], w[8];
        if constexpr (NB > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h[b][i];
        } else {
            input(b, v);
        }
        if (a.sum) block_store<R>(a.sum, row * a.lds + c, n, a.vec, turn, R::rounded(v));
        weights8(a.w, a.w_kind, a.vec_w, c + 8 * lane, n - 8 * lane, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 8 * lane + i < n ? __fmul_rn(__fmul_rn(v[i], rstd), w[i]) : 0.0f;
        const typename R::Raw y = R::rounded(v);
        if (a.out) block_store<R>(a.out, row * a.ldo + c, n, a.vec, turn, y);
        if (a.held.r_codes) hold_rows<R>(a.held, row, c + 8 * lane, y);
    }
}

// ---------------------------------------------- 32 rows, shared by columns --

constexpr int TILE_ROWS = 32;
constexpr int TILE_COLS = 512;       // of 8 warps; K times as many of a CTA
constexpr int tile_smem(int k) { return TILE_ROWS * TILE_COLS * k * 4; }
constexpr int64_t TILE_MOST = 8 * 3 * TILE_COLS;     // columns that a cluster holds
constexpr int ROWS_EACH = TILE_ROWS / WARPS;         // rows of a warp, 512 columns of each

__device__ __forceinline__ void async16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void async_wait(int pending) {            // for all but the last `pending` groups; a constant where it is inlined
    if (pending >= 3) asm volatile("cp.async.wait_group 3;" : : : "memory");
    else if (pending == 2) asm volatile("cp.async.wait_group 2;" : : : "memory");
    else if (pending == 1) asm volatile("cp.async.wait_group 1;" : : : "memory");
    else asm volatile("cp.async.wait_group 0;" : : : "memory");
}

// A row of a tile in shared memory, 16 bits: as it is, a lane's 8 side by side;
// 32 bits: in each block of 256 pieces of four side by side over the lanes, so
// that no two lanes of a load meet in a bank.
template <class R>
struct TileRow {
    typename R::Elem *at;            // of a block of 256 columns
    __device__ __forceinline__ uint4 *piece(int lane, int half) const {
        return reinterpret_cast<uint4 *>(at + (R::SIZE == 2 ? 8 * lane : 128 * half + 4 * lane));
    }
    __device__ __forceinline__ typename R::Raw get() const {
        const int lane = threadIdx.x & 31;
        if constexpr (R::SIZE == 2) return *piece(lane, 0);
        else return {*piece(lane, 0), *piece(lane, 1)};
    }
    __device__ __forceinline__ void put(const typename R::Raw &r) const {
        const int lane = threadIdx.x & 31;
        if constexpr (R::SIZE == 2) *piece(lane, 0) = r;
        else {
            *piece(lane, 0) = r.a;
            *piece(lane, 1) = r.b;
        }
    }
    // the block of a matrix on its way here; `there` columns exist.  What a lane
    // gets is its own to read once its copies have landed (vec), or at once.
    __device__ __forceinline__ void fetch(const void *p, int64_t from, int there, bool vec, typename R::Elem *turn) const {
        const int lane = threadIdx.x & 31;
        if (vec && there - 8 * lane >= 8) {
            const typename R::Elem *q = static_cast<const typename R::Elem *>(p) + from + 8 * lane;
            async16(piece(lane, 0), q);
            if (R::SIZE == 4) async16(piece(lane, 1), q + 4);
        } else {
            put(block_load<R>(p, from, there, vec, turn));
        }
    }
};
__device__ __forceinline__ int column_at(int place) {        // the column of a 32-bit place, in its block of 256
    return 8 * ((place & 127) >> 2) + 4 * ((place >> 7) & 1) + (place & 3);
}

// What a cluster's CTAs tell one another: a pair for each row and 8 warps.
struct Exchange {
    float2 pairs[2][TILE_ROWS][4];
    double wides[TILE_ROWS][4];
};

// The form along the columns of a tile of 32 rows: a thread takes two columns
// (the two of a word of 16-bit values), and 32 rows of each.
template <class R, int K>
__device__ __forceinline__ void hold_tile(const NormHeld &h, int64_t rb, int64_t col0, const typename R::Elem *tile) {
    constexpr int PITCH = TILE_COLS * K;
    float v[32];
    if constexpr (R::SIZE == 2) {
        const uint32_t *from = reinterpret_cast<const uint32_t *>(tile) + threadIdx.x;
        uint32_t w[32], two = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = from[i * (PITCH / 2)];
#pragma unroll
        for (int i = 0; i < 32; ++i) max_two<typename R::Type>(two, w[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = R::Type::to_f32(j ? w[i] >> 16 : w[i] & 0xFFFFu);
            hold_column(h, rb, col0 + 2 * (int)threadIdx.x + j, R::Type::to_f32(j ? two >> 16 : two & 0xFFFFu), v);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int place = (int)threadIdx.x + j * (PITCH / 2);
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(tile[i * PITCH + place]);
#pragma unroll
            for (int i = 0; i < 32; i += 2) max_abs3(top, v[i], v[i + 1]);
            hold_column(h, rb, col0 + (place & ~255) + column_at(place & 255), top, v);
        }
    }
}

// A cluster of ceil(cols / (512 K)) CTAs takes 32 rows, a warp 4 of them, 512
// columns of each.  All of a warp's inputs are on their way to shared memory at
// once (what is in flight decides: with loads into registers, two rows at a
// time, 4096 x 4096 bf16 in both forms took 57 us).  The rows' sums of squares;
// the exchange; then the result in its own type in x's place, its form along the
// rows from registers (4 lanes a group), and through shared memory the one along
// the columns.  16 bits: x and the residual lie there and are added again for
// the result; 32 bits: their sum takes x's place.
template <class R, int K>
__global__ void __launch_bounds__(THREADS *K, K == 1 ? 3 : 1)
rms_tile_kernel(NormArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ Exchange ex;
    __shared__ float rstds[TILE_ROWS];
    __shared__ __align__(16) typename R::Elem turns[WARPS * K][256];
    constexpr int PITCH = TILE_COLS * K;
    constexpr bool TWO = R::SIZE == 2;               // both inputs in shared memory
    typename R::Elem *xs = reinterpret_cast<typename R::Elem *>(raw), *rs = xs + TILE_ROWS * PITCH;
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kk = warp / WARPS, rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int64_t rows = a.held.rows, cols = a.held.cols, rb = blockIdx.x / ranks, row0 = TILE_ROWS * rb;
    const int64_t col0 = (int64_t)rank * PITCH + TILE_COLS * kk;                         // of the warp
    const int there[2] = {part(cols, col0), part(cols, col0 + 256)};
    typename R::Elem *turn = turns[warp];
    auto row_at = [&](typename R::Elem *of, int i, int b) { return TileRow<R>{of + (warp % WARPS + WARPS * i) * PITCH + TILE_COLS * kk + 256 * b}; };
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i) {
        const int64_t row = row0 + warp % WARPS + WARPS * i;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int n = row < rows ? there[b] : 0;
            row_at(xs, i, b).fetch(a.x, row * a.ldx + col0 + 256 * b, n, a.vec, turn);
            if (TWO && a.residual) row_at(rs, i, b).fetch(a.residual, row * a.ldr + col0 + 256 * b, n, a.vec, turn);
        }
        asm volatile("cp.async.commit_group;" : : : "memory");
    }
    auto input = [&](int i, int b, int64_t row, f2 h[4]) {           // x + residual
        float v[8], q[8];
        R::floats(row_at(xs, i, b).get(), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = f2pack(v[2 * j], v[2 * j + 1]);
        if (!a.residual) return;
        if constexpr (TWO) R::floats(row_at(rs, i, b).get(), q);
        else R::floats(block_load<R>(a.residual, row * a.ldr + col0 + 256 * b, row < rows ? there[b] : 0, a.vec, turn), q);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = add2(h[j], f2pack(q[2 * j], q[2 * j + 1]));
    };
    float hi[ROWS_EACH], lo[ROWS_EACH];
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i) {
        const int64_t row = row0 + warp % WARPS + WARPS * i;
        async_wait(ROWS_EACH - 1 - i);
        f2 h[2][4];
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            input(i, b, row, h[b]);
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f2unpack(h[b][j], v[2 * j], v[2 * j + 1]);
                max_abs3(top, v[2 * j], v[2 * j + 1]);
            }
            if (a.residual) {
                block_store<R>(a.sum, row * a.lds + col0 + 256 * b, row < rows ? there[b] : 0, a.vec, turn, R::rounded(v));
                if (!TWO) row_at(xs, i, b).put(R::rounded(v));
            }
        }
        Dot d;
        const bool ok = d.begin<2>(top, top);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) d.add(h[b][j], h[b][j]);
        d.end(hi[i], lo[i]);
        if (!ok) hi[i] = __uint_as_float(0x7F800000u);
    }
    warp_pair4(hi, lo);
    if ((lane & 7) == 0) ex.pairs[0][warp % WARPS + WARPS * (lane >> 3)][kk] = make_float2(hi[0], lo[0]);
    cluster.sync();
    float all = 0.0f, rest = 0.0f;
    if (threadIdx.x < TILE_ROWS) {
        for (int q = 0; q < ranks; ++q) {
            const Exchange *other = cluster.map_shared_rank(&ex, q);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float2 p = other->pairs[0][threadIdx.x][k];
                add22(all, rest, p.x, p.y);
            }
        }
        rstds[threadIdx.x] = rstd_of(all, rest, a.mean, a.eps);
    }
    // the sum as the result is made from it: the residual is added again where it lies beside x
    auto total = [&](int i, int b, int64_t row, f2 h[4]) {
        if constexpr (TWO) {
            input(i, b, row, h);
        } else {
            float v[8];
            R::floats(row_at(xs, i, b).get(), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = f2pack(v[2 * j], v[2 * j + 1]);
        }
    };
    // too large for float32's squares (or not finite): in 64 bits; every CTA of
    // the cluster has seen the same sums and comes here, or none does
    if (__syncthreads_or(!finite_f32(all))) {
#pragma unroll 1
        for (int i = 0; i < ROWS_EACH; ++i) {
            double s = 0.0;
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                f2 h[4];
                total(i, b, row0 + warp % WARPS + WARPS * i, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x, y;
                    f2unpack(h[j], x, y);
                    s = __dadd_rn(s, __dadd_rn(__dmul_rn((double)x, (double)x), __dmul_rn((double)y, (double)y)));
                }
            }
            s = warp_double(s);
            if (lane == 0) ex.wides[warp % WARPS + WARPS * i][kk] = s;
        }
        cluster.sync();
        if (threadIdx.x < TILE_ROWS && !finite_f32(all)) {
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
        float w[8];
        weights8(a.w, a.w_kind, a.vec_w, c + 8 * lane, there[b] - 8 * lane, w);
#pragma unroll 2
        for (int i = 0; i < ROWS_EACH; ++i) {
            const int64_t row = row0 + warp % WARPS + WARPS * i;
            const int n = row < rows ? there[b] : 0;
            f2 h[4];
            total(i, b, row, h);
            const f2 rstd = both(rstds[warp % WARPS + WARPS * i]);
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) f2unpack(mul2(mul2(h[j], rstd), f2pack(w[2 * j], w[2 * j + 1])), v[2 * j], v[2 * j + 1]);
            if (n < 256) {
#pragma unroll
                for (int j = 0; j < 8; ++j) if (8 * lane + j >= n) v[j] = 0.0f;
            }
            const typename R::Raw y = R::rounded(v);
            if (a.out) block_store<R>(a.out, row * a.ldo + c, n, a.vec, turn, y);
            row_at(xs, i, b).put(y);
            if (a.held.r_codes) hold_rows<R>(a.held, row, c + 8 * lane, y);
        }
    }
    __syncthreads();
    hold_tile<R, K>(a.held, rb, (int64_t)rank * PITCH, xs);
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
    bool vec, vec_w;
    float minus_one;                 // -1, which the compiler does not know
    Mean mean;
    NormHeld held;
    int64_t row_blocks;
};

// As rms_tile_kernel, a cluster taking row blocks b, b + clusters, ...: a lane
// adds up its columns' part of dw over all of them.  Shared memory keeps both
// inputs of 16 bits; of 32 bits x alone, and dy is read again.
template <class R, int K>
__global__ void __launch_bounds__(THREADS *K, K == 1 ? 2 : 1)
rms_back_kernel(BackArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ Exchange ex;
    __shared__ float slopes[TILE_ROWS], rstds[TILE_ROWS];
    __shared__ __align__(16) typename R::Elem turns[WARPS * K][256];
    constexpr int PITCH = TILE_COLS * K;
    constexpr bool TWO = R::SIZE == 2;
    typename R::Elem *xs = reinterpret_cast<typename R::Elem *>(raw), *ys = xs + TILE_ROWS * PITCH;
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kk = warp / WARPS, rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int64_t rows = a.held.rows, cols = a.held.cols, col0 = (int64_t)rank * PITCH + TILE_COLS * kk;
    const int there[2] = {part(cols, col0), part(cols, col0 + 256)};
    typename R::Elem *turn = turns[warp];
    auto row_at = [&](typename R::Elem *of, int i, int b) { return TileRow<R>{of + (warp % WARPS + WARPS * i) * PITCH + TILE_COLS * kk + 256 * b}; };
    pdl_wait();
    pdl_trigger();
    f2 w[2][4], dw[2][4] = {};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float v[8];
        weights8(a.w, a.w_kind, a.vec_w, col0 + 256 * b + 8 * lane, there[b] - 8 * lane, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[b][j] = f2pack(v[2 * j], v[2 * j + 1]);
    }
    int turns_taken = 0;
    for (int64_t rb = blockIdx.x / ranks; rb < a.row_blocks; rb += gridDim.x / ranks, turns_taken ^= 1) {
        const int64_t row0 = TILE_ROWS * rb;
#pragma unroll
        for (int i = 0; i < ROWS_EACH; ++i) {
            const int64_t row = row0 + warp % WARPS + WARPS * i;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int n = row < rows ? there[b] : 0;
                row_at(xs, i, b).fetch(a.x, row * a.ldx + col0 + 256 * b, n, a.vec, turn);
                if (TWO) row_at(ys, i, b).fetch(a.dy, row * a.lddy + col0 + 256 * b, n, a.vec, turn);
            }
            asm volatile("cp.async.commit_group;" : : : "memory");
        }
        auto gradient = [&](int i, int b, int64_t row, f2 g[4]) {
            float v[8];
            if constexpr (TWO) R::floats(row_at(ys, i, b).get(), v);
            else R::floats(block_load<R>(a.dy, row * a.lddy + col0 + 256 * b, row < rows ? there[b] : 0, a.vec, turn), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = f2pack(v[2 * j], v[2 * j + 1]);
        };
        float hi[ROWS_EACH], lo[ROWS_EACH];
#pragma unroll
        for (int i = 0; i < ROWS_EACH; ++i) {
            const int64_t row = row0 + warp % WARPS + WARPS * i;
            const f2 rstd = both(row < rows ? a.rstd[row] : 0.0f);
            async_wait(ROWS_EACH - 1 - i);
            f2 g[2][4], x[2][4];
            float tg = 0.0f, tx = 0.0f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float v[8];
                gradient(i, b, row, g[b]);
                R::floats(row_at(xs, i, b).get(), v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[b][j] = f2pack(v[2 * j], v[2 * j + 1]);
                    dw[b][j] = fma2(g[b][j], mul2(x[b][j], rstd), dw[b][j]);
                    g[b][j] = mul2(g[b][j], w[b][j]);
                    float p, q;
                    f2unpack(g[b][j], p, q);
                    max_abs3(tg, p, q);
                    max_abs3(tx, v[2 * j], v[2 * j + 1]);
                }
            }
            Dot d;
            if (d.begin<2>(tg, tx)) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) d.add(g[b][j], x[b][j]);
                d.end(hi[i], lo[i]);
            } else {                                 // far outside of any gradient's range: in 64 bits
                double s = 0.0;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float p, q, u, v;
                        f2unpack(g[b][j], p, q);
                        f2unpack(x[b][j], u, v);
                        s = __dadd_rn(s, __dadd_rn(__dmul_rn((double)p, (double)u), __dmul_rn((double)q, (double)v)));
                    }
                hi[i] = (float)s;
                lo[i] = finite_f32(hi[i]) ? (float)(s - (double)hi[i]) : 0.0f;
            }
        }
        warp_pair4(hi, lo);
        if ((lane & 7) == 0) ex.pairs[turns_taken][warp % WARPS + WARPS * (lane >> 3)][kk] = make_float2(hi[0], lo[0]);
        cluster.sync();
        if (threadIdx.x < TILE_ROWS) {
            float all = 0.0f, rest = 0.0f;
            for (int q = 0; q < ranks; ++q) {
                const Exchange *other = cluster.map_shared_rank(&ex, q);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 p = other->pairs[turns_taken][threadIdx.x][k];
                    add22(all, rest, p.x, p.y);
                }
            }
            const float rstd = row0 + threadIdx.x < rows ? a.rstd[row0 + threadIdx.x] : 0.0f;
            rstds[threadIdx.x] = rstd;
            slopes[threadIdx.x] = slope_of(all, rest, a.mean, rstd);
        }
        __syncthreads();
        const f2 minus = both(a.minus_one);
#pragma unroll 2
        for (int i = 0; i < ROWS_EACH; ++i) {
            const int64_t row = row0 + warp % WARPS + WARPS * i;
            const f2 rstd = both(rstds[warp % WARPS + WARPS * i]), slope = both(slopes[warp % WARPS + WARPS * i]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int64_t c = col0 + 256 * b;
                const int n = row < rows ? there[b] : 0;
                float x[8], v[8];
                typename R::Raw q;
                if (a.residual) q = block_load<R>(a.residual, row * a.ldr + c, n, a.vec, turn);
                f2 g[4];
                gradient(i, b, row, g);
                R::floats(row_at(xs, i, b).get(), x);
                // (g w - x slope) rstd, each rounded
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f2unpack(mul2(fma2(mul2(f2pack(x[2 * j], x[2 * j + 1]), slope), minus, mul2(g[j], w[b][j])), rstd), v[2 * j], v[2 * j + 1]);
                if (a.residual) {
                    float r[8];
                    R::floats(q, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], r[j]);
                }
                if (n < 256) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) if (8 * lane + j >= n) v[j] = 0.0f;
                }
                const typename R::Raw y = R::rounded(v);
                block_store<R>(a.dx, row * a.ldd + c, n, a.vec, turn, y);
                if (a.held.c_codes) row_at(xs, i, b).put(y);
                if (a.held.r_codes) hold_rows<R>(a.held, row, c + 8 * lane, y);
            }
        }
        __syncthreads();
        if (a.held.c_codes) {
            hold_tile<R, K>(a.held, rb, (int64_t)rank * PITCH, xs);
            __syncthreads();
        }
    }
    // the 8 warps' parts of dw, in their order
    if (a.dw_parts) {
        float *tile = reinterpret_cast<float *>(raw);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) f2unpack(dw[b][j], v[2 * j], v[2 * j + 1]);
            TileRow<RowF32>{reinterpret_cast<uint32_t *>(tile + (warp % WARPS) * PITCH + TILE_COLS * kk + 256 * b)}.put(RowF32::rounded(v));
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
    __shared__ __align__(16) typename R::Elem turns[WARPS][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x, cols = a.held.cols;
    typename R::Elem *turn = turns[warp];
    pdl_wait();
    pdl_trigger();
    const float rstd = a.rstd[row];
    float hi = 0.0f, lo = 0.0f;
    auto inputs = [&](int64_t c, float g[8], float x[8]) {           // g: times the weight
        float w[8];
        const int n = part(cols, c);
        R::floats(block_load<R>(a.dy, row * a.lddy + c, n, a.vec, turn), g);
        R::floats(block_load<R>(a.x, row * a.ldx + c, n, a.vec, turn), x);
        weights8(a.w, a.w_kind, a.vec_w, c + 8 * lane, n - 8 * lane, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], w[j]);
    };
    for (int64_t c = 256 * warp; c < cols; c += 8 * THREADS) {
        float g[8], x[8], tg = 0.0f, tx = 0.0f;
        inputs(c, g, x);
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
    for (int64_t c = 256 * warp; c < cols; c += 8 * THREADS) {
        float v[8], x[8];
        const int n = part(cols, c);
        inputs(c, v, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fsub_rn(v[j], __fmul_rn(x[j], slope)), rstd);
        if (a.residual) {
            float q[8];
            R::floats(block_load<R>(a.residual, row * a.ldr + c, n, a.vec, turn), q);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], q[j]);
        }
        block_store<R>(a.dx, row * a.ldd + c, n, a.vec, turn, R::rounded(v));
    }
}
// Their part of dw: 2048 columns of the rows b, b + gridDim.y, ...
template <class R>
__global__ void __launch_bounds__(THREADS)
rms_back_weight_kernel(BackArgs a) {
    __shared__ __align__(16) typename R::Elem turns[WARPS][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cols = a.held.cols, c = 256 * ((int64_t)blockIdx.x * WARPS + warp);
    const int n = part(cols, c);
    pdl_wait();
    pdl_trigger();
    float dw[8] = {};
    for (int64_t row = blockIdx.y; row < a.held.rows; row += gridDim.y) {
        const float rstd = a.rstd[row];
        float v[8], x[8];
        R::floats(block_load<R>(a.dy, row * a.lddy + c, n, a.vec, turns[warp]), v);
        R::floats(block_load<R>(a.x, row * a.ldx + c, n, a.vec, turns[warp]), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = __fmaf_rn(v[j], __fmul_rn(x[j], rstd), dw[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) if (8 * lane + j < n) a.dw_parts[blockIdx.y * cols + c + 8 * lane + j] = dw[j];
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
    if (c < cols) {
        int i = warp;
        for (; i + 7 * WARPS < n; i += 8 * WARPS) {          // 8 loads in flight
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = parts[(i + j * WARPS) * cols + c];
#pragma unroll
            for (int j = 0; j < 8; ++j) s = __fadd_rn(s, v[j]);
        }
        for (; i < n; i += WARPS) s = __fadd_rn(s, parts[i * cols + c]);
    }
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

// Parts of dw: a number of the sizes alone, so that a sum has the same bits
// whatever forms are asked for.  256 of them keep scratch small and the GPU busy.
static int64_t back_parts(int64_t rows, int64_t cols) {
    const int64_t blocks = (rows + TILE_ROWS - 1) / TILE_ROWS, most = cols > TILE_MOST ? 64 : 256;
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
    if (vec) *vec = addr(p) % 16 == 0;
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
    bool vec, vec_w = true;
    zs_status r = check(m, rows, cols, dtype, &vec, fn);
    if (r) return r;
    if (sum && !residual) return zs_fail(ZS_EINVAL, "%s: sum without a residual is x itself", fn);
    if (!(eps >= 0.0f) || eps > 3e38f) return zs_fail(ZS_EINVAL, "%s: eps %g", fn, (double)eps);
    if ((r = check_held(r_codes, r_scales, "along rows", fn)) || (r = check_held(c_codes, c_scales, "along columns", fn))) return r;
    if (rows == 0 || cols == 0) {
        zs_clear_error();
        return ZS_OK;
    }
    if ((r = check_vector(weight, weight_dtype, true, &vec_w, "weight", fn)) || (r = check_vector(rstd, ZS_DTYPE_FP32, true, nullptr, "rstd", fn)))
        return r;
    if (!out && !r_codes && !c_codes) return zs_fail(ZS_EINVAL, "%s: no form of the result is asked for", fn);
    using namespace zsk;
    if (c_codes && cols > TILE_MOST && !out)
        return zs_fail(ZS_EINVAL, "%s: along the columns of more than %d columns needs out", fn, (int)TILE_MOST);
    NormArgs a;
    a.x = x; a.residual = residual; a.w = weight; a.sum = sum; a.out = out; a.rstd = rstd;
    a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldo = ldo;
    a.w_kind = weight_dtype; a.vec = vec; a.vec_w = vec_w; a.eps = eps; a.mean = mean_of(cols);
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
    bool vec, vec_w = true;
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
    if ((r = check_vector(weight, weight_dtype, true, &vec_w, "weight", fn)) || (r = check_vector(rstd, ZS_DTYPE_FP32, true, nullptr, "rstd", fn)))
        return r;
    if (dw && (!scratch || addr(scratch) % 16)) return zs_fail(ZS_EINVAL, "%s: scratch NULL or not 16-byte aligned", fn);
    using namespace zsk;
    const bool tiles = cols <= TILE_MOST;
    BackArgs a;
    a.dy = dy; a.x = x; a.w = weight; a.residual = residual; a.rstd = rstd; a.dx = dx; a.dw_parts = dw ? scratch : nullptr;
    a.lddy = lddy; a.ldx = ldx; a.ldr = ldr; a.ldd = lddx;
    a.w_kind = weight_dtype; a.vec = vec; a.vec_w = vec_w; a.minus_one = -1.0f; a.mean = mean_of(cols);
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
