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
// float32 pairs, good to 2^-37 of the magnitudes' sum at worst, and rstd is the
// float32 nearest to the formula's value but where that lies within 2^-38 of the
// middle of two.
//
// A result held along its columns needs 32 rows at a time, which no SM holds
// whole.  One kernel makes the rows' sums, another takes tiles of 32 rows by 512
// columns and reads the inputs again, from L2 as far as they lie there: 4096 x
// 4096 bf16 in both forms takes 36 us.  The backward pass, whose dx is always
// written, reads its inputs once and makes the forms from dx (41 us; by tiles 51,
// which rows of more than 8192 columns take).  Taking long matrices by as
// many rows as fit L2 costs more in the kernels' ends than it gains (backward
// pass of 16384 x 4096 bf16: 215 us by 64 MB, 186 by 128 MB, 161 whole), and the
// reverse order of tiles changes nothing (within 1 %).  Clusters that hold 32 rows and
// exchange their sums through distributed shared memory read once, but took 41
// us: 57 of them fit the GPU, and the 128 blocks of rows need three turns of all
// that lies between two barriers.
#include <atomic>
#include <limits>

#include "zs_launch.h"
#include "zs_mx4.cuh"

namespace zsk {

typedef unsigned long long f2;

constexpr float MOST_F32 = 3.402823466e38f;

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

// A lane's 8 of a block of 256 columns from p on, `there` of which exist (any
// integer), on their way.  VEC: rows are 16-byte aligned and whole pieces of 8.
// Otherwise lanes load neighbouring elements (8 loads of 2 or 4 bytes that share
// their sectors, instead of 8 that each meet another one), which the warp's turn
// (256 elements of shared memory) deals out once all of them are needed.
template <class R, bool VEC>
struct Load {
    typename R::Raw r;
    __device__ __forceinline__ Load() {}
    __device__ __forceinline__ Load(const typename R::Elem *p, int there) {
        const int lane = threadIdx.x & 31;
        r = 8 * lane < there ? *reinterpret_cast<const typename R::Raw *>(p + 8 * lane) : R::zero();
    }
    __device__ __forceinline__ typename R::Raw take(typename R::Elem *) const { return r; }
};
template <class R>
struct Load<R, false> {
    uint32_t v[8];
    __device__ __forceinline__ Load() {}
    __device__ __forceinline__ Load(const typename R::Elem *p, int there) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 32 * i + lane < there ? (uint32_t)p[32 * i + lane] : 0u;
    }
    __device__ __forceinline__ typename R::Raw take(typename R::Elem *turn) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 8; ++i) turn[32 * i + lane] = (typename R::Elem)v[i];
        __syncwarp();
        const typename R::Raw r = *reinterpret_cast<const typename R::Raw *>(turn + 8 * lane);
        __syncwarp();
        return r;
    }
};
template <class R, bool VEC>
__device__ __forceinline__ void block_store(typename R::Elem *p, int there, typename R::Elem *turn, const typename R::Raw &r) {
    const int lane = threadIdx.x & 31;
    if constexpr (VEC) {
        if (8 * lane < there) *reinterpret_cast<typename R::Raw *>(p + 8 * lane) = r;
    } else {
        *reinterpret_cast<typename R::Raw *>(turn + 8 * lane) = r;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) if (32 * i + lane < there) p[32 * i + lane] = turn[32 * i + lane];
        __syncwarp();
    }
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

// Blocks of 8 pairs that a lane adds to one accumulator: 4096 x 4096 bf16 whole
// 25.1 us, backward 28.8; with one block 25.8 and 29.5.
constexpr int RUN = 2;

// A sum of products a b as hi + lo.  The accumulator begins at 3 * 2^m, 2^m
// above the sum of the magnitudes, and so stays in [2^(m+1), 2^(m+2)); of
// squares at 2^m, and stays in [2^m, 2^(m+1)).  Then
//   s = a b + h;  d = h - s (exact);  e = a b + d (the rounding error of s)
// four paired instructions for two products.  2^m is at most 16 times the
// largest product (two blocks; from the factors' largest magnitudes, which may
// belong to different columns, it could be anything above), and at least 2^-100.
// Of two blocks: each e is at most 2^(m-23), rounded once itself, and 8 of them
// are added in float32: off by 25 2^(m-47) a half, 16 2^(m-47) more where the
// halves meet, together 2^-36.9 of the largest product; squares half of that.
template <bool SQUARES>
struct Dot {
    f2 h, l;
    float start;
    // of at most 8 N pairs with |a b| <= top, rounded; false: too large
    template <int N>
    __device__ __forceinline__ bool begin(float top) {
        static_assert(N <= RUN, "blocks");
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        constexpr int LOG = N == 1 ? 2 : 3;          // of the products of one half
        const int m = max(e + 1 + LOG, -100);
        const bool ok = e < 115;                     // infinities and NaN have 128
        start = __uint_as_float(!ok ? 0x7F800000u : SQUARES ? (uint32_t)(m + 127) << 23 : (uint32_t)(m + 1 + 127) << 23 | 0x400000u);
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
// The same of the pairs of a row's WPR warps, by lanes of one of them: fewer
// instructions than one pair after another in every lane (2048 x 8192 bf16
// backward 31 us, not 35), but a longer way for a row that waits for nothing else
// (4096 x 4096 bf16 forward along the rows 29 us, 27 one after another).
template <int WPR>
__device__ __forceinline__ void row_pair(float &hi, float &lo) {
#pragma unroll
    for (int off = 1; off < WPR; off <<= 1) {
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
    if (!(hi >= 1.1754944e-38f) || hi > 3e38f) return 0.0f;                 // summed in 64 bits instead
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
// rstd^2 mean(g x), by one rstd after the other: the square alone leaves float32
// where x is below 2^-63
__device__ __forceinline__ float slope_of(float hi, float lo, const Mean &mean, float rstd) {
    times(hi, lo, mean.hi, mean.lo);
    times(hi, lo, rstd, 0.0f);
    times(hi, lo, rstd, 0.0f);
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

// A warp's index in a form that the compiler knows to be the same in all lanes:
// what follows from it is then worked out once a warp.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0); }

// Where the values of a warp's block of 256 columns from `col` on, of the rows
// from `row` on, go in the form along the rows: worked out once, since offsets of
// 64 bits cost as much as the values do.
struct RowsOut {
    uint8_t *codes, *scales;         // of the lane's 8 columns
    int64_t bytes;                   // of a row of codes
    uint32_t in, writes;             // bit b: of this block and the next, the group exists; this lane writes its scale
    __device__ __forceinline__ RowsOut(const NormHeld &h, int64_t row, int64_t col) {
        const int lane = threadIdx.x & 31;
        bytes = mx4_row_bytes(h.cols);
        codes = h.r_codes + (row * bytes + col / 2) + 4 * lane;
        const int64_t atoms = mx4_atoms(h.cols), atom = col / (4 * MX4_GROUP);
        scales = h.r_scales + ((row >> 7) * atoms + atom) * MX4_ATOM + mx4_in_atom((int)(row & 127), 0) + MX4_ATOM * (lane >> 4) + ((lane >> 2) & 3);
        const int groups = (int)min((int64_t)16, mx4_groups(h.cols) - col / MX4_GROUP), left = row < 128 * mx4_row_tiles(h.rows) ? (int)min((int64_t)4, atoms - atom) : 0;
        in = ((lane >> 2) < groups ? 1u : 0u) | (8 + (lane >> 2) < groups ? 2u : 0u);
        writes = (lane & 3) ? 0u : ((lane >> 4) < left ? 1u : 0u) | (2 + (lane >> 4) < left ? 2u : 0u);
    }
    // y: 8 values a lane, 4 neighbouring lanes a group, 0 past the matrix; of the
    // row `down` below, inside the same 32, which exists or not
    template <class R>
    __device__ __forceinline__ void hold(const typename R::Raw &y, int down, int block, bool exists) const {
        const uint32_t byte = mx4_scale_byte(__float_as_uint(R::top4(y)) >> 23);
        float v[8];
        R::floats(y, v);
        const uint32_t word = byte == 255u ? 0u : encode8(v, byte == 255u ? 0.0f : mx4_inverse(byte));
        if ((in >> block & 1) && exists) *reinterpret_cast<uint32_t *>(codes + down * bytes + 128 * block) = word;
        if (writes >> block & 1) scales[16 * down + 2 * MX4_ATOM * block] = (uint8_t)byte;
    }
};

// 32 values of one column: the rows from 32 g on.  codes, scale: where they go, or NULL.
__device__ __forceinline__ void hold_column(uint8_t *codes, uint8_t *scale, float top, const float v[32]) {
    const uint32_t byte = mx4_scale_byte(__float_as_uint(top) >> 23);
    const float inv = byte == 255u ? 0.0f : mx4_inverse(byte);
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = byte == 255u ? 0u : encode8(v + 8 * j, inv);
    if (codes) *reinterpret_cast<uint4 *>(codes) = make_uint4(q[0], q[1], q[2], q[3]);
    if (scale) *scale = (uint8_t)byte;
}

// ------------------------------------------------------- forward, rows --

struct NormArgs {
    const void *x, *residual, *w;
    void *sum, *out;
    float *rstd;
    int64_t ldx, ldr, lds, ldo;
    int32_t w_kind;
    bool vec, vec_w;                 // every matrix has 16-byte aligned rows; so does the weight
    float eps, least;                // least: of least_sum
    Mean mean;
    NormHeld held;
};

// WPR warps take a row, 8 values a lane and block of 256 columns; a lane keeps
// its NB blocks (NB 0: more than registers hold, read again).  Bandwidth
// bounds many rows of 32 bits (4096 x 4096 along the rows: 34 us, 31 at a copy's
// rate); of 16 bits the issue of instructions (28 us, 16: 43 a value, issue slots
// 72 % busy, DRAM 42 %), and past 8192 columns the few rows that are in flight (2048
// x 16384: 50 us, 40); the way through the sum's exchange a few rows (24 x 4096
// bf16: 2.6 us in a graph).
template <class R, int WPR, int NB, bool VEC>
__global__ void __launch_bounds__(THREADS)
rms_rows_kernel(NormArgs a) {
    constexpr int ROWS = WARPS / WPR, KEEP = NB > 0 ? NB : 1;
    __shared__ float2 parts[WARPS];
    __shared__ double wides[WARPS];
    __shared__ __align__(16) typename R::Elem turns[VEC ? 1 : WARPS][VEC ? 8 : 256];
    const int lane = threadIdx.x & 31, warp = warp_index(), mine = warp % WPR;
    const int64_t rows = a.held.rows, cols = a.held.cols, row = (int64_t)blockIdx.x * ROWS + warp / WPR;
    const int blocks = NB > 0 ? NB : (int)((cols + 256 * WPR - 1) / (256 * WPR));
    const bool there = row < rows;
    typedef typename R::Elem Elem;
    Elem *turn = turns[VEC ? 0 : warp];
    const Elem *x = static_cast<const Elem *>(a.x) + row * a.ldx, *residual = static_cast<const Elem *>(a.residual) + row * a.ldr;
    Elem *sum = static_cast<Elem *>(a.sum) + row * a.lds, *out = static_cast<Elem *>(a.out) + row * a.ldo;
    auto column = [&](int b) { return 256 * (int64_t)(mine + WPR * b); };
    auto exist = [&](int b) { return there ? part(cols, column(b)) : 0; };
    pdl_wait();
    pdl_trigger();
    auto add = [&](const Load<R, VEC> &first, const Load<R, VEC> &second, float h[8]) {
        R::floats(first.take(turn), h);
        if (!a.residual) return;
        float r[8];
        R::floats(second.take(turn), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __fadd_rn(h[i], r[i]);
    };
    auto input = [&](int b, float h[8]) {
        const Load<R, VEC> first(x + column(b), exist(b)), second(residual + column(b), a.residual ? exist(b) : 0);
        add(first, second, h);
    };
    float h[KEEP][8];
    float hi = 0.0f, lo = 0.0f;
    auto square = [&](auto &v) {                     // of one or all blocks
        constexpr int ALL = sizeof(v) / 32, N = ALL < RUN ? ALL : RUN;
#pragma unroll
        for (int b0 = 0; b0 < ALL; b0 += N) {
            float top = 0.0f;
#pragma unroll
            for (int b = b0; b < b0 + N; ++b)
#pragma unroll
                for (int i = 0; i < 8; i += 2) max_abs3(top, v[b][i], v[b][i + 1]);
            Dot<true> d;
            const bool ok = d.template begin<N>(__fmul_rn(top, top));
#pragma unroll
            for (int b = b0; b < b0 + N; ++b)
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const f2 p = f2pack(v[b][i], v[b][i + 1]);
                    d.add(p, p);
                }
            float dh, dl;
            d.end(dh, dl);
            add22(hi, lo, ok ? dh : __uint_as_float(0x7F800000u), dl);
        }
    };
    if constexpr (NB > 0) {
        Load<R, VEC> first[KEEP], second[KEEP];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            first[b] = Load<R, VEC>(x + column(b), exist(b));
            second[b] = Load<R, VEC>(residual + column(b), a.residual ? exist(b) : 0);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) add(first[b], second[b], h[b]);
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
    // too large or too small for float32's squares (or not finite): in 64 bits
    const bool wide = !(hi >= a.least && hi <= MOST_F32);
    if (__syncthreads_or(wide)) {
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
        if (wide) rstd = rstd_of(s, (double)cols, a.eps);
    }
    if (there && mine == 0 && lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int b = 0; b < blocks; ++b) {
        const int64_t c = column(b);
        const int n = exist(b);
        float v[8], w[8];
        if constexpr (NB > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h[b][i];
        } else {
            input(b, v);
        }
        if (a.sum) block_store<R, VEC>(sum + c, n, turn, R::rounded(v));
        weights8(a.w, a.w_kind, a.vec_w, c + 8 * lane, n - 8 * lane, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 8 * lane + i < n ? __fmul_rn(__fmul_rn(v[i], rstd), w[i]) : 0.0f;
        const typename R::Raw y = R::rounded(v);
        if (a.out) block_store<R, VEC>(out + c, n, turn, y);
        if (a.held.r_codes) RowsOut(a.held, row, c).template hold<R>(y, 0, 0, there);
    }
}

// ------------------------------------------------- the sums of many rows --

// rstd of every row (h: x + residual), or of the backward pass c, rstd^2 times
// the mean of g x: WPR warps a row, two blocks of 256 columns of both inputs on
// their way while two are summed.  Neither bandwidth nor the issue of instructions
// alone bounds it: 4096 x 4096 bf16 takes 15 us from cold caches (10 at a copy's
// rate; DRAM 56 %, issue slots 44 % busy), 4096 x 12288 backward 44 (30; 58 and 64
// %).  VEC: rows are 16-byte aligned and whole pieces of 8.
struct SumArgs {
    const void *x, *other, *w;       // other: the residual or NULL; dy
    int64_t ldx, ldo, rows, cols;
    int32_t w_kind;
    bool vec_w;
    float eps, least;
    Mean mean;
    const float *rstd;               // of the backward pass
    float *result;                   // [rows]
};

template <class R, int WPR, bool BACK, bool VEC>
__global__ void __launch_bounds__(THREADS, R::SIZE == 2 ? 4 : 3)
rms_sums_kernel(SumArgs a) {
    constexpr int BLOCKS = 2;
    __shared__ float2 parts[WARPS];
    __shared__ double wides[WARPS];
    __shared__ __align__(16) typename R::Elem turns[VEC ? 1 : WARPS][VEC ? 8 : 256];
    const int lane = threadIdx.x & 31, warp = warp_index(), mine = warp % WPR;
    const int64_t row = (int64_t)blockIdx.x * (WARPS / WPR) + warp / WPR;
    const bool there = row < a.rows;
    typename R::Elem *turn = turns[VEC ? 0 : warp];
    const typename R::Elem *x = static_cast<const typename R::Elem *>(a.x) + row * a.ldx, *other = static_cast<const typename R::Elem *>(a.other) + row * a.ldo;
    pdl_wait();
    pdl_trigger();
    // block c: u v summed over its columns, u = v = h or u = g, v = x
    auto inputs = [&](const typename R::Raw &rx, const typename R::Raw &ro, int64_t c, int n, f2 u[4], f2 v[4]) {
        float x[8], o[8];
        R::floats(rx, x);
        R::floats(ro, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = f2pack(x[2 * j], x[2 * j + 1]);
        if constexpr (BACK) {
            float w[8];
            weights8(a.w, a.w_kind, a.vec_w, c + 8 * lane, n - 8 * lane, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = mul2(f2pack(o[2 * j], o[2 * j + 1]), f2pack(w[2 * j], w[2 * j + 1]));
        } else {
            if (a.other)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = add2(v[j], f2pack(o[2 * j], o[2 * j + 1]));
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = v[j];
        }
    };
    float hi = 0.0f, lo = 0.0f;
    Load<R, VEC> next_x[BLOCKS], next_o[BLOCKS];
    auto fetch = [&](int64_t c0) {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int64_t c = c0 + 256 * WPR * b;
            const int n = there ? part(a.cols, c) : 0;
            next_x[b] = Load<R, VEC>(x + c, n);
            next_o[b] = Load<R, VEC>(other + c, a.other ? n : 0);
        }
    };
    fetch(256 * mine);
#pragma unroll 1
    for (int64_t c0 = 256 * mine; c0 < a.cols; c0 += 256 * WPR * BLOCKS) {
        typename R::Raw rx[BLOCKS], ro[BLOCKS];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            rx[b] = next_x[b].take(turn);
            ro[b] = next_o[b].take(turn);
        }
        if (c0 + 256 * WPR * BLOCKS < a.cols) fetch(c0 + 256 * WPR * BLOCKS);
        f2 u[BLOCKS][4], v[BLOCKS][4];
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int64_t c = c0 + 256 * WPR * b;
            inputs(rx[b], ro[b], c, there ? part(a.cols, c) : 0, u[b], v[b]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p, q;
                f2unpack(BACK ? mul2(u[b][j], v[b][j]) : v[b][j], p, q);
                max_abs3(top, p, q);
            }
        }
        Dot<!BACK> d;
        const bool ok = d.template begin<BLOCKS>(BACK ? top : __fmul_rn(top, top));
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) d.add(u[b][j], v[b][j]);
        float dh, dl;
        d.end(dh, dl);
        add22(hi, lo, ok ? dh : __uint_as_float(0x7F800000u), dl);
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
    const float given = BACK && there ? a.rstd[row] : 0.0f;
    float result = BACK ? slope_of(hi, lo, a.mean, given) : rstd_of(hi, lo, a.mean, a.eps);
    // too large for float32's products, squares too small (or not finite): in 64 bits
    const bool wide = !((BACK ? fabsf(hi) : hi) >= a.least && (BACK ? fabsf(hi) : hi) <= MOST_F32);
    if (__syncthreads_or(wide)) {
        double s = 0.0;
#pragma unroll 1
        for (int64_t c = 256 * mine; c < a.cols; c += 256 * WPR) {
            const int n = there ? part(a.cols, c) : 0;
            const typename R::Raw rx = Load<R, VEC>(x + c, n).take(turn), ro = Load<R, VEC>(other + c, a.other ? n : 0).take(turn);
            f2 u[4], v[4];
            inputs(rx, ro, c, n, u, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p, q, y, z;
                f2unpack(u[j], p, q);
                f2unpack(v[j], y, z);
                s = __dadd_rn(s, __dadd_rn(__dmul_rn((double)p, (double)y), __dmul_rn((double)q, (double)z)));
            }
        }
        s = warp_double(s);
        if (lane == 0) wides[warp] = s;
        __syncthreads();
        s = 0.0;
        for (int k = 0; k < WPR; ++k) s = __dadd_rn(s, wides[warp - mine + k]);
        if (wide) {
            if (BACK) result = (float)__dmul_rn(__ddiv_rn(s, (double)a.cols), __dmul_rn((double)given, (double)given));
            else result = rstd_of(s, (double)a.cols, a.eps);
        }
    }
    if (there && mine == 0 && lane == 0) a.result[row] = result;
}

// --------------------------------------------- tiles of 32 rows, 512 columns --

constexpr int TILE_ROWS = 32, TILE_COLS = 512;
constexpr int ROWS_EACH = TILE_ROWS / WARPS;         // rows of a warp

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
    // a lane's 8 on their way here: its own to read once the copies have landed
    __device__ __forceinline__ void fetch(const typename R::Elem *q, bool exists) const {
        const int lane = threadIdx.x & 31;
        if (!exists) return put(R::zero());
        async16(piece(lane, 0), q);
        if (R::SIZE == 4) async16(piece(lane, 1), q + 4);
    }
    // neighbouring elements, for the whole warp to read after its __syncwarp()
    __device__ __forceinline__ void put(const Load<R, false> &l) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 32 * i + (threadIdx.x & 31);
            at[R::SIZE == 2 ? c : 128 * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3)] = (typename R::Elem)l.v[i];
        }
    }
};
__device__ __forceinline__ int column_at(int place) {        // the column of a 32-bit place, in its block of 256
    return 8 * ((place & 127) >> 2) + 4 * ((place >> 7) & 1) + (place & 3);
}

// The form along the columns of a tile: a thread takes two columns (the two of a
// word of 16-bit values), and 32 rows of each.
template <class R>
__device__ __forceinline__ void hold_tile(const NormHeld &h, int64_t rb, int64_t col0, const typename R::Elem *tile) {
    const int64_t bytes = mx4_row_bytes(h.rows), atoms = mx4_atoms(h.rows), most = 128 * mx4_row_tiles(h.cols);
    const bool in = rb < mx4_groups(h.rows);
    auto column = [&](int64_t col, float top, const float v[32]) {
        hold_column(in && col < h.cols ? h.c_codes + col * bytes + 16 * rb : nullptr,
                    col < most ? h.c_scales + ((col >> 7) * atoms + (rb >> 2)) * MX4_ATOM + mx4_in_atom((int)(col & 127), (int)(rb & 3)) : nullptr, top, v);
    };
    float v[32];
    if constexpr (R::SIZE == 2) {
        const uint32_t *from = reinterpret_cast<const uint32_t *>(tile) + threadIdx.x;
        uint32_t w[32], two = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = from[i * (TILE_COLS / 2)];
#pragma unroll
        for (int i = 0; i < 32; ++i) max_two<typename R::Type>(two, w[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = R::Type::to_f32(j ? w[i] >> 16 : w[i] & 0xFFFFu);
            column(col0 + 2 * (int)threadIdx.x + j, R::Type::to_f32(j ? two >> 16 : two & 0xFFFFu), v);
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
            const int place = (int)threadIdx.x + j * (TILE_COLS / 2);
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(tile[i * TILE_COLS + place]);
#pragma unroll
            for (int i = 0; i < 32; i += 2) max_abs3(top, v[i], v[i + 1]);
            column(col0 + (place & ~255) + column_at(place & 255), top, v);
        }
    }
}

// A warp's share of a matrix: 4 rows, 8 apart, and two blocks of 256 columns.
template <class R, bool VEC>
struct Share {
    typename R::Elem *at;
    int64_t step;
    __device__ __forceinline__ Share(const void *p, int64_t ld, int64_t row, int64_t col)
        : at(static_cast<typename R::Elem *>(const_cast<void *>(p)) + (row * ld + col)), step(8 * ld) {}
    __device__ __forceinline__ typename R::Elem *of(int i, int b) const { return at + i * step + 256 * b; }
    // `there`: of the block's 256 columns, how many exist
    __device__ __forceinline__ Load<R, VEC> load(int i, int b, int there) const { return Load<R, VEC>(of(i, b), there); }
    __device__ __forceinline__ void store(int i, int b, int there, typename R::Elem *turn, const typename R::Raw &r) const {
        block_store<R, VEC>(of(i, b), there, turn, r);
    }
    __device__ __forceinline__ void fetch(const TileRow<R> &to, int i, int b, int there) const {
        const int lane = threadIdx.x & 31;
        if constexpr (VEC) to.fetch(of(i, b) + 8 * lane, 8 * lane < there);
        else to.put(load(i, b, there));
    }
    // y with nothing past the matrix
    static __device__ __forceinline__ typename R::Raw cut(const float v[8], int there) {
        const int lane = threadIdx.x & 31;
        typename R::Raw y = R::rounded(v);
        if (there >= 256) return y;
        if (VEC) return 8 * lane >= there ? R::zero() : y;
        float u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 8 * lane + j >= there ? 0.0f : v[j];
        return R::rounded(u);
    }
};

// Bytes of shared memory: inputs of 16 bits lie there (x, and the residual; of
// the backward pass x, dy and what reaches the stream), of 32 bits x alone.
template <class R>
constexpr int tile_smem(bool back) { return TILE_ROWS * TILE_COLS * (R::SIZE == 4 ? 4 : back ? 6 : 4); }
template <class R>
constexpr int tile_ctas(bool back) { return R::SIZE == 4 || !back ? 3 : 2; }         // an SM

// The result of a tile, rstd being known: a warp takes 4 rows, and all of its
// inputs are on their way to shared memory at once.  The new stream; the result
// in its own type in x's place, its form along the rows from registers (4 lanes
// a group), and through shared memory the one along the columns.  4096 x 4096
// bf16 from cold caches: 27 us, 30 instructions a value, issue slots 57 % busy and
// warps waiting for their first inputs.  (Tiles of 256 columns by 4 warps: within
// 2 %.  Greatest magnitudes by one instruction instead of two: the same.)
template <class R, bool VEC>
__global__ void __launch_bounds__(THREADS, tile_ctas<R>(false))
rms_tile_kernel(NormArgs a, int col_blocks) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ __align__(16) typename R::Elem turns[VEC ? 1 : WARPS][VEC ? 8 : 256];
    constexpr bool TWO = R::SIZE == 2;               // both inputs in shared memory
    const int lane = threadIdx.x & 31, warp = warp_index();
    const int64_t rb = blockIdx.x / col_blocks, row0 = TILE_ROWS * rb, col0 = (int64_t)(blockIdx.x % col_blocks) * TILE_COLS;
    const int64_t rows = a.held.rows, cols = a.held.cols;
    const int exist = (int)min((int64_t)TILE_ROWS, max((int64_t)0, rows - row0)), first = part(cols, col0), second = part(cols, col0 + 256);
    typename R::Elem *turn = turns[VEC ? 0 : warp];
    typename R::Elem *xs = reinterpret_cast<typename R::Elem *>(raw), *mine = xs + warp * TILE_COLS, *mine_r = mine + TILE_ROWS * TILE_COLS;
    auto there = [&](int i, int b) { return warp + WARPS * i >= exist ? 0 : b ? second : first; };
    auto place = [&](typename R::Elem *of, int i, int b) { return TileRow<R>{of + WARPS * i * TILE_COLS + 256 * b}; };
    const Share<R, VEC> x(a.x, a.ldx, row0 + warp, col0), residual(a.residual, a.ldr, row0 + warp, col0), sum(a.sum, a.lds, row0 + warp, col0),
        out(a.out, a.ldo, row0 + warp, col0);
    const RowsOut rows_out(a.held, row0 + warp, col0);
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            x.fetch(place(mine, i, b), i, b, there(i, b));
            if (TWO && a.residual) residual.fetch(place(mine_r, i, b), i, b, there(i, b));
        }
        asm volatile("cp.async.commit_group;" : : : "memory");
    }
    if (!VEC) __syncwarp();
    float rstds[ROWS_EACH];
    f2 w[2][4];
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i) rstds[i] = warp + WARPS * i < exist ? a.rstd[row0 + warp + WARPS * i] : 0.0f;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float v[8];
        weights8(a.w, a.w_kind, a.vec_w, col0 + 256 * b + 8 * lane, (b ? second : first) - 8 * lane, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[b][j] = f2pack(v[2 * j], v[2 * j + 1]);
    }
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i) {
        async_wait(ROWS_EACH - 1 - i);
        const f2 rstd = both(rstds[i]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int n = there(i, b);
            f2 h[4];
            float v[8];
            R::floats(place(mine, i, b).get(), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = f2pack(v[2 * j], v[2 * j + 1]);
            if (a.residual) {
                float q[8];
                if constexpr (TWO) R::floats(place(mine_r, i, b).get(), q);
                else R::floats(residual.load(i, b, n).take(turn), q);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = add2(h[j], f2pack(q[2 * j], q[2 * j + 1]));
                    f2unpack(h[j], v[2 * j], v[2 * j + 1]);
                }
                sum.store(i, b, n, turn, R::rounded(v));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) f2unpack(mul2(mul2(h[j], rstd), w[b][j]), v[2 * j], v[2 * j + 1]);
            const typename R::Raw y = Share<R, VEC>::cut(v, n);
            if (a.out) out.store(i, b, n, turn, y);
            place(mine, i, b).put(y);
            if (a.held.r_codes) rows_out.template hold<R>(y, WARPS * i, b, warp + WARPS * i < exist);
        }
    }
    __syncthreads();
    hold_tile<R>(a.held, rb, col0, xs);
}

// ------------------------------------------------------------- backward --

struct BackArgs {
    const void *dy, *x, *w, *residual;
    const float *rstd;
    void *dx;
    float *dw_parts;                 // [parts][parts_pitch(cols)], or NULL
    float *slopes;                   // [rows]
    int64_t lddy, ldx, ldr, ldd, parts;
    int32_t w_kind;
    bool vec, vec_w;
    float minus_one;                 // -1, which the compiler does not know
    Mean mean;
    NormHeld held;
};

__host__ __device__ constexpr int64_t parts_pitch(int64_t cols) { return (cols + TILE_COLS - 1) / TILE_COLS * TILE_COLS; }

// The same of the backward pass, c being known: a CTA takes its 512 columns of
// the row blocks b, b + parts, ... and adds up their part of dw.  Bandwidth bounds
// it: 4096 x 12288 bf16 takes 61 us from cold caches, 59 at a copy's rate.  (The
// residual by plain loads and three CTAs an SM took 4 % more.)
template <class R, bool VEC>
__global__ void __launch_bounds__(THREADS, tile_ctas<R>(true))
rms_back_kernel(BackArgs a, int64_t blocks, int col_blocks) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ __align__(16) typename R::Elem turns[VEC ? 1 : WARPS][VEC ? 8 : 256];
    constexpr bool TWO = R::SIZE == 2;
    constexpr int TILE = TILE_ROWS * TILE_COLS;
    const int lane = threadIdx.x & 31, warp = warp_index();
    const int64_t part_index = blockIdx.x / col_blocks, col0 = (int64_t)(blockIdx.x % col_blocks) * TILE_COLS;
    const int64_t rows = a.held.rows, cols = a.held.cols;
    const int first = part(cols, col0), second = part(cols, col0 + 256);
    typename R::Elem *turn = turns[VEC ? 0 : warp];
    typename R::Elem *xs = reinterpret_cast<typename R::Elem *>(raw), *mine = xs + warp * TILE_COLS;
    auto place = [&](int matrix, int i, int b) { return TileRow<R>{mine + matrix * TILE + WARPS * i * TILE_COLS + 256 * b}; };
    pdl_wait();
    pdl_trigger();
    f2 w[2][4], dw[2][4] = {};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float v[8];
        weights8(a.w, a.w_kind, a.vec_w, col0 + 256 * b + 8 * lane, (b ? second : first) - 8 * lane, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[b][j] = f2pack(v[2 * j], v[2 * j + 1]);
    }
    const f2 minus = both(a.minus_one);
    for (int64_t rb = part_index; rb < blocks; rb += a.parts) {
        const int64_t row0 = TILE_ROWS * rb;
        const int exist = (int)min((int64_t)TILE_ROWS, max((int64_t)0, rows - row0));
        auto there = [&](int i, int b) { return warp + WARPS * i >= exist ? 0 : b ? second : first; };
        const Share<R, VEC> x(a.x, a.ldx, row0 + warp, col0), dy(a.dy, a.lddy, row0 + warp, col0), residual(a.residual, a.ldr, row0 + warp, col0),
            dx(a.dx, a.ldd, row0 + warp, col0);
        const RowsOut rows_out(a.held, row0 + warp, col0);
#pragma unroll
        for (int i = 0; i < ROWS_EACH; ++i) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                x.fetch(place(0, i, b), i, b, there(i, b));
                if (TWO) dy.fetch(place(1, i, b), i, b, there(i, b));
                if (TWO && a.residual) residual.fetch(place(2, i, b), i, b, there(i, b));
            }
            asm volatile("cp.async.commit_group;" : : : "memory");
        }
        if (!VEC) __syncwarp();
        float rstds[ROWS_EACH], slopes[ROWS_EACH];
#pragma unroll
        for (int i = 0; i < ROWS_EACH; ++i) {
            const bool in = warp + WARPS * i < exist;
            rstds[i] = in ? a.rstd[row0 + warp + WARPS * i] : 0.0f;
            slopes[i] = in ? a.slopes[row0 + warp + WARPS * i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < ROWS_EACH; ++i) {
            async_wait(ROWS_EACH - 1 - i);
            const f2 rstd = both(rstds[i]), slope = both(slopes[i]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int n = there(i, b);
                float u[8], v[8];
                if constexpr (TWO) R::floats(place(1, i, b).get(), v);
                else R::floats(dy.load(i, b, n).take(turn), v);
                R::floats(place(0, i, b).get(), u);
                // dw; (g w - x slope) rstd, each rounded
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 g = f2pack(v[2 * j], v[2 * j + 1]), z = f2pack(u[2 * j], u[2 * j + 1]);
                    dw[b][j] = fma2(g, mul2(z, rstd), dw[b][j]);
                    f2unpack(mul2(fma2(mul2(z, slope), minus, mul2(g, w[b][j])), rstd), v[2 * j], v[2 * j + 1]);
                }
                if (a.residual) {
                    float r[8];
                    if constexpr (TWO) R::floats(place(2, i, b).get(), r);
                    else R::floats(residual.load(i, b, n).take(turn), r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], r[j]);
                }
                const typename R::Raw y = Share<R, VEC>::cut(v, n);
                dx.store(i, b, n, turn, y);
                if (a.held.c_codes) place(0, i, b).put(y);
                if (a.held.r_codes) rows_out.template hold<R>(y, WARPS * i, b, warp + WARPS * i < exist);
            }
        }
        if (a.held.c_codes) {
            __syncthreads();
            hold_tile<R>(a.held, rb, col0, xs);
            __syncthreads();
        }
    }
    // the 8 warps' parts of dw, in their order
    if (!a.dw_parts) return;
    __syncthreads();
    float *tile = reinterpret_cast<float *>(raw);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f2unpack(dw[b][j], v[2 * j], v[2 * j + 1]);
        TileRow<RowF32>{reinterpret_cast<uint32_t *>(tile + warp * TILE_COLS + 256 * b)}.put(RowF32::rounded(v));
    }
    __syncthreads();
    for (int at = threadIdx.x; at < TILE_COLS; at += THREADS) {
        float s = tile[at];
#pragma unroll
        for (int i = 1; i < WARPS; ++i) s = __fadd_rn(s, tile[i * TILE_COLS + at]);
        a.dw_parts[part_index * parts_pitch(cols) + col0 + (at & ~255) + column_at(at & 255)] = s;
    }
}

// The backward pass in one reading, dx as it is: WPR warps take a
// row, two blocks of 256 columns each, from its sum to its result.  VEC: the next
// rows' x, dy and residual are on their way to shared memory, a lane's 8 to a
// place of its own (32 bits: two fours, each beside the neighbours', since a
// warp's copies then read whole sectors; 4096 x 4096: 49 us, not 76); other rows
// go through registers.  A CTA takes WARPS / WPR
// rows at a time and leaves its part of dw.  4096 x 4096 bf16: 29 us with
// rms_weight_kernel (20 at a copy's rate; the two readings of rms_back_kernel: 39),
// fp32 48 (40; 107), 1333 x 1490 fp16 10 (20).  Bandwidth bounds rows of 32 bits; of
// 16 bits nothing is full (34 instructions a value, issue slots 51 % and DRAM 49 %
// busy): four warps a scheduler wait for one another's sums.  A few rows wait for
// the way through their sum.
// Three CTAs an SM spill; a ring of four rows takes as long as one of three.
__host__ __device__ constexpr int whole_cta_warps(int wpr) { return wpr > WARPS ? wpr : WARPS; }
__host__ __device__ constexpr int whole_ctas(int wpr) { return wpr > WARPS ? 1 : 2; }             // an SM
template <class R>
__host__ __device__ constexpr int whole_depth() { return R::SIZE == 4 ? 2 : 3; }                  // rows of the ring
template <class R>
__host__ __device__ constexpr int whole_stage(int wpr) { return 3 * 2 * 8 * R::SIZE * 32 * whole_cta_warps(wpr); }
// bytes of shared memory: the ring, and the warps' parts of dw in its place
template <class R, bool VEC>
constexpr int whole_smem(int wpr) { return VEC ? whole_depth<R>() * whole_stage<R>(wpr) : whole_cta_warps(wpr) * 2 * 256 * 4; }

template <class R, int WPR, bool VEC>
__global__ void __launch_bounds__(32 * whole_cta_warps(WPR), whole_ctas(WPR))
rms_back_rows_kernel(BackArgs a) {
    constexpr int NB = 2, W = whole_cta_warps(WPR), ROWS = W / WPR, DEPTH = whole_depth<R>(), STAGE = whole_stage<R>(WPR), PIECES = R::SIZE / 2;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ float2 parts[2][W];
    __shared__ double wides[W];
    __shared__ __align__(16) typename R::Elem turns[VEC ? 1 : W][VEC ? 8 : 256];
    typedef typename R::Elem Elem;
    const int lane = threadIdx.x & 31, warp = warp_index(), mine = warp % WPR, sub = warp / WPR;
    const int64_t rows = a.held.rows, cols = a.held.cols, step = a.parts * ROWS;
    Elem *turn = turns[VEC ? 0 : warp];
    auto column = [&](int b) { return 256 * (mine + WPR * b); };
    const int exist[NB] = {part(cols, column(0)), part(cols, column(1))};
    constexpr bool FOURS = VEC && R::SIZE == 4;
    auto four = [&](int h) { return FOURS ? 128 * h + 4 * lane : 8 * lane + 4 * h; };       // the first column of half h of a lane's 8
    pdl_wait();
    pdl_trigger();
    f2 w[NB][4], dw[NB][4] = {};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float v[8];
        if constexpr (FOURS) {
            float u[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                weights8(a.w, a.w_kind, false, column(b) + four(h), min(4, exist[b] - four(h)), u);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = u[j];
            }
        } else {
            weights8(a.w, a.w_kind, a.vec_w, column(b) + 8 * lane, exist[b] - 8 * lane, v);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[b][j] = f2pack(v[2 * j], v[2 * j + 1]);
    }
    const f2 minus = both(a.minus_one);
    const int64_t first = (int64_t)blockIdx.x * ROWS + sub;
    int64_t ahead = first;                           // the next row of the ring
    int slot = 0, place = 0;
    uint8_t *own = raw + 16 * threadIdx.x;
    auto piece = [&](int at, int matrix, int b, int h) { return own + at + ((matrix * NB + b) * PIECES + h) * (16 * 32 * W); };
    auto copy = [&] {
        if constexpr (VEC) {
            if (ahead < rows) {
                const Elem *from[3] = {static_cast<const Elem *>(a.x) + ahead * a.ldx, static_cast<const Elem *>(a.dy) + ahead * a.lddy,
                                       static_cast<const Elem *>(a.residual) + ahead * a.ldr};
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < PIECES; ++h)
                        if (four(h) < exist[b])
#pragma unroll
                            for (int k = 0; k < 3; ++k)
                                if (k < 2 || a.residual) async16(piece(slot, k, b, h), from[k] + column(b) + four(h));
            }
            asm volatile("cp.async.commit_group;" : : : "memory");
            slot = slot + STAGE == DEPTH * STAGE ? 0 : slot + STAGE;
            ahead += step;
        }
    };
    for (int i = 0; i < DEPTH - 1; ++i) copy();
    int at = 0;                                      // of the two places for the warps' sums
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < rows; row0 += step, at ^= 1) {
        const int64_t row = row0 + sub;
        const bool there = row < rows;
        const float given = there ? a.rstd[row] : 0.0f;
        typename R::Raw held[3][VEC ? 1 : NB];       // x, dy and the residual of a row that is not VEC
        if constexpr (VEC) {
            copy();
            async_wait(DEPTH - 1);
        } else {
            Load<R, false> l[3][NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int n = there ? exist[b] : 0;
                l[0][b] = Load<R, false>(static_cast<const Elem *>(a.x) + row * a.ldx + column(b), n);
                l[1][b] = Load<R, false>(static_cast<const Elem *>(a.dy) + row * a.lddy + column(b), n);
                l[2][b] = Load<R, false>(static_cast<const Elem *>(a.residual) + row * a.ldr + column(b), a.residual ? n : 0);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 3; ++k) held[k][b] = l[k][b].take(turn);
        }
        auto values = [&](int k, int b, float v[8]) {
            if constexpr (VEC) {
                uint4 r[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
#pragma unroll
                for (int h = 0; h < PIECES; ++h)
                    if (there && four(h) < exist[b]) r[h] = *reinterpret_cast<const uint4 *>(piece(place, k, b, h));
                if constexpr (R::SIZE == 2) R::floats(r[0], v);
                else R::floats({r[0], r[1]}, v);
            } else {
                R::floats(held[k][b], v);
            }
        };
        // dy and x of block b in pairs
        auto inputs = [&](int b, f2 u[4], f2 v[4]) {
            float x[8], y[8];
            values(0, b, x);
            values(1, b, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = f2pack(x[2 * j], x[2 * j + 1]);
                u[j] = f2pack(y[2 * j], y[2 * j + 1]);
            }
        };
        f2 g[NB][4], z[NB][4];
        float top = 0.0f, hi, lo;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            inputs(b, g[b], z[b]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p, q;
                f2unpack(mul2(mul2(g[b][j], w[b][j]), z[b][j]), p, q);
                max_abs3(top, p, q);
            }
        }
        {
            Dot<false> d;
            const bool ok = d.template begin<NB>(top);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) d.add(mul2(g[b][j], w[b][j]), z[b][j]);
            d.end(hi, lo);
            if (!ok) hi = __uint_as_float(0x7F800000u);
        }
        warp_pair(hi, lo);
        // too large for float32's products (or not finite): the row in 64 bits
        bool wide = !(fabsf(hi) <= 1e30f);           // sixteen such sums are finite
        int any = wide;
        if (WPR > 1) {
            if (lane == 0) parts[at][warp] = make_float2(hi, lo);
            any = __syncthreads_or(wide);
            const float2 p = parts[at][warp - mine + lane % WPR];
            hi = p.x;
            lo = p.y;
            wide = __any_sync(0xFFFFFFFFu, !(fabsf(hi) <= 1e30f));
            row_pair<WPR>(hi, lo);
        }
        float c = slope_of(hi, lo, a.mean, given);
        if (any) {
            double s = 0.0;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float p, q, x, y;
                    f2unpack(mul2(g[b][j], w[b][j]), p, q);
                    f2unpack(z[b][j], x, y);
                    s = __dadd_rn(s, __dadd_rn(__dmul_rn((double)p, (double)x), __dmul_rn((double)q, (double)y)));
                }
            s = warp_double(s);
            if (WPR > 1) {
                if (lane == 0) wides[warp] = s;
                __syncthreads();
                s = 0.0;
                for (int k = 0; k < WPR; ++k) s = __dadd_rn(s, wides[warp - mine + k]);
            }
            if (wide) c = (float)__dmul_rn(__ddiv_rn(s, (double)cols), __dmul_rn((double)given, (double)given));
        }
        const f2 rstd = both(given), slope = both(c);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dw[b][j] = fma2(g[b][j], mul2(z[b][j], rstd), dw[b][j]);
                f2unpack(mul2(fma2(mul2(z[b][j], slope), minus, mul2(g[b][j], w[b][j])), rstd), v[2 * j], v[2 * j + 1]);
            }
            if (a.residual) {
                float r[8];
                values(2, b, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], r[j]);
            }
            Elem *to = static_cast<Elem *>(a.dx) + row * a.ldd + column(b);
            if constexpr (FOURS) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (there && four(h) < exist[b]) *reinterpret_cast<float4 *>(to + four(h)) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            } else {
                block_store<R, VEC>(to, there ? exist[b] : 0, turn, R::rounded(v));
            }
        }
        place = place + STAGE == DEPTH * STAGE ? 0 : place + STAGE;
    }
    if (!a.dw_parts) return;
    // the rows' parts of dw, in their order
    __syncthreads();
    float *tile = reinterpret_cast<float *>(raw);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f2unpack(dw[b][j], v[2 * j], v[2 * j + 1]);
        TileRow<RowF32>{reinterpret_cast<uint32_t *>(tile + (warp * NB + b) * 256)}.put(RowF32::rounded(v));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < WPR * NB * 256; i += 32 * W) {
        const int block = i >> 8, from = (block % WPR * NB + block / WPR) * 256 + (i & 255), col = 256 * block + (FOURS ? i & 255 : column_at(i & 255));
        float s = tile[from];
#pragma unroll
        for (int k = 1; k < ROWS; ++k) s = __fadd_rn(s, tile[k * (WPR * NB * 256) + from]);
        if (col < cols) a.dw_parts[blockIdx.x * parts_pitch(cols) + col] = s;
    }
}

// dw from its parts: 32 columns a CTA, 32 warps' shares of the parts, then a
// tree over the shares.
constexpr int WEIGHT_WARPS = 32;
constexpr int MOST_WHOLE_PARTS = 152, MOST_TILE_PARTS = 256;     // the former for each CTA of an SM, two at most
constexpr int WEIGHT_LOADS = (2 * MOST_WHOLE_PARTS + WEIGHT_WARPS - 1) / WEIGHT_WARPS;
static_assert(WEIGHT_LOADS * WEIGHT_WARPS >= MOST_TILE_PARTS, "parts of dw");
__global__ void __launch_bounds__(32 * WEIGHT_WARPS)
rms_weight_kernel(const float *parts, int n, int64_t cols, int64_t pitch, void *dw, int kind) {
    __shared__ float share[WEIGHT_WARPS][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = 32 * (int64_t)blockIdx.x;
    pdl_wait();
    pdl_trigger();
    float s = 0.0f;
    if (c0 + lane < cols) {
        float v[WEIGHT_LOADS];                       // all in flight
#pragma unroll
        for (int j = 0; j < WEIGHT_LOADS; ++j) v[j] = warp + j * WEIGHT_WARPS < n ? parts[(warp + j * WEIGHT_WARPS) * pitch + c0 + lane] : 0.0f;
#pragma unroll
        for (int j = 0; j < WEIGHT_LOADS; ++j) s = __fadd_rn(s, v[j]);
    }
    share[warp][lane] = s;
    __syncthreads();
    s = share[lane][warp];                           // a column a warp
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, off));
    const int64_t c = c0 + warp;
    if (lane != 0 || c >= cols) return;
    if (kind == ZS_DTYPE_FP32) static_cast<float *>(dw)[c] = s;
    else static_cast<uint16_t *>(dw)[c] = (uint16_t)(kind == ZS_DTYPE_FP16 ? FP16T::from_f32(s) : BF16T::from_f32(s));
}

// ------------------------------------------------------------- launches --

// The sum of squares below which a row is summed in 64 bits: the errors that
// float32's least number leaves (2^-149 a square) would count, unless eps hides them.
// With an eps that may take the mean out of float32, every row.
static float least_sum(int64_t cols, float eps) {
    return eps < 0x1p-100f ? (float)cols * 0x1p-100f : eps > 0x1p120f ? std::numeric_limits<float>::infinity() : 0.0f;
}

template <class R, int WPR, int NB>
static cudaError_t rows_launch(const NormArgs &a, int64_t grid_rows, cudaStream_t s) {
    const int64_t per = WARPS / WPR, grid = (grid_rows + per - 1) / per;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) { return launch_dependent(kernel, (unsigned)grid, THREADS, 0, 1, s, a); };
    return a.vec && a.held.cols % 8 == 0 ? go(rms_rows_kernel<R, WPR, NB, true>) : go(rms_rows_kernel<R, WPR, NB, false>);
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

template <class R, bool BACK, bool VEC>
static cudaError_t sums_launch(const SumArgs &a, cudaStream_t s) {
    // as many warps a row as give every SM 16 (with 32, 4096 x 4096 bf16 took 2 us
    // more); of the backward pass rows are wider than 8192 here, and their number decides
    const int64_t rows = a.rows;
    auto go = [&](auto kernel, int wpr) { return launch_dependent(kernel, (unsigned)((rows * wpr + WARPS - 1) / WARPS), THREADS, 0, 1, s, a); };
    if (rows >= 2432 || a.cols <= 1024) return go(rms_sums_kernel<R, 1, BACK, VEC>, 1);
    if (rows >= 1216 || a.cols <= 2048) return go(rms_sums_kernel<R, 2, BACK, VEC>, 2);
    if (rows >= 608 || a.cols <= 4096) return go(rms_sums_kernel<R, 4, BACK, VEC>, 4);
    return go(rms_sums_kernel<R, 8, BACK, VEC>, 8);
}

template <class... P>
static cudaError_t tile_launch(void (*kernel)(P...), std::atomic<bool> (&set)[64], int smem, int64_t grid, int threads, cudaStream_t s, const P &...args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    return launch_dependent(kernel, (unsigned)grid, threads, smem, 1, s, args...);
}

static int col_blocks_of(int64_t cols) { return (int)((cols + TILE_COLS - 1) / TILE_COLS); }

template <class R, bool VEC>
static cudaError_t norm_tiles(const NormArgs &a, cudaStream_t s) {
    static std::atomic<bool> set[64];
    const int64_t rows = a.held.rows, cols = a.held.cols;
    const int cb = col_blocks_of(cols);
    const SumArgs sums = {a.x, a.residual, nullptr, a.ldx, a.ldr, rows, cols, 0, true, a.eps, a.least, a.mean, nullptr, a.rstd};
    const cudaError_t e = sums_launch<R, false, VEC>(sums, s);
    return e != cudaSuccess ? e : tile_launch(rms_tile_kernel<R, VEC>, set, tile_smem<R>(false), 4 * mx4_atoms(rows) * cb, THREADS, s, a, cb);
}

// Parts of dw, by tiles and by whole rows: numbers of the sizes alone, so that a
// sum has the same bits every time, whatever forms are asked for.  256 of the
// former keep scratch small and the GPU busy; the latter are a CTA each, one or two an SM.
static int64_t back_parts(int64_t rows) {
    const int64_t blocks = (rows + TILE_ROWS - 1) / TILE_ROWS;
    return blocks < MOST_TILE_PARTS ? blocks : MOST_TILE_PARTS;
}

// One reading of a row: as many warps as give each lane 16 columns.
constexpr int64_t WHOLE_MOST = 8192;                 // columns
static int whole_warps(int64_t cols) { return cols <= 512 ? 1 : cols <= 2048 ? 4 : cols <= 4096 ? 8 : 16; }
static int64_t whole_parts(int64_t rows, int64_t cols) {
    const int64_t per = cols <= 2048 ? WARPS / whole_warps(cols) : 1, n = (rows + per - 1) / per;
    const int64_t most = MOST_WHOLE_PARTS * whole_ctas(whole_warps(cols));
    return n < most ? n : most;
}

// Floats of parts that a matrix of these sizes or of smaller ones can leave, by
// any type and alignment.  A wide matrix leaves fewer parts than a narrower one
// that is read in one go, and may then need less: so the most that each of the
// ways asks for up to this width, which grows with either size.
static int64_t scratch_parts(int64_t rows, int64_t cols) {
    int64_t most = 0;
    for (const int64_t edge : {(int64_t)4096, WHOLE_MOST}) {       // up to here parts grow with the width
        const int64_t c = cols < edge ? cols : edge, n = whole_parts(rows, c) * parts_pitch(c);
        if (n > most) most = n;
    }
    const int64_t n = back_parts(rows) * parts_pitch(cols);
    return n > most ? n : most;
}

template <class R, int WPR, bool VEC>
static cudaError_t whole_launch(BackArgs &a, cudaStream_t s) {
    static std::atomic<bool> set[64];
    a.parts = whole_parts(a.held.rows, a.held.cols);
    return tile_launch(rms_back_rows_kernel<R, WPR, VEC>, set, whole_smem<R, VEC>(WPR), a.parts, 32 * whole_cta_warps(WPR), s, a);
}
template <class R, bool VEC>
static cudaError_t back_whole(BackArgs &a, cudaStream_t s) {
    switch (whole_warps(a.held.cols)) {
        case 1: return whole_launch<R, 1, VEC>(a, s);
        case 4: return whole_launch<R, 4, VEC>(a, s);
        case 8: return whole_launch<R, 8, VEC>(a, s);
        default: return whole_launch<R, 16, VEC>(a, s);
    }
}

template <class R, bool VEC>
static cudaError_t back_tiles(const BackArgs &a, cudaStream_t s) {
    static std::atomic<bool> set[64];
    const int64_t rows = a.held.rows, cols = a.held.cols;
    const int64_t blocks = a.held.c_codes ? 4 * mx4_atoms(rows) : a.held.r_codes ? 4 * mx4_row_tiles(rows) : (rows + TILE_ROWS - 1) / TILE_ROWS;
    const int cb = col_blocks_of(cols);
    const SumArgs sums = {a.x, a.dy, a.w, a.ldx, a.lddy, rows, cols, a.w_kind, a.vec_w, 0.0f, 0.0f, a.mean, a.rstd, a.slopes};
    const cudaError_t e = sums_launch<R, true, VEC>(sums, s);
    return e != cudaSuccess ? e : tile_launch(rms_back_kernel<R, VEC>, set, tile_smem<R>(true), a.parts * cb, THREADS, s, a, blocks, cb);
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
    NormArgs a;
    a.x = x; a.residual = residual; a.w = weight; a.sum = sum; a.out = out; a.rstd = rstd;
    a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldo = ldo;
    a.w_kind = weight_dtype; a.vec = vec; a.vec_w = vec_w; a.eps = eps; a.least = least_sum(cols, eps); a.mean = mean_of(cols);
    a.held = {static_cast<uint8_t *>(r_codes), static_cast<uint8_t *>(r_scales), static_cast<uint8_t *>(c_codes), static_cast<uint8_t *>(c_scales), rows, cols};
    const cudaStream_t s = (cudaStream_t)stream;
    if (!c_codes) {
        // the rows' tiles of scales have to be whole
        const int64_t grid_rows = r_codes ? 128 * mx4_row_tiles(rows) : rows;
        return cuda_status(by_type(dtype, [&](auto t) { return rows_of<decltype(t)>(a, grid_rows, s); }), fn);
    }
    return cuda_status(by_type(dtype, [&](auto t) {
        return a.vec && cols % 8 == 0 ? norm_tiles<decltype(t), true>(a, s) : norm_tiles<decltype(t), false>(a, s);
    }), fn);
}

zs_status zs_rms_norm_scratch(int64_t rows, int64_t cols, int64_t *bytes) {
    const char *fn = "zs_rms_norm_scratch";
    if (!bytes) return zs_fail(ZS_EINVAL, "%s: NULL result", fn);
    if (rows < 0 || cols < 0 || rows >= MOST || cols >= MOST)
        return zs_fail(ZS_EINVAL, "%s: %lld x %lld out of range", fn, (long long)rows, (long long)cols);
    *bytes = rows > 0 && cols > 0 ? 4 * (zsk::scratch_parts(rows, cols) + rows) : 0;
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
    if (!scratch || addr(scratch) % 16) return zs_fail(ZS_EINVAL, "%s: scratch NULL or not 16-byte aligned", fn);
    using namespace zsk;
    BackArgs a;
    a.dy = dy; a.x = x; a.w = weight; a.residual = residual; a.rstd = rstd; a.dx = dx;
    // one reading where a row fits the registers, and the forms from dx, which then
    // lies in L2: 4096 x 4096 bf16 in both 41 us, by tiles 51; fp32 62 and 104; 4000 x
    // 4003 bf16 63 and 88; 300 x 1000 bf16 8 and 14; 16384 x 1024 bf16 52 and 51
    const bool whole = cols <= WHOLE_MOST;
    a.parts = whole ? 0 : back_parts(rows);     // 0: set with the launch
    a.dw_parts = dw ? scratch : nullptr;
    a.slopes = scratch + a.parts * parts_pitch(cols);
    a.lddy = lddy; a.ldx = ldx; a.ldr = ldr; a.ldd = lddx;
    a.w_kind = weight_dtype; a.vec = vec; a.vec_w = vec_w; a.minus_one = -1.0f; a.mean = mean_of(cols);
    a.held = {static_cast<uint8_t *>(r_codes), static_cast<uint8_t *>(r_scales), static_cast<uint8_t *>(c_codes),
              static_cast<uint8_t *>(c_scales), rows, cols};
    cudaError_t e = by_type(dtype, [&](auto t) {
        using R = decltype(t);
        const bool pieces = a.vec && cols % 8 == 0;
        if (whole) return pieces ? back_whole<R, true>(a, s) : back_whole<R, false>(a, s);
        return pieces ? back_tiles<R, true>(a, s) : back_tiles<R, false>(a, s);
    });
    if (e == cudaSuccess && dw)
        e = launch_dependent(rms_weight_kernel, (unsigned)((cols + 31) / 32), 32 * WEIGHT_WARPS, 0, 1, s, a.dw_parts, (int)a.parts, cols, parts_pitch(cols), dw, dw_dtype);
    if (e == cudaSuccess && whole && (r_codes || c_codes))
        return zs_mx4_quantize(dx, rows, cols, lddx, dtype, r_codes, r_scales, c_codes, c_scales, stream);
    return cuda_status(e, fn);
}

}  // extern "C"
