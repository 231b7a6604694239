// Adam(W) over a list of separate tensors in one launch, moments in 32 bits
// or in 8 (zs_build_tensors, zs_adam_tensors).
//
// The host cuts every tensor into chunks and writes one
// record per chunk, with the addresses already advanced to it, so that a CTA
// finds all it needs in one load whatever the number of tensors.
//
// 8-bit moments.  A block is 256 consecutive elements of a tensor (the last
// one may be short).  exp_avg is held as e4m3 codes, exp_avg_sq as the e4m3
// codes of its square root: the root has half the octaves, so that e4m3's 18
// octaves span what 36 would of the square itself.  A block has one float32
// scale for each, 2^(floor(log2 max) - 7): e4m3 is a floating format, so a
// power of two costs no precision, makes scaling exact and leaves its largest
// value in [128, 256), which no rounding takes past 448.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <new>
#include <utility>

#include "zs_launch.h"
#include "zs_tensors.cuh"

// Elements per CTA: a list long enough to fill the GPU takes the chunk at
// which its kernel was fastest (32-bit moments 8192: 833 us for 202M
// elements; 8-bit 6144: 470 us rounded to nearest, against 488 at 4096 and at
// 8192); a short one takes small chunks, spread over more SMs.
constexpr int CHUNK32 = 8192, CHUNK8 = 6144, CHUNK_SHORT = 2048;
static_assert(CHUNK32 <= CHUNK_MOST && CHUNK8 <= CHUNK_MOST, "chunks");
constexpr int64_t SHORT_ELEMS = 304ll * CHUNK8;     // two chunks an SM
constexpr int STATE_BLOCK = 256;     // elements per scale: 8 a lane of one warp

namespace zsk {

struct Adam8C {
    float b1, b2, omb1, omb2, eps, wd, lr_wd, step_size, root, root_2_32;
    int adamw;
    uint32_t k0, k1, step;
    // the same and 1 twice, for the paired instructions
    struct { unsigned long long b1, b2, omb1, omb2, eps, wd, lr_wd, step_size, root_2_32, one, minus_one; } two;
};

__device__ __forceinline__ void load8f(const float *a, float o[8]) {
    const float4 x = *reinterpret_cast<const float4 *>(a);
    const float4 y = *reinterpret_cast<const float4 *>(a + 4);
    o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
    o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
}
__device__ __forceinline__ void store8f(float *a, const float o[8]) {
    *reinterpret_cast<float4 *>(a) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4 *>(a + 4) = make_float4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ uint16_t cast1(float p, bool fp16) {
    return (uint16_t)(fp16 ? FP16T::from_f32(p) : BF16T::from_f32(p));
}

// ------------------------------------------------------ 32-bit moments --
// 28 bytes an element with 16-bit gradients and a 16-bit copy; the update is
// adam_elem, so that a list over a plan's shards gives zs_adam_step's bits.
// Bandwidth bounds it: 202M elements in 833 us, 6.8 TB/s, the rate of a copy.
template <class G>
__global__ void __launch_bounds__(THREADS)
tensors32_kernel(const ZsChunk *chunks, AdamC c, const float *d_coef,
                 const int32_t *d_flags, bool fp16) {
    pdl_wait();
    pdl_trigger();
    const ZsChunk k = chunks[blockIdx.x];
    const float coef = d_coef ? *d_coef : 1.0f;
    if (d_flags && (*d_flags & ZS_SKIP_NONFINITE)) return;
    float *pm = static_cast<float *>(k.m), *pv = static_cast<float *>(k.v);
    uint16_t *param = static_cast<uint16_t *>(k.param);
    const int vec = k.tensor < 0 ? 0 : k.len & ~7;
    for (int x = 8 * threadIdx.x; x < vec; x += 8 * THREADS) {
        float g[8], p[8], m[8], v[8];
        G::load8(k.grad, x, g);
        load8f(k.master + x, p);
        load8f(pm + x, m);
        load8f(pv + x, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) adam_elem(p[i], m[i], v[i], g[i], coef, c);
        store8f(k.master + x, p);
        store8f(pm + x, m);
        store8f(pv + x, v);
        if (param) *reinterpret_cast<uint4 *>(param + x) = cast8(p, fp16);
    }
    for (int x = vec + threadIdx.x; x < k.len; x += THREADS) {
        float p = k.master[x], m = pm[x], v = pv[x];
        adam_elem(p, m, v, G::load1(k.grad, x), coef, c);
        k.master[x] = p;
        pm[x] = m;
        pv[x] = v;
        if (param) param[x] = cast1(p, fp16);
    }
}

// ------------------------------------------------------- 8-bit moments --

// Philox4x32 (Salmon, Moraes, Dror, Shaw 2011) with 7 rounds, the fewest
// that its authors found to pass every test of their batteries.
__device__ __forceinline__ void philox7(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1, uint32_t w[4]) {
#pragma unroll
    for (int r = 0; r < 7; ++r) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

// e4m3 codes of two floats, nearest even (lo in the low byte)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 codes -> float
__device__ __forceinline__ void e4m3_decode8(uint2 c, float o[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint16_t two = (uint16_t)((j < 2 ? c.x : c.y) >> (16 * (j & 1)));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h));
        o[2 * j] = f.x;
        o[2 * j + 1] = f.y;
    }
}

// a >= 0 (< 256) to a value of e4m3, up when its random bits say so: random
// is 16 r + 8 for 16 random bits r, the middle of the interval that they name,
// so the probability of the upper neighbour is a's place between the two, to
// 2^-16.  The equally spaced range below 2^-6 is shifted into the binade
// [2^-6, 2^-5), whose spacing is the same 2^-9.  Adding to the bits below the
// kept mantissa carries into it, and past it into the exponent, as rounding up
// does.  (2^-6 - a) 2^100, saturated, is 1 below 2^-6 and 0 from it on: fused
// products keep the comparison off the integer pipe, which is the busier one.
__device__ __forceinline__ float e4m3_dither(float a, uint32_t random) {
    float low;
    asm("fma.rn.sat.f32 %0, %1, 0fF1800000, 0f6E800000;" : "=f"(low) : "f"(a));     // -2^100, 2^94
    const uint32_t u = __float_as_uint(__fmaf_rn(low, 0.015625f, a)) + random;
    return __fmaf_rn(low, -0.015625f, __uint_as_float(u & 0xFFF00000u));
}

__device__ __forceinline__ bool finite_bits(float x) {
    return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// The e4m3 codes of 8 values x times inv (a power of two).  ROOT: x >= 0, and
// a positive value never gets code 0 (it divides the update).
template <bool ROOT, bool DITHER>
__device__ __forceinline__ uint2 encode8(const float x[8], float inv, const uint32_t random[8]) {
    constexpr float BIG = 1.2676506002282294e30f;    // 2^100: takes the smallest positive root past 2^-9
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn(x[i], inv);
        if (DITHER)
            y[i] = ROOT ? e4m3_dither(y[i], random[i]) : copysignf(e4m3_dither(fabsf(y[i]), random[i]), y[i]);
        if (ROOT) y[i] = fmaxf(y[i], fminf(__fmul_rn(x[i], BIG), 0.001953125f));   // 0 for 0
    }
    return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                      e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

// A block's largest magnitude, as bits (a NaN's if there is one), from 8
// values a lane.
__device__ __forceinline__ uint32_t block_top(const float x[8]) {
    float top = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
    return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top) & 0x7FFFFFFFu);
}

__device__ __forceinline__ void random8(int64_t elem, int32_t tensor, const Adam8C &c, uint32_t lo[8], uint32_t hi[8]) {
    const uint64_t q = (uint64_t)elem >> 2;
    const uint32_t t = (uint32_t)tensor & 0x7FFFFFFFu;
    uint32_t w[8];
    philox7((uint32_t)q, (uint32_t)(q >> 32), t, c.step, c.k0, c.k1, w);
    philox7((uint32_t)q | 1u, (uint32_t)(q >> 32), t, c.step, c.k0, c.k1, w + 4);    // q is even
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = (w[i] & 0xFFFFu) * 16u + 8u;
        hi[i] = (w[i] >> 16) * 16u + 8u;
    }
}

// Pairs of floats: the paired instructions round each half as the scalar ones
// do and issue once for two elements.  A paired sum of a paired product is
// fused with it in spite of both .rn, which would round once where the update
// rounds twice; so a sum is written as one operand times ONE, an argument that
// the compiler does not know, plus the other.
typedef unsigned long long f2;
__device__ __forceinline__ f2 both(float x) { return f2pack(x, x); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b, const Adam8C &c) { return fma2(a, c.two.one, b); }
__device__ __forceinline__ f2 sub2(f2 a, f2 b, const Adam8C &c) { return fma2(b, c.two.minus_one, a); }

// 2^32 sqrt(v) of two, correctly rounded and without a branch, so that a
// lane's roots overlap.  Markstein's correction of an approximate root s of
// w = 2^64 v: the residual w - s s is exact in one fused operation, and
// s + (w - s s) / (2 sqrt(w)) rounds as the root does.  2^64 keeps the
// residual of the smallest v among the normal numbers; zs_test_root compares
// it with the library's root on every v below 2^64.  Infinities and NaN give
// NaN, and so does v >= 2^64.
__device__ __forceinline__ f2 root_2_32(f2 v) {
    const f2 w = mul2(v, both(18446744073709551616.0f)), minus_w = mul2(v, both(-18446744073709551616.0f));
    float a, b;
    f2unpack(w, a, b);
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(fmaxf(a, 7.8886090522101181e-31f)));   // 2^-100: v = 0 gives 0
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(fmaxf(b, 7.8886090522101181e-31f)));
    const f2 y = f2pack(a, b), s = mul2(w, y);
    return fma2(fma2(s, s, minus_w), mul2(both(-0.5f), y), s);
}

constexpr uint32_t ROOT_END = 0x5F800000u;       // 2^64
__global__ void root_test_kernel(unsigned long long *bad) {
    unsigned long long mine = 0;
    for (uint32_t u = 2 * (blockIdx.x * blockDim.x + threadIdx.x); u < ROOT_END; u += 2 * gridDim.x * blockDim.x) {
        const float a = __uint_as_float(u), b = __uint_as_float(u + 1);
        float x, y;
        f2unpack(root_2_32(f2pack(a, b)), x, y);
        mine += (__float_as_uint(x) != __float_as_uint(__fmul_rn(__fsqrt_rn(a), 4294967296.0f))) +
                (__float_as_uint(y) != __float_as_uint(__fmul_rn(__fsqrt_rn(b), 4294967296.0f)));
    }
    if (mine) atomicAdd(bad, mine);
}

// a / b to 2 units in the last place, b normal or 0 (a root times at least 1,
// plus eps): without the scaling that other denominators need.
__device__ __forceinline__ float quick_quotient(float a, float b) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
    return __fmul_rn(a, y);
}

// New moment and square of one element; g: the gradient times coef (and the
// decay of Adam-L2), p: decayed (AdamW).
__device__ __forceinline__ void adam8_moments(float &p, float &m, float &v, float g, float r, float sm, float sr,
                                              float coef, const Adam8C &c) {
    float gi = __fmul_rn(g, coef);
    if (c.adamw)
        p = __fsub_rn(p, __fmul_rn(c.lr_wd, p));
    else
        gi = __fadd_rn(gi, __fmul_rn(c.wd, p));
    const float r0 = __fmul_rn(r, sr);
    m = __fadd_rn(__fmul_rn(c.b1, __fmul_rn(m, sm)), __fmul_rn(c.omb1, gi));
    v = __fadd_rn(__fmul_rn(c.b2, __fmul_rn(r0, r0)), __fmul_rn(c.omb2, __fmul_rn(gi, gi)));
}

// One block, any length and alignment, with moments that are not finite: such
// an element becomes a NaN code and does not count for the scale.
template <class G, bool DITHER>
__device__ __noinline__ void adam8_block(const ZsChunk *chunk, const Adam8C c, float coef, bool fp16, int b) {
    const ZsChunk k = *chunk;
    uint8_t *cm = static_cast<uint8_t *>(k.m), *cv = static_cast<uint8_t *>(k.v);
    uint16_t *param = static_cast<uint16_t *>(k.param);
    const int lane = threadIdx.x & 31, x = b * STATE_BLOCK + 8 * lane;
    const int n = min(8, k.len - x);             // of this lane, may be negative
    float m[8], r[8];
    const float sm = k.m_scale[b], sr = k.v_scale[b];
    uint2 qm = make_uint2(0, 0), qr = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = i < n ? cm[x + i] : 0u, d = i < n ? cv[x + i] : 0u;
        if (i < 4) { qm.x |= a << (8 * i); qr.x |= d << (8 * i); }
        else { qm.y |= a << (8 * i - 32); qr.y |= d << (8 * i - 32); }
    }
    e4m3_decode8(qm, m);
    e4m3_decode8(qr, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) {
            m[i] = r[i] = 0.0f;
            continue;
        }
        float p = k.master[x + i], v;
        adam8_moments(p, m[i], v, G::load1(k.grad, x + i), r[i], sm, sr, coef, c);
        r[i] = __fsqrt_rn(v);
        const float den = __fadd_rn(__fmul_rn(r[i], c.root), c.eps);
        p = __fsub_rn(p, __fmul_rn(c.step_size, quick_quotient(m[i], den)));
        k.master[x + i] = p;
        if (param) param[x + i] = cast1(p, fp16);
    }
    bool bad_m[8], bad_r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bad_m[i] = !finite_bits(m[i]);
        bad_r[i] = !finite_bits(r[i]);
        if (bad_m[i]) m[i] = 0.0f;
        if (bad_r[i]) r[i] = 0.0f;
    }
    const uint32_t fm = max(block_top(m) >> 23, 8u), fr = max(block_top(r) >> 23, 8u);
    uint32_t lo[8], hi[8];
    if (DITHER) random8(k.elem + x, k.tensor, c, lo, hi);
    qm = encode8<false, DITHER>(m, __uint_as_float((261u - fm) << 23), lo);
    qr = encode8<true, DITHER>(r, __uint_as_float((261u - fr) << 23), hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) continue;
        cm[x + i] = bad_m[i] ? 0x7F : (uint8_t)((i < 4 ? qm.x : qm.y) >> (8 * (i & 3)));
        cv[x + i] = bad_r[i] ? 0x7F : (uint8_t)((i < 4 ? qr.x : qr.y) >> (8 * (i & 3)));
    }
    if (lane == 0) {
        k.m_scale[b] = __uint_as_float((fm - 7u) << 23);
        k.v_scale[b] = __uint_as_float((fr - 7u) << 23);
    }
}

// Stages of a chunk in shared memory: GROUP blocks each, one a warp.
constexpr int STAGES8 = CHUNK8 / STATE_BLOCK / WARPS;
constexpr int STAGE_ELEMS = STATE_BLOCK * WARPS;
template <class G>
constexpr int SMEM8 = CHUNK8 * (G::SIZE + 4 + 1 + 1);
constexpr uint64_t BULK_NS = 1000000000ull;      // one wait gives up after 1 s

__device__ int g_tensors_wait_timeouts;          // waits that gave up

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :
                 : "r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A CTA has its whole chunk fetched by bulk copies at once, in stages of one
// block a warp; a warp then takes its block of each stage as it lands, 8
// consecutive elements a lane.  16 bytes an element with 16-bit gradients and
// a 16-bit copy: at the copy bandwidth that leaves about 85 instructions an
// element, so the arithmetic counts as much as the bytes, and the copies keep
// memory busy while every warp of the SM computes (loads into registers took
// 623 us and more for 202M elements).  Rounded to nearest 465 us, 7.0 TB/s;
// stochastically 491 us, 6.6 TB/s: there instructions bound it, 73 an element,
// 24 of them the random bits and their rounding (529 us with 81, before the
// estimates of the reciprocal and the root went without scaling; 3 or 5 CTAs an
// SM 520 us and more).  The quotient m / den is
// the quick one (its last two bits may be off: 2^-22 of one update, far below
// a rounding of p); the root is exact, since codes hang on it.
// give_up, for tests: the stage whose wait runs out (its barrier expects bytes
// that never come), or -1.
template <class G, bool DITHER>
__global__ void __launch_bounds__(THREADS, 4)
tensors8_kernel(const ZsChunk *chunks, Adam8C c, const float *d_coef,
                const int32_t *d_flags, bool fp16, int give_up) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[STAGES8];
    pdl_wait();
    pdl_trigger();
    const ZsChunk k = chunks[blockIdx.x];
    const float coef = d_coef ? *d_coef : 1.0f;
    if (d_flags && (*d_flags & ZS_SKIP_NONFINITE)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int full = k.tensor >= 0 ? k.len / STATE_BLOCK : 0;    // blocks of the vector path
    const uint32_t sg = smem_u32(smem), sp = sg + CHUNK8 * G::SIZE, sm = sp + CHUNK8 * 4, sr = sm + CHUNK8, bar = smem_u32(bars);
    if (threadIdx.x == 0 && full > 0) {
        for (int i = 0; i < STAGES8; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" : : "r"(bar + 8 * i) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" : : : "memory");
        for (int i = 0, at = 0; at < full * STATE_BLOCK; ++i, at += STAGE_ELEMS) {
            const uint32_t n = (uint32_t)min(STAGE_ELEMS, full * STATE_BLOCK - at);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" : : "r"(bar + 8 * i), "r"(n * (G::SIZE + 6) + (i == give_up ? 16 : 0)) : "memory");
            bulk_load(sg + at * G::SIZE, static_cast<const char *>(k.grad) + (int64_t)at * G::SIZE, n * G::SIZE, bar + 8 * i);
            bulk_load(sp + at * 4, k.master + at, n * 4, bar + 8 * i);
            bulk_load(sm + at, static_cast<const uint8_t *>(k.m) + at, n, bar + 8 * i);
            bulk_load(sr + at, static_cast<const uint8_t *>(k.v) + at, n, bar + 8 * i);
        }
    }
    // the warp's scales: block warp + 8 i in lane i
    float hm = 0.0f, hr = 0.0f;
    if (lane < STAGES8 && warp + WARPS * lane < full) {
        hm = k.m_scale[warp + WARPS * lane];
        hr = k.v_scale[warp + WARPS * lane];
    }
    __syncthreads();
    for (int i = 0, b = warp; b * STATE_BLOCK < k.len; ++i, b += WARPS) {
        if (b >= full) {
            adam8_block<G, DITHER>(chunks + blockIdx.x, c, coef, fp16, b);
            continue;
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_quick(bar + 8 * i, 0, BULK_NS))) {
            if (lane == 0) atomicAdd(&g_tensors_wait_timeouts, 1);
            mbar_wait_quick(bar + 8 * i, 0, BULK_NS);       // shared memory stays until the copies land
            continue;
        }
        const int x = b * STATE_BLOCK + 8 * lane;
        float g[8], p[8], m[8], r[8];
        G::shared8(sg + x * G::SIZE, g);
        floats4(lds16(sp + 4 * x), p);
        floats4(lds16(sp + 4 * x + 16), p + 4);
        e4m3_decode8(lds8(sm + x), m);
        e4m3_decode8(lds8(sr + x), r);
        const float scale_m = __shfl_sync(0xFFFFFFFFu, hm, i), scale_r = __shfl_sync(0xFFFFFFFFu, hr, i);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            f2 g2 = mul2(f2pack(g[e], g[e + 1]), both(coef)), p2 = f2pack(p[e], p[e + 1]);
            if (c.adamw)
                p2 = sub2(p2, mul2(c.two.lr_wd, p2), c);
            else
                g2 = add2(g2, mul2(c.two.wd, p2), c);
            const f2 m0 = mul2(f2pack(m[e], m[e + 1]), both(scale_m)), r0 = mul2(f2pack(r[e], r[e + 1]), both(scale_r));
            const f2 v2 = add2(mul2(c.two.b2, mul2(r0, r0)), mul2(c.two.omb2, mul2(g2, g2)), c);
            f2unpack(p2, p[e], p[e + 1]);
            f2unpack(add2(mul2(c.two.b1, m0), mul2(c.two.omb1, g2), c), m[e], m[e + 1]);
            f2unpack(root_2_32(v2), r[e], r[e + 1]);
        }
        const uint32_t tm = block_top(m), tr = block_top(r);
        if (max(tm, tr) >= 0x7F800000u) {         // the same in all lanes; nothing is written yet
            adam8_block<G, DITHER>(chunks + blockIdx.x, c, coef, fp16, b);
            continue;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float a, b;
            f2unpack(add2(mul2(f2pack(r[e], r[e + 1]), c.two.root_2_32), c.two.eps, c), a, b);
            const f2 q = f2pack(quick_quotient(m[e], a), quick_quotient(m[e + 1], b));
            f2unpack(sub2(f2pack(p[e], p[e + 1]), mul2(c.two.step_size, q), c), p[e], p[e + 1]);
        }
        store8f(k.master + x, p);
        if (k.param) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(k.param) + x) = cast8(p, fp16);
        const uint32_t fm = max(tm >> 23, 8u), fr = (uint32_t)max((int)(tr >> 23) - 32, 8);
        uint32_t lo[8], hi[8];
        if (DITHER) random8(k.elem + x, k.tensor, c, lo, hi);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(k.m) + x) = encode8<false, DITHER>(m, __uint_as_float((261u - fm) << 23), lo);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(k.v) + x) = encode8<true, DITHER>(r, __uint_as_float((229u - fr) << 23), hi);   // 2^-32 of the root's factor
        if (lane == 0) {
            k.m_scale[b] = __uint_as_float((fm - 7u) << 23);
            k.v_scale[b] = __uint_as_float((fr - 7u) << 23);
        }
    }
}

template <class G, bool DITHER>
static cudaError_t launch8(const zs_tensors *L, const Adam8C &c, const float *d_coef, const int32_t *d_flags, bool fp16,
                           cudaStream_t s) {
    static std::atomic<bool> set[64];            // the kernel's shared memory, per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(tensors8_kernel<G, DITHER>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM8<G>);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    return launch_dependent(tensors8_kernel<G, DITHER>, (unsigned)L->chunks.size(), THREADS, SMEM8<G>, 1, s, L->d_chunks, c,
                            d_coef, d_flags, fp16, zsl_test_give_up());
}

template <class G>
static cudaError_t launch(const zs_tensors *L, const ZsAdamScalars &a, const Adam8C &c8, bool dither,
                          const float *d_coef, const int32_t *d_flags, cudaStream_t s) {
    const unsigned grid = (unsigned)L->chunks.size();
    const bool fp16 = L->cfg.param_dtype == ZS_DTYPE_FP16;
    if (L->cfg.state_bits == 32) {
        AdamC c;
        c.lr = a.lr; c.b1 = a.b1; c.b2 = a.b2; c.omb1 = a.omb1; c.omb2 = a.omb2; c.eps = a.eps;
        c.wd = a.wd; c.lr_wd = a.lr_wd; c.bc1 = a.bc1; c.bc2 = a.bc2; c.adamw = a.adamw;
        return launch_dependent(tensors32_kernel<G>, grid, THREADS, 0, 1, s, L->d_chunks, c, d_coef, d_flags, fp16);
    }
    return dither ? launch8<G, true>(L, c8, d_coef, d_flags, fp16, s) : launch8<G, false>(L, c8, d_coef, d_flags, fp16, s);
}

}  // namespace zsk

cudaError_t zsl_tensors_wait_timeouts(int *count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, zsk::g_tensors_wait_timeouts, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(zsk::g_tensors_wait_timeouts, &zero, sizeof(int));
    }
    return e;
}

namespace {

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

int dtype_size(int32_t t) { return t == ZS_DTYPE_FP32 ? 4 : 2; }

}  // namespace

extern "C" {

zs_status zs_build_tensors(const zs_tensors_config *cfg, int32_t n, const zs_tensor *t,
                           zs_tensors **out) {
    const char *fn = "zs_build_tensors";
    if (!cfg || !out || n < 0 || (n > 0 && !t)) return zs_fail(ZS_EINVAL, "%s: NULL argument or n < 0", fn);
    *out = nullptr;
    if (cfg->state_bits != 8 && cfg->state_bits != 32)
        return zs_fail(ZS_EINVAL, "%s: state_bits %d is neither 8 nor 32", fn, cfg->state_bits);
    if (cfg->grad_dtype < ZS_DTYPE_BF16 || cfg->grad_dtype > ZS_DTYPE_FP32)
        return zs_fail(ZS_EINVAL, "%s: grad_dtype %d", fn, cfg->grad_dtype);
    if (cfg->param_dtype != ZS_DTYPE_BF16 && cfg->param_dtype != ZS_DTYPE_FP16)
        return zs_fail(ZS_EINVAL, "%s: param_dtype %d is not a 16-bit type", fn, cfg->param_dtype);
    if (cfg->reserved != 0) return zs_fail(ZS_EINVAL, "%s: reserved must be 0", fn);
    const bool eight = cfg->state_bits == 8;
    const int gsize = dtype_size(cfg->grad_dtype);
    int64_t chunks = 0, numel = 0;
    for (int32_t i = 0; i < n && numel < SHORT_ELEMS; ++i) numel += t[i].numel > 0 && t[i].numel < SHORT_ELEMS ? t[i].numel : t[i].numel > 0 ? SHORT_ELEMS : 0;
    const int64_t chunk = numel < SHORT_ELEMS ? CHUNK_SHORT : eight ? CHUNK8 : CHUNK32;
    for (int32_t i = 0; i < n; ++i) {
        const zs_tensor &x = t[i];
        if (x.numel < 0) return zs_fail(ZS_EINVAL, "%s: tensor %d: numel %lld < 0", fn, i, (long long)x.numel);
        if (x.numel == 0) continue;
        const struct { const void *p; unsigned size; bool used; const char *name; } items[] = {
            {x.grad, (unsigned)gsize, true, "grad"},
            {x.param, 2, x.param != nullptr, "param"},
            {x.master, 4, true, "master"},
            {x.exp_avg, eight ? 1u : 4u, true, "exp_avg"},
            {x.exp_avg_sq, eight ? 1u : 4u, true, "exp_avg_sq"},
            {x.exp_avg_scale, 4, eight, "exp_avg_scale"},
            {x.exp_avg_sq_scale, 4, eight, "exp_avg_sq_scale"},
        };
        for (const auto &it : items)
            if (it.used && (!it.p || addr(it.p) % it.size))
                return zs_fail(ZS_EINVAL, "%s: tensor %d: %s NULL or not aligned to its elements", fn, i, it.name);
        if (x.numel > (int64_t)1 << 48) return zs_fail(ZS_EINVAL, "%s: tensor %d: numel too large", fn, i);
        chunks += (x.numel + chunk - 1) / chunk;
    }
    if (chunks > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: more than 2^31 chunks of %d elements", fn, (int)chunk);
    zs_tensors *L = new (std::nothrow) zs_tensors;
    if (!L) return zs_fail(ZS_ENOMEM, "%s: out of host memory", fn);
    L->cfg = *cfg;
    L->n = n;
    try {
        L->chunks.reserve((size_t)chunks);
        std::vector<std::pair<uintptr_t, uintptr_t>> grads;              // first byte, past the last
        grads.reserve((size_t)n);
        for (int32_t i = 0; i < n; ++i)
            if (t[i].numel > 0) grads.emplace_back(addr(t[i].grad), addr(t[i].grad) + (uintptr_t)(t[i].numel * gsize));
        std::sort(grads.begin(), grads.end());
        for (size_t i = 1; i < grads.size(); ++i) L->grads_apart &= grads[i - 1].second <= grads[i].first;
    } catch (const std::bad_alloc &) {
        delete L;
        return zs_fail(ZS_ENOMEM, "%s: out of host memory", fn);
    }
    for (int32_t i = 0; i < n; ++i) {
        const zs_tensor &x = t[i];
        const bool aligned = addr(x.grad) % 16 == 0 && addr(x.param) % 16 == 0 && addr(x.master) % 16 == 0 &&
                             addr(x.exp_avg) % 16 == 0 && addr(x.exp_avg_sq) % 16 == 0;
        L->numel += x.numel;
        L->blocks += (x.numel + STATE_BLOCK - 1) / STATE_BLOCK;
        for (int64_t e = 0; e < x.numel; e += chunk) {
            const int64_t w = eight ? 1 : 4;
            ZsChunk k;
            k.grad = static_cast<const char *>(x.grad) + e * gsize;
            k.param = x.param ? static_cast<char *>(x.param) + 2 * e : nullptr;
            k.master = x.master + e;
            k.m = static_cast<char *>(x.exp_avg) + w * e;
            k.v = static_cast<char *>(x.exp_avg_sq) + w * e;
            k.m_scale = eight ? x.exp_avg_scale + e / STATE_BLOCK : nullptr;
            k.v_scale = eight ? x.exp_avg_sq_scale + e / STATE_BLOCK : nullptr;
            k.elem = e;
            k.len = (int32_t)(x.numel - e < chunk ? x.numel - e : chunk);
            k.tensor = aligned ? i : (int32_t)((uint32_t)i | 0x80000000u);
            L->chunks.push_back(k);
        }
    }
    *out = L;
    zs_clear_error();
    return ZS_OK;
}

void zs_free_tensors(zs_tensors *list) { delete list; }

zs_status zs_tensors_info(const zs_tensors *L, zs_tensors_info_t *out) {
    if (!L || !out) return zs_fail(ZS_EINVAL, "zs_tensors_info: NULL argument");
    out->n_tensors = L->n;
    out->state_bits = L->cfg.state_bits;
    out->numel = L->numel;
    out->n_chunks = (int64_t)L->chunks.size();
    out->n_blocks = L->blocks;
    out->device_table_bytes = (int64_t)(L->chunks.size() * sizeof(ZsChunk));
    zs_clear_error();
    return ZS_OK;
}

zs_status zs_tensors_upload(zs_tensors *L, void *d_table, int64_t bytes, void *stream) {
    const char *fn = "zs_tensors_upload";
    if (!L) return zs_fail(ZS_EINVAL, "%s: NULL list", fn);
    const int64_t need = (int64_t)(L->chunks.size() * sizeof(ZsChunk));
    if (need > 0) {
        if (!d_table || addr(d_table) % 16)
            return zs_fail(ZS_EINVAL, "%s: table NULL or not 16-byte aligned", fn);
        if (bytes < need)
            return zs_fail(ZS_EINVAL, "%s: %lld bytes < %lld needed", fn, (long long)bytes, (long long)need);
        const cudaError_t e = cudaMemcpyAsync(d_table, L->chunks.data(), (size_t)need,
                                              cudaMemcpyHostToDevice, (cudaStream_t)stream);
        if (e != cudaSuccess)
            return zs_fail(ZS_ECUDA, "%s: cudaMemcpyAsync: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
        L->d_chunks = static_cast<const ZsChunk *>(d_table);
    }
    zs_clear_error();
    return ZS_OK;
}

zs_status zs_test_root(int64_t *d_count, void *stream) {
    if (!d_count || addr(d_count) % 8) return zs_fail(ZS_EINVAL, "zs_test_root: count NULL or misaligned");
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaMemsetAsync(d_count, 0, 8, s);
    if (e == cudaSuccess) {
        zsk::root_test_kernel<<<1216, zsk::THREADS, 0, s>>>(reinterpret_cast<unsigned long long *>(d_count));
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "zs_test_root: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

zs_status zs_adam_tensors(const zs_tensors *L, const zs_adam_hparams *hp, int64_t step,
                          int32_t rounding, uint64_t seed, const float *d_clip_coef,
                          const int32_t *d_flags, void *stream) {
    const char *fn = "zs_adam_tensors";
    if (!L) return zs_fail(ZS_EINVAL, "%s: NULL list", fn);
    ZsAdamScalars a;
    zs_status r = zs_adam_scalars(hp, step, &a, fn);
    if (r) return r;
    if (rounding != ZS_ROUND_NEAREST && !(rounding == ZS_ROUND_STOCHASTIC && L->cfg.state_bits == 8))
        return zs_fail(ZS_EINVAL, "%s: rounding %d (stochastic rounding needs 8-bit moments)", fn, rounding);
    if (addr(d_clip_coef) % 4 || addr(d_flags) % 4)
        return zs_fail(ZS_EINVAL, "%s: d_clip_coef / d_flags misaligned", fn);
    if (L->chunks.empty()) {
        zs_clear_error();
        return ZS_OK;
    }
    if (!L->d_chunks) return zs_fail(ZS_ESTATE, "%s: list not uploaded (call zs_tensors_upload first)", fn);
    zsk::Adam8C c;
    c.b1 = a.b1; c.b2 = a.b2; c.omb1 = a.omb1; c.omb2 = a.omb2;
    c.eps = a.eps > 0.0f && a.eps < 0x1p-126f ? 0x1p-126f : a.eps;      // the quick quotient takes no subnormal denominator
    c.wd = a.wd; c.lr_wd = a.lr_wd; c.step_size = a.step_size; c.root = a.root; c.root_2_32 = a.root * 0x1p-32f;
    c.adamw = a.adamw;
    auto both = [](float x) {
        uint32_t u;
        memcpy(&u, &x, 4);
        return (unsigned long long)u << 32 | u;
    };
    c.two = {both(c.b1), both(c.b2), both(c.omb1), both(c.omb2), both(c.eps), both(c.wd), both(c.lr_wd), both(c.step_size),
             both(c.root_2_32), both(1.0f), both(-1.0f)};
    c.k0 = (uint32_t)seed;
    c.k1 = (uint32_t)(seed >> 32);
    c.step = (uint32_t)step;
    const bool dither = rounding == ZS_ROUND_STOCHASTIC;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (L->cfg.grad_dtype == ZS_DTYPE_FP32) e = zsk::launch<zsk::F32G>(L, a, c, dither, d_clip_coef, d_flags, s);
    else if (L->cfg.grad_dtype == ZS_DTYPE_FP16) e = zsk::launch<zsk::H16G<zsk::FP16T>>(L, a, c, dither, d_clip_coef, d_flags, s);
    else e = zsk::launch<zsk::H16G<zsk::BF16T>>(L, a, c, dither, d_clip_coef, d_flags, s);
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

}  // extern "C"
