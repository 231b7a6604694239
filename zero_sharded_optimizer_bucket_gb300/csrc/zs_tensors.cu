// Adam(W) over a list of separate tensors in one launch, moments in 32 bits
// or in 8 (zs_build_tensors, zs_adam_tensors).
//
// The host cuts every tensor into chunks of CHUNK elements and writes one
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
#include <new>
#include <vector>

#include "zs_device.cuh"
#include "zs_launch.h"

constexpr int CHUNK = 8192;          // elements per CTA
constexpr int STATE_BLOCK = 256;     // elements per scale: 8 a lane of one warp

struct ZsChunk {
    const void *grad;
    void *param;                     // 16-bit copy, or NULL
    float *master;
    void *m, *v;                     // float32, or e4m3 codes
    float *m_scale, *v_scale;        // 8-bit moments: of the chunk's first block
    int64_t elem;                    // index of the first element in its tensor
    int32_t len;
    int32_t tensor;                  // index in the list; bit 31: not every address is aligned
};
static_assert(sizeof(ZsChunk) == 72, "chunk layout");

struct zs_tensors {
    zs_tensors_config cfg;
    int32_t n = 0;
    int64_t numel = 0, blocks = 0;
    std::vector<ZsChunk> chunks;
    const ZsChunk *d_chunks = nullptr;   // caller memory given to zs_tensors_upload
};

namespace zsk {

struct Adam8C {
    float b1, b2, omb1, omb2, eps, wd, lr_wd, step_size, root;
    int adamw;
    uint32_t k0, k1, step;
};

struct F32G {
    static __device__ __forceinline__ void load8(const void *p, int64_t i, float g[8]) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4));
        g[0] = x.x; g[1] = x.y; g[2] = x.z; g[3] = x.w;
        g[4] = y.x; g[5] = y.y; g[6] = y.z; g[7] = y.w;
    }
    static __device__ __forceinline__ float load1(const void *p, int64_t i) {
        return static_cast<const float *>(p)[i];
    }
};
template <class T>
struct H16G {
    static __device__ __forceinline__ void load8(const void *p, int64_t i, float g[8]) {
        const uint4 v = ldg16(static_cast<const uint16_t *>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = T::to_f32(lane16(v, j));
    }
    static __device__ __forceinline__ float load1(const void *p, int64_t i) {
        return T::to_f32(static_cast<const uint16_t *>(p)[i]);
    }
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

// The 16-bit copy of 8 new parameters (fp16: the type is a launch argument,
// uniform over the grid).
__device__ __forceinline__ uint4 cast8(const float p[8], bool fp16) {
    uint32_t r[8];
    if (fp16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = FP16T::from_f32(p[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = BF16T::from_f32(p[i]);
    }
    return pack8(r);
}
__device__ __forceinline__ uint16_t cast1(float p, bool fp16) {
    return (uint16_t)(fp16 ? FP16T::from_f32(p) : BF16T::from_f32(p));
}

// ------------------------------------------------------ 32-bit moments --
// 28 bytes an element with 16-bit gradients and a 16-bit copy; the update is
// adam_elem, so that a list over a plan's shards gives zs_adam_step's bits.
template <class G>
__global__ void __launch_bounds__(THREADS)
tensors32_kernel(const ZsChunk *__restrict__ chunks, AdamC c, const float *__restrict__ d_coef,
                 const int32_t *__restrict__ d_flags, bool fp16) {
    if (d_flags && (*d_flags & ZS_SKIP_NONFINITE)) return;
    const float coef = d_coef ? *d_coef : 1.0f;
    const ZsChunk k = chunks[blockIdx.x];
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
        const uint32_t h0 = __umulhi(c0, 0xD2511F53u), l0 = c0 * 0xD2511F53u;
        const uint32_t h1 = __umulhi(c2, 0xCD9E8D57u), l1 = c2 * 0xCD9E8D57u;
        c0 = h1 ^ c1 ^ k0;
        c1 = l1;
        c2 = h0 ^ c3 ^ k1;
        c3 = l0;
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

// y (|y| < 256) to a value of e4m3, up when its 16 random bits say so: the
// probability of the upper neighbour is y's place between the two, to 2^-16.
// The equally spaced range below 2^-6 is shifted into the binade [2^-6, 2^-5),
// whose spacing is the same 2^-9.  Adding to the bits below the kept mantissa
// carries into it, and past it into the exponent, as rounding up does.
__device__ __forceinline__ float e4m3_dither(float y, uint32_t random16) {
    const float a = fabsf(y);
    const float off = a < 0.015625f ? 0.015625f : 0.0f;
    const uint32_t u = __float_as_uint(__fadd_rn(a, off)) + ((random16 << 4) | 8u);
    return copysignf(__fsub_rn(__uint_as_float(u & 0xFFF00000u), off), y);
}

__device__ __forceinline__ bool finite_bits(float x) {
    return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// The scale of a block's moment and the 8 codes of this lane.  All 32 lanes
// call it.  ROOT: x >= 0, and a positive value never gets code 0 (it divides
// the update).  Elements that are not finite become NaN codes and do not
// count for the scale.
template <bool ROOT, bool DITHER>
__device__ __forceinline__ uint2 encode8(float x[8], const uint32_t random[8], float &scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const bool odd = top >= 0x7F800000u;         // the same in every lane
    if (odd) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (finite_bits(x[i])) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
    }
    const uint32_t field = max(top >> 23, 8u);
    scale = __uint_as_float((field - 7u) << 23);
    const float inv = __uint_as_float((261u - field) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn(x[i], inv);
        if (DITHER) y[i] = e4m3_dither(y[i], random[i]);
        if (ROOT && x[i] > 0.0f) y[i] = fmaxf(y[i], 0.001953125f);
        if (odd && !finite_bits(x[i])) y[i] = __uint_as_float(0x7FC00000u);
    }
    return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                      e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

// One warp takes a block at a time, 8 consecutive elements a lane.
// 16 bytes an element with 16-bit gradients and a 16-bit copy.
template <class G, bool DITHER>
__global__ void __launch_bounds__(THREADS)
tensors8_kernel(const ZsChunk *__restrict__ chunks, Adam8C c, const float *__restrict__ d_coef,
                const int32_t *__restrict__ d_flags, bool fp16) {
    if (d_flags && (*d_flags & ZS_SKIP_NONFINITE)) return;
    const float coef = d_coef ? *d_coef : 1.0f;
    const ZsChunk k = chunks[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t *cm = static_cast<uint8_t *>(k.m), *cv = static_cast<uint8_t *>(k.v);
    uint16_t *param = static_cast<uint16_t *>(k.param);
    const bool aligned = k.tensor >= 0;
    for (int b = warp; b * STATE_BLOCK < k.len; b += WARPS) {
        const int x = b * STATE_BLOCK + 8 * lane;
        const int n = min(8, k.len - x);         // of this lane, may be negative
        const bool vec = aligned && n == 8;
        float g[8], p[8], m[8], r[8];
        uint2 qm = make_uint2(0, 0), qv = make_uint2(0, 0);
        if (vec) {
            G::load8(k.grad, x, g);
            load8f(k.master + x, p);
            qm = *reinterpret_cast<const uint2 *>(cm + x);
            qv = *reinterpret_cast<const uint2 *>(cv + x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = i < n;
                g[i] = in ? G::load1(k.grad, x + i) : 0.0f;
                p[i] = in ? k.master[x + i] : 0.0f;
                const uint32_t a = in ? cm[x + i] : 0u, d = in ? cv[x + i] : 0u;
                if (i < 4) { qm.x |= a << (8 * i); qv.x |= d << (8 * i); }
                else { qm.y |= a << (8 * i - 32); qv.y |= d << (8 * i - 32); }
            }
        }
        const float sm = k.m_scale[b], sv = k.v_scale[b];
        e4m3_decode8(qm, m);
        e4m3_decode8(qv, r);
        uint32_t lo[8], hi[8];
        if (DITHER) {
            const uint64_t q = (uint64_t)(k.elem + x) >> 2;
            const uint32_t t = (uint32_t)k.tensor & 0x7FFFFFFFu;
            uint32_t w[8];
            philox7((uint32_t)q, (uint32_t)(q >> 32), t, c.step, c.k0, c.k1, w);
            philox7((uint32_t)(q + 1), (uint32_t)((q + 1) >> 32), t, c.step, c.k0, c.k1, w + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[i] = w[i] & 0xFFFFu;
                hi[i] = w[i] >> 16;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float gi = __fmul_rn(g[i], coef);
            if (c.adamw)
                p[i] = __fsub_rn(p[i], __fmul_rn(c.lr_wd, p[i]));
            else
                gi = __fadd_rn(gi, __fmul_rn(c.wd, p[i]));
            const float r0 = __fmul_rn(r[i], sv);
            m[i] = __fadd_rn(__fmul_rn(c.b1, __fmul_rn(m[i], sm)), __fmul_rn(c.omb1, gi));
            r[i] = __fsqrt_rn(__fadd_rn(__fmul_rn(c.b2, __fmul_rn(r0, r0)),
                                        __fmul_rn(c.omb2, __fmul_rn(gi, gi))));
            const float den = __fadd_rn(__fmul_rn(r[i], c.root), c.eps);
            p[i] = __fsub_rn(p[i], __fmul_rn(c.step_size, __fdiv_rn(m[i], den)));
        }
        float ns, nv;
        if (n < 8) {   // past the end: nothing that the scales could see
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= n) m[i] = r[i] = 0.0f;
        }
        qm = encode8<false, DITHER>(m, lo, ns);
        qv = encode8<true, DITHER>(r, hi, nv);
        if (vec) {
            store8f(k.master + x, p);
            *reinterpret_cast<uint2 *>(cm + x) = qm;
            *reinterpret_cast<uint2 *>(cv + x) = qv;
            if (param) *reinterpret_cast<uint4 *>(param + x) = cast8(p, fp16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= n) continue;
                k.master[x + i] = p[i];
                cm[x + i] = (uint8_t)((i < 4 ? qm.x : qm.y) >> (8 * (i & 3)));
                cv[x + i] = (uint8_t)((i < 4 ? qv.x : qv.y) >> (8 * (i & 3)));
                if (param) param[x + i] = cast1(p[i], fp16);
            }
        }
        if (lane == 0) {
            k.m_scale[b] = ns;
            k.v_scale[b] = nv;
        }
    }
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
        tensors32_kernel<G><<<grid, THREADS, 0, s>>>(L->d_chunks, c, d_coef, d_flags, fp16);
    } else if (dither) {
        tensors8_kernel<G, true><<<grid, THREADS, 0, s>>>(L->d_chunks, c8, d_coef, d_flags, fp16);
    } else {
        tensors8_kernel<G, false><<<grid, THREADS, 0, s>>>(L->d_chunks, c8, d_coef, d_flags, fp16);
    }
    return cudaGetLastError();
}

}  // namespace zsk

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
    int64_t chunks = 0;
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
        chunks += (x.numel + CHUNK - 1) / CHUNK;
    }
    if (chunks > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: more than 2^31 chunks of %d elements", fn, CHUNK);
    zs_tensors *L = new (std::nothrow) zs_tensors;
    if (!L) return zs_fail(ZS_ENOMEM, "%s: out of host memory", fn);
    L->cfg = *cfg;
    L->n = n;
    try {
        L->chunks.reserve((size_t)chunks);
    } catch (const std::bad_alloc &) {
        delete L;
        return zs_fail(ZS_ENOMEM, "%s: out of host memory", fn);
    }
    for (int32_t i = 0; i < n; ++i) {
        const zs_tensor &x = t[i];
        const uintptr_t state = eight ? 8 : 16;
        const bool aligned = addr(x.grad) % 16 == 0 && addr(x.param) % 16 == 0 && addr(x.master) % 16 == 0 &&
                             addr(x.exp_avg) % state == 0 && addr(x.exp_avg_sq) % state == 0;
        L->numel += x.numel;
        L->blocks += (x.numel + STATE_BLOCK - 1) / STATE_BLOCK;
        for (int64_t e = 0; e < x.numel; e += CHUNK) {
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
            k.len = (int32_t)(x.numel - e < CHUNK ? x.numel - e : CHUNK);
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
    c.b1 = a.b1; c.b2 = a.b2; c.omb1 = a.omb1; c.omb2 = a.omb2; c.eps = a.eps;
    c.wd = a.wd; c.lr_wd = a.lr_wd; c.step_size = a.step_size; c.root = a.root; c.adamw = a.adamw;
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
