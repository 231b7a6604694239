// The global gradient norm over a list of tensors, and clipping in place
// (zs_norm_tensors, zs_clip_tensors).
//
// norm = sqrt(sum of squares) / S over every gradient of the list, with the
// coefficient and the flag that zs_adam_tensors takes.  One read of the
// gradients: 2 or 4 bytes an element at two to four instructions, so bandwidth
// bounds it.  202M bf16 gradients: 77 us with the caches flushed before, 5.3 TB/s
// (0.78 of a copy's rate; instructions and loads share the issue slots).  100M
// fp16 gradients clipped in place, norm included: 97 us, 6.2 TB/s of two reads
// and a write.  A short list is two launches: 4.5 us in a graph.
#include <atomic>

#include "zs_launch.h"
#include "zs_norm.cuh"
#include "zs_tensors.cuh"

namespace zsk {

// 128 threads with up to 8 groups of 8 elements each: a chunk of 8192.  Fewer
// threads with more groups share the work that a thread has with a chunk over
// more squares (256 threads of 4 groups: 94 us for 202M bf16 gradients).
constexpr int NORM_THREADS = 128, NORM_GROUPS = 8, NORM_DEPTH = 2;
static_assert(8 * NORM_THREADS * NORM_GROUPS >= CHUNK_MOST, "a chunk at a time");
template <class G>
__host__ __device__ constexpr int norm_stage() { return 8 * NORM_THREADS * NORM_GROUPS * G::SIZE; }
template <class G>
__host__ __device__ constexpr int norm_ring() { return NORM_DEPTH * norm_stage<G>(); }      // 192 KB an SM
template <class G>
__host__ __device__ constexpr int norm_ctas() { return G::SIZE == 2 ? 6 : 3; }

// 8 gradients as they lie in memory.
template <class G>
struct Raw8;
template <class T>
struct Raw8<H16G<T>> {
    uint4 w;
    __device__ __forceinline__ void shared(uint32_t at, bool) { w = lds16(at); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    // element i of the 8
    __device__ __forceinline__ void put(const void *p, int x, int i) {
        const uint32_t v = (uint32_t)static_cast<const uint16_t *>(p)[x] << (i & 1 ? 16 : 0);
        uint32_t &u = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        u |= v;
    }
};
template <>
struct Raw8<F32G> {
    uint4 a, b;
    __device__ __forceinline__ void shared(uint32_t at, bool second) {
        a = lds16(at);
        if (second) b = lds16(at + 16 * NORM_THREADS);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void put(const void *p, int x, int i) {
        const uint32_t v = __float_as_uint(static_cast<const float *>(p)[x]);
        uint4 &q = i < 4 ? a : b;
        uint32_t &u = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
        u = v;
    }
};

// Sum of squares of a thread's groups as a pair hi + lo, good to about 2^-32
// of it (vt_sumsq).  p.ok false: the magnitudes leave the range of the method,
// and squares() is to be used.
template <class T>
__device__ __forceinline__ VtPair pair_of(const Raw8<H16G<T>> (&r)[NORM_GROUPS], int n) {
    uint4 w[NORM_GROUPS];
#pragma unroll
    for (int g = 0; g < NORM_GROUPS; ++g) w[g] = r[g].w;
    return vt_sumsq<T>(w, n);
}
// The same for float32.  A square is not exact here: s = x x + h is rounded
// once, d = h - s is exact (both in [B, 2B)), and x x + d is the rounding error
// of s, kept to 24 bits of its own.
__device__ __forceinline__ VtPair pair_of(const Raw8<F32G> (&r)[NORM_GROUPS], int n) {
    float top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int g = 0; g < NORM_GROUPS; ++g) {
        if (g >= n) continue;
        float x[8];
        floats4(r[g].a, x);
        floats4(r[g].b, x + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
    }
    VtPair p;
    p.hi = p.lo = 0.0f;
    const uint32_t field = __float_as_uint(top) >> 23;
    bad = top != 0.0f && !(field >= 87u && field < 183u);        // [2^-40, 2^56)
    p.ok = !bad;
    if (bad || top == 0.0f) return p;
    const float B = __uint_as_float((2u * field - 254u + 7u + 127u) << 23);     // 2^(2E + 7), above 32 top^2
    const unsigned long long BB = f2pack(B, B);
    unsigned long long h = BB, l = 0;
#pragma unroll
    for (int g = 0; g < NORM_GROUPS; ++g) {
        if (g >= n) continue;
        float x[8];
        floats4(r[g].a, x);
        floats4(r[g].b, x + 4);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const unsigned long long v = f2pack(x[i], x[i + 1]);
            unsigned long long s, d, e;
            asm("fma.rn.f32x2 %0, %1, %1, %2;" : "=l"(s) : "l"(v), "l"(h));
            asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(h), "l"(s));
            asm("fma.rn.f32x2 %0, %1, %1, %2;" : "=l"(e) : "l"(v), "l"(d));
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(l) : "l"(l), "l"(e));
            h = s;
        }
    }
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(h) : "l"(h), "l"(BB));                // exact
    float he, ho, le, lo;
    f2unpack(h, he, ho);
    f2unpack(l, le, lo);
    add22(he, le, ho, lo);
    p.hi = he;
    p.lo = le;
    return p;
}

template <class T>
__device__ __forceinline__ double squares(const Raw8<H16G<T>> (&r)[NORM_GROUPS], int n) {
    uint4 w[NORM_GROUPS];
#pragma unroll
    for (int g = 0; g < NORM_GROUPS; ++g) w[g] = r[g].w;
    return vt_sumsq_f64<T>(w, n);
}
__device__ __forceinline__ double squares(const Raw8<F32G> (&r)[NORM_GROUPS], int n) {
    double s = 0.0;
#pragma unroll
    for (int g = 0; g < NORM_GROUPS; ++g) {
        if (g >= n) continue;
        float x[8];
        floats4(r[g].a, x);
        floats4(r[g].b, x + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = __dadd_rn(s, __dmul_rn((double)x[i], (double)x[i]));
    }
    return s;
}

__device__ __forceinline__ void async16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(to), "l"(from) : "memory");
}

// CTA b takes chunks b, b + grid, ...; a thread adds its groups' squares to a
// pair of floats over all of them, and the CTA leaves one double.  Which
// thread takes what depends on the list and the grid alone, so the same call
// gives the same bits.  The next chunks' groups are on their way to shared
// memory, each thread's to a place of its own, so that nothing but its own
// copies holds a thread up (loaded into registers when their turn came, 202M
// bf16 gradients took 100 us).
template <class G>
__global__ void __launch_bounds__(NORM_THREADS, norm_ctas<G>())
norm_tensors_kernel(const ZsChunk *chunks, int n_chunks, double *partials) {
    extern __shared__ __align__(16) uint8_t ring[];
    // a group is one or two pieces of 16 bytes, each beside the neighbours': a
    // warp's copies then read whole sectors (two pieces side by side: 59 us for 51M
    // fp32 gradients, 38 so)
    constexpr int PIECES = G::SIZE / 2, ONE = 16 / G::SIZE;
    __shared__ double red[NORM_THREADS / 32];
    pdl_wait();
    pdl_trigger();
    float hi = 0.0f, lo = 0.0f;
    double wide = 0.0;
    const int t = threadIdx.x;
    const uint32_t mine = smem_u32(ring) + 16 * t;                   // 16-byte pieces side by side over the threads
    const void *grad = nullptr;                                      // of the next chunk to be copied
    int vec = 0, ahead = blockIdx.x, slot = 0;
    auto look = [&] {
        vec = 0;
        if (ahead >= n_chunks) return;
        grad = chunks[ahead].grad;
        vec = chunks[ahead].tensor < 0 ? 0 : chunks[ahead].len & ~7;
    };
    auto copy = [&] {
#pragma unroll
        for (int p = 0; p < NORM_GROUPS * PIECES; ++p) {
            if (ONE * (t + NORM_THREADS * p) >= vec) break;
            async16(mine + slot + p * (16 * NORM_THREADS), static_cast<const char *>(grad) + 16 * (t + NORM_THREADS * p));
        }
        asm volatile("cp.async.commit_group;" : : : "memory");
        slot = slot + norm_stage<G>() == norm_ring<G>() ? 0 : slot + norm_stage<G>();
        ahead += gridDim.x;
        look();
    };
    look();
    copy();
    int place = 0;
    auto add = [&](const Raw8<G> (&r)[NORM_GROUPS], int n) {
        const VtPair p = pair_of(r, n);
        if (p.ok) add22(hi, lo, p.hi, p.lo);
        else wide = __dadd_rn(wide, squares(r, n));
        if (hi > 1.0e30f) {                          // far below where another pair could overflow it
            wide = __dadd_rn(wide, __dadd_rn((double)hi, (double)lo));
            hi = lo = 0.0f;
        }
    };
#pragma unroll 1
    for (int c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        copy();
        const int len = chunks[c].len, whole = chunks[c].tensor < 0 ? 0 : len & ~7;
        asm volatile("cp.async.wait_group %0;" : : "n"(NORM_DEPTH - 1) : "memory");
        if (ONE * t < whole) {
            Raw8<G> r[NORM_GROUPS];
            int n = 0;
#pragma unroll
            for (int g = 0; g < NORM_GROUPS; ++g) {
                r[g].zero();
                const int x = ONE * (t + NORM_THREADS * PIECES * g);
                if (x < whole) {
                    r[g].shared(mine + place + g * PIECES * (16 * NORM_THREADS), x + ONE * NORM_THREADS < whole);
                    n = g + 1;
                }
            }
            add(r, n);
        }
        place = place + norm_stage<G>() == norm_ring<G>() ? 0 : place + norm_stage<G>();
        // the rest, or all of a chunk that is not aligned: lanes side by side
        if (whole == len) continue;
        const void *from = chunks[c].grad;
#pragma unroll 1
        for (int x0 = whole + t; x0 < len; x0 += 8 * NORM_THREADS * NORM_GROUPS) {
            Raw8<G> r[NORM_GROUPS];
            int n = 0;
#pragma unroll
            for (int g = 0; g < NORM_GROUPS; ++g) {
                r[g].zero();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int x = x0 + NORM_THREADS * (8 * g + i);
                    if (x < len) {
                        r[g].put(from, x, i);
                        n = g + 1;
                    }
                }
            }
            add(r, n);
        }
    }
    double s = __dadd_rn(__dadd_rn((double)hi, (double)lo), wide);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s = __dadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, off));
    if ((t & 31) == 0) red[t >> 5] = s;
    __syncthreads();
    if (t != 0) return;
    for (int w = 1; w < NORM_THREADS / 32; ++w) s = __dadd_rn(s, red[w]);
    partials[blockIdx.x] = s;
}

__global__ void __launch_bounds__(THREADS)
norm_tensors_finish_kernel(const double *partials, int n, float max_norm, float *d_norm, float *d_coef,
                           int32_t *d_flags, ZsScaleArgs sc) {
    __shared__ double red[WARPS];
    pdl_wait();
    pdl_trigger();
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) v = __dadd_rn(v, partials[i]);
    const double s = block_sum(v, red);
    if (threadIdx.x == 0) norm_finish(s, max_norm, d_norm, d_coef, d_flags, sc);
}

// g = g coef, rounded once to the gradients' type.
template <class G>
__global__ void __launch_bounds__(THREADS)
clip_tensors_kernel(const ZsChunk *chunks, const float *d_coef, const int32_t *d_flags, int kind) {
    pdl_wait();
    pdl_trigger();
    const float coef = *d_coef;
    if (d_flags && (*d_flags & ZS_SKIP_NONFINITE)) return;
    if (coef == 1.0f) return;                        // every gradient stays what it is
    // the last chunks first: the norm, whose coefficient this is, has just read them
    const ZsChunk &k = chunks[gridDim.x - 1 - blockIdx.x];
    void *grad = const_cast<void *>(k.grad);
    const int len = k.len, vec = k.tensor < 0 ? 0 : len & ~7;
    for (int x = 8 * threadIdx.x; x < vec; x += 8 * THREADS) {
        float g[8];
        G::load8(grad, x, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(g[i], coef);
        if (G::SIZE == 4) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(grad) + x);
            o[0] = make_float4(g[0], g[1], g[2], g[3]);
            o[1] = make_float4(g[4], g[5], g[6], g[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(grad) + x) = cast8(g, kind == ZS_DTYPE_FP16);
        }
    }
    for (int x = vec + threadIdx.x; x < len; x += THREADS) {
        const float g = __fmul_rn(G::load1(grad, x), coef);
        if (G::SIZE == 4) static_cast<float *>(grad)[x] = g;
        else static_cast<uint16_t *>(grad)[x] = (uint16_t)(kind == ZS_DTYPE_FP16 ? FP16T::from_f32(g) : BF16T::from_f32(g));
    }
}

template <class G>
static cudaError_t norm_launch(const zs_tensors *L, double *partials, int64_t *grid, cudaStream_t s) {
    static std::atomic<int> known[64];               // SMs, once the kernel's shared memory is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = known[dev].load(std::memory_order_relaxed);
    if (sms <= 0) {
        e = cudaFuncSetAttribute(norm_tensors_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, norm_ring<G>());
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    const int64_t n = (int64_t)L->chunks.size(), wave = (int64_t)sms * norm_ctas<G>();
    *grid = n < wave ? n : wave;
    return launch_dependent(norm_tensors_kernel<G>, (unsigned)*grid, NORM_THREADS, norm_ring<G>(), 1, s, L->d_chunks, (int)n, partials);
}

// f with the gradient type of the list
template <class F>
static cudaError_t by_type(int32_t dtype, F f) {
    if (dtype == ZS_DTYPE_FP32) return f(F32G());
    if (dtype == ZS_DTYPE_FP16) return f(H16G<FP16T>());
    return f(H16G<BF16T>());
}

}  // namespace zsk

namespace {

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
bool al(const void *p, unsigned n) { return p && addr(p) % n == 0; }

zs_status cuda_status(cudaError_t e, const char *fn) {
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

}  // namespace

extern "C" {

zs_status zs_norm_tensors(const zs_tensors *L, double *scratch, float max_norm, const zs_loss_scaler *scaler,
                          float *d_norm, float *d_clip_coef, int32_t *d_flags, void *stream) {
    const char *fn = "zs_norm_tensors";
    if (!L) return zs_fail(ZS_EINVAL, "%s: NULL list", fn);
    ZsScaleArgs sc = {};
    if (scaler) {
        const zs_status r = zs_scale_args(scaler, &sc, fn);
        if (r) return r;
    }
    if (!al(d_norm, 4) || !al(d_clip_coef, 4) || !al(d_flags, 4))
        return zs_fail(ZS_EINVAL, "%s: d_norm, d_clip_coef or d_flags NULL or misaligned", fn);
    const int64_t n = (int64_t)L->chunks.size();
    if (n > 0 && !al(scratch, 8)) return zs_fail(ZS_EINVAL, "%s: scratch NULL or not 8-byte aligned", fn);
    if (n > 0 && !L->d_chunks) return zs_fail(ZS_ESTATE, "%s: list not uploaded (call zs_tensors_upload first)", fn);
    using namespace zsk;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    int64_t grid = 0;
    if (n > 0) e = by_type(L->cfg.grad_dtype, [&](auto g) { return norm_launch<decltype(g)>(L, scratch, &grid, s); });
    if (e == cudaSuccess)
        e = launch_dependent(norm_tensors_finish_kernel, 1, THREADS, 0, 1, s, scratch, (int)grid, max_norm, d_norm, d_clip_coef, d_flags, sc);
    return cuda_status(e, fn);
}

zs_status zs_clip_tensors(const zs_tensors *L, const float *d_clip_coef, const int32_t *d_flags, void *stream) {
    const char *fn = "zs_clip_tensors";
    if (!L) return zs_fail(ZS_EINVAL, "%s: NULL list", fn);
    if (!al(d_clip_coef, 4) || addr(d_flags) % 4)
        return zs_fail(ZS_EINVAL, "%s: d_clip_coef NULL or misaligned, or d_flags misaligned", fn);
    if (!L->grads_apart) return zs_fail(ZS_EINVAL, "%s: gradients of the list overlap", fn);
    if (L->chunks.empty()) {
        zs_clear_error();
        return ZS_OK;
    }
    if (!L->d_chunks) return zs_fail(ZS_ESTATE, "%s: list not uploaded (call zs_tensors_upload first)", fn);
    using namespace zsk;
    return cuda_status(by_type(L->cfg.grad_dtype, [&](auto g) {
        return launch_dependent(clip_tensors_kernel<decltype(g)>, (unsigned)L->chunks.size(), THREADS, 0, 1, (cudaStream_t)stream,
                                L->d_chunks, d_clip_coef, d_flags, (int)L->cfg.grad_dtype);
    }), fn);
}

}  // extern "C"
