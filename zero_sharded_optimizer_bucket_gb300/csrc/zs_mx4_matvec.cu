// A few tokens of 16 or 32 bits through a weight held in 4 bits
// (zs_mx4_matvec): out[m][n] = sum over k of x[m][k] w[n][k].
//
// The weight's 0.53 bytes an element are read once and decoded in registers;
// products go to the tensor cores in fp16 (mma m16n8k16): a code is exact
// there, a token's values are after a power of two of their own (fp32 ones as
// two numbers of 11 bits), sums are fp32, and a group's scale is multiplied to
// its 32 products' sum.
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
    int32_t out_kind, row_tiles;     // row tiles of 16 a CTA (1, 2, 4, 8)
};

constexpr int MV_CHUNK = 128;        // k of one atom of scales: 4 groups
// k of x that lies in shared memory at a time
__host__ __device__ constexpr int mv_stage(int nb) { return nb == 1 ? 4096 : nb == 2 ? 2048 : 1024; }
__host__ __device__ constexpr int mv_pitch(int nb) { return mv_stage(nb) + 32; }         // halves; 64 bytes past 128: two tokens' pieces side by side
__host__ __device__ constexpr int mv_smem(int nb) { return 8 * nb * mv_pitch(nb) * 2; }

// codes j and j + 4 of 8 as two halves, 2^-14 of their values: the sign to the
// top, exponent and mantissa to the lowest exponent bits and the highest
// mantissa bit (1/2 is subnormal there, and exact)
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j) {
    const uint32_t t = j == 3 ? w : w << (12 - 4 * j);
    return (t & 0x80008000u) | ((t >> 3) & 0x0E000E00u);
}

__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int KIND>
__device__ __forceinline__ float mv_value(const void *x, int64_t at) {
    if (KIND == ZS_DTYPE_FP32) return static_cast<const float *>(x)[at];
    const uint32_t b = static_cast<const uint16_t *>(x)[at];
    return KIND == ZS_DTYPE_FP16 ? FP16T::to_f32(b) : BF16T::to_f32(b);
}

// floor(log2) of a token's largest magnitude, from its bits; at least what
// float32 has powers of two for
__device__ __forceinline__ int mv_exponent(int top) { return max((int)((uint32_t)top >> 23) - 127, -112); }
__device__ __forceinline__ float mv_power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }     // e of normal numbers

// A CTA takes 16 * row_tiles rows of the weight and, of a cluster of S, one
// S-th of k, its warps sharing both; 8 NB columns of tokens (fp32: two columns
// a token) lie in shared memory as halves.
template <int KIND, int NB>
__global__ void __launch_bounds__(THREADS)
mx4_matvec_kernel(MatvecArgs a) {
    constexpr int COLS = 8 * NB, PER = KIND == ZS_DTYPE_FP32 ? 2 : 1, TOKENS = COLS / PER, PITCH = mv_pitch(NB);
    extern __shared__ __align__(16) uint8_t raw[];
    __half *xs = reinterpret_cast<__half *>(raw);
    __shared__ float share[COLS * 128];
    __shared__ int top[TOKENS];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = lane >> 2, t = lane & 3;
    const int parts = WARPS / a.row_tiles, part = warp / a.row_tiles, tile = warp % a.row_tiles;
    const int64_t row0 = ((int64_t)(blockIdx.x / ranks) * a.row_tiles + tile) * 16, token0 = (int64_t)blockIdx.y * TOKENS;
    const int tokens = (int)min((int64_t)TOKENS, a.m - token0);
    const int64_t groups = mx4_groups(a.k), chunks = (groups + 3) / 4, row_bytes = mx4_row_bytes(a.k), atoms = mx4_atoms(a.k);
    const int64_t first = chunks * rank / ranks, last = chunks * (rank + 1) / ranks;
    if (threadIdx.x < TOKENS) top[threadIdx.x] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    // the largest finite magnitude of each token in this part of k
    const int64_t k0 = first * MV_CHUNK, k1 = min(last * MV_CHUNK, a.k);
    for (int i = 0; i < tokens; ++i) {
        uint32_t most = 0;
        for (int64_t k = k0 + threadIdx.x; k < k1; k += THREADS) {
            const uint32_t b = __float_as_uint(mv_value<KIND>(a.x, (token0 + i) * a.ldx + k)) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) most = max(most, b);
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (lane == 0) atomicMax(&top[i], (int)most);
    }
    __syncthreads();
    // sums are held as those of the largest token, so that none overflows before it does
    int most = 0;
    for (int i = 0; i < tokens; ++i) most = max(most, top[i]);
    const int common = mv_exponent(most);
    const float up = mv_power(min(common, 126));
    float acc[NB][4] = {};
    const int64_t ra = row0 + q, rb = ra + 8;
    const bool has_a = ra < a.n, has_b = rb < a.n;
    const uint8_t *ca = a.codes + ra * row_bytes + 4 * t, *cb = a.codes + rb * row_bytes + 4 * t;
    const uint8_t *sa = a.scales + (ra >> 7) * atoms * MX4_ATOM + mx4_in_atom((int)(ra & 127), 0);
    const uint8_t *sb = a.scales + (rb >> 7) * atoms * MX4_ATOM + mx4_in_atom((int)(rb & 127), 0);
    constexpr int STAGE = mv_stage(NB) / MV_CHUNK;
    for (int64_t c0 = first; c0 < last; c0 += STAGE) {
        const int n = (int)min((int64_t)STAGE, last - c0);
        if (c0 > first) __syncthreads();
        // tokens to halves, times 2^(14 - E), element 8 i + j at 8 i + 2 (j % 4) + j / 4: a lane's 8 codes in the order of its pairs
        for (int i = warp; i < tokens; i += WARPS) {
            const float f = mv_power(14 - mv_exponent(top[i]));
            for (int kk = lane; kk < n * MV_CHUNK; kk += 32) {
                const int64_t k = c0 * MV_CHUNK + kk;
                const float v = k < a.k ? __fmul_rn(mv_value<KIND>(a.x, (token0 + i) * a.ldx + k), f) : 0.0f;
                const int at = (kk & ~7) + 2 * (kk & 3) + ((kk >> 2) & 1);
                const __half h = __float2half_rn(v);
                xs[PER * i * PITCH + at] = h;
                if (PER == 2) xs[(PER * i + 1) * PITCH + at] = __hisinf(h) || __hisnan(h) ? __half(0.0f) : __float2half_rn(__fmul_rn(__fsub_rn(v, __half2float(h)), 2048.0f));
            }
        }
        __syncthreads();
        for (int c = part; c < n; c += parts) {
            const int64_t g0 = 4 * (c0 + c);
            uint32_t wa[4], wb[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                wa[g] = has_a && g0 + g < groups ? *reinterpret_cast<const uint32_t *>(ca + 16 * (g0 + g)) : 0u;
                wb[g] = has_b && g0 + g < groups ? *reinterpret_cast<const uint32_t *>(cb + 16 * (g0 + g)) : 0u;
            }
            const uint32_t za = has_a ? *reinterpret_cast<const uint32_t *>(sa + (c0 + c) * MX4_ATOM) : 0u;
            const uint32_t zb = has_b ? *reinterpret_cast<const uint32_t *>(sb + (c0 + c) * MX4_ATOM) : 0u;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t pa[4], pb[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pa[j] = code_pair(wa[g], j);
                    pb[j] = code_pair(wb[g], j);
                }
                const float fa = __fmul_rn(mx4_scale((za >> (8 * g)) & 255u), up), fb = __fmul_rn(mx4_scale((zb >> (8 * g)) & 255u), up);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (8 * b + q < PER * tokens) v = *reinterpret_cast<const uint4 *>(xs + (8 * b + q) * PITCH + c * MV_CHUNK + 32 * g + 8 * t);
                    float d[4] = {};
                    mma16816(d, pa[0], pb[0], pa[1], pb[1], v.x, v.y);
                    mma16816(d, pa[2], pb[2], pa[3], pb[3], v.z, v.w);
                    acc[b][0] = __fmaf_rn(d[0], fa, acc[b][0]);
                    acc[b][1] = __fmaf_rn(d[1], fa, acc[b][1]);
                    acc[b][2] = __fmaf_rn(d[2], fb, acc[b][2]);
                    acc[b][3] = __fmaf_rn(d[3], fb, acc[b][3]);
                }
            }
        }
    }
    __syncthreads();
    // the warps' parts of k, in their order: [warp][column][16 rows]
    float *red = reinterpret_cast<float *>(raw);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[(warp * COLS + 8 * b + 2 * t + (i & 1)) * 16 + q + 8 * (i >> 1)] = acc[b][i];
    __syncthreads();
    const int rows = 16 * a.row_tiles;
    for (int i = threadIdx.x; i < tokens * rows; i += THREADS) {
        const int token = i / rows, r = i % rows;
        const int down = mv_exponent(top[token]) - min(common, 126);
        float s[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            s[p] = 0.0f;
            for (int w = 0; w < parts; ++w) s[p] = __fadd_rn(s[p], red[((w * a.row_tiles + r / 16) * COLS + PER * token + p) * 16 + r % 16]);
        }
        float v = s[0];
        if (PER == 2) v = __fmaf_rn(s[PER - 1], 1.0f / 2048, v);
        // the codes' 2^-14 and the token's 2^14 are one another's
        share[token * rows + r] = __fmul_rn(__fmul_rn(v, mv_power(down >> 1)), mv_power(down - (down >> 1)));
    }
    cluster.sync();
    const int64_t block0 = (int64_t)(blockIdx.x / ranks) * rows;
    for (int i = rank * THREADS + threadIdx.x; i < tokens * rows; i += THREADS * ranks) {
        float s = 0.0f;
        for (int r = 0; r < ranks; ++r) s = __fadd_rn(s, cluster.map_shared_rank(share, r)[i]);
        const int64_t row = block0 + i % rows, at = (token0 + i / rows) * a.ldo + row;
        if (row >= a.n) continue;
        if (a.out_kind == ZS_DTYPE_FP32) static_cast<float *>(a.out)[at] = s;
        else static_cast<uint16_t *>(a.out)[at] = (uint16_t)(a.out_kind == ZS_DTYPE_FP16 ? FP16T::from_f32(s) : BF16T::from_f32(s));
    }
    cluster.sync();                  // the others may still read this CTA's sums
}

template <int KIND, int NB>
static cudaError_t matvec_launch(MatvecArgs a, cudaStream_t s) {
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(mx4_matvec_kernel<KIND, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, mv_smem(NB));
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    const int64_t tokens = 8 * NB / (KIND == ZS_DTYPE_FP32 ? 2 : 1), ty = (a.m + tokens - 1) / tokens, tiles = (a.n + 15) / 16;
    const int64_t chunks = (mx4_groups(a.k) + 3) / 4;
    // enough CTAs for two an SM: first by parts of k, then by fewer rows each
    int split = 1;
    a.row_tiles = 8;
    auto ctas = [&] { return (tiles + a.row_tiles - 1) / a.row_tiles * split * ty; };
    while (ctas() < 304 && split < 8 && chunks >= 2 * split * (WARPS / a.row_tiles)) split *= 2;
    while (ctas() < 304 && a.row_tiles > 1 && chunks >= 2 * split * (WARPS / a.row_tiles)) a.row_tiles /= 2;
    const int64_t blocks = (tiles + a.row_tiles - 1) / a.row_tiles * split;
    if (blocks > 0x7FFFFFFF || ty > 65535) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)ty);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = mv_smem(NB);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
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
        e = dtype == ZS_DTYPE_FP32 ? zsk::matvec_of<ZS_DTYPE_FP32>(a, s)
          : dtype == ZS_DTYPE_FP16 ? zsk::matvec_of<ZS_DTYPE_FP16>(a, s) : zsk::matvec_of<ZS_DTYPE_BF16>(a, s);
    }
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}
