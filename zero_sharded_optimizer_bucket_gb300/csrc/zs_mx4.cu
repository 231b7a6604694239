// 16- or 32-bit matrices to microscaled 4-bit floating point and back
// (zs_mx4_quantize, zs_mx4_dequantize).
//
// Along the rows a group is 32 consecutive elements of a row; along the
// columns, 32 consecutive elements of a column, and the result is the
// transposed matrix.  A training step needs both of every operand (a product
// sums along one dimension, its gradients along the other), so one launch
// makes both from one read.
#include "zs_launch.h"
#include "zs_mx4.cuh"

namespace zsk {

constexpr int QT = 128;      // a CTA takes a tile of 128 x 128: one scale atom each way


// 8 consecutive elements of a row as floats, zero outside the matrix
template <class T, bool F32, bool VEC>
struct Row8 {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *x, int64_t at, int n) {
        if (n <= 0) {
#pragma unroll
            for (auto &v : w) v = make_uint4(0, 0, 0, 0);
        } else if (VEC && n >= 8) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(x) + at * (F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = __ldg(p + i);
        } else {
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = i < n ? (F32 ? static_cast<const uint32_t *>(x)[at + i]
                                    : (uint32_t)static_cast<const uint16_t *>(x)[at + i]) : 0u;
            if (F32) {
                w[0] = make_uint4(r[0], r[1], r[2], r[3]);
                w[F32 ? 1 : 0] = make_uint4(r[4], r[5], r[6], r[7]);
            } else {
                w[0] = pack8(r);
            }
        }
    }
    __device__ __forceinline__ void get(float y[8]) const {
        if (F32) {
            y[0] = __uint_as_float(w[0].x); y[1] = __uint_as_float(w[0].y);
            y[2] = __uint_as_float(w[0].z); y[3] = __uint_as_float(w[0].w);
            y[4] = __uint_as_float(w[F32 ? 1 : 0].x); y[5] = __uint_as_float(w[F32 ? 1 : 0].y);
            y[6] = __uint_as_float(w[F32 ? 1 : 0].z); y[7] = __uint_as_float(w[F32 ? 1 : 0].w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = T::to_f32(lane16(w[0], i));
        }
    }
};

// codes of 8 values of a group whose scale byte is known
__device__ __forceinline__ uint32_t mx4_encode8(const float y[8], uint32_t byte) {
    if (byte == 255u) return 0u;
    const float inv = mx4_inverse(byte);
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __fmul_rn(y[i], inv);
    return e2m1x8(z);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

struct Mx4Args {
    const void *x;
    int64_t rows, cols, ld;
    uint8_t *r_codes, *r_scales;     // along the rows; NULL: not wanted
    uint8_t *c_codes, *c_scales;     // along the columns
    int64_t tiles_c;                 // tiles along the columns of the grid
};

template <class T, bool F32, bool VEC, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256)
mx4_quantize_kernel(Mx4Args a) {
    extern __shared__ __align__(16) uint8_t tile[];              // COLS: the tile as it was read
    __shared__ __align__(16) uint8_t rs[MX4_ATOM], cs[MX4_ATOM];
    constexpr int ES = F32 ? 4 : 2;
    const int t = threadIdx.x;
    const int64_t rt = blockIdx.x / a.tiles_c, ct = blockIdx.x - rt * a.tiles_c;
    const int64_t row0 = rt * QT, col0 = ct * QT;
    const int c8 = (t & 15) * 8;
    const int ncol = (int)min((int64_t)QT, a.cols - col0) - c8;  // of this thread's 8
    constexpr int PASSES = QT / 16;
    Row8<T, F32, VEC> v[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int64_t row = row0 + 16 * i + (t >> 4);
        v[i].load(a.x, row * a.ld + col0 + c8, row < a.rows ? ncol : 0);
    }
    const int64_t row_bytes = mx4_row_bytes(a.cols);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = 16 * i + (t >> 4);
        if (COLS) {
            uint4 *dst = reinterpret_cast<uint4 *>(tile + ((size_t)r * QT + c8) * ES);
#pragma unroll
            for (int j = 0; j < (F32 ? 2 : 1); ++j) dst[j] = v[i].w[j];
        }
        if (ROWS) {
            float y[8];
            v[i].get(y);
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, abs_bits(y[j]));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const uint32_t byte = mx4_scale_byte(top >> 23);
            if ((t & 3) == 0) rs[mx4_in_atom(r, (t & 15) >> 2)] = (uint8_t)byte;
            const int64_t at = (col0 + c8) / 2;
            if (row0 + r < a.rows && at < row_bytes)
                *reinterpret_cast<uint32_t *>(a.r_codes + (row0 + r) * row_bytes + at) = mx4_encode8(y, byte);
        }
    }
    __syncthreads();
    if (COLS) {
        // a thread takes 32 rows of two neighbouring columns
        const int c = 2 * (t & 63), g = t >> 6;
        float y[2][32];
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const size_t at = (size_t)(32 * g + i) * QT + c;
            if (F32) {
                const float2 w = *reinterpret_cast<const float2 *>(tile + at * ES);
                y[0][i] = w.x;
                y[1][i] = w.y;
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + at * ES);
                y[0][i] = T::to_f32(w & 0xFFFFu);
                y[1][i] = T::to_f32(w >> 16);
            }
            top[0] = max(top[0], abs_bits(y[0][i]));
            top[1] = max(top[1], abs_bits(y[1][i]));
        }
        const int64_t bytes = mx4_row_bytes(a.rows), at = row0 / 2 + 16 * g;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t byte = mx4_scale_byte(top[j] >> 23);
            cs[mx4_in_atom(c + j, g)] = (uint8_t)byte;
            if (col0 + c + j < a.cols && at < bytes)
                *reinterpret_cast<uint4 *>(a.c_codes + (col0 + c + j) * bytes + at) =
                    make_uint4(mx4_encode8(y[j], byte), mx4_encode8(y[j] + 8, byte),
                               mx4_encode8(y[j] + 16, byte), mx4_encode8(y[j] + 24, byte));
        }
        __syncthreads();
    }
    // the tile's scale atoms, padding (zero values: scale byte 0) included
    if (ROWS && t < 32 && rt < mx4_row_tiles(a.rows))
        reinterpret_cast<uint4 *>(a.r_scales + (rt * mx4_atoms(a.cols) + ct) * MX4_ATOM)[t] =
            reinterpret_cast<const uint4 *>(rs)[t];
    if (COLS && t >= 32 && t < 64 && ct < mx4_row_tiles(a.cols))
        reinterpret_cast<uint4 *>(a.c_scales + (ct * mx4_atoms(a.rows) + rt) * MX4_ATOM)[t - 32] =
            reinterpret_cast<const uint4 *>(cs)[t - 32];
}

// 8 elements a thread: 4 bytes of codes to 16 or 32 bytes of values
template <class T, bool F32, bool VEC>
__global__ void __launch_bounds__(256)
mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                      int64_t rows, int64_t cols, void *__restrict__ out, int64_t ldo) {
    const int64_t row_bytes = mx4_row_bytes(cols), per = row_bytes / 4, atoms = mx4_atoms(cols);
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= rows * per) return;
    const int64_t row = u / per, c = 8 * (u - row * per), g = c / MX4_GROUP;
    const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(codes) + u);
    const float s = mx4_scale(__ldg(scales + ((row >> 7) * atoms + (g >> 2)) * MX4_ATOM + mx4_in_atom((int)(row & 127), (int)(g & 3))));
    float y[8];
    e2m1_decode8(q, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(y[i], s);
    const int n = (int)min((int64_t)8, cols - c);
    if (F32) {
        float *o = static_cast<float *>(out) + row * ldo + c;
        if (VEC && n == 8) {
            reinterpret_cast<float4 *>(o)[0] = make_float4(y[0], y[1], y[2], y[3]);
            reinterpret_cast<float4 *>(o)[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i < n) o[i] = y[i];
        }
    } else {
        uint16_t *o = static_cast<uint16_t *>(out) + row * ldo + c;
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = T::from_f32(y[i]);
        if (VEC && n == 8) {
            *reinterpret_cast<uint4 *>(o) = pack8(r);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i < n) o[i] = (uint16_t)r[i];
        }
    }
}

struct F32X {
    static __device__ __forceinline__ float to_f32(uint32_t) { return 0.0f; }
    static __device__ __forceinline__ uint32_t from_f32(float) { return 0u; }
};

template <class T, bool F32, bool VEC, bool ROWS, bool COLS>
static cudaError_t quantize_launch(const Mx4Args &a, int64_t grid, cudaStream_t s) {
    const int smem = COLS ? QT * QT * (F32 ? 4 : 2) : 0;
    if (smem > 48 * 1024 - 2 * MX4_ATOM) {
        const cudaError_t e = cudaFuncSetAttribute(mx4_quantize_kernel<T, F32, VEC, ROWS, COLS>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    mx4_quantize_kernel<T, F32, VEC, ROWS, COLS><<<(unsigned)grid, 256, smem, s>>>(a);
    return cudaGetLastError();
}

template <class T, bool F32, bool VEC>
static cudaError_t quantize_ways(const Mx4Args &a, int64_t grid, cudaStream_t s) {
    if (a.r_codes && a.c_codes) return quantize_launch<T, F32, VEC, true, true>(a, grid, s);
    if (a.r_codes) return quantize_launch<T, F32, VEC, true, false>(a, grid, s);
    return quantize_launch<T, F32, VEC, false, true>(a, grid, s);
}

}  // namespace zsk

namespace {

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
bool al16(const void *p) { return p && (addr(p) & 15) == 0; }
bool dtype_ok(int32_t t) { return t >= ZS_DTYPE_BF16 && t <= ZS_DTYPE_FP32; }
constexpr int64_t MX4_MOST = (int64_t)1 << 31;       // rows, columns

zs_status check_held(const void *codes, const void *scales, int64_t rows, int64_t cols, const char *what, const char *fn) {
    if (rows > 0 && cols > 0 && (!al16(codes) || !al16(scales)))
        return zs_fail(ZS_EINVAL, "%s: %s: codes or scales NULL or not 16-byte aligned", fn, what);
    return ZS_OK;
}

zs_status cuda_status(cudaError_t e, const char *fn) {
    if (e != cudaSuccess)
        return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}

zs_status check_matrix(int64_t rows, int64_t cols, const void *p, int64_t ld, int32_t dtype, const char *fn) {
    if (rows < 0 || cols < 0 || rows >= MX4_MOST || cols >= MX4_MOST)
        return zs_fail(ZS_EINVAL, "%s: %lld x %lld out of range", fn, (long long)rows, (long long)cols);
    if (!dtype_ok(dtype)) return zs_fail(ZS_EINVAL, "%s: dtype %d", fn, dtype);
    if (ld < cols) return zs_fail(ZS_EINVAL, "%s: row stride %lld < %lld columns", fn, (long long)ld, (long long)cols);
    if (rows > 0 && cols > 0 && (!p || addr(p) % (dtype == ZS_DTYPE_FP32 ? 4 : 2)))
        return zs_fail(ZS_EINVAL, "%s: matrix NULL or not aligned to its elements", fn);
    return ZS_OK;
}

}  // namespace

extern "C" {

zs_status zs_mx4_sizes(int64_t rows, int64_t cols, int64_t *row_bytes, int64_t *code_bytes, int64_t *scale_bytes) {
    const char *fn = "zs_mx4_sizes";
    if (!row_bytes || !code_bytes || !scale_bytes) return zs_fail(ZS_EINVAL, "%s: NULL result", fn);
    if (rows < 0 || cols < 0 || rows >= MX4_MOST || cols >= MX4_MOST)
        return zs_fail(ZS_EINVAL, "%s: %lld x %lld out of range", fn, (long long)rows, (long long)cols);
    *row_bytes = mx4_row_bytes(cols);
    *code_bytes = rows * mx4_row_bytes(cols);
    *scale_bytes = mx4_row_tiles(rows) * mx4_atoms(cols) * MX4_ATOM;
    zs_clear_error();
    return ZS_OK;
}

zs_status zs_mx4_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                          void *r_codes, void *r_scales, void *c_codes, void *c_scales, void *stream) {
    const char *fn = "zs_mx4_quantize";
    zs_status r = check_matrix(rows, cols, x, ld, dtype, fn);
    if (r) return r;
    const bool along_rows = r_codes || r_scales, along_cols = c_codes || c_scales;
    if (along_rows && (r = check_held(r_codes, r_scales, rows, cols, "along rows", fn))) return r;
    if (along_cols && (r = check_held(c_codes, c_scales, rows, cols, "along columns", fn))) return r;
    if (!along_rows && !along_cols && rows > 0 && cols > 0)
        return zs_fail(ZS_EINVAL, "%s: neither form is asked for", fn);
    if (rows == 0 || cols == 0) {
        zs_clear_error();
        return ZS_OK;
    }
    zsk::Mx4Args a;
    a.x = x; a.rows = rows; a.cols = cols; a.ld = ld;
    a.r_codes = static_cast<uint8_t *>(r_codes);
    a.r_scales = static_cast<uint8_t *>(r_scales);
    a.c_codes = static_cast<uint8_t *>(c_codes);
    a.c_scales = static_cast<uint8_t *>(c_scales);
    // every scale atom is some tile's, the padding ones included
    a.tiles_c = along_rows ? mx4_atoms(cols) : mx4_row_tiles(cols);
    const int64_t tiles_r = along_cols ? mx4_atoms(rows) : mx4_row_tiles(rows);
    const int64_t grid = a.tiles_c * tiles_r;
    if (grid > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: %lld tiles", fn, (long long)grid);
    const cudaStream_t s = (cudaStream_t)stream;
    const int64_t per16 = dtype == ZS_DTYPE_FP32 ? 4 : 8;
    const bool vec = (addr(x) & 15) == 0 && ld % per16 == 0;
    using namespace zsk;
    cudaError_t e;
    if (dtype == ZS_DTYPE_FP32) e = vec ? quantize_ways<F32X, true, true>(a, grid, s) : quantize_ways<F32X, true, false>(a, grid, s);
    else if (dtype == ZS_DTYPE_FP16) e = vec ? quantize_ways<FP16T, false, true>(a, grid, s) : quantize_ways<FP16T, false, false>(a, grid, s);
    else e = vec ? quantize_ways<BF16T, false, true>(a, grid, s) : quantize_ways<BF16T, false, false>(a, grid, s);
    return cuda_status(e, fn);
}

zs_status zs_mx4_dequantize(const void *codes, const void *scales, int64_t rows, int64_t cols, void *out,
                            int64_t ldo, int32_t dtype, void *stream) {
    const char *fn = "zs_mx4_dequantize";
    zs_status r = check_matrix(rows, cols, out, ldo, dtype, fn);
    if (r) return r;
    if ((r = check_held(codes, scales, rows, cols, "matrix", fn))) return r;
    if (rows == 0 || cols == 0) {
        zs_clear_error();
        return ZS_OK;
    }
    const int64_t units = rows * (mx4_row_bytes(cols) / 4), grid = (units + 255) / 256;
    if (grid > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: %lld x %lld too large", fn, (long long)rows, (long long)cols);
    const cudaStream_t s = (cudaStream_t)stream;
    const bool vec = (addr(out) & 15) == 0 && ldo % (dtype == ZS_DTYPE_FP32 ? 4 : 8) == 0;
    const uint8_t *c = static_cast<const uint8_t *>(codes), *sc = static_cast<const uint8_t *>(scales);
    using namespace zsk;
    const dim3 g((unsigned)grid), b(256);
    if (dtype == ZS_DTYPE_FP32) {
        if (vec) mx4_dequantize_kernel<F32X, true, true><<<g, b, 0, s>>>(c, sc, rows, cols, out, ldo);
        else mx4_dequantize_kernel<F32X, true, false><<<g, b, 0, s>>>(c, sc, rows, cols, out, ldo);
    } else if (dtype == ZS_DTYPE_FP16) {
        if (vec) mx4_dequantize_kernel<FP16T, false, true><<<g, b, 0, s>>>(c, sc, rows, cols, out, ldo);
        else mx4_dequantize_kernel<FP16T, false, false><<<g, b, 0, s>>>(c, sc, rows, cols, out, ldo);
    } else {
        if (vec) mx4_dequantize_kernel<BF16T, false, true><<<g, b, 0, s>>>(c, sc, rows, cols, out, ldo);
        else mx4_dequantize_kernel<BF16T, false, false><<<g, b, 0, s>>>(c, sc, rows, cols, out, ldo);
    }
    return cuda_status(cudaGetLastError(), fn);
}

}  // extern "C"
