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
            for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = p[i];
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

// m = the larger magnitudes of two pairs of 16-bit values; a NaN stays
template <class T>
__device__ __forceinline__ void max_abs2(uint32_t &m, uint32_t w);
template <>
__device__ __forceinline__ void max_abs2<BF16T>(uint32_t &m, uint32_t w) {
    asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %1;\n\tmax.NaN.bf16x2 %0, %0, a;\n\t}" : "+r"(m) : "r"(w));
}
template <>
__device__ __forceinline__ void max_abs2<FP16T>(uint32_t &m, uint32_t w) {
    asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %1;\n\tmax.NaN.f16x2 %0, %0, a;\n\t}" : "+r"(m) : "r"(w));
}

// codes of 8 values times 2^(127 - byte)
__device__ __forceinline__ uint32_t encode_floats(float y[8], unsigned long long inv) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        unsigned long long two = f2pack(y[i], y[i + 1]);
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(two) : "l"(inv));
        f2unpack(two, y[i], y[i + 1]);
    }
    return e2m1x8(y);
}
template <class T>
__device__ __forceinline__ uint32_t encode_words(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, unsigned long long inv) {
    float y[8];
    const uint32_t w[4] = {w0, w1, w2, w3};
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = T::to_f32(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
    return encode_floats(y, inv);
}

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
    pdl_wait();
    pdl_trigger();
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

// 16-bit matrices whose rows are 16-byte aligned: a persistent CTA walks tiles,
// fetched ahead by tensor copies (two boxes of 64 columns, 128-byte swizzle;
// zeros outside the matrix) into a ring of stages, and makes both forms from
// shared memory.  Along the rows 4 lanes share a group, 8 elements each; along
// the columns a thread takes 32 rows of two neighbouring columns; neither
// access has a bank conflict under the swizzle.  Bandwidth bounds it: 2 bytes
// read and 0.53 written an element and form.
// 8 warps on three CTAs an SM; for both forms every warp makes one after the
// other (8 warps for each on two CTAs took 34 us for 14336 x 4096, this 30).
constexpr int QS_BOX = 64 * 128 * 2, QS_STAGE = 2 * QS_BOX, QS_STAGES = 2, QS_CTAS = 3;
constexpr int QS_SMEM = QS_STAGES * QS_STAGE + 1024;
constexpr uint64_t QS_WAIT_NS = 1000000000ull;       // one wait gives up after 1 s

__device__ int g_quantize_wait_timeouts;             // waits that gave up

template <class T, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256, QS_CTAS)
mx4_quantize_tiles_kernel(const __grid_constant__ CUtensorMap map, Mx4Args a, int tiles) {
    extern __shared__ uint8_t raw[];
    __shared__ __align__(16) uint8_t rs[2][MX4_ATOM], cs[2][MX4_ATOM];
    __shared__ __align__(8) uint64_t bars[QS_STAGES];
    const int t = threadIdx.x;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, bar = smem_u32(bars);
    const int tiles_c = (int)a.tiles_c;
    auto fetch = [&](int i) {                        // the i-th tile of this CTA
        const int tile = (int)blockIdx.x + i * (int)gridDim.x, s = i % QS_STAGES;
        const int rt = tile / tiles_c, ct = tile - rt * tiles_c;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" : : "r"(bar + 8 * s), "r"(QS_STAGE) : "memory");
        tma2d(base + s * QS_STAGE, &map, ct * QT, rt * QT, bar + 8 * s);
        tma2d(base + s * QS_STAGE + QS_BOX, &map, ct * QT + 64, rt * QT, bar + 8 * s);
    };
    const int mine = ((int)(tiles - blockIdx.x) + (int)gridDim.x - 1) / (int)gridDim.x;
    if (t == 0) {
        for (int i = 0; i < QS_STAGES; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" : : "r"(bar + 8 * i) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" : : : "memory");
        pdl_wait();
        pdl_trigger();
        for (int i = 0; i < QS_STAGES && i < mine; ++i) fetch(i);
    }
    __syncthreads();
    const int64_t r_bytes = mx4_row_bytes(a.cols), c_bytes = mx4_row_bytes(a.rows);
    const int64_t r_atoms = mx4_atoms(a.cols), c_atoms = mx4_atoms(a.rows);
    for (int i = 0; i < mine; ++i) {
        const int tile = (int)blockIdx.x + i * (int)gridDim.x, s = i % QS_STAGES;
        const int64_t rt = tile / tiles_c, ct = tile - rt * tiles_c;
        const int64_t row0 = rt * QT, col0 = ct * QT;
        const uint32_t at = base + s * QS_STAGE;
        bool landed = true;
        if (t < 32) landed = mbar_wait_quick(bar + 8 * s, (uint32_t)((i / QS_STAGES) & 1), QS_WAIT_NS);
        if (!__syncthreads_and(landed)) {
            // give up, once the copies in flight have landed
            if (t == 0) {
                atomicAdd(&g_quantize_wait_timeouts, 1);
                for (int j = i; j < i + QS_STAGES && j < mine; ++j)
                    mbar_wait_quick(bar + 8 * (j % QS_STAGES), (uint32_t)((j / QS_STAGES) & 1), QS_WAIT_NS);
            }
            __syncthreads();
            return;
        }
        if (ROWS) {
            // a thread takes a group: 4 lanes a row, 8 rows a warp.  The second
            // box's pieces are read two apart in turn, so that 8 lanes meet 8
            // different pieces of the banks.
            const int g = t & 3, box = g >> 1;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 64 * j + (t >> 2);
                uint32_t w[16], two = 0;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int piece = 4 * (g & 1) + (h ^ (2 * box));
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[4 * h]), "=r"(w[4 * h + 1]), "=r"(w[4 * h + 2]), "=r"(w[4 * h + 3])
                                 : "r"(at + box * QS_BOX + 128 * r + 16 * (piece ^ (r & 7))));
                }
#pragma unroll
                for (int h = 0; h < 16; ++h) max_abs2<T>(two, w[h]);
                const uint32_t byte = mx4_scale_byte(__float_as_uint(T::to_f32(max(two & 0xFFFFu, two >> 16))) >> 23);
                const float inv = byte == 255u ? 0.0f : mx4_inverse(byte);
                uint32_t q[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    q[h] = byte == 255u ? 0u : encode_words<T>(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3], f2pack(inv, inv));
                rs[i & 1][mx4_in_atom(r, g)] = (uint8_t)byte;
                if (row0 + r < a.rows && col0 / 2 + 16 * g < r_bytes)
                    *reinterpret_cast<uint4 *>(a.r_codes + (row0 + r) * r_bytes + col0 / 2 + 16 * g) =
                        box ? make_uint4(q[2], q[3], q[0], q[1]) : make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        if (COLS) {
            // a thread takes 32 rows of two columns; lanes 16 on the same
            // columns' next 32, so that a warp's stores fill sectors.  They
            // read rows 4 apart in turn: other pieces of the banks.
            const int upper = (t >> 4) & 1, g = 2 * (t >> 7) + upper;
            const int box = (t >> 5) & 1, word = 16 * ((t >> 6) & 1) + (t & 15), c = 64 * box + 2 * word;
            uint32_t w[32], two = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {            // rows e, e + 8, ...: the same turn of the swizzle
                const int r = e ^ (4 * upper);
                const uint32_t from = at + box * QS_BOX + 4096 * g + 128 * r + 16 * ((word >> 2) ^ r) + 4 * (word & 3);
#pragma unroll
                for (int h = 0; h < 4; ++h) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[8 * h + e]) : "r"(from + 1024 * h));
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) max_abs2<T>(two, w[e]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t byte = mx4_scale_byte(__float_as_uint(T::to_f32(j ? two >> 16 : two & 0xFFFFu)) >> 23);
                const float inv = byte == 255u ? 0.0f : mx4_inverse(byte);
                cs[i & 1][mx4_in_atom(c + j, g)] = (uint8_t)byte;
                uint32_t q[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = T::to_f32(j ? w[8 * h + e] >> 16 : w[8 * h + e] & 0xFFFFu);
                    const uint32_t x = byte == 255u ? 0u : encode_floats(y, f2pack(inv, inv));
                    q[h] = upper ? __funnelshift_l(x, x, 16) : x;
                }
                if (col0 + c + j < a.cols && row0 / 2 + 16 * g < c_bytes)
                    *reinterpret_cast<uint4 *>(a.c_codes + (col0 + c + j) * c_bytes + row0 / 2 + 16 * g) = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        __syncthreads();                             // the stage is read, the scales are in rs and cs
        if (t == 0 && i + QS_STAGES < mine) fetch(i + QS_STAGES);
        if (ROWS && t >= 32 && t < 64 && rt < mx4_row_tiles(a.rows))
            reinterpret_cast<uint4 *>(a.r_scales + (rt * r_atoms + ct) * MX4_ATOM)[t - 32] = reinterpret_cast<const uint4 *>(rs[i & 1])[t - 32];
        if (COLS && t >= 64 && t < 96 && ct < mx4_row_tiles(a.cols))
            reinterpret_cast<uint4 *>(a.c_scales + (ct * c_atoms + rt) * MX4_ATOM)[t - 64] = reinterpret_cast<const uint4 *>(cs[i & 1])[t - 64];
    }
}

// 32 bytes of values a thread (8 or 16 elements), in 4 rows at a time, so
// that loads overlap and a warp stores whole lines.  Bandwidth bounds it.
// Where the rows of out are not 16-byte aligned a warp turns its 256 values
// through shared memory, and its lanes store neighbours (stored by the thread
// that decoded them, 14335 x 4095 bf16 took 312 us instead of 33; fp32 goes this
// way always, 56 -> 42 us for 14336 x 4096).
constexpr int DQ_ROWS = 4;
__host__ __device__ constexpr int dq_each(bool f32, bool vec) { return vec && !f32 ? 16 : 8; }
template <class T, bool F32, bool VEC>
__global__ void __launch_bounds__(256)
mx4_dequantize_kernel(const uint8_t *codes, const uint8_t *scales,
                      int64_t rows, int64_t cols, void *out, int64_t ldo, uint32_t tiles_c) {
    constexpr int E = dq_each(F32, VEC);
    constexpr bool TURN = F32 || !VEC;
    __shared__ __align__(16) float turn[TURN ? 8 : 1][TURN ? 256 : 1];
    const int64_t row_bytes = mx4_row_bytes(cols), atoms = mx4_atoms(cols);
    const uint32_t rt = blockIdx.x / tiles_c, ct = blockIdx.x - rt * tiles_c;
    const int64_t row0 = (int64_t)rt * DQ_ROWS, c = (int64_t)ct * (256 * E) + E * (int)threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (!TURN && c >= cols) return;
    const int64_t g = c / MX4_GROUP;
    const int n = (int)max((int64_t)0, min((int64_t)E, cols - c));
    uint2 q[DQ_ROWS];
    uint32_t byte[DQ_ROWS];
#pragma unroll
    for (int i = 0; i < DQ_ROWS; ++i) {
        const int64_t row = row0 + i;
        if (row >= rows || n == 0) continue;
        if (E == 8) q[i].x = *reinterpret_cast<const uint32_t *>(codes + row * row_bytes + c / 2);
        else q[i] = *reinterpret_cast<const uint2 *>(codes + row * row_bytes + c / 2);
        byte[i] = scales[((row >> 7) * atoms + (g >> 2)) * MX4_ATOM + mx4_in_atom((int)(row & 127), (int)(g & 3))];
    }
#pragma unroll
    for (int i = 0; i < DQ_ROWS; ++i) {
        const int64_t row = row0 + i;
        if (row >= rows) continue;
        const float s = mx4_scale(byte[i]);
        float y[E];
        e2m1_decode8(q[i].x, y);
        if (E == 16) e2m1_decode8(q[i].y, y + E - 8);
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = __fmul_rn(y[e], s);
        if (TURN) {
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
            const int64_t c0 = c - 8 * lane;         // of the warp
            float4 *t = reinterpret_cast<float4 *>(turn[warp] + 8 * lane);
            t[0] = make_float4(y[0], y[1], y[2], y[3]);
            t[1] = make_float4(y[4], y[5], y[6], y[7]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t col = c0 + 32 * e + lane;
                const float v = turn[warp][32 * e + lane];
                if (col >= cols) continue;
                if (F32) static_cast<float *>(out)[row * ldo + col] = v;
                else static_cast<uint16_t *>(out)[row * ldo + col] = (uint16_t)T::from_f32(v);
            }
            __syncwarp();
            continue;
        }
        uint16_t *o = static_cast<uint16_t *>(out) + row * ldo + c;
        uint32_t r[E];
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = T::from_f32(y[e]);
        if (n == E) {
#pragma unroll
            for (int e = 0; e < E; e += 8) *reinterpret_cast<uint4 *>(o + e) = pack8(r + e);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) if (e < n) o[e] = (uint16_t)r[e];
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
    return launch_dependent(mx4_quantize_kernel<T, F32, VEC, ROWS, COLS>, (unsigned)grid, 256, (size_t)smem, 1, s, a);
}

template <class T, bool ROWS, bool COLS>
static cudaError_t tiles_launch(const Mx4Args &a, int64_t tiles, cudaStream_t s) {
    static std::atomic<int> known[64];           // SMs, once the kernel's shared memory is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = known[dev].load(std::memory_order_relaxed);
    if (sms <= 0) {
        e = cudaFuncSetAttribute(mx4_quantize_tiles_kernel<T, ROWS, COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, QS_SMEM);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    const EncodeTiled f = encode_tiled();
    if (!f) return cudaErrorNotSupported;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)a.cols, (cuuint64_t)a.rows}, strides[1] = {(cuuint64_t)a.ld * 2};
    const cuuint32_t boxes[2] = {64, 128}, ones[2] = {1, 1};
    if (f(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(a.x), dims, strides, boxes, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const int64_t wave = QS_CTAS * (int64_t)sms, grid = tiles < wave ? tiles : wave;
    return launch_dependent(mx4_quantize_tiles_kernel<T, ROWS, COLS>, (unsigned)grid, 256, QS_SMEM, 1, s, map, a, (int)tiles);
}

template <class T>
static cudaError_t tiles_ways(const Mx4Args &a, int64_t tiles, cudaStream_t s) {
    if (a.r_codes && a.c_codes) return tiles_launch<T, true, true>(a, tiles, s);
    if (a.r_codes) return tiles_launch<T, true, false>(a, tiles, s);
    return tiles_launch<T, false, true>(a, tiles, s);
}

template <class T, bool F32, bool VEC>
static cudaError_t quantize_ways(const Mx4Args &a, int64_t grid, cudaStream_t s) {
    if (a.r_codes && a.c_codes) return quantize_launch<T, F32, VEC, true, true>(a, grid, s);
    if (a.r_codes) return quantize_launch<T, F32, VEC, true, false>(a, grid, s);
    return quantize_launch<T, F32, VEC, false, true>(a, grid, s);
}

}  // namespace zsk

cudaError_t zsl_quantize_wait_timeouts(int *count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, zsk::g_quantize_wait_timeouts, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(zsk::g_quantize_wait_timeouts, &zero, sizeof(int));
    }
    return e;
}

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
    else if (dtype == ZS_DTYPE_FP16) e = vec ? tiles_ways<FP16T>(a, grid, s) : quantize_ways<FP16T, false, false>(a, grid, s);
    else e = vec ? tiles_ways<BF16T>(a, grid, s) : quantize_ways<BF16T, false, false>(a, grid, s);
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
    const bool vec = (addr(out) & 15) == 0 && ldo % (dtype == ZS_DTYPE_FP32 ? 4 : 8) == 0;
    const int64_t span = 256 * zsk::dq_each(dtype == ZS_DTYPE_FP32, vec), tiles_c = (cols + span - 1) / span, grid = tiles_c * ((rows + zsk::DQ_ROWS - 1) / zsk::DQ_ROWS);
    if (grid > 0x7FFFFFFF) return zs_fail(ZS_EINVAL, "%s: %lld x %lld too large", fn, (long long)rows, (long long)cols);
    const cudaStream_t s = (cudaStream_t)stream;
    const uint8_t *c = static_cast<const uint8_t *>(codes), *sc = static_cast<const uint8_t *>(scales);
    using namespace zsk;
    auto launch = [&](auto kernel) {
        return launch_dependent(kernel, (unsigned)grid, 256, 0, 1, s, c, sc, rows, cols, out, ldo, (uint32_t)tiles_c);
    };
    cudaError_t e;
    if (dtype == ZS_DTYPE_FP32) e = launch(mx4_dequantize_kernel<F32X, true, false>);
    else if (dtype == ZS_DTYPE_FP16) e = vec ? launch(mx4_dequantize_kernel<FP16T, false, true>) : launch(mx4_dequantize_kernel<FP16T, false, false>);
    else e = vec ? launch(mx4_dequantize_kernel<BF16T, false, true>) : launch(mx4_dequantize_kernel<BF16T, false, false>);
    return cuda_status(e, fn);
}

}  // extern "C"
