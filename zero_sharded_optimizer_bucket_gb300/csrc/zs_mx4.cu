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
// m = the larger of m and |x|; a NaN stays
__device__ __forceinline__ void max_abs(float &m, float x) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x)));
}

struct Mx4Args {
    const void *x;
    int64_t rows, cols, ld;
    uint8_t *r_codes, *r_scales;     // along the rows; NULL: not wanted
    uint8_t *c_codes, *c_scales;     // along the columns
    int64_t tiles_c;                 // tiles along the columns of the grid
    int32_t give_up;                 // for tests: the unit of each CTA whose wait runs out, or -1
};

// The scale byte of a group and the factor of its values (0 for a NaN group,
// whose codes are 0), from its largest magnitude.
struct Mx4Scale {
    uint32_t byte;
    float inv;
    // a code word of the group
    __device__ __forceinline__ uint32_t codes(float y[8]) const { return byte == 255u ? 0u : encode_floats(y, f2pack(inv, inv)); }
};
__device__ __forceinline__ Mx4Scale mx4_scale(float top) {
    const uint32_t byte = mx4_scale_byte(__float_as_uint(top) >> 23);
    return {byte, byte == 255u ? 0.0f : mx4_inverse(byte)};
}

// A persistent CTA walks tiles, each in units of 32 KB (a tile of 16-bit
// values, or half the columns of an fp32 one), and makes both forms from shared
// memory.  A unit lies there as two boxes of 128 rows by 128 bytes, 16-byte
// pieces turned by the row (128-byte swizzle).  Along the rows a thread takes
// groups of 32 elements; along the columns, 32 rows of two neighbouring
// columns (fp32: of one); neither has a bank conflict under the swizzle, and a
// warp's stores fill sectors.  Bandwidth bounds it: 2 or 4 bytes read and 0.53
// written an element and form.
// BOXES: the rows of x are 16-byte aligned, and tensor copies fetch the units
// ahead into a ring of stages, with zeros outside the matrix.  Otherwise lanes
// load neighbouring elements of a row, whatever its address; the CTAs of an SM
// overlap one another's loads, and how many are in flight bounds it.
// 8 warps on three CTAs an SM; for both forms every warp makes one after the
// other (8 warps for each on two CTAs took 34 us for 14336 x 4096, this 30).
// 14336 x 4096 along the rows, the columns, both: bf16 24, 25 and 30 us (6.1,
// 5.9, 6.0 TB/s), fp32 41, 41 and 48 (6.5, 6.4, 6.2); 14335 x 4095: bf16 42, 47
// and 58 us (3.6, 3.2, 3.1 TB/s), fp32 46, 51 and 62 (5.7, 5.2, 4.8).
constexpr int QS_BOX = 128 * 128, QS_STAGE = 2 * QS_BOX, QS_STAGES = 2, QS_CTAS = 3;
constexpr uint64_t QS_WAIT_NS = 1000000000ull;       // one wait gives up after 1 s
constexpr int qs_smem(bool boxes) { return (boxes ? QS_STAGES : 1) * QS_STAGE + 1024; }

__device__ int g_quantize_wait_timeouts;             // waits that gave up

template <class T, bool F32, bool BOXES, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256, QS_CTAS)
mx4_quantize_kernel(const __grid_constant__ CUtensorMap map, Mx4Args a, int tiles) {
    constexpr int UNITS = F32 ? 2 : 1;               // of a tile
    constexpr int BOX_COLS = F32 ? 32 : 64, UNIT_COLS = 2 * BOX_COLS;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(16) uint8_t rs[2][MX4_ATOM], cs[2][MX4_ATOM];
    __shared__ __align__(8) uint64_t bars[QS_STAGES];
    const int t = threadIdx.x;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, bar = smem_u32(bars);
    const int tiles_c = (int)a.tiles_c;
    auto fetch = [&](int u) {                        // the u-th unit of this CTA
        const int tile = (int)blockIdx.x + u / UNITS * (int)gridDim.x, s = u % QS_STAGES;
        const int rt = tile / tiles_c, ct = tile - rt * tiles_c;
        const int col = ct * QT + u % UNITS * UNIT_COLS;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" : : "r"(bar + 8 * s), "r"(QS_STAGE + (u == a.give_up ? 16 : 0)) : "memory");
        tma2d(base + s * QS_STAGE, &map, col, rt * QT, bar + 8 * s);
        tma2d(base + s * QS_STAGE + QS_BOX, &map, col + BOX_COLS, rt * QT, bar + 8 * s);
    };
    const int mine = ((int)(tiles - blockIdx.x) + (int)gridDim.x - 1) / (int)gridDim.x * UNITS;
    if (BOXES && t == 0) {
        for (int i = 0; i < QS_STAGES; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" : : "r"(bar + 8 * i) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" : : : "memory");
    }
    if (!BOXES || t == 0) {
        pdl_wait();
        pdl_trigger();
    }
    if (BOXES && t == 0)
        for (int u = 0; u < QS_STAGES && u < mine; ++u) fetch(u);
    __syncthreads();
    const int64_t r_bytes = mx4_row_bytes(a.cols), c_bytes = mx4_row_bytes(a.rows);
    const int64_t r_atoms = mx4_atoms(a.cols), c_atoms = mx4_atoms(a.rows);
    for (int u = 0; u < mine; ++u) {
        const int i = u / UNITS, half = u % UNITS;
        const int tile = (int)blockIdx.x + i * (int)gridDim.x, s = BOXES ? u % QS_STAGES : 0;
        const int64_t rt = tile / tiles_c, ct = tile - rt * tiles_c;
        const int64_t row0 = rt * QT, col0 = ct * QT + half * UNIT_COLS;
        const uint32_t at = base + s * QS_STAGE;
        if (BOXES) {
            bool landed = true;
            if (t < 32) landed = mbar_wait_quick(bar + 8 * s, (uint32_t)((u / QS_STAGES) & 1), QS_WAIT_NS);
            if (!__syncthreads_and(landed)) {
                // give up, once the copies in flight have landed
                if (t == 0) {
                    atomicAdd(&g_quantize_wait_timeouts, 1);
                    for (int j = u; j < u + QS_STAGES && j < mine; ++j)
                        mbar_wait_quick(bar + 8 * (j % QS_STAGES), (uint32_t)((j / QS_STAGES) & 1), QS_WAIT_NS);
                }
                __syncthreads();
                return;
            }
        } else {
            // a warp takes every 8th row, with LOADS loads of a lane in flight
            // (14335 x 4095 bf16 along the rows: 54 us with half as many; pairs
            // of elements in one load, which odd rows cannot use, 54 and more)
            constexpr int A_ROW = UNIT_COLS / 32, LOADS = 32, PER = LOADS / A_ROW;
            const int lane = t & 31;
#pragma unroll 1
            for (int r0 = t >> 5; r0 < QT; r0 += 8 * PER) {
                uint32_t w[LOADS];
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const int64_t row = row0 + r0 + 8 * (j / A_ROW), col = col0 + 32 * (j % A_ROW) + lane;
                    w[j] = 0;
                    if (row < a.rows && col < a.cols)
                        w[j] = F32 ? static_cast<const uint32_t *>(a.x)[row * a.ld + col]
                                   : (uint32_t)static_cast<const uint16_t *>(a.x)[row * a.ld + col];
                }
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const int r = r0 + 8 * (j / A_ROW), c = 32 * (j % A_ROW) + lane, b = (c % BOX_COLS) * (F32 ? 4 : 2);
                    const uint32_t to = at + c / BOX_COLS * QS_BOX + 128 * r + 16 * ((b >> 4) ^ (r & 7)) + (b & 15);
                    if (F32) asm volatile("st.shared.b32 [%0], %1;" : : "r"(to), "r"(w[j]) : "memory");
                    else asm volatile("st.shared.u16 [%0], %1;" : : "r"(to), "h"((uint16_t)w[j]) : "memory");
                }
            }
            __syncthreads();
        }
        if (ROWS) {
            // a thread takes a group, of 64 or 128 bytes of a row.  The second
            // box's pieces are read two (fp32: four) apart in turn, so that 8
            // lanes meet 8 different pieces of the banks.
            constexpr int A_ROW = UNIT_COLS / 32;    // groups
            const int g = t % A_ROW, box = g / (A_ROW / 2);
#pragma unroll
            for (int j = 0; j < A_ROW / 2; ++j) {
                const int r = 256 / A_ROW * j + t / A_ROW;
                uint32_t q[4];
                uint32_t byte;
                if constexpr (F32) {
                    float w[32], top = 0.0f;
#pragma unroll
                    for (int h = 0; h < 8; ++h)
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(w[4 * h]), "=f"(w[4 * h + 1]), "=f"(w[4 * h + 2]), "=f"(w[4 * h + 3])
                                     : "r"(at + box * QS_BOX + 128 * r + 16 * (h ^ (4 * box) ^ (r & 7))));
#pragma unroll
                    for (int h = 0; h < 32; ++h) max_abs(top, w[h]);
                    const Mx4Scale sc = mx4_scale(top);
                    byte = sc.byte;
#pragma unroll
                    for (int h = 0; h < 4; ++h) q[h] = sc.codes(w + 8 * h);
                } else {
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
                    const Mx4Scale sc = mx4_scale(T::to_f32(max(two & 0xFFFFu, two >> 16)));
                    byte = sc.byte;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = T::to_f32(e & 1 ? w[4 * h + (e >> 1)] >> 16 : w[4 * h + (e >> 1)] & 0xFFFFu);
                        q[h] = sc.codes(y);
                    }
                }
                rs[i & 1][mx4_in_atom(r, A_ROW * half + g)] = (uint8_t)byte;
                if (row0 + r < a.rows && col0 / 2 + 16 * g < r_bytes)
                    *reinterpret_cast<uint4 *>(a.r_codes + (row0 + r) * r_bytes + col0 / 2 + 16 * g) =
                        box ? make_uint4(q[2], q[3], q[0], q[1]) : make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        if (COLS) {
            // a thread takes 32 rows of a word (two columns, or one fp32);
            // lanes 16 on the same words' next 32, so that a warp's stores
            // fill sectors.  They read rows 4 apart in turn: other pieces of
            // the banks.
            constexpr int COLUMNS = F32 ? 1 : 2;     // of a word
            const int upper = (t >> 4) & 1, g = 2 * (t >> 7) + upper;
            const int box = (t >> 5) & 1, word = 16 * ((t >> 6) & 1) + (t & 15), c = BOX_COLS * box + COLUMNS * word;
            uint32_t w[32], two = 0;
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {            // rows e, e + 8, ...: the same turn of the swizzle
                const int r = e ^ (4 * upper);
                const uint32_t from = at + box * QS_BOX + 4096 * g + 128 * r + 16 * ((word >> 2) ^ r) + 4 * (word & 3);
#pragma unroll
                for (int h = 0; h < 4; ++h) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[8 * h + e]) : "r"(from + 1024 * h));
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if constexpr (F32) max_abs(top, __uint_as_float(w[e]));
                else max_abs2<T>(two, w[e]);
            }
#pragma unroll
            for (int j = 0; j < COLUMNS; ++j) {
                if constexpr (!F32) top = T::to_f32(j ? two >> 16 : two & 0xFFFFu);
                const Mx4Scale sc = mx4_scale(top);
                cs[i & 1][mx4_in_atom(half * UNIT_COLS + c + j, g)] = (uint8_t)sc.byte;
                uint32_t q[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = F32 ? __uint_as_float(w[8 * h + e]) : T::to_f32(j ? w[8 * h + e] >> 16 : w[8 * h + e] & 0xFFFFu);
                    const uint32_t x = sc.codes(y);
                    q[h] = upper ? __funnelshift_l(x, x, 16) : x;
                }
                if (col0 + c + j < a.cols && row0 / 2 + 16 * g < c_bytes)
                    *reinterpret_cast<uint4 *>(a.c_codes + (col0 + c + j) * c_bytes + row0 / 2 + 16 * g) = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        __syncthreads();                             // the stage is read, the scales are in rs and cs
        if (BOXES && t == 0 && u + QS_STAGES < mine) fetch(u + QS_STAGES);
        if (half != UNITS - 1) continue;
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
// way always, 56 -> 41 us for 14336 x 4096, 6.5 TB/s; bf16 26 us, 5.8 TB/s).
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

template <class T, bool F32, bool BOXES, bool ROWS, bool COLS>
static cudaError_t quantize_launch(const Mx4Args &a, int64_t tiles, cudaStream_t s) {
    static std::atomic<int> known[64];           // SMs, once the kernel's shared memory is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = known[dev].load(std::memory_order_relaxed);
    if (sms <= 0) {
        e = cudaFuncSetAttribute(mx4_quantize_kernel<T, F32, BOXES, ROWS, COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, qs_smem(BOXES));
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    CUtensorMap map = {};
    if (BOXES) {
        const EncodeTiled f = encode_tiled();
        if (!f) return cudaErrorNotSupported;
        const cuuint64_t dims[2] = {(cuuint64_t)a.cols, (cuuint64_t)a.rows}, strides[1] = {(cuuint64_t)a.ld * (F32 ? 4 : 2)};
        const cuuint32_t boxes[2] = {F32 ? 32 : 64, 128}, ones[2] = {1, 1};
        if (f(&map, F32 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(a.x), dims, strides, boxes, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const int64_t wave = QS_CTAS * (int64_t)sms, grid = tiles < wave ? tiles : wave;
    return launch_dependent(mx4_quantize_kernel<T, F32, BOXES, ROWS, COLS>, (unsigned)grid, 256, qs_smem(BOXES), 1, s, map, a, (int)tiles);
}

template <class T, bool F32, bool BOXES>
static cudaError_t quantize_ways(const Mx4Args &a, int64_t tiles, cudaStream_t s) {
    if (a.r_codes && a.c_codes) return quantize_launch<T, F32, BOXES, true, true>(a, tiles, s);
    if (a.r_codes) return quantize_launch<T, F32, BOXES, true, false>(a, tiles, s);
    return quantize_launch<T, F32, BOXES, false, true>(a, tiles, s);
}

template <class T, bool F32>
static cudaError_t quantize_rows(const Mx4Args &a, int64_t tiles, bool boxes, cudaStream_t s) {
    return boxes ? quantize_ways<T, F32, true>(a, tiles, s) : quantize_ways<T, F32, false>(a, tiles, s);
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
    a.give_up = zsl_test_give_up();
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
    // tensor copies: aligned rows, and a stride that a tensor map holds (2^40 bytes)
    const bool boxes = (addr(x) & 15) == 0 && ld % per16 == 0 && ld < ((int64_t)1 << 37);
    using namespace zsk;
    cudaError_t e;
    if (dtype == ZS_DTYPE_FP32) e = quantize_rows<F32X, true>(a, grid, boxes, s);
    else if (dtype == ZS_DTYPE_FP16) e = quantize_rows<FP16T, false>(a, grid, boxes, s);
    else e = quantize_rows<BF16T, false>(a, grid, boxes, s);
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
