// Microscaled 4-bit matrices: layout and conversions shared by the quantiser
// and the product.
#pragma once

#include <cuda.h>

#include <atomic>

#include "zs_device.cuh"

constexpr int MX4_GROUP = 32;          // elements that share a scale
constexpr int MX4_ATOM = 512;          // bytes of scales of 128 rows x 4 groups

__host__ __device__ inline int64_t mx4_groups(int64_t cols) { return (cols + MX4_GROUP - 1) / MX4_GROUP; }
__host__ __device__ inline int64_t mx4_row_bytes(int64_t cols) { return 16 * mx4_groups(cols); }
// scale atoms along a row: an even number, so that a 256-element step of the
// product always finds two
__host__ __device__ inline int64_t mx4_atoms(int64_t cols) { return 2 * ((mx4_groups(cols) + 7) / 8); }
__host__ __device__ inline int64_t mx4_row_tiles(int64_t rows) { return (rows + 127) / 128; }
// byte of (row, group) inside its atom: the order in which the tensor cores'
// copy takes scales (32 lanes of 16 bytes, a lane's four rows 32 apart)
__host__ __device__ inline int mx4_in_atom(int row, int group) {
    return (row & 31) * 16 + ((row >> 5) & 3) * 4 + (group & 3);
}

namespace zsk {

// The shared scale of a group whose largest magnitude has this exponent
// field: 2^(floor(log2 max) - 2), stored with bias 127; 255 (NaN) when the
// group holds an infinity or NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t field) {
    return field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
}
__device__ __forceinline__ float mx4_inverse(uint32_t byte) {   // 2^(127 - byte), byte <= 252
    return __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float mx4_scale(uint32_t byte) {     // 2^(byte - 127), NaN for 255
    return byte == 0u ? __uint_as_float(1u << 22)
                      : byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// e2m1 codes of 8 floats, nearest even, saturating at 6; element i in bits
// [4i, 4i + 4)
__device__ __forceinline__ uint32_t e2m1x8(const float y[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// the values of 8 codes
__device__ __forceinline__ void e2m1_decode8(uint32_t codes, float o[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        o[2 * j] = f.x;
        o[2 * j + 1] = f.y;
    }
}

// One wait of a whole warp: the same answer in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_quick(bar, parity, limit_ns));
}

// True in one lane of a converged warp.  The warps that issue loads and
// products run their loops with all lanes and elect one for the issue: under
// `if (lane == 0)` around the whole loop the compiler cannot know that the
// operands are uniform and serialises each instruction, which took 858
// cycles for a stage of products that elected take 512, the tensor cores' own
// rate (2 x 128 x 256 x 256, operands already in shared memory).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void tma2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :
        : "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// cuTensorMapEncodeTiled, through the runtime (no link against the driver).
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static std::atomic<void *> fn{nullptr};
    void *p = fn.load(std::memory_order_relaxed);
    if (!p) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

}  // namespace zsk
