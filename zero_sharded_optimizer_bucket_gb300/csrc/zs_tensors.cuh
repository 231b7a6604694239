// A list of separate tensors, cut into chunks: what its kernels share.
#pragma once

#include <vector>

#include "zs_device.cuh"

constexpr int CHUNK_MOST = 8192;     // elements of a chunk

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
    bool grads_apart = true;         // no element is in two gradients
    std::vector<ZsChunk> chunks;
    const ZsChunk *d_chunks = nullptr;   // caller memory given to zs_tensors_upload
};

namespace zsk {

__device__ __forceinline__ void floats4(const uint4 &v, float o[4]) {
    o[0] = __uint_as_float(v.x); o[1] = __uint_as_float(v.y);
    o[2] = __uint_as_float(v.z); o[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

// Gradient types: 8 elements from global and from shared memory, or one.
struct F32G {
    static constexpr int SIZE = 4;
    static __device__ __forceinline__ void load8(const void *p, int64_t i, float g[8]) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
        floats4(q[0], g);
        floats4(q[1], g + 4);
    }
    static __device__ __forceinline__ void shared8(uint32_t a, float g[8]) {
        floats4(lds16(a), g);
        floats4(lds16(a + 16), g + 4);
    }
    static __device__ __forceinline__ float load1(const void *p, int64_t i) {
        return static_cast<const float *>(p)[i];
    }
};
template <class T>
struct H16G {
    static constexpr int SIZE = 2;
    static __device__ __forceinline__ void convert(const uint4 &v, float g[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = T::to_f32(lane16(v, j));
    }
    static __device__ __forceinline__ void load8(const void *p, int64_t i, float g[8]) {
        convert(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i), g);
    }
    static __device__ __forceinline__ void shared8(uint32_t a, float g[8]) { convert(lds16(a), g); }
    static __device__ __forceinline__ float load1(const void *p, int64_t i) {
        return T::to_f32(static_cast<const uint16_t *>(p)[i]);
    }
};

// The 16-bit copy of 8 new parameters (fp16: the type is a launch argument,
// uniform over the grid).
__device__ __forceinline__ uint4 cast8(const float p[8], bool fp16) {
    uint32_t r[4];
    if (fp16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(p[2 * i], p[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * i], p[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace zsk
