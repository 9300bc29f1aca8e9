// The activation types (float32, bfloat16, float16) as float32 registers, shared by the scan and norm
// kernels.  The type is a run-time value that is the same for a whole launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/stepq.h"

namespace sq {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Round to nearest, ties to even; NaN stays NaN (one conversion instruction on gfx950).
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    const __bf16 v = (__bf16)x;
    uint16_t b;
    __builtin_memcpy(&b, &v, 2);
    return b;
}

__device__ __forceinline__ float f16_val(uint32_t h) {
    const uint16_t b = (uint16_t)h;
    _Float16 v;
    __builtin_memcpy(&v, &b, 2);
    return (float)v;
}
__device__ __forceinline__ uint32_t f16_bits(float x) {
    const _Float16 v = (_Float16)x;
    uint16_t b;
    __builtin_memcpy(&b, &v, 2);
    return b;
}

__device__ __forceinline__ void store1(void* p, int dt, int64_t i, float x) {
    if (dt == SQ_DTYPE_F32) static_cast<float*>(p)[i] = x;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)(dt == SQ_DTYPE_BF16 ? bf16_bits(x) : f16_bits(x));
}

// Eight consecutive elements, 16-byte aligned (float32 in two accesses).
__device__ __forceinline__ void store8(void* p, int dt, int64_t i, const float* x) {
    if (dt == SQ_DTYPE_F32) {
        f32x4 a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) { a[j] = x[j]; b[j] = x[4 + j]; }
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        d[0] = a;
        d[1] = b;
        return;
    }
    u32x4v w;
    if (dt == SQ_DTYPE_BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16_bits(x[2 * j]) | (bf16_bits(x[2 * j + 1]) << 16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f16_bits(x[2 * j]) | (f16_bits(x[2 * j + 1]) << 16);
    }
    *reinterpret_cast<u32x4v*>(static_cast<uint16_t*>(p) + i) = w;
}

template <int V>
__device__ __forceinline__ void storev(void* p, int dt, int64_t i, const float* x) {
    if constexpr (V == 8) store8(p, dt, i, x);
    else store1(p, dt, i, x[0]);
}

}  // namespace sq
