// V adjacent elements of an activation type known at compile time: as loaded, as float32, and stored with one rounding each.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vec.h"

namespace sq {

template <int DT>
constexpr int kBytes = DT == SQ_DTYPE_F32 ? 4 : 2;

template <int DT, int V>
struct Elems {
    static constexpr int kWords = (V * kBytes<DT> + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    // from element i of p; V > 1: aligned to the V elements (at most 16 bytes an access)
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const char* s = static_cast<const char*>(p) + i * kBytes<DT>;
        if constexpr (V * kBytes<DT> == 2) w[0] = *reinterpret_cast<const uint16_t*>(s);
        else if constexpr (kWords == 1) w[0] = *reinterpret_cast<const uint32_t*>(s);
        else if constexpr (kWords == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(s);
            w[0] = x.x;
            w[1] = x.y;
        } else {
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                const u32x4v x = reinterpret_cast<const u32x4v*>(s)[k];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * k + j] = x[j];
            }
        }
    }
    // element `lane` of the row at element `row` of p: the row the same for the wave, so that it stays in scalar registers
    __device__ __forceinline__ void load(const void* p, int64_t row, uint32_t lane) {
        load(static_cast<const char*>(p) + row * kBytes<DT> + (uint64_t)(lane * (uint32_t)kBytes<DT>), 0);
    }
    __device__ __forceinline__ void store(void* p, int64_t row, uint32_t lane) const {
        store(static_cast<char*>(p) + row * kBytes<DT> + (uint64_t)(lane * (uint32_t)kBytes<DT>), 0);
    }
    __device__ __forceinline__ void store_once(void* p, int64_t row, uint32_t lane) const {
        store_once(static_cast<char*>(p) + row * kBytes<DT> + (uint64_t)(lane * (uint32_t)kBytes<DT>), 0);
    }
    // the bits as they are
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        char* s = static_cast<char*>(p) + i * kBytes<DT>;
        if constexpr (V * kBytes<DT> == 2) *reinterpret_cast<uint16_t*>(s) = (uint16_t)w[0];
        else if constexpr (kWords == 1) *reinterpret_cast<uint32_t*>(s) = w[0];
        else if constexpr (kWords == 2) *reinterpret_cast<uint2*>(s) = uint2{w[0], w[1]};
        else {
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                u32x4v x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = w[4 * k + j];
                reinterpret_cast<u32x4v*>(s)[k] = x;
            }
        }
    }
    // the same past the caches' usual order: rows that the launch does not read again
    __device__ __forceinline__ void store_once(void* p, int64_t i) const {
        char* s = static_cast<char*>(p) + i * kBytes<DT>;
        if constexpr (V * kBytes<DT> == 2) __builtin_nontemporal_store((uint16_t)w[0], reinterpret_cast<uint16_t*>(s));
        else {
#pragma unroll
            for (int k = 0; k < kWords; ++k) __builtin_nontemporal_store(w[k], reinterpret_cast<uint32_t*>(s) + k);
        }
    }
    __device__ __forceinline__ float at(int j) const {
        if constexpr (DT == SQ_DTYPE_F32) return __uint_as_float(w[j]);
        else if constexpr (DT == SQ_DTYPE_BF16) return (j & 1) ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
        else return f16_val((j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
    }
    __device__ __forceinline__ void set(const float* x) {
        if constexpr (DT == SQ_DTYPE_F32) {
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = __float_as_uint(x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const float hi = 2 * j + 1 < V ? x[2 * j + 1] : 0.f;
                w[j] = DT == SQ_DTYPE_BF16 ? bf16_bits(x[2 * j]) | (bf16_bits(hi) << 16) : f16_bits(x[2 * j]) | (f16_bits(hi) << 16);
            }
        }
    }
};

// 1 / (1 + exp(-z)) to 9 2^-24 of itself for |z| up to 64, with exp(-z) = 2^a (1 - r): a = -z log2(e) rounded, r = a ln 2 + z, exact but for ln 2's own
// rounding (2^-28), so that the error does not grow with |z| by more than that.  Beyond 200 the power is zero or infinite either way, and r
// stays small.  The reciprocal is the hardware's, off by at most one unit in the last place.  A NaN gives a number: every gate is
// multiplied by z itself.  Rows of 16 bits have float32 results too (sums over tokens, gradients of states), so they get the same gates.
__device__ __forceinline__ float sigmoid(float z) {
    const float x = __builtin_amdgcn_fmed3f(z, -200.f, 200.f), a = -x * 1.44269504089f;
    return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(a), 1.f - fmaf(a, 0.69314718056f, x), 1.f));
}

}  // namespace sq
