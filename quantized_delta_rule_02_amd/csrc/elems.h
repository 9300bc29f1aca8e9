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

// exp(-z) from the hardware's 2^x.  EXACT: the rounding of z log2(e) is put back as a factor, so that its error does not grow with
// |z| (up to 5e-6 of the value at 88 without); results that 16 bits round by 2^-12 or more need it not.  From a = 128 on 2^a is
// infinity, and infinity times a remainder of zero or below would be NaN; far below -126 it is zero: there 2^a stays as it is.
template <bool EXACT>
__device__ __forceinline__ float exp_minus(float z) {
    constexpr float l2e = 1.44269504089f, ln2 = 0.69314718056f;
    const float a = -z * l2e;
    const float e = __builtin_amdgcn_exp2f(a);
    if constexpr (!EXACT) return e;
    const float lo = fmaf(-z, l2e, -a);
    return a < 128.f && a > -200.f ? fmaf(e, lo * ln2, e) : e;
}
// 1 / (1 + exp(-z)); the reciprocal is the hardware's, off by at most one unit in the last place
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + exp_minus<EXACT>(z)); }

}  // namespace sq
