// Device helpers of the selective scan: lane layout, steps, sums over lanes.
//
// A lane holds four states of one channel: lane = channel * (N / 4) + quarter, so a wave holds 256 / N channels, a channel's
// states lie 16 bytes a lane and a wave's states are 1 KB in one piece.
#pragma once
#include <hip/hip_runtime.h>

#include "elems.h"
#include "ssm.h"

namespace sq {

constexpr int kSsmThreads = kSsmWaves * 64;
constexpr float kLog2e = 1.44269504089f;

template <int N>
struct SsmLane {
    static constexpr int kPer = N / 4;                  // lanes of a channel
    static constexpr int kWaveCh = 64 / kPer;           // channels of a wave
    static constexpr int kBlockCh = kSsmWaves * kWaveCh;
};

// ln(1 + e^x) = max(x, 0) + ln(1 + w), w = e^-|x|, by the series of the inverse hyperbolic tangent:
// ln(1 + w) = 2 artanh(v) = 2 v (1 + v^2 / 3 + v^4 / 5 + ...), v = w / (2 + w) <= 1 / 3.  The first term left out, v^16 / 17, is
// below 2^-29; small w keep their digits, which a logarithm of the rounded 1 + w would lose.
__device__ __forceinline__ float softplus(float x) {
    const float w = exp_minus<true>(fabsf(x));
    const float v = w * __builtin_amdgcn_rcpf(2.f + w), q = v * v;
    float s = 1.f / 15.f;
    s = fmaf(s, q, 1.f / 13.f);
    s = fmaf(s, q, 1.f / 11.f);
    s = fmaf(s, q, 1.f / 9.f);
    s = fmaf(s, q, 1.f / 7.f);
    s = fmaf(s, q, 1.f / 5.f);
    s = fmaf(s, q, 1.f / 3.f);
    s = fmaf(s, q, 1.f);
    return fmaf(2.f * v, s, x > 0.f ? x : x <= 0.f ? 0.f : x);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e, kDppHalfMirror = 0x141, kDppMirror = 0x140, kDppRor4 = 0x124, kDppRor8 = 0x128;

// a of lanes l and l ^ 32 (16) exchanged so that each sum of the two results is a sum over both: after it the lower half (even
// rows) has a's sums and the upper half (odd rows) b's.
__device__ __forceinline__ float join32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float join16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over a channel's PER lanes; all of them get it.
template <int PER>
__device__ __forceinline__ float channel_sum(float x) {
    if constexpr (PER >= 2) x += dpp<kDppXor1>(x);
    if constexpr (PER >= 4) x += dpp<kDppXor2>(x);
    if constexpr (PER >= 8) x += dpp<kDppHalfMirror>(x);
    if constexpr (PER >= 16) x += dpp<kDppMirror>(x);
    if constexpr (PER >= 32) x = join16(x, x);
    return x;
}

// Where block `blk` of a launch has its channels: the first one, and how many (none of two groups).
struct SsmBlock {
    int group, c0, n;
};
__device__ __forceinline__ SsmBlock block_channels(const SsmParams& p, int blk, int per) {
    const int in_group = (p.group_channels + per - 1) / per, g = blk / in_group, at = (blk - g * in_group) * per;
    const int left = p.group_channels - at;
    return SsmBlock{g, g * p.group_channels + at, left < per ? left : per};
}

// Four adjacent elements, of which n (maybe none) are there; the others are zero.
template <int DT, bool VEC>
struct Four {
    Elems<DT, VEC ? 4 : 1> e[VEC ? 1 : 4];
    __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
        if constexpr (VEC) {
            e[0].zero();
            if (n > 0) e[0].load(p, i);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                e[j].zero();
                if (j < n) e[j].load(p, i + j);
            }
        }
    }
    __device__ __forceinline__ float at(int j) const {
        if constexpr (VEC) return e[0].at(j);
        else return e[j].at(0);
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, int n, const float* x) {
        if constexpr (VEC) {
            Elems<DT, 4> o;
            o.set(x);
            if (n > 0) o.store(p, i);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Elems<DT, 1> o;
                o.set(x + j);
                if (j < n) o.store(p, i + j);
            }
        }
    }
};

__device__ __forceinline__ f32x4 load_states(const float* p, int64_t i, bool there) {
    f32x4 h{0.f, 0.f, 0.f, 0.f};
    if (there) h = *reinterpret_cast<const f32x4*>(p + i);
    return h;
}

#define SQ_SSM_DISPATCH_DT(fn, N, ...)                                                                        \
    do {                                                                                                      \
        if (p.dtype == SQ_DTYPE_BF16) return vec ? fn<SQ_DTYPE_BF16, N, true>(__VA_ARGS__) : fn<SQ_DTYPE_BF16, N, false>(__VA_ARGS__); \
        if (p.dtype == SQ_DTYPE_F16) return vec ? fn<SQ_DTYPE_F16, N, true>(__VA_ARGS__) : fn<SQ_DTYPE_F16, N, false>(__VA_ARGS__);    \
        return vec ? fn<SQ_DTYPE_F32, N, true>(__VA_ARGS__) : fn<SQ_DTYPE_F32, N, false>(__VA_ARGS__);          \
    } while (0)
#define SQ_SSM_DISPATCH(fn, ...)                                          \
    do {                                                                  \
        if (p.d_state == 8) SQ_SSM_DISPATCH_DT(fn, 8, __VA_ARGS__);        \
        if (p.d_state == 16) SQ_SSM_DISPATCH_DT(fn, 16, __VA_ARGS__);      \
        if (p.d_state == 32) SQ_SSM_DISPATCH_DT(fn, 32, __VA_ARGS__);      \
        if (p.d_state == 64) SQ_SSM_DISPATCH_DT(fn, 64, __VA_ARGS__);      \
        if (p.d_state == 128) SQ_SSM_DISPATCH_DT(fn, 128, __VA_ARGS__);    \
        return hipErrorInvalidValue;                                      \
    } while (0)

}  // namespace sq
