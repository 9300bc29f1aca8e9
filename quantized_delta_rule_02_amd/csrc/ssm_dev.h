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
    static constexpr int kPad = (kWaveCh + 3) / 4 * 4;  // between rows of a tile: four tokens of a wave meet no bank twice, and rows
                                                        // stay aligned to the four elements that are read from them at a time
    static_assert(kBlockCh % 4 == 0 && (kBlockCh + kPad) % 4 == 0, "rows are accessed four elements at a time");
};

// ln(1 + e^x) = max(x, 0) + ln(1 + w), w = e^-|x|.  w comes from 2^y with the rounding of y = -|x| log2(e) put back (|x| + y ln 2 is
// exact but for ln 2's own rounding, 2^-28); beyond 150 it is below every float32 (min drops a NaN there, the last line brings it
// back).  ln(1 + w) = w P(w) with the polynomial of degree 8 that has the least relative error on [0, 1], 2^-25 (by Remez exchange),
// so that small w keep their digits, which a logarithm of the rounded 1 + w would lose.
struct SoftPlus {
    float w, value;
};
__device__ __forceinline__ SoftPlus softplus(float x) {
    const float m = fminf(fabsf(x), 150.f), y = -m * kLog2e;
    float w = __builtin_amdgcn_exp2f(y);
    w = fmaf(w, fmaf(-y, 0.69314718056f, -m), w);
    float s = 0.0052326940931379795f;
    s = fmaf(s, w, -0.02950523979961872f);
    s = fmaf(s, w, 0.07822595536708832f);
    s = fmaf(s, w, -0.13663245737552643f);
    s = fmaf(s, w, 0.19106006622314453f);
    s = fmaf(s, w, -0.2484298199415207f);
    s = fmaf(s, w, 0.3331909775733948f);
    s = fmaf(s, w, -0.4999949336051941f);
    s = fmaf(s, w, 0.9999999403953552f);
    return SoftPlus{w, fmaf(w, s, x <= 0.f ? 0.f : x)};
}
// its derivative 1 / (1 + e^-x) from the same w
__device__ __forceinline__ float softplus_slope(float x, float w) {
    const float r = __builtin_amdgcn_rcpf(1.f + w);
    return x <= 0.f ? w * r : r;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e, kDppHalfMirror = 0x141, kDppMirror = 0x140, kDppRor4 = 0x124, kDppRor8 = 0x128;
constexpr int kDppShl4 = 0x104, kDppShl8 = 0x108;      // lane i gets lane i + 4, i + 8 of its row of 16

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

// Sums over a channel's lanes of four tokens' values at a time: lane q < 4 of the channel gets token q's (PER = 2: lane q < 2 those of
// tokens q and q + 2).  Each exchange sends the half of the tokens that the lane does not keep, so four sums take nine instructions
// instead of the eight and four masked stores of one after another.  The order of the additions is channel_sum's.
template <int PER>
__device__ __forceinline__ void channel_sums4(float (&v)[4]) {
    const int lane = (int)threadIdx.x;
    const bool odd = lane & 1, high = lane & 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {                        // tokens 2 k and 2 k + 1
        const float keep = odd ? v[2 * k + 1] : v[2 * k], send = odd ? v[2 * k] : v[2 * k + 1];
        v[2 * k] = keep + dpp<kDppXor1>(send);
    }
    if constexpr (PER >= 4) {
        const float keep = high ? v[2] : v[0], send = high ? v[0] : v[2];
        v[0] = keep + dpp<kDppXor2>(send);
        // lanes q, q + 4, ... now hold the same token's sums of their quads
        if constexpr (PER >= 8) v[0] += dpp<kDppShl4>(v[0]);
        if constexpr (PER >= 16) v[0] += dpp<kDppShl8>(v[0]);
        if constexpr (PER >= 32) v[0] = join16(v[0], v[0]);
    }
}

// Where lane `quarter` of a channel puts what channel_sums4 left it: put(token, value).
template <int PER, class Put>
__device__ __forceinline__ void put_sums4(const float (&v)[4], int quarter, Put put) {
    if constexpr (PER == 2) {
        put(quarter, v[0]);
        put(quarter + 2, v[2]);
    } else if constexpr (PER == 4) {
        put(quarter, v[0]);
    } else {
        if (quarter < 4) put(quarter, v[0]);
    }
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
