// Rows of a cache held in 8 or 4 bits: quantised as they are written, and read back (gfx950).
//
//   s = max |x| / Q over a group of a row, rounded to float32;   code = the format's value nearest to x / s, ties to even
//   value read back = code * s                                    Q = 127 (int8), 7 (int4), 448 (e4m3)
//
// The code is that of the exact quotient of x and the stored s: a rounded quotient could fall on the middle between two codes.
// With k the nearest step count of an approximate quotient, x - k u s (u the step, 1 for integers) is exact in one fused
// multiply-add: k u has at most 8 bits, so k u s and x differ by a multiple of the last place of u s of at most half of u s or a
// little more; comparing it with u s / 2 tells whether k is the nearest one.
//
// An approximate quotient settles nearly all codes: with x / s to 2^-22, only values within 2^-11 of half a step of a middle take the
// exact way (one wave in ten has one).  12301 rows of 1024 bfloat16 elements into int8: 11.4 us (3.3 TB/s; every code the exact way:
// 13.1), of which 3 are the launch; 65536 such rows read back from slots in any order: 44 us, 4.6 TB/s (52 with each row's slot,
// codes and scale one after another instead of four of each in flight).  64 rows: the launch, 4 us on the GPU, 8.5 of host time.
//
// Memory bounds both: every row is read and written once.  A thread holds eight elements (16 bytes of a 16-bit type) and the
// threads of a group, a power of two of one wave, find its maximum by lane exchanges; the group's bits are compared as
// integers, so that a NaN or an infinity is the maximum and makes the scale NaN.  Rows of odd strides go element by element: 12301 rows of 1024
// written in 34 us (aligned 11.9), read in 17 (7.8, one set of inputs).
#include <hip/hip_runtime.h>

#include "cache.h"
#include "elems.h"

namespace sq {

constexpr int kThreads = 256;

template <int F>
constexpr float kTop = F == SQ_CACHE_INT8 ? 127.f : F == SQ_CACHE_INT4 ? 7.f : 448.f;

// A group's scale, and what its codes are found with: x and s times `up` (a power of two that keeps tiny scales normal).
struct Scale {
    float s, su, inv, up;
};
template <int F>
__device__ __forceinline__ Scale scale_of(uint32_t max_bits) {
    Scale k;
    k.s = max_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(max_bits) / kTop<F>;
    k.up = k.s < 0x1p-100f ? 0x1p64f : 1.f;
    k.su = k.s * k.up;
    k.inv = k.s > 0.f ? __builtin_amdgcn_rcpf(k.su) : 0.f;      // a scale of zero or NaN: codes of zero
    return k;
}

// The nearest code as the number it stands for (before the scale).
template <int F>
__device__ __forceinline__ float code_of(const Scale& k, float x) {
    const float xu = x * k.up, y = k.inv == 0.f ? 0.f : xu * k.inv;
    float u = 1.f, n;
    if constexpr (F == SQ_CACHE_E4M3) {                          // steps of 2^(e - 3), e the exponent, of 2^-9 below 2^-6
        int e = (int)((__float_as_uint(y) >> 23) & 255u);
        e = e < 121 ? 121 : e;
        u = __uint_as_float((uint32_t)(e - 3) << 23);
        n = rintf(y * __uint_as_float((uint32_t)(254 - (e - 3)) << 23));
    } else {
        n = rintf(y);
    }
    const float us = u * k.su, r2 = 2.f * fmaf(-n * u, k.su, xu);
    const bool odd = ((int)n & 1) != 0;
    if (r2 > us || (r2 == us && odd)) n += 1.f;
    else if (r2 < -us || (r2 == -us && odd)) n -= 1.f;
    n = k.inv == 0.f ? 0.f : n * u;
    return fminf(fmaxf(n, -kTop<F>), kTop<F>);
}

// n / d for n below 2^31: with l = ceil(log2 d) and m = floor(2^(31 + l) / d) + 1, m d is 2^(31 + l) + e, 0 < e <= d <= 2^l, so that
// n m / 2^(31 + l) exceeds n / d by less than 1 / d.
struct Div {
    uint32_t m;
    int32_t s;
    explicit Div(uint32_t d) {
        int l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        s = 31 + l;
        m = (uint32_t)((uint64_t(1) << s) / d + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> s); }
};

// Eight codes as stored: 8 bytes, or 4 for 4-bit codes (the first of two in the low half of its byte).
template <int F>
__device__ __forceinline__ uint2 pack8(const float* v) {
    uint2 w{0, 0};
    if constexpr (F == SQ_CACHE_E4M3) {
        w.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        w.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], (int)w.x, true);
        w.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
        w.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], (int)w.y, true);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = (uint32_t)(int)v[j];
            if constexpr (F == SQ_CACHE_INT4) w.x |= (c & 15u) << (4 * j);
            else if (j < 4) w.x |= (c & 255u) << (8 * j);
            else w.y |= (c & 255u) << (8 * (j - 4));
        }
    }
    return w;
}
template <int F>
__device__ __forceinline__ float unpack1(uint32_t c) {           // of a code in the low bits
    if constexpr (F == SQ_CACHE_E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)(c & 255u), 0);
    else if constexpr (F == SQ_CACHE_INT8) return (float)(int8_t)(c & 255u);
    else return (float)((int32_t)(c << 28) >> 28);
}

// Eight codes by the approximate quotient; `near` grows to 1 or more where one of them comes within 2^-11 of half a step of the
// middle between two codes (the quotient is off by 2^-22 of itself, 2^-15 of a step at most): there only the exact remainder tells.
template <int F>
__device__ __forceinline__ uint2 quick8(const Scale& k, const float* x, float& near) {
    uint2 w{0, 0};
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j] * k.inv;
    if constexpr (F == SQ_CACHE_E4M3) {
        w.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        w.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], (int)w.x, true);
        w.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
        w.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], (int)w.y, true);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int word = (int)(j < 4 ? w.x : w.y);
            const float v = j % 4 == 0 ? __builtin_amdgcn_cvt_f32_fp8(word, 0) : j % 4 == 1 ? __builtin_amdgcn_cvt_f32_fp8(word, 1)
                          : j % 4 == 2 ? __builtin_amdgcn_cvt_f32_fp8(word, 2) : __builtin_amdgcn_cvt_f32_fp8(word, 3);
            // half a step is 2^(e - 4), e the exponent but not below -6
            const float top = fmaxf(__uint_as_float(__float_as_uint(y[j]) & 0x7f800000u), 0x1p-6f);
            near = fmaxf(near, fabsf(y[j] - v) >= top * (0.0625f * (1.f - 0x1p-11f)) ? 1.f : 0.f);
        }
    } else {
        // adding 1.5 2^23 rounds to an integer, ties to even, and leaves it in the low bits
        constexpr float kRound = 12582912.f;
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = y[j] + kRound;
            b[j] = __float_as_uint(t);
            near = fmaxf(near, fabsf(y[j] - (t - kRound)) * (2.f * (1.f + 0x1p-11f)));
        }
        if constexpr (F == SQ_CACHE_INT4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w.x |= (b[j] & 15u) << (4 * j);
        } else {
            // bytes 0 of the two sources, then the pairs
            w.x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
            w.y = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[7], b[6], 0x0c0c0400u), __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u), 0x05040100u);
        }
    }
    return w;
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
    return o > x ? o : x;
}
// The maximum over 2^log adjacent lanes; all of them get it.
__device__ __forceinline__ uint32_t group_max(uint32_t x, int log) {
    if (log > 0) x = max_dpp<0xb1>(x);                           // lane ^ 1
    if (log > 1) x = max_dpp<0x4e>(x);                           // lane ^ 2
    if (log > 2) x = max_dpp<0x141>(x);                          // 7 - lane of 8
    if (log > 3) x = max_dpp<0x140>(x);                          // 15 - lane of 16
    if (log > 4) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = r[0] > r[1] ? r[0] : r[1];
    }
    if (log > 5) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = r[0] > r[1] ? r[0] : r[1];
    }
    return x;
}

// K vectors of eight elements a thread; 2^lanes_log threads belong to a group, of which those with elements work.
template <int DT, int F, int K>
__global__ void __launch_bounds__(kThreads) k_cache_write(const CacheParams p, int lanes_log, uint32_t groups, Div by_groups) {
    const int lanes = 1 << lanes_log, lane = (int)threadIdx.x & (lanes - 1);
    const int64_t item = (int64_t)blockIdx.x * (kThreads >> lanes_log) + ((int)threadIdx.x >> lanes_log);
    const uint32_t row = by_groups((uint32_t)item), g = (uint32_t)item - row * groups;
    const bool in = item < p.n_rows * groups;
    const int64_t e0 = (int64_t)g * p.group;
    Elems<DT, 8> x[K];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int at = (k * lanes + lane) * 8;
        x[k].zero();
        if (in && at < p.group) x[k].load(p.x.p, (int64_t)row * p.x.stride + e0 + at);
    }
    // in flight beside the row, which is read whether its slot is there or not
    const int64_t slot = !in ? -1 : p.slots ? (int64_t)p.slots[row] : (int64_t)row;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(x[k].at(j)) & 0x7fffffffu;
            most = b > most ? b : most;
        }
    const bool live = slot >= 0 && slot < p.n_slots;             // the same for a group; the wave's other groups go on
    const Scale s = scale_of<F>(group_max(most, lanes_log));
    if (live && lane == 0) p.scales[slot * groups + g] = s.s;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int at = (k * lanes + lane) * 8;
        float v[8], near = s.up == 1.f ? 0.f : 1.f;              // scaled quotients go the exact way
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[k].at(j);
        uint2 w = quick8<F>(s, v, near);
        if (s.inv == 0.f) w = uint2{0, 0};                       // a group of zeros, or one with a value that is not finite
        else if (near >= 1.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = code_of<F>(s, v[j]);
            w = pack8<F>(v);
        }
        if (!live || at >= p.group) continue;
        uint8_t* to = p.codes + slot * p.row_bytes + (F == SQ_CACHE_INT4 ? (e0 + at) / 2 : e0 + at);
        if constexpr (F == SQ_CACHE_INT4) *reinterpret_cast<uint32_t*>(to) = w.x;
        else *reinterpret_cast<uint2*>(to) = w;
    }
}

// Any group and alignment: a wave a group, two elements a lane at a time.
template <int DT, int F>
__global__ void __launch_bounds__(kThreads) k_cache_write_any(const CacheParams p, uint32_t groups) {
    constexpr int kSteps = kCacheMaxGroup / 128;
    const int lane = (int)threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + ((int)threadIdx.x >> 6);
    if (item >= p.n_rows * groups) return;
    const uint32_t row = (uint32_t)item / groups, g = (uint32_t)item - row * groups;
    const int64_t slot = p.slots ? (int64_t)p.slots[row] : (int64_t)row;
    if (slot < 0 || slot >= p.n_slots) return;
    const int64_t e0 = (int64_t)g * p.group;
    Elems<DT, 1> x[kSteps][2];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = k * 128 + lane * 2 + j;
            x[k][j].zero();
            if (at < p.group) x[k][j].load(p.x.p, (int64_t)row * p.x.stride + e0 + at);
            const uint32_t b = __float_as_uint(x[k][j].at(0)) & 0x7fffffffu;
            most = b > most ? b : most;
        }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)most, m);
        most = o > most ? o : most;
    }
    const Scale s = scale_of<F>(most);
    if (lane == 0) p.scales[slot * groups + g] = s.s;
    uint8_t* to = p.codes + slot * p.row_bytes;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int at = k * 128 + lane * 2;
        if (at >= p.group) continue;
        float v[8] = {code_of<F>(s, x[k][0].at(0)), code_of<F>(s, x[k][1].at(0)), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const uint2 w = pack8<F>(v);
        if constexpr (F == SQ_CACHE_INT4) {
            to[(e0 + at) / 2] = (uint8_t)w.x;                    // groups of 4-bit codes are even
        } else {
            to[e0 + at] = (uint8_t)w.x;
            if (at + 1 < p.group) to[e0 + at + 1] = (uint8_t)(w.x >> 8);
        }
    }
}

// V elements a thread (8, or 2 for any alignment), U of them with their loads in flight together.
template <int DT, int F, int V, int U>
__global__ void __launch_bounds__(kThreads) k_cache_read(const CacheParams p, uint32_t groups, uint32_t per_row, int64_t n_items, Div by_row, Div by_group) {
    const int64_t base = (int64_t)blockIdx.x * (kThreads * U) + (int)threadIdx.x;
    uint32_t c[U][2], row[U];
    float s[U], s2[U];
    int64_t to[U], slot[U];
    int at[U];
    // all slots, then all codes and scales: two latencies for U items
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + u * kThreads;
        const uint32_t item = (uint32_t)(i < n_items ? i : n_items - 1);
        row[u] = by_row(item);
        at[u] = (int)(item - row[u] * per_row) * V;
        slot[u] = p.slots ? (int64_t)p.slots[row[u]] : (int64_t)row[u];
        to[u] = i < n_items ? (int64_t)row[u] * p.x.stride + at[u] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        c[u][0] = c[u][1] = 0;
        s[u] = s2[u] = 0.f;
        if (slot[u] < 0 || slot[u] >= p.n_slots) to[u] = -1;
        if (to[u] < 0) continue;
        const uint8_t* from = p.codes + slot[u] * p.row_bytes + (F == SQ_CACHE_INT4 ? at[u] / 2 : at[u]);
        s[u] = p.scales[slot[u] * groups + by_group((uint32_t)at[u])];
        if constexpr (V == 8) {
            if constexpr (F == SQ_CACHE_INT4) {
                c[u][0] = *reinterpret_cast<const uint32_t*>(from);
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(from);
                c[u][0] = w.x;
                c[u][1] = w.y;
            }
        } else {
            c[u][0] = from[0];
            if (at[u] + 1 < p.d) {
                if constexpr (F != SQ_CACHE_INT4) c[u][0] |= (uint32_t)from[1] << 8;
                s2[u] = p.scales[slot[u] * groups + by_group((uint32_t)(at[u] + 1))];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (to[u] < 0) continue;
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            constexpr int kBits = F == SQ_CACHE_INT4 ? 4 : 8;
            const int bit = j * kBits;
            v[j] = unpack1<F>(c[u][bit / 32] >> (bit % 32)) * (V == 8 || j == 0 ? s[u] : s2[u]);
        }
        if constexpr (V == 8) {
            Elems<DT, 8> o;
            o.set(v);
            o.store(p.x.p, to[u]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (at[u] + j < p.d) {
                    Elems<DT, 1> o;
                    o.set(v + j);
                    o.store(p.x.p, to[u] + j);
                }
        }
    }
}

// ------------------------------------------------------------------ launches

template <int DT, int F>
static hipError_t launch_write(const CacheParams& p, bool vec, hipStream_t s) {
    const uint32_t groups = (uint32_t)(p.d / p.group);
    const int64_t items = p.n_rows * groups;
    if (!vec) {
        k_cache_write_any<DT, F><<<dim3((unsigned)((items + 3) / 4)), kThreads, 0, s>>>(p, groups);
        return hipGetLastError();
    }
    int lanes_log = 0;
    while (lanes_log < 6 && (8 << lanes_log) < p.group) ++lanes_log;
    const int64_t per = kThreads >> lanes_log;
    const dim3 grid((unsigned)((items + per - 1) / per));
    if (p.group <= 512) k_cache_write<DT, F, 1><<<grid, kThreads, 0, s>>>(p, lanes_log, groups, Div(groups));
    else k_cache_write<DT, F, 2><<<grid, kThreads, 0, s>>>(p, lanes_log, groups, Div(groups));
    return hipGetLastError();
}

template <int DT, int F>
static hipError_t launch_read(const CacheParams& p, bool vec, hipStream_t s) {
    const uint32_t groups = (uint32_t)(p.d / p.group), per_row = vec ? (uint32_t)p.d / 8 : ((uint32_t)p.d + 1) / 2;
    const int64_t items = p.n_rows * per_row;
    constexpr int kU = 4;
    const dim3 grid((unsigned)((items + kThreads * kU - 1) / (kThreads * kU)));
    if (vec) k_cache_read<DT, F, 8, kU><<<grid, kThreads, 0, s>>>(p, groups, per_row, items, Div(per_row), Div((uint32_t)p.group));
    else k_cache_read<DT, F, 2, kU><<<grid, kThreads, 0, s>>>(p, groups, per_row, items, Div(per_row), Div((uint32_t)p.group));
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_dt(const CacheParams& p, bool vec, bool write, hipStream_t s) {
    if (p.format == SQ_CACHE_INT8) return write ? launch_write<DT, SQ_CACHE_INT8>(p, vec, s) : launch_read<DT, SQ_CACHE_INT8>(p, vec, s);
    if (p.format == SQ_CACHE_INT4) return write ? launch_write<DT, SQ_CACHE_INT4>(p, vec, s) : launch_read<DT, SQ_CACHE_INT4>(p, vec, s);
    return write ? launch_write<DT, SQ_CACHE_E4M3>(p, vec, s) : launch_read<DT, SQ_CACHE_E4M3>(p, vec, s);
}
static hipError_t launch_any(const CacheParams& p, bool vec, bool write, hipStream_t s) {
    if (p.dtype == SQ_DTYPE_BF16) return launch_dt<SQ_DTYPE_BF16>(p, vec, write, s);
    if (p.dtype == SQ_DTYPE_F16) return launch_dt<SQ_DTYPE_F16>(p, vec, write, s);
    return launch_dt<SQ_DTYPE_F32>(p, vec, write, s);
}

hipError_t launch_cache_write(const CacheParams& p, bool vec, hipStream_t s) { return launch_any(p, vec, true, s); }
hipError_t launch_cache_read(const CacheParams& p, bool vec, hipStream_t s) { return launch_any(p, vec, false, s); }

}  // namespace sq
