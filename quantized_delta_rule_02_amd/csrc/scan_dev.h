// Device helpers of the gated delta scan: float32 products on the bfloat16 matrix units.
//
// A float32 value is exactly the sum of three bfloat16 values (8 significand bits each, by truncation), so a
// product of two float32 matrices is six bfloat16 products (the three smallest of the nine, below 2^-21 of the
// largest, are left out): about float32 accuracy at 2500 / 6 TFLOP/s, where the float32 matrix instructions
// reach 157.  An operand that is a bfloat16 input already is one plane and needs three products.
//
// MFMA 16x16x32: A lane (i = l & 15, g = l >> 4) holds 8 elements of row i, B lane (n, g) the same 8 positions of
// column n, D lane (n, g) rows 4g + r, r < 4.  Which k a position (g, e) stands for is free as long as A and B agree.
// Here position (g, 4t + r) of a block of 32 is k = 16 t + 4 g + r: then two D tiles of a lane are, as they stand,
// a B operand of the next product, and states and updates never leave their registers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "scan.h"
#include "vec.h"

namespace sq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

template <int N>
struct Frag {
    u32x4v p[N];
};

__device__ __forceinline__ uint32_t hi16_pair(float a, float b) {   // the upper halves of a (low) and b (high)
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float trunc_bf16(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

template <int N>
__device__ __forceinline__ Frag<N> split8(const float* x) {
    Frag<N> f;
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = x[j];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f.p[n][j] = hi16_pair(m[2 * j], m[2 * j + 1]);
        if (n + 1 < N) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] -= trunc_bf16(m[j]);
        }
    }
    return f;
}

// Four elements: the dwords of plane n.
template <int N>
__device__ __forceinline__ void split4(const float* x, u32x2* out) {
    float m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = x[j];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        out[n][0] = hi16_pair(m[0], m[1]);
        out[n][1] = hi16_pair(m[2], m[3]);
        if (n + 1 < N) {
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] -= trunc_bf16(m[j]);
        }
    }
}

template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = 2; s >= 0; --s) {       // smallest terms first
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.p[i]),
                                                              __builtin_bit_cast(bf16x8, b.p[j]), acc, 0, 0, 0);
        }
    }
}

// Position of column c of a matrix row inside the row's storage: blocks of 32 in the order described above.
__device__ __forceinline__ constexpr int kpos(int c) {
    return (c & ~31) | ((c & 12) << 1) | ((c & 16) >> 2) | (c & 3);
}

struct Seq {
    int64_t start;
    int64_t len;
};
// Sequence b, with offsets outside the packed arrays pulled inside (nothing beyond them is read or written).
__device__ __forceinline__ Seq sequence(const ScanParams& p, int b) {
    if (!p.seq_start) return Seq{0, p.n_tokens};
    int64_t s = p.seq_start[b], e = p.seq_start[b + 1];
    s = s < 0 ? 0 : s > p.n_tokens ? p.n_tokens : s;
    e = e < s ? s : e > p.n_tokens ? p.n_tokens : e;
    return Seq{s, e - s};
}
__device__ __forceinline__ int64_t first_slot(const Seq& q, int b) { return (q.start >> 5) + b; }

// Where the backward pass divides by a gate it counts gates below this as it: terms scaled by 1e-30 are lost in float32
// either way, and the quotient stays one of normal numbers, also for a gate of zero.  The states take the gates as they are.
constexpr float kGateMin = 1e-30f;

// gate per key row: float32 operands whatever the inputs' type (three planes); one gate per head: the inputs' own planes
#define SQ_SCAN_DISPATCH(fn, ...)                                                            \
    do {                                                                                     \
        const int np = p.dtype == SQ_DTYPE_BF16 ? 1 : p.dtype == SQ_DTYPE_F16 ? 2 : 3;       \
        if (p.form == SQ_FORM_KDA) {                                                         \
            if (p.dk == 16) return fn<16, 3, true>(__VA_ARGS__);                             \
            if (p.dk == 64) return fn<64, 3, true>(__VA_ARGS__);                             \
            if (p.dk == 128) return fn<128, 3, true>(__VA_ARGS__);                           \
        } else {                                                                             \
            if (p.dk == 16) return np == 1 ? fn<16, 1, false>(__VA_ARGS__) : np == 2 ? fn<16, 2, false>(__VA_ARGS__) : fn<16, 3, false>(__VA_ARGS__);       \
            if (p.dk == 64) return np == 1 ? fn<64, 1, false>(__VA_ARGS__) : np == 2 ? fn<64, 2, false>(__VA_ARGS__) : fn<64, 3, false>(__VA_ARGS__);       \
            if (p.dk == 128) return np == 1 ? fn<128, 1, false>(__VA_ARGS__) : np == 2 ? fn<128, 2, false>(__VA_ARGS__) : fn<128, 3, false>(__VA_ARGS__);   \
        }                                                                                    \
        return hipErrorInvalidValue;                                                         \
    } while (0)

}  // namespace sq
