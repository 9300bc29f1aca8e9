// Device helpers of the gated delta scan: float32 products on the bfloat16 matrix units.
//
// A float32 value is the sum of three bfloat16 values (rounded to nearest, then what is left, twice), so a product of
// two float32 matrices is six bfloat16 products (the three smallest of the nine, up to 2^-24 of the largest, are left
// out): about float32 accuracy at 2500 / 6 TFLOP/s, where the float32 matrix instructions reach 157.  An operand that is
// a bfloat16 input already is one plane and needs three products.
//
// MFMA 16x16x32: A lane (i = l & 15, g = l >> 4) holds 8 elements of row i, B lane (n, g) the same 8 positions of
// column n, D lane (n, g) rows 4g + r, r < 4.  Which k a position (g, e) stands for is free as long as A and B agree.
// Here position (g, 4t + r) of a block of 32 is k = 16 t + 4 g + r: then two D tiles of a lane are, as they stand,
// an operand of the next product, and states and updates never leave their registers.
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

// Two float32 rounded to bfloat16 (a low), and what rounding left of each: x - bf16(x) is exact in float32, and one
// instruction as the two-element dot product with (-1, 0) or (0, -1), half of what masking and subtracting takes.  The
// constants come from registers: as an inline constant 0xbf800000 stands for another pair.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t round_pair(float a, float b) {
    bf16x2 r;
    r[0] = (__bf16)a;
    r[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ void rest_pair(uint32_t pair, float& a, float& b) {
    uint32_t lo = 0x0000bf80u, hi = 0xbf800000u;
    __asm__("" : "+s"(lo));
    __asm__("" : "+s"(hi));
    const bf16x2 p = __builtin_bit_cast(bf16x2, pair);
    a = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2, lo), a, false);
    b = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2, hi), b, false);
}

template <int N>
__device__ __forceinline__ Frag<N> split8(const float* x) {
    Frag<N> f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            f.p[n][j] = round_pair(a, b);
            if (n + 1 < N) rest_pair(f.p[n][j], a, b);
        }
    }
    return f;
}

// A choice between two values (a ?: of two array elements is a choice of their addresses, which takes an array out of the
// registers).
__device__ __forceinline__ float pick(bool c, float a, float b) { return c ? a : b; }

// The value, of which the compiler knows nothing: addresses formed from it are formed where they are used and not kept in
// registers over a loop.
__device__ __forceinline__ int opaque(int x) {
    __asm__ volatile("" : "+v"(x));
    return x;
}

// Four elements: the dwords of plane n.
template <int N>
__device__ __forceinline__ void split4(const float* x, u32x2* out) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            out[n][j] = round_pair(a, b);
            if (n + 1 < N) rest_pair(out[n][j], a, b);
        }
    }
}

// acc += a b, the terms of planes i and j with i + j <= ORD, the smallest first.
template <int ORD, int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = ORD; s >= 0; --s) {
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.p[i]),
                                                              __builtin_bit_cast(bf16x8, b.p[j]), acc, 0, 0, 0);
        }
    }
}

// Position of column c of a matrix row inside the row's storage, in the order described above.
__device__ __forceinline__ constexpr int kpos32(int c) {
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

// The i-th sequence longer than short_len, or -1.  A whole wave looks at 64 sequences at a time.
__device__ __forceinline__ int long_sequence(const ScanParams& p, int i) {
    for (int b0 = 0; b0 < p.n_seq; b0 += 64) {
        const int b = b0 + ((int)threadIdx.x & 63);
        uint64_t m = __ballot(b < p.n_seq && sequence(p, b < p.n_seq ? b : 0).len > p.short_len);
        const int c = __popcll(m);
        if (i < c) {
            while (i-- > 0) m &= m - 1;
            return b0 + __builtin_ctzll(m);
        }
        i -= c;
    }
    return -1;
}

// The chunk of a slot: its first token and how many it has (0: no chunk uses the slot, or not the chunked scan's).  Of the
// sequences whose first slot is not above the slot it is the last one's: a search by 64 lanes at a time (one round for 64
// sequences, two for 4096), since a round is a load's latency.
struct ChunkAt {
    int64_t tok0;
    int rem;
};
__device__ __forceinline__ ChunkAt chunk_of_slot(const ScanParams& p, int64_t slot) {
    int lo = 0, n = p.n_seq;                         // it is one of the n from lo
    while (n > 1) {
        const int step = (n + 63) / 64, at = ((int)threadIdx.x & 63) * step;
        const bool below = at < n && first_slot(sequence(p, lo + at), lo + at) <= slot;
        const int last = 63 - __builtin_clzll(__ballot(below) | 1);
        lo += last * step;
        n = n - last * step < step ? n - last * step : step;
    }
    const Seq q = sequence(p, lo);
    const int64_t c0 = (slot - first_slot(q, lo)) * kChunk;
    const int start = __builtin_amdgcn_readfirstlane((int)(q.start + c0));
    int64_t rem = c0 < 0 || q.len <= p.short_len ? 0 : q.len - c0;
    rem = rem < 0 ? 0 : rem > kChunk ? kChunk : rem;
    return ChunkAt{start, __builtin_amdgcn_readfirstlane((int)rem)};
}

// Products of one token's gates within its block of 2^lev tokens: up to it, after it, and of the whole block.
template <typename T>
struct GateLevels {
    T pre, suf, full;
    GateLevels() = default;
    __device__ __forceinline__ explicit GateLevels(T a) : pre(a), suf(1), full(a) {}
    // joins the sibling block, whose gates multiply to `other`; odd: this token lies in the second of the two
    __device__ __forceinline__ void grow(bool odd, T other) {
        pre = odd ? pre * other : pre;
        suf = odd ? suf : suf * other;
        full *= other;
    }
};

// Orders a wave's own LDS accesses.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int NP>
__device__ __forceinline__ Frag<NP> lds_frag(const uint16_t* base, int plane_stride, int off) {
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = *reinterpret_cast<const u32x4v*>(base + i * plane_stride + off);
    return f;
}

// A barrier for LDS contents only: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A window of memory whose loads give 0 and whose stores do nothing beyond `bytes`: the rows behind a sequence's end need
// no branch.  The base is the same for the whole wave; offsets are 32 bits (the stride limit keeps a chunk below 4 GiB).
struct Window {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ Window(const void* base, uint32_t bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000)) {}
};
template <int DT>
__device__ __forceinline__ uint32_t win_load1(const Window& w, uint32_t off) {
    if constexpr (DT == SQ_DTYPE_F32) return __builtin_amdgcn_raw_buffer_load_b32(w.r, off, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b16(w.r, off, 0, 0);
}
template <int DT>
__device__ __forceinline__ float val1(uint32_t x) {
    return DT == SQ_DTYPE_F32 ? __uint_as_float(x) : DT == SQ_DTYPE_BF16 ? bf16_lo(x) : f16_val(x);
}
template <int DT>
__device__ __forceinline__ void win_store1(const Window& w, uint32_t off, float x) {
    if constexpr (DT == SQ_DTYPE_F32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), w.r, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(DT == SQ_DTYPE_BF16 ? bf16_bits(x) : f16_bits(x)), w.r, off, 0, 0);
}

// N adjacent elements as loaded, and their values.
template <int DT, int N>
struct Raw {
    static constexpr int W = N * (DT == SQ_DTYPE_F32 ? 4 : 2) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const Window& b, uint32_t off) {
        if constexpr (W == 1) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(b.r, off, 0, 0);
        } else if constexpr (W == 2) {
            const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(b.r, off, 0, 0);
            w[0] = x[0];
            w[1] = x[1];
        } else {
            static_assert(W == 4);
            const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(b.r, off, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = x[i];
        }
    }
    __device__ __forceinline__ float at(int j) const {
        if constexpr (DT == SQ_DTYPE_F32) return __uint_as_float(w[j]);
        else return val1<DT>((j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
    }
};

constexpr int planes_of(int dt) { return dt == SQ_DTYPE_BF16 ? 1 : dt == SQ_DTYPE_F16 ? 2 : 3; }   // that hold it exactly

#define SQ_SCAN_DISPATCH_DT(fn, DK, KDA, ...)                                                    \
    do {                                                                                         \
        if (p.dtype == SQ_DTYPE_BF16) return fn<DK, SQ_DTYPE_BF16, KDA>(__VA_ARGS__);             \
        if (p.dtype == SQ_DTYPE_F16) return fn<DK, SQ_DTYPE_F16, KDA>(__VA_ARGS__);               \
        return fn<DK, SQ_DTYPE_F32, KDA>(__VA_ARGS__);                                           \
    } while (0)
#define SQ_SCAN_DISPATCH(fn, ...)                                                                \
    do {                                                                                         \
        const bool kda = p.form == SQ_FORM_KDA;                                                  \
        if (p.dk == 16 && kda) SQ_SCAN_DISPATCH_DT(fn, 16, true, __VA_ARGS__);                    \
        if (p.dk == 16) SQ_SCAN_DISPATCH_DT(fn, 16, false, __VA_ARGS__);                          \
        if (p.dk == 64 && kda) SQ_SCAN_DISPATCH_DT(fn, 64, true, __VA_ARGS__);                    \
        if (p.dk == 64) SQ_SCAN_DISPATCH_DT(fn, 64, false, __VA_ARGS__);                          \
        if (p.dk == 128 && kda) SQ_SCAN_DISPATCH_DT(fn, 128, true, __VA_ARGS__);                  \
        if (p.dk == 128) SQ_SCAN_DISPATCH_DT(fn, 128, false, __VA_ARGS__);                        \
        return hipErrorInvalidValue;                                                             \
    } while (0)

}  // namespace sq
