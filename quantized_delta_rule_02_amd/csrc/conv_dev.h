// What the convolution's kernels share: filters and the inputs before a run.
#pragma once
#include <hip/hip_runtime.h>

#include "conv.h"
#include "elems.h"

namespace sq {

constexpr int kThreads = 256, kU = 8, kUb = 4;         // threads of a workgroup; tokens whose loads are in flight together (gradients)

template <int DT, int W, int V>
struct Filter {
    float w[V][W], b[V];
    __device__ __forceinline__ void load(const ConvParams& p, uint32_t c) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[v][j] = p.weight[(int64_t)(c + v) * W + j];
            b[v] = p.bias ? p.bias[c + v] : 0.f;
        }
    }
};

// Inputs W - 1 .. 1 places before the run's first token.
template <int DT, int W, int V>
__device__ __forceinline__ void inputs_before(const ConvParams& p, const RunAt& r, uint32_t c, Elems<DT, V> (&e)[W - 1]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (!r.first) e[j].load(p.x.p, (r.tok0 - (W - 1) + j) * p.x.stride, c);     // a run has at least W - 1 tokens before the next
        else if (p.s0) e[j].load(p.s0, ((int64_t)r.seq * (W - 1) + j) * p.channels, c);
        else e[j].zero();
    }
}

// `fn` for the call's taps, type and alignment: BYTES a thread, or one element where the arrays do not allow it.
#define SQ_CONV_WIDTH(fn, DT, V, ...)                                \
    switch (p.width) {                                               \
        case 2: return fn<DT, 2, V>(__VA_ARGS__);                    \
        case 3: return fn<DT, 3, V>(__VA_ARGS__);                    \
        case 4: return fn<DT, 4, V>(__VA_ARGS__);                    \
        case 5: return fn<DT, 5, V>(__VA_ARGS__);                    \
        case 6: return fn<DT, 6, V>(__VA_ARGS__);                    \
        case 7: return fn<DT, 7, V>(__VA_ARGS__);                    \
        case 8: return fn<DT, 8, V>(__VA_ARGS__);                    \
        default: return hipErrorInvalidValue;                        \
    }
#define SQ_CONV_DISPATCH(fn, BYTES, ...)                                                 \
    do {                                                                                 \
        if (p.dtype == SQ_DTYPE_BF16 && vec) SQ_CONV_WIDTH(fn, SQ_DTYPE_BF16, (BYTES) / 2, __VA_ARGS__) \
        if (p.dtype == SQ_DTYPE_BF16) SQ_CONV_WIDTH(fn, SQ_DTYPE_BF16, 1, __VA_ARGS__)    \
        if (p.dtype == SQ_DTYPE_F16 && vec) SQ_CONV_WIDTH(fn, SQ_DTYPE_F16, (BYTES) / 2, __VA_ARGS__) \
        if (p.dtype == SQ_DTYPE_F16) SQ_CONV_WIDTH(fn, SQ_DTYPE_F16, 1, __VA_ARGS__)      \
        if (vec) SQ_CONV_WIDTH(fn, SQ_DTYPE_F32, (BYTES) / 4, __VA_ARGS__)                \
        SQ_CONV_WIDTH(fn, SQ_DTYPE_F32, 1, __VA_ARGS__)                                   \
    } while (0)

}  // namespace sq
