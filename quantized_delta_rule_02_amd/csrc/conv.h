// Launchers of the causal convolution (conv.hip), called by the C ABI (mix_api.cpp).
#pragma once
#include "runs.h"

namespace sq {

constexpr int kConvMaxWidth = 8;

struct ConvParams {
    Runs runs;
    int32_t channels, dtype, act, width;
    int32_t once;                    // forward: y is written past the caches' usual order
    Rows x, y, dy, dx;
    const float* weight;             // [channels][width]
    const float* bias;               // [channels] or NULL
    const void* s0;                  // [n_seq][width - 1][channels], oldest input first, or NULL
    void* s1;
    const void* ds1;
    void* ds0;
    float* part;                     // backward: [slot][width + 1][channels] sums of dweight and dbias over a run
    float* dweight;
    float* dbias;
    // one token of each request
    const int32_t* slots;            // or NULL: request b has slot b
    int64_t n_slots, batch;
    void* window;                    // [n_slots][width - 1][channels]
};

constexpr int kConvBwdLog = 6, kConvBwdRuns = 8;     // log2 of the tokens of a wave and of a workgroup of the backward pass
int conv_run_log(int64_t n_tokens, int64_t n_seq, int32_t channels);    // of the forward pass
// `vec`: every array allows the accesses of `vec` elements at a time (conv_vec) that the kernels make.
int conv_vec(int32_t dtype);
hipError_t launch_conv(const ConvParams& p, bool vec, hipStream_t s);
hipError_t launch_conv_bwd(const ConvParams& p, bool vec, hipStream_t s);
hipError_t launch_conv_step(const ConvParams& p, bool vec, hipStream_t s);

}  // namespace sq
