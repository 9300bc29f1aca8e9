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
constexpr int kConvLog = 4;                          // of a run of the forward pass
// Bytes that a thread accesses at a time, forward, backward and for one token: adjacent channels of a row.  Forward and backward as many as
// registers allow (at the kernels).  One token is a chain of loads of a slot, its window and the filters, which many threads of few
// channels hide best: 64 requests of 8192 channels in bfloat16 with 4 taps take 3.7 us with 4 bytes, 4.2 with 8 and 5.8 with 16, 256 of
// them 7.6, 10.0 and 15.7, one of 512 2.1, 2.1 and 2.4; float32 4.5, 4.9 and 5.1, 14.3, 14.5 and 16.9, 2.2, 2.1 and 2.2.
constexpr int kConvBytes = 8, kConvBwdBytes = 4, kConvStepBytes = 4;
// `vec`: every array and the channels allow these accesses; otherwise they are of one element.
hipError_t launch_conv(const ConvParams& p, bool vec, hipStream_t s);
hipError_t launch_conv_bwd(const ConvParams& p, bool vec, hipStream_t s);
hipError_t launch_conv_step(const ConvParams& p, bool vec, hipStream_t s);

}  // namespace sq
