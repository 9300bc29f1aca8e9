// Short causal convolution over packed sequences, one filter a channel, with its activation (gfx950).
//
//   p_t = bias + sum_j w_j x_{t - W + 1 + j},   y_t = p_t or p_t sigmoid(p_t)        (x before a sequence: s0, or zero)
//
// Memory bounds the forward pass: x is read once and y written once.  A thread owns V adjacent channels and walks a run of tokens
// with the last W - 1 inputs in registers; the only inputs read twice are the W - 1 before each run.  Runs start at a sequence's
// start, so no run holds two sequences, and the run that reads s0 is also the one that writes s1 (each thread its own channels,
// after its reads), so that both may be the same array.  12301 tokens of 8192 channels in bfloat16, four taps, new inputs every pass:
// 82 us, 4.9 TB/s (a copy: 6.0).  Four channels a thread (8-byte accesses) leave 62 registers, so that 8 waves a SIMD hide the
// latency: eight channels took 97 us on one set of inputs, four 85.  Runs of 16 tokens with 8 loads in flight: 82 us, of 32: 86, of 8: 92.
// Single elements, where strides or channels do not allow 8 bytes: 61 us where four take 48 (8190 tokens of 8192 channels, one set of inputs).
#include <hip/hip_runtime.h>

#include "conv_dev.h"

namespace sq {

// The last W - 1 inputs of a sequence: rows of x, or of s0 where the sequence is shorter.  All reads come before the writes.
template <int DT, int W, int V>
__device__ __forceinline__ void last_inputs(const ConvParams& p, const RunAt& r, uint32_t c) {
    Elems<DT, V> e[W - 1];
    const int64_t s = (int64_t)r.seq * (W - 1);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t at = r.len - (W - 1) + j;
        if (at >= 0) e[j].load(p.x.p, (r.start + at) * p.x.stride, c);
        else if (p.s0) e[j].load(p.s0, (s + at + W - 1) * p.channels, c);
        else e[j].zero();
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) e[j].store(p.s1, (s + j) * p.channels, c);
}

template <int DT, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads) k_conv(const ConvParams p, int n_blocks) {
    const uint32_t c = (((int)blockIdx.x % n_blocks) * kThreads + (int)threadIdx.x) * V;
    Filter<DT, W, V> f;
    if (c < (uint32_t)p.channels) f.load(p, c);
    const RunAt r = run_of_slot(p.runs, (int64_t)((int)blockIdx.x / n_blocks));
    if (c >= (uint32_t)p.channels) return;
    Elems<DT, V> before[W - 1];
    float x[W - 1 + kU][V];
    if (r.n > 0) {
        inputs_before<DT, W, V>(p, r, c, before);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) x[j][v] = before[j].at(v);
    }
    if (r.first && p.s1) last_inputs<DT, W, V>(p, r, c);
    if (r.n == 0) return;
    Elems<DT, V> in[kU], next[kU];
    auto fetch = [&](int t, Elems<DT, V>(&e)[kU]) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (t + u < r.n) e[u].load(p.x.p, (r.tok0 + t + u) * p.x.stride, c);
    };
    fetch(0, next);
    for (int t = 0; t < r.n; t += kU) {
#pragma unroll
        for (int u = 0; u < kU; ++u) in[u] = next[u];
        fetch(t + kU, next);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (t + u >= r.n) break;
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[W - 1 + u][v] = in[u].at(v);
                float s = f.b[v];
#pragma unroll
                for (int j = 0; j < W; ++j) s = fmaf(f.w[v][j], x[u + j][v], s);
                y[v] = SILU ? s * sigmoid(s) : s;
            }
            Elems<DT, V> o;
            o.set(y);
            if (p.once) o.store_once(p.y.p, (r.tok0 + t + u) * p.y.stride, c);
            else o.store(p.y.p, (r.tok0 + t + u) * p.y.stride, c);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) x[j][v] = x[j + kU][v];
    }
}

// One token of each request, its last W - 1 inputs in a slot of the pool: window and x in, y and the window moved by one out.
template <int DT, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads) k_conv_step(const ConvParams p, int n_blocks) {
    const uint32_t c = (((int)blockIdx.x % n_blocks) * kThreads + (int)threadIdx.x) * V;
    const int64_t b = (int)blockIdx.x / n_blocks;
    const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
    if (c >= (uint32_t)p.channels || slot < 0 || slot >= p.n_slots) return;
    const int64_t base = slot * (W - 1) * p.channels + c;
    Elems<DT, V> e[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) e[j].load(p.window, base + (int64_t)j * p.channels);
    e[W - 1].load(p.x.p, b * p.x.stride, c);
    Filter<DT, W, V> f;
    f.load(p, c);
    float y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = f.b[v];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(f.w[v][j], e[j].at(v), s);
        y[v] = SILU ? s * sigmoid(s) : s;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) e[j + 1].store(p.window, base + (int64_t)j * p.channels);
    Elems<DT, V> o;
    o.set(y);
    o.store(p.y.p, b * p.y.stride, c);
}

// ------------------------------------------------------------------ launches

template <int DT, int W, int V>
static hipError_t fwd_n(const ConvParams& p, hipStream_t s) {
    const int n_blocks = (p.channels + kThreads * V - 1) / (kThreads * V);
    const dim3 grid((unsigned)(run_slots(p.runs.n_tokens, p.runs.n_seq, p.runs.log) * n_blocks));
    if (p.act == SQ_ACT_SILU) k_conv<DT, W, V, true><<<grid, kThreads, 0, s>>>(p, n_blocks);
    else k_conv<DT, W, V, false><<<grid, kThreads, 0, s>>>(p, n_blocks);
    return hipGetLastError();
}
template <int DT, int W, int V>
static hipError_t step_n(const ConvParams& p, hipStream_t s) {
    const int n_blocks = (p.channels + kThreads * V - 1) / (kThreads * V);
    const dim3 grid((unsigned)(p.batch * n_blocks));
    if (p.act == SQ_ACT_SILU) k_conv_step<DT, W, V, true><<<grid, kThreads, 0, s>>>(p, n_blocks);
    else k_conv_step<DT, W, V, false><<<grid, kThreads, 0, s>>>(p, n_blocks);
    return hipGetLastError();
}

hipError_t launch_conv(const ConvParams& p, bool vec, hipStream_t s) { SQ_CONV_DISPATCH(fwd_n, kConvBytes, p, s); }
hipError_t launch_conv_step(const ConvParams& p, bool vec, hipStream_t s) { SQ_CONV_DISPATCH(step_n, kConvStepBytes, p, s); }

}  // namespace sq
