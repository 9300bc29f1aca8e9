// Gradients of the short causal convolution (gfx950).
//
//   p_t = bias + sum_j w_j x_{t - W + 1 + j},   y_t = act(p_t)
//   dp = dy act'(p),  dx_t = sum_j w_j dp_{t + W - 1 - j} (+ ds1),  dw_j = sum_t dp_t x_{t - W + 1 + j},  dbias = sum_t dp_t
//
// They are bound by the vector unit, 39 instructions an element (p again, its derivative, W products each for dx and
// dweight) with 73 % of its time used, beside memory: 8190 tokens of 8192 channels 95 us, floor by memory 67.  Measured at 37 instructions
// (gates of fewer digits): two channels a thread (82 registers) 89 us, four 97; runs of 64 tokens a wave 87 us, of 32: 89, of 16: 97
// (W - 1 more steps each).  Single elements: 126 us where two take 95.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "conv_dev.h"

namespace sq {

// A workgroup has kThreads / 64 runs of 2^kConvBwdLog tokens one after the other, a wave each, over 64 V channels: their sums
// meet in LDS and go out as one row of `part`.  A wave's walk goes W - 1 tokens past its run's end (their dp belongs to the run's
// last dx), and dx follows W - 1 tokens behind.  What reaches inputs before the sequence is ds0's.
template <int DT, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(const ConvParams p, int n_blocks) {
    constexpr int kWaves = kThreads / 64;
    __shared__ float s_sum[kWaves][(W + 1) * V][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const uint32_t c = (((int)blockIdx.x % n_blocks) * 64 + lane) * V;
    const int64_t slot = (int)blockIdx.x / n_blocks;
    RunAt r = run_of_slot(p.runs, slot);
    {                                                          // the wave's part of it
        const int at = __builtin_amdgcn_readfirstlane(wave << kConvBwdLog), most = 1 << kConvBwdLog, n = r.n - at;
        r.n = n < 0 ? 0 : n < most ? n : most;
        r.tok0 += at;
        r.first = r.first && at == 0;
    }
    float dw[V][W], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[v][j] = 0.f;
    }
    if (c < (uint32_t)p.channels && (r.n > 0 || r.first)) {
        Filter<DT, W, V> f;
        f.load(p, c);
        float x[W - 1 + kUb][V], dp[W - 1 + kUb][V];           // W - 1 inputs and gradients before a step's kUb tokens, and these
        {
            Elems<DT, V> before[W - 1];
            inputs_before<DT, W, V>(p, r, c, before);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[j][v] = before[j].at(v);
                    dp[j][v] = 0.f;
                }
        }
        const int64_t off = r.tok0 - r.start, s = (int64_t)r.seq * (W - 1);
        const int left = (int)(r.len - off), end = r.n + W - 1;        // tokens to the sequence's end; dx of token t - (W - 1) at step t
        Elems<DT, V> ex[kUb], ey[kUb];
        auto fetch = [&](int t) {
#pragma unroll
            for (int u = 0; u < kUb; ++u) {
                ex[u].zero();
                ey[u].zero();
                if (t + u < left && t + u < end) {
                    ex[u].load(p.x.p, (r.tok0 + t + u) * p.x.stride, c);
                    ey[u].load(p.dy.p, (r.tok0 + t + u) * p.dy.stride, c);
                }
            }
        };
        // kUb steps; INNER: all of them the run's own tokens, their dx rows the run's too and none of them among the last inputs
        auto steps = [&](auto inner, int t) {
            constexpr bool INNER = decltype(inner)::value;
#pragma unroll
            for (int u = 0; u < kUb; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[W - 1 + u][v] = ex[u].at(v);
                    dp[W - 1 + u][v] = ey[u].at(v);
                }
            fetch(t + kUb);
#pragma unroll
            for (int u = 0; u < kUb; ++u) {
                if (!INNER && t + u >= end) break;
                if (INNER || t + u < left) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float g = dp[W - 1 + u][v];
                        if constexpr (SILU) {
                            float a = f.b[v];
#pragma unroll
                            for (int j = 0; j < W; ++j) a = fmaf(f.w[v][j], x[u + j][v], a);
                            const float sg = sigmoid(a);
                            g *= sg * fmaf(a, 1.f - sg, 1.f);
                            dp[W - 1 + u][v] = g;
                        }
                        if (INNER || t + u < r.n) {
                            db[v] += g;
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[v][j] = fmaf(g, x[u + j][v], dw[v][j]);
                        }
                    }
                }
                // dx's token in its sequence; below 0: a row of s0.  A later run's first steps see inputs of the run before it: theirs.
                const int64_t at = off + t + u - (W - 1);
                if (!INNER && (at >= 0 ? t + u < W - 1 : !r.first || !p.ds0)) continue;
                float d[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) d[v] = fmaf(f.w[v][W - 1 - j], dp[u + j][v], d[v]);
                }
                const int64_t kept = at - (r.len - (W - 1));           // its row of s1, where it is one of the last inputs
                if (!INNER && p.ds1 && kept >= 0) {
                    Elems<DT, V> e;
                    e.load(p.ds1, (s + kept) * p.channels, c);
#pragma unroll
                    for (int v = 0; v < V; ++v) d[v] += e.at(v);
                }
                Elems<DT, V> o;
                o.set(d);
                if (INNER || at >= 0) o.store(p.dx.p, (r.start + at) * p.dx.stride, c);
                else o.store(p.ds0, (s + at + W - 1) * p.channels, c);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[j][v] = x[j + kUb][v];
                    dp[j][v] = dp[j + kUb][v];
                }
        };
        fetch(0);
        for (int t = 0; t < end; t += kUb) {
            if (t >= W - 1 && t + kUb <= r.n && off + t + kUb <= r.len) steps(std::true_type{}, t);
            else steps(std::false_type{}, t);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j <= W; ++j) s_sum[wave][j * V + v][lane] = j < W ? dw[v][j < W ? j : 0] : db[v];
    __syncthreads();
    float* part = p.part + slot * (W + 1) * p.channels;
    const int c0 = ((int)blockIdx.x % n_blocks) * 64 * V;
    for (int i = (int)threadIdx.x; i < (W + 1) * V * 64; i += kThreads) {          // in the order of the row's columns
        const int j = i / (V * 64), at = i % (V * 64);
        if (c0 + at >= p.channels) continue;
        float s = s_sum[0][j * V + at % V][at / V];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += s_sum[w][j * V + at % V][at / V];
        part[(int64_t)j * p.channels + c0 + at] = s;
    }
}

// dweight and dbias: the rows of `part` added in a fixed order, 64 columns a workgroup, the rows in 16 interleaved parts.
__global__ void __launch_bounds__(1024) k_conv_sum(const ConvParams p, int64_t n_rows) {
    __shared__ float s_part[16][64];
    const int lane = (int)threadIdx.x & 63, sub = (int)threadIdx.x >> 6;
    const int64_t n_cols = (int64_t)(p.width + 1) * p.channels, col = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (col < n_cols)
        for (int64_t i = sub; i < n_rows; i += 16) s += p.part[i * n_cols + col];
    s_part[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || col >= n_cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += s_part[k][lane];
    const int64_t j = col / p.channels, c = col % p.channels;
    if (j < p.width) { if (p.dweight) p.dweight[c * p.width + j] = s; }
    else if (p.dbias) p.dbias[c] = s;
}

// ------------------------------------------------------------------ launches

template <int DT, int W, int V>
static hipError_t bwd_n(const ConvParams& p, int64_t slots, hipStream_t s) {
    const int n_blocks = (p.channels + 64 * V - 1) / (64 * V);
    const dim3 grid((unsigned)(slots * n_blocks));
    if (p.act == SQ_ACT_SILU) k_conv_bwd<DT, W, V, true><<<grid, kThreads, 0, s>>>(p, n_blocks);
    else k_conv_bwd<DT, W, V, false><<<grid, kThreads, 0, s>>>(p, n_blocks);
    return hipGetLastError();
}
static hipError_t launch_runs(const ConvParams& p, bool vec, int64_t slots, hipStream_t s) { SQ_CONV_DISPATCH(bwd_n, kConvBwdBytes, p, slots, s); }

hipError_t launch_conv_bwd(const ConvParams& p, bool vec, hipStream_t s) {
    const int64_t slots = p.runs.n_seq > 0 ? run_slots(p.runs.n_tokens, p.runs.n_seq, p.runs.log) : 0;
    if (slots > 0) {
        const hipError_t e = launch_runs(p, vec, slots, s);
        if (e != hipSuccess) return e;
    }
    if (!p.dweight && !p.dbias) return hipSuccess;
    const int64_t cols = (int64_t)(p.width + 1) * p.channels;
    k_conv_sum<<<dim3((unsigned)((cols + 63) / 64)), 1024, 0, s>>>(p, slots);
    return hipGetLastError();
}

}  // namespace sq
