// Short causal convolution over packed sequences, one filter a channel, with its activation and gradients (gfx950).
//
//   p_t = bias + sum_j w_j x_{t - W + 1 + j},   y_t = p_t or p_t sigmoid(p_t)        (x before a sequence: s0, or zero)
//   dp = dy act'(p),  dx_t = sum_j w_j dp_{t + W - 1 - j} (+ ds1),  dw_j = sum_t dp_t x_{t - W + 1 + j},  dbias = sum_t dp_t
//
// Memory bounds the forward pass: x is read once and y written once.  A thread owns V adjacent channels and walks a run of tokens
// with the last W - 1 inputs in registers; the only inputs read twice are the W - 1 before each run.  Runs start at a sequence's
// start, so no run holds two sequences, and the run that reads s0 is also the one that writes s1 (each thread its own channels,
// after its reads), so that both may be the same array.  12301 tokens of 8192 channels in bfloat16, four taps, new inputs every pass:
// 84 us, 4.8 TB/s (a copy: 6.0).  Four channels a thread (8-byte accesses) leave 62 registers, so that 8 waves a SIMD hide the
// latency: eight channels took 97 us on one set of inputs, four 85.  Runs of 16 tokens with 8 loads in flight: 82 us, of 32: 86, of 8: 92.
// The gradients are bound by the vector unit, 37 instructions an element (p again, its derivative, W products each for dx and
// dweight) with 69 to 80 % of its time used: 8190 tokens of 8192 channels 96 us, floor by memory 67.  Two channels a thread (82
// registers) 89 us, four 97; runs of 64 tokens a wave 87 us, of 32: 89, of 16: 97 (W - 1 more steps each).
#include <hip/hip_runtime.h>

#include <type_traits>

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
                y[v] = SILU ? s * sigmoid<DT == SQ_DTYPE_F32>(s) : s;
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
        y[v] = SILU ? s * sigmoid<DT == SQ_DTYPE_F32>(s) : s;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) e[j + 1].store(p.window, base + (int64_t)j * p.channels);
    Elems<DT, V> o;
    o.set(y);
    o.store(p.y.p, b * p.y.stride, c);
}

// Gradients.  A workgroup has kThreads / 64 runs of 2^kConvBwdLog tokens one after the other, a wave each, over 64 V channels: their sums
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
                            const float sg = sigmoid<DT == SQ_DTYPE_F32>(a);
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

template <int DT>
constexpr int kVec = 16 / kBytes<DT>;
int conv_vec(int32_t dtype) { return dtype == SQ_DTYPE_F32 ? 4 : 8; }

enum { kOpFwd, kOpStep, kOpBwd };

template <int OP, int DT, int W, int V>
static hipError_t launch_w(const ConvParams& p, hipStream_t s) {
    constexpr int kCols = (OP == kOpBwd ? 64 : kThreads) * V;          // channels of a workgroup
    const int n_blocks = (p.channels + kCols - 1) / kCols;
    const int64_t n = OP == kOpStep ? p.batch : p.runs.n_seq > 0 ? run_slots(p.runs.n_tokens, p.runs.n_seq, p.runs.log) : 0;
    if (n == 0) return hipSuccess;
    const dim3 grid((unsigned)(n * n_blocks));
    const bool silu = p.act == SQ_ACT_SILU;
    auto kernel = OP == kOpFwd ? (silu ? k_conv<DT, W, V, true> : k_conv<DT, W, V, false>)
                : OP == kOpStep ? (silu ? k_conv_step<DT, W, V, true> : k_conv_step<DT, W, V, false>)
                                : (silu ? k_conv_bwd<DT, W, V, true> : k_conv_bwd<DT, W, V, false>);
    kernel<<<grid, kThreads, 0, s>>>(p, n_blocks);
    return hipGetLastError();
}

template <int OP, int DT, int V>
static hipError_t launch_v(const ConvParams& p, hipStream_t s) {
    switch (p.width) {
        case 2: return launch_w<OP, DT, 2, V>(p, s);
        case 3: return launch_w<OP, DT, 3, V>(p, s);
        case 4: return launch_w<OP, DT, 4, V>(p, s);
        case 5: return launch_w<OP, DT, 5, V>(p, s);
        case 6: return launch_w<OP, DT, 6, V>(p, s);
        case 7: return launch_w<OP, DT, 7, V>(p, s);
        case 8: return launch_w<OP, DT, 8, V>(p, s);
    }
    return hipErrorInvalidValue;
}

template <int OP>
static hipError_t launch_op(const ConvParams& p, bool vec, hipStream_t s) {
    constexpr int kDiv = OP == kOpBwd ? 4 : OP == kOpFwd ? 2 : 1;         // of the vector: the gradients keep W + 1 sums an element
    if (p.dtype == SQ_DTYPE_BF16)
        return vec ? launch_v<OP, SQ_DTYPE_BF16, kVec<SQ_DTYPE_BF16> / kDiv>(p, s) : launch_v<OP, SQ_DTYPE_BF16, 1>(p, s);
    if (p.dtype == SQ_DTYPE_F16)
        return vec ? launch_v<OP, SQ_DTYPE_F16, kVec<SQ_DTYPE_F16> / kDiv>(p, s) : launch_v<OP, SQ_DTYPE_F16, 1>(p, s);
    return vec ? launch_v<OP, SQ_DTYPE_F32, kVec<SQ_DTYPE_F32> / kDiv>(p, s) : launch_v<OP, SQ_DTYPE_F32, 1>(p, s);
}

int conv_run_log(int64_t, int64_t, int32_t) { return 4; }

hipError_t launch_conv(const ConvParams& p, bool vec, hipStream_t s) { return launch_op<kOpFwd>(p, vec, s); }
hipError_t launch_conv_step(const ConvParams& p, bool vec, hipStream_t s) { return launch_op<kOpStep>(p, vec, s); }
hipError_t launch_conv_bwd(const ConvParams& p, bool vec, hipStream_t s) {
    hipError_t e = launch_op<kOpBwd>(p, vec, s);
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    const int64_t cols = (int64_t)(p.width + 1) * p.channels;
    k_conv_sum<<<dim3((unsigned)((cols + 63) / 64)), 1024, 0, s>>>(
        p, p.runs.n_seq > 0 ? run_slots(p.runs.n_tokens, p.runs.n_seq, p.runs.log) : 0);
    return hipGetLastError();
}

}  // namespace sq
