// Selective state space scan over packed sequences: a gate for every channel and state (gfx950).
//
//   delta = softplus(dt + bias),  h_t = exp(delta_t a) h_{t-1} + delta_t u_t B_t,  p_t = C_t . h_t + d u_t,  y_t = p_t silu(z_t)
//
// There is no matrix product in it: the decay differs from state to state of every channel.  What bounds it is the vector unit,
// one exponential (at half the rate: 8 cycles a wave) and four operations (4 cycles each) for every token, channel and state, 123 us for
// 12301 tokens of 4096 channels of 16 states where memory needs 68.  It takes 333 us: 35 instructions for a token of four states a
// lane, 20 of them the recurrence, 2 the sum over a channel's lanes, the rest steps, gate and conversions; and whole sequences of
// different lengths on 448 workgroups keep 60 % of the vector unit busy.  Four states a lane: a channel
// of 16 states is four lanes, so one sequence of 4096 channels is 256 waves.  A workgroup's tile of tokens is prepared in LDS,
// every step (softplus) and product delta u once; B and C are read from there by all lanes, and y, complete after a sum over a
// channel's lanes, goes back through LDS so that gate and stores are made in rows.
//
// Few and long sequences leave most of the GPU idle that way, so they are cut into segments that run side by side: each from a
// state of zero (k_ssm with LOCAL: the state after it, and the sum of its steps, whose exponential is the product of its
// decays), then the states before the segments one after another (k_ssm_join), then each segment with its outputs.
#include <hip/hip_runtime.h>

#include "ssm_dev.h"

namespace sq {

// TT: tokens staged at a time.
template <int DT, int N, bool VEC, bool LOCAL, int TT>
__global__ void __launch_bounds__(kSsmThreads) k_ssm(const SsmParams p, int n_blocks) {
    using L = SsmLane<N>;
    constexpr int CB = L::kBlockCh, NV = CB / 4, kItems = (TT * NV + kSsmThreads - 1) / kSsmThreads;
    constexpr int kRows = LOCAL ? 1 : 2, kBc = (TT * kRows * (N / 4) + kSsmThreads - 1) / kSsmThreads;
    __shared__ __attribute__((aligned(16))) float2 s_d[TT][CB];           // delta, delta u
    __shared__ __attribute__((aligned(16))) float s_y[LOCAL ? 1 : TT][CB + L::kPad];
    __shared__ f32x4 s_bc[kRows][TT][N / 4];
    const int tid = (int)threadIdx.x, blk = (int)blockIdx.x % n_blocks;
    const int64_t slot = (int)blockIdx.x / n_blocks;
    const bool seg = p.runs.log >= 0;
    int seq, len;
    int64_t tok0;
    if (seg) {
        const RunAt r = run_of_slot(p.runs, slot);
        if (r.n == 0) return;
        seq = r.seq; len = r.n; tok0 = r.tok0;
    } else {
        const Span q = span_of(p.runs, (int)slot);
        seq = (int)slot; len = (int)q.len; tok0 = q.start;
    }
    const SsmBlock bc = block_channels(p, blk, CB);
    const int ch = tid / L::kPer, quarter = tid % L::kPer;            // the lane's channel of the block, its four states
    const bool there = ch < bc.n;
    const int64_t at = ((int64_t)bc.c0 + ch) * N + 4 * quarter;
    const int64_t states = (int64_t)p.channels * N;
    f32x4 a2 = load_states(p.a, at, there), h{0.f, 0.f, 0.f, 0.f};
    if constexpr (!LOCAL) {
        if (seg) h = load_states(p.hseg, slot * states + at, there);
        else if (p.s0) h = load_states(p.s0, seq * states + at, there);
    }
    float dsum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) a2[j] *= kLog2e;
    // staging: item i of a thread is four channels of one token, the same channels for all its items
    static_assert(kSsmThreads % NV == 0, "a thread's items have one column");
    const int c4 = tid % NV * 4;
    float bias[4], dw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        bias[j] = p.dt_bias && c4 + j < bc.n ? p.dt_bias[bc.c0 + c4 + j] : 0.f;
        dw[j] = !LOCAL && p.d && c4 + j < bc.n ? p.d[bc.c0 + c4 + j] : 0.f;
    }
    Four<DT, VEC> ru[kItems], rd[kItems], rbc[kBc];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int e = i * kSsmThreads + tid, t = t0 + e / NV;
            const int n = e < TT * NV && t < len ? bc.n - c4 : 0;
            ru[i].load(p.u.p, (tok0 + t) * p.u.stride + bc.c0 + c4, n);
            rd[i].load(p.dt.p, (tok0 + t) * p.dt.stride + bc.c0 + c4, n);
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = i * kSsmThreads + tid, k = e % (N / 4), t = t0 + e / (N / 4) % TT, w = e / (N / 4 * TT);
            const int n = w < kRows && t < len ? 4 : 0;
            const Rows& r = w ? p.c : p.b;
            rbc[i].load(r.p, (tok0 + t) * r.stride + bc.group * N + 4 * k, n);
        }
    };
    fetch(0);
    for (int t0 = 0; t0 < len; t0 += TT) {
        const int nt = len - t0 < TT ? len - t0 : TT;
        Four<DT, VEC> cu[kItems], cz[LOCAL ? 1 : kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int e = i * kSsmThreads + tid, t = e / NV;
            cu[i] = ru[i];
            if (e < TT * NV && t < nt) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = rd[i].at(j) + bias[j];
                if (p.softplus) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = softplus(x[j]).value;
                }
#pragma unroll
                for (int j = 0; j < 4; j += 2)
                    *reinterpret_cast<f32x4*>(&s_d[t][c4 + j]) = f32x4{x[j], x[j] * ru[i].at(j), x[j + 1], x[j + 1] * ru[i].at(j + 1)};
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = i * kSsmThreads + tid, k = e % (N / 4), t = e / (N / 4) % TT, w = e / (N / 4 * TT);
            f32x4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = rbc[i].at(j);
            if (w < kRows) s_bc[w][t][k] = x;
        }
        __syncthreads();
        if (t0 + TT < len) fetch(t0 + TT);
        if constexpr (!LOCAL) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int e = i * kSsmThreads + tid, t = e / NV;
                cz[i].load(p.z.p, (tok0 + t0 + t) * p.z.stride + bc.c0 + c4, p.z.p && e < TT * NV && t < nt ? bc.n - c4 : 0);
            }
        }
        auto step = [&](const float2& d, const f32x4& b, const f32x4& c) {
            float y = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(__builtin_amdgcn_exp2f(d.x * a2[j]), h[j], d.y * b[j]);
                if constexpr (!LOCAL) y = fmaf(h[j], c[j], y);
            }
            if constexpr (LOCAL) dsum += d.x;
            return y;
        };
        int t = 0;
        for (; t + 4 <= nt; t += 4) {
            float2 d[4];
            f32x4 b[4], c[4];
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                d[k] = s_d[t + k][ch];
                b[k] = s_bc[0][t + k][quarter];
                if constexpr (!LOCAL) c[k] = s_bc[kRows - 1][t + k][quarter];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = step(d[k], b[k], c[k]);
            if constexpr (!LOCAL) {
                channel_sums4<L::kPer>(y);
                put_sums4<L::kPer>(y, quarter, [&](int k, float v) { s_y[t + k][ch] = v; });
            }
        }
        for (; t < nt; ++t) {
            f32x4 c{0.f, 0.f, 0.f, 0.f};
            if constexpr (!LOCAL) c = s_bc[kRows - 1][t][quarter];
            float y = step(s_d[t][ch], s_bc[0][t][quarter], c);
            if constexpr (!LOCAL) {
                y = channel_sum<L::kPer>(y);
                if (quarter == 0) s_y[t][ch] = y;
            }
        }
        __syncthreads();
        if constexpr (!LOCAL) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int e = i * kSsmThreads + tid, t = e / NV;
                if (e >= TT * NV || t >= nt) continue;
                const f32x4 sum = *reinterpret_cast<const f32x4*>(&s_y[t][c4]);
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = sum[j];
                if (p.d) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fmaf(dw[j], cu[i].at(j), y[j]);
                }
                if (p.z.p) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] *= cz[i].at(j) * sigmoid(cz[i].at(j));
                }
                Four<DT, VEC>::store(p.y.p, (tok0 + t0 + t) * p.y.stride + bc.c0 + c4, bc.n - c4, y);
            }
        }
    }
    if (!there) return;
    if constexpr (LOCAL) {
        *reinterpret_cast<f32x4*>(p.hseg + slot * states + at) = h;
        if (quarter == 0) p.dsum[slot * p.channels + bc.c0 + ch] = dsum;
    } else if (!seg && p.s1) {
        *reinterpret_cast<f32x4*>(p.s1 + seq * states + at) = h;
    }
}

// The states before a sequence's segments, one after another (blockIdx.y of 1: the gradients of the states after them,
// from the last to the first): h <- exp(a sum of steps) h + what the segment makes from zero.  Four states a thread; the
// loads of eight segments are in flight together.
__global__ void __launch_bounds__(256) k_ssm_join(const SsmParams p, int n_blocks) {
    const int blk = (int)blockIdx.x % n_blocks, seq = (int)blockIdx.x / n_blocks;
    const bool rev = blockIdx.y != 0;
    const int64_t states = (int64_t)p.channels * p.d_state, at = ((int64_t)blk * 256 + (int)threadIdx.x) * 4;
    if (at >= states) return;
    const int64_t c = at / p.d_state;
    const Span q = span_of(p.runs, seq);
    const int64_t slot0 = run_slot0(p.runs, q, seq), n = (q.len + (int64_t(1) << p.runs.log) - 1) >> p.runs.log;
    const float* first = rev ? p.ds1 : p.s0;
    float* last = rev ? p.ds0 : p.s1;
    float* w = (rev ? p.kseg : p.hseg) + at;
    f32x4 h = load_states(first, seq * states + at, first != nullptr), a2 = load_states(p.a, at, true);
#pragma unroll
    for (int j = 0; j < 4; ++j) a2[j] *= kLog2e;
    constexpr int K = 8;
    for (int64_t i0 = 0; i0 < n; i0 += K) {
        f32x4 x[K];
        float ds[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t s = slot0 + (rev ? n - 1 - (i0 + k) : i0 + k);
            if (i0 + k < n) {
                x[k] = *reinterpret_cast<const f32x4*>(w + s * states);
                ds[k] = p.dsum[s * p.channels + c];
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t s = slot0 + (rev ? n - 1 - (i0 + k) : i0 + k);
            if (i0 + k >= n) break;
            *reinterpret_cast<f32x4*>(w + s * states) = h;
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = fmaf(__builtin_amdgcn_exp2f(ds[k] * a2[j]), h[j], x[k][j]);
        }
    }
    if (last) *reinterpret_cast<f32x4*>(last + seq * states + at) = h;
}

// One token of each request, the state in a slot of the pool: bound by reading and writing the states (256 requests of 4096 x 16 float32
// states: 28.7 us, 5.0 TB/s).
template <int DT, int N, bool VEC>
__global__ void __launch_bounds__(kSsmThreads) k_ssm_step(const SsmParams p, int n_blocks) {
    using L = SsmLane<N>;
    const int tid = (int)threadIdx.x, blk = (int)blockIdx.x % n_blocks;
    const int64_t r = (int)blockIdx.x / n_blocks;
    const int64_t slot = p.slots ? (int64_t)p.slots[r] : r;
    const SsmBlock bc = block_channels(p, blk, L::kBlockCh);
    const int ch = tid / L::kPer, quarter = tid % L::kPer;
    if (slot < 0 || slot >= p.n_slots || ch >= bc.n) return;
    const int64_t c = bc.c0 + ch;
    float* state = p.state + (slot * p.channels + c) * N + 4 * quarter;
    f32x4 h = *reinterpret_cast<const f32x4*>(state);
    const f32x4 a = *reinterpret_cast<const f32x4*>(p.a + c * N + 4 * quarter);
    Elems<DT, 1> eu, ed, ez;
    Four<DT, VEC> eb, ec;
    eu.load(p.u.p, r * p.u.stride + c);
    ed.load(p.dt.p, r * p.dt.stride + c);
    if (p.z.p) ez.load(p.z.p, r * p.z.stride + c);
    eb.load(p.b.p, r * p.b.stride + bc.group * N + 4 * quarter, 4);
    ec.load(p.c.p, r * p.c.stride + bc.group * N + 4 * quarter, 4);
    float delta = ed.at(0) + (p.dt_bias ? p.dt_bias[c] : 0.f);
    if (p.softplus) delta = softplus(delta).value;
    const float du = delta * eu.at(0);
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(__builtin_amdgcn_exp2f(delta * (a[j] * kLog2e)), h[j], du * eb.at(j));
        y = fmaf(h[j], ec.at(j), y);
    }
    *reinterpret_cast<f32x4*>(state) = h;
    y = channel_sum<L::kPer>(y);
    if (quarter != 0) return;
    if (p.d) y = fmaf(p.d[c], eu.at(0), y);
    if (p.z.p) {
        const float z = ez.at(0);
        y *= z * sigmoid(z);
    }
    Elems<DT, 1> o;
    o.set(&y);
    o.store(p.y.p, r * p.y.stride + c);
}

// ------------------------------------------------------------------ launches

// The gradients always go by segments: of 128 tokens where they still give every CU several workgroups (less to join: 16 us instead of 27
// of 850 for 8190 tokens of 4096 x 16), of 32 where 64 would leave CUs without one (us with 32 / 64 tokens: 500 tokens of 256 x 16: 42/54, of
// 1024 x 16: 42/55, of 256 x 128: 49/63; 1000 of 1024 x 16: 51/60; 250 of 4096 x 16: 49/61).
//
// The forward pass walks the tokens twice with segments and takes two launches more, so it takes them only where whole sequences leave much of the GPU
// idle for long.  With g workgroups of whole sequences of L tokens, a sequence takes 0.115 L us whatever g is, up to one a CU, and segments 0.0004 g L
// and 20 us more: L (288 - g) >= 50000.  Above 256 CUs have two and take longer (from 1563 tokens on), from 352 on segments cost more at equal lengths (us with
// segments / without, bfloat16, 16 states, sequences x channels of tokens; 256 x 16 states are 4 workgroups):
//   1 x 4096 of 160: 27/21, 192: 27/25, 224: 26/29, 320: 28/39, 777: 41/89, 4000: 137/448
//   2 x 4096 of 192: 29/26, 256: 29/32, 320: 35/39, 2000: 127/228      8 x 1024 of 224: 33/29, 256: 35/32, 320: 35/40, 1500: 98/170
//   40 x 256 of 150: 34/22, 256: 42/33, 320: 43/40, 400: 49/49         3 x 4096 of 2000: 174/229
//   4 x 4096 of 160: 35/23, 400: 64/51, 2000: 222/231                  8 x 2048 of 1500: 173/174
//   5 x 4096 of 2000: 280/321    80 x 256 of 400: 75/66                6 x 4096 of 1757: 303/284    7 x 4096 of 1757: 347/286
// Other numbers of states are alike (C x N = 65536, 1 x 4000, 3 x 2000, 7 x 1757: N = 8: 186/618, 254/330, 508/382; N = 32: 123/387, 156/201, 308/243; N = 64:
// 116/364, 152/189, 300/235; N = 128: 120/403, 158/209, 307/251).  The rule goes by the mean, since the lengths are on the device: one long sequence among
// many short ones goes without segments (one of 8000 beside 63 of 8 tokens of 4096 x 16: 1035 us, 247 with them; in a call of its own 233).
// A segment is at least 64 tokens, longer once 2048 workgroups are there.
int ssm_segment_log(int64_t n_tokens, int64_t n_seq, int64_t blocks, bool backward) {
    if (backward) return (n_tokens >> 7) * blocks >= 2048 ? 7 : (n_tokens >> 6) * blocks >= 512 ? 6 : 5;
    const int64_t groups = n_seq * blocks, left = groups < 256 ? 288 - groups : 32;
    if (n_seq < 1 || groups >= 352 || n_tokens / n_seq * left < 50000) return -1;
    int log = 6;
    while (log < 12 && (n_tokens >> (log + 1)) * blocks >= 2048) ++log;
    return log;
}

hipError_t launch_ssm_join(const SsmParams& p, int directions, hipStream_t s) {
    const int jb = (int)(((int64_t)p.channels * p.d_state + 1023) / 1024);
    k_ssm_join<<<dim3((unsigned)((int64_t)p.runs.n_seq * jb), (unsigned)directions), 256, 0, s>>>(p, jb);
    return hipGetLastError();
}

// Up to how many workgroups whole sequences of 64 tokens and more are staged 64 tokens at a time: as many as their LDS lets the GPU's 256 CUs of
// 160 KB hold at once, each waiting at its own barriers; beyond that the workgroups that 32 tokens leave room for hide more.
// us with 64 / 32 tokens, bfloat16, C x N = 65536 (64 workgroups a sequence), sequences x tokens:
//    N = 8:    7 x 1757: 688/550   16 x 700: 477/336   64 x 188: 512/344   7 x 100: 38/27   1 x 100: 19/19
//    N = 16:   7 x 1757: 415/444   8 x 1500: 324/350   12 x 1000: 299/248   64 x 188: 256/211   7 x 100: 21.7/21.9
//    N = 32:   7 x 1757: 351/380   12 x 1000: 208/213   16 x 700: 175/183   64 x 188: 182/179   7 x 100: 19.5/19.7
//    N = 64:   7 x 1757: 349/366   12 x 1000: 205/212   16 x 700: 173/178   64 x 188: 181/176   7 x 100: 19.0/19.7
//    N = 128:  7 x 1757: 368/387   8 x 1500: 288/303   12 x 1000: 264/219   64 x 188: 228/183   7 x 100: 20.5/20.9
// float32 is alike (7 x 1757: 748/584, 435/454, 366/401, 348/369, 378/391).  With 8 states one workgroup of 64 tokens fills a CU, and it is never
// faster.  Sequences of a few tokens need no more than 32 (64 of 4 tokens: 30 us with 64, 19 with 32).
template <int N>
constexpr int64_t kSsmLong = N == 8 ? 0 : 256 * (160 * 1024 / int64_t(sizeof(float) * 64 * (3 * SsmLane<N>::kBlockCh + SsmLane<N>::kPad + 2 * N)));
static_assert(kSsmLong<16> == 512 && kSsmLong<32> == 768 && kSsmLong<64> == 768 && kSsmLong<128> == 512, "workgroups that 160 KB hold");

template <int DT, int N, bool VEC>
static hipError_t scan_n(const SsmParams& p, hipStream_t s) {
    const int blocks = (int)ssm_blocks(p.channels, p.n_groups, N);
    if (p.runs.log < 0) {
        const int64_t groups = (int64_t)p.runs.n_seq * blocks;
        const dim3 grid((unsigned)groups);
        if constexpr (kSsmLong<N> > 0) {
            if (groups <= kSsmLong<N> && p.runs.n_tokens >= 64 * (int64_t)p.runs.n_seq) {
                k_ssm<DT, N, VEC, false, 64><<<grid, kSsmThreads, 0, s>>>(p, blocks);
                return hipGetLastError();
            }
        }
        k_ssm<DT, N, VEC, false, 32><<<grid, kSsmThreads, 0, s>>>(p, blocks);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(run_slots(p.runs.n_tokens, p.runs.n_seq, p.runs.log) * blocks));
    k_ssm<DT, N, VEC, true, 32><<<grid, kSsmThreads, 0, s>>>(p, blocks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = launch_ssm_join(p, 1, s);
    if (e != hipSuccess) return e;
    k_ssm<DT, N, VEC, false, 32><<<grid, kSsmThreads, 0, s>>>(p, blocks);
    return hipGetLastError();
}
template <int DT, int N, bool VEC>
static hipError_t step_n(const SsmParams& p, hipStream_t s) {
    const int blocks = (int)ssm_blocks(p.channels, p.n_groups, N);
    k_ssm_step<DT, N, VEC><<<dim3((unsigned)(p.batch * blocks)), kSsmThreads, 0, s>>>(p, blocks);
    return hipGetLastError();
}

hipError_t launch_ssm(const SsmParams& p, bool vec, hipStream_t s) { SQ_SSM_DISPATCH(scan_n, p, s); }
hipError_t launch_ssm_step(const SsmParams& p, bool vec, hipStream_t s) { SQ_SSM_DISPATCH(step_n, p, s); }

}  // namespace sq
