// Gradients of the selective state space scan (gfx950).
//
//   dp = dy silu(z),  G_t = C_t dp_t + e_{t+1} G_{t+1} (after the last token: + ds1),  e_t = exp(delta_t a)
//   dC_t = sum_c dp h_t,  dB_t = sum_c G_t delta u,  du = d dp + delta sum_n G B,  ddelta = sum_n G (a e h_{t-1} + u B),
//   ddt = ddelta sigmoid(dt + bias),  da = sum_t G delta e h_{t-1},  dd = sum_t dp u,  dz = dy p silu'(z),  ds0 = e_1 G_1
//
// Nothing of the forward call is kept.  Sequences are cut into segments of 32 to 128 tokens.  k_ssm_ends finds, for all of them side by
// side, the state after a segment from a state of zero and the gradient before it from a gradient of zero, in one walk: the
// latter is sum_t (e_1 ... e_t) C_t dp_t; it also keeps the state before every 8th token.  k_ssm_join turns the ends into the states
// before and the gradients after the segments.  k_ssm_grad takes a segment's tiles of 8 tokens from the last to the first: the state
// before the tile from what k_ssm_ends kept and the decayed state before the segment, forward with every decay and decayed state in
// registers, then backward.  Sums over a channel's states are lane exchanges; dB
// and dC are sums over all channels: over the wave's by exchanges that halve the values a lane holds each time, over the
// workgroup's waves in LDS, over the workgroups by k_ssm_sum_bc, all in a fixed order.
//
// The vector unit bounds it: 43 instructions for a token of four states a lane in k_ssm_ends (all of its time used), 102 in k_ssm_grad
// (61 %).  8190 tokens of 4096 channels of 16 states in bfloat16: 711 us a pass; floor by memory 79 us, by the vector unit 205.  Under a
// tracer, where each kernel runs by itself and some 10 % longer, 181 us are the ends, 16 joining, 579 the gradients, 20 the sums.  Keeping the states before
// every 8th token (8 bytes a token and channel, written and read) instead of walking the segment again: 689 -> 604 us.  What staging makes stays in LDS, and
// the products of two tokens are scheduled apart, or the loads of all eight move up: three waves a SIMD (168 registers, some 20 of them spilled) 557 us,
// two (no spills) 605; in float32 and from 64 states on, where 26 to 44 would spill, two waves are faster (36 against 29 us for 515
// tokens of 256 x 64 in segments of 64).  Rows of single elements (4095 channels): 1084 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ssm_dev.h"

namespace sq {

constexpr int kTile = kSsmTile;

template <int DT, int N, bool VEC>
__global__ void __launch_bounds__(kSsmThreads) k_ssm_ends(const SsmParams p, int n_blocks) {
    using L = SsmLane<N>;
    constexpr int TT = 32, CB = L::kBlockCh, NV = CB / 4, kItems = (TT * NV + kSsmThreads - 1) / kSsmThreads;
    constexpr int kBc = (TT * 2 * (N / 4) + kSsmThreads - 1) / kSsmThreads;
    __shared__ __attribute__((aligned(16))) float2 s_d[TT][CB];           // delta, delta u
    __shared__ __attribute__((aligned(16))) float s_p[TT][CB];            // dp
    __shared__ f32x4 s_bc[2][TT][N / 4];
    const int tid = (int)threadIdx.x, blk = (int)blockIdx.x % n_blocks;
    const int64_t slot = (int)blockIdx.x / n_blocks;
    const RunAt r = run_of_slot(p.runs, slot);
    if (r.n == 0) return;
    const SsmBlock bc = block_channels(p, blk, CB);
    const int ch = tid / L::kPer, quarter = tid % L::kPer;
    const bool there = ch < bc.n;
    const int64_t at = ((int64_t)bc.c0 + ch) * N + 4 * quarter;
    f32x4 a2 = load_states(p.a, at, there), h{0.f, 0.f, 0.f, 0.f}, k{0.f, 0.f, 0.f, 0.f}, e{1.f, 1.f, 1.f, 1.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) a2[j] *= kLog2e;
    float dsum = 0.f, bias[4];
    static_assert(kSsmThreads % NV == 0, "a thread's items have one column");
    const int c4 = tid % NV * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = p.dt_bias && c4 + j < bc.n ? p.dt_bias[bc.c0 + c4 + j] : 0.f;
    for (int t0 = 0; t0 < r.n; t0 += TT) {
        const int nt = r.n - t0 < TT ? r.n - t0 : TT;
        Four<DT, VEC> eu[kItems], ed[kItems], ey[kItems], ez[kItems], eb[kBc];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int x = i * kSsmThreads + tid, t = x / NV;
            const int n = x < TT * NV && t < nt ? bc.n - c4 : 0;
            const int64_t tok = r.tok0 + t0 + t;
            eu[i].load(p.u.p, tok * p.u.stride + bc.c0 + c4, n);
            ed[i].load(p.dt.p, tok * p.dt.stride + bc.c0 + c4, n);
            ey[i].load(p.dy.p, tok * p.dy.stride + bc.c0 + c4, n);
            ez[i].load(p.z.p, tok * p.z.stride + bc.c0 + c4, p.z.p ? n : 0);
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int x = i * kSsmThreads + tid, q = x % (N / 4), t = x / (N / 4) % TT, w = x / (N / 4 * TT);
            const Rows& rows = w ? p.c : p.b;
            eb[i].load(rows.p, (r.tok0 + t0 + t) * rows.stride + bc.group * N + 4 * q, w < 2 && t < nt ? 4 : 0);
        }
        if (t0) __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int x = i * kSsmThreads + tid, t = x / NV;
            if (x >= TT * NV || t >= nt) continue;
            float d[4];
            f32x4 g;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j] = ed[i].at(j) + bias[j];
                g[j] = ey[i].at(j);
            }
            if (p.softplus) {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = softplus(d[j]).value;
            }
            if (p.z.p) {
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] *= ez[i].at(j) * sigmoid(ez[i].at(j));
            }
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                *reinterpret_cast<f32x4*>(&s_d[t][c4 + j]) = f32x4{d[j], d[j] * eu[i].at(j), d[j + 1], d[j + 1] * eu[i].at(j + 1)};
            *reinterpret_cast<f32x4*>(&s_p[t][c4]) = g;
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int x = i * kSsmThreads + tid, q = x % (N / 4), t = x / (N / 4) % TT, w = x / (N / 4 * TT);
            f32x4 f;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = eb[i].at(j);
            if (w < 2) s_bc[w][t][q] = f;
        }
        __syncthreads();
        for (int t8 = 0; t8 < nt; t8 += kTile) {
            if (there && t0 + t8 > 0) {                   // what k_ssm_grad starts its tiles from
                const int64_t tile = (r.tok0 + t0 + t8) / kTile;
                *reinterpret_cast<f32x4*>(p.htile + tile * p.channels * N + at) = h;
                if (quarter == 0) p.dtile[tile * p.channels + bc.c0 + ch] = dsum;
            }
            auto step = [&](int t) {
                const float2 d = s_d[t][ch];
                const float dp = s_p[t][ch];
                const f32x4 b = s_bc[0][t][quarter], c = s_bc[1][t][quarter];
                dsum += d.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = __builtin_amdgcn_exp2f(d.x * a2[j]);
                    h[j] = fmaf(x, h[j], d.y * b[j]);
                    e[j] *= x;
                    k[j] = fmaf(e[j], c[j] * dp, k[j]);
                }
            };
            if (t8 + kTile <= nt) {
#pragma unroll
                for (int t = 0; t < kTile; ++t) step(t8 + t);
            } else {
                for (int t = t8; t < nt; ++t) step(t);
            }
        }
    }
    if (!there) return;
    const int64_t to = slot * p.channels * N + at;
    *reinterpret_cast<f32x4*>(p.hseg + to) = h;
    *reinterpret_cast<f32x4*>(p.kseg + to) = k;
    if (quarter == 0) p.dsum[slot * p.channels + bc.c0 + ch] = dsum;
}

template <int N>
struct Grad {
    static constexpr int kWaves = N == 8 ? 2 : N <= 64 ? 4 : 8, kThreads = kWaves * 64;
    static constexpr int kPer = N / 4, kWaveCh = 64 / kPer, CB = kWaves * kWaveCh;
    static constexpr int TS = 16;                         // tokens staged at a time
    static constexpr int kPad = (kWaveCh + 3) / 4 * 4;    // rows apart so that a wave's tokens meet no bank twice, and aligned to four elements
    static constexpr int NV = CB / 4, kItems = (TS * NV + kThreads - 1) / kThreads;
    static constexpr int kBc = (TS * 2 * kPer + kThreads - 1) / kThreads;
    static constexpr int kGroups = kThreads / NV;         // threads that share a channel in the sums over tokens
    static_assert(CB % 4 == 0 && (CB + kPad) % 4 == 0, "rows are accessed four elements at a time");
};

// One token's v[0..3], of the lane's four states, summed over the wave's channels.  Each exchange joins two values' halves, so that
// the sums end up spread over the lanes; `out` is a row of N floats.
template <int PER>
__device__ __forceinline__ void wave_sums(const float (&v)[4], float* out) {
    const int lane = (int)threadIdx.x & 63;
    const float a0 = join32(v[0], v[2]), a1 = join32(v[1], v[3]);              // upper half: states 2 and 3
    float* to = out + 4 * (lane % PER) + (lane & 32 ? 2 : 0);
    if constexpr (PER == 32) {
        *reinterpret_cast<float2*>(to) = float2{a0, a1};
    } else {
        float b = join16(a0, a1);                                              // odd rows: states 1 and 3
        if constexpr (PER <= 8) b += dpp<kDppRor8>(b);
        if constexpr (PER <= 4) b += dpp<kDppRor4>(b);
        if constexpr (PER <= 2) b += dpp<kDppXor2>(b);
        if ((lane & 15) < PER) to[lane & 16 ? 1 : 0] = b;
    }
}

template <int DT, int N, bool VEC>
__global__ void __launch_bounds__(Grad<N>::kThreads, DT != SQ_DTYPE_F32 && N <= 32 ? 3 : 2) k_ssm_grad(const SsmParams p, int n_blocks) {
    using K = Grad<N>;
    constexpr int TB = kTile, TS = K::TS, CB = K::CB, NV = K::NV, kT = K::kThreads, PER = K::kPer;
    // All that a token and channel needs lives here between staging and the gradients' rows: registers are for the states.
    __shared__ __attribute__((aligned(16))) float2 s_d[TS][CB];           // delta, delta u
    __shared__ __attribute__((aligned(16))) float s_p[TS][CB];            // dp
    __shared__ __attribute__((aligned(16))) float s_sl[TS][CB], s_sz[TS][CB];                                  // sigmoid of dt + bias, of z
    __shared__ __attribute__((aligned(16))) float s_y[TS][CB + K::kPad], s_gb[TS][CB + K::kPad], s_ga[TS][CB + K::kPad];   // sums of C h, G B, a G e h
    __shared__ __attribute__((aligned(16))) float s_par[2][CB];           // dt_bias, d
    __shared__ f32x4 s_acc[2][kT];                        // sums of dd and ddt_bias over a staging thread's tokens, four channels
    __shared__ f32x4 s_bc[2][TS][N / 4];
    __shared__ __attribute__((aligned(16))) float s_w[K::kWaves][TB][2 * N];   // dB and dC of a tile's tokens over a wave's channels
    const int tid = (int)threadIdx.x, wave = tid >> 6, blk = (int)blockIdx.x % n_blocks;
    const int64_t slot = (int)blockIdx.x / n_blocks;
    const RunAt r = run_of_slot(p.runs, slot);
    const SsmBlock bc = block_channels(p, blk, CB);
    const int ch = tid / PER, quarter = tid % PER;
    const bool there = ch < bc.n;
    const int64_t states = (int64_t)p.channels * N, at = ((int64_t)bc.c0 + ch) * N + 4 * quarter;
    f32x4 da{0.f, 0.f, 0.f, 0.f};
    static_assert(kT % NV == 0, "a thread's items have one column");
    const int c4 = tid % NV * 4;
    s_acc[0][tid] = s_acc[1][tid] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (r.n > 0) {
        // Lanes without a channel hold zeros throughout (dp, u, the gradient and the states before the segment), so they add nothing
        f32x4 a2 = load_states(p.a, at, there);
#pragma unroll
        for (int j = 0; j < 4; ++j) a2[j] *= kLog2e;
        const f32x4 h0 = load_states(p.hseg, slot * states + at, there);
        f32x4 gk = load_states(p.kseg, slot * states + at, there);
        if (tid < CB) {
            s_par[0][tid] = p.dt_bias && tid < bc.n ? p.dt_bias[bc.c0 + tid] : 0.f;
            s_par[1][tid] = p.d && tid < bc.n ? p.d[bc.c0 + tid] : 0.f;
        }
        __syncthreads();
        Four<DT, VEC> ru[K::kItems], rd[K::kItems], ry[K::kItems], rz[K::kItems], rbc[K::kBc];
        auto fetch = [&](int t0) {
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                const int x = i * kT + tid, t = t0 + x / NV;
                const int n = x < TS * NV && t < r.n ? bc.n - c4 : 0;
                const int64_t tok = r.tok0 + t;
                ru[i].load(p.u.p, tok * p.u.stride + bc.c0 + c4, n);
                rd[i].load(p.dt.p, tok * p.dt.stride + bc.c0 + c4, n);
                ry[i].load(p.dy.p, tok * p.dy.stride + bc.c0 + c4, n);
                rz[i].load(p.z.p, tok * p.z.stride + bc.c0 + c4, p.z.p ? n : 0);
            }
#pragma unroll
            for (int i = 0; i < K::kBc; ++i) {
                const int x = i * kT + tid, q = x % (N / 4), t = t0 + x / (N / 4) % TS, w = x / (N / 4 * TS);
                const Rows& rows = w ? p.c : p.b;
                rbc[i].load(rows.p, (r.tok0 + t) * rows.stride + bc.group * N + 4 * q, w < 2 && t < r.n ? 4 : 0);
            }
        };
        // the state before a tile: what its segment made so far from zero, and what is left of the state before the segment
        f32x4 hl;
        float dl;
        auto fetch_state = [&](int tile) {
            const int64_t i = r.tok0 / kTile + tile;             // (r.tok0 + kTile tile) / kTile
            hl = load_states(p.htile, i * states + at, there);
            dl = there ? p.dtile[i * p.channels + bc.c0 + ch] : 0.f;
        };
        auto row4 = [&](float* at4) -> f32x4& { return *reinterpret_cast<f32x4*>(at4); };
        auto stage = [&](int nt) {
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                const int x = i * kT + tid, t = x / NV;
                if (x >= TS * NV || t >= nt) continue;
                f32x4 d = row4(&s_par[0][c4]), g;
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += rd[i].at(j);
                if (p.softplus) {
                    f32x4 slope;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const SoftPlus s = softplus(d[j]);
                        slope[j] = softplus_slope(d[j], s.w);
                        d[j] = s.value;
                    }
                    row4(&s_sl[t][c4]) = slope;
                }
#pragma unroll
                for (int j = 0; j < 4; j += 2)
                    row4(&s_d[t][c4 + j].x) = f32x4{d[j], d[j] * ru[i].at(j), d[j + 1], d[j + 1] * ru[i].at(j + 1)};
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] = ry[i].at(j);
                if (p.z.p) {
                    f32x4 sz;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sz[j] = sigmoid(rz[i].at(j));
                        g[j] *= rz[i].at(j) * sz[j];
                    }
                    row4(&s_sz[t][c4]) = sz;
                }
                row4(&s_p[t][c4]) = g;
            }
#pragma unroll
            for (int i = 0; i < K::kBc; ++i) {
                const int x = i * kT + tid, q = x % (N / 4), t = x / (N / 4) % TS, w = x / (N / 4 * TS);
                f32x4 f;
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = rbc[i].at(j);
                if (w < 2) s_bc[w][t][q] = f;
            }
        };
        // a tile, `base` its place among the staged tokens, nt (all of them if FULL) its tokens; `hs` the state before it
        auto tile_back = [&](auto full, int base, int nt, const f32x4& hs) {
            constexpr bool FULL = decltype(full)::value;
            f32x4 eh[TB], e[TB], h = hs;                  // decayed states, decays
#pragma unroll
            for (int t4 = 0; t4 < TB; t4 += 4) {
                float y[4];
#pragma unroll
                for (int t = t4; t < t4 + 4; ++t) {
                    if (!FULL && t >= nt) break;
                    const float2 d = s_d[base + t][ch];
                    const float dpt = s_p[base + t][ch];
                    const f32x4 b = s_bc[0][base + t][quarter], c = s_bc[1][base + t][quarter];
                    float s = 0.f, v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e[t][j] = __builtin_amdgcn_exp2f(d.x * a2[j]);
                        eh[t][j] = e[t][j] * h[j];
                        h[j] = fmaf(d.y, b[j], eh[t][j]);
                        s = fmaf(h[j], c[j], s);
                        v[j] = dpt * h[j];
                    }
                    wave_sums<PER>(v, &s_w[wave][t][N]);
                    if (t & 1) __builtin_amdgcn_sched_barrier(0);      // else the loads of all eight tokens move up and registers spill
                    y[t - t4] = s;
                    if (!FULL) {
                        s = channel_sum<PER>(s);
                        if (quarter == 0) s_y[base + t][ch] = s;
                    }
                }
                if (FULL && p.z.p) {
                    channel_sums4<PER>(y);
                    put_sums4<PER>(y, quarter, [&](int k, float v) { s_y[base + t4 + k][ch] = v; });
                }
            }
#pragma unroll
            for (int t4 = TB - 4; t4 >= 0; t4 -= 4) {
                float gb[4], ga[4];
#pragma unroll
                for (int t = t4 + 3; t >= t4; --t) {
                    if (!FULL && t >= nt) continue;
                    const float2 d = s_d[base + t][ch];
                    const float dpt = s_p[base + t][ch];
                    const f32x4 b = s_bc[0][base + t][quarter], c = s_bc[1][base + t][quarter];
                    float v[4], sb = 0.f, sa = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float g = fmaf(c[j], dpt, gk[j]), through = g * eh[t][j];
                        sb = fmaf(g, b[j], sb);
                        sa = fmaf(a2[j], through, sa);
                        da[j] = fmaf(through, d.x, da[j]);
                        v[j] = g * d.y;
                        gk[j] = g * e[t][j];
                    }
                    wave_sums<PER>(v, &s_w[wave][t][0]);
                    if (!(t & 1)) __builtin_amdgcn_sched_barrier(0);
                    gb[t - t4] = sb;
                    ga[t - t4] = sa;
                    if (!FULL) {
                        sb = channel_sum<PER>(sb);
                        sa = channel_sum<PER>(sa);
                        if (quarter == 0) {
                            s_gb[base + t][ch] = sb;
                            s_ga[base + t][ch] = sa;
                        }
                    }
                }
                if (FULL) {
                    channel_sums4<PER>(gb);
                    channel_sums4<PER>(ga);
                    put_sums4<PER>(gb, quarter, [&](int k, float v) { s_gb[base + t4 + k][ch] = v; });
                    put_sums4<PER>(ga, quarter, [&](int k, float v) { s_ga[base + t4 + k][ch] = v; });
                }
            }
        };
        const int n_staged = (r.n + TS - 1) / TS;
        fetch((n_staged - 1) * TS);
        if ((r.n - 1) / TB > 0) fetch_state((r.n - 1) / TB);
        for (int st = n_staged - 1; st >= 0; --st) {
            const int t0 = st * TS, nt = r.n - t0 < TS ? r.n - t0 : TS;
            stage(nt);
            __syncthreads();
#pragma unroll
            for (int half = TS / TB - 1; half >= 0; --half) {
                const int tile = st * (TS / TB) + half, n = nt - half * TB;
                if (n <= 0) continue;
                f32x4 hs = h0;
                if (tile > 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) hs[j] = fmaf(__builtin_amdgcn_exp2f(dl * a2[j]), h0[j], hl[j]);
                }
                if (tile > 1) fetch_state(tile - 1);
                if (n >= TB) tile_back(std::true_type{}, half * TB, TB, hs);
                else tile_back(std::false_type{}, half * TB, n, hs);
                __syncthreads();
                // dB and dC of the tile's tokens over the waves, and out
                const int most = n < TB ? n : TB;
                float* part = p.bc_part + ((int64_t)blk * p.runs.n_tokens + r.tok0 + t0 + half * TB) * (2 * N);
                for (int x = tid; x < most * 2 * N; x += kT) {
                    float s = (&s_w[0][0][0])[x];
#pragma unroll
                    for (int w = 1; w < K::kWaves; ++w) s += (&s_w[w][0][0])[x];
                    part[x] = s;
                }
                if (half > 0) __syncthreads();            // after the last one the next staging has its own
            }
            // the rows of these tokens: du, ddt, dz
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                const int x = i * kT + tid, t = x / NV;
                if (x >= TS * NV || t >= nt) continue;
                const int64_t tok = r.tok0 + t0 + t;
                const f32x4 g = row4(&s_p[t][c4]), gb = row4(&s_gb[t][c4]), ga = row4(&s_ga[t][c4]), dw = row4(&s_par[1][c4]);
                float du[4], ddt[4];
                f32x4 dd = s_acc[0][tid], db = s_acc[1][tid];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = ru[i].at(j);
                    du[j] = s_d[t][c4 + j].x * gb[j];
                    ddt[j] = fmaf(ga[j], 0.69314718056f, u * gb[j]);
                    dd[j] = fmaf(g[j], u, dd[j]);
                }
                s_acc[0][tid] = dd;
                if (p.d) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) du[j] = fmaf(dw[j], g[j], du[j]);
                }
                if (p.softplus) {
                    const f32x4 slope = row4(&s_sl[t][c4]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) ddt[j] *= slope[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) db[j] += ddt[j];
                s_acc[1][tid] = db;
                Four<DT, VEC>::store(p.du.p, tok * p.du.stride + bc.c0 + c4, bc.n - c4, du);
                Four<DT, VEC>::store(p.ddt.p, tok * p.ddt.stride + bc.c0 + c4, bc.n - c4, ddt);
                if (!p.dz.p) continue;
                const f32x4 sz = row4(&s_sz[t][c4]), y4 = row4(&s_y[t][c4]);
                float dz[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float z = rz[i].at(j), y = p.d ? fmaf(dw[j], ru[i].at(j), y4[j]) : y4[j];
                    dz[j] = ry[i].at(j) * y * (sz[j] * fmaf(z, 1.f - sz[j], 1.f));
                }
                Four<DT, VEC>::store(p.dz.p, tok * p.dz.stride + bc.c0 + c4, bc.n - c4, dz);
            }
            if (st > 0) fetch(t0 - TS);                   // in flight beside other workgroups' work: no registers for them before
        }
    }
    // the segment's sums (of zero for a slot without tokens)
    if (there) *reinterpret_cast<f32x4*>(p.hseg + slot * states + at) = da;           // read above by this lane alone
    __syncthreads();
    if (tid < 2 * CB) {                                   // the threads of four channels in order
        const int which = tid / CB, c = tid % CB;
        float s = 0.f;
        for (int k = 0; k < K::kGroups; ++k) s += s_acc[which][k * NV + c / 4][c % 4];
        if (c < bc.n) p.dd_part[(slot * 2 + which) * p.channels + bc.c0 + c] = s;
    }
}

// da, dd and ddt_bias (the columns of one row of partial sums after the other): the segments' rows added in a fixed order, 64
// columns a workgroup, the rows in 16 interleaved parts.
__global__ void __launch_bounds__(1024) k_ssm_sum(const SsmParams p, int64_t n_rows) {
    __shared__ float s_part[16][64];
    const int lane = (int)threadIdx.x & 63, sub = (int)threadIdx.x >> 6;
    const int64_t states = (int64_t)p.channels * p.d_state, col = (int64_t)blockIdx.x * 64 + lane, c = col - states;
    const bool in_da = c < 0, in = c < 2 * (int64_t)p.channels;
    const float* part = in_da ? p.hseg + col : p.dd_part + c;
    const int64_t row = in_da ? states : 2 * (int64_t)p.channels;
    float s = 0.f;
    if (in) {
#pragma unroll 4
        for (int64_t i = sub; i < n_rows; i += 16) s += part[i * row];
    }
    s_part[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || !in) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += s_part[k][lane];
    if (in_da) { if (p.da) p.da[col] = s; }
    else if (c < p.channels) { if (p.dd) p.dd[c] = s; }
    else if (p.ddt_bias) p.ddt_bias[c - p.channels] = s;
}

// dB and dC: over the blocks of channels of each group.  Tokens outside the sequences are left as they are.
template <int DT>
__global__ void __launch_bounds__(256) k_ssm_sum_bc(const SsmParams p, int blocks_per_group) {
    const int N = p.d_state, w = 2 * N;
    const int64_t first = span_of(p.runs, 0).start;
    const Span q = span_of(p.runs, p.runs.n_seq - 1);
    const int64_t n = (q.start + q.len - first) * w * p.n_groups;
    for (int64_t x = (int64_t)blockIdx.x * 256 + (int)threadIdx.x; x < n; x += (int64_t)gridDim.x * 256) {
        const int i = (int)(x % w), g = (int)(x / w % p.n_groups);
        const int64_t tok = first + x / w / p.n_groups;
        const float* part = p.bc_part + ((int64_t)g * blocks_per_group * p.runs.n_tokens + tok) * w + i;
        float s = 0.f;
#pragma unroll 8
        for (int b = 0; b < blocks_per_group; ++b) s += part[(int64_t)b * p.runs.n_tokens * w];
        const Rows& to = i < N ? p.db : p.dc;
        Elems<DT, 1> o;
        o.set(&s);
        o.store(to.p, tok * to.stride + g * N + (i < N ? i : i - N));
    }
}

// ------------------------------------------------------------------ launches

#define SQ_LAUNCHED() do { const hipError_t e_ = hipGetLastError(); if (e_ != hipSuccess) return e_; } while (0)

template <int DT, int N, bool VEC>
static hipError_t grad_n(const SsmParams& p, hipStream_t s) {
    using K = Grad<N>;
    const int64_t slots = p.runs.n_seq > 0 ? run_slots(p.runs.n_tokens, p.runs.n_seq, p.runs.log) : 0;      // rows of sums
    const int ends = (int)ssm_blocks(p.channels, p.n_groups, N);
    const bool tokens = p.runs.n_tokens > 0 && p.runs.n_seq > 0;
    if (tokens) {
        k_ssm_ends<DT, N, VEC><<<dim3((unsigned)(slots * ends)), kSsmThreads, 0, s>>>(p, ends);
        SQ_LAUNCHED();
    }
    const int per_group = (p.group_channels + K::CB - 1) / K::CB, blocks = p.n_groups * per_group;
    if (p.runs.n_seq > 0) {
        const hipError_t e = launch_ssm_join(p, 2, s);
        if (e != hipSuccess) return e;
        k_ssm_grad<DT, N, VEC><<<dim3((unsigned)(slots * blocks)), K::kThreads, 0, s>>>(p, blocks);
        SQ_LAUNCHED();
    }
    if (p.da || p.dd || p.ddt_bias) {
        k_ssm_sum<<<dim3((unsigned)(((int64_t)p.channels * (N + 2) + 63) / 64)), 1024, 0, s>>>(p, slots);
        SQ_LAUNCHED();
    }
    if (tokens) {
        int64_t n = (p.runs.n_tokens * 2 * N * p.n_groups + 255) / 256;
        if (n > 8192) n = 8192;
        k_ssm_sum_bc<DT><<<dim3((unsigned)n), 256, 0, s>>>(p, per_group);
        SQ_LAUNCHED();
    }
    return hipSuccess;
}

hipError_t launch_ssm_bwd(const SsmParams& p, bool vec, hipStream_t s) { SQ_SSM_DISPATCH(grad_n, p, s); }
int64_t ssm_grad_blocks(int channels, int n_groups, int d_state) {
    const int per = d_state == 8 ? Grad<8>::CB : d_state == 16 ? Grad<16>::CB : d_state == 32 ? Grad<32>::CB : d_state == 64 ? Grad<64>::CB : Grad<128>::CB;
    const int g = channels / n_groups;
    return int64_t(n_groups) * ((g + per - 1) / per);
}

}  // namespace sq
