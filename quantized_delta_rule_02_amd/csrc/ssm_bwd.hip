// Gradients of the selective state space scan (gfx950).
//
//   dp = dy silu(z),  G_t = C_t dp_t + e_{t+1} G_{t+1} (after the last token: + ds1),  e_t = exp(delta_t a)
//   dC_t = sum_c dp h_t,  dB_t = sum_c G_t delta u,  du = d dp + delta sum_n G B,  ddelta = sum_n G (a e h_{t-1} + u B),
//   ddt = ddelta sigmoid(dt + bias),  da = sum_t G delta e h_{t-1},  dd = sum_t dp u,  dz = dy p silu'(z),  ds0 = e_1 G_1
//
// Nothing of the forward call is kept.  Sequences are cut into segments of 64 tokens.  k_ssm_ends finds, for all of them side by
// side, the state after a segment from a state of zero and the gradient before it from a gradient of zero, in one walk: the
// latter is sum_t (e_1 ... e_t) C_t dp_t.  k_ssm_join turns them into the states before and the gradients after the segments.
// k_ssm_grad walks a segment forward, keeping the state every 8 tokens in LDS, then its tiles of 8 tokens from the last to the
// first: forward with every state and decay in registers, then backward.  Sums over a channel's states are lane exchanges; dB
// and dC are sums over all channels: over the wave's by exchanges that halve the values a lane holds each time, over the
// workgroup's waves in LDS, over the workgroups by k_ssm_sum_bc, all in a fixed order.
#include <hip/hip_runtime.h>

#include "ssm_dev.h"

namespace sq {

constexpr int kSegLog = 6, kSeg = 1 << kSegLog;

template <int DT, int N, bool VEC>
__global__ void __launch_bounds__(kSsmThreads) k_ssm_ends(const SsmParams p, int n_blocks) {
    using L = SsmLane<N>;
    constexpr int TT = 32, CB = L::kBlockCh, NV = CB / 4, kItems = (TT * NV + kSsmThreads - 1) / kSsmThreads;
    constexpr int kBc = (TT * 2 * (N / 4) + kSsmThreads - 1) / kSsmThreads;
    __shared__ float2 s_d[TT][CB];                        // delta, delta u
    __shared__ float s_p[TT][CB];                         // dp
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
    float dsum = 0.f;
    for (int t0 = 0; t0 < r.n; t0 += TT) {
        const int nt = r.n - t0 < TT ? r.n - t0 : TT;
        if (t0) __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int x = i * kSsmThreads + tid, t = x / NV, c = x % NV * 4;
            const int n = x < TT * NV && t < nt ? bc.n - c : 0;
            const int64_t tok = r.tok0 + t0 + t;
            Four<DT, VEC> eu, ed, ey, ez;
            eu.load(p.u.p, tok * p.u.stride + bc.c0 + c, n);
            ed.load(p.dt.p, tok * p.dt.stride + bc.c0 + c, n);
            ey.load(p.dy.p, tok * p.dy.stride + bc.c0 + c, n);
            ez.load(p.z.p, tok * p.z.stride + bc.c0 + c, p.z.p ? n : 0);
            if (x < TT * NV && t < nt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float bias = p.dt_bias && c + j < bc.n ? p.dt_bias[bc.c0 + c + j] : 0.f;
                    float d = ed.at(j) + bias, g = ey.at(j);
                    d = p.softplus ? softplus(d) : d;
                    s_d[t][c + j] = float2{d, d * eu.at(j)};
                    if (p.z.p) g *= ez.at(j) * sigmoid<DT == SQ_DTYPE_F32>(ez.at(j));
                    s_p[t][c + j] = g;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int x = i * kSsmThreads + tid, q = x % (N / 4), t = x / (N / 4) % TT, w = x / (N / 4 * TT);
            const Rows& rows = w ? p.c : p.b;
            Four<DT, VEC> v;
            v.load(rows.p, (r.tok0 + t0 + t) * rows.stride + bc.group * N + 4 * q, w < 2 && t < nt ? 4 : 0);
            f32x4 f;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = v.at(j);
            if (w < 2) s_bc[w][t][q] = f;
        }
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
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
    static constexpr int kWaves = N <= 16 ? 4 : 8, kThreads = kWaves * 64;
    static constexpr int kPer = N / 4, kWaveCh = 64 / kPer, CB = kWaves * kWaveCh;
    static constexpr int TB = 8, kTiles = kSeg / TB;
    static constexpr int NV = CB / 4, kItems = (TB * NV + kThreads - 1) / kThreads;
    static constexpr int kBc = (TB * 2 * kPer + kThreads - 1) / kThreads;
    static constexpr int kFlush = N <= 64 ? 8 : 4;        // tokens whose dB and dC wait in LDS
    static constexpr int kGroups = kThreads / NV;         // threads that share a channel in the sums over tokens
};

// dB and dC of one token over the wave's channels: v[0..3] of dB, v[4..7] of dC, of the lane's four states.  Each exchange joins
// two values' halves, so the sums end up spread over the lanes; `out` is the wave's row of 2 N floats.
template <int PER>
__device__ __forceinline__ void wave_sums(const float* v, float* out) {
    const int lane = (int)threadIdx.x & 63, q = lane % PER;
    float a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = join32(v[j], v[4 + j]);                 // upper half: dC
    float* row = out + (lane >= 32 ? 4 * PER : 0) + 4 * q;
    if constexpr (PER == 32) {
        *reinterpret_cast<f32x4*>(row) = f32x4{a[0], a[1], a[2], a[3]};
        return;
    } else {
        float b0 = join16(a[0], a[2]), b1 = join16(a[1], a[3]);                // odd rows: states 2 and 3
        if constexpr (PER <= 8) { b0 += dpp<kDppRor8>(b0); b1 += dpp<kDppRor8>(b1); }
        if constexpr (PER <= 4) { b0 += dpp<kDppRor4>(b0); b1 += dpp<kDppRor4>(b1); }
        if constexpr (PER <= 2) { b0 += dpp<kDppXor2>(b0); b1 += dpp<kDppXor2>(b1); }
        if ((lane & 15) < PER) *reinterpret_cast<float2*>(row + (lane & 16 ? 2 : 0)) = float2{b0, b1};
    }
}

template <int DT, int N, bool VEC>
__global__ void __launch_bounds__(Grad<N>::kThreads, Grad<N>::kWaves == 4 ? 3 : 2) k_ssm_grad(const SsmParams p, int n_blocks) {
    using K = Grad<N>;
    constexpr int TB = K::TB, CB = K::CB, NV = K::NV, kT = K::kThreads, PER = K::kPer;
    __shared__ float2 s_d[TB][CB];                        // delta, delta u
    __shared__ float s_p[TB][CB];                         // dp
    __shared__ float s_o[3][TB][CB];                      // sum of G B, of a G e h, and p - d u
    __shared__ f32x4 s_bc[2][TB][N / 4];
    __shared__ f32x4 s_h[K::kTiles - 1][kT];              // the lane's states before tiles 1, 2, ...
    __shared__ __attribute__((aligned(16))) float s_w[K::kWaves][K::kFlush][2 * N];
    const int tid = (int)threadIdx.x, wave = tid >> 6, blk = (int)blockIdx.x % n_blocks;
    const int64_t slot = (int)blockIdx.x / n_blocks;
    const RunAt r = run_of_slot(p.runs, slot);
    const SsmBlock bc = block_channels(p, blk, CB);
    const int ch = tid / PER, quarter = tid % PER;
    const bool there = ch < bc.n;
    const int64_t at = ((int64_t)bc.c0 + ch) * N + 4 * quarter, to = slot * p.channels * N + at;
    f32x4 da{0.f, 0.f, 0.f, 0.f};
    float dd[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};      // sums over tokens of the staging thread's channels
    const int c4 = tid % NV * 4;
    if (r.n > 0) {
        f32x4 a2 = load_states(p.a, at, there);
#pragma unroll
        for (int j = 0; j < 4; ++j) a2[j] *= kLog2e;
        const f32x4 h0 = load_states(p.hseg, to, there);
        f32x4 gk = load_states(p.kseg, to, there);
        Four<DT, VEC> ru[K::kItems], rd[K::kItems], ry[K::kItems], rz[K::kItems], rbc[K::kBc];
        auto fetch = [&](int t0, bool back) {
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                const int x = i * kT + tid, t = t0 + x / NV;
                const int n = x < TB * NV && t < r.n ? bc.n - c4 : 0;
                const int64_t tok = r.tok0 + t;
                ru[i].load(p.u.p, tok * p.u.stride + bc.c0 + c4, n);
                rd[i].load(p.dt.p, tok * p.dt.stride + bc.c0 + c4, n);
                if (!back) continue;
                ry[i].load(p.dy.p, tok * p.dy.stride + bc.c0 + c4, n);
                rz[i].load(p.z.p, tok * p.z.stride + bc.c0 + c4, p.z.p ? n : 0);
            }
#pragma unroll
            for (int i = 0; i < K::kBc; ++i) {
                const int x = i * kT + tid, q = x % (N / 4), t = t0 + x / (N / 4) % TB, w = x / (N / 4 * TB);
                const Rows& rows = w ? p.c : p.b;
                rbc[i].load(rows.p, (r.tok0 + t) * rows.stride + bc.group * N + 4 * q, w < (back ? 2 : 1) && t < r.n ? 4 : 0);
            }
        };
        float raw[K::kItems][4];                          // dt + bias
        auto stage = [&](int nt, bool back) {
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                const int x = i * kT + tid, t = x / NV;
                if (x >= TB * NV || t >= nt) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float bias = p.dt_bias && c4 + j < bc.n ? p.dt_bias[bc.c0 + c4 + j] : 0.f;
                    raw[i][j] = rd[i].at(j) + bias;
                    const float d = p.softplus ? softplus(raw[i][j]) : raw[i][j];
                    s_d[t][c4 + j] = float2{d, d * ru[i].at(j)};
                    if (!back) continue;
                    float g = ry[i].at(j);
                    if (p.z.p) g *= rz[i].at(j) * sigmoid<DT == SQ_DTYPE_F32>(rz[i].at(j));
                    s_p[t][c4 + j] = g;
                }
            }
#pragma unroll
            for (int i = 0; i < K::kBc; ++i) {
                const int x = i * kT + tid, q = x % (N / 4), t = x / (N / 4) % TB, w = x / (N / 4 * TB);
                f32x4 f;
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = rbc[i].at(j);
                if (w < (back ? 2 : 1)) s_bc[w][t][q] = f;
            }
        };
        const int n_tiles = (r.n + TB - 1) / TB;
        // forward, the states before every tile but the first kept
        {
            f32x4 h = h0;
            fetch(0, n_tiles == 1);
            for (int tile = 0; tile + 1 < n_tiles; ++tile) {
                stage(TB, false);
                __syncthreads();
                fetch((tile + 1) * TB, tile + 2 == n_tiles);
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const float2 d = s_d[t][ch];
                    const f32x4 b = s_bc[0][t][quarter];
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = fmaf(__builtin_amdgcn_exp2f(d.x * a2[j]), h[j], d.y * b[j]);
                }
                s_h[tile][tid] = h;
                __syncthreads();
            }
        }
        for (int tile = n_tiles - 1; tile >= 0; --tile) {
            const int t0 = tile * TB, nt = r.n - t0 < TB ? r.n - t0 : TB;
            stage(nt, true);
            Four<DT, VEC> cu[K::kItems], cy[K::kItems], cz[K::kItems];
            float craw[K::kItems][4];
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                cu[i] = ru[i];
                cy[i] = ry[i];
                cz[i] = rz[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) craw[i][j] = raw[i][j];
            }
            __syncthreads();
            if (tile > 0) fetch(t0 - TB, true);
            const f32x4 hs = tile > 0 ? s_h[tile > 0 ? tile - 1 : 0][tid] : h0;
            f32x4 h[TB], e[TB];
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                if (t < nt) {
                    const float2 d = s_d[t][ch];
                    const f32x4 b = s_bc[0][t][quarter], prev = t ? h[t ? t - 1 : 0] : hs;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e[t][j] = __builtin_amdgcn_exp2f(d.x * a2[j]);
                        h[t][j] = fmaf(e[t][j], prev[j], d.y * b[j]);
                    }
                    if (p.z.p) {
                        const f32x4 c = s_bc[1][t][quarter];
                        float y = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) y = fmaf(h[t][j], c[j], y);
                        y = channel_sum<PER>(y);
                        if (quarter == 0) s_o[2][t][ch] = y;
                    }
                }
            }
#pragma unroll
            for (int t = TB - 1; t >= 0; --t) {
                if (t < nt) {
                    const float2 d = s_d[t][ch];
                    const float dp = s_p[t][ch];
                    const f32x4 b = s_bc[0][t][quarter], c = s_bc[1][t][quarter], prev = t ? h[t ? t - 1 : 0] : hs;
                    float v[8], gb = 0.f, ga = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float g = fmaf(c[j], dp, gk[j]), through = g * (e[t][j] * prev[j]);
                        gb = fmaf(g, b[j], gb);
                        ga = fmaf(a2[j], through, ga);
                        da[j] = fmaf(through, d.x, da[j]);
                        v[j] = g * d.y;
                        v[4 + j] = dp * h[t][j];
                        gk[j] = g * e[t][j];
                    }
                    if (!there) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = 0.f;
                    }
                    wave_sums<PER>(v, s_w[wave][t % K::kFlush]);
                    gb = channel_sum<PER>(gb);
                    ga = channel_sum<PER>(ga);
                    if (quarter == 0) {
                        s_o[0][t][ch] = gb;
                        s_o[1][t][ch] = ga;
                    }
                }
                if (t % K::kFlush == 0) {
                    __syncthreads();
                    // over the waves, and out
                    const int most = nt - t < K::kFlush ? nt - t : K::kFlush;
                    for (int x = tid; x < most * 2 * N; x += kT) {
                        const int tt = x / (2 * N), i = x % (2 * N);
                        float s = s_w[0][tt][i];
#pragma unroll
                        for (int w = 1; w < K::kWaves; ++w) s += s_w[w][tt][i];
                        p.bc_part[((int64_t)blk * p.runs.n_tokens + r.tok0 + t0 + t + tt) * (2 * N) + i] = s;
                    }
                    if (t > 0) __syncthreads();
                }
            }
            // the rows of this tile: du, ddt, dz
#pragma unroll
            for (int i = 0; i < K::kItems; ++i) {
                const int x = i * kT + tid, t = x / NV;
                if (x >= TB * NV || t >= nt) continue;
                const int64_t tok = r.tok0 + t0 + t;
                float du[4], ddt[4], dz[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float dw = p.d && c4 + j < bc.n ? p.d[bc.c0 + c4 + j] : 0.f;
                    const float u = cu[i].at(j), g = s_p[t][c4 + j], gb = s_o[0][t][c4 + j], delta = s_d[t][c4 + j].x;
                    du[j] = delta * gb;
                    if (p.d) du[j] = fmaf(dw, g, du[j]);
                    ddt[j] = fmaf(s_o[1][t][c4 + j], 0.69314718056f, u * gb);
                    if (p.softplus) ddt[j] *= sigmoid<true>(craw[i][j]);
                    dd[j] = fmaf(g, u, dd[j]);
                    db[j] += ddt[j];
                    if (p.z.p) {
                        const float z = cz[i].at(j), sg = sigmoid<DT == SQ_DTYPE_F32>(z);
                        const float y = p.d ? fmaf(dw, u, s_o[2][t][c4 + j]) : s_o[2][t][c4 + j];
                        dz[j] = cy[i].at(j) * y * (sg * fmaf(z, 1.f - sg, 1.f));
                    }
                }
                Four<DT, VEC>::store(p.du.p, tok * p.du.stride + bc.c0 + c4, bc.n - c4, du);
                Four<DT, VEC>::store(p.ddt.p, tok * p.ddt.stride + bc.c0 + c4, bc.n - c4, ddt);
                if (p.dz.p) Four<DT, VEC>::store(p.dz.p, tok * p.dz.stride + bc.c0 + c4, bc.n - c4, dz);
            }
            __syncthreads();
        }
    }
    // the segment's sums (of zero for a slot without tokens)
    if (there) *reinterpret_cast<f32x4*>(p.da_part + to) = da;
    float* red = &s_w[0][0][0];                           // [8][threads that share channels][NV]: in pieces of one column
    static_assert(K::kWaves * K::kFlush * 2 * N >= kT, "room for one value a thread");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        __syncthreads();
        red[tid] = j < 4 ? dd[j & 3] : db[j & 3];
        __syncthreads();
        if (tid < NV && c4 + (j & 3) < bc.n) {
            float s = 0.f;
            for (int k = 0; k < K::kGroups; ++k) s += red[k * NV + tid];
            p.dd_part[(slot * 2 + (j >> 2)) * p.channels + bc.c0 + c4 + (j & 3)] = s;
        }
    }
}

// da, dd and ddt_bias: the segments' rows added in a fixed order, 64 columns a workgroup, the rows in 16 interleaved parts.
__global__ void __launch_bounds__(1024) k_ssm_sum(const float* part, int64_t n_rows, int64_t row, int64_t n_cols, float* out) {
    __shared__ float s_part[16][64];
    const int lane = (int)threadIdx.x & 63, sub = (int)threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (col < n_cols)
        for (int64_t i = sub; i < n_rows; i += 16) s += part[i * row + col];
    s_part[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || col >= n_cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += s_part[k][lane];
    out[col] = s;
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
    const int64_t states = (int64_t)p.channels * N;
    if (p.da) k_ssm_sum<<<dim3((unsigned)((states + 63) / 64)), 1024, 0, s>>>(p.da_part, slots, states, states, p.da);
    SQ_LAUNCHED();
    const dim3 cols((unsigned)((p.channels + 63) / 64));
    if (p.dd) k_ssm_sum<<<cols, 1024, 0, s>>>(p.dd_part, slots, 2 * (int64_t)p.channels, p.channels, p.dd);
    SQ_LAUNCHED();
    if (p.ddt_bias) k_ssm_sum<<<cols, 1024, 0, s>>>(p.dd_part + p.channels, slots, 2 * (int64_t)p.channels, p.channels, p.ddt_bias);
    SQ_LAUNCHED();
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
