// Norms before and after a block, with the residual add, channel scale and gate fused (gfx950).
//
//   in :  h = x + s c r;            n = f w h i(h)
//   out:  o = x + s c (w y i(y) act(z))
//   i(a) = 1 / sqrt(sum(a^2) / div + eps), div = d (RMS) or 1 (unit L2 norm)
//
// and their gradients, from  d(a i(a)): da = i (g - a i^2 (g . a) / div)  for an incoming g.
//
// All four are bound by memory: every row is read once into registers (both sums of a backward pass
// are taken from there) and written once.  A row of d elements belongs to TPR threads with K vectors of
// V elements each, so that one workgroup of 256 threads holds 256 / TPR rows: head rows (d <= 512 with 16-byte
// accesses) live in part of a wave and need no LDS, longer ones take the whole workgroup.  Rows above 2048 elements that cannot
// be read 16 bytes at a time take 1024 threads, the widest of them a kernel that reads them twice (k_norm_wide).
// dweight and dchan_scale are sums over all rows: each thread keeps its columns' sums in registers over the
// workgroup's rows, the workgroup adds its row groups in LDS and writes one partial row, and a second
// kernel adds the partial rows in a fixed order (no atomics, so results do not depend on the schedule).
#include <hip/hip_runtime.h>

#include "norm.h"
#include "vec.h"

namespace sq {

constexpr int norm_threads(int tpr) { return tpr > kNormThreads ? tpr : kNormThreads; }    // of a workgroup

struct Sum2 { float a, b; };

// Sums over the TPR threads of a row; every thread gets them.
template <int TPR>
__device__ __forceinline__ Sum2 row_sum(Sum2 v, float* lds) {
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int m = 1; m < W; m <<= 1) {
        v.a += __shfl_xor(v.a, m);
        v.b += __shfl_xor(v.b, m);
    }
    if constexpr (TPR > 64) {
        const int wave = (int)threadIdx.x >> 6;
        __syncthreads();                       // the previous row's sums have been read
        if ((threadIdx.x & 63) == 0) { lds[2 * wave] = v.a; lds[2 * wave + 1] = v.b; }
        __syncthreads();
        v = Sum2{0.f, 0.f};
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) { v.a += lds[2 * w]; v.b += lds[2 * w + 1]; }
    }
    return v;
}

// exp(-z) from the hardware's 2^x: the rounding of z log2(e) is put back as a factor, so that its error does not grow with |z|.
// From a = 128 on 2^a is infinity, and infinity times a remainder of zero or below would be NaN; far below -126 it is zero,
// and the remainder of an infinite a is NaN: there 2^a stays as it is.
__device__ __forceinline__ float exp_neg(float z) {
    constexpr float l2e = 1.44269504089f, ln2 = 0.69314718056f;
    const float a = -z * l2e, lo = fmaf(-z, l2e, -a), e = __builtin_amdgcn_exp2f(a);
    return a < 128.f && a > -200.f ? fmaf(e, lo * ln2, e) : e;
}
// The reciprocal is the hardware's, off by at most one unit in the last place of float32 (2^-23 of the gate): an output in
// float32 carries some five roundings of that size, one in 16 bits is rounded by 2^-11 or more.
__device__ __forceinline__ void act_of(int act, float z, float& g, float& dg) {
    const float e = exp_neg(z), s = __builtin_amdgcn_rcpf(1.f + e);
    if (act == SQ_ACT_SILU) {
        g = z * s;
        dg = s * fmaf(z, 1.f - s, 1.f);
    } else {                                   // SQ_ACT_SIGMOID
        // 1 - s = sigmoid(-z): the difference loses all its digits as s nears 1, e s loses none there
        g = s;
        dg = s * (z > 0.f ? e * s : 1.f - s);
    }
}

// A row index of a launch fits 32 bits (checked by the caller): the split into outer and inner is a 32-bit division.
__device__ __forceinline__ int64_t row_at(const NormRows& a, uint32_t outer, uint32_t inner, int d) {
    return (int64_t)outer * a.stride + (int64_t)(inner * (uint32_t)d);
}

// Elements as loaded: what follows a load waits for it, so all loads of a row come before the first conversion.
template <int V>
struct RawV {
    u32x4v a, b;
    __device__ __forceinline__ void load(const NormRows& r, int dt, int64_t i) {
        if constexpr (V == 8) {
            if (dt == SQ_DTYPE_F32) {
                const u32x4v* s = reinterpret_cast<const u32x4v*>(static_cast<const float*>(r.p) + i);
                a = s[0];
                b = s[1];
            } else {
                a = *reinterpret_cast<const u32x4v*>(static_cast<const uint16_t*>(r.p) + i);
            }
        } else {
            a[0] = dt == SQ_DTYPE_F32 ? static_cast<const uint32_t*>(r.p)[i] : static_cast<const uint16_t*>(r.p)[i];
        }
    }
    __device__ __forceinline__ void get(int dt, float* x) const {
        if constexpr (V == 8) {
            if (dt == SQ_DTYPE_F32) {
#pragma unroll
                for (int j = 0; j < 4; ++j) { x[j] = __uint_as_float(a[j]); x[4 + j] = __uint_as_float(b[j]); }
            } else if (dt == SQ_DTYPE_BF16) {
#pragma unroll
                for (int j = 0; j < 4; ++j) { x[2 * j] = bf16_lo(a[j]); x[2 * j + 1] = bf16_hi(a[j]); }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) { x[2 * j] = f16_val(a[j] & 0xffffu); x[2 * j + 1] = f16_val(a[j] >> 16); }
            }
        } else {
            x[0] = dt == SQ_DTYPE_F32 ? __uint_as_float(a[0]) : dt == SQ_DTYPE_BF16 ? bf16_lo(a[0]) : f16_val(a[0]);
        }
    }
};

// U rows at a time: their loads are in flight together.
// EXTRA (gradients of the first norm): dh or r is there.
template <int OP, int V, int TPR, int K, int U, bool EXTRA>
__global__ void __launch_bounds__(norm_threads(TPR), V == 8 && K == 1 ? 4 : 1) k_norm(const NormParams p) {
    constexpr int NT = norm_threads(TPR), RPB = NT / TPR;
    constexpr bool kBwd = OP == kNormInBwd || OP == kNormOutBwd;
    constexpr bool kIn = OP == kNormIn || OP == kNormInBwd;
    constexpr bool kAll = K <= 2;              // few enough registers to load every array at once
    __shared__ float s_red[2 * NT / 64];
    __shared__ float s_col[kBwd && RPB > 1 ? NT * V * K : 1];
    const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR;
    const int d = p.d;
    // first: the row the norm is of, its addend or gate, the incoming gradient; second: what only the result needs
    const NormRows& ra = OP == kNormIn ? p.x : OP == kNormInBwd ? p.h : p.y;
    const NormRows& rt = OP == kNormIn ? p.r : p.z;
    const NormRows& rg = OP == kNormInBwd ? p.dn : p.d_o;
    const NormRows& re = OP == kNormInBwd ? p.dh : p.x;
    const bool has_t = OP == kNormIn ? p.has_r : kIn ? false : p.has_z;
    const bool has_e = OP == kNormInBwd ? EXTRA && p.has_dh : OP == kNormOut ? p.has_x : false;
    const bool has_r = EXTRA && p.has_r;
    const int dt_t = OP == kNormIn ? p.dtype : p.dtype_out, dt_e = OP == kNormInBwd ? p.dtype : p.dtype_out;
    RawV<V> xa[U][K], xt[U][K], xg[kBwd ? U : 1][K], xe[U][K], xr[OP == kNormInBwd ? U : 1][K];
    int col[K];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        col[k] = (k * TPR + lane) * V;
        in[k] = col[k] < d;
    }
    uint32_t outer[U], inner[U];
    bool live[U];
    auto load_second = [&](int u, int k) {
        if (has_e) xe[u][k].load(re, dt_e, row_at(re, outer[u], inner[u], d) + col[k]);
        if constexpr (OP == kNormInBwd) {
            if (has_r) xr[u][k].load(p.r, p.dtype, row_at(p.r, outer[u], inner[u], d) + col[k]);
        }
    };
    auto load_rows = [&](int64_t row0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * RPB + sub;
            live[u] = row < p.n_rows;
            outer[u] = (uint32_t)row / (uint32_t)p.n_inner;
            inner[u] = (uint32_t)row % (uint32_t)p.n_inner;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!(live[u] && in[k])) continue;
                xa[u][k].load(ra, p.dtype, row_at(ra, outer[u], inner[u], d) + col[k]);
                if (has_t) xt[u][k].load(rt, dt_t, row_at(rt, outer[u], inner[u], d) + col[k]);
                if constexpr (kBwd) xg[kBwd ? u : 0][k].load(rg, p.dtype_out, row_at(rg, outer[u], inner[u], d) + col[k]);
                if constexpr (kAll) load_second(u, k);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB * U;
    int64_t row0 = (int64_t)blockIdx.x * RPB * U;
    if (row0 < p.n_rows) load_rows(row0);
    float w[K][V], c[K][V], sw[K][V], sc[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[k][j] = (p.weight && in[k]) ? p.weight[col[k] + j] : 1.f;
            c[k][j] = (p.chan_scale && in[k]) ? p.chan_scale[col[k] + j] * p.res_scale : p.res_scale;
            sw[k][j] = sc[k][j] = 0.f;
        }
    // every thread of a workgroup makes the same number of rounds: the row sums hold barriers
    for (; row0 < p.n_rows; row0 += step) {
        float a[U][K][V], g[U][K][V], t[U][K][V], e[U][K][V], q[U][K][V];   // t: act(z), q: its derivative (or r)
        Sum2 s[U];
        uint32_t o_[U], i_[U];
        bool lv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = Sum2{0.f, 0.f};
            o_[u] = outer[u];
            i_[u] = inner[u];
            lv[u] = live[u];
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    a[u][k][j] = g[u][k][j] = e[u][k][j] = q[u][k][j] = 0.f;
                    t[u][k][j] = kIn ? 0.f : 1.f;
                }
                if (!(lv[u] && in[k])) continue;
                xa[u][k].get(p.dtype, a[u][k]);
                if (has_t) {
                    xt[u][k].get(dt_t, t[u][k]);
                    if constexpr (!kIn) {
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float z = t[u][k][j];
                            act_of(p.act, z, t[u][k][j], q[u][k][j]);
                        }
                    }
                }
                if constexpr (kBwd) xg[kBwd ? u : 0][k].get(p.dtype_out, g[u][k]);
                if constexpr (kAll) {
                    if (has_e) xe[u][k].get(dt_e, e[u][k]);
                    if constexpr (OP == kNormInBwd) {
                        if (has_r) xr[OP == kNormInBwd ? u : 0][k].get(p.dtype, q[u][k]);
                    }
                }
            }
        }
        if constexpr (kAll) {
            if (row0 + step < p.n_rows) load_rows(row0 + step);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if constexpr (OP == kNormIn) a[u][k][j] = has_t ? fmaf(c[k][j], t[u][k][j], a[u][k][j]) : a[u][k][j];
                    s[u].a = fmaf(a[u][k][j], a[u][k][j], s[u].a);
                    if constexpr (OP == kNormInBwd) s[u].b = fmaf(g[u][k][j] * w[k][j], a[u][k][j], s[u].b);
                    if constexpr (OP == kNormOutBwd) s[u].b = fmaf(g[u][k][j] * c[k][j] * w[k][j] * t[u][k][j], a[u][k][j], s[u].b);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = row_sum<TPR>(s[u], s_red);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float inv = 1.f / sqrtf(fmaf(s[u].a, p.inv_div, p.eps));
            [[maybe_unused]] float back = 0.f;
            if constexpr (OP == kNormInBwd) back = s[u].b * p.out_scale * inv * inv * p.inv_div;
            if constexpr (OP == kNormOutBwd) back = s[u].b * inv * inv * p.inv_div;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!(lv[u] && in[k])) continue;
                if constexpr (!kAll) {
                    load_second(u, k);
                    if (has_e) xe[u][k].get(dt_e, e[u][k]);
                    if constexpr (OP == kNormInBwd) {
                        if (has_r) xr[OP == kNormInBwd ? u : 0][k].get(p.dtype, q[u][k]);
                    }
                }
                auto put = [&](const NormRows& r, int dt, const float* v) { storev<V>(r.p, dt, row_at(r, o_[u], i_[u], d) + col[k], v); };
                float o[V], e2[V];
                if constexpr (OP == kNormIn) {
                    if (p.write_h) put(p.h, p.dtype, a[u][k]);
                    const float f = inv * p.out_scale;
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = a[u][k][j] * f * w[k][j];
                    put(p.n, p.dtype_out, o);
                } else if constexpr (OP == kNormInBwd) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float gf = g[u][k][j] * p.out_scale;
                        o[j] = fmaf(inv, gf * w[k][j] - a[u][k][j] * back, e[u][k][j]);
                        sw[k][j] = fmaf(gf * inv, a[u][k][j], sw[k][j]);
                        if constexpr (EXTRA) sc[k][j] = fmaf(o[j] * p.res_scale, q[u][k][j], sc[k][j]);   // q: r, or 0 where nobody asks
                        e2[j] = o[j] * c[k][j];
                    }
                    if (p.write_dr) put(p.dr, p.dtype, e2);
                    put(p.dx, p.dtype, o);
                } else if constexpr (OP == kNormOut) {
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = fmaf(a[u][k][j] * inv * w[k][j] * t[u][k][j], c[k][j], e[u][k][j]);
                    put(p.o, p.dtype_out, o);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float yh = a[u][k][j] * inv, gc = g[u][k][j] * c[k][j];
                        o[j] = inv * (gc * w[k][j] * t[u][k][j] - a[u][k][j] * back);
                        e2[j] = gc * w[k][j] * yh * q[u][k][j];
                        sw[k][j] = fmaf(gc * t[u][k][j], yh, sw[k][j]);
                        sc[k][j] = fmaf(g[u][k][j] * p.res_scale * t[u][k][j], w[k][j] * yh, sc[k][j]);
                    }
                    if (p.write_dz) put(p.dz, p.dtype_out, e2);
                    put(p.dy, p.dtype, o);
                }
            }
        }
        if constexpr (!kAll) {
            if (row0 + step < p.n_rows) load_rows(row0 + step);
        }
    }
    if constexpr (kBwd) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (!(which ? p.dchan_scale : p.dweight)) continue;
            float(&v)[K][V] = which ? sc : sw;
            if constexpr (RPB > 1) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) s_col[sub * (TPR * V * K) + (k * TPR + lane) * V + j] = v[k][j];
                __syncthreads();
            }
            float* out = p.part + ((size_t)which * p.n_blocks + blockIdx.x) * d;
            if constexpr (RPB > 1) {
                for (int i = (int)threadIdx.x; i < d; i += NT) {
                    float t = 0.f;
                    for (int r = 0; r < RPB; ++r) t += s_col[r * (TPR * V * K) + i];
                    out[i] = t;
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (in[k]) {
#pragma unroll
                        for (int j = 0; j < V; ++j) out[col[k] + j] = v[k][j];
                    }
            }
        }
    }
}

// Rows above 4096 elements that are read one at a time: 1024 threads take a row in groups of four elements each, once for its
// sums and once more for its results (from the caches: a row is 64 KiB at most), so that no array of a row is held and only the
// column sums stay in registers.
constexpr int kWideThreads = 1024;
template <int OP>
__global__ void __launch_bounds__(kWideThreads) k_norm_wide(const NormParams p) {
    constexpr int NT = kWideThreads, G = 4, NK = kNormMaxD / NT;
    constexpr bool kBwd = OP == kNormInBwd || OP == kNormOutBwd;
    constexpr bool kIn = OP == kNormIn || OP == kNormInBwd;
    __shared__ float s_red[2 * NT / 64];
    const int lane = (int)threadIdx.x, d = p.d;
    const NormRows& ra = OP == kNormIn ? p.x : OP == kNormInBwd ? p.h : p.y;
    const NormRows& rt = OP == kNormIn ? p.r : p.z;
    const NormRows& rg = OP == kNormInBwd ? p.dn : p.d_o;
    const NormRows& re = OP == kNormInBwd ? p.dh : p.x;
    const bool has_t = OP == kNormIn ? p.has_r : kIn ? false : p.has_z;
    const bool has_e = OP == kNormInBwd ? p.has_dh : OP == kNormOut ? p.has_x : false;
    const int dt_t = OP == kNormIn ? p.dtype : p.dtype_out, dt_e = OP == kNormInBwd ? p.dtype : p.dtype_out;
    float sw[kBwd ? NK : 1], sc[kBwd ? NK : 1];
#pragma unroll
    for (int k = 0; k < (kBwd ? NK : 1); ++k) sw[k] = sc[k] = 0.f;
    for (int64_t row = blockIdx.x; row < p.n_rows; row += gridDim.x) {
        const uint32_t outer = (uint32_t)row / (uint32_t)p.n_inner, inner = (uint32_t)row % (uint32_t)p.n_inner;
        RawV<1> xa[G], xt[G], xg[G], xe[G], xr[G];
        float w[G], c[G];
        auto col = [&](int k, int u) { return (k + u) * NT + lane; };
        auto load = [&](const NormRows& r, int dt, RawV<1>& x, int i) { x.load(r, dt, row_at(r, outer, inner, d) + i); };
        auto fetch = [&](int k) {
#pragma unroll
            for (int u = 0; u < G; ++u) {
                const int i = col(k, u);
                if (i >= d) continue;
                load(ra, p.dtype, xa[u], i);
                if (has_t) load(rt, dt_t, xt[u], i);
                if constexpr (kBwd) load(rg, p.dtype_out, xg[u], i);
                w[u] = p.weight ? p.weight[i] : 1.f;
                c[u] = p.chan_scale ? p.chan_scale[i] * p.res_scale : p.res_scale;
            }
        };
        // the row's element (norm_in: h), the gate and its derivative, the incoming gradient
        auto element = [&](int u, float& a, float& t, float& q, float& g) {
            xa[u].get(p.dtype, &a);
            t = 1.f;
            q = g = 0.f;
            if (has_t) {
                xt[u].get(dt_t, &t);
                if constexpr (kIn) a = fmaf(c[u], t, a);
                else act_of(p.act, t, t, q);
            }
            if constexpr (kBwd) xg[u].get(p.dtype_out, &g);
        };
        Sum2 s{0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k * NT < d; k += G) {
            fetch(k);
#pragma unroll
            for (int u = 0; u < G; ++u) {
                if (col(k, u) >= d) continue;
                float a, t, q, g;
                element(u, a, t, q, g);
                s.a = fmaf(a, a, s.a);
                if constexpr (OP == kNormInBwd) s.b = fmaf(g * w[u], a, s.b);
                if constexpr (OP == kNormOutBwd) s.b = fmaf(g * c[u] * w[u] * t, a, s.b);
            }
        }
        s = row_sum<NT>(s, s_red);
        const float inv = 1.f / sqrtf(fmaf(s.a, p.inv_div, p.eps));
        const float back = s.b * (OP == kNormInBwd ? p.out_scale : 1.f) * inv * inv * p.inv_div;
#pragma unroll(kBwd ? NK / G : 1)
        for (int k = 0; k < NK; k += G) {
            if (k * NT < d) {
                fetch(k);
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    if (col(k, u) >= d) continue;
                    if (has_e) load(re, dt_e, xe[u], col(k, u));
                    if constexpr (OP == kNormInBwd) {
                        if (p.has_r) load(p.r, p.dtype, xr[u], col(k, u));
                    }
                }
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    const int i = col(k, u), n = kBwd ? k + u : 0;
                    if (i >= d) continue;
                    float a, t, q, g, e = 0.f, r = 0.f;
                    element(u, a, t, q, g);
                    if (has_e) xe[u].get(dt_e, &e);
                    if constexpr (OP == kNormInBwd) {
                        if (p.has_r) xr[u].get(p.dtype, &r);
                    }
                    auto put = [&](const NormRows& to, int dt, float v) { store1(to.p, dt, row_at(to, outer, inner, d) + i, v); };
                    if constexpr (OP == kNormIn) {
                        if (p.write_h) put(p.h, p.dtype, a);
                        put(p.n, p.dtype_out, a * (inv * p.out_scale) * w[u]);
                    } else if constexpr (OP == kNormInBwd) {
                        const float gf = g * p.out_scale, o = fmaf(inv, gf * w[u] - a * back, e);
                        sw[n] = fmaf(gf * inv, a, sw[n]);
                        sc[n] = fmaf(o * p.res_scale, r, sc[n]);
                        if (p.write_dr) put(p.dr, p.dtype, o * c[u]);
                        put(p.dx, p.dtype, o);
                    } else if constexpr (OP == kNormOut) {
                        put(p.o, p.dtype_out, fmaf(a * inv * w[u] * t, c[u], e));
                    } else {
                        const float yh = a * inv, gc = g * c[u];
                        sw[n] = fmaf(gc * t, yh, sw[n]);
                        sc[n] = fmaf(g * p.res_scale * t, w[u] * yh, sc[n]);
                        if (p.write_dz) put(p.dz, p.dtype_out, gc * w[u] * yh * q);
                        put(p.dy, p.dtype, inv * (gc * w[u] * t - a * back));
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);           // one group's loads at a time
        }
    }
    if constexpr (kBwd) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (!(which ? p.dchan_scale : p.dweight)) continue;
            float* out = p.part + ((size_t)which * p.n_blocks + blockIdx.x) * d;
#pragma unroll
            for (int k = 0; k < NK; ++k)
                if (k * NT + lane < d) out[k * NT + lane] = which ? sc[k] : sw[k];
        }
    }
}

// Adds the partial rows: 16 columns x 64 row groups per workgroup, the groups in LDS, in a fixed order (with 16 groups a sum
// of 1024 rows of 128 columns took 20 us).
constexpr int kSumGroups = 64;
__global__ void __launch_bounds__(16 * kSumGroups) k_norm_sum(const NormParams p) {
    __shared__ float s[kSumGroups][17];
    const int ci = (int)threadIdx.x & 15, g = (int)threadIdx.x >> 4;
    const int which = (int)blockIdx.y, col = (int)blockIdx.x * 16 + ci;
    float* out = which ? p.dchan_scale : p.dweight;
    if (!out) return;
    const float* in = p.part + (size_t)which * p.n_blocks * p.d;
    float t = 0.f;
    if (col < p.d) {
#pragma unroll 4
        for (int b = g; b < p.n_blocks; b += kSumGroups) t += in[(size_t)b * p.d + col];
    }
    s[g][ci] = t;
    __syncthreads();
    if (g < 4) {
        for (int r = g + 4; r < kSumGroups; r += 4) t += s[r][ci];
        s[g][ci] = t;
    }
    __syncthreads();
    if (g == 0 && col < p.d) out[col] = s[0][ci] + s[1][ci] + s[2][ci] + s[3][ci];
}

// K = 0: k_norm_wide.
template <int OP, int V, int TPR, int K>
static hipError_t launch_t(const NormParams& p0, hipStream_t s) {
    constexpr int RPB = norm_threads(TPR) / TPR;
    constexpr int U = V == 8 && K == 1 && TPR < 256 && OP == kNormIn ? 2 : 1;
    constexpr bool kBwd = OP == kNormInBwd || OP == kNormOutBwd;
    NormParams p = p0;
    int64_t blocks = (p.n_rows + RPB * U - 1) / (RPB * U);
    if (kBwd) {
        const int64_t cap = norm_bwd_blocks(p.n_rows, p.d);
        if (blocks > cap) blocks = cap;
    } else if (blocks > 8192) {
        blocks = 8192;                         // the weights are loaded once per workgroup and kept over its rows
    }
    p.n_blocks = (int32_t)blocks;
    const dim3 grid((unsigned)blocks), blk(norm_threads(TPR));
    if (blocks > 0) {
        constexpr bool kChoice = OP == kNormInBwd;
        if constexpr (K == 0) k_norm_wide<OP><<<grid, blk, 0, s>>>(p);
        else if (kChoice && !p.has_dh && !p.has_r) k_norm<OP, V, TPR, K, U, !kChoice><<<grid, blk, 0, s>>>(p);
        else k_norm<OP, V, TPR, K, U, true><<<grid, blk, 0, s>>>(p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !kBwd || !(p.dweight || p.dchan_scale)) return e;
    k_norm_sum<<<dim3((unsigned)((p.d + 15) / 16), 2), dim3(16 * kSumGroups), 0, s>>>(p);
    return hipGetLastError();
}

template <int OP>
static hipError_t launch_op(bool vec, const NormParams& p, hipStream_t s) {
    const int d = p.d;
    if (vec) {
        const int n = d / 8;                   // 16-byte vectors of a row
        if (n <= 2) return launch_t<OP, 8, 2, 1>(p, s);
        if (n <= 8) return launch_t<OP, 8, 8, 1>(p, s);
        if (n <= 16) return launch_t<OP, 8, 16, 1>(p, s);
        if (n <= 32) return launch_t<OP, 8, 32, 1>(p, s);
        if (n <= 64) return launch_t<OP, 8, 64, 1>(p, s);
        if (n <= 256) return launch_t<OP, 8, 256, 1>(p, s);
        if (n <= 512) return launch_t<OP, 8, 256, 2>(p, s);
        if (n <= 1024) return launch_t<OP, 8, 256, 4>(p, s);
        return launch_t<OP, 8, 256, 8>(p, s);
    }
    if (d <= 16) return launch_t<OP, 1, 16, 1>(p, s);
    if (d <= 64) return launch_t<OP, 1, 64, 1>(p, s);
    if (d <= 256) return launch_t<OP, 1, 64, 4>(p, s);
    if (d <= 2048) return launch_t<OP, 1, 256, 8>(p, s);
    // Wider rows take 1024 threads, with at most 8 elements of every array in a thread's registers (the gradients of the second
    // norm: 4), or k_norm_wide.  With 256 threads of 64 elements they spilled up to 5549 registers.  bfloat16, 16 million
    // elements, no 16-byte accesses, us now / with 256 threads / plain torch:
    //   first norm, residual: 2049: 76 / 504 / 215   4095: 56 / 327 / 216   8191: 66 / 220 / 216   16383: 73 / 344 / 212
    //   its gradients:        2049: 136 / 1256 / 844  4095: 105 / 1017 / 769  8191: 94 / 976 / 732  16383: 226 / 948 / 724
    //   second norm:          2049: 76 / 568 / 370   4095: 59 / 392 / 371   8191: 74 / 292 / 368   16383: 99 / 376 / 367
    //   its gradients:        2049: 128 / 2501 / 1325  4095: 98 / 1823 / 1254  8191: 211 / 1453 / 1211  16383: 207 / 1658 / 1202
    // k_norm_wide from 4097 elements on: 92, 249, 126, 234 us at 4097, where 8 held elements take 86, 118, 95 and (spilled) 367.
    if (d <= 4096) return launch_t<OP, 1, 1024, 4>(p, s);
    if constexpr (OP != kNormOutBwd) {
        if (d <= 8192) return launch_t<OP, 1, 1024, 8>(p, s);
    }
    return launch_t<OP, 1, kWideThreads, 0>(p, s);
}

hipError_t launch_norm(int op, bool vec, const NormParams& p, hipStream_t s) {
    switch (op) {
        case kNormIn: return launch_op<kNormIn>(vec, p, s);
        case kNormInBwd: return launch_op<kNormInBwd>(vec, p, s);
        case kNormOut: return launch_op<kNormOut>(vec, p, s);
        case kNormOutBwd: return launch_op<kNormOutBwd>(vec, p, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace sq
