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
// accesses) live in part of a wave and need no LDS, longer ones take the whole workgroup.
// dweight and dchan_scale are sums over all rows: each thread keeps its columns' sums in registers over the
// workgroup's rows, the workgroup adds its row groups in LDS and writes one partial row, and a second
// kernel adds the partial rows in a fixed order (no atomics, so results do not depend on the schedule).
#include <hip/hip_runtime.h>

#include "norm.h"
#include "vec.h"

namespace sq {

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
        v.a = lds[0] + lds[2] + lds[4] + lds[6];
        v.b = lds[1] + lds[3] + lds[5] + lds[7];
    }
    return v;
}

__device__ __forceinline__ void act_of(int act, float z, float& g, float& dg) {
    if (act == SQ_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        g = z * s;
        dg = s * (1.f + z * (1.f - s));
    } else {                                   // SQ_ACT_SIGMOID
        g = 1.f / (1.f + expf(-z));
        dg = g * (1.f - g);
    }
}

// A row index of a launch fits 32 bits (checked by the caller): the split into outer and inner is a 32-bit division.
__device__ __forceinline__ int64_t row_at(const NormRows& a, uint32_t outer, uint32_t inner, int d) {
    return (int64_t)outer * a.stride + (int64_t)(inner * (uint32_t)d);
}

template <int OP, int V, int TPR, int K>
__global__ void __launch_bounds__(kNormThreads) k_norm(const NormParams p) {
    constexpr int RPB = kNormThreads / TPR;
    constexpr bool kBwd = OP == kNormInBwd || OP == kNormOutBwd;
    __shared__ float s_red[8];
    __shared__ float s_col[kBwd && RPB > 1 ? kNormThreads * V * K : 1];
    const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR;
    const int d = p.d;
    int col[K];
    bool in[K];
    float w[K][V], c[K][V], sw[K][V], sc[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        col[k] = (k * TPR + lane) * V;
        in[k] = col[k] < d;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[k][j] = (p.weight && in[k]) ? p.weight[col[k] + j] : 1.f;
            c[k][j] = (p.chan_scale && in[k]) ? p.chan_scale[col[k] + j] * p.res_scale : p.res_scale;
            sw[k][j] = sc[k][j] = 0.f;
        }
    }
    // every thread of a workgroup makes the same number of rounds: the row sums hold barriers
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < p.n_rows; row0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = row0 + sub;
        const bool live = row < p.n_rows;
        const uint32_t outer = (uint32_t)row / (uint32_t)p.n_inner, inner = (uint32_t)row % (uint32_t)p.n_inner;
        float a[K][V], g[K][V], t[K][V];
        Sum2 s{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool on = live && in[k];
#pragma unroll
            for (int j = 0; j < V; ++j) a[k][j] = g[k][j] = t[k][j] = 0.f;
            if (!on) continue;
            if constexpr (OP == kNormIn) {
                loadv<V>(p.x.p, p.dtype, row_at(p.x, outer, inner, d) + col[k], a[k]);
                if (p.has_r) {
                    loadv<V>(p.r.p, p.dtype, row_at(p.r, outer, inner, d) + col[k], t[k]);
#pragma unroll
                    for (int j = 0; j < V; ++j) a[k][j] = fmaf(c[k][j], t[k][j], a[k][j]);
                }
            } else if constexpr (OP == kNormInBwd) {
                loadv<V>(p.h.p, p.dtype, row_at(p.h, outer, inner, d) + col[k], a[k]);
                loadv<V>(p.dn.p, p.dtype_out, row_at(p.dn, outer, inner, d) + col[k], g[k]);
            } else {
                loadv<V>(p.y.p, p.dtype, row_at(p.y, outer, inner, d) + col[k], a[k]);
                if (p.has_z) loadv<V>(p.z.p, p.dtype_out, row_at(p.z, outer, inner, d) + col[k], t[k]);
                if constexpr (OP == kNormOutBwd)
                    loadv<V>(p.d_o.p, p.dtype_out, row_at(p.d_o, outer, inner, d) + col[k], g[k]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) s.a = fmaf(a[k][j], a[k][j], s.a);
            if constexpr (OP == kNormInBwd) {
#pragma unroll
                for (int j = 0; j < V; ++j) s.b = fmaf(g[k][j] * w[k][j], a[k][j], s.b);
            }
            if constexpr (OP == kNormOutBwd) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float act = 1.f, dact = 0.f;
                    if (p.has_z) act_of(p.act, t[k][j], act, dact);
                    s.b = fmaf(g[k][j] * c[k][j] * w[k][j] * act, a[k][j], s.b);
                }
            }
        }
        s = row_sum<TPR>(s, s_red);
        const float inv = 1.f / sqrtf(fmaf(s.a, p.inv_div, p.eps));
        [[maybe_unused]] float back = 0.f;
        if constexpr (OP == kNormInBwd) back = s.b * p.out_scale * inv * inv * p.inv_div;
        if constexpr (OP == kNormOutBwd) back = s.b * inv * inv * p.inv_div;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!(live && in[k])) continue;
            float o[V];
            if constexpr (OP == kNormIn) {
                if (p.write_h) storev<V>(p.h.p, p.dtype, row_at(p.h, outer, inner, d) + col[k], a[k]);
                const float f = inv * p.out_scale;
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = a[k][j] * f * w[k][j];
                storev<V>(p.n.p, p.dtype_out, row_at(p.n, outer, inner, d) + col[k], o);
            } else if constexpr (OP == kNormInBwd) {
                float e[V];
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] = 0.f;
                if (p.has_dh) loadv<V>(p.dh.p, p.dtype, row_at(p.dh, outer, inner, d) + col[k], e);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float gf = g[k][j] * p.out_scale;
                    o[j] = fmaf(inv, gf * w[k][j] - a[k][j] * back, e[j]);
                    sw[k][j] = fmaf(gf * inv, a[k][j], sw[k][j]);
                }
                if (p.has_r) {                 // only dchan_scale needs r
                    loadv<V>(p.r.p, p.dtype, row_at(p.r, outer, inner, d) + col[k], t[k]);
#pragma unroll
                    for (int j = 0; j < V; ++j) sc[k][j] = fmaf(o[j] * p.res_scale, t[k][j], sc[k][j]);
                }
                if (p.write_dr) {
#pragma unroll
                    for (int j = 0; j < V; ++j) e[j] = o[j] * c[k][j];
                    storev<V>(p.dr.p, p.dtype, row_at(p.dr, outer, inner, d) + col[k], e);
                }
                storev<V>(p.dx.p, p.dtype, row_at(p.dx, outer, inner, d) + col[k], o);
            } else if constexpr (OP == kNormOut) {
                float e[V];
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] = 0.f;
                if (p.has_x) loadv<V>(p.x.p, p.dtype_out, row_at(p.x, outer, inner, d) + col[k], e);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float act = 1.f, dact = 0.f;
                    if (p.has_z) act_of(p.act, t[k][j], act, dact);
                    o[j] = fmaf(a[k][j] * inv * w[k][j] * act, c[k][j], e[j]);
                }
                storev<V>(p.o.p, p.dtype_out, row_at(p.o, outer, inner, d) + col[k], o);
            } else {
                float e[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float act = 1.f, dact = 0.f;
                    if (p.has_z) act_of(p.act, t[k][j], act, dact);
                    const float yh = a[k][j] * inv, gc = g[k][j] * c[k][j];
                    o[j] = inv * (gc * w[k][j] * act - a[k][j] * back);
                    e[j] = gc * w[k][j] * yh * dact;
                    sw[k][j] = fmaf(gc * act, yh, sw[k][j]);
                    sc[k][j] = fmaf(g[k][j] * p.res_scale * act, w[k][j] * yh, sc[k][j]);
                }
                if (p.write_dz) storev<V>(p.dz.p, p.dtype_out, row_at(p.dz, outer, inner, d) + col[k], e);
                storev<V>(p.dy.p, p.dtype, row_at(p.dy, outer, inner, d) + col[k], o);
            }
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
                for (int i = (int)threadIdx.x; i < d; i += kNormThreads) {
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

// Adds the partial rows: 16 columns x 16 row groups per workgroup, the groups in LDS, in a fixed order.
__global__ void __launch_bounds__(kNormThreads) k_norm_sum(const NormParams p) {
    __shared__ float s[16][17];
    const int ci = (int)threadIdx.x & 15, g = (int)threadIdx.x >> 4;
    const int which = (int)blockIdx.y, col = (int)blockIdx.x * 16 + ci;
    float* out = which ? p.dchan_scale : p.dweight;
    if (!out) return;
    const float* in = p.part + (size_t)which * p.n_blocks * p.d;
    float t = 0.f;
    if (col < p.d)
        for (int b = g; b < p.n_blocks; b += 16) t += in[(size_t)b * p.d + col];
    s[g][ci] = t;
    __syncthreads();
    if (g == 0 && col < p.d) {
        for (int r = 1; r < 16; ++r) t += s[r][ci];
        out[col] = t;
    }
}

template <int OP, int V, int TPR, int K>
static hipError_t launch_t(const NormParams& p0, hipStream_t s) {
    constexpr int RPB = kNormThreads / TPR;
    constexpr bool kBwd = OP == kNormInBwd || OP == kNormOutBwd;
    NormParams p = p0;
    int64_t blocks = (p.n_rows + RPB - 1) / RPB;
    if (kBwd) {
        const int64_t cap = norm_bwd_blocks(p.n_rows, p.d);
        if (blocks > cap) blocks = cap;
    } else if (blocks > 8192) {
        blocks = 8192;                         // the weights are loaded once per workgroup and kept over its rows
    }
    p.n_blocks = (int32_t)blocks;
    if (blocks > 0) k_norm<OP, V, TPR, K><<<dim3((unsigned)blocks), dim3(kNormThreads), 0, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !kBwd || !(p.dweight || p.dchan_scale)) return e;
    k_norm_sum<<<dim3((unsigned)((p.d + 15) / 16), 2), dim3(kNormThreads), 0, s>>>(p);
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
    return launch_t<OP, 1, 256, 64>(p, s);
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
