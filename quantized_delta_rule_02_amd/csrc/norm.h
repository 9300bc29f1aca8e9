// Launchers of the norm kernels (norm.hip), called by the C ABI (ops_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sq {

constexpr int kNormMaxD = 16384;     // widest row: 256 threads hold it in 64 registers each
constexpr int kNormThreads = 256;

// Row arrays: element (row, j) of an array sits at p[(row / n_inner) * stride + (row % n_inner) * d + j].
struct NormRows {
    void* p;
    int64_t stride;
};

struct NormParams {
    int64_t n_rows;
    int32_t n_inner, d, dtype, dtype_out, act, n_blocks;
    int32_t has_r, has_z, has_x, has_dh, write_h, write_dr, write_dz;
    float inv_div;                   // 1 / d (RMS) or 1 (unit L2)
    float eps, res_scale, out_scale;
    const float* weight;             // [d] or NULL = 1
    const float* chan_scale;         // [d] or NULL = 1
    NormRows x, r, h, n, z, y, o;    // forward
    NormRows dn, dh, dx, dr, d_o, dy, dz;
    float* part;                     // backward: [2][n_blocks][d] partial sums of dweight and dchan_scale
    float* dweight;
    float* dchan_scale;
};

// Workgroups of a backward launch: at most one per row, and few enough that their partial sums stay small.
inline int64_t norm_bwd_blocks(int64_t n_rows, int d) {
    int64_t cap = (int64_t(1) << 21) / d;
    if (cap > 1024) cap = 1024;
    if (cap < 256) cap = 256;
    return n_rows < cap ? n_rows : cap;
}

enum : int { kNormIn = 0, kNormInBwd = 1, kNormOut = 2, kNormOutBwd = 3 };
// `vec`: every array is 16-byte aligned with strides and d multiples of 8.
hipError_t launch_norm(int op, bool vec, const NormParams& p, hipStream_t s);

}  // namespace sq
