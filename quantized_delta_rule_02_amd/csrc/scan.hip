// Gated delta scan over packed sequences (gfx950): per (sequence, head), S in float32,
//
//   S' = D_t S;  e_t = v_t - S'^T k_t;  S = S' + k_t (beta_t e_t)^T;  y_t = S^T q_t,   D_t = alpha_t I or diag(alpha_t)
//
// in chunks of 32 tokens.  With gamma_t the product of the chunk's gates up to t and Gamma_tj = gamma_t / gamma_j (formed
// as a product of gates, so no gate is divided by and strong decay cannot overflow):
//
//   A_tj = k_t . Gamma_tj k_j (j < t),  P_tj = q_t . Gamma_tj k_j (j <= t),  That = (I + A diag(beta))^-1
//   e = That (V - (gamma K) S);  u = beta e;  y = (gamma Q) S + P u;  S <- gamma_C S + ((gamma_C / gamma) K)^T u
//
// k_prep: That and P of every chunk and head, one wave each, all chunks at once.
// k_scan: the recurrence over a sequence's chunks.  A wave owns 16 value columns of one state (the columns do not
// interact), in 4 registers per 16 x 16 tile; see scan_dev.h for why no register has to move between products.
#include <hip/hip_runtime.h>

#include "scan_dev.h"

namespace sq {

__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- prep

constexpr int kPrepWaves = 4;
constexpr int kPrepLd = 36;          // 16-byte aligned rows, 4 banks apart

template <int DK, int NPL, bool KDA, bool BWD>
__global__ void __launch_bounds__(kPrepWaves * 64) k_prep(const ScanParams p) {
    constexpr int NKB = (DK + 31) / 32;
    __shared__ __align__(16) float s_n[kPrepWaves][2][32][kPrepLd];
    __shared__ __align__(16) float s_p[kPrepWaves][32][kPrepLd];
    __shared__ float s_g[KDA ? 1 : kPrepWaves][32][33];
    __shared__ float s_b[kPrepWaves][32];
    const int wave = (int)threadIdx.x >> 6, l = (int)threadIdx.x & 63, n = l & 15, g = l >> 4;
    const int64_t id = (int64_t)blockIdx.x * kPrepWaves + wave;
    if (id >= p.n_slots * p.n_heads) return;         // no workgroup barrier below: each wave works alone
    const int h = (int)(id % p.n_heads);
    const int64_t slot = id / p.n_heads;
    // the sequence whose first slot is the last one not above this slot
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_slot(sequence(p, mid), mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    const Seq sq_ = sequence(p, lo);
    const int64_t c0 = (slot - first_slot(sq_, lo)) * kChunk;
    if (c0 < 0 || c0 >= sq_.len) return;             // a slot that no chunk uses
    const int rem = (int)(sq_.len - c0 < kChunk ? sq_.len - c0 : kChunk);
    const int64_t tok0 = sq_.start + c0;
    const int hk = h / (p.n_heads / p.n_heads_k);
    constexpr float gmin = BWD ? kGateMin : 0.f;

    float(&N)[2][32][kPrepLd] = s_n[wave];
    float(&Pm)[32][kPrepLd] = s_p[wave];
    if (l < 32) s_b[wave][l] = l < rem ? p.beta[(tok0 + l) * p.n_heads + h] : 0.f;
    if constexpr (!KDA) {
        // column j of Gamma: a running product down the rows
        const float al = (l & 31) < rem ? fmaxf(p.gate[(tok0 + (l & 31)) * p.n_heads + h], gmin) : 1.f;
        if (l < 32) {
            float x = 0.f;
            for (int i = 0; i < 32; ++i) {
                const float ai = __shfl(al, i, 32);
                x = i == l ? 1.f : x * ai;
                s_g[wave][i][l] = x;
            }
        }
    }

    f32x4 aA[3], aP[3];                              // tiles (0,0), (1,0), (1,1)
#pragma unroll
    for (int t = 0; t < 3; ++t) aA[t] = aP[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    [[maybe_unused]] float diag[2] = {0.f, 0.f};
    for (int kb = 0; kb < NKB; ++kb) {
        float kx[2][8], qx[2][8], ax[2][8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 16 * t + n, ch = 32 * kb + 8 * g;
            const bool on = tok < rem && ch < DK;
#pragma unroll
            for (int j = 0; j < 8; ++j) { kx[t][j] = qx[t][j] = 0.f; ax[t][j] = 1.f; }
            if (on) {
                load8(p.k.p, p.dtype, (tok0 + tok) * p.k.stride + hk * DK + ch, kx[t]);
                load8(p.q.p, p.dtype, (tok0 + tok) * p.q.stride + hk * DK + ch, qx[t]);
                if constexpr (KDA) {
                    load8(p.gate, SQ_DTYPE_F32, ((tok0 + tok) * p.n_heads + h) * DK + ch, ax[t]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ax[t][j] = fmaxf(ax[t][j], gmin);
                }
            }
        }
        if constexpr (!KDA) {
            Frag<NPL> kf[2], qf[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) { kf[t] = split8<NPL>(kx[t]); qf[t] = split8<NPL>(qx[t]); }
            mma(aA[0], kf[0], kf[0]); mma(aP[0], qf[0], kf[0]);
            mma(aA[1], kf[1], kf[0]); mma(aP[1], qf[1], kf[0]);
            mma(aA[2], kf[1], kf[1]); mma(aP[2], qf[1], kf[1]);
        } else {
            // Pairs (i, j), j < i, by the highest bit in which i and j differ: with blocks of 2^lev tokens, i lies in an odd
            // block and j in the even one before it, and Gamma_ij is (gates of i's block up to i) x (gates of j's block
            // after j), both at most 1.  Five levels cover the triangle.
            float pre[2][8], suf[2][8], full[2][8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    diag[t] = fmaf(qx[t][j], kx[t][j], diag[t]);
                    pre[t][j] = full[t][j] = ax[t][j];
                    suf[t][j] = 1.f;
                }
#pragma unroll
            for (int lev = 0; lev < 4; ++lev) {
                const bool odd = (n >> lev) & 1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float kr[8], qr[8], kc[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        kr[j] = odd ? kx[t][j] * pre[t][j] : 0.f;
                        qr[j] = odd ? qx[t][j] * pre[t][j] : 0.f;
                        kc[j] = odd ? 0.f : kx[t][j] * suf[t][j];
                    }
                    const Frag<3> fk = split8<3>(kr), fq = split8<3>(qr), fc = split8<3>(kc);
                    f32x4 ta{0.f, 0.f, 0.f, 0.f}, tp{0.f, 0.f, 0.f, 0.f};
                    mma(ta, fk, fc);
                    mma(tp, fq, fc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool pair = ((4 * g + r) >> (lev + 1)) == (n >> (lev + 1));
                        aA[2 * t][r] += pair ? ta[r] : 0.f;
                        aP[2 * t][r] += pair ? tp[r] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float other = __shfl_xor(full[t][j], 1 << lev);
                        if (odd) pre[t][j] *= other;
                        else suf[t][j] *= other;
                        full[t][j] *= other;
                    }
                }
            }
            float kr[8], qr[8], kc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                kr[j] = kx[1][j] * pre[1][j];
                qr[j] = qx[1][j] * pre[1][j];
                kc[j] = kx[0][j] * suf[0][j];
            }
            const Frag<3> fk = split8<3>(kr), fq = split8<3>(qr), fc = split8<3>(kc);
            mma(aA[1], fk, fc);
            mma(aP[1], fq, fc);
        }
    }
    wave_sync();
    float* ap = nullptr;
    if constexpr (BWD && !KDA) ap = p.mat_ap + id * 2 * 32 * 32;
#pragma unroll
    for (int tl = 0; tl < 3; ++tl) {
        const int ti = tl > 0, tj = tl > 1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * ti + 4 * g + r, j = 16 * tj + n;
            float a = aA[tl][r], pv = aP[tl][r];
            if constexpr (!KDA) {
                const float gm = s_g[wave][i][j];
                a *= gm;
                pv *= gm;
            }
            a = j < i ? a : 0.f;
            pv = j <= i ? pv : 0.f;
            N[0][i][j] = a * s_b[wave][j];
            if constexpr (BWD) N[1][i][j] = a * s_b[wave][i];
            Pm[i][j] = pv;
            if constexpr (BWD && !KDA) {
                ap[i * 32 + j] = a;
                ap[1024 + i * 32 + j] = pv;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) Pm[4 * g + r][16 + n] = 0.f;     // the tile above the diagonal
    if constexpr (KDA) {
        wave_sync();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float x = diag[t];
            x += __shfl_xor(x, 16);
            x += __shfl_xor(x, 32);
            if (g == 0) Pm[16 * t + n][16 * t + n] = x;
        }
    }
    wave_sync();
    // (I + N) X = I by rows: lane c holds column c; lanes 0-31 take A diag(beta), lanes 32-63 diag(beta) A
    const int which = BWD ? l >> 5 : 0, cl = l & 31;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float s0 = i == cl ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int jj = 0; jj < (i + 3) / 4; ++jj) {
            const f32x4 row = *reinterpret_cast<const f32x4*>(&N[which][i][4 * jj]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * jj + j < i) {
                    if (j & 1) s1 = fmaf(-row[j], x[4 * jj + j], s1);
                    else s0 = fmaf(-row[j], x[4 * jj + j], s0);
                }
        }
        x[i] = s0 + s1;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 32; ++i) N[which][i][cl] = x[i];         // without BWD both halves write the same values
    wave_sync();
    const size_t mo = (size_t)id * kMatShorts;
    auto put = [&](uint16_t* mat, int ti, const float* v) {
        const Frag<3> f = split8<3>(v);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl)
            *reinterpret_cast<u32x4v*>(mat + mo + ((ti * 3 + pl) * 64 + l) * 8) = f.p[pl];
    };
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
        float v[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = 16 * (e >> 2) + 4 * g + (e & 3);
            v[e] = N[0][16 * ti + n][c];
            w[e] = Pm[16 * ti + n][c];
        }
        put(p.mat_th, ti, v);
        if constexpr (!BWD) put(p.mat_p, ti, w);
        if constexpr (BWD) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = 16 * (e >> 2) + 4 * g + (e & 3);
                v[e] = N[1][c][16 * ti + n];
                w[e] = Pm[c][16 * ti + n];
            }
            put(p.mat_tt, ti, v);
            put(p.mat_pt, ti, w);
        }
    }
}

// ---------------------------------------------------------------- scan

// MODE: forward with outputs; forward for the backward pass (keeps e and the chunks' first states, no y);
// reverse (the gradient of the state from the last chunk to the first).
enum : int { kScanOut = 0, kScanKeep = 1, kScanRev = 2 };

template <int NP>
__device__ __forceinline__ Frag<NP> lds_frag(const uint16_t* base, int plane_stride, int off) {
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = *reinterpret_cast<const u32x4v*>(base + i * plane_stride + off);
    return f;
}

__device__ __forceinline__ Frag<3> mat_frag(const uint16_t* mat, size_t id, int ti, int l) {
    Frag<3> f;
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
        f.p[pl] = *reinterpret_cast<const u32x4v*>(mat + id * kMatShorts + ((ti * 3 + pl) * 64 + l) * 8);
    return f;
}

__device__ __forceinline__ void load4(const void* p, int dt, int64_t i, float* x) {
    if (dt == SQ_DTYPE_F32) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = a[j];
        return;
    }
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        x[2 * j] = dt == SQ_DTYPE_BF16 ? bf16_lo(w[j]) : f16_val(w[j] & 0xffffu);
        x[2 * j + 1] = dt == SQ_DTYPE_BF16 ? bf16_hi(w[j]) : f16_val(w[j] >> 16);
    }
}

template <int DK, int NPL, bool KDA, int MODE>
__global__ void __launch_bounds__(512) k_scan(const ScanParams p) {
    constexpr bool REV = MODE == kScanRev;
    constexpr int NP = KDA ? 3 : NPL;                // planes of the staged operands (gates make them float32)
    constexpr int NT = DK / 16, NKB = (DK + 31) / 32;
    constexpr int LDK = 32 * NKB + 8, LDT = 40;      // rows 4 (resp. 20) banks apart
    constexpr bool kTwoT = REV;                      // the reverse scan needs K^T and Q^T, the forward one Q and K^T
    __shared__ __align__(16) uint16_t s_k[NP][32][LDK];          // token-major operands
    __shared__ __align__(16) uint16_t s_q[kTwoT || MODE == kScanKeep ? 1 : NP][32][LDK];
    __shared__ __align__(16) uint16_t s_kt[NP][DK][LDT];         // key-major operands
    __shared__ __align__(16) uint16_t s_qt[kTwoT ? NP : 1][DK][LDT];
    __shared__ __align__(16) float s_pre[32], s_suf[32], s_beta[32], s_last[KDA ? DK : 4];

    const int tid = (int)threadIdx.x, nthr = (int)blockDim.x;
    const int wave = tid >> 6, l = tid & 63, n = l & 15, g = l >> 4;
    const int H = p.n_heads, dv = p.dv;
    const int bh = (int)(blockIdx.x % (unsigned)(H * p.n_seq)), sg = (int)(blockIdx.x / (unsigned)(H * p.n_seq));
    const int b = bh / H, h = bh % H, hk = h / (H / p.n_heads_k);
    const Seq seq = sequence(p, b);
    const int64_t slot0 = first_slot(seq, b);
    const int col = (sg * (nthr >> 6) + wave) * 16 + n;          // this lane's value column
    const int64_t nc = (seq.len + kChunk - 1) / kChunk;

    f32x4 S[NT];
    const float* init = REV ? p.ds1 : p.s0;
    const size_t sbase = (size_t)bh * DK * dv + col;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = init ? init[sbase + (size_t)(16 * t + 4 * g + r) * dv] : 0.f;
    if constexpr (DK < 32) {                         // the unused half of a block of 32 key rows stays zero
        for (int i = tid; i < NP * 32 * LDK; i += nthr) (&s_k[0][0][0])[i] = 0;
        if constexpr (MODE == kScanOut)
            for (int i = tid; i < NP * 32 * LDK; i += nthr) (&s_q[0][0][0])[i] = 0;
    }

    for (int64_t ci = 0; ci < nc; ++ci) {
        const int64_t c = REV ? nc - 1 - ci : ci;
        const int64_t tok0 = seq.start + c * kChunk;
        const int rem = (int)(seq.len - c * kChunk < kChunk ? seq.len - c * kChunk : kChunk);
        const size_t id = (size_t)(slot0 + c) * H + h;
        const Frag<3> m0[2] = {mat_frag(REV ? p.mat_tt : p.mat_th, id, 0, l), mat_frag(REV ? p.mat_tt : p.mat_th, id, 1, l)};
        float xin[2][4];                             // v (forward) or dy (reverse)
        const ScanRows& xr = REV ? p.dy : p.v;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = 16 * t + 4 * g + r;
                xin[t][r] = tok < rem ? load1(xr.p, p.dtype, (tok0 + tok) * xr.stride + (int64_t)h * dv + col) : 0.f;
            }
        __syncthreads();                             // the previous chunk's operands have been read
        if (tid < 64) {
            const int t = l & 31;
            if (l < 32) s_beta[t] = t < rem ? p.beta[(tok0 + t) * H + h] : 0.f;
            if constexpr (!KDA) {
                float pr = t < rem ? p.gate[(tok0 + t) * H + h] : 1.f, sf = pr;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float a = __shfl_up(pr, o, 32), z = __shfl_down(sf, o, 32);
                    if (t >= o) pr *= a;
                    if (t + o < 32) sf *= z;
                }
                sf = __shfl_down(sf, 1, 32);
                if (l < 32) {
                    s_pre[t] = pr;
                    s_suf[t] = t == 31 ? 1.f : sf;
                    if (t == 31) s_last[0] = pr;
                }
            }
        }
        for (int u = tid; u < 8 * DK / 4; u += nthr) {           // 4 tokens x 4 key rows each
            const int tq = u & 7, cq = u >> 3;
            float kx[4][4], qx[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int tok = 4 * tq + j;
#pragma unroll
                for (int i = 0; i < 4; ++i) kx[j][i] = qx[j][i] = 0.f;
                if (tok < rem) {
                    load4(p.k.p, p.dtype, (tok0 + tok) * p.k.stride + hk * DK + 4 * cq, kx[j]);
                    if constexpr (MODE != kScanKeep)
                        load4(p.q.p, p.dtype, (tok0 + tok) * p.q.stride + hk * DK + 4 * cq, qx[j]);
                }
            }
            float pre[4][4], suf[4][4];
            if constexpr (KDA) {
                float al[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) al[j][i] = 1.f;
                    if (4 * tq + j < rem)
                        load4(p.gate, SQ_DTYPE_F32, ((tok0 + 4 * tq + j) * H + h) * DK + 4 * cq, al[j]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pre[0][i] = al[0][i];
                    suf[3][i] = 1.f;
#pragma unroll
                    for (int j = 1; j < 4; ++j) pre[j][i] = pre[j - 1][i] * al[j][i];
#pragma unroll
                    for (int j = 2; j >= 0; --j) suf[j][i] = suf[j + 1][i] * al[j + 1][i];
                    float up = pre[3][i], dn = pre[3][i];        // products over the eight token quads
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) {
                        const float a = __shfl_up(up, o, 8), z = __shfl_down(dn, o, 8);
                        if (tq >= o) up *= a;
                        if (tq + o < 8) dn *= z;
                    }
                    if (tq == 7) s_last[4 * cq + i] = up;
                    float before = __shfl_up(up, 1, 8), after = __shfl_down(dn, 1, 8);
                    before = tq == 0 ? 1.f : before;
                    after = tq == 7 ? 1.f : after;
#pragma unroll
                    for (int j = 0; j < 4; ++j) { pre[j][i] *= before; suf[j][i] *= after; }
                }
            }
            // token-major: forward gamma K (and gamma Q), reverse (gamma_C / gamma) K; key-major: the other way round
            float a[4][4], bq[4][4], kt[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[j][i] = kx[j][i] * (KDA ? (REV ? suf[j][i] : pre[j][i]) : 1.f);
                    bq[j][i] = qx[j][i] * (KDA ? pre[j][i] : 1.f);
                    kt[i][j] = kx[j][i] * (KDA ? (REV ? pre[j][i] : suf[j][i]) : 1.f);
                }
            const int pc = kpos(4 * cq), pt = kpos(4 * tq);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x2 w[NP];
                split4<NP>(a[j], w);
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x2*>(&s_k[i][4 * tq + j][pc]) = w[i];
                split4<NP>(kt[j], w);
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x2*>(&s_kt[i][4 * cq + j][pt]) = w[i];
                if constexpr (MODE == kScanOut) {
                    split4<NP>(bq[j], w);
#pragma unroll
                    for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x2*>(&s_q[i][4 * tq + j][pc]) = w[i];
                }
                if constexpr (REV) {
                    const float qt[4] = {bq[0][j], bq[1][j], bq[2][j], bq[3][j]};
                    split4<NP>(qt, w);
#pragma unroll
                    for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x2*>(&s_qt[i][4 * cq + j][pt]) = w[i];
                }
            }
        }
        __syncthreads();

        if constexpr (MODE != kScanOut) {            // the backward pass reads the states at the chunk borders
            float* keep = (REV ? p.gt : p.st) + id * (size_t)DK * dv + col;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) keep[(size_t)(16 * t + 4 * g + r) * dv] = S[t][r];
        }
        const f32x4 zero{0.f, 0.f, 0.f, 0.f};
        f32x4 z[2] = {zero, zero}, yq[2] = {zero, zero};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            float sx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) sx[e] = 2 * kb + (e >> 2) < NT ? S[2 * kb + (e >> 2)][e & 3] : 0.f;
            const Frag<3> sf = split8<3>(sx);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int off = (16 * t + n) * LDK + 32 * kb + 8 * g;
                mma(z[t], lds_frag<NP>(&s_k[0][0][0], 32 * LDK, off), sf);
                if constexpr (MODE == kScanOut) mma(yq[t], lds_frag<NP>(&s_q[0][0][0], 32 * LDK, off), sf);
            }
        }
        float pre[2][4], suf[2][4], be[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                pre[t][r] = KDA ? 1.f : s_pre[16 * t + 4 * g + r];
                suf[t][r] = KDA ? 1.f : s_suf[16 * t + 4 * g + r];
                be[t][r] = s_beta[16 * t + 4 * g + r];
            }
        float w8[8];
        if constexpr (!REV) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = xin[e >> 2][e & 3] - pre[e >> 2][e & 3] * z[e >> 2][e & 3];
            const Frag<3> rf = split8<3>(w8);
            f32x4 ev[2] = {zero, zero};
#pragma unroll
            for (int t = 0; t < 2; ++t) mma(ev[t], m0[t], rf);
            if constexpr (MODE == kScanKeep) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int tok = 16 * t + 4 * g + r;
                        if (tok < rem) p.e[((tok0 + tok) * H + h) * dv + col] = ev[t][r];
                    }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = ev[e >> 2][e & 3] * be[e >> 2][e & 3];
            if constexpr (MODE == kScanOut) {
                const Frag<3> uf = split8<3>(w8);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 y;
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = yq[t][r] * pre[t][r];
                    mma(y, mat_frag(p.mat_p, id, t, l), uf);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int tok = 16 * t + 4 * g + r;
                        if (tok < rem) store1(p.y.p, p.dtype, (tok0 + tok) * p.y.stride + (int64_t)h * dv + col, y[r]);
                    }
                }
            }
            if constexpr (!KDA) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w8[e] *= suf[e >> 2][e & 3];
            }
            const Frag<3> uf = split8<3>(w8);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] *= s_last[KDA ? 16 * t + 4 * g + r : 0];
                mma(S[t], lds_frag<NP>(&s_kt[0][0][0], DK * LDT, (16 * t + n) * LDT + 8 * g), uf);
            }
        } else {
            // R = (gamma_C / gamma) K G + P^T dy;  du = T^T R;  G <- gamma_C G + (gamma Q)^T dy - (gamma K)^T (beta du)
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = xin[e >> 2][e & 3];
            const Frag<3> dyf = split8<3>(w8);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) z[t][r] *= suf[t][r];
                mma(z[t], mat_frag(p.mat_pt, id, t, l), dyf);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = z[e >> 2][e & 3];
            const Frag<3> rf = split8<3>(w8);
            f32x4 du[2] = {zero, zero};
#pragma unroll
            for (int t = 0; t < 2; ++t) mma(du[t], m0[t], rf);
            float q8[8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = 16 * t + 4 * g + r;
                    const float w = du[t][r] * be[t][r];
                    if (tok < rem) {
                        p.du[((tok0 + tok) * H + h) * dv + col] = du[t][r];
                        store1(p.dvv.p, p.dtype, (tok0 + tok) * p.dvv.stride + (int64_t)h * dv + col, w);
                    }
                    w8[4 * t + r] = -w * pre[t][r];
                    q8[4 * t + r] = xin[t][r] * pre[t][r];
                }
            const Frag<3> wf = split8<3>(w8), qf = split8<3>(q8);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] *= s_last[KDA ? 16 * t + 4 * g + r : 0];
                const int off = (16 * t + n) * LDT + 8 * g;
                mma(S[t], lds_frag<NP>(&s_kt[0][0][0], DK * LDT, off), wf);
                mma(S[t], lds_frag<NP>(&s_qt[0][0][0], DK * LDT, off), qf);
            }
        }
    }
    float* fin = REV ? p.ds0 : MODE == kScanOut ? p.s1 : nullptr;
    if (fin) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) fin[sbase + (size_t)(16 * t + 4 * g + r) * dv] = S[t][r];
    }
}

// ---------------------------------------------------------------- launchers

template <int DK, int NPL, bool KDA>
static hipError_t prep_t(const ScanParams& p, bool backward, hipStream_t s) {
    const int64_t blocks = (p.n_slots * p.n_heads + kPrepWaves - 1) / kPrepWaves;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), blk(kPrepWaves * 64);
    if (backward) k_prep<DK, NPL, KDA, true><<<grid, blk, 0, s>>>(p);
    else k_prep<DK, NPL, KDA, false><<<grid, blk, 0, s>>>(p);
    return hipGetLastError();
}

template <int DK, int NPL, bool KDA>
static hipError_t scan_t(const ScanParams& p, int mode, hipStream_t s) {
    const int slices = p.dv / 16, nw = slices < 8 ? slices : 8;
    const int64_t blocks = (int64_t)p.n_seq * p.n_heads * (slices / nw);
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), blk(nw * 64);
    switch (mode) {
        case kScanOut: k_scan<DK, NPL, KDA, kScanOut><<<grid, blk, 0, s>>>(p); break;
        case kScanKeep: k_scan<DK, NPL, KDA, kScanKeep><<<grid, blk, 0, s>>>(p); break;
        default: k_scan<DK, NPL, KDA, kScanRev><<<grid, blk, 0, s>>>(p); break;
    }
    return hipGetLastError();
}

hipError_t launch_scan_prep(const ScanParams& p, bool backward, hipStream_t s) { SQ_SCAN_DISPATCH(prep_t, p, backward, s); }
hipError_t launch_scan_fwd(const ScanParams& p, bool keep, hipStream_t s) {
    const int mode = keep ? kScanKeep : kScanOut;
    SQ_SCAN_DISPATCH(scan_t, p, mode, s);
}
hipError_t launch_scan_rev(const ScanParams& p, hipStream_t s) { SQ_SCAN_DISPATCH(scan_t, p, kScanRev, s); }

}  // namespace sq
