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

// ---------------------------------------------------------------- prep

constexpr int kPrepWaves = 4;
constexpr int kPrepLd = 36;          // 16-byte aligned rows, 4 banks apart

// One wave per chunk and head.  Its LDS is one 32 x 32 matrix (two for the backward pass), used in turn for I + N, for
// its inverse and for P, so that four and more waves fit on a SIMD: with all of them side by side (18 KiB a wave, two
// waves) the launch took 118 us where it now takes 61 (12301 tokens, 32 heads, bfloat16).
template <int DK, int DT, bool KDA, bool BWD>
__global__ void __launch_bounds__(kPrepWaves * 64) k_prep(const ScanParams p) {
    constexpr int NKB = (DK + 31) / 32, NPL = planes_of(DT), NM = BWD ? 2 : 1, ES = DT == SQ_DTYPE_F32 ? 4 : 2;
    __shared__ __align__(16) float s_m[kPrepWaves][NM][32][kPrepLd];
    __shared__ float s_gt[KDA ? 1 : kPrepWaves][2][5][32];
    __shared__ float s_b[kPrepWaves][32];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l = (int)threadIdx.x & 63, n = l & 15, g = l >> 4;
    const int64_t id = (int64_t)blockIdx.x * kPrepWaves + wave;
    if (id >= p.n_slots * p.n_heads) return;         // no workgroup barrier below: each wave works alone
    const int h = (int)(id % p.n_heads);
    const ChunkAt ck = chunk_of_slot(p, id / p.n_heads);
    if (ck.rem <= 0) return;                         // a slot that no chunk uses
    const int rem = ck.rem, H = p.n_heads, hk = h / (H / p.n_heads_k);
    const int64_t tok0 = ck.tok0;
    constexpr float gmin = BWD ? kGateMin : 0.f;

    float(&M)[NM][32][kPrepLd] = s_m[wave];
    if (l < 32) s_b[wave][l] = l < rem ? p.beta[(tok0 + l) * H + h] : 0.f;
    if constexpr (!KDA) {
        const int t = l & 31;
        const float a = t < rem ? p.gate[(tok0 + t) * H + h] : 1.f;
        GateLevels<float> lv(fmaxf(a, gmin));
#pragma unroll
        for (int lev = 0; lev < 5; ++lev) {
            if (l < 32) {
                s_gt[wave][0][lev][t] = lv.pre;
                s_gt[wave][1][lev][t] = lv.suf;
            }
            lv.grow((t >> lev) & 1, __shfl_xor(lv.full, 1 << lev));
        }
        // the gates' products up to each token and after it, for the scan (which takes the gates as they are)
        if constexpr (BWD) {
            lv = GateLevels<float>(a);
#pragma unroll
            for (int lev = 0; lev < 5; ++lev) lv.grow((t >> lev) & 1, __shfl_xor(lv.full, 1 << lev));
        }
        if (l < 32) {
            p.mat_gb[id * 64 + t] = lv.pre;
            p.mat_gb[id * 64 + 32 + t] = lv.suf;
        }
    }

    f32x4 aA[3], aP[3];                              // tiles (0,0), (1,0), (1,1)
#pragma unroll
    for (int t = 0; t < 3; ++t) aA[t] = aP[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    [[maybe_unused]] float diag[2] = {0.f, 0.f};
    const uint32_t ks = (uint32_t)p.k.stride * ES, qs = (uint32_t)p.q.stride * ES, gs = (uint32_t)H * DK * 4;
    const Window wk(static_cast<const char*>(p.k.p) + tok0 * ks, rem * ks), wq(static_cast<const char*>(p.q.p) + tok0 * qs, rem * qs);
    const Window wg(reinterpret_cast<const char*>(p.gate) + tok0 * gs, KDA ? rem * gs : 0);
    constexpr int RW = DT == SQ_DTYPE_F32 ? 2 : 1;   // 16-byte loads of 8 elements
    struct Rows { Raw<DT, 8 / RW> k[2][RW], q[2][RW]; Raw<SQ_DTYPE_F32, 4> a[2][KDA ? 2 : 1]; };
    auto fetch = [&](int kb) {                       // key rows 32 kb + 8 g .. + 7 of tokens 16 t + n
        Rows r;
        const int ch = 32 * kb + 8 * g;
        auto at = [&](uint32_t off) { return DK < 32 && ch >= DK ? 0xfffffff0u : off; };   // beyond the rows: zeros
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                r.k[t][i].load(wk, at((16 * t + n) * ks + (hk * DK + ch + 4 * i) * ES));
                r.q[t][i].load(wq, at((16 * t + n) * qs + (hk * DK + ch + 4 * i) * ES));
            }
            if constexpr (KDA) {
#pragma unroll
                for (int i = 0; i < 2; ++i) r.a[t][i].load(wg, at((16 * t + n) * gs + (h * DK + ch + 4 * i) * 4));
            }
        }
        return r;
    };
    Rows next = fetch(0);
#pragma unroll(KDA ? 1 : NKB)
    for (int kb = 0; kb < NKB; ++kb) {
        const Rows cur = next;
        if (kb + 1 < NKB) next = fetch(kb + 1);
        float kx[2][8], qx[2][8];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                kx[t][j] = RW == 2 ? cur.k[t][RW - 1 ? j >> 2 : 0].at(j & 3) : cur.k[t][0].at(j);
                qx[t][j] = RW == 2 ? cur.q[t][RW - 1 ? j >> 2 : 0].at(j & 3) : cur.q[t][0].at(j);
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
            // after j), both at most 1.  Five levels cover the triangle.  At a level a token is a row or a column, never
            // both: one scaled and split k serves as either operand.
            GateLevels<float> lv[2][8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    diag[t] = fmaf(qx[t][j], kx[t][j], diag[t]);
                    const bool on = 16 * t + n < rem && (DK >= 32 || 32 * kb + 8 * g < DK);
                    lv[t][j] = GateLevels<float>(on ? fmaxf(cur.a[t][KDA ? j >> 2 : 0].at(j & 3), gmin) : 1.f);
                }
#pragma unroll
            for (int lev = 0; lev < 4; ++lev) {
                const bool odd = (n >> lev) & 1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float ku[8], qu[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ku[j] = kx[t][j] * pick(odd, lv[t][j].pre, lv[t][j].suf);
                        qu[j] = qx[t][j] * lv[t][j].pre;
                    }
                    const Frag<3> fk = split8<3>(ku), fq = split8<3>(qu);
                    f32x4 ta{0.f, 0.f, 0.f, 0.f}, tp{0.f, 0.f, 0.f, 0.f};
                    mma(ta, fk, fk);
                    mma(tp, fq, fk);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = 4 * g + r;
                        const bool pair = ((i ^ n) >> lev) == 1 && i > n;
                        aA[2 * t][r] += pair ? ta[r] : 0.f;
                        aP[2 * t][r] += pair ? tp[r] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) lv[t][j].grow(odd, __shfl_xor(lv[t][j].full, 1 << lev));
                }
            }
            float kr[8], qr[8], kc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                kr[j] = kx[1][j] * lv[1][j].pre;
                qr[j] = qx[1][j] * lv[1][j].pre;
                kc[j] = kx[0][j] * lv[0][j].suf;
            }
            const Frag<3> fk = split8<3>(kr), fq = split8<3>(qr), fc = split8<3>(kc);
            mma(aA[1], fk, fc);
            mma(aP[1], fq, fc);
        }
    }
    wave_sync();
    float* ap = nullptr;
    if constexpr (BWD && !KDA) ap = p.mat_ap + id * 2 * 32 * 32;
    if constexpr (KDA) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            diag[t] += __shfl_xor(diag[t], 16);      // lane n: q_i . k_i of token 16 t + n
            diag[t] += __shfl_xor(diag[t], 32);
        }
    }
#pragma unroll
    for (int tl = 0; tl < 3; ++tl) {
        const int ti = tl > 0, tj = tl > 1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * ti + 4 * g + r, j = 16 * tj + n;
            float a = aA[tl][r], pv = aP[tl][r];
            if constexpr (!KDA) {
                const int lev = j < i ? 31 - __builtin_clz(i ^ j) : 0;
                const float gm = s_gt[wave][0][lev][i] * s_gt[wave][1][lev][j];
                a *= gm;
                pv *= i == j ? 1.f : gm;
            } else if (ti == tj) {
                pv = i == j ? diag[ti] : pv;
            }
            a = j < i ? a : 0.f;
            pv = j <= i ? pv : 0.f;
            aP[tl][r] = pv;
            M[0][i][j] = a * s_b[wave][j];
            if constexpr (BWD) M[NM - 1][i][j] = a * s_b[wave][i];
            if constexpr (BWD && !KDA) {
                ap[i * 32 + j] = a;
                ap[1024 + i * 32 + j] = pv;
            }
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
            const f32x4 row = *reinterpret_cast<const f32x4*>(&M[which][i][4 * jj]);
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
    for (int i = 0; i < 32; ++i) M[which][i][cl] = x[i];         // without BWD both halves write the same values
    wave_sync();
    const size_t mo = (size_t)id * kMatShorts;
    auto put = [&](uint16_t* mat, const float (&m)[32][kPrepLd], bool transposed) {
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = 16 * (e >> 2) + 4 * g + (e & 3);
                v[e] = transposed ? m[c][16 * ti + n] : m[16 * ti + n][c];
            }
            const Frag<3> f = split8<3>(v);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl)
                *reinterpret_cast<u32x4v*>(mat + mo + ((ti * 3 + pl) * 64 + l) * 8) = f.p[pl];
        }
    };
    put(p.mat_th, M[0], false);
    if constexpr (BWD) put(p.mat_tt, M[NM - 1], true);
    wave_sync();
#pragma unroll
    for (int tl = 0; tl < 3; ++tl)
#pragma unroll
        for (int r = 0; r < 4; ++r) M[0][16 * (tl > 0) + 4 * g + r][16 * (tl > 1) + n] = aP[tl][r];
#pragma unroll
    for (int r = 0; r < 4; ++r) M[0][4 * g + r][16 + n] = 0.f;   // the tile above the diagonal
    wave_sync();
    put(BWD ? p.mat_pt : p.mat_p, M[0], BWD);
}

// ---------------------------------------------------------------- scan

// MODE: forward with outputs; forward for the backward pass (keeps e and the chunks' first states, no y);
// reverse (the gradient of the state from the last chunk to the first).
enum : int { kScanOut = 0, kScanKeep = 1, kScanRev = 2 };

// The scan's LDS: operands of one chunk.  Token-major rows are 4 banks apart, key-major ones 20.
template <int DK, int NP, int MODE>
struct ScanLds {
    static constexpr bool REV = MODE == kScanRev;
    static constexpr int NKB = (DK + 31) / 32, LDK = 32 * NKB + 8, LDT = 40, NMAT = MODE == kScanKeep ? 1 : 2;
    uint16_t k[NP][32][LDK];                             // token-major: gamma K forward, (gamma_C / gamma) K in reverse
    uint16_t q[MODE == kScanOut ? NP : 1][MODE == kScanOut ? 32 : 1][LDK];
    uint16_t kt[NP][DK][LDT];                            // key-major: the other of the two
    uint16_t qt[REV ? NP : 1][REV ? DK : 1][LDT];
    uint16_t m[NMAT][kMatShorts];                        // That, P (forward); T^T, P^T (reverse)
    float pre[32], suf[32], beta[32], last[DK];
};

// One workgroup of DK / 16 waves per DK value columns of a state, so that each thread stages 4 tokens x 2 key rows of a
// chunk.  The loads of the next chunk are in flight while this one is computed.
template <int DK, int DT, bool KDA, int MODE>
__device__ __forceinline__ void scan_body(const ScanParams& p, unsigned block, ScanLds<DK, KDA ? 3 : planes_of(DT), MODE>& s) {
    constexpr bool REV = MODE == kScanRev, OUT = MODE == kScanOut;
    constexpr int NPL = planes_of(DT);
    constexpr int NP = KDA ? 3 : NPL;                // planes of the staged operands (gates make them float32)
    using Lds = ScanLds<DK, NP, MODE>;
    constexpr int NT = DK / 16, NKB = Lds::NKB, LDK = Lds::LDK, LDT = Lds::LDT, NMAT = Lds::NMAT;
    constexpr int NW = DK / 16, NTHR = NW * 64, CH = 8 * DK / NTHR, ES = DT == SQ_DTYPE_F32 ? 4 : 2;
    static_assert(CH == 2);

    const int tid = (int)threadIdx.x;
    const int wave = tid >> 6, l = tid & 63, n = l & 15, g = l >> 4;
    const int H = p.n_heads, dv = p.dv;
    const int bh = (int)(block % (unsigned)(H * p.n_seq)), sg = (int)(block / (unsigned)(H * p.n_seq));
    const int b = bh / H, h = bh % H, hk = h / (H / p.n_heads_k);
    const Seq sv = sequence(p, b);
    const int start = __builtin_amdgcn_readfirstlane((int)sv.start), len = __builtin_amdgcn_readfirstlane((int)sv.len);
    const int64_t slot0 = (start >> 5) + b;
    const int col = (sg * NW + wave) * 16 + n;                   // this lane's value column
    const int nc = (len + kChunk - 1) / kChunk;
    // staging: token quad and key rows of this thread; the gates' products run over the quads, eight neighbouring lanes
    const int tq = KDA ? tid & 7 : tid / (DK / CH), cq = KDA ? tid >> 3 : tid % (DK / CH);

    f32x4 S[NT];
    const float* init = REV ? p.ds1 : p.s0;
    const size_t sbase = (size_t)bh * DK * dv + col;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = init ? init[sbase + (size_t)(16 * t + 4 * g + r) * dv] : 0.f;
    if constexpr (DK < 32) {                         // the unused half of a block of 32 key rows stays zero
        for (int i = tid; i < NP * 32 * LDK; i += NTHR) (&s.k[0][0][0])[i] = 0;
        if constexpr (OUT)
            for (int i = tid; i < NP * 32 * LDK; i += NTHR) (&s.q[0][0][0])[i] = 0;
    }

    constexpr int MU = (NMAT * kMatShorts / 8 + NTHR - 1) / NTHR;   // 16-byte units of the chunk's matrices per thread
    Raw<DT, CH> kx[4], qx[4];
    Raw<SQ_DTYPE_F32, CH> ax[4];
    u32x4v mx[MU];
    uint32_t xn[2][4];
    float gb0 = 0.f, gb1 = 0.f;
    const ScanRows& xr = REV ? p.dy : p.v;
    const uint32_t ks = (uint32_t)p.k.stride * ES, qs = (uint32_t)p.q.stride * ES, xs = (uint32_t)xr.stride * ES;
    const uint32_t gs = (uint32_t)H * DK * 4;
    const uint32_t ko = 4 * tq * ks + (hk * DK + CH * cq) * ES, qo = 4 * tq * qs + (hk * DK + CH * cq) * ES;
    const uint32_t go = 4 * tq * gs + (h * DK + CH * cq) * 4, xo = 4 * g * xs + (h * dv + col) * ES;
    auto fetch = [&](int c) {                        // chunk c into registers
        const int64_t tok0 = start + (int64_t)c * kChunk;
        const uint32_t rem = len - c * kChunk < kChunk ? len - c * kChunk : kChunk;
        const size_t id = (size_t)(slot0 + c) * H + h;
        const Window wk(static_cast<const char*>(p.k.p) + tok0 * ks, rem * ks);
        const Window wx(static_cast<const char*>(xr.p) + tok0 * xs, rem * xs);
#pragma unroll
        for (int j = 0; j < 4; ++j) kx[j].load(wk, ko + j * ks);
        if constexpr (MODE != kScanKeep) {
            const Window wq(static_cast<const char*>(p.q.p) + tok0 * qs, rem * qs);
#pragma unroll
            for (int j = 0; j < 4; ++j) qx[j].load(wq, qo + j * qs);
        }
        if constexpr (KDA) {
            const Window wg(reinterpret_cast<const char*>(p.gate) + tok0 * gs, rem * gs);
#pragma unroll
            for (int j = 0; j < 4; ++j) ax[j].load(wg, go + j * gs);
        } else if (tid < 64) {
            gb0 = p.mat_gb[id * 64 + tid];           // the products of the gates, from k_prep
        }
        if (tid < 32) {
            const Window wb(p.beta + tok0 * H, rem * H * 4);
            gb1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(wb.r, (tid * H + h) * 4, 0, 0));
        }
#pragma unroll
        for (int u = 0; u < MU; ++u) {
            const int i = tid + u * NTHR, which = i / (kMatShorts / 8);
            if (NMAT * kMatShorts / 8 % NTHR == 0 || i < NMAT * kMatShorts / 8) {
                const uint16_t* m = which ? (REV ? p.mat_pt : p.mat_p) : (REV ? p.mat_tt : p.mat_th);
                mx[u] = *reinterpret_cast<const u32x4v*>(m + id * kMatShorts + (i - which * (kMatShorts / 8)) * 8);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) xn[t][r] = win_load1<DT>(wx, xo + (16 * t + r) * xs);
    };
    if (nc > 0) fetch(REV ? nc - 1 : 0);

    for (int ci = 0; ci < nc; ++ci) {
        const int c = REV ? nc - 1 - ci : ci;
        const int64_t tok0 = start + (int64_t)c * kChunk;
        const int rem = len - c * kChunk < kChunk ? len - c * kChunk : kChunk;
        const size_t id = (size_t)(slot0 + c) * H + h;
        lds_barrier();                               // the previous chunk's operands have been read
        if (!KDA && tid < 64) (&s.pre[0])[tid] = gb0;            // pre, then suf
        if (tid < 32) s.beta[tid] = gb1;
        if (!KDA && tid == 31) s.last[0] = gb0;                  // pre of the last token: all gates
#pragma unroll
        for (int u = 0; u < MU; ++u) {
            const int i = tid + u * NTHR;
            if (NMAT * kMatShorts / 8 % NTHR == 0 || i < NMAT * kMatShorts / 8)
                *reinterpret_cast<u32x4v*>(&s.m[0][0] + i * 8) = mx[u];
        }
        {
            float pre[4][CH], suf[4][CH];
            if constexpr (KDA) {
                float al[4][CH];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < CH; ++i) al[j][i] = 4 * tq + j < rem ? ax[j].at(i) : 1.f;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
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
                    if (tq == 7) s.last[CH * cq + i] = up;
                    float before = __shfl_up(up, 1, 8), after = __shfl_down(dn, 1, 8);
                    before = tq == 0 ? 1.f : before;
                    after = tq == 7 ? 1.f : after;
#pragma unroll
                    for (int j = 0; j < 4; ++j) { pre[j][i] *= before; suf[j][i] *= after; }
                }
            }
            // token-major: forward gamma K (and gamma Q), reverse (gamma_C / gamma) K; key-major: the other way round
            const int pc = kpos(CH * cq), pt = kpos(4 * tq);
            auto put_row = [&](auto& arr, const float* x, int row) {        // CH adjacent key rows of a token
                float m[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) m[i] = x[i];
#pragma unroll
                for (int pl = 0; pl < NP; ++pl) {
                    uint32_t* at = reinterpret_cast<uint32_t*>(&arr[pl][row][pc]);
                    at[0] = hi16_pair(m[0], m[1]);
#pragma unroll
                    for (int i = 0; i < CH; ++i) m[i] -= trunc_bf16(m[i]);
                }
            };
            auto put_col = [&](auto& arr, const float* x, int row) {        // four tokens of a key row
                u32x2 w[NP];
                split4<NP>(x, w);
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x2*>(&arr[i][row][pt]) = w[i];
            };
            float kt[CH][4], qt[CH][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a[CH], bq[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const float kv = kx[j].at(i);
                    a[i] = kv * (KDA ? (REV ? suf[j][i] : pre[j][i]) : 1.f);
                    kt[i][j] = kv * (KDA ? (REV ? pre[j][i] : suf[j][i]) : 1.f);
                    if constexpr (MODE != kScanKeep) bq[i] = qt[i][j] = qx[j].at(i) * (KDA ? pre[j][i] : 1.f);
                }
                put_row(s.k, a, 4 * tq + j);
                if constexpr (OUT) put_row(s.q, bq, 4 * tq + j);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                put_col(s.kt, kt[i], CH * cq + i);
                if constexpr (REV) put_col(s.qt, qt[i], CH * cq + i);
            }
        }
        float xin[2][4];                             // v (forward) or dy (reverse)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) xin[t][r] = val1<DT>(xn[t][r]);
        lds_barrier();
        if (ci + 1 < nc) fetch(REV ? c - 1 : c + 1);

        if constexpr (!OUT) {                        // the backward pass reads the states at the chunk borders
            float* keep = (REV ? p.gt : p.st) + id * (size_t)DK * dv;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) keep[(uint32_t)((16 * t + 4 * g + r) * dv + col)] = S[t][r];
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
                mma(z[t], lds_frag<NP>(&s.k[0][0][0], 32 * LDK, off), sf);
                if constexpr (OUT) mma(yq[t], lds_frag<NP>(&s.q[0][0][0], 32 * LDK, off), sf);
            }
        }
        float pre[2][4], suf[2][4], be[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                pre[t][r] = KDA ? 1.f : s.pre[16 * t + 4 * g + r];
                suf[t][r] = KDA ? 1.f : s.suf[16 * t + 4 * g + r];
                be[t][r] = s.beta[16 * t + 4 * g + r];
            }
        auto mat = [&](int which, int t) { return lds_frag<3>(&s.m[0][0], 512, which * kMatShorts + t * 1536 + 8 * l); };
        float w8[8];
        if constexpr (!REV) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = xin[e >> 2][e & 3] - pre[e >> 2][e & 3] * z[e >> 2][e & 3];
            const Frag<3> rf = split8<3>(w8);
            f32x4 ev[2] = {zero, zero};
#pragma unroll
            for (int t = 0; t < 2; ++t) mma(ev[t], mat(0, t), rf);
            if constexpr (MODE == kScanKeep) {
                const Window we(p.e + tok0 * H * dv, (uint32_t)rem * H * dv * 4);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        win_store1<SQ_DTYPE_F32>(we, ((16 * t + 4 * g + r) * H * dv + h * dv + col) * 4, ev[t][r]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = ev[e >> 2][e & 3] * be[e >> 2][e & 3];
            if constexpr (OUT) {
                const Frag<3> uf = split8<3>(w8);
                const uint32_t ys = (uint32_t)p.y.stride * ES, yo = 4 * g * ys + (h * dv + col) * ES;
                const Window wy(static_cast<const char*>(p.y.p) + tok0 * ys, (uint32_t)rem * ys);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 y;
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = yq[t][r] * pre[t][r];
                    mma(y, mat(1, t), uf);
#pragma unroll
                    for (int r = 0; r < 4; ++r) win_store1<DT>(wy, yo + (16 * t + r) * ys, y[r]);
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
                for (int r = 0; r < 4; ++r) S[t][r] *= s.last[KDA ? 16 * t + 4 * g + r : 0];
                mma(S[t], lds_frag<NP>(&s.kt[0][0][0], DK * LDT, (16 * t + n) * LDT + 8 * g), uf);
            }
        } else {
            // R = (gamma_C / gamma) K G + P^T dy;  du = T^T R;  G <- gamma_C G + (gamma Q)^T dy - (gamma K)^T (beta du)
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = xin[e >> 2][e & 3];
            const Frag<NPL> dyf = split8<NPL>(w8);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) z[t][r] *= suf[t][r];
                mma(z[t], mat(1, t), dyf);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w8[e] = z[e >> 2][e & 3];
            const Frag<3> rf = split8<3>(w8);
            f32x4 du[2] = {zero, zero};
#pragma unroll
            for (int t = 0; t < 2; ++t) mma(du[t], mat(0, t), rf);
            float q8[8];
            const uint32_t vs = (uint32_t)p.dvv.stride * ES, vo = 4 * g * vs + (h * dv + col) * ES;
            const Window wd(p.du + tok0 * H * dv, (uint32_t)rem * H * dv * 4);
            const Window wv(static_cast<const char*>(p.dvv.p) + tok0 * vs, (uint32_t)rem * vs);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float w = du[t][r] * be[t][r];
                    win_store1<SQ_DTYPE_F32>(wd, ((16 * t + 4 * g + r) * H * dv + h * dv + col) * 4, du[t][r]);
                    win_store1<DT>(wv, vo + (16 * t + r) * vs, w);
                    w8[4 * t + r] = -w * pre[t][r];
                    q8[4 * t + r] = xin[t][r] * pre[t][r];
                }
            const Frag<3> wf = split8<3>(w8);
            const Frag<KDA ? NPL : 3> qf = split8<KDA ? NPL : 3>(q8);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] *= s.last[KDA ? 16 * t + 4 * g + r : 0];
                const int off = (16 * t + n) * LDT + 8 * g;
                mma(S[t], lds_frag<NP>(&s.qt[0][0][0], DK * LDT, off), qf);
                mma(S[t], lds_frag<NP>(&s.kt[0][0][0], DK * LDT, off), wf);
            }
        }
    }
    float* fin = REV ? p.ds0 : OUT ? p.s1 : nullptr;
    if (fin) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) fin[sbase + (size_t)(16 * t + 4 * g + r) * dv] = S[t][r];
    }
}

template <int DK, int DT, bool KDA>
__global__ void __launch_bounds__(4 * DK) k_scan(const ScanParams p) {
    __shared__ __align__(16) ScanLds<DK, KDA ? 3 : planes_of(DT), kScanOut> s;
    scan_body<DK, DT, KDA, kScanOut>(p, blockIdx.x, s);
}

// The two scans of the backward pass, which do not depend on each other, side by side in one launch.
template <int DK, int DT, bool KDA>
__global__ void __launch_bounds__(4 * DK) k_scan_both(const ScanParams p, unsigned n_rev) {
    constexpr int NP = KDA ? 3 : planes_of(DT);
    __shared__ __align__(16) union U {
        ScanLds<DK, NP, kScanKeep> f;
        ScanLds<DK, NP, kScanRev> r;
    } s;
    // the reverse scans are the longer ones: they start first
    if (blockIdx.x < n_rev) scan_body<DK, DT, KDA, kScanRev>(p, blockIdx.x, s.r);
    else scan_body<DK, DT, KDA, kScanKeep>(p, blockIdx.x - n_rev, s.f);
}

// ---------------------------------------------------------------- launchers

template <int DK, int DT, bool KDA>
static hipError_t prep_t(const ScanParams& p, bool backward, hipStream_t s) {
    const int64_t blocks = (p.n_slots * p.n_heads + kPrepWaves - 1) / kPrepWaves;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), blk(kPrepWaves * 64);
    if (backward) k_prep<DK, DT, KDA, true><<<grid, blk, 0, s>>>(p);
    else k_prep<DK, DT, KDA, false><<<grid, blk, 0, s>>>(p);
    return hipGetLastError();
}

template <int DK, int DT, bool KDA>
static hipError_t scan_t(const ScanParams& p, bool backward, hipStream_t s) {
    if (p.dv % DK != 0) return hipErrorInvalidValue;
    const int64_t blocks = (int64_t)p.n_seq * p.n_heads * (p.dv / DK) * (backward ? 2 : 1);
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), blk(4 * DK);
    if (backward) k_scan_both<DK, DT, KDA><<<grid, blk, 0, s>>>(p, (unsigned)(blocks / 2));
    else k_scan<DK, DT, KDA><<<grid, blk, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_scan_prep(const ScanParams& p, bool backward, hipStream_t s) { SQ_SCAN_DISPATCH(prep_t, p, backward, s); }
hipError_t launch_scan(const ScanParams& p, bool backward, hipStream_t s) { SQ_SCAN_DISPATCH(scan_t, p, backward, s); }

}  // namespace sq
