// The chunked scan's preparation, and the scan of short sequences, which needs none (gfx950).  See scan.hip for the recurrence.
#include <hip/hip_runtime.h>

#include "scan_dev.h"

namespace sq {

// ---------------------------------------------------------------- short sequences

// Token by token, for a few drafted tokens, or one, per request.
//
// A state is read once and written once, 128 KiB a 128 x 128 state, and that is what bounds it: 64 x 32 states take 52 us,
// 5.1 TB/s, where the chunked scan, which keeps a CU's LDS and registers for one or two states whose loads, products and
// stores follow one another, takes 80 after its preparation's 15.  Here a wave owns 32 value columns of a state (a row's piece
// is one cache line of 128 bytes) and nothing else, without LDS and barriers: lane l holds the columns 4 (l & 7) .. + 3 of the
// key rows DK / 8 (l >> 3) .. + DK / 8 - 1.  Per token, with S' = D S,
//
//   u = beta (v - S'^T k);   y = S'^T q + (q . k) u;   S = S' + k u^T
//
// so that both products over the key rows are summed over the lanes in one round.  A token costs a wave some 330 vector
// instructions, which the memory traffic hides up to about eight tokens.

template <int DK, int DT, bool KDA>
__device__ __forceinline__ void short_sequences(const ScanParams& p, unsigned block) {
    constexpr int R = DK / 8, ES = DT == SQ_DTYPE_F32 ? 4 : 2, W = 16 / ES;      // key rows of a lane; elements per 16 bytes
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l = (int)threadIdx.x & 63, cl = l & 7, kl = l >> 3;
    const int H = p.n_heads, dv = p.dv, parts = dv / 32;
    const int64_t id = (int64_t)block * 4 + wave;
    const int64_t st = id / parts;
    if (st >= (int64_t)p.n_seq * H) return;
    const int col = (int)(id - st * parts) * 32 + 4 * cl, b = (int)(st / H), h = (int)(st - (int64_t)b * H), hk = h / (H / p.n_heads_k);
    const Seq sv = sequence(p, b);
    if (sv.len > p.short_len) return;                // the chunked scan's
    const int len = __builtin_amdgcn_readfirstlane((int)sv.len);
    const int64_t start = __builtin_amdgcn_readfirstlane((int)sv.start);

    // all addresses are one wave's base, a lane's 32-bit offset and a row's: none takes registers of its own
    const uint32_t at = (uint32_t)(kl * R * dv + col) * 4, bytes = (uint32_t)(DK * dv) * 4;
    f32x4 S[R];
    if (p.s0) {
        const Window w0(p.s0 + st * DK * dv, bytes);
#pragma unroll
        for (int j = 0; j < R; ++j) S[j] = __builtin_bit_cast(f32x4, (u32x4v)__builtin_amdgcn_raw_buffer_load_b128(w0.r, at, j * dv * 4, 0));
    } else {
        // not a window of no bytes: whether an offset is beyond it is decided by the lane's offset against its size less the
        // row's, which would be below zero here
#pragma unroll
        for (int j = 0; j < R; ++j) S[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    using Words = std::conditional_t<ES == 4, u32x4v, u32x2>;       // four elements
    struct Token {                                   // as loaded
        u32x4v k[R / W], q[R / W], a[KDA ? R / 4 : 1];
        Words v;
        float gate, beta;
    };
    auto load = [&](int64_t t) {
        Token x;
        const Window wk(static_cast<const char*>(p.k.p) + (t * p.k.stride + hk * DK) * ES, DK * ES);
        const Window wq(static_cast<const char*>(p.q.p) + (t * p.q.stride + hk * DK) * ES, DK * ES);
        const Window wv(static_cast<const char*>(p.v.p) + (t * p.v.stride + h * dv) * ES, dv * ES);
#pragma unroll
        for (int i = 0; i < R / W; ++i) {
            x.k[i] = __builtin_amdgcn_raw_buffer_load_b128(wk.r, kl * R * ES + 16 * i, 0, 0);
            x.q[i] = __builtin_amdgcn_raw_buffer_load_b128(wq.r, kl * R * ES + 16 * i, 0, 0);
        }
        if constexpr (ES == 4) x.v = __builtin_amdgcn_raw_buffer_load_b128(wv.r, col * ES, 0, 0);
        else x.v = __builtin_amdgcn_raw_buffer_load_b64(wv.r, col * ES, 0, 0);
        if constexpr (KDA) {
            const Window wa(p.gate + (t * H + h) * DK, DK * 4);
#pragma unroll
            for (int i = 0; i < R / 4; ++i) x.a[i] = __builtin_amdgcn_raw_buffer_load_b128(wa.r, kl * R * 4 + 16 * i, 0, 0);
        } else {
            x.gate = p.gate[t * H + h];
        }
        x.beta = p.beta[t * H + h];
        return x;
    };
    auto value = [](const auto& w, int j) {          // element j of 16-bit pairs or float32 words
        if constexpr (DT == SQ_DTYPE_F32) return __uint_as_float(w[j]);
        else return val1<DT>((j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
    };
    Token next;
    if (len > 0) next = load(start);
    for (int t = 0; t < len; ++t) {
        const Token x = next;
        if (t + 1 < len) next = load(start + t + 1);
        f32x4 sk{0.f, 0.f, 0.f, 0.f}, sq{0.f, 0.f, 0.f, 0.f};
        float qk = 0.f;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float kj = value(x.k[j / W], j % W), qj = value(x.q[j / W], j % W);
            S[j] *= KDA ? __uint_as_float(x.a[KDA ? j / 4 : 0][j & 3]) : x.gate;
            sk += kj * S[j];
            sq += qj * S[j];
            qk = fmaf(qj, kj, qk);
        }
#pragma unroll
        for (int m = 8; m < 64; m <<= 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sk[c] += __shfl_xor(sk[c], m);
                sq[c] += __shfl_xor(sq[c], m);
            }
            qk += __shfl_xor(qk, m);
        }
        f32x4 u;
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = x.beta * (value(x.v, c) - sk[c]);
#pragma unroll
        for (int j = 0; j < R; ++j) S[j] += value(x.k[j / W], j % W) * u;
        if (kl == 0) {
            const f32x4 y = sq + qk * u;
            const Window wy(static_cast<const char*>(p.y.p) + ((start + t) * p.y.stride + h * dv) * ES, dv * ES);
            if constexpr (DT == SQ_DTYPE_F32) {
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, y), wy.r, col * ES, 0, 0);
            } else {
                u32x2 w;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[i] = DT == SQ_DTYPE_BF16 ? round_pair(y[2 * i], y[2 * i + 1]) : f16_bits(y[2 * i]) | f16_bits(y[2 * i + 1]) << 16;
                __builtin_amdgcn_raw_buffer_store_b64(w, wy.r, col * ES, 0, 0);
            }
        }
    }
    if (p.s1) {
        const Window w1(p.s1 + st * DK * dv, bytes);
#pragma unroll
        for (int j = 0; j < R; ++j) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, S[j]), w1.r, at, j * dv * 4, 0);
    }
}

// ---------------------------------------------------------------- prep

constexpr int kPrepWaves = 4;
constexpr int kPrepLd = 36;          // 16-byte aligned rows, 4 banks apart

// One wave per chunk and head.  Its LDS is one 32 x 32 matrix (two for the backward pass), used in turn for I + N, for
// its inverse and for P, so that four and more waves fit on a SIMD: with all of them side by side (18 KiB a wave, two
// waves) the launch took 118 us where it now takes 61 (12301 tokens, 32 heads, bfloat16).
// SHORT: the workgroups from n_prep on take the short sequences (see above): the two do not depend on each other, and the few
// chunks beside many short sequences would leave most CUs idle.
template <int DK, int DT, bool KDA, bool BWD, bool SHORT>
__global__ void __launch_bounds__(kPrepWaves * 64, !SHORT ? 1 : DT == SQ_DTYPE_F32 || KDA ? 2 : 4) k_prep(const ScanParams p, unsigned n_prep) {
    if constexpr (SHORT) {
        if (blockIdx.x >= n_prep) {
            short_sequences<DK, DT, KDA>(p, blockIdx.x - n_prep);
            return;
        }
    }
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
    // Forward, a gate counts as it is (NaN stays NaN); the matrices of the backward pass are those of gates of at least kGateMin.
    auto counted = [](float a) { return BWD ? fmaxf(a, kGateMin) : a; };

    float(&M)[NM][32][kPrepLd] = s_m[wave];
    if (l < 32) s_b[wave][l] = l < rem ? p.beta[(tok0 + l) * H + h] : 0.f;
    if constexpr (!KDA) {
        const int t = l & 31;
        const float a = t < rem ? p.gate[(tok0 + t) * H + h] : 1.f;
        GateLevels<float> lv(counted(a));
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
#pragma unroll KDA ? 1 : NKB
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
            mma<2>(aA[0], kf[0], kf[0]); mma<2>(aP[0], qf[0], kf[0]);
            mma<2>(aA[1], kf[1], kf[0]); mma<2>(aP[1], qf[1], kf[0]);
            mma<2>(aA[2], kf[1], kf[1]); mma<2>(aP[2], qf[1], kf[1]);
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
                    lv[t][j] = GateLevels<float>(on ? counted(cur.a[t][KDA ? j >> 2 : 0].at(j & 3)) : 1.f);
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
                    mma<2>(ta, fk, fk);
                    mma<2>(tp, fq, fk);
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
            mma<2>(aA[1], fk, fc);
            mma<2>(aP[1], fq, fc);
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
    auto put = [&](uint16_t* mat, const float (&m)[32][kPrepLd], bool transposed, float scale0, float scale1) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {                // rows 16 t + n
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = 16 * (e >> 2) + 4 * g + (e & 3);
                v[e] = transposed ? m[c][16 * t + n] : m[16 * t + n][c] * pick(t, scale1, scale0);
            }
            const Frag<3> f = split8<3>(v);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl)
                *reinterpret_cast<u32x4v*>(mat + ((t * 3 + pl) * 64 + l) * 8) = f.p[pl];
        }
    };
    put(p.mat_f + id * (BWD ? 1 : 2) * kMatShorts, M[0], false, BWD ? 1.f : s_b[wave][n], BWD ? 1.f : s_b[wave][16 + n]);
    if constexpr (BWD) put(p.mat_r + id * 2 * kMatShorts, M[NM - 1], true, 1.f, 1.f);
    wave_sync();
#pragma unroll
    for (int tl = 0; tl < 3; ++tl)
#pragma unroll
        for (int r = 0; r < 4; ++r) M[0][16 * (tl > 0) + 4 * g + r][16 * (tl > 1) + n] = aP[tl][r];
#pragma unroll
    for (int r = 0; r < 4; ++r) M[0][4 * g + r][16 + n] = 0.f;   // the tile above the diagonal
    wave_sync();
    put(BWD ? p.mat_r + (id * 2 + 1) * kMatShorts : p.mat_f + (id * 2 + 1) * kMatShorts, M[0], BWD, 1.f, 1.f);
}

// ---------------------------------------------------------------- launchers

static int64_t prep_blocks(const ScanParams& p) { return (p.n_slots * p.n_heads + kPrepWaves - 1) / kPrepWaves; }

template <int DK, int DT, bool KDA>
static hipError_t prep_t(const ScanParams& p, bool backward, hipStream_t s) {
    const int64_t blocks = prep_blocks(p);
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), blk(kPrepWaves * 64);
    if (backward) k_prep<DK, DT, KDA, true, false><<<grid, blk, 0, s>>>(p, 0);
    else k_prep<DK, DT, KDA, false, false><<<grid, blk, 0, s>>>(p, 0);
    return hipGetLastError();
}

template <int DK, int DT, bool KDA>
static hipError_t short_t(const ScanParams& p, bool prep, hipStream_t s) {
    if constexpr (DK < 64) {
        return hipErrorInvalidValue;
    } else {
        if (p.dv % 32 != 0) return hipErrorInvalidValue;
        const int64_t n_prep = prep ? prep_blocks(p) : 0, blocks = n_prep + ((int64_t)p.n_seq * p.n_heads * (p.dv / 32) + 3) / 4;
        if (blocks > 0x7fffffff) return hipErrorInvalidValue;
        k_prep<DK, DT, KDA, false, true><<<dim3((unsigned)blocks), dim3(kPrepWaves * 64), 0, s>>>(p, (unsigned)n_prep);
        return hipGetLastError();
    }
}

hipError_t launch_scan_prep(const ScanParams& p, bool backward, hipStream_t s) { SQ_SCAN_DISPATCH(prep_t, p, backward, s); }
hipError_t launch_scan_short(const ScanParams& p, bool prep, hipStream_t s) { SQ_SCAN_DISPATCH(short_t, p, prep, s); }

}  // namespace sq
