// Gradients of the gated delta scan, the part that is parallel over chunks (gfx950).
//
// Given, per chunk and head, the state S before the chunk, the gradient G of the state after it (k_scan's forward and
// reverse passes), e and du = G_t^T k_t for every token; u = beta e, w = beta du:
//
//   X1 = dY S^T, X2 = W S^T, X3 = U G^T;   B1_tj = dy_t . u_j (j <= t), B2_tj = w_t . u_j (j < t)
//   dq_t = gamma_t X1_t + sum_j Gamma_tj k_j B1_tj
//   dk_t = (gamma_C/gamma_t) X3_t - gamma_t X2_t + sum_{i>=t} Gamma_it q_i B1_it
//          - sum_{i>t} Gamma_it k_i B2_it - sum_{j<t} Gamma_tj k_j B2_tj
//   dbeta_t = du_t . e_t
//   alpha_t dalpha_t = the sum of all terms that hold alpha_t: pairs j < t <= i of
//          E_ij = Gamma_ij (q_i k_j B1_ij - k_i k_j B2_ij), rows i >= t of gamma_i (q_i X1_i - k_i X2_i), columns j < t of
//          (gamma_C/gamma_j) k_j X3_j, and gamma_C S.G  (per key row, or summed over the key rows for one gate per head).
// The last sum is taken over exactly those terms, not as a difference of running sums over all of them: each term is
// proportional to alpha_t, so that the quotient by alpha_t keeps its relative accuracy for small gates.
//
// One workgroup per (chunk, q/k head), a wave per 16 key rows; the value heads that share q and k follow one another and
// their dq and dk add up in registers, in a fixed order.
//
// Reads 128 KiB of states and gradients per chunk and head (128 x 128), 1.06 GB at 8190 tokens and 32 heads: 174 us at the rate
// of a copy; the launch takes 465 us there (one gate per head), 253 us at 3001 tokens with gates per key row.  Its 79 million
// vector instructions are 128 us at four cycles each on 1024 SIMDs, its 10 million products of 16 cycles 66; the rest is waiting
// for the states with two waves a SIMD.  The value heads of a q/k head come one after another, so a call of few chunks and q/k
// heads leaves CUs idle.  A wave per 32 key
// rows is as fast (480 us) with one gate per head and slower with a gate per key row (307 us), where its registers spill; 16 waves
// a CU (128 registers, spilling) take 589 and 367 us; all of a workgroup's states in flight at once (spilling) 677 and 322.
#include <hip/hip_runtime.h>

#include "scan_dev.h"

namespace sq {

// val[t][r] belongs to token 16 t + 4 g + r.  Inclusive suffix sums and exclusive prefix sums inside blocks of 2^LEV tokens.
template <int LEV>
__device__ __forceinline__ void suffix_in(float (&v)[2][4], int g) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if constexpr (LEV == 1) { v[t][0] += v[t][1]; v[t][2] += v[t][3]; }
        if constexpr (LEV >= 2) { v[t][2] += v[t][3]; v[t][1] += v[t][2]; v[t][0] += v[t][1]; }
    }
    if constexpr (LEV >= 3) {
        float tot[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float mine = v[t][0], o1 = __shfl_xor(mine, 16);
            float add = (g & 1) ? 0.f : o1;
            if constexpr (LEV >= 4) {
                const float pair = mine + o1, o2 = __shfl_xor(pair, 32);
                add += (g & 2) ? 0.f : o2;
                tot[t] = pair + o2;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) v[t][r] += add;
        }
        if constexpr (LEV >= 5) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[0][r] += tot[1];
        }
    }
}
template <int LEV>
__device__ __forceinline__ void prefix_before(float (&v)[2][4], int g) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if constexpr (LEV == 0) { v[t][0] = v[t][1] = v[t][2] = v[t][3] = 0.f; }
        if constexpr (LEV == 1) { v[t][1] = v[t][0]; v[t][3] = v[t][2]; v[t][0] = v[t][2] = 0.f; }
    }
    if constexpr (LEV >= 2) {
        float tot[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float a0 = v[t][0], a1 = a0 + v[t][1], a2 = a1 + v[t][2], mine = a2 + v[t][3];
            float add = 0.f;
            if constexpr (LEV >= 3) {
                const float o1 = __shfl_xor(mine, 16);
                add = (g & 1) ? o1 : 0.f;
                if constexpr (LEV >= 4) {
                    const float pair = mine + o1, o2 = __shfl_xor(pair, 32);
                    add += (g & 2) ? o2 : 0.f;
                    tot[t] = pair + o2;
                }
            }
            v[t][0] = add;
            v[t][1] = add + a0;
            v[t][2] = add + a1;
            v[t][3] = add + a2;
        }
        if constexpr (LEV >= 5) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[1][r] += tot[0];
        }
    }
}

template <int DK, int DT, bool KDA>
struct GradLds {
    static constexpr int NPL = planes_of(DT), NW = DK / 16;
    static constexpr int VB = DK, VBP = VB < 32 ? 32 : VB, LDV = VBP + 8;    // value columns staged at a time
    union {
        struct { uint16_t dy[NPL][32][LDV], u[3][32][LDV], w[3][32][LDV]; };
        // rows as A operands, three planes each.  GDN: M1 = Gamma B1, M1^T, -(M2 + M2^T) with M2 = Gamma B2;
        // KDA: B1 below the diagonal, its transpose, B2 and its transpose
        uint16_t m[KDA ? 4 : 3][3][32][40];
    };
    float b1[32][36], b2[32][36], e[KDA ? 1 : 32][36];
    float gt[2][KDA ? 1 : 6][32], row[NW][32], col[NW][32], corner[NW];
};

// Sixteen values of each of 16 neighbouring lanes n: lane n gets the lanes' sum of value n.
__device__ __forceinline__ float transpose_sum16(float (&v)[16], int n) {
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) {
        const bool up = n & m;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float a = pick(up, v[i + m], v[i]), b = pick(up, v[i], v[i + m]);
            v[i] = a + __shfl_xor(b, m);
        }
    }
    return v[0];
}

template <int DK, int DT, bool KDA>
__global__ void __launch_bounds__(DK * 4, DK < 64 ? 1 : 2) k_grad(const ScanParams p) {
    using Lds = GradLds<DK, DT, KDA>;
    constexpr int NPL = Lds::NPL, NW = Lds::NW, ND = DK / 16 / NW, NTHR = NW * 64, ES = DT == SQ_DTYPE_F32 ? 4 : 2;
    constexpr int VB = Lds::VB, VBP = Lds::VBP, LDV = Lds::LDV, OCT = VB / 8, UPT = 32 * OCT / NTHR, JOBS = (6 + NW - 1) / NW;
    __shared__ __align__(16) Lds s;

    const int tid = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = p.n_heads, Hk = p.n_heads_k, dv = p.dv, grp = H / Hk;
    const int hk = (int)(blockIdx.x % (unsigned)Hk);
    const int64_t slot = blockIdx.x / (unsigned)Hk;
    const ChunkAt ck = chunk_of_slot(p, slot);
    if (ck.rem <= 0) return;                         // a slot that no chunk uses (the whole workgroup leaves)
    const int rem = ck.rem;
    const int64_t tok0 = ck.tok0;
    const uint32_t ks = (uint32_t)p.k.stride * ES, qs = (uint32_t)p.q.stride * ES;
    const Window wk(static_cast<const char*>(p.k.p) + tok0 * ks, rem * ks), wq(static_cast<const char*>(p.q.p) + tok0 * qs, rem * qs);
    uint32_t kraw[ND][2][4], qraw[ND][2][4];
    auto kv = [&](int nd, int t, int r) { return val1<DT>(kraw[nd][t][r]); };
    auto qv = [&](int nd, int t, int r) { return val1<DT>(qraw[nd][t][r]); };
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};
    f32x4 dq[ND][2], dk[ND][2];
#pragma unroll
    for (int nd = 0; nd < ND; ++nd) dq[nd][0] = dq[nd][1] = dk[nd][0] = dk[nd][1] = zero;
    if constexpr (VB < 32) {                         // the unused half of a block of 32 value columns stays zero
        for (int i = tid; i < 3 * 32 * LDV; i += NTHR) {
            (&s.u[0][0][0])[i] = 0;
            (&s.w[0][0][0])[i] = 0;
            if (i < NPL * 32 * LDV) (&s.dy[0][0][0])[i] = 0;
        }
    }

    for (int gi = 0; gi < grp; ++gi) {
        const int h = hk * grp + gi;
        const int64_t id = slot * H + h;
        const int l = opaque(tid & 63), n = l & 15, g = l >> 4;
        const int d0 = 16 * ND * wave + n;           // this lane's key rows: d0 + 16 nd
        const Window ws(p.st + id * DK * dv, (uint32_t)(DK * dv) * 4), wg(p.gt + id * DK * dv, (uint32_t)(DK * dv) * 4);
        Raw<SQ_DTYPE_F32, 4> sn[ND][2], gn[ND][2];   // the next 32 value columns of S and G
        auto fetch_states = [&](int v0) {
            // blocks of 16 value columns: [dv / 16][DK][16]
            const int at = opaque((d0 + (g >> 1) * DK) * 16 + 8 * (g & 1)) + v0 * DK;
#pragma unroll
            for (int nd = 0; nd < ND; ++nd)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t off = (at + 16 * nd * 16 + 4 * i) * 4;
                    if (VB < 32 && 8 * g >= VB) off = 0xfffffff0u;
                    sn[nd][i].load(ws, off);
                    gn[nd][i].load(wg, off);
                }
        };
        fetch_states(0);
        uint32_t araw[KDA ? ND : 1][2][4];
        // k, q and the gates of this lane's key rows: needed after the products over the value columns, loaded during the last
        auto fetch_rows = [&] {
            const int g4 = opaque(4 * g);
            const Window wa(p.gate + tok0 * H * (KDA ? DK : 1), KDA ? (uint32_t)rem * H * DK * 4 : 0);
#pragma unroll
            for (int nd = 0; nd < ND; ++nd)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t tok = 16 * t + g4 + r, c = d0 + 16 * nd;
                        kraw[nd][t][r] = win_load1<DT>(wk, tok * ks + (hk * DK + c) * ES);
                        qraw[nd][t][r] = win_load1<DT>(wq, tok * qs + (hk * DK + c) * ES);
                        if constexpr (KDA) araw[KDA ? nd : 0][t][r] = win_load1<SQ_DTYPE_F32>(wa, (tok * H * DK + h * DK + c) * 4);
                    }
        };
        float alpha = 1.f;
        if (!KDA && wave == 0) {
            const int t = l & 31;
            alpha = t < rem ? fmaxf(p.gate[(tok0 + t) * H + h], kGateMin) : 1.f;
        }
        lds_barrier();                               // the previous head's LDS contents have been read
        if (VB < 32 && gi > 0) {                     // the unused halves were overwritten by the small matrices
            for (int i = tid; i < 3 * 32 * LDV; i += NTHR) {
                (&s.u[0][0][0])[i] = 0;
                (&s.w[0][0][0])[i] = 0;
                if (i < NPL * 32 * LDV) (&s.dy[0][0][0])[i] = 0;
            }
            lds_barrier();
        }
        if constexpr (!KDA) {
            if (wave == 0) {
                const int t = l & 31;
                GateLevels<float> lv(alpha);
#pragma unroll
                for (int lev = 0; lev < 6; ++lev) {
                    if (l < 32) {
                        s.gt[0][lev][t] = lv.pre;
                        s.gt[1][lev][t] = lv.suf;
                    }
                    if (lev < 5) lv.grow((t >> lev) & 1, __shfl_xor(lv.full, 1 << lev));
                }
            }
        }
        f32x4 x1[ND][2], x2[ND][2], x3[ND][2], bj[JOBS];
#pragma unroll
        for (int nd = 0; nd < ND; ++nd)
#pragma unroll
            for (int t = 0; t < 2; ++t) x1[nd][t] = x2[nd][t] = x3[nd][t] = zero;
#pragma unroll
        for (int j = 0; j < JOBS; ++j) bj[j] = zero;
        float corner[ND] = {}, dbeta[UPT] = {};
        const int oct = tid % OCT, stok = tid / OCT;             // staging: eight value columns of tokens stok + u NTHR / OCT
        const uint32_t ds = (uint32_t)p.dy.stride * ES;
        const Window wy(static_cast<const char*>(p.dy.p) + tok0 * ds, rem * ds), we(p.e + id * dv * kChunk, dv * kChunk * 4),
            wu(p.du + id * dv * kChunk, dv * kChunk * 4), wb(p.beta + tok0 * H, (uint32_t)rem * H * 4);
        float sbeta[UPT];
#pragma unroll
        for (int u = 0; u < UPT; ++u)
            sbeta[u] = __uint_as_float(win_load1<SQ_DTYPE_F32>(wb, ((stok + u * (NTHR / OCT)) * H + h) * 4));
        for (int vb = 0; vb < dv; vb += VB) {
            constexpr int RW = DT == SQ_DTYPE_F32 ? 2 : 1;
            Raw<DT, 8 / RW> yr[UPT][RW];
            Raw<SQ_DTYPE_F32, 4> er[UPT][2], ur[UPT][2];
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                const uint32_t tok = stok + u * (NTHR / OCT), c = h * dv + vb + 8 * oct;
#pragma unroll
                for (int i = 0; i < RW; ++i) yr[u][i].load(wy, tok * ds + (c + 4 * i) * ES);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // blocks of 16 value columns: [dv / 16][32][16], zero behind the sequence's end
                    const uint32_t o = (((vb + 8 * oct) >> 4) * (kChunk * 16) + tok * 16 + 8 * (oct & 1) + 4 * i) * 4;
                    er[u][i].load(we, o);
                    ur[u][i].load(wu, o);
                }
            }
            if (vb) lds_barrier();
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                const int tok = stok + u * (NTHR / OCT);
                float y8[8], e8[8], u8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y8[j] = RW == 2 ? yr[u][RW - 1 ? j >> 2 : 0].at(j & 3) : yr[u][0].at(j);
                    e8[j] = er[u][j >> 2].at(j & 3);
                    u8[j] = ur[u][j >> 2].at(j & 3);
                    dbeta[u] = fmaf(e8[j], u8[j], dbeta[u]);
                    e8[j] *= sbeta[u];
                    u8[j] *= sbeta[u];
                }
                const Frag<NPL> fy = split8<NPL>(y8);
                const Frag<3> fu = split8<3>(e8), fw = split8<3>(u8);
#pragma unroll
                for (int i = 0; i < NPL; ++i) *reinterpret_cast<u32x4v*>(&s.dy[i][tok][8 * oct]) = fy.p[i];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    *reinterpret_cast<u32x4v*>(&s.u[i][tok][8 * oct]) = fu.p[i];
                    *reinterpret_cast<u32x4v*>(&s.w[i][tok][8 * oct]) = fw.p[i];
                }
            }
            lds_barrier();
#pragma unroll 1
            for (int kb = 0; kb < VBP / 32; ++kb) {
                __builtin_amdgcn_sched_barrier(0);
                Raw<SQ_DTYPE_F32, 4> sc[ND][2], gc[ND][2];
#pragma unroll
                for (int nd = 0; nd < ND; ++nd)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sc[nd][i] = sn[nd][i];
                        gc[nd][i] = gn[nd][i];
                    }
                const int v1 = vb + 32 * (kb + 1);
                if (v1 < dv) fetch_states(v1);
                else fetch_rows();
                const int off = n * LDV + 32 * kb + 8 * g;
                {
                    Frag<3> f[ND];
#pragma unroll
                    for (int nd = 0; nd < ND; ++nd) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            v[j] = sc[nd][j >> 2].at(j & 3);
                            corner[nd] = fmaf(v[j], gc[nd][j >> 2].at(j & 3), corner[nd]);
                        }
                        f[nd] = split8<3>(v);
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const Frag<NPL> fy = lds_frag<NPL>(&s.dy[0][0][0], 32 * LDV, off + 16 * t * LDV);
#pragma unroll
                        for (int nd = 0; nd < ND; ++nd) mma<2>(x1[nd][t], fy, f[nd]);
                        const Frag<3> fw = lds_frag<3>(&s.w[0][0][0], 32 * LDV, off + 16 * t * LDV);
#pragma unroll
                        for (int nd = 0; nd < ND; ++nd) mma<2>(x2[nd][t], fw, f[nd]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);   // keeps the registers of the two halves apart
                {
                    Frag<3> f[ND];
#pragma unroll
                    for (int nd = 0; nd < ND; ++nd) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = gc[nd][j >> 2].at(j & 3);
                        f[nd] = split8<3>(v);
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const Frag<3> fu = lds_frag<3>(&s.u[0][0][0], 32 * LDV, off + 16 * t * LDV);
#pragma unroll
                        for (int nd = 0; nd < ND; ++nd) mma<2>(x3[nd][t], fu, f[nd]);
                    }
                }
#pragma unroll
                for (int j = 0; j < JOBS; ++j) {
                    const int jb = wave + NW * j;                // tiles (0,0), (1,0), (1,1) of B2, then of B1
                    if (jb < 6) {
                        const int tl = jb % 3, ti = tl > 0, tj = tl > 1;
                        const Frag<3> fu = lds_frag<3>(&s.u[0][0][0], 32 * LDV, off + 16 * tj * LDV);
                        const int oi = off + 16 * ti * LDV;
                        if (jb < 3) mma<2>(bj[j], lds_frag<3>(&s.w[0][0][0], 32 * LDV, oi), fu);
                        else mma<2>(bj[j], lds_frag<NPL>(&s.dy[0][0][0], 32 * LDV, oi), fu);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
#pragma unroll
            for (int o = 1; o < OCT; o <<= 1) dbeta[u] += __shfl_xor(dbeta[u], o);
            const int tok = stok + u * (NTHR / OCT);
            if (oct == 0 && tok < rem) p.dbeta[(tok0 + tok) * H + h] = dbeta[u];
        }
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const int jb = wave + NW * j;
            if (jb < 6) {
                const int tl = jb % 3, ti = tl > 0, tj = tl > 1;
                float(&out)[32][36] = jb < 3 ? s.b2 : s.b1;
#pragma unroll
                for (int r = 0; r < 4; ++r) out[16 * ti + 4 * g + r][16 * tj + n] = bj[j][r];
            }
        }
        constexpr int MPT = NTHR < 256 ? 256 / NTHR : 1;         // units (row, four columns) per thread
        if constexpr (!KDA) {
            // sums over the key rows of the terms with the chunk's first state and last gradient
            float sums[16];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float a = 0.f, c = 0.f;
#pragma unroll
                    for (int nd = 0; nd < ND; ++nd) {
                        a += qv(nd, t, r) * x1[nd][t][r] - kv(nd, t, r) * x2[nd][t][r];
                        c += kv(nd, t, r) * x3[nd][t][r];
                    }
                    sums[4 * t + r] = a;
                    sums[8 + 4 * t + r] = c;
                }
            const float mine = transpose_sum16(sums, n);
            (n < 8 ? s.row : s.col)[wave][16 * ((n >> 2) & 1) + 4 * g + (n & 3)] = mine;
            float cor = 0.f;
#pragma unroll
            for (int nd = 0; nd < ND; ++nd) cor += corner[nd];
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) cor += __shfl_xor(cor, o);
            if (l == 0) s.corner[wave] = cor;
        }
        lds_barrier();
        // the small matrices as A operands, over the staged rows
#pragma unroll 1
        for (int u = 0; u < MPT; ++u) {
            if (NTHR > 256 && tid >= 256) break;
            const int i = (tid + u * NTHR) >> 3, j0 = 4 * ((tid + u * NTHR) & 7);
            if constexpr (!KDA) {
                const float* ap = p.mat_ap + id * 2048 + i * 32 + j0;
                const f32x4 a4 = *reinterpret_cast<const f32x4*>(ap), p4 = *reinterpret_cast<const f32x4*>(ap + 1024);
                float m1[4], mt[4], ms[4];
                f32x4 e4;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + c, hi = i > j ? i : j, lo = i > j ? j : i;
                    const int lev = i == j ? 0 : 31 - __builtin_clz(i ^ j);
                    const float gm = i == j ? 1.f : s.gt[0][lev][hi] * s.gt[1][lev][lo];
                    const float v1 = s.b1[hi][lo], v2 = s.b2[hi][lo];
                    m1[c] = j <= i ? v1 * gm : 0.f;
                    mt[c] = j >= i ? v1 * gm : 0.f;
                    ms[c] = i == j ? 0.f : -v2 * gm;
                    e4[c] = j < i ? p4[c] * v1 - a4[c] * v2 : 0.f;
                }
                *reinterpret_cast<f32x4*>(&s.e[i][j0]) = e4;
                u32x2 w[3];
                auto put = [&](int which, const float* v) {
                    split4<3>(v, w);
#pragma unroll
                    for (int pl = 0; pl < 3; ++pl) *reinterpret_cast<u32x2*>(&s.m[which][pl][i][kpos32(j0)]) = w[pl];
                };
                put(0, m1);
                put(1, mt);
                put(2, ms);
            } else {
                float m[4][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + c, hi = i > j ? i : j, lo = i > j ? j : i;
                    const float v1 = s.b1[hi][lo], v2 = s.b2[hi][lo];
                    m[0][c] = j < i ? v1 : 0.f;
                    m[1][c] = j > i ? v1 : 0.f;
                    m[2][c] = j < i ? v2 : 0.f;
                    m[3][c] = j > i ? v2 : 0.f;
                }
                u32x2 w[3];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    split4<3>(m[q], w);
#pragma unroll
                    for (int pl = 0; pl < 3; ++pl) *reinterpret_cast<u32x2*>(&s.m[KDA ? q : 0][pl][i][kpos32(j0)]) = w[pl];
                }
            }
        }
        lds_barrier();
        auto mfrag = [&](int which, int t) { return lds_frag<3>(&s.m[which][0][0][0], 32 * 40, (16 * t + n) * 40 + 8 * g); };
        if constexpr (!KDA) {
            float pre[2][4], suf[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    pre[t][r] = s.gt[0][5][16 * t + 4 * g + r];
                    suf[t][r] = s.gt[1][5][16 * t + 4 * g + r];
                }
            Frag<NPL> kf[ND], qf[ND];
#pragma unroll
            for (int nd = 0; nd < ND; ++nd) {
                float k8[8], q8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    k8[e] = kv(nd, e >> 2, e & 3);
                    q8[e] = qv(nd, e >> 2, e & 3);
                }
                kf[nd] = split8<NPL>(k8);
                qf[nd] = split8<NPL>(q8);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const Frag<3> m1 = mfrag(0, t), mt = mfrag(1, t), ms = mfrag(2, t);
#pragma unroll
                for (int nd = 0; nd < ND; ++nd) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        dq[nd][t][r] = fmaf(pre[t][r], x1[nd][t][r], dq[nd][t][r]);
                        dk[nd][t][r] += suf[t][r] * x3[nd][t][r] - pre[t][r] * x2[nd][t][r];
                    }
                    mma<2>(dq[nd][t], m1, kf[nd]);
                    mma<2>(dk[nd][t], mt, qf[nd]);
                    mma<2>(dk[nd][t], ms, kf[nd]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (wave == 0) {
                // Sums of E over j < t: a product with the matrix of ones above the diagonal; then over i >= t
                Frag<3> ef[2];
                Frag<1> ones[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float v[8];
                    const f32x4 lo = *reinterpret_cast<const f32x4*>(&s.e[16 * t + n][8 * g]);
                    const f32x4 hi = *reinterpret_cast<const f32x4*>(&s.e[16 * t + n][8 * g + 4]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) { v[j] = lo[j]; v[4 + j] = hi[j]; }
                    ef[t] = split8<3>(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 8 * g + j < 16 * t + n ? 1.f : 0.f;
                    ones[t] = split8<1>(v);
                }
                float out[2] = {0.f, 0.f}, cor = 0.f;
                const float last = s.gt[0][5][31];
#pragma unroll
                for (int w = 0; w < NW; ++w) cor += s.corner[w];
#pragma unroll
                for (int ti = 0; ti < 2; ++ti) {
                    float row[4], col[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = 16 * ti + 4 * g + r;
                        row[r] = col[r] = 0.f;
#pragma unroll
                        for (int w = 0; w < NW; ++w) { row[r] += s.row[w][i]; col[r] += s.col[w][i]; }
                        row[r] *= pre[ti][r];
                        col[r] *= suf[ti][r];
                    }
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt) {
                        f32x4 f = zero;
                        mma<2>(f, ef[ti], ones[tt]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) out[tt] += pick(16 * ti + 4 * g + r >= 16 * tt + n, f[r] + row[r], col[r]);
                    }
                }
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    out[tt] += __shfl_xor(out[tt], 16);
                    out[tt] += __shfl_xor(out[tt], 32);
                }
                // lane t < 32 holds the gate of token t and writes its gradient
                if (l < rem) p.dgate[(tok0 + l) * H + h] = (pick(l < 16, out[0], out[1]) + cor * last) / alpha;
            }
        } else {
            // Pairs by the highest differing bit of their tokens (see k_prep): at level lev the rows of odd blocks of 2^lev
            // tokens meet the columns of the even block before.
            float dlog[ND][2][4], al[2][4];
            GateLevels<float> lv[2][4];
            auto gates = [&](int nd) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        al[t][r] = 16 * t + 4 * g + r < rem ? fmaxf(__uint_as_float(araw[KDA ? nd : 0][t][r]), kGateMin) : 1.f;
                        lv[t][r] = GateLevels<float>(al[t][r]);
                    }
            };
            auto odd = [&](int lev, int t, int r) { return ((16 * t + 4 * g + r) >> lev) & 1; };
            auto grow = [&](auto tag) {              // from blocks of 2^LEV tokens to twice that
                constexpr int LEV = decltype(tag)::value;
                float other[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if constexpr (LEV < 2) other[t][r] = lv[t][r ^ (1 << (LEV & 1))].full;
                        else if constexpr (LEV < 4) other[t][r] = __shfl_xor(lv[t][r].full, 4 << LEV);
                        else other[t][r] = lv[t ^ 1][r].full;
                    }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) lv[t][r].grow(odd(LEV, t, r), other[t][r]);
            };
            // the terms with the chunk's first state and last gradient, and the diagonal (which has no gate)
#pragma unroll
            for (int nd = 0; nd < ND; ++nd) {
                gates(nd);
                grow(std::integral_constant<int, 0>{});
                grow(std::integral_constant<int, 1>{});
                grow(std::integral_constant<int, 2>{});
                grow(std::integral_constant<int, 3>{});
                grow(std::integral_constant<int, 4>{});
                float cor = corner[nd], rowv[2][4], colv[2][4];
                cor += __shfl_xor(cor, 16);
                cor += __shfl_xor(cor, 32);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float a = lv[t][r].pre * x1[nd][t][r], b = lv[t][r].pre * x2[nd][t][r];
                        const float c = lv[t][r].suf * x3[nd][t][r], e = s.b1[16 * t + 4 * g + r][16 * t + 4 * g + r];
                        dq[nd][t][r] += fmaf(e, kv(nd, t, r), a);
                        dk[nd][t][r] += fmaf(e, qv(nd, t, r), c - b);
                        rowv[t][r] = qv(nd, t, r) * a - kv(nd, t, r) * b;
                        colv[t][r] = kv(nd, t, r) * c;
                    }
                suffix_in<5>(rowv, g);
                prefix_before<5>(colv, g);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) dlog[nd][t][r] = rowv[t][r] + colv[t][r] + lv[0][0].full * cor;
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int nd = 0; nd < ND; ++nd) {
                gates(nd);
                auto level = [&](auto tag) {
                    constexpr int LEV = decltype(tag)::value;
                    // rows come from odd blocks only, columns from even ones: the masks of the matrices leave nothing else
                    float kc[8], qr[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = e >> 2, r = e & 3;
                        kc[e] = kv(nd, t, r) * pick(odd(LEV, t, r), -lv[t][r].pre, lv[t][r].suf);
                        qr[e] = qv(nd, t, r) * lv[t][r].pre;
                    }
                    const Frag<3> fc = split8<3>(kc), fq = split8<3>(qr);
                    // which columns of this lane's row pair with it at this level: within its own 16 tokens below
                    // level 4, all of the other 16 at level 4
                    const int y = n ^ (4 * g);
                    auto on = [&](int r) { return ((y ^ r) >> (LEV < 4 ? LEV : 0)) == 1; };
                    const uint32_t k0 = (on(0) ? 0xffffu : 0u) | (on(1) ? 0xffff0000u : 0u);
                    const uint32_t k1 = (on(2) ? 0xffffu : 0u) | (on(3) ? 0xffff0000u : 0u);
                    auto frag = [&](int which, int t) {
                        Frag<3> f = mfrag(which, t);
#pragma unroll
                        for (int pl = 0; pl < 3; ++pl) {
                            const int keep = LEV < 4 ? t : 1 - t;
                            f.p[pl][2 * keep] &= LEV < 4 ? k0 : ~0u;
                            f.p[pl][2 * keep + 1] &= LEV < 4 ? k1 : ~0u;
                            f.p[pl][2 * (1 - keep)] = f.p[pl][2 * (1 - keep) + 1] = 0;
                        }
                        return f;
                    };
                    float rowv[2][4], colv[2][4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        f32x4 da = zero, db = zero, dc = zero;
                        if (LEV < 4 || t == 1) {
                            mma<2>(da, frag(0, t), fc);
                            mma<2>(db, frag(KDA ? 2 : 0, t), fc);
                        }
                        if (LEV < 4 || t == 0) {
                            mma<2>(dc, frag(1, t), fq);
                            mma<2>(dc, frag(KDA ? 3 : 0, t), fc);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float a = lv[t][r].pre * da[r], b = lv[t][r].pre * db[r], c = lv[t][r].suf * dc[r];
                            const bool o = odd(LEV, t, r);
                            dq[nd][t][r] += o ? a : 0.f;
                            dk[nd][t][r] += o ? -b : c;
                            rowv[t][r] = o ? qv(nd, t, r) * a - kv(nd, t, r) * b : 0.f;
                            colv[t][r] = o ? 0.f : kv(nd, t, r) * c;
                        }
                    }
                    suffix_in<LEV>(rowv, g);
                    prefix_before<LEV>(colv, g);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) dlog[nd][t][r] += pick(odd(LEV, t, r), rowv[t][r], colv[t][r]);
                    if constexpr (LEV < 4) grow(tag);
                    __builtin_amdgcn_sched_barrier(0);
                };
                level(std::integral_constant<int, 0>{});
                level(std::integral_constant<int, 1>{});
                level(std::integral_constant<int, 2>{});
                level(std::integral_constant<int, 3>{});
                level(std::integral_constant<int, 4>{});
                const Window wo(p.dgate + tok0 * H * DK, (uint32_t)rem * H * DK * 4);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        win_store1<SQ_DTYPE_F32>(wo, ((16 * t + 4 * g + r) * H * DK + h * DK + d0 + 16 * nd) * 4,
                                                 dlog[nd][t][r] / al[t][r]);
            }
        }
    }
    const int l = tid & 63, n = l & 15, g = l >> 4, d0 = 16 * ND * wave + n;
    const uint32_t os = (uint32_t)p.dq.stride * ES, oks = (uint32_t)p.dkk.stride * ES;
    const Window wdq(static_cast<const char*>(p.dq.p) + tok0 * os, rem * os);
    const Window wdk(static_cast<const char*>(p.dkk.p) + tok0 * oks, rem * oks);
#pragma unroll
    for (int nd = 0; nd < ND; ++nd)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t c = (hk * DK + d0 + 16 * nd) * ES;
                win_store1<DT>(wdq, (16 * t + 4 * g + r) * os + c, dq[nd][t][r]);
                win_store1<DT>(wdk, (16 * t + 4 * g + r) * oks + c, dk[nd][t][r]);
            }
}

template <int DK, int DT, bool KDA>
static hipError_t grad_t(const ScanParams& p, hipStream_t s) {
    const int64_t blocks = p.n_slots * p.n_heads_k;
    if (blocks > 0x7fffffff || p.dv % DK != 0) return hipErrorInvalidValue;
    k_grad<DK, DT, KDA><<<dim3((unsigned)blocks), dim3(DK * 4), 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_scan_grad(const ScanParams& p, hipStream_t s) { SQ_SCAN_DISPATCH(grad_t, p, s); }

}  // namespace sq
