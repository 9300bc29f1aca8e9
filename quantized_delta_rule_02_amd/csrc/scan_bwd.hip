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

template <int DK, int NPL, bool KDA>
__global__ void __launch_bounds__(DK * 4) k_grad(const ScanParams p) {
    constexpr int NW = DK / 16, NT = NW * 64;
    constexpr int VB = DK == 16 ? 16 : 64, VBP = VB < 32 ? 32 : VB, LDV = VBP + 8;   // value columns staged at a time
    constexpr int OCT = VB / 8, JOBS = (6 + NW - 1) / NW;
    static_assert(32 * OCT <= NT, "one staging unit per thread");
    __shared__ __align__(16) uint16_t s_dy[NPL][32][LDV], s_u[3][32][LDV], s_w[3][32][LDV];
    __shared__ __align__(16) float s_b1[32][36], s_b2[32][36];
    __shared__ float s_e[KDA ? 1 : 32][33], s_gam[KDA ? 1 : 32][33];
    __shared__ float s_row[NW][32], s_col[NW][32], s_corner[NW], s_pre[32], s_suf[32];

    const int tid = (int)threadIdx.x, wave = tid >> 6, l = tid & 63, n = l & 15, g = l >> 4;
    const int H = p.n_heads, Hk = p.n_heads_k, dv = p.dv, grp = H / Hk;
    const int hk = (int)(blockIdx.x % (unsigned)Hk);
    const int64_t slot = blockIdx.x / (unsigned)Hk;
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_slot(sequence(p, mid), mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    const Seq seq = sequence(p, lo);
    const int64_t c0 = (slot - first_slot(seq, lo)) * kChunk;
    if (c0 < 0 || c0 >= seq.len) return;             // a slot that no chunk uses (the whole workgroup leaves)
    const int rem = (int)(seq.len - c0 < kChunk ? seq.len - c0 : kChunk);
    const int64_t tok0 = seq.start + c0;
    const int d = 16 * wave + n;                     // this lane's key row

    float kv[2][4], qv[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = 16 * t + 4 * g + r;
            kv[t][r] = tok < rem ? load1(p.k.p, p.dtype, (tok0 + tok) * p.k.stride + hk * DK + d) : 0.f;
            qv[t][r] = tok < rem ? load1(p.q.p, p.dtype, (tok0 + tok) * p.q.stride + hk * DK + d) : 0.f;
        }
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};
    f32x4 dq[2] = {zero, zero}, dk[2] = {zero, zero};
    if constexpr (VB < 32) {                         // the unused half of a block of 32 value columns stays zero
        for (int i = tid; i < 3 * 32 * LDV; i += NT) {
            (&s_u[0][0][0])[i] = 0;
            (&s_w[0][0][0])[i] = 0;
            if (i < NPL * 32 * LDV) (&s_dy[0][0][0])[i] = 0;
        }
    }

    for (int gi = 0; gi < grp; ++gi) {
        const int h = hk * grp + gi;
        const size_t id = (size_t)slot * H + h;
        __syncthreads();                             // the previous head's LDS contents have been read
        float pre[2][4], suf[2][4], al[2][4], last = 1.f;
        if constexpr (!KDA) {
            if (wave == 0) {
                const int t = l & 31;
                const float a = t < rem ? fmaxf(p.gate[(tok0 + t) * H + h], kGateMin) : 1.f;
                float pr = a, sf = a, x = 0.f;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float up = __shfl_up(pr, o, 32), dn = __shfl_down(sf, o, 32);
                    if (t >= o) pr *= up;
                    if (t + o < 32) sf *= dn;
                }
                sf = __shfl_down(sf, 1, 32);
                for (int i = 0; i < 32; ++i) {
                    const float ai = __shfl(a, i, 32);
                    x = i == t ? 1.f : x * ai;
                    if (l < 32) s_gam[i][t] = x;
                }
                if (l < 32) {
                    s_pre[t] = pr;
                    s_suf[t] = t == 31 ? 1.f : sf;
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = 16 * t + 4 * g + r;
                    al[t][r] = tok < rem ? fmaxf(p.gate[((tok0 + tok) * H + h) * DK + d], kGateMin) : 1.f;
                }
        }
        f32x4 x1[2] = {zero, zero}, x2[2] = {zero, zero}, x3[2] = {zero, zero}, bj[JOBS];
#pragma unroll
        for (int j = 0; j < JOBS; ++j) bj[j] = zero;
        float corner = 0.f, dbeta = 0.f;
        const int oct = tid % OCT, stok = tid / OCT;             // staging: token and eight value columns of this thread
        const bool stage = tid < 32 * OCT, slive = stage && stok < rem;
        const float sbeta = slive ? p.beta[(tok0 + stok) * H + h] : 0.f;
        for (int vb = 0; vb < dv; vb += VB) {
            if (vb) __syncthreads();
            if (stage) {
                float y8[8], e8[8], u8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y8[j] = e8[j] = u8[j] = 0.f;
                if (slive) {
                    const int64_t at = ((tok0 + stok) * H + h) * dv + vb + 8 * oct;
                    load8(p.dy.p, p.dtype, (tok0 + stok) * p.dy.stride + (int64_t)h * dv + vb + 8 * oct, y8);
                    load8(p.e, SQ_DTYPE_F32, at, e8);
                    load8(p.du, SQ_DTYPE_F32, at, u8);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dbeta = fmaf(e8[j], u8[j], dbeta);
                    e8[j] *= sbeta;
                    u8[j] *= sbeta;
                }
                const Frag<NPL> fy = split8<NPL>(y8);
                const Frag<3> fu = split8<3>(e8), fw = split8<3>(u8);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    if (i < NPL) *reinterpret_cast<u32x4v*>(&s_dy[i < NPL ? i : 0][stok][8 * oct]) = fy.p[i < NPL ? i : 0];
                    *reinterpret_cast<u32x4v*>(&s_u[i][stok][8 * oct]) = fu.p[i];
                    *reinterpret_cast<u32x4v*>(&s_w[i][stok][8 * oct]) = fw.p[i];
                }
            }
            __syncthreads();
#pragma unroll
            for (int kb = 0; kb < VBP / 32; ++kb) {
                auto frag = [&](auto& arr, int t) {
                    constexpr int N = sizeof(arr) / (32 * LDV * 2);
                    Frag<N> f;
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        f.p[i] = *reinterpret_cast<const u32x4v*>(&arr[i][16 * t + n][32 * kb + 8 * g]);
                    return f;
                };
                float sv[8], gv[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) sv[j] = gv[j] = 0.f;
                if (32 * kb + 8 * g < VB) {
                    const int64_t at = ((int64_t)id * DK + d) * dv + vb + 32 * kb + 8 * g;
                    load8(p.st, SQ_DTYPE_F32, at, sv);
                    load8(p.gt, SQ_DTYPE_F32, at, gv);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) corner = fmaf(sv[j], gv[j], corner);
                const Frag<3> sf = split8<3>(sv), gf = split8<3>(gv);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    mma(x1[t], frag(s_dy, t), sf);
                    mma(x2[t], frag(s_w, t), sf);
                    mma(x3[t], frag(s_u, t), gf);
                }
#pragma unroll
                for (int j = 0; j < JOBS; ++j) {
                    const int jb = wave + NW * j;                // tiles (0,0), (1,0), (1,1) of B1, then of B2
                    if (jb < 6) {
                        const int tl = jb % 3, ti = tl > 0, tj = tl > 1;
                        const Frag<3> uf = frag(s_u, tj);
                        if (jb < 3) mma(bj[j], frag(s_dy, ti), uf);
                        else mma(bj[j], frag(s_w, ti), uf);
                    }
                }
            }
        }
        if (stage) {
#pragma unroll
            for (int o = 1; o < OCT; o <<= 1) dbeta += __shfl_xor(dbeta, o);
            if (slive && oct == 0) p.dbeta[(tok0 + stok) * H + h] = dbeta;
        }
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const int jb = wave + NW * j;
            if (jb < 6) {
                const int tl = jb % 3, ti = tl > 0, tj = tl > 1;
                float(&out)[32][36] = jb < 3 ? s_b1 : s_b2;
#pragma unroll
                for (int r = 0; r < 4; ++r) out[16 * ti + 4 * g + r][16 * tj + n] = bj[j][r];
            }
        }
        if constexpr (!KDA) {
            // sums over the key rows of the terms with the chunk's first state and last gradient
            float rowv[2][4], colv[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    rowv[t][r] = qv[t][r] * x1[t][r] - kv[t][r] * x2[t][r];
                    colv[t][r] = kv[t][r] * x3[t][r];
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) {
                        rowv[t][r] += __shfl_xor(rowv[t][r], o);
                        colv[t][r] += __shfl_xor(colv[t][r], o);
                    }
                    if (n == 0) {
                        s_row[wave][16 * t + 4 * g + r] = rowv[t][r];
                        s_col[wave][16 * t + 4 * g + r] = colv[t][r];
                    }
                }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) corner += __shfl_xor(corner, o);
            if (l == 0) s_corner[wave] = corner;
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    pre[t][r] = s_pre[16 * t + 4 * g + r];
                    suf[t][r] = s_suf[16 * t + 4 * g + r];
                }
            const float* ap = p.mat_ap + id * 2048;
            for (int i = tid; i < 1024; i += NT) {   // E below the diagonal; B1 and B2 times Gamma, zero above it
                const int a = i >> 5, c = i & 31;
                const float gm = s_gam[a][c], b1 = c <= a ? s_b1[a][c] : 0.f, b2 = c < a ? s_b2[a][c] : 0.f;
                s_e[a][c] = c < a ? ap[1024 + i] * b1 - ap[i] * b2 : 0.f;
                s_b1[a][c] = b1 * gm;
                s_b2[a][c] = b2 * gm;
            }
            __syncthreads();
            const Frag<3> kf = split8<3>(&kv[0][0]), qf = split8<3>(&qv[0][0]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float m1[8], m1t[8], ms[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 16 * t + n, j = 16 * (e >> 2) + 4 * g + (e & 3);
                    m1[e] = s_b1[i][j];
                    m1t[e] = s_b1[j][i];
                    ms[e] = -(s_b2[i][j] + s_b2[j][i]);          // one of the two is zero
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dq[t][r] = fmaf(pre[t][r], x1[t][r], dq[t][r]);
                    dk[t][r] += suf[t][r] * x3[t][r] - pre[t][r] * x2[t][r];
                }
                mma(dq[t], split8<3>(m1), kf);
                mma(dk[t], split8<3>(m1t), qf);
                mma(dk[t], split8<3>(ms), kf);
            }
            if (wave == 0 && l < 32) {
                float row = 0.f, colt = 0.f, cor = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) { row += s_row[w][l]; colt += s_col[w][l]; cor += s_corner[w]; }
                row *= s_pre[l];
                colt *= s_suf[l];
                cor *= s_pre[31];
                // row l: sums of E over the columns before each t, with the row's own term
                float f = row;
                for (int t = 0; t < 32; ++t) {
                    const float e = s_e[l][t];
                    s_e[l][t] = f;
                    f += e;
                }
                s_col[0][l] = colt;
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                float a = cor;
                for (int i = 0; i < 32; ++i) {
                    if (i >= l) a += s_e[i][l];
                    else a += s_col[0][i];
                }
                if (l < rem) {
                    const float alpha = fmaxf(p.gate[(tok0 + l) * H + h], kGateMin);
                    p.dgate[(tok0 + l) * H + h] = a / alpha;
                }
            }
        } else {
            corner += __shfl_xor(corner, 16);
            corner += __shfl_xor(corner, 32);
            __syncthreads();
            float full[2][4], dlog[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    pre[t][r] = full[t][r] = al[t][r];
                    suf[t][r] = 1.f;
                    dlog[t][r] = 0.f;
                    const int tok = 16 * t + 4 * g + r;          // the diagonal has no gate
                    const float b = s_b1[tok][tok];
                    dq[t][r] = fmaf(b, kv[t][r], dq[t][r]);
                    dk[t][r] = fmaf(b, qv[t][r], dk[t][r]);
                }
            // Pairs by the highest differing bit of their tokens (see k_prep): at level lev the rows of odd blocks of 2^lev
            // tokens meet the columns of the even block before.
            auto level = [&](auto tag) {
                constexpr int LEV = decltype(tag)::value;
                float kc[8], qr[8], kr[8];
                bool odd[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        odd[t][r] = ((16 * t + 4 * g + r) >> LEV) & 1;
                        kc[4 * t + r] = odd[t][r] ? 0.f : kv[t][r] * suf[t][r];
                        qr[4 * t + r] = odd[t][r] ? qv[t][r] * pre[t][r] : 0.f;
                        kr[4 * t + r] = odd[t][r] ? -kv[t][r] * pre[t][r] : 0.f;
                    }
                const Frag<3> fc = split8<3>(kc), fq = split8<3>(qr), fr = split8<3>(kr);
                float rowv[2][4], colv[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float r1[8], r2[8], c1[8], c2[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = 16 * t + n, j = 16 * (e >> 2) + 4 * g + (e & 3);
                        const bool pair = ((i ^ j) >> LEV) == 1;
                        const bool lower = pair && j < i, upper = pair && j > i;
                        r1[e] = lower ? s_b1[i][j] : 0.f;
                        r2[e] = lower ? s_b2[i][j] : 0.f;
                        c1[e] = upper ? s_b1[j][i] : 0.f;
                        c2[e] = upper ? s_b2[j][i] : 0.f;
                    }
                    f32x4 d1 = zero, d2 = zero, d3 = zero;
                    mma(d1, split8<3>(r1), fc);
                    mma(d2, split8<3>(r2), fc);
                    mma(d3, split8<3>(c1), fq);
                    mma(d3, split8<3>(c2), fr);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float a = pre[t][r] * d1[r], b = pre[t][r] * d2[r], c = suf[t][r] * d3[r];
                        if (odd[t][r]) {
                            dq[t][r] += a;
                            dk[t][r] -= b;
                        } else {
                            dk[t][r] += c;
                        }
                        rowv[t][r] = odd[t][r] ? qv[t][r] * a - kv[t][r] * b : 0.f;
                        colv[t][r] = odd[t][r] ? 0.f : kv[t][r] * c;
                    }
                }
                suffix_in<LEV>(rowv, g);
                prefix_before<LEV>(colv, g);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) dlog[t][r] += odd[t][r] ? rowv[t][r] : colv[t][r];
                // blocks of twice the size
                float other[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if constexpr (LEV < 2) other[t][r] = full[t][r ^ (1 << LEV)];
                        else if constexpr (LEV < 4) other[t][r] = __shfl_xor(full[t][r], 4 << LEV);
                        else other[t][r] = full[t ^ 1][r];
                    }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (odd[t][r]) pre[t][r] *= other[t][r];
                        else suf[t][r] *= other[t][r];
                        full[t][r] *= other[t][r];
                    }
            };
            level(std::integral_constant<int, 0>{});
            level(std::integral_constant<int, 1>{});
            level(std::integral_constant<int, 2>{});
            level(std::integral_constant<int, 3>{});
            level(std::integral_constant<int, 4>{});
            last = full[0][0];
            float rowv[2][4], colv[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float a = pre[t][r] * x1[t][r], b = pre[t][r] * x2[t][r], c = suf[t][r] * x3[t][r];
                    dq[t][r] += a;
                    dk[t][r] += c - b;
                    rowv[t][r] = qv[t][r] * a - kv[t][r] * b;
                    colv[t][r] = kv[t][r] * c;
                }
            suffix_in<5>(rowv, g);
            prefix_before<5>(colv, g);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = 16 * t + 4 * g + r;
                    if (tok < rem)
                        p.dgate[((tok0 + tok) * H + h) * DK + d] =
                            (dlog[t][r] + rowv[t][r] + colv[t][r] + last * corner) / al[t][r];
                }
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = 16 * t + 4 * g + r;
            if (tok < rem) {
                store1(p.dq.p, p.dtype, (tok0 + tok) * p.dq.stride + hk * DK + d, dq[t][r]);
                store1(p.dkk.p, p.dtype, (tok0 + tok) * p.dkk.stride + hk * DK + d, dk[t][r]);
            }
        }
}

template <int DK, int DT, bool KDA>
static hipError_t grad_t(const ScanParams& p, hipStream_t s) {
    constexpr int NPL = DT == SQ_DTYPE_BF16 ? 1 : DT == SQ_DTYPE_F16 ? 2 : 3;
    const int64_t blocks = p.n_slots * p.n_heads_k;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    k_grad<DK, NPL, KDA><<<dim3((unsigned)blocks), dim3(DK * 4), 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_scan_grad(const ScanParams& p, hipStream_t s) { SQ_SCAN_DISPATCH(grad_t, p, s); }

}  // namespace sq
