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
// k_prep (scan_prep.hip): That and P of every chunk and head, one wave each, all chunks at once.
// k_scan: the recurrence over a sequence's chunks.  A wave owns 16 value columns of one state (the columns do not
// interact), in 4 registers per 16 x 16 tile; see scan_dev.h for why no register has to move between products.
#include <hip/hip_runtime.h>

#include "scan_dev.h"

namespace sq {

// ---------------------------------------------------------------- scan

// MODE: forward with outputs; forward for the backward pass (keeps e and the chunks' first states, no y);
// reverse (the gradient of the state from the last chunk to the first).
enum : int { kScanOut = 0, kScanKeep = 1, kScanRev = 2 };

// The scan's LDS: operands of a chunk.  What the first half of a step reads is there twice, so that the next chunk's can be
// written meanwhile; the key-major operands, read by the second half only, once.  Token-major rows are 4 banks apart,
// key-major ones 20.
template <int DK, int DT, bool KDA, int MODE, int NC>
struct ScanLds {
    static constexpr bool REV = MODE == kScanRev, OUT = MODE == kScanOut;
    static constexpr bool VL = DT != SQ_DTYPE_F32;       // v through LDS (there is no room for it in float32)
    static constexpr int NP = KDA ? 3 : planes_of(DT);   // planes of the operands (gates make them float32)
    // A y of 16 bits takes three planes too: what two leave out, 2^-16 of an operand, is above the rounding of a y that is small
    // against its terms.
    static constexpr int LDK = (DK < 32 ? 32 : DK) + 8, LDT = 40, NMAT = MODE == kScanKeep ? 1 : 2;
    // The chunk's matrices go through LDS where the operands are one or two planes (a prefill of one-plane operands that reads
    // them from memory: 288 -> 313 us).  With three, both copies (24 KiB) do not fit beside the 144 KiB of 16-bit rows with
    // a gate per key row, and LDS is what a step waits for most: the computing waves read them from memory, a step ahead.
    static constexpr bool ML = NP < 3;
    struct First {
        uint16_t k[NP][32][LDK];                         // token-major: gamma K forward, (gamma_C / gamma) K in reverse
        uint16_t q[OUT ? NP : 1][OUT ? 32 : 1][LDK];
        uint16_t m[ML ? NMAT : 1][ML ? kMatShorts : 8];  // That, P (forward); T^T, P^T (reverse)
        float pre[32], suf[32], beta[32];
    } first[2];
    uint16_t kt[NP][DK][LDT];                            // key-major: the other of the two K
    uint16_t qt[REV ? NP : 1][REV ? DK : 1][LDT];
    uint16_t v[VL ? 16 * NC : 1][LDT];                       // v (forward) or dy (reverse), value-major, the 16-bit inputs' bits
    float last[DK];                                      // all gates of the chunk
};

// One workgroup per 16 NC value columns of a state: NC waves compute, NS others bring the chunks' operands into LDS, one
// chunk ahead.  Two barriers a step: (1) the chunk's first operands and v are there and the key-major ones of the chunk
// before are free, (2) its key-major ones are there and v is free.
//
// A computing wave owns 16 value columns and keeps S in its registers.  A step is a chain (S, e, u, S) on one or two waves a
// SIMD, so its length is instructions issued, four cycles each, plus what the chain waits for.  Measured (one gate per head,
// bfloat16, 128 x 128): 2.2 us a step where a CU has one state's half to itself, 3.3 us a state where all CUs are full
// (12301 tokens in 7 prompts, 32 heads: 280 us).  The chain's own 309 vector instructions (200 of them split float32 operands)
// and 96 products of 16 cycles a step and wave are 1.2 us, 2.3 us for the two waves of a full SIMD; the rest is LDS latency
// and the barriers.  Forms that were slower when y took two planes (270 us then; 225 with the staging left out): loading and
// staging by the computing waves (309 us; KDA prefill 366 against 315), 32 columns a wave with 32x32x16 products (281 us, one
// prompt of 777 tokens 78 us against 60), LDS reads issued a block ahead (361 us: the registers for it leave room for one
// workgroup a CU).
template <int DK, int DT, bool KDA, int MODE, int NC>
struct Scan {
    using Lds = ScanLds<DK, DT, KDA, MODE, NC>;
    static constexpr bool REV = MODE == kScanRev, OUT = MODE == kScanOut, VL = Lds::VL;
    static constexpr int NPL = planes_of(DT), NP = Lds::NP;
    static constexpr int NT = DK / 16, NKB = (DK + 31) / 32, LDK = Lds::LDK, LDT = Lds::LDT, NMAT = Lds::NMAT;
    static constexpr bool ML = Lds::ML;
    static constexpr int NS = DK < 32 ? 1 : 4, NTHR = NS * 64, CH = 8 * DK / NTHR, ES = DT == SQ_DTYPE_F32 ? 4 : 2;
    static_assert(CH == 2 || CH == 4);

    const ScanParams& p;
    Lds& s;
    int H, b, h, sg, start, len, nc;
    int64_t slot0;

    __device__ __forceinline__ Scan(const ScanParams& p_, Lds& s_, unsigned block) : p(p_), s(s_) {
        H = p.n_heads;
        const int bh = (int)(block % (unsigned)(H * p.n_long));
        sg = (int)(block / (unsigned)(H * p.n_long));
        b = bh / H;
        h = bh % H;
        if (p.short_len >= 0) b = __builtin_amdgcn_readfirstlane(long_sequence(p, b));
        if (b < 0) return;                           // see run()
        const Seq sv = sequence(p, b);
        start = __builtin_amdgcn_readfirstlane((int)sv.start);
        len = __builtin_amdgcn_readfirstlane((int)sv.len);
        slot0 = (start >> 5) + b;
        nc = (len + kChunk - 1) / kChunk;
    }
    __device__ __forceinline__ int chunk(int i) const { return REV ? nc - 1 - i : i; }       // of step i
    __device__ __forceinline__ int tokens(int c) const { return len - c * kChunk < kChunk ? len - c * kChunk : kChunk; }
    __device__ __forceinline__ size_t id(int c) const { return (size_t)(slot0 + c) * H + h; }

    __device__ __forceinline__ void stage(int tid);
    __device__ __forceinline__ void compute(int wave, int l);
    __device__ __forceinline__ void run() {
        if (b < 0) return;                           // no such sequence: the whole workgroup leaves
        const int tid = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        if constexpr (DK < 32) {                     // the unused half of a block of 32 key rows stays zero
            for (int i = tid; i < 2 * NP * 32 * LDK; i += (NC + NS) * 64) {
                const int j = i % (NP * 32 * LDK);
                typename Lds::First& f = s.first[i / (NP * 32 * LDK)];
                (&f.k[0][0][0])[j] = 0;
                if (OUT) (&f.q[0][0][0])[j] = 0;
            }
            lds_barrier();
        }
        if (wave < NC) {
            __builtin_amdgcn_s_setprio(2);           // the chain goes before the staging on its SIMD
            compute(wave, tid & 63);
        } else {
            stage(tid - NC * 64);
        }
    }
};

// The staging waves: each thread brings 4 tokens x CH key rows of a chunk.
template <int DK, int DT, bool KDA, int MODE, int NC>
__device__ __forceinline__ void Scan<DK, DT, KDA, MODE, NC>::stage(int tid) {
    const int hk = h / (H / p.n_heads_k);
    // token quad and key rows of this thread; the gates' products run over the quads, eight neighbouring lanes (and so spread,
    // the LDS writes of both layouts meet no bank twice; with the key rows on neighbouring lanes the key-major ones met
    // each sixteen times)
    const int tq = tid & 7, cq = tid >> 3;
    const int pc = kpos32(CH * cq), pt = kpos32(4 * tq);
    constexpr int MU = ML ? NMAT * kMatShorts / 8 / NTHR : 0;   // 16-byte units of the matrices per thread, and some left
    constexpr int MR = ML ? NMAT * kMatShorts / 8 % NTHR : 0;
    u32x4v mx[MU + 1];
    Raw<DT, CH> kx[4], qx[4];
    Raw<SQ_DTYPE_F32, CH> ax[4];
    u32x2 ktw[CH][NP], qtw[REV ? CH : 1][NP];        // the key-major operands of the next second half
    float gb0 = 0.f, gb1 = 0.f, lastw[CH];
    // v: 4 tokens x 2 value columns per unit
    constexpr int VU = NC * 64 / NTHR;
    Raw<VL ? DT : SQ_DTYPE_BF16, 2> vx[VU][VL ? 4 : 1];
    const ScanRows& xr = REV ? p.dy : p.v;
    const int vq = tid & 7, vc = tid >> 3;
    const uint32_t xs = (uint32_t)xr.stride * ES, xo = 4 * vq * xs + (h * p.dv + sg * 16 * NC + 2 * vc) * ES;
    auto fetch_v = [&](int c) {
        if constexpr (VL) {
            const Window wx(static_cast<const char*>(xr.p) + (start + (int64_t)c * kChunk) * xs, tokens(c) * xs);
#pragma unroll
            for (int u = 0; u < VU; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) vx[u][j].load(wx, xo + j * xs + u * (NTHR / 4) * ES);
        }
    };
    auto put_v = [&] {
        if constexpr (VL) {
#pragma unroll
            for (int u = 0; u < VU; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    u32x2 w;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w[j] = __builtin_amdgcn_perm(vx[u][2 * j + 1].w[0], vx[u][2 * j].w[0], i ? 0x07060302u : 0x05040100u);
                    *reinterpret_cast<u32x2*>(&s.v[2 * vc + i + u * (NTHR / 4)][kpos32(4 * vq)]) = w;
                }
        }
    };
    const uint32_t ks = (uint32_t)p.k.stride * ES, qs = (uint32_t)p.q.stride * ES, gs = (uint32_t)H * DK * 4;
    const uint32_t ko = 4 * tq * ks + (hk * DK + CH * cq) * ES, qo = 4 * tq * qs + (hk * DK + CH * cq) * ES;
    const uint32_t go = 4 * tq * gs + (h * DK + CH * cq) * 4;
    auto fetch = [&](int c) {                        // chunk c into registers
        const int64_t tok0 = start + (int64_t)c * kChunk;
        const uint32_t rem = tokens(c);
        const Window wk(static_cast<const char*>(p.k.p) + tok0 * ks, rem * ks);
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
            gb0 = p.mat_gb[id(c) * 64 + tid];        // the products of the gates, from k_prep
        }
        if (tid < 32) {
            const Window wb(p.beta + tok0 * H, rem * H * 4);
            gb1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(wb.r, (tid * H + h) * 4, 0, 0));
        }
        if constexpr (ML) {
            const u32x4v* m = reinterpret_cast<const u32x4v*>((REV ? p.mat_r : p.mat_f) + id(c) * (NMAT * kMatShorts));
#pragma unroll
            for (int u = 0; u < MU; ++u) mx[u] = m[tid + u * NTHR];
            if (MR && tid < MR) mx[MU] = m[tid + MU * NTHR];
        }
    };
    auto put_first = [&](int c, typename Lds::First& f) {        // what the first half of a step reads; makes ktw, qtw, lastw
        const int rem = tokens(c);
        if (!KDA && tid < 64) (&f.pre[0])[tid] = gb0;            // pre, then suf
        if (tid < 32) f.beta[tid] = gb1;
        if (!KDA) lastw[0] = gb0;                                // thread 31: pre of the last token
        if constexpr (ML) {
#pragma unroll
            for (int u = 0; u < MU; ++u) *reinterpret_cast<u32x4v*>(&f.m[0][0] + (tid + u * NTHR) * 8) = mx[u];
            if (MR && tid < MR) *reinterpret_cast<u32x4v*>(&f.m[0][0] + (tid + MU * NTHR) * 8) = mx[MU];
        }
        if constexpr (!KDA && DT == SQ_DTYPE_BF16) {             // the inputs' bits as they are
            auto rows = [&](auto& arr, const Raw<DT, CH>* x) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t* to = reinterpret_cast<uint32_t*>(&arr[0][4 * tq + j][pc]);
                    if constexpr (CH == 4) *reinterpret_cast<u32x2*>(to) = u32x2{x[j].w[0], x[j].w[CH / 2 - 1]};
                    else to[0] = x[j].w[0];
                }
            };
            auto cols = [&](auto& out, const Raw<DT, CH>* x) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        out[i][0][j] = __builtin_amdgcn_perm(x[2 * j + 1].w[i / 2], x[2 * j].w[i / 2], (i & 1) ? 0x07060302u : 0x05040100u);
            };
            rows(f.k, kx);
            cols(ktw, kx);
            if constexpr (OUT) rows(f.q, qx);
            if constexpr (REV) cols(qtw, qx);
        } else {
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
                    GateLevels<float> lv(pre[3][i]);             // over the eight token quads
                    float before = 1.f;
#pragma unroll
                    for (int o = 0; o < 3; ++o) {
                        const bool odd = (tq >> o) & 1;
                        const float other = __shfl_xor(lv.full, 1 << o);
                        before = odd ? before * other : before;
                        lv.grow(odd, other);
                    }
                    lastw[i] = lv.full;
#pragma unroll
                    for (int j = 0; j < 4; ++j) { pre[j][i] *= before; suf[j][i] *= lv.suf; }
                }
            }
            // token-major: forward gamma K (and gamma Q), reverse (gamma_C / gamma) K; key-major: the other way round
            auto put_row = [&](auto& arr, const float* x, int row) {   // CH adjacent key rows of a token
                if constexpr (CH == 4) {
                    u32x2 w[NP];
                    split4<NP>(x, w);
#pragma unroll
                    for (int pl = 0; pl < NP; ++pl) *reinterpret_cast<u32x2*>(&arr[pl][row][pc]) = w[pl];
                } else {
                    float a = x[0], b2 = x[1];
#pragma unroll
                    for (int pl = 0; pl < NP; ++pl) {
                        const uint32_t w = round_pair(a, b2);
                        *reinterpret_cast<uint32_t*>(&arr[pl][row][pc]) = w;
                        if (pl + 1 < NP) rest_pair(w, a, b2);
                    }
                }
            };
            float kt[CH][4], qt[CH][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a[CH], bq[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const float kv = kx[j].at(i);
                    a[i] = kv * (KDA ? pick(REV, suf[j][i], pre[j][i]) : 1.f);
                    kt[i][j] = kv * (KDA ? pick(REV, pre[j][i], suf[j][i]) : 1.f);
                    if constexpr (MODE != kScanKeep) bq[i] = qt[i][j] = qx[j].at(i) * (KDA ? pre[j][i] : 1.f);
                }
                put_row(f.k, a, 4 * tq + j);
                if constexpr (OUT) put_row(f.q, bq, 4 * tq + j);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                split4<NP>(kt[i], ktw[i]);
                if constexpr (REV) split4<NP>(qt[i], qtw[i]);
            }
        }
    };
    if (nc > 0) {
        fetch_v(chunk(0));
        fetch(chunk(0));
        put_v();
        put_first(chunk(0), s.first[0]);
        if (nc > 1) {
            fetch_v(chunk(1));
            fetch(chunk(1));
        }
    }
    for (int i = 0; i < nc; ++i) {
        lds_barrier();                               // (1)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) {
                *reinterpret_cast<u32x2*>(&s.kt[pl][CH * cq + c][pt]) = ktw[c][pl];
                if constexpr (REV) *reinterpret_cast<u32x2*>(&s.qt[pl][CH * cq + c][pt]) = qtw[c][pl];
            }
        if constexpr (KDA) {
            if (tq == 0) {
#pragma unroll
                for (int c = 0; c < CH; ++c) s.last[CH * cq + c] = lastw[c];
            }
        } else if (tid == 31) {
            s.last[0] = lastw[0];
        }
        if (i + 1 < nc) {
            put_first(chunk(i + 1), s.first[(i + 1) & 1]);
            if (i + 2 < nc) fetch(chunk(i + 2));
        }
        lds_barrier();                               // (2)
        if (i + 1 < nc) {
            put_v();
            if (i + 2 < nc) fetch_v(chunk(i + 2));
        }
    }
}

// The computing waves: 16 value columns each.
template <int DK, int DT, bool KDA, int MODE, int NC>
__device__ __forceinline__ void Scan<DK, DT, KDA, MODE, NC>::compute(int wave, int l) {
    const int n = l & 15, g = l >> 4, dv = p.dv, c0 = (sg * NC + wave) * 16, col = c0 + n;
    // lane (n, g), register r of tile t: key row (or token) 16 t + 4 g + r, value column c0 + n
    f32x4 S[NT];
    const float* init = REV ? p.ds1 : p.s0;
    const size_t sbase = (size_t)(b * H + h) * DK * dv;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = init ? init[sbase + (uint32_t)((16 * t + 4 * g + r) * dv + col)] : 0.f;

    // A product with its operands exchanged has the transposed result: lane (n, g) then holds token (or key row) 16 t + n and
    // in its four registers the value columns c0 + 4 g + r, which are adjacent in memory.  Outputs are made that way: one
    // access of 4 elements instead of four.
    auto store4 = [&](auto type, const Window& w, uint32_t off, const f32x4& x) {
        constexpr int T = decltype(type)::value;
        if constexpr (T == SQ_DTYPE_F32) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, x), w.r, off, 0, 0);
        } else {
            u32x2 b;
#pragma unroll
            for (int r = 0; r < 2; ++r)
                b[r] = T == SQ_DTYPE_BF16 ? round_pair(x[2 * r], x[2 * r + 1]) : f16_bits(x[2 * r]) | f16_bits(x[2 * r + 1]) << 16;
            __builtin_amdgcn_raw_buffer_store_b64(b, w.r, off, 0, 0);
        }
    };
    constexpr std::integral_constant<int, DT> row_type{};
    constexpr std::integral_constant<int, SQ_DTYPE_F32> f32_type{};
    // states and e, du for the backward pass: blocks of 16 value columns (a wave writes whole kilobytes)
    const uint32_t oc = opaque((n * 16 + 4 * g) * 4);

    uint32_t xn[VL ? 1 : 8];
    auto fetch = [&](int c) {                        // v (forward) or dy (reverse), in float32
        if constexpr (!VL) {
            const ScanRows& xr = REV ? p.dy : p.v;
            const uint32_t xs = (uint32_t)xr.stride * ES, o = opaque(4 * g * xs + (h * dv + col) * ES);
            const Window wx(static_cast<const char*>(xr.p) + (start + (int64_t)c * kChunk) * xs, tokens(c) * xs);
#pragma unroll
            for (int e = 0; e < 8; ++e) xn[VL ? 0 : e] = win_load1<DT>(wx, o + (16 * (e >> 2) + (e & 3)) * xs);
        }
    };
    if (nc > 0) fetch(chunk(0));
    Frag<1> unit[OUT ? 1 : 2];                       // the unit matrix: 32 key rows against key rows 16 t + n
    if constexpr (!OUT) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 16 * (e >> 2) + 4 * g + (e & 3) == 16 * t + n ? 1.f : 0.f;
            unit[OUT ? 0 : t] = split8<1>(v);
        }
    }

    // The chunk's matrices, That and P (reverse: T^T and P^T): rows 16 t + n as A operands, or as B operands of the transposed
    // product; from LDS when they are used, or from memory a step before.
    Frag<3> m0[2], m1[2];
    auto load_mat = [&](Frag<3>(&m)[2], const uint16_t* from) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 3; ++i) m[t].p[i] = *reinterpret_cast<const u32x4v*>(from + (uint32_t)((t * 3 + i) * 512 + 8 * l));
    };
    auto next_mat = [&](Frag<3>(&m)[2], int which, int step) {
        if constexpr (!ML) {
            if (step < nc) load_mat(m, (REV ? p.mat_r : p.mat_f) + (id(chunk(step)) * NMAT + which) * kMatShorts);
        }
    };
    next_mat(m0, 0, 0);
    if constexpr (NMAT == 2) next_mat(m1, 1, 0);
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};
    for (int ci = 0; ci < nc; ++ci) {
        const int c = chunk(ci), rem = tokens(c);
        const int64_t tok0 = start + (int64_t)c * kChunk;
        typename Lds::First& f = s.first[ci & 1];
        float x[8];                                  // v (forward) or dy (reverse)
        if constexpr (!VL) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = val1<DT>(xn[VL ? 0 : e]);
        }
        lds_barrier();                               // (1)
        if (!VL && ci + 1 < nc) fetch(chunk(ci + 1));
        if constexpr (VL) {
            const u32x4v b8 = *reinterpret_cast<const u32x4v*>(&s.v[16 * wave + n][8 * g]);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = val1<DT>((e & 1) ? b8[e >> 1] >> 16 : b8[e >> 1] & 0xffffu);
        }
        f32x4 pre[2], suf[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (!KDA) {
                pre[t] = *reinterpret_cast<const f32x4*>(&f.pre[16 * t + 4 * g]);
                suf[t] = *reinterpret_cast<const f32x4*>(&f.suf[16 * t + 4 * g]);
            }
        }
        f32x4 z[2] = {zero, zero}, yq[2] = {zero, zero};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {           // 32 key rows each: two tiles of S are the B operand
            float sx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) sx[e] = 2 * kb + (e >> 2) < NT ? S[2 * kb + (e >> 2) < NT ? 2 * kb + (e >> 2) : 0][e & 3] : 0.f;
            const Frag<3> sf = split8<3>(sx);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int off = (16 * t + n) * LDK + 32 * kb + 8 * g;
                mma<2>(z[t], lds_frag<NP>(&f.k[0][0][0], 32 * LDK, off), sf);
                if constexpr (OUT) mma<2>(yq[t], sf, lds_frag<NP>(&f.q[0][0][0], 32 * LDK, off));
            }
            if constexpr (!OUT) {
                // the backward pass reads the states at the chunk borders: transposed by a product with the unit matrix
                const Window wk((REV ? p.gt : p.st) + (id(c) * dv + c0) * DK, DK * 64);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (2 * kb + t >= NT) continue;
                    f32x4 border = zero;
                    mma<2>(border, sf, unit[OUT ? 0 : t]);
                    store4(f32_type, wk, oc + (32 * kb + 16 * t) * 64, border);
                }
            }
        }
        // S <- gamma_C S + the chunk's update, tile by tile
        auto update = [&](auto add) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (KDA) S[t] *= *reinterpret_cast<const f32x4*>(&s.last[16 * t + 4 * g]);
                else S[t] *= s.last[0];
                const int off = (16 * t + n) * LDT + 8 * g;
                const Frag<NP> kt = lds_frag<NP>(&s.kt[0][0][0], DK * LDT, off);
                if constexpr (REV) add(t, kt, lds_frag<NP>(&s.qt[0][0][0], DK * LDT, off));
                else add(t, kt, kt);
            }
        };
        float w[8];
        if constexpr (!REV) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = KDA ? x[e] - z[e >> 2][e & 3] : x[e] - pre[e >> 2][e & 3] * z[e >> 2][e & 3];
            const Frag<3> rf = split8<3>(w);
            if constexpr (ML) load_mat(m0, &f.m[0][0]);
            f32x4 ev[2] = {zero, zero};              // beta e; e itself for the backward pass
#pragma unroll
            for (int t = 0; t < 2; ++t) mma<2>(ev[t], m0[t], rf);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (MODE == kScanKeep) {
                    f32x4 et = zero;
                    mma<2>(et, rf, m0[t]);
                    store4(f32_type, Window(p.e + (id(c) * dv + c0) * kChunk, kChunk * 64), oc + 16 * t * 64, et);
                }
            }
            next_mat(m0, 0, ci + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (MODE == kScanKeep) ev[t] *= *reinterpret_cast<const f32x4*>(&f.beta[16 * t + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) w[4 * t + r] = ev[t][r];
            }
            if constexpr (OUT) {
                if constexpr (ML) load_mat(m1, &f.m[ML ? 1 : 0][0]);
                const Frag<3> uf = split8<3>(w);
                const uint32_t ys = (uint32_t)p.y.stride * ES;
                const Window wy(static_cast<const char*>(p.y.p) + tok0 * ys, (uint32_t)rem * ys);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if constexpr (!KDA) yq[t] *= f.pre[16 * t + n];
                    mma<2>(yq[t], uf, m1[t]);
                    store4(row_type, wy, (16 * t + n) * ys + (h * dv + c0 + 4 * g) * ES, yq[t]);
                }
                next_mat(m1, 1, ci + 1);
            }
            if constexpr (!KDA) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] *= suf[e >> 2][e & 3];
            }
            const Frag<3> uf = split8<3>(w);
            lds_barrier();                           // (2)
            update([&](int t, const Frag<NP>& kt, const Frag<NP>&) { mma<2>(S[t], kt, uf); });
        } else {
            // R = (gamma_C / gamma) K G + P^T dy;  du = T^T R;  G <- gamma_C G + (gamma Q)^T dy - (gamma K)^T (beta du)
            if constexpr (ML) load_mat(m1, &f.m[ML ? 1 : 0][0]);
            const Frag<NPL> xf = split8<NPL>(x);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (!KDA) z[t] *= suf[t];
                mma<2>(z[t], m1[t], xf);
#pragma unroll
                for (int r = 0; r < 4; ++r) w[4 * t + r] = z[t][r];
            }
            next_mat(m1, 1, ci + 1);
            if constexpr (ML) load_mat(m0, &f.m[0][0]);
            const Frag<3> rf = split8<3>(w);
            const uint32_t vs = (uint32_t)p.dvv.stride * ES;
            const Window wd(p.du + (id(c) * dv + c0) * kChunk, kChunk * 64);
            const Window wv(static_cast<const char*>(p.dvv.p) + tok0 * vs, (uint32_t)rem * vs);
            f32x4 du[2] = {zero, zero};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 dt = zero;
                mma<2>(du[t], m0[t], rf);
                mma<2>(dt, rf, m0[t]);
                store4(f32_type, wd, oc + 16 * t * 64, dt);
                dt *= f.beta[16 * t + n];
                store4(row_type, wv, (16 * t + n) * vs + (h * dv + c0 + 4 * g) * ES, dt);
            }
            next_mat(m0, 0, ci + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                du[t] *= *reinterpret_cast<const f32x4*>(&f.beta[16 * t + 4 * g]);
                if constexpr (!KDA) du[t] *= pre[t];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    w[4 * t + r] = -du[t][r];
                    if constexpr (!KDA) x[4 * t + r] *= pre[t][r];
                }
            }
            constexpr int NY = KDA ? NPL : 3;
            const Frag<3> wf = split8<3>(w);
            const Frag<NY> yf = split8<NY>(x);
            lds_barrier();                           // (2)
            update([&](int t, const Frag<NP>& kt, const Frag<NP>& qt) {
                mma<2>(S[t], qt, yf);
                mma<2>(S[t], kt, wf);
            });
        }
    }
    float* fin = REV ? p.ds0 : OUT ? p.s1 : nullptr;
    if (fin) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) fin[sbase + (uint32_t)((16 * t + 4 * g + r) * dv + col)] = S[t][r];
    }
}

constexpr int scan_threads(int dk, int nc) { return (nc + (dk < 32 ? 1 : 4)) * 64; }

template <int DK, int DT, bool KDA, int NC>
__global__ void __launch_bounds__(scan_threads(DK, NC)) k_scan(const ScanParams p) {
    __shared__ __align__(16) ScanLds<DK, DT, KDA, kScanOut, NC> s;
    Scan<DK, DT, KDA, kScanOut, NC>(p, s, blockIdx.x).run();
}

// The two scans of the backward pass, which do not depend on each other, side by side in one launch.
template <int DK, int DT, bool KDA, int NC>
__global__ void __launch_bounds__(scan_threads(DK, NC)) k_scan_both(const ScanParams p, unsigned n_rev) {
    __shared__ __align__(16) union U {
        ScanLds<DK, DT, KDA, kScanKeep, NC> f;
        ScanLds<DK, DT, KDA, kScanRev, NC> r;
    } s;
    // the reverse scans are the longer ones: they start first
    if (blockIdx.x < n_rev) Scan<DK, DT, KDA, kScanRev, NC>(p, s.r, blockIdx.x).run();
    else Scan<DK, DT, KDA, kScanKeep, NC>(p, s.f, blockIdx.x - n_rev).run();
}

// ---------------------------------------------------------------- launchers

template <int DK, int DT, bool KDA, int NC>
static hipError_t scan_nc(const ScanParams& p, bool backward, hipStream_t s) {
    if (p.dv % (16 * NC) != 0) return hipErrorInvalidValue;
    const int64_t blocks = (int64_t)p.n_long * p.n_heads * (p.dv / (16 * NC)) * (backward ? 2 : 1);
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), blk(scan_threads(DK, NC));
    if (backward) k_scan_both<DK, DT, KDA, NC><<<grid, blk, 0, s>>>(p, (unsigned)(blocks / 2));
    else k_scan<DK, DT, KDA, NC><<<grid, blk, 0, s>>>(p);
    return hipGetLastError();
}

template <int DK, int DT, bool KDA>
static hipError_t scan_t(const ScanParams& p, bool backward, hipStream_t s) {
    // Eight computing waves share the operands of four staging waves where there are more workgroups of four than CUs (256);
    // below that, four put the columns on twice as many CUs (a prompt of 777 tokens: 56 us, with eight 74; seven prompts of
    // 12301 tokens, 448 workgroups of four: 314 us, with eight 285; a backward call of 8190 tokens, 512 workgroups of four:
    // 1004 us, with eight 992).  With a gate per key row a workgroup of either size fills a CU's LDS: there 320 of four, one and a
    // quarter for each CU, are still a little faster (prefill of 6150 tokens: 426 us a call, with eight 443).
    if constexpr (DK == 128) {
        if ((int64_t)p.n_long * p.n_heads * (p.dv / 64) * (backward ? 2 : 1) > 256) return scan_nc<DK, DT, KDA, 8>(p, backward, s);
    }
    return scan_nc<DK, DT, KDA, DK < 32 ? 1 : 4>(p, backward, s);
}

hipError_t launch_scan(const ScanParams& p, bool backward, hipStream_t s) { SQ_SCAN_DISPATCH(scan_t, p, backward, s); }

}  // namespace sq
