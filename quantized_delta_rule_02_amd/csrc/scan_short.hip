// The gated delta scan of short sequences (gfx950), token by token: a few drafted tokens, or one, per request.
//
// A state is read once and written once, 128 KiB a 128 x 128 state, and that is what bounds the launch; the chunked scan keeps
// a CU's LDS and registers for one or two states, whose loads, products and stores follow one another.  Here a wave owns 32
// value columns of a state (a row's piece is one cache line of 128 bytes) and nothing else, without LDS and barriers:
// lane l holds the columns 4 (l & 7) .. + 3 of the key rows DK / 8 (l >> 3) .. + DK / 8 - 1.  Per token, with S' = D S,
//
//   u = beta (v - S'^T k);   y = S'^T q + (q . k) u;   S = S' + k u^T
//
// so that both products over the key rows are summed over the lanes in one round.
#include <hip/hip_runtime.h>

#include "scan_dev.h"

namespace sq {

typedef float f32x4w __attribute__((ext_vector_type(4), aligned(4)));   // states are aligned to their elements only

template <int DK, int DT, bool KDA>
__global__ void __launch_bounds__(256, DT == SQ_DTYPE_F32 || KDA ? 2 : 4) k_short(const ScanParams p) {
    constexpr int R = DK / 8, ES = DT == SQ_DTYPE_F32 ? 4 : 2, W = 16 / ES;      // key rows of a lane; elements per 16 bytes
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l = (int)threadIdx.x & 63, cl = l & 7, kl = l >> 3;
    const int H = p.n_heads, dv = p.dv, parts = dv / 32;
    const int64_t id = (int64_t)blockIdx.x * 4 + wave;
    const int64_t st = id / parts;
    if (st >= (int64_t)p.n_seq * H) return;
    const int col = (int)(id - st * parts) * 32 + 4 * cl, b = (int)(st / H), h = (int)(st - (int64_t)b * H), hk = h / (H / p.n_heads_k);
    const Seq sv = sequence(p, b);
    if (sv.len > p.short_len) return;                // the chunked scan's
    const int len = __builtin_amdgcn_readfirstlane((int)sv.len);

    const int64_t at = (st * DK + kl * R) * dv + col;
    f32x4 S[R];
#pragma unroll
    for (int j = 0; j < R; ++j) S[j] = p.s0 ? f32x4(*reinterpret_cast<const f32x4w*>(p.s0 + at + (int64_t)j * dv)) : f32x4{0.f, 0.f, 0.f, 0.f};

    using Words = std::conditional_t<ES == 4, u32x4v, u32x2>;       // four elements
    struct Token {                                   // as loaded
        u32x4v k[R / W], q[R / W], a[KDA ? R / 4 : 1];
        Words v;
        float gate, beta;
    };
    auto load = [&](int64_t t) {
        Token x;
        const char* kp = static_cast<const char*>(p.k.p) + (t * p.k.stride + hk * DK + kl * R) * ES;
        const char* qp = static_cast<const char*>(p.q.p) + (t * p.q.stride + hk * DK + kl * R) * ES;
#pragma unroll
        for (int i = 0; i < R / W; ++i) {
            x.k[i] = reinterpret_cast<const u32x4v*>(kp)[i];
            x.q[i] = reinterpret_cast<const u32x4v*>(qp)[i];
        }
        x.v = *reinterpret_cast<const Words*>(static_cast<const char*>(p.v.p) + (t * p.v.stride + h * dv + col) * ES);
        if constexpr (KDA) {
            const u32x4v* ap = reinterpret_cast<const u32x4v*>(p.gate + (t * H + h) * DK + kl * R);
#pragma unroll
            for (int i = 0; i < R / 4; ++i) x.a[i] = ap[i];
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
    if (len > 0) next = load(sv.start);
    for (int t = 0; t < len; ++t) {
        const Token x = next;
        if (t + 1 < len) next = load(sv.start + t + 1);
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
            char* yp = static_cast<char*>(p.y.p) + ((sv.start + t) * p.y.stride + h * dv + col) * ES;
            if constexpr (DT == SQ_DTYPE_F32) {
                *reinterpret_cast<f32x4*>(yp) = y;
            } else {
                u32x2 w;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[i] = DT == SQ_DTYPE_BF16 ? round_pair(y[2 * i], y[2 * i + 1]) : f16_bits(y[2 * i]) | f16_bits(y[2 * i + 1]) << 16;
                *reinterpret_cast<u32x2*>(yp) = w;
            }
        }
    }
    if (p.s1) {
#pragma unroll
        for (int j = 0; j < R; ++j) *reinterpret_cast<f32x4w*>(p.s1 + at + (int64_t)j * dv) = S[j];
    }
}

template <int DK, int DT, bool KDA>
static hipError_t short_t(const ScanParams& p, hipStream_t s) {
    if constexpr (DK < 64) {
        return hipErrorInvalidValue;
    } else {
        if (p.dv % 32 != 0) return hipErrorInvalidValue;
        const int64_t blocks = ((int64_t)p.n_seq * p.n_heads * (p.dv / 32) + 3) / 4;
        if (blocks > 0x7fffffff) return hipErrorInvalidValue;
        k_short<DK, DT, KDA><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(p);
        return hipGetLastError();
    }
}

hipError_t launch_scan_short(const ScanParams& p, hipStream_t s) { SQ_SCAN_DISPATCH(short_t, p, s); }

}  // namespace sq
