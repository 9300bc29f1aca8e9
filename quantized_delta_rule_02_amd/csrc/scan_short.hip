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
    const int64_t start = __builtin_amdgcn_readfirstlane((int)sv.start);

    // all addresses are one wave's base, a lane's 32-bit offset and a row's: none takes registers of its own
    const uint32_t at = (uint32_t)(kl * R * dv + col) * 4, bytes = (uint32_t)(DK * dv) * 4;
    const Window w0(p.s0 + st * DK * dv, p.s0 ? bytes : 0);      // no first states: zeros
    f32x4 S[R];
#pragma unroll
    for (int j = 0; j < R; ++j) S[j] = __builtin_bit_cast(f32x4, (u32x4v)__builtin_amdgcn_raw_buffer_load_b128(w0.r, at, j * dv * 4, 0));

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
