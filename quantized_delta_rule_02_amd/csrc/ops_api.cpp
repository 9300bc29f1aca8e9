// C ABI of the gated delta scan and the norms around it: argument validation, workspace layout and launches.
// See include/stepq.h for the contract.
#include <hip/hip_runtime.h>

#include <cmath>

#include "checks.h"
#include "norm.h"
#include "scan.h"

using namespace sq;

// ------------------------------------------------------------------ scan

namespace {

struct ScanWork {                    // byte offsets of the workspace's parts
    size_t mf, gb, mr, ap, e, du, st, gt, total;
};

ScanWork scan_work(const sq_scan_cfg& c, bool backward) {
    ScanWork w{};
    size_t at = 0;
    auto take = [&at](size_t bytes) { const size_t o = at; at += (bytes + 255) & ~size_t(255); return o; };
    const size_t mats = size_t(scan_slots(c.n_tokens, c.n_seq)) * size_t(c.n_heads);
    const size_t vals = mats * kChunk * size_t(c.d_v) * 4;
    w.mf = take(mats * kMatShorts * (backward ? 2 : 4));
    if (c.form == SQ_FORM_GDN) w.gb = take(mats * 2 * kChunk * 4);
    if (backward) {
        w.mr = take(mats * kMatShorts * 4);
        if (c.form == SQ_FORM_GDN) w.ap = take(mats * 2 * kChunk * kChunk * 4);
        w.e = take(vals);
        w.du = take(vals);
        w.st = take(mats * size_t(c.d_k) * size_t(c.d_v) * 4);
        w.gt = take(mats * size_t(c.d_k) * size_t(c.d_v) * 4);
    }
    w.total = at;
    return w;
}

sq_status check_scan_cfg(const sq_scan_cfg* c) {
    if (!c) { set_error("cfg is NULL"); return SQ_ERR_ARG; }
    if (c->form != SQ_FORM_GDN && c->form != SQ_FORM_KDA) { set_error("form %d", c->form); return SQ_ERR_ARG; }
    if (!dtype_ok(c->dtype)) { set_error("dtype %d", c->dtype); return SQ_ERR_ARG; }
    if (c->n_heads < 1 || c->n_heads > 4096 || c->n_heads_k < 1 || c->n_heads % c->n_heads_k != 0) {
        set_error("n_heads %d / n_heads_k %d: heads in 1..4096, n_heads_k a divisor", c->n_heads, c->n_heads_k);
        return SQ_ERR_ARG;
    }
    if (!shape_supported(c->d_k, c->d_v)) {
        set_error("state shape %dx%d is not compiled in", c->d_k, c->d_v);
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->n_seq < 0 || c->n_tokens < 0 || c->n_tokens > 0x7fffffff) {
        set_error("n_seq %d / n_tokens %lld out of range", c->n_seq, (long long)c->n_tokens);
        return SQ_ERR_ARG;
    }
    // one workgroup per 16..128 value columns of a state, and at most one per chunk slot and head
    if ((scan_slots(c->n_tokens, c->n_seq) + c->n_seq) * c->n_heads * 2 > int64_t(0x7fffffff)) {
        set_error("too many sequences, tokens and heads in one call");
        return SQ_ERR_ARG;
    }
    return SQ_OK;
}

// Threads of the launch over all states: 8 computing and 4 staging waves per 128 value columns, 4 and 4 per 64, 1 and 1 per 16.
int64_t scan_launch_threads(const sq_scan_cfg& c, bool backward) {
    const int64_t per_col = c.d_k >= 128 ? 768 / 128 : c.d_k >= 64 ? 512 / 64 : 128 / 16;
    return int64_t(c.n_seq) * c.n_heads * c.d_v * per_col * (backward ? 2 : 1);
}

// Sequences of at most 16 tokens go token by token where the mean is at most 12 (the lengths themselves are the device's) and
// d_k is 64 or more.  Microseconds on the GPU, this way / in chunks, ragged sequences x 32 heads, at means of 1, 4, 8, 12, 16:
//   one gate per head, bfloat16, 128 x 128:  64:  47/87 55/89 74/91 88/92 94/96     8:  7/20 15/20 19/20 29/21 30/21
//   one gate per head, float32, 128 x 128:   64:  48/102 61/105 82/107 102/110 113/110    8:  7/23 15/22 20/24 30/24 32/24
//   a gate per key row, bfloat16, 128 x 128: 64:  48/130 62/144 92/146 116/153 123/147    8:  7/34 14/34 21/34 34/35 39/35
//   a gate per key row, float32, 128 x 256:  64:  109/213 123/230 174/231 208/242 221/236 8:  13/47 22/47 28/47 41/48 38/48
// 256 sequences and 64 x 64 states are alike, and so is one token of 32 heads: 5 against 13 to 29.  It loses where a few
// sequences with one gate per head have means of 9 to 12 (the chain of one sequence's tokens, 29 against 21).
constexpr int kShortLen = 16, kShortMean = 12;
bool takes_short(const sq_scan_cfg& c) { return c.d_k >= 64 && c.n_tokens <= int64_t(kShortMean) * c.n_seq; }

// A row array of `heads` x d elements of type dt per token (accessed up to 16 bytes at a time).
sq_status check_rows(const sq_rows* a, const char* name, int64_t heads, int64_t d, int32_t dt) {
    if (!a || !a->d_ptr) { set_error("%s is NULL", name); return SQ_ERR_ARG; }
    if (a->stride < heads * d) { set_error("%s: stride %lld below %lld", name, (long long)a->stride, (long long)(heads * d)); return SQ_ERR_SHAPE; }
    if (a->stride >= (int64_t(1) << 24)) { set_error("%s: stride %lld, below 2^24 elements is supported", name, (long long)a->stride); return SQ_ERR_SHAPE; }
    if (!aligned(a->d_ptr, 16) || a->stride * esize(dt) % 16 != 0) {
        set_error("%s: address and stride must be multiples of 16 bytes", name);
        return SQ_ERR_ARG;
    }
    return SQ_OK;
}

sq_status check_states(const float* a, const char* name) { return a ? check_f32(a, name, 4) : SQ_OK; }

ScanRows rows_of(const sq_rows* a) { return a ? ScanRows{a->d_ptr, a->stride} : ScanRows{nullptr, 0}; }

ScanParams scan_params(const sq_scan_cfg& c, const ScanWork& w, void* work, bool backward) {
    ScanParams p{};
    p.form = c.form; p.dtype = c.dtype; p.n_heads = c.n_heads; p.n_heads_k = c.n_heads_k; p.dk = c.d_k; p.dv = c.d_v;
    p.short_len = -1;
    p.n_long = c.n_seq;
    p.n_seq = c.n_seq; p.n_tokens = c.n_tokens; p.n_slots = scan_slots(c.n_tokens, c.n_seq); p.seq_start = c.d_seq_start;
    char* base = static_cast<char*>(work);
    auto u16 = [base](size_t o) { return reinterpret_cast<uint16_t*>(base + o); };
    auto f32 = [base](size_t o) { return reinterpret_cast<float*>(base + o); };
    p.mat_f = u16(w.mf);
    p.mat_gb = f32(w.gb);
    if (backward) {
        p.mat_r = u16(w.mr); p.mat_ap = f32(w.ap);
        p.e = f32(w.e); p.du = f32(w.du); p.st = f32(w.st); p.gt = f32(w.gt);
    }
    return p;
}

}  // namespace

extern "C" sq_status sq_delta_scan_bytes(const sq_scan_cfg* cfg, int32_t backward, size_t* bytes) {
    if (!bytes) { set_error("bytes is NULL"); return SQ_ERR_ARG; }
    SQ_TRY(check_scan_cfg(cfg));
    *bytes = scan_work(*cfg, backward != 0).total;
    return SQ_OK;
}

// What both directions share; *empty: there is no sequence and nothing to do.
static sq_status check_scan(const sq_scan_cfg* cfg, bool backward, const sq_rows* q, const sq_rows* k, const sq_rows* v,
                            const float* d_gate, const float* d_beta, bool* empty) {
    SQ_TRY(check_scan_cfg(cfg));
    *empty = cfg->n_seq == 0;
    if (*empty) return SQ_OK;
    if (scan_launch_threads(*cfg, backward) > int64_t(0xffffffffu)) {    // what one launch can have
        set_error("%d sequences of %d heads: too many states in one call", cfg->n_seq, cfg->n_heads);
        return SQ_ERR_ARG;
    }
    if (!cfg->d_seq_start && cfg->n_seq != 1) { set_error("d_seq_start is NULL with %d sequences", cfg->n_seq); return SQ_ERR_ARG; }
    if (cfg->n_tokens == 0) return SQ_OK;    // only empty sequences: the row arrays are not read
    SQ_TRY(check_rows(q, "q", cfg->n_heads_k, cfg->d_k, cfg->dtype));
    SQ_TRY(check_rows(k, "k", cfg->n_heads_k, cfg->d_k, cfg->dtype));
    SQ_TRY(check_rows(v, "v", cfg->n_heads, cfg->d_v, cfg->dtype));
    SQ_TRY(check_f32(d_gate, "gate", cfg->form == SQ_FORM_KDA ? 16 : 4));
    SQ_TRY(check_f32(d_beta, "beta", 4));
    return SQ_OK;
}

extern "C" sq_status sq_delta_scan(const sq_scan_cfg* cfg, const sq_rows* q, const sq_rows* k, const sq_rows* v,
                                   const float* d_gate, const float* d_beta, const float* d_s0, const sq_rows* y,
                                   float* d_s1, void* d_work, size_t work_bytes, void* stream) {
    bool empty = false;
    SQ_TRY(check_scan(cfg, false, q, k, v, d_gate, d_beta, &empty));
    if (empty) return SQ_OK;
    if (cfg->n_tokens > 0) SQ_TRY(check_rows(y, "y", cfg->n_heads, cfg->d_v, cfg->dtype));
    const ScanWork w = scan_work(*cfg, false);
    SQ_TRY(check_work(d_work, work_bytes, w.total));
    SQ_TRY(check_states(d_s0, "s0"));
    SQ_TRY(check_states(d_s1, "s1"));
    ScanParams p = scan_params(*cfg, w, d_work, false);
    p.q = rows_of(q); p.k = rows_of(k); p.v = rows_of(v); p.y = rows_of(y);
    p.gate = d_gate; p.beta = d_beta; p.s0 = d_s0; p.s1 = d_s1;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (takes_short(*cfg)) {
        p.short_len = kShortLen;
        const int64_t n_long = cfg->n_tokens / (kShortLen + 1);          // no more sequences can be longer
        if (n_long < p.n_long) p.n_long = int32_t(n_long);
        e = launch_scan_short(p, n_long > 0, s);
        if (e != hipSuccess) return fail_hip(e, "short scan launch");
        if (n_long == 0) return SQ_OK;
    } else {
        if (cfg->n_tokens > 0) e = launch_scan_prep(p, false, s);
        if (e != hipSuccess) return fail_hip(e, "scan preparation launch");
    }
    e = launch_scan(p, false, s);
    return e == hipSuccess ? SQ_OK : fail_hip(e, "scan launch");
}

extern "C" sq_status sq_delta_scan_bwd(const sq_scan_cfg* cfg, const sq_rows* q, const sq_rows* k, const sq_rows* v,
                                       const float* d_gate, const float* d_beta, const float* d_s0, const sq_rows* dy,
                                       const float* d_ds1, const sq_rows* dq, const sq_rows* dk, const sq_rows* dv,
                                       float* d_dgate, float* d_dbeta, float* d_ds0, void* d_work, size_t work_bytes,
                                       void* stream) {
    bool empty = false;
    SQ_TRY(check_scan(cfg, true, q, k, v, d_gate, d_beta, &empty));
    if (empty) return SQ_OK;
    if (cfg->n_tokens > 0) {
        SQ_TRY(check_rows(dy, "dy", cfg->n_heads, cfg->d_v, cfg->dtype));
        SQ_TRY(check_rows(dq, "dq", cfg->n_heads_k, cfg->d_k, cfg->dtype));
        SQ_TRY(check_rows(dk, "dk", cfg->n_heads_k, cfg->d_k, cfg->dtype));
        SQ_TRY(check_rows(dv, "dv", cfg->n_heads, cfg->d_v, cfg->dtype));
        SQ_TRY(check_f32(d_dgate, "dgate", 4));
        SQ_TRY(check_f32(d_dbeta, "dbeta", 4));
    }
    const ScanWork w = scan_work(*cfg, true);
    SQ_TRY(check_work(d_work, work_bytes, w.total));
    SQ_TRY(check_states(d_s0, "s0"));
    SQ_TRY(check_states(d_ds1, "ds1"));
    SQ_TRY(check_states(d_ds0, "ds0"));
    ScanParams p = scan_params(*cfg, w, d_work, true);
    p.q = rows_of(q); p.k = rows_of(k); p.v = rows_of(v); p.dy = rows_of(dy);
    p.dq = rows_of(dq); p.dkk = rows_of(dk); p.dvv = rows_of(dv);
    p.gate = d_gate; p.beta = d_beta; p.s0 = d_s0; p.ds1 = d_ds1; p.ds0 = d_ds0; p.dgate = d_dgate; p.dbeta = d_dbeta;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (cfg->n_tokens > 0) {
        e = launch_scan_prep(p, true, s);
        if (e != hipSuccess) return fail_hip(e, "scan preparation launch");
    }
    e = launch_scan(p, true, s);
    if (e != hipSuccess) return fail_hip(e, "scan launch");
    if (cfg->n_tokens > 0) e = launch_scan_grad(p, s);
    return e == hipSuccess ? SQ_OK : fail_hip(e, "scan gradient launch");
}

// ------------------------------------------------------------------ norms

namespace {

sq_status check_norm_cfg(const sq_norm_cfg* c, bool out) {
    if (!c) { set_error("cfg is NULL"); return SQ_ERR_ARG; }
    if (!dtype_ok(c->dtype) || !dtype_ok(c->dtype_out)) { set_error("dtype %d / dtype_out %d", c->dtype, c->dtype_out); return SQ_ERR_ARG; }
    if (c->kind != SQ_NORM_RMS && c->kind != SQ_NORM_L2) { set_error("kind %d", c->kind); return SQ_ERR_ARG; }
    if (out && c->act != SQ_ACT_SILU && c->act != SQ_ACT_SIGMOID) { set_error("act %d", c->act); return SQ_ERR_ARG; }
    if (c->d < 1 || c->d > kNormMaxD) { set_error("rows of %d elements: 1..%d are supported", c->d, kNormMaxD); return SQ_ERR_UNSUPPORTED; }
    if (c->n_outer < 0 || c->n_inner < 1 || c->n_outer > 0x7fffffff || c->n_outer * c->n_inner > 0x7fffffff ||
        int64_t(c->n_inner) * c->d > 0x7fffffff) {
        set_error("%lld x %d rows of %d elements: too many", (long long)c->n_outer, c->n_inner, c->d);
        return SQ_ERR_SHAPE;
    }
    if (!(c->eps >= 0.f) || !std::isfinite(c->eps) || !std::isfinite(c->res_scale) || !std::isfinite(c->out_scale)) {
        set_error("eps %g must not be negative, scales must be finite", double(c->eps));
        return SQ_ERR_ARG;
    }
    return SQ_OK;
}

// The arrays of one call: checked one by one, and all of them allow 16-byte accesses or none is read so.
struct NormCheck {
    const sq_norm_cfg& c;
    bool vec;
    sq_status st = SQ_OK;
    explicit NormCheck(const sq_norm_cfg& cfg) : c(cfg), vec(cfg.d % 8 == 0) {}
    NormRows operator()(const sq_rows* a, const char* name, int32_t dt, bool needed) {
        if (!a || !a->d_ptr) {
            if (needed && st == SQ_OK) { set_error("%s is NULL", name); st = SQ_ERR_ARG; }
            return NormRows{nullptr, 0};
        }
        if (st != SQ_OK) return NormRows{nullptr, 0};
        if ((c.n_outer > 1 && a->stride < int64_t(c.n_inner) * c.d) || a->stride > (int64_t(1) << 40)) {
            set_error("%s: stride %lld below %lld", name, (long long)a->stride, (long long)c.n_inner * c.d);
            st = SQ_ERR_SHAPE;
        } else if (!aligned(a->d_ptr, uintptr_t(esize(dt)))) {
            set_error("%s is not aligned to its element size", name);
            st = SQ_ERR_ARG;
        }
        vec = vec && aligned(a->d_ptr, 16) && (a->stride % 8 == 0 || c.n_outer <= 1);
        return NormRows{a->d_ptr, a->stride};
    }
};

sq_status check_params(const float* w, const float* cs) {
    if (!aligned(w, 4) || !aligned(cs, 4)) { set_error("weight / chan_scale not aligned"); return SQ_ERR_ARG; }
    return SQ_OK;
}

NormParams norm_params(const sq_norm_cfg& c, const float* w, const float* cs) {
    NormParams p{};
    p.n_rows = c.n_outer * c.n_inner;
    p.n_inner = c.n_inner; p.d = c.d; p.dtype = c.dtype; p.dtype_out = c.dtype_out; p.act = c.act;
    p.inv_div = c.kind == SQ_NORM_RMS ? float(1.0 / c.d) : 1.f;
    p.eps = c.eps; p.res_scale = c.res_scale; p.out_scale = c.out_scale;
    p.weight = w; p.chan_scale = cs;
    return p;
}

size_t norm_bytes(int64_t n_rows, int32_t d) { return size_t(2) * size_t(norm_bwd_blocks(n_rows, d)) * size_t(d) * 4; }

sq_status launch_norm_bwd(int op, bool vec, NormParams& p, float* dw, float* dcs, void* work, size_t bytes, void* stream) {
    p.dweight = dw; p.dchan_scale = dcs;
    if (dw || dcs) {
        SQ_TRY(check_work(work, bytes, norm_bytes(p.n_rows, p.d)));
        p.part = static_cast<float*>(work);
    }
    const hipError_t e = launch_norm(op, vec, p, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "norm gradient launch");
}

}  // namespace

extern "C" sq_status sq_norm_bytes(int64_t n_rows, int32_t d, size_t* bytes) {
    if (!bytes) { set_error("bytes is NULL"); return SQ_ERR_ARG; }
    if (n_rows < 0 || n_rows > 0x7fffffff || d < 1 || d > kNormMaxD) { set_error("%lld rows of %d elements", (long long)n_rows, d); return SQ_ERR_ARG; }
    *bytes = norm_bytes(n_rows, d);
    return SQ_OK;
}

extern "C" sq_status sq_norm_in(const sq_norm_cfg* cfg, const sq_rows* x, const sq_rows* r, const float* d_weight,
                                const float* d_chan_scale, const sq_rows* h, const sq_rows* n, void* stream) {
    SQ_TRY(check_norm_cfg(cfg, false));
    SQ_TRY(check_params(d_weight, d_chan_scale));
    if (cfg->n_outer == 0) return SQ_OK;     // nothing to do
    NormParams p = norm_params(*cfg, d_weight, d_chan_scale);
    NormCheck ck(*cfg);
    p.x = ck(x, "x", cfg->dtype, true);
    p.r = ck(r, "r", cfg->dtype, false);
    p.h = ck(h, "h", cfg->dtype, false);
    p.n = ck(n, "n", cfg->dtype_out, true);
    if (ck.st != SQ_OK) return ck.st;
    p.has_r = p.r.p != nullptr;
    p.write_h = p.h.p != nullptr;
    const hipError_t e = launch_norm(kNormIn, ck.vec, p, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "norm launch");
}

extern "C" sq_status sq_norm_in_bwd(const sq_norm_cfg* cfg, const sq_rows* h, const sq_rows* dn, const sq_rows* dh,
                                    const sq_rows* r, const float* d_weight, const float* d_chan_scale, const sq_rows* dx,
                                    const sq_rows* dr, float* d_dweight, float* d_dchan_scale, void* d_work,
                                    size_t work_bytes, void* stream) {
    SQ_TRY(check_norm_cfg(cfg, false));
    SQ_TRY(check_params(d_weight, d_chan_scale));
    NormParams p = norm_params(*cfg, d_weight, d_chan_scale);
    NormCheck ck(*cfg);
    const bool rows = cfg->n_outer > 0;
    p.h = ck(h, "h", cfg->dtype, rows);
    p.dn = ck(dn, "dn", cfg->dtype_out, rows);
    p.dh = ck(dh, "dh", cfg->dtype, false);
    p.r = d_dchan_scale ? ck(r, "r (needed for dchan_scale)", cfg->dtype, rows) : NormRows{nullptr, 0};
    p.dx = ck(dx, "dx", cfg->dtype, rows);
    p.dr = ck(dr, "dr", cfg->dtype, false);
    if (ck.st != SQ_OK) return ck.st;
    p.has_dh = p.dh.p != nullptr;
    p.has_r = p.r.p != nullptr;
    p.write_dr = p.dr.p != nullptr;
    return launch_norm_bwd(kNormInBwd, ck.vec, p, d_dweight, d_dchan_scale, d_work, work_bytes, stream);
}

extern "C" sq_status sq_norm_out(const sq_norm_cfg* cfg, const sq_rows* y, const sq_rows* z, const sq_rows* x,
                                 const float* d_weight, const float* d_chan_scale, const sq_rows* o, void* stream) {
    SQ_TRY(check_norm_cfg(cfg, true));
    SQ_TRY(check_params(d_weight, d_chan_scale));
    if (cfg->n_outer == 0) return SQ_OK;     // nothing to do
    NormParams p = norm_params(*cfg, d_weight, d_chan_scale);
    NormCheck ck(*cfg);
    p.y = ck(y, "y", cfg->dtype, true);
    p.z = ck(z, "z", cfg->dtype_out, false);
    p.x = ck(x, "x", cfg->dtype_out, false);
    p.o = ck(o, "o", cfg->dtype_out, true);
    if (ck.st != SQ_OK) return ck.st;
    p.has_z = p.z.p != nullptr;
    p.has_x = p.x.p != nullptr;
    const hipError_t e = launch_norm(kNormOut, ck.vec, p, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "norm launch");
}

extern "C" sq_status sq_norm_out_bwd(const sq_norm_cfg* cfg, const sq_rows* y, const sq_rows* z, const sq_rows* d_o,
                                     const float* d_weight, const float* d_chan_scale, const sq_rows* dy,
                                     const sq_rows* dz, float* d_dweight, float* d_dchan_scale, void* d_work,
                                     size_t work_bytes, void* stream) {
    SQ_TRY(check_norm_cfg(cfg, true));
    SQ_TRY(check_params(d_weight, d_chan_scale));
    NormParams p = norm_params(*cfg, d_weight, d_chan_scale);
    NormCheck ck(*cfg);
    const bool rows = cfg->n_outer > 0;
    p.y = ck(y, "y", cfg->dtype, rows);
    p.z = ck(z, "z", cfg->dtype_out, false);
    p.d_o = ck(d_o, "do", cfg->dtype_out, rows);
    p.dy = ck(dy, "dy", cfg->dtype, rows);
    p.dz = ck(dz, "dz", cfg->dtype_out, false);
    if (ck.st != SQ_OK) return ck.st;
    if (p.dz.p && !p.z.p && rows) { set_error("dz without z"); return SQ_ERR_ARG; }
    p.has_z = p.z.p != nullptr;
    p.write_dz = p.dz.p != nullptr;
    return launch_norm_bwd(kNormOutBwd, ck.vec, p, d_dweight, d_dchan_scale, d_work, work_bytes, stream);
}
