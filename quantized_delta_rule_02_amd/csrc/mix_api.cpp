// C ABI of the causal convolution, the selective scan and the quantised row cache: argument validation, workspace layout and
// launches.  See include/stepq.h for the contract.
#include <hip/hip_runtime.h>

#include "cache.h"
#include "checks.h"
#include "conv.h"
#include "ssm.h"

using namespace sq;

namespace {

constexpr int64_t kMaxThreads = 0xffffffffll;    // of one launch

// The packed sequences of a call.
sq_status check_seqs(int32_t n_seq, int64_t n_tokens, const int32_t* start) {
    if (n_seq < 0 || n_tokens < 0 || n_tokens > 0x7fffffff) {
        set_error("n_seq %d / n_tokens %lld out of range", n_seq, (long long)n_tokens);
        return SQ_ERR_ARG;
    }
    if (!aligned(start, 4)) { set_error("d_seq_start is not aligned"); return SQ_ERR_ARG; }
    return SQ_OK;
}
sq_status check_start(int32_t n_seq, const int32_t* start) {
    if (!start && n_seq > 1) { set_error("d_seq_start is NULL with %d sequences", n_seq); return SQ_ERR_ARG; }
    return SQ_OK;
}

// Row arrays of one call: checked one by one; `vec` stays true as long as all of them allow accesses of `v` elements.
struct RowCheck {
    int32_t dtype;
    int64_t n_rows;
    int v;
    bool vec = true;
    sq_status st = SQ_OK;
    Rows operator()(const sq_rows* a, const char* name, int64_t width, bool needed) {
        if (!a || !a->d_ptr) {
            if (needed && st == SQ_OK) { set_error("%s is NULL", name); st = SQ_ERR_ARG; }
            return Rows{nullptr, 0};
        }
        if (st != SQ_OK) return Rows{nullptr, 0};
        if ((n_rows > 1 && a->stride < width) || a->stride > (int64_t(1) << 40)) {
            set_error("%s: stride %lld below %lld or too large", name, (long long)a->stride, (long long)width);
            st = SQ_ERR_SHAPE;
        } else if (!aligned(a->d_ptr, uintptr_t(esize(dtype)))) {
            set_error("%s is not aligned to its element size", name);
            st = SQ_ERR_ARG;
        }
        vec = vec && aligned(a->d_ptr, uintptr_t(v * esize(dtype))) && (a->stride % v == 0 || n_rows <= 1) && width % v == 0;
        return Rows{a->d_ptr, n_rows > 1 ? a->stride : width};
    }
    // a plain array of the same type
    void plain(const void* a, const char* name) {
        if (st == SQ_OK && !aligned(a, uintptr_t(esize(dtype)))) {
            set_error("%s is not aligned to its element size", name);
            st = SQ_ERR_ARG;
        }
        vec = vec && aligned(a, uintptr_t(v * esize(dtype)));
    }
};

sq_status check_optional(const float* a, const char* name, uintptr_t to = 4) { return a ? check_f32(a, name, to) : SQ_OK; }

}  // namespace

// ------------------------------------------------------------------ convolution

namespace {

sq_status check_conv_cfg(const sq_conv_cfg* c) {
    if (!c) { set_error("cfg is NULL"); return SQ_ERR_ARG; }
    if (!dtype_ok(c->dtype)) { set_error("dtype %d", c->dtype); return SQ_ERR_ARG; }
    if (c->act != SQ_ACT_SILU && c->act != SQ_ACT_NONE) { set_error("act %d", c->act); return SQ_ERR_ARG; }
    if (c->channels < 1 || c->channels > (1 << 24)) { set_error("channels %d: 1..2^24", c->channels); return SQ_ERR_ARG; }
    if (c->width < 2 || c->width > kConvMaxWidth) {
        set_error("filters of %d taps: 2..%d are supported", c->width, kConvMaxWidth);
        return SQ_ERR_UNSUPPORTED;
    }
    SQ_TRY(check_seqs(c->n_seq, c->n_tokens, c->d_seq_start));
    // a thread an element where accesses are single, in the shortest runs; the gradients' workgroups have 64 channels there
    if (((c->n_tokens >> 4) + c->n_seq) * ((int64_t(c->channels) + 255) / 256) * 256 > kMaxThreads ||
        run_slots(c->n_tokens, c->n_seq, kConvBwdRuns) * ((int64_t(c->channels) + 63) / 64) * 256 > kMaxThreads ||
        int64_t(c->width + 1) * c->channels * 16 > kMaxThreads) {
        set_error("%lld tokens of %d channels in %d sequences: too many for one call", (long long)c->n_tokens, c->channels, c->n_seq);
        return SQ_ERR_ARG;
    }
    return SQ_OK;
}

size_t conv_bytes(const sq_conv_cfg& c) {
    return size_t(run_slots(c.n_tokens, c.n_seq, kConvBwdRuns)) * size_t(c.width + 1) * size_t(c.channels) * 4;
}

ConvParams conv_params(const sq_conv_cfg& c, int log, const float* weight, const float* bias) {
    ConvParams p{};
    p.runs = Runs{c.d_seq_start, c.n_tokens, c.n_seq, log};
    p.channels = c.channels; p.dtype = c.dtype; p.act = c.act; p.width = c.width;
    p.weight = weight; p.bias = bias;
    return p;
}

}  // namespace

extern "C" sq_status sq_conv_bytes(const sq_conv_cfg* cfg, size_t* bytes) {
    if (!bytes) { set_error("bytes is NULL"); return SQ_ERR_ARG; }
    SQ_TRY(check_conv_cfg(cfg));
    *bytes = conv_bytes(*cfg);
    return SQ_OK;
}

extern "C" sq_status sq_conv(const sq_conv_cfg* cfg, const sq_rows* x, const float* d_weight, const float* d_bias,
                             const void* d_s0, const sq_rows* y, void* d_s1, void* stream) {
    SQ_TRY(check_conv_cfg(cfg));
    if (cfg->n_seq == 0) return SQ_OK;
    SQ_TRY(check_start(cfg->n_seq, cfg->d_seq_start));
    SQ_TRY(check_f32(d_weight, "weight", 4));
    SQ_TRY(check_optional(d_bias, "bias"));
    ConvParams p = conv_params(*cfg, kConvLog, d_weight, d_bias);
    RowCheck ck{cfg->dtype, cfg->n_tokens, kConvBytes / int(esize(cfg->dtype))};
    p.x = ck(x, "x", cfg->channels, cfg->n_tokens > 0);
    p.y = ck(y, "y", cfg->channels, cfg->n_tokens > 0);
    ck.plain(d_s0, "s0");
    ck.plain(d_s1, "s1");
    if (ck.st != SQ_OK) return ck.st;
    p.s0 = d_s0; p.s1 = d_s1;
    // x and y beyond what the last cache holds: y would push out x's rows, and be gone itself when the next call reads it (12301 tokens of
    // 8192 channels in bfloat16: 82 us so, 88 otherwise; below, the next call finds y there)
    p.once = cfg->n_tokens * cfg->channels * esize(cfg->dtype) * 2 > (int64_t(256) << 20);
    const hipError_t e = launch_conv(p, ck.vec && cfg->channels % ck.v == 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "convolution launch");
}

extern "C" sq_status sq_conv_bwd(const sq_conv_cfg* cfg, const sq_rows* x, const float* d_weight, const float* d_bias,
                                 const void* d_s0, const sq_rows* dy, const void* d_ds1, const sq_rows* dx, float* d_dweight,
                                 float* d_dbias, void* d_ds0, void* d_work, size_t work_bytes, void* stream) {
    SQ_TRY(check_conv_cfg(cfg));
    SQ_TRY(check_start(cfg->n_seq, cfg->d_seq_start));
    SQ_TRY(check_f32(d_weight, "weight", 4));
    SQ_TRY(check_optional(d_bias, "bias"));
    SQ_TRY(check_optional(d_dweight, "dweight"));
    SQ_TRY(check_optional(d_dbias, "dbias"));
    ConvParams p = conv_params(*cfg, kConvBwdRuns, d_weight, d_bias);
    RowCheck ck{cfg->dtype, cfg->n_tokens, kConvBwdBytes / int(esize(cfg->dtype))};
    const bool rows = cfg->n_tokens > 0 && cfg->n_seq > 0;
    p.x = ck(x, "x", cfg->channels, rows);
    p.dy = ck(dy, "dy", cfg->channels, rows);
    p.dx = ck(dx, "dx", cfg->channels, rows);
    ck.plain(d_s0, "s0");
    ck.plain(d_ds1, "ds1");
    ck.plain(d_ds0, "ds0");
    if (ck.st != SQ_OK) return ck.st;
    p.s0 = d_s0; p.ds1 = d_ds1; p.ds0 = d_ds0;
    p.dweight = d_dweight; p.dbias = d_dbias;
    if (d_dweight || d_dbias) {
        SQ_TRY(check_work(d_work, work_bytes, conv_bytes(*cfg)));
        p.part = static_cast<float*>(d_work);
    }
    const hipError_t e = launch_conv_bwd(p, ck.vec && cfg->channels % ck.v == 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "convolution gradient launch");
}

extern "C" sq_status sq_conv_step(const sq_conv_cfg* cfg, const sq_rows* x, const float* d_weight, const float* d_bias,
                                  const int32_t* d_slots, int64_t n_slots, void* d_window, const sq_rows* y, void* stream) {
    SQ_TRY(check_conv_cfg(cfg));
    if (cfg->n_tokens == 0) return SQ_OK;
    if (n_slots < 0 || n_slots > 0x7fffffff) { set_error("n_slots %lld", (long long)n_slots); return SQ_ERR_ARG; }
    if (n_slots == 0) return SQ_OK;          // every slot is outside
    SQ_TRY(check_f32(d_weight, "weight", 4));
    SQ_TRY(check_optional(d_bias, "bias"));
    if (!aligned(d_slots, 4)) { set_error("d_slots is not aligned"); return SQ_ERR_ARG; }
    if (cfg->n_tokens * ((int64_t(cfg->channels) + 255) / 256) * 256 > kMaxThreads) {
        set_error("%lld requests of %d channels: too many for one call", (long long)cfg->n_tokens, cfg->channels);
        return SQ_ERR_ARG;
    }
    ConvParams p = conv_params(*cfg, 0, d_weight, d_bias);
    RowCheck ck{cfg->dtype, cfg->n_tokens, kConvStepBytes / int(esize(cfg->dtype))};
    p.x = ck(x, "x", cfg->channels, true);
    p.y = ck(y, "y", cfg->channels, true);
    if (!d_window && ck.st == SQ_OK) { set_error("window is NULL"); return SQ_ERR_ARG; }
    ck.plain(d_window, "window");
    if (ck.st != SQ_OK) return ck.st;
    p.slots = d_slots; p.n_slots = n_slots; p.batch = cfg->n_tokens; p.window = d_window;
    const hipError_t e = launch_conv_step(p, ck.vec && cfg->channels % ck.v == 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "convolution step launch");
}

// ------------------------------------------------------------------ selective scan

namespace {

struct SsmWork {                     // byte offsets of the workspace's parts
    size_t hseg, kseg, dsum, htile, dtile, dd, bc, total;
};

int64_t ssm_fwd_blocks(const sq_ssm_cfg& c) { return ssm_blocks(c.channels, c.n_groups, c.d_state); }

SsmWork ssm_work(const sq_ssm_cfg& c, bool backward, int log) {
    SsmWork w{};
    size_t at = 0;
    auto take = [&at](size_t bytes) { const size_t o = at; at += (bytes + 255) & ~size_t(255); return o; };
    if (log >= 0) {
        const size_t slots = size_t(run_slots(c.n_tokens, c.n_seq, log)), states = slots * size_t(c.channels) * size_t(c.d_state) * 4;
        w.hseg = take(states);
        w.dsum = take(slots * size_t(c.channels) * 4);
        if (backward) {
            w.kseg = take(states);
            const size_t tiles = (size_t(c.n_tokens) + kSsmTile - 1) / kSsmTile;
            w.htile = take(tiles * size_t(c.channels) * size_t(c.d_state) * 4);
            w.dtile = take(tiles * size_t(c.channels) * 4);
            w.dd = take(slots * 2 * size_t(c.channels) * 4);
            w.bc = take(size_t(ssm_grad_blocks(c.channels, c.n_groups, c.d_state)) * size_t(c.n_tokens) * 2 * size_t(c.d_state) * 4);
        }
    }
    w.total = at;
    return w;
}

sq_status check_ssm_cfg(const sq_ssm_cfg* c) {
    if (!c) { set_error("cfg is NULL"); return SQ_ERR_ARG; }
    if (!dtype_ok(c->dtype)) { set_error("dtype %d", c->dtype); return SQ_ERR_ARG; }
    if (c->d_state != 8 && c->d_state != 16 && c->d_state != 32 && c->d_state != 64 && c->d_state != 128) {
        set_error("%d states a channel: 8, 16, 32, 64 and 128 are compiled in", c->d_state);
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->channels < 1 || c->channels > (1 << 20) || c->n_groups < 1 || c->channels % c->n_groups != 0) {
        set_error("channels %d / n_groups %d: channels in 1..2^20, n_groups a divisor", c->channels, c->n_groups);
        return SQ_ERR_ARG;
    }
    if (c->softplus != 0 && c->softplus != 1) { set_error("softplus %d", c->softplus); return SQ_ERR_ARG; }
    SQ_TRY(check_seqs(c->n_seq, c->n_tokens, c->d_seq_start));
    if (run_slots(c->n_tokens, c->n_seq, 6) * ssm_fwd_blocks(*c) * 512 > kMaxThreads ||
        int64_t(c->n_seq) * ((int64_t(c->channels) * c->d_state + 1023) / 1024) * 256 > kMaxThreads) {
        set_error("%lld tokens of %d channels in %d sequences: too many for one call", (long long)c->n_tokens, c->channels, c->n_seq);
        return SQ_ERR_ARG;
    }
    return SQ_OK;
}

SsmParams ssm_params(const sq_ssm_cfg& c, int log) {
    SsmParams p{};
    p.runs = Runs{c.d_seq_start, c.n_tokens, c.n_seq, log};
    p.dtype = c.dtype; p.channels = c.channels; p.d_state = c.d_state; p.n_groups = c.n_groups;
    p.group_channels = c.channels / c.n_groups; p.softplus = c.softplus;
    return p;
}

// The inputs that all three calls share; accesses of four elements where all arrays allow them and no group ends inside one.
sq_status take_inputs(const sq_ssm_cfg& c, SsmParams& p, RowCheck& ck, const sq_ssm_in* in, bool rows) {
    if (!in) { set_error("inputs are NULL"); return SQ_ERR_ARG; }
    const int64_t bc = int64_t(c.n_groups) * c.d_state;
    p.u = ck(in->u, "u", c.channels, rows);
    p.dt = ck(in->dt, "dt", c.channels, rows);
    p.b = ck(in->b, "b", bc, rows);
    p.c = ck(in->c, "c", bc, rows);
    p.z = ck(in->z, "z", c.channels, false);
    if (ck.st != SQ_OK) return ck.st;
    SQ_TRY(check_f32(in->d_a, "a", 16));
    SQ_TRY(check_optional(in->d_d, "d"));
    SQ_TRY(check_optional(in->d_dt_bias, "dt_bias"));
    p.a = in->d_a; p.d = in->d_d; p.dt_bias = in->d_dt_bias;
    ck.vec = ck.vec && p.group_channels % 4 == 0;
    return SQ_OK;
}

int ssm_log(const sq_ssm_cfg& c, bool backward) { return ssm_segment_log(c.n_tokens, c.n_seq, ssm_fwd_blocks(c), backward); }

}  // namespace

extern "C" sq_status sq_ssm_scan_bytes(const sq_ssm_cfg* cfg, int32_t backward, size_t* bytes) {
    if (!bytes) { set_error("bytes is NULL"); return SQ_ERR_ARG; }
    SQ_TRY(check_ssm_cfg(cfg));
    *bytes = ssm_work(*cfg, backward != 0, ssm_log(*cfg, backward != 0)).total;
    return SQ_OK;
}

extern "C" sq_status sq_ssm_scan(const sq_ssm_cfg* cfg, const sq_ssm_in* in, const float* d_s0, const sq_rows* y, float* d_s1,
                                 void* d_work, size_t work_bytes, void* stream) {
    SQ_TRY(check_ssm_cfg(cfg));
    if (cfg->n_seq == 0) return SQ_OK;
    SQ_TRY(check_start(cfg->n_seq, cfg->d_seq_start));
    const int log = ssm_log(*cfg, false);
    SsmParams p = ssm_params(*cfg, log);
    RowCheck ck{cfg->dtype, cfg->n_tokens, 4};
    p.y = ck(y, "y", cfg->channels, cfg->n_tokens > 0);
    SQ_TRY(take_inputs(*cfg, p, ck, in, cfg->n_tokens > 0));
    SQ_TRY(check_optional(d_s0, "s0", 16));
    SQ_TRY(check_optional(d_s1, "s1", 16));
    p.s0 = d_s0; p.s1 = d_s1;
    const SsmWork w = ssm_work(*cfg, false, log);
    SQ_TRY(check_work(d_work, work_bytes, w.total));
    if (log >= 0) {
        char* base = static_cast<char*>(d_work);
        p.hseg = reinterpret_cast<float*>(base + w.hseg);
        p.dsum = reinterpret_cast<float*>(base + w.dsum);
    }
    const hipError_t e = launch_ssm(p, ck.vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "selective scan launch");
}

extern "C" sq_status sq_ssm_scan_bwd(const sq_ssm_cfg* cfg, const sq_ssm_in* in, const float* d_s0, const sq_rows* dy,
                                     const float* d_ds1, const sq_ssm_grads* out, float* d_ds0, void* d_work, size_t work_bytes,
                                     void* stream) {
    SQ_TRY(check_ssm_cfg(cfg));
    SQ_TRY(check_start(cfg->n_seq, cfg->d_seq_start));
    if (!out) { set_error("gradients are NULL"); return SQ_ERR_ARG; }
    const int log = ssm_log(*cfg, true);
    const bool rows = cfg->n_tokens > 0 && cfg->n_seq > 0;
    SsmParams p = ssm_params(*cfg, log);
    RowCheck ck{cfg->dtype, cfg->n_tokens, 4};
    const int64_t bc = int64_t(cfg->n_groups) * cfg->d_state;
    p.dy = ck(dy, "dy", cfg->channels, rows);
    p.du = ck(out->du, "du", cfg->channels, rows);
    p.ddt = ck(out->ddt, "ddt", cfg->channels, rows);
    p.dz = ck(out->dz, "dz", cfg->channels, false);
    RowCheck bk{cfg->dtype, cfg->n_tokens, 1};       // written element by element
    p.db = bk(out->db, "db", bc, rows);
    p.dc = bk(out->dc, "dc", bc, rows);
    SQ_TRY(take_inputs(*cfg, p, ck, in, rows));
    if (bk.st != SQ_OK) return bk.st;
    if (p.dz.p && !p.z.p && rows) { set_error("dz without z"); return SQ_ERR_ARG; }
    SQ_TRY(check_optional(out->d_da, "da"));
    SQ_TRY(check_optional(out->d_dd, "dd"));
    SQ_TRY(check_optional(out->d_ddt_bias, "ddt_bias"));
    SQ_TRY(check_optional(d_s0, "s0", 16));
    SQ_TRY(check_optional(d_ds1, "ds1", 16));
    SQ_TRY(check_optional(d_ds0, "ds0", 16));
    const SsmWork w = ssm_work(*cfg, true, log);
    SQ_TRY(check_work(d_work, work_bytes, w.total));
    auto f32 = [d_work](size_t o) { return reinterpret_cast<float*>(static_cast<char*>(d_work) + o); };
    p.hseg = f32(w.hseg); p.kseg = f32(w.kseg); p.dsum = f32(w.dsum); p.htile = f32(w.htile); p.dtile = f32(w.dtile); p.dd_part = f32(w.dd); p.bc_part = f32(w.bc);
    p.s0 = d_s0; p.ds1 = d_ds1; p.ds0 = d_ds0;
    p.da = out->d_da; p.dd = out->d_dd; p.ddt_bias = out->d_ddt_bias;
    const hipError_t e = launch_ssm_bwd(p, ck.vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "selective scan gradient launch");
}

extern "C" sq_status sq_ssm_step(const sq_ssm_cfg* cfg, const sq_ssm_in* in, const int32_t* d_slots, int64_t n_slots,
                                 float* d_state, const sq_rows* y, void* stream) {
    SQ_TRY(check_ssm_cfg(cfg));
    if (cfg->n_tokens == 0) return SQ_OK;
    if (n_slots < 0 || n_slots > 0x7fffffff) { set_error("n_slots %lld", (long long)n_slots); return SQ_ERR_ARG; }
    if (n_slots == 0) return SQ_OK;          // every slot is outside
    if (!aligned(d_slots, 4)) { set_error("d_slots is not aligned"); return SQ_ERR_ARG; }
    if (cfg->n_tokens * ssm_fwd_blocks(*cfg) * 256 > kMaxThreads) {
        set_error("%lld requests of %d channels: too many for one call", (long long)cfg->n_tokens, cfg->channels);
        return SQ_ERR_ARG;
    }
    SsmParams p = ssm_params(*cfg, -1);
    RowCheck ck{cfg->dtype, cfg->n_tokens, 4};
    p.y = ck(y, "y", cfg->channels, true);
    SQ_TRY(take_inputs(*cfg, p, ck, in, true));
    SQ_TRY(check_f32(d_state, "state", 16));
    p.slots = d_slots; p.n_slots = n_slots; p.batch = cfg->n_tokens; p.state = d_state;
    const hipError_t e = launch_ssm_step(p, ck.vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "selective scan step launch");
}

// ------------------------------------------------------------------ quantised row cache

namespace {

sq_status cache_call(const sq_cache_cfg* c, const sq_rows* x, const int32_t* d_slots, const void* codes, const float* scales,
                     CacheParams& p, bool& vec, bool& empty) {
    if (!c) { set_error("cfg is NULL"); return SQ_ERR_ARG; }
    if (!dtype_ok(c->dtype)) { set_error("dtype %d", c->dtype); return SQ_ERR_ARG; }
    if (c->format != SQ_CACHE_INT8 && c->format != SQ_CACHE_INT4 && c->format != SQ_CACHE_E4M3) { set_error("format %d", c->format); return SQ_ERR_ARG; }
    if (c->group < 1 || c->group > kCacheMaxGroup || (c->format == SQ_CACHE_INT4 && c->group % 2 != 0)) {
        set_error("groups of %d elements: 1..%d, even for 4-bit codes", c->group, kCacheMaxGroup);
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->d < 1 || c->d % c->group != 0) { set_error("rows of %d elements in groups of %d", c->d, c->group); return SQ_ERR_SHAPE; }
    if (c->n_rows < 0 || c->n_slots < 0 || c->n_slots > 0x7fffffff) {
        set_error("n_rows %lld / n_slots %lld out of range", (long long)c->n_rows, (long long)c->n_slots);
        return SQ_ERR_ARG;
    }
    // a wave a group, or a thread two elements
    if (c->n_rows > 0x7fffffff || c->n_rows * (c->d / c->group) * 64 > kMaxThreads || c->n_rows * ((int64_t(c->d) + 1) / 2) > 0x7fffffff) {
        set_error("%lld rows of %d elements: too many for one call", (long long)c->n_rows, c->d);
        return SQ_ERR_SHAPE;
    }
    empty = c->n_rows == 0 || c->n_slots == 0;      // with no slots every slot is outside
    if (empty) return SQ_OK;
    RowCheck ck{c->dtype, c->n_rows, 8};
    ck.v = 16 / int(esize(c->dtype));                // float32 rows of eight elements are two accesses
    p.x = ck(x, "x", c->d, true);
    if (ck.st != SQ_OK) return ck.st;
    if (!codes) { set_error("codes is NULL"); return SQ_ERR_ARG; }
    SQ_TRY(check_f32(scales, "scales", 4));
    if (!aligned(d_slots, 4)) { set_error("d_slots is not aligned"); return SQ_ERR_ARG; }
    vec = ck.vec && c->group % 8 == 0 && aligned(codes, c->format == SQ_CACHE_INT4 ? 4 : 8);
    p.dtype = c->dtype; p.format = c->format; p.d = c->d; p.group = c->group; p.n_rows = c->n_rows; p.n_slots = c->n_slots;
    p.row_bytes = c->format == SQ_CACHE_INT4 ? c->d / 2 : c->d;
    p.slots = d_slots;
    p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    p.scales = const_cast<float*>(scales);
    return SQ_OK;
}

}  // namespace

extern "C" sq_status sq_cache_write(const sq_cache_cfg* cfg, const sq_rows* x, const int32_t* d_slots, void* d_codes,
                                    float* d_scales, void* stream) {
    CacheParams p{};
    bool vec = false, empty = false;
    SQ_TRY(cache_call(cfg, x, d_slots, d_codes, d_scales, p, vec, empty));
    if (empty) return SQ_OK;
    const hipError_t e = launch_cache_write(p, vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "cache write launch");
}

extern "C" sq_status sq_cache_read(const sq_cache_cfg* cfg, const void* d_codes, const float* d_scales, const int32_t* d_slots,
                                   const sq_rows* out, void* stream) {
    CacheParams p{};
    bool vec = false, empty = false;
    SQ_TRY(cache_call(cfg, out, d_slots, d_codes, d_scales, p, vec, empty));
    if (empty) return SQ_OK;
    const hipError_t e = launch_cache_read(p, vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SQ_OK : fail_hip(e, "cache read launch");
}
