/*
 * stepq.h -- C ABI of the MI355X (gfx950) quantized gated-delta state step.
 *
 * The library implements the decode-time hot path of STEPQuant (Yao et al.,
 * 2026, "STEPQuant: When and Where Errors Matter in Delta-Rule Recurrent State
 * Quantization"): every (request, layer, head) recurrent state S (d_k x d_v)
 * lives in a packed pool as mixed-width integer codes with a binary16 factor
 * per key row and a binary16 scale per value column, plus binary16 "pivot"
 * rows kept unquantized.  One step dequantizes the state, applies the gated
 * delta update, emits the readout y = X^T q from the float state, then refits
 * the row factors and column scales and packs the state back.
 *
 * Passages the calls follow (STEPQuant pages):
 *   - rcap.io post, decode-step pseudocode: unpack -> gated delta update ->
 *     readout before requantization -> row scales sqrt(row_mag)/sqrt(impact)
 *     -> weighted column fit -> quantize at each unit's width.
 *   - hyper.ai summary, section 方法 (Method): lifetime-aware bit allocation and
 *     FP16 pivot selection run offline; a fused kernel does chunked state
 *     reconstruction, the delta update and the readout; the dual-axis fit and
 *     packed write-back run on a separate stream, keeping the state compressed
 *     between tokens.
 *
 * Conventions
 *   - All sizes are element counts unless named *_bytes.
 *   - "d_" prefixed pointers are device pointers (HIP device memory on the
 *     current device); "h_" or unprefixed pointers in sq_plan_cfg are host.
 *   - Streams are passed as void* and hold a hipStream_t (NULL = the null stream).
 *   - Per-step arrays are laid out [n_layers][batch][H][d] (row-major, fp32).
 *     Device inputs must be finite (the kernels run with IEEE mode off and do
 *     not screen NaN or infinity); a non-finite input leaves the touched states
 *     unspecified, never memory outside them.
 *   - A call over an empty range (batch = 0 or n_layers = 0) validates its
 *     sizes and returns SQ_OK without touching any array (they may be NULL).
 *   - Host threads: a plan is read-only after creation and may be shared; calls
 *     on one pool may come from several threads (the split arrangement
 *     serializes its own set-up per pool).  Device work that touches the same
 *     slots must still be ordered by the caller (streams, events).
 *   - Every call validates its arguments on the host before enqueuing work and
 *     returns a negative sq_status on failure, with a message available from
 *     sq_last_error() on the calling thread.  Device work is asynchronous: a
 *     device fault surfaces at the caller's next synchronization.  No C++
 *     exception crosses this boundary.
 */
#ifndef STEPQ_H
#define STEPQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t sq_status;
#define SQ_OK                 0
#define SQ_ERR_ARG           -1   /* null pointer, bad enum, bad count */
#define SQ_ERR_SHAPE         -2   /* sizes inconsistent with the plan or the buffer */
#define SQ_ERR_UNSUPPORTED   -3   /* (d_k, d_v), width or grid size not compiled in */
#define SQ_ERR_SLOT          -4   /* slot out of range or repeated (validate mode) */
#define SQ_ERR_PLAN_MISMATCH -5   /* pool bound to another plan / layer range out of plan */
#define SQ_ERR_NOMEM         -6   /* host or device allocation failed */
#define SQ_ERR_HIP           -7   /* a HIP runtime call failed */

#define SQ_FORM_GDN 0             /* one retention gate per head: D = alpha I        */
#define SQ_FORM_KDA 1             /* one retention gate per key row: D = diag(alpha) */
#define SQ_UNIT_HEAD 0            /* allocation unit: a whole head state             */
#define SQ_UNIT_ROW  1            /* allocation unit: one key row of a head state    */
#define SQ_QUANT_DUAL_AXIS 0      /* row factors sqrt(m / w) + impact-weighted column fit (the method) */
#define SQ_QUANT_ROW_ABSMAX 1     /* per-row absmax r = m / qmax, column scales 1 (ablation: no fit) */

#define SQ_DTYPE_F32  0            /* element types of the scan's and the norms' row arrays */
#define SQ_DTYPE_BF16 1
#define SQ_DTYPE_F16  2
#define SQ_NORM_RMS 0             /* divide by sqrt(mean(x^2) + eps) */
#define SQ_NORM_L2  1             /* divide by sqrt(sum(x^2) + eps)  */
#define SQ_ACT_SILU    0          /* gate g(z) = z sigmoid(z) */
#define SQ_ACT_SIGMOID 1          /* gate g(z) = sigmoid(z)   */

#define SQ_MAX_WIDTHS 8
#define SQ_MAX_GRID   8
#define SQ_PIVOT_BITS 16          /* width reported for a pivot (binary16) unit/row  */

/* Plan configuration (host memory; read during sq_plan_create only). */
typedef struct sq_plan_cfg {
    int32_t form;                 /* SQ_FORM_GDN or SQ_FORM_KDA */
    int32_t unit;                 /* SQ_UNIT_HEAD or SQ_UNIT_ROW */
    int32_t n_layers, n_heads, d_k, d_v;
    int32_t n_widths;             /* candidate code widths, each in {2, 3, 4, 6, 8} */
    int32_t widths[SQ_MAX_WIDTHS];
    int32_t budget_milli;         /* average bits x 1000 over non-pivot units */
    int32_t pivot_ppm;            /* pivot units: ceil(pivot_ppm * units / 1e6) */
    int32_t n_grid;               /* column-scale candidates gamma (1..8), relative to the column base */
    float   grid[SQ_MAX_GRID];
    const float* gate;            /* alpha per unit for calibration: [L][H] (GDN) or [L][H][d_k] (KDA) */
    const float* impact;          /* row-impact score w [L][H][d_k]; NULL = estimate from the traces */
    const int32_t* unit_bits;     /* optional fixed allocation per unit (a candidate width, 16 = pivot); NULL = plan */
    /* calibration traces; NULL q = draw them with the built-in Philox-4x32-10 generator */
    const float* calib_q;         /* [L][H][S][T][d_k] */
    const float* calib_k;         /* [L][H][S][T][d_k] */
    const float* calib_v;         /* [L][H][S][T][d_v] */
    const float* calib_beta;      /* [L][H][S][T] */
    uint64_t calib_seed;
    int32_t calib_segments;       /* S */
    int32_t calib_len;            /* T */
    int32_t n_threads;            /* planner threads; 0 = all hardware threads */
    int32_t quantizer;            /* SQ_QUANT_DUAL_AXIS (0) or SQ_QUANT_ROW_ABSMAX (1; rcap.io post, the
                                     ablation paragraph: the allocation without the dual-axis fit) */
} sq_plan_cfg;

typedef struct sq_plan sq_plan;   /* host-side plan (opaque) */
typedef struct sq_pool sq_pool;   /* a device pool bound to a plan (opaque) */

/* Summary of a plan's layout. */
typedef struct sq_plan_desc {
    int32_t n_layers, n_heads, d_k, d_v, form, unit, n_units, n_pivot_units;
    int32_t n_grid;
    int32_t n_widths;
    int32_t widths[SQ_MAX_WIDTHS];/* candidate widths, ascending */
    uint64_t slot_bytes;          /* bytes of one slot (all layers and heads of one request) */
    double code_bits_per_entry;   /* allocated bits per state entry, pivots at 16, scales excluded */
    double stored_bits_per_entry; /* slot_bytes * 8 / (L * H * d_k * d_v): codes + scales + padding */
    double compression_vs_fp32;   /* 32 / stored_bits_per_entry */
    int32_t quantizer;            /* SQ_QUANT_* */
} sq_plan_desc;

/* ---- plan (CPU) --------------------------------------------------------
 * Offline planner (hyper.ai summary, 方法, lifetime-aware bit allocation and
 * the row-impact score): lifetime weight per unit from its mean log retention,
 * reconstruction distortion at each candidate width on calibration snapshots,
 * FP16 pivots for the riskiest units, an exact budgeted allocation of widths,
 * and the packed layout.  Runs on the host only; the plan owns host memory.
 * Errors: SQ_ERR_ARG / SQ_ERR_UNSUPPORTED on bad configuration. */
sq_status sq_plan_create(const sq_plan_cfg* cfg, sq_plan** out);
void      sq_plan_destroy(sq_plan* plan);
sq_status sq_plan_describe(const sq_plan* plan, sq_plan_desc* out);
/* Per-unit planner quantities (host arrays of n_units; any pointer may be NULL):
 * mean log retention, lifetime weight, distortion [n_units][n_widths], width (16 = pivot). */
sq_status sq_plan_units(const sq_plan* plan, double* lbar, double* lifetime, double* distortion,
                        int32_t* unit_bits);
/* Per-row tables in canonical row order (host arrays [L][H][d_k]; any may be NULL):
 * quantization width (16 = pivot row) and the row-impact score used by the step. */
sq_status sq_plan_rows(const sq_plan* plan, int32_t* row_bits, float* impact);
/* Serialize to / restore from a byte buffer (host).  With buf == NULL, *bytes
 * receives the size needed.  sq_plan_load validates the buffer. */
sq_status sq_plan_save(const sq_plan* plan, void* buf, size_t* bytes);
sq_status sq_plan_load(const void* buf, size_t bytes, sq_plan** out);
/* The built-in calibration generator for one (layer, head): q, k [S][T][d_k]
 * (unit L2 norm), v [S][T][d_v], beta [S][T] (host arrays, fp32). */
sq_status sq_calib_generate(uint64_t seed, int32_t layer, int32_t head, int32_t n_seg,
                            int32_t seg_len, int32_t d_k, int32_t d_v,
                            float* q, float* k, float* v, float* beta);

/* ---- pool (device) -----------------------------------------------------
 * The caller owns the pool memory: n_slots slots of desc.slot_bytes each.  A
 * request's state for (layer l, head h) lives in its slot at the plan's
 * offset for (l, h).  Binding copies the plan's layout tables to the current
 * device (the pool object owns those small allocations until destroyed); calls
 * on the pool must run with that device current, otherwise SQ_ERR_ARG.  A slot
 * whose bytes are all zero holds the zero state (its scales are 0), so a new
 * request's slot may be cleared instead of imported.  Every call below that
 * takes d_slots skips a request whose slot lies outside [0, n_slots): no pool
 * byte is touched for it and its outputs keep their previous contents
 * (sq_state_step with SQ_STEP_VALIDATE returns SQ_ERR_SLOT instead). */
sq_status sq_pool_bytes(const sq_plan* plan, int32_t n_slots, size_t* bytes);
sq_status sq_pool_create(const sq_plan* plan, void* d_pool, size_t pool_bytes, int32_t n_slots,
                         sq_pool** out);
void      sq_pool_destroy(sq_pool* pool);
/* The same three calls under the names the method's decode-step interface is usually described
 * with: sq_plan_info = sq_plan_describe, sq_pool_bind = sq_pool_create (the caller's device buffer
 * is bound, not allocated), sq_pool_release = sq_pool_destroy. */
sq_status sq_plan_info(const sq_plan* plan, sq_plan_desc* out);
sq_status sq_pool_bind(const sq_plan* plan, void* d_pool, size_t pool_bytes, int32_t n_slots,
                       sq_pool** out);
void      sq_pool_release(sq_pool* pool);

#define SQ_STEP_SPLIT    1u       /* two kernels: readout on stream_main, fit + pack on stream_aux */
#define SQ_STEP_VALIDATE 2u       /* copy the slot list to the host and check range and uniqueness */
#define SQ_STEP_NO_JOIN  4u       /* with SQ_STEP_SPLIT: return without making stream_main wait for stream_aux */

/* ---- state_step --------------------------------------------------------
 * One decode step for batch requests over layers [layer0, layer0 + n_layers)
 * and every head (rcap.io post, decode-step pseudocode; hyper.ai 方法):
 *   S = unpack(codes, r, c, pivots);  X = D S + beta k (v^T - k^T D S);
 *   y = X^T q (written to d_y before requantization);
 *   r = binary16(sqrt(rowmax|X| / w));  c = argmin over the grid of the
 *   impact-weighted reconstruction error;  codes = clamp(rint(X / (r c))).
 * d_slots[b] is the pool slot of request b (int32, device).  d_q, d_k
 * [n_layers][batch][H][d_k]; d_v, d_y [..][d_v]; d_beta [..]; d_gate is alpha
 * in (0, 1]: [n_layers][batch][H] (GDN) or [n_layers][batch][H][d_k] (KDA).
 * Slots must be distinct within a call (otherwise the result is undefined;
 * SQ_STEP_VALIDATE checks it and returns SQ_ERR_SLOT).  Enqueued on
 * stream_main (and stream_aux with SQ_STEP_SPLIT; ordered by events, the call
 * returns with stream_main waiting for all of its work).
 * SQ_STEP_SPLIT | SQ_STEP_NO_JOIN leaves the fit + pack of the call running on
 * stream_aux so that later work on stream_main (another layer's readout, the
 * model's own kernels) overlaps it (hyper.ai summary, 方法, the second-stream
 * arrangement).  The caller then orders anything that touches the same layers
 * (the next step's call for them, sq_export, ...) after stream_aux; calls for
 * other layers may follow on stream_main at once.  The split scratch holds one
 * region per (layer, slot index < n_slots), so such calls do not share it. */
sq_status sq_state_step(sq_pool* pool, int32_t layer0, int32_t n_layers, int32_t batch,
                        const int32_t* d_slots, const float* d_q, const float* d_k,
                        const float* d_v, const float* d_gate, const float* d_beta, float* d_y,
                        void* stream_main, void* stream_aux, uint32_t flags);

/* ---- state_step, split, without allocation -----------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * two kernels as sq_state_step with SQ_STEP_SPLIT, both on one stream, with
 * the scratch e = v - k^T D S in a fixed array of SQ_SPLIT_STATIC_MAX_FLOATS
 * floats that the library holds on each GPU until the process ends (its
 * address is looked up when a pool is created on that GPU).  Same arguments
 * and layouts as sq_state_step; bitwise the same y and pool bytes.
 * n_layers * batch * H * d_v above the limit: SQ_ERR_ARG, nothing enqueued.
 * Every call on one GPU uses the same array: calls that overlap on that GPU
 * (other streams, other host threads, other pools) race and their results
 * are undefined; order them.  Makes no device allocation and no host copy. */
#define SQ_SPLIT_STATIC_MAX_FLOATS (8ll << 20)
sq_status sq_state_step_split_static(sq_pool* pool, int32_t layer0, int32_t n_layers,
                                     int32_t batch, const int32_t* d_slots, const float* d_q,
                                     const float* d_k, const float* d_v, const float* d_gate,
                                     const float* d_beta, float* d_y, void* stream);

/* ---- pack / unpack -----------------------------------------------------
 * sq_pack quantizes float states d_X [n_layers][batch][H][d_k][d_v] into the
 * slots (row factors, column fit, rounding; the requantization half of a
 * step).  sq_unpack writes the dequantized states r_i c_j Q_ij (binary16
 * value on pivot rows) to d_X in the same layout (rcap.io pseudocode, unpack). */
sq_status sq_pack(sq_pool* pool, int32_t layer0, int32_t n_layers, int32_t batch,
                  const int32_t* d_slots, const float* d_X, void* stream);
sq_status sq_unpack(sq_pool* pool, int32_t layer0, int32_t n_layers, int32_t batch,
                    const int32_t* d_slots, float* d_X, void* stream);

/* ---- export / import ---------------------------------------------------
 * Canonical (layout-independent) form of the packed states, in canonical
 * key-row order: d_codes int16 [n_layers][batch][H][d_k][d_v] holds the
 * signed code on code rows and the binary16 bit pattern on pivot rows;
 * d_r uint16 [..][d_k] binary16 row factors (1.0 on pivot rows); d_c uint16
 * [..][d_v] binary16 column scales.  Import clamps codes to each row's range. */
sq_status sq_export(sq_pool* pool, int32_t layer0, int32_t n_layers, int32_t batch,
                    const int32_t* d_slots, int16_t* d_codes, uint16_t* d_r, uint16_t* d_c,
                    void* stream);
sq_status sq_import(sq_pool* pool, int32_t layer0, int32_t n_layers, int32_t batch,
                    const int32_t* d_slots, const int16_t* d_codes, const uint16_t* d_r,
                    const uint16_t* d_c, void* stream);

/* ---- comparators (same inputs, other state formats) --------------------
 * Uniform INT8 per-row state (the baseline the pages compare against): state
 * i = (layer * n_slots + slot) * H + head holds d_k*d_v int8 codes at
 * d_codes + i*d_k*d_v and a binary32 row scale [d_k] at d_scales + i*d_k;
 * step: S = s_i Q, the same update and readout, s_i = max_j |X_ij| / 127,
 * Q = clamp(rint(X / s_i), +-127).  The codes of a state are group-interleaved
 * like the pool's 8-bit containers: with cpl = max(1, d_v / 64) columns per lane,
 * lpr = d_v / cpl lanes and gr = 16 / cpl rows per group, code (i, j) sits at
 * byte ((i / gr) * lpr + j / cpl) * 16 + (i % gr) * cpl + j % cpl of the state.
 * sq_fp32_step keeps float states d_S [(layer * n_slots + slot) * H + head]
 * [d_k][d_v] row-major (no quantization).  Alignment: d_codes to 16 bytes, d_S
 * to 4 * cpl bytes; otherwise SQ_ERR_ARG. */
sq_status sq_int8_step(int32_t form, int32_t n_heads, int32_t dim_k, int32_t dim_v, int32_t n_slots,
                       int32_t layer0, int32_t n_layers, int32_t batch, const int32_t* d_slots,
                       int8_t* d_codes, float* d_scales, const float* d_q, const float* d_k,
                       const float* d_v, const float* d_gate, const float* d_beta, float* d_y,
                       void* stream);
sq_status sq_fp32_step(int32_t form, int32_t n_heads, int32_t dim_k, int32_t dim_v, int32_t n_slots,
                       int32_t layer0, int32_t n_layers, int32_t batch, const int32_t* d_slots,
                       float* d_S, const float* d_q, const float* d_k, const float* d_v,
                       const float* d_gate, const float* d_beta, float* d_y, void* stream);
/* Streaming copy of n_bytes (multiple of 16, 16-byte aligned) for measuring achievable HBM bandwidth. */
sq_status sq_copy(const void* d_src, void* d_dst, size_t n_bytes, void* stream);
/* VALU issue-rate probe for measuring the instruction-issue ceiling of the step's occupancy:
 * n_blocks workgroups of 256 threads (4 wave64, one per SIMD), each lane running 8 independent
 * chains of 1024 fp32 FMAs, with dynamic LDS reserved so that at most waves_per_simd (1..8)
 * workgroups, i.e. waves per SIMD, are resident on a CU.  d_out (device, caller-owned) receives
 * n_blocks * 256 floats (the chains' sums).  On return *n_fma holds the wave-level FMA
 * instructions the launch issues (n_blocks * 4 * 8192) and *blocks_per_cu the residency the
 * runtime reports for that LDS reservation; time the launch on `stream` with events.
 * SQ_ERR_ARG for NULL pointers or out-of-range sizes; SQ_ERR_UNSUPPORTED when the device's LDS
 * cannot cap residency at waves_per_simd (the per-workgroup LDS limit); asynchronous otherwise. */
sq_status sq_valu_probe(int32_t waves_per_simd, int32_t n_blocks, float* d_out, uint64_t* n_fma,
                        int32_t* blocks_per_cu, void* stream);

/* ---- scan: the recurrence over whole sequences ---------------------------
 * The float form of the step's recurrence over packed sequences (a prompt, several drafted tokens,
 * a training batch): per sequence b and head h, from S = d_s0[b][h] (zero if d_s0 is NULL), for the
 * tokens t of the sequence in order,
 *   X = D_t S + beta_t k_t (v_t - (D_t S)^T k_t)^T;  y_t = X^T q_t;  S = X,
 * and d_s1[b][h] = S at the end (the layout sq_pack takes and sq_unpack and sq_fp32_step have, one layer).
 * Sequence b holds the tokens [d_seq_start[b], d_seq_start[b + 1]) of the packed arrays (int32, device,
 * n_seq + 1 values, not decreasing, within [0, n_tokens]; NULL: one sequence of n_tokens).  A sequence
 * may be empty (its state is copied); tokens outside every sequence are neither read nor written.
 * Offsets that break these rules give unspecified results and touch nothing outside the arrays.
 *
 * Row arrays (sq_rows): element (token, head, j) at d_ptr[token * stride + head * d + j], so that q, k and
 * v may be parts of one wider array.  q, k: n_heads_k heads (a divisor of n_heads) of d_k elements; head h
 * reads q and k of head h / (n_heads / n_heads_k).  v, y: n_heads heads of d_v elements.  All four have the
 * element type cfg->dtype; gates, beta, states and the arithmetic are float32 (the chunks' products on the bfloat16
 * matrix units with every float32 operand split into three parts), each output rounded once.
 * d_gate: alpha in [0, 1], [n_tokens][n_heads] (GDN) or [n_tokens][n_heads][d_k] (KDA); d_beta
 * [n_tokens][n_heads].  (The gradients of q, k and gate count gates below 1e-30 as 1e-30.)
 * Alignment: row arrays 16 bytes, with stride * element size a multiple of 16; d_gate (KDA) 16 bytes;
 * the workspace 256 bytes.  Strides at least heads * d and below 2^24 elements.
 * d_s0 and d_s1 may be the same array; no other two arrays may overlap.
 *
 * Workspace: sq_delta_scan_bytes bytes of device memory, the caller's, free again when the call's work on
 * `stream` is done; calls that may overlap (two streams, or two captured graphs whose replays overlap)
 * need one each.  No call allocates or synchronizes, so all of them can be captured.
 * The result does not depend on what else runs (no atomics; sums in a fixed order).  sq_delta_scan takes the sequences of at
 * most 16 tokens of a call with 12 or fewer a sequence token by token if d_k is 64 or more; all others, and everything in
 * sq_delta_scan_bwd, go in chunks of 32 tokens from a sequence's start.  The two ways agree to float32 rounding for finite
 * values.  A result that the formula makes NaN or infinite (from an input or a state, or a value above 3.38e38 on the way)
 * is not finite here either, but in chunks it may be NaN where the formula keeps an infinity, and the same head's results of
 * the other tokens of its chunk, those before it among them, may be NaN too.  Chunks before it in sq_delta_scan, other heads
 * and other sequences keep their results. */
typedef struct sq_rows {
    void* d_ptr;
    int64_t stride;               /* elements from one token (row) to the next */
} sq_rows;

typedef struct sq_scan_cfg {
    int32_t form;                 /* SQ_FORM_GDN or SQ_FORM_KDA */
    int32_t dtype;                /* SQ_DTYPE_*: q, k, v, y and their gradients */
    int32_t n_heads, n_heads_k;   /* heads of v, y and the states; heads of q and k */
    int32_t d_k, d_v;             /* a pair of sq_supported_shapes */
    int32_t n_seq;
    int64_t n_tokens;             /* tokens of the packed arrays, below 2^31 */
    const int32_t* d_seq_start;
} sq_scan_cfg;

/* Bytes of workspace for sq_delta_scan (backward = 0) or sq_delta_scan_bwd (1); d_seq_start is not read. */
sq_status sq_delta_scan_bytes(const sq_scan_cfg* cfg, int32_t backward, size_t* bytes);
sq_status sq_delta_scan(const sq_scan_cfg* cfg, const sq_rows* q, const sq_rows* k, const sq_rows* v,
                        const float* d_gate, const float* d_beta, const float* d_s0, const sq_rows* y,
                        float* d_s1, void* d_work, size_t work_bytes, void* stream);
/* Gradients of sq_delta_scan: from dy (the gradient of y) and d_ds1 (of the final states, NULL = zero) the
 * gradients of q, k, v (dtype; dq and dk summed over the heads that share them), gate, beta and the first
 * states (float32, the inputs' layouts; d_ds0 may be NULL, and may be d_ds1).  Nothing of the forward call
 * is needed: the states are computed again.  d_s0 as in the forward call. */
sq_status sq_delta_scan_bwd(const sq_scan_cfg* cfg, const sq_rows* q, const sq_rows* k, const sq_rows* v,
                            const float* d_gate, const float* d_beta, const float* d_s0, const sq_rows* dy,
                            const float* d_ds1, const sq_rows* dq, const sq_rows* dk, const sq_rows* dv,
                            float* d_dgate, float* d_dbeta, float* d_ds0, void* d_work, size_t work_bytes,
                            void* stream);

/* ---- norms around the recurrence -----------------------------------------
 * Rows of d elements: row (i, j), i < n_outer, j < n_inner, at d_ptr[i * stride + j * d] (a token's heads
 * lie side by side; n_inner = 1 for plain rows), of any length d from 1 to 16384.  Statistics and sums in float32,
 * each output rounded once.  inv(a) = 1 / sqrt(mean(a^2) + eps) (SQ_NORM_RMS) or 1 / sqrt(sum(a^2) + eps)
 * (SQ_NORM_L2: rows of unit norm, as the step and the scan take q and k).
 *   sq_norm_in  (before a block):  h = x + res_scale * chan_scale * r;   n = out_scale * weight * h * inv(h)
 *   sq_norm_out (after a block):   o = x + res_scale * chan_scale * (weight * y * inv(y) * act(z))
 * weight and chan_scale: float32 [d], NULL = 1.  r (with h), z and x may be NULL: no residual, no gate.
 * Types: in: x, r, h cfg->dtype, n cfg->dtype_out; out: y cfg->dtype, z, x, o cfg->dtype_out; gradients have
 * their array's type, those of weight and chan_scale are float32.
 * An output may be an input's own array if its type and stride are the same; arrays must not overlap otherwise.
 * Rows whose arrays all start at 16 bytes, with strides and d multiples of 8, are read 16 bytes at a time.
 *
 * sq_norm_in_bwd: from h, dn and (optional) dh, the gradient that reaches h past the norm:
 *   dx = dh + d(n)/d(h) dn;  dr = res_scale * chan_scale * dx;  dweight = sum over rows of out_scale * dn * h * inv(h);
 *   dchan_scale = sum over rows of res_scale * dx * r.
 * sq_norm_out_bwd: from y, z, do: dy, dz, dweight, dchan_scale (the gradient of x is do itself).
 * dr, dz, d_dweight, d_dchan_scale may be NULL; r is needed for d_dchan_scale only.  With no rows the sums are written as zero.
 * Sums over rows are taken in a fixed order through a workspace of sq_norm_bytes bytes (used if d_dweight or
 * d_dchan_scale is given), under the rules of the scan's. */
typedef struct sq_norm_cfg {
    int32_t dtype, dtype_out;     /* SQ_DTYPE_* */
    int32_t kind;                 /* SQ_NORM_RMS or SQ_NORM_L2 */
    int32_t act;                  /* SQ_ACT_*, sq_norm_out only */
    int64_t n_outer;
    int32_t n_inner, d;
    float eps, res_scale, out_scale;
} sq_norm_cfg;

sq_status sq_norm_bytes(int64_t n_rows, int32_t d, size_t* bytes);
sq_status sq_norm_in(const sq_norm_cfg* cfg, const sq_rows* x, const sq_rows* r, const float* d_weight,
                     const float* d_chan_scale, const sq_rows* h, const sq_rows* n, void* stream);
sq_status sq_norm_in_bwd(const sq_norm_cfg* cfg, const sq_rows* h, const sq_rows* dn, const sq_rows* dh,
                         const sq_rows* r, const float* d_weight, const float* d_chan_scale, const sq_rows* dx,
                         const sq_rows* dr, float* d_dweight, float* d_dchan_scale, void* d_work,
                         size_t work_bytes, void* stream);
sq_status sq_norm_out(const sq_norm_cfg* cfg, const sq_rows* y, const sq_rows* z, const sq_rows* x,
                      const float* d_weight, const float* d_chan_scale, const sq_rows* o, void* stream);
sq_status sq_norm_out_bwd(const sq_norm_cfg* cfg, const sq_rows* y, const sq_rows* z, const sq_rows* d_o,
                          const float* d_weight, const float* d_chan_scale, const sq_rows* dy, const sq_rows* dz,
                          float* d_dweight, float* d_dchan_scale, void* d_work, size_t work_bytes, void* stream);

/* ---- errors / info ------------------------------------------------------ */
const char* sq_status_str(sq_status s);
const char* sq_last_error(void);          /* thread-local; "" if none */
/* Shapes (d_k, d_v) the step kernels are compiled for, as pairs: out[2i], out[2i+1]. */
int32_t     sq_supported_shapes(int32_t* out, int32_t max_pairs);

#ifdef __cplusplus
}
#endif
#endif /* STEPQ_H */
