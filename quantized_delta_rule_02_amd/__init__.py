"""Python binding of libstepq (the MI355X quantized gated-delta state step).

Thin marshalling over the C ABI in include/stepq.h: every function here has the
name of the C call it wraps, converts its arguments (numpy arrays for host
data, torch CUDA tensors for device data, torch streams) and raises StepQError
on a negative status.  All computation runs in the library's HIP kernels and
C++ runtime; there is no Python or CPU fallback.
"""
from __future__ import annotations

import ctypes
from ctypes import POINTER, byref, c_double, c_float, c_int32, c_size_t, c_uint64, c_void_p

import numpy as np

from . import _lib
from ._lib import (SQ_ACT_NONE, SQ_ACT_SIGMOID, SQ_ACT_SILU, SQ_CACHE_E4M3, SQ_CACHE_INT4, SQ_CACHE_INT8, SQ_DTYPE_BF16, SQ_DTYPE_F16, SQ_DTYPE_F32, SQ_NORM_L2, SQ_NORM_RMS, SQ_FORM_GDN, SQ_FORM_KDA, SQ_PIVOT_BITS, SQ_QUANT_DUAL_AXIS, SQ_QUANT_ROW_ABSMAX,
                   SQ_SPLIT_STATIC_MAX_FLOATS, SQ_STEP_NO_JOIN, SQ_STEP_SPLIT, SQ_STEP_VALIDATE, SQ_UNIT_HEAD,
                   SQ_UNIT_ROW)

__all__ = [
    "StepQError", "Plan", "Pool", "sq_plan_create", "sq_plan_describe", "sq_plan_info", "sq_pool_bind", "sq_pool_release", "sq_plan_units", "sq_plan_rows",
    "sq_plan_save", "sq_plan_load", "sq_calib_generate", "sq_pool_bytes", "sq_pool_create", "sq_state_step", "sq_state_step_split_static",
    "sq_pack", "sq_unpack", "sq_export", "sq_import", "sq_int8_step", "sq_fp32_step", "sq_copy", "sq_valu_probe",
    "sq_delta_scan_bytes", "sq_delta_scan", "sq_delta_scan_bwd", "sq_norm_bytes", "sq_norm_in", "sq_norm_in_bwd", "sq_norm_out", "sq_norm_out_bwd",
    "sq_conv_bytes", "sq_conv", "sq_conv_bwd", "sq_conv_step", "sq_ssm_scan_bytes", "sq_ssm_scan", "sq_ssm_scan_bwd", "sq_ssm_step",
    "sq_cache_write", "sq_cache_read", "SQ_ACT_NONE", "SQ_CACHE_INT8", "SQ_CACHE_INT4", "SQ_CACHE_E4M3",
    "SQ_DTYPE_F32", "SQ_DTYPE_BF16", "SQ_DTYPE_F16", "SQ_NORM_RMS", "SQ_NORM_L2", "SQ_ACT_SILU", "SQ_ACT_SIGMOID",
    "sq_supported_shapes", "SQ_FORM_GDN", "SQ_FORM_KDA", "SQ_UNIT_HEAD", "SQ_UNIT_ROW", "SQ_STEP_SPLIT",
    "SQ_STEP_VALIDATE", "SQ_STEP_NO_JOIN", "SQ_SPLIT_STATIC_MAX_FLOATS", "SQ_PIVOT_BITS", "SQ_QUANT_DUAL_AXIS", "SQ_QUANT_ROW_ABSMAX",
]


class StepQError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib.load()
        self.status = status
        msg = lib.sq_last_error().decode()
        super().__init__(f"{where}: {lib.sq_status_str(status).decode()} ({status}): {msg}")


def _check(status: int, where: str):
    if status != 0:
        raise StepQError(status, where)


def _fptr(a, dtype=np.float32, ctype=c_float):
    if a is None:
        return None, None
    arr = np.ascontiguousarray(a, dtype=dtype)
    return arr, arr.ctypes.data_as(POINTER(ctype))


# ---------------------------------------------------------------- plan

class Plan:
    """Owns an sq_plan handle (host memory)."""

    def __init__(self, handle: int):
        self.handle = c_void_p(handle)
        self.desc = sq_plan_describe(self)

    def close(self):
        if self.handle and self.handle.value:
            _lib.load().sq_plan_destroy(self.handle)
            self.handle = c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sq_plan_create(*, form, unit, n_layers, n_heads, d_k, d_v, widths, budget_milli, pivot_ppm, grid, gate,
                   impact=None, unit_bits=None, calib=None, calib_seed=0, calib_segments=32, calib_len=512,
                   n_threads=0, quantizer=SQ_QUANT_DUAL_AXIS) -> Plan:
    """Run the offline planner.  gate/impact/unit_bits/calib are host arrays (calib = (q, k, v, beta))."""
    lib = _lib.load()
    cfg = _lib.SqPlanCfg()
    cfg.form, cfg.unit = int(form), int(unit)
    cfg.n_layers, cfg.n_heads, cfg.d_k, cfg.d_v = int(n_layers), int(n_heads), int(d_k), int(d_v)
    widths = list(widths)
    if not 1 <= len(widths) <= _lib.SQ_MAX_WIDTHS:
        raise ValueError(f"between 1 and {_lib.SQ_MAX_WIDTHS} candidate widths")
    cfg.n_widths = len(widths)
    for i, b in enumerate(widths):
        cfg.widths[i] = int(b)
    cfg.budget_milli, cfg.pivot_ppm = int(budget_milli), int(pivot_ppm)
    grid = list(grid)
    if not 1 <= len(grid) <= _lib.SQ_MAX_GRID:
        raise ValueError("between 1 and 8 grid candidates")
    cfg.n_grid = len(grid)
    for i, g in enumerate(grid):
        cfg.grid[i] = float(g)
    keep = []
    n_gate = n_layers * n_heads * (d_k if form == SQ_FORM_KDA else 1)
    g_arr, cfg.gate = _fptr(gate)
    if g_arr.size != n_gate:
        raise ValueError(f"gate has {g_arr.size} values, expected {n_gate}")
    keep.append(g_arr)
    if impact is not None:
        i_arr, cfg.impact = _fptr(impact)
        if i_arr.size != n_layers * n_heads * d_k:
            raise ValueError("impact must have L * H * d_k values")
        keep.append(i_arr)
    if unit_bits is not None:
        u_arr, cfg.unit_bits = _fptr(unit_bits, np.int32, c_int32)
        n_units = n_layers * n_heads * (d_k if unit == SQ_UNIT_ROW else 1)
        if u_arr.size != n_units:
            raise ValueError(f"unit_bits has {u_arr.size} values, expected {n_units}")
        keep.append(u_arr)
    if calib is not None:
        q, k, v, b = calib
        nt = n_layers * n_heads * calib_segments * calib_len
        arrs = []
        for a, per in ((q, d_k), (k, d_k), (v, d_v), (b, 1)):
            arr, _ = _fptr(a)
            if arr.size != nt * per:
                raise ValueError("calibration trace size does not match L * H * segments * len")
            arrs.append(arr)
        keep.extend(arrs)
        cfg.calib_q = arrs[0].ctypes.data_as(POINTER(c_float))
        cfg.calib_k = arrs[1].ctypes.data_as(POINTER(c_float))
        cfg.calib_v = arrs[2].ctypes.data_as(POINTER(c_float))
        cfg.calib_beta = arrs[3].ctypes.data_as(POINTER(c_float))
    cfg.calib_seed = int(calib_seed)
    cfg.calib_segments, cfg.calib_len, cfg.n_threads = int(calib_segments), int(calib_len), int(n_threads)
    cfg.quantizer = int(quantizer)
    out = c_void_p()
    _check(lib.sq_plan_create(byref(cfg), byref(out)), "sq_plan_create")
    return Plan(out.value)


def sq_plan_describe(plan: Plan, _entry="sq_plan_describe") -> dict:
    d = _lib.SqPlanDesc()
    _check(getattr(_lib.load(), _entry)(plan.handle, byref(d)), _entry)
    out = {name: getattr(d, name) for name, _ in d._fields_}
    out["widths"] = [int(d.widths[i]) for i in range(d.n_widths)]
    return out


def sq_plan_info(plan: Plan) -> dict:
    """sq_plan_describe under its other name (the C ABI exports both)."""
    return sq_plan_describe(plan, _entry="sq_plan_info")


def sq_plan_units(plan: Plan) -> dict:
    d = plan.desc
    U = d["n_units"]
    nw = len(d["widths"])
    lbar = np.zeros(U, np.float64)
    L = np.zeros(U, np.float64)
    D = np.zeros((U, nw), np.float64)
    ub = np.zeros(U, np.int32)
    _check(_lib.load().sq_plan_units(plan.handle, lbar.ctypes.data_as(POINTER(c_double)),
                                     L.ctypes.data_as(POINTER(c_double)), D.ctypes.data_as(POINTER(c_double)),
                                     ub.ctypes.data_as(POINTER(c_int32))), "sq_plan_units")
    return {"lbar": lbar, "lifetime": L, "distortion": D, "unit_bits": ub}


def sq_plan_rows(plan: Plan):
    d = plan.desc
    n = d["n_layers"] * d["n_heads"] * d["d_k"]
    rb = np.zeros(n, np.int32)
    w = np.zeros(n, np.float32)
    _check(_lib.load().sq_plan_rows(plan.handle, rb.ctypes.data_as(POINTER(c_int32)),
                                    w.ctypes.data_as(POINTER(c_float))), "sq_plan_rows")
    shape = (d["n_layers"], d["n_heads"], d["d_k"])
    return rb.reshape(shape), w.reshape(shape)


def sq_plan_save(plan: Plan) -> bytes:
    lib = _lib.load()
    n = c_size_t(0)
    _check(lib.sq_plan_save(plan.handle, None, byref(n)), "sq_plan_save")
    buf = ctypes.create_string_buffer(n.value)
    _check(lib.sq_plan_save(plan.handle, buf, byref(n)), "sq_plan_save")
    return buf.raw[: n.value]


def sq_plan_load(data: bytes) -> Plan:
    out = c_void_p()
    buf = ctypes.create_string_buffer(bytes(data), len(data))
    _check(_lib.load().sq_plan_load(buf, len(data), byref(out)), "sq_plan_load")
    return Plan(out.value)


def sq_calib_generate(seed, layer, head, n_seg, seg_len, d_k, d_v):
    q = np.zeros((n_seg, seg_len, d_k), np.float32)
    k = np.zeros_like(q)
    v = np.zeros((n_seg, seg_len, d_v), np.float32)
    b = np.zeros((n_seg, seg_len), np.float32)
    P = POINTER(c_float)
    _check(_lib.load().sq_calib_generate(int(seed), layer, head, n_seg, seg_len, d_k, d_v, q.ctypes.data_as(P),
                                         k.ctypes.data_as(P), v.ctypes.data_as(P), b.ctypes.data_as(P)),
           "sq_calib_generate")
    return q, k, v, b


def sq_supported_shapes():
    lib = _lib.load()
    n = lib.sq_supported_shapes(None, 0)
    buf = (c_int32 * (2 * n))()
    lib.sq_supported_shapes(buf, n)
    return [(buf[2 * i], buf[2 * i + 1]) for i in range(n)]


# ---------------------------------------------------------------- device helpers

def _dev(t, dtype, numel, name):
    """Device pointer of a contiguous CUDA tensor with at least numel elements of dtype."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return c_void_p(t.data_ptr())


def _stream(s):
    import torch
    if s is None:
        s = torch.cuda.current_stream()
    return c_void_p(s.cuda_stream if hasattr(s, "cuda_stream") else int(s))


class Pool:
    """An sq_pool bound to caller-owned device memory (the tensor is kept alive here)."""

    def __init__(self, handle: int, plan: Plan, memory, n_slots: int):
        self.handle = c_void_p(handle)
        self.plan = plan
        self.memory = memory
        self.n_slots = n_slots
        d = plan.desc
        self.L, self.H, self.d_k, self.d_v, self.form = d["n_layers"], d["n_heads"], d["d_k"], d["d_v"], d["form"]

    def close(self):
        if self.handle and self.handle.value:
            _lib.load().sq_pool_destroy(self.handle)
            self.handle = c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sq_pool_bytes(plan: Plan, n_slots: int) -> int:
    n = c_size_t(0)
    _check(_lib.load().sq_pool_bytes(plan.handle, n_slots, byref(n)), "sq_pool_bytes")
    return n.value


def sq_pool_create(plan: Plan, memory, n_slots: int, _entry="sq_pool_create") -> Pool:
    """memory: a uint8 CUDA tensor of at least sq_pool_bytes(plan, n_slots) bytes."""
    import torch
    nbytes = sq_pool_bytes(plan, n_slots)
    ptr = _dev(memory, torch.uint8, nbytes, "pool memory")
    out = c_void_p()
    _check(getattr(_lib.load(), _entry)(plan.handle, ptr, memory.numel(), n_slots, byref(out)), _entry)
    return Pool(out.value, plan, memory, n_slots)


def sq_pool_bind(plan: Plan, memory, n_slots: int) -> Pool:
    """sq_pool_create under its other name (the C ABI exports both): binds caller-owned memory."""
    return sq_pool_create(plan, memory, n_slots, _entry="sq_pool_bind")


def sq_pool_release(pool: Pool) -> None:
    """Release a pool's device tables (the C ABI's sq_pool_release); the caller's memory stays."""
    if pool.handle and pool.handle.value:
        _lib.load().sq_pool_release(pool.handle)
        pool.handle = c_void_p(None)


def sq_state_step(pool: Pool, layer0, n_layers, batch, slots, q, k, v, gate, beta, y,
                  stream_main=None, stream_aux=None, flags=0):
    import torch
    n = n_layers * batch * pool.H
    f = torch.float32
    n_gate = n * (pool.d_k if pool.form == SQ_FORM_KDA else 1)
    aux = _stream(stream_aux) if stream_aux is not None else None
    _check(_lib.load().sq_state_step(
        pool.handle, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
        _dev(q, f, n * pool.d_k, "q"), _dev(k, f, n * pool.d_k, "k"), _dev(v, f, n * pool.d_v, "v"),
        _dev(gate, f, n_gate, "gate"), _dev(beta, f, n, "beta"), _dev(y, f, n * pool.d_v, "y"),
        _stream(stream_main), aux, int(flags)), "sq_state_step")


def sq_state_step_split_static(pool: Pool, layer0, n_layers, batch, slots, q, k, v, gate, beta, y, stream=None):
    """The split step with the library's fixed per-GPU scratch (no device allocation)."""
    import torch
    n = n_layers * batch * pool.H
    f = torch.float32
    n_gate = n * (pool.d_k if pool.form == SQ_FORM_KDA else 1)
    _check(_lib.load().sq_state_step_split_static(
        pool.handle, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
        _dev(q, f, n * pool.d_k, "q"), _dev(k, f, n * pool.d_k, "k"), _dev(v, f, n * pool.d_v, "v"),
        _dev(gate, f, n_gate, "gate"), _dev(beta, f, n, "beta"), _dev(y, f, n * pool.d_v, "y"),
        _stream(stream)), "sq_state_step_split_static")


def sq_pack(pool: Pool, layer0, n_layers, batch, slots, X, stream=None):
    import torch
    n = n_layers * batch * pool.H * pool.d_k * pool.d_v
    _check(_lib.load().sq_pack(pool.handle, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
                               _dev(X, torch.float32, n, "X"), _stream(stream)), "sq_pack")


def sq_unpack(pool: Pool, layer0, n_layers, batch, slots, X, stream=None):
    import torch
    n = n_layers * batch * pool.H * pool.d_k * pool.d_v
    _check(_lib.load().sq_unpack(pool.handle, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
                                 _dev(X, torch.float32, n, "X"), _stream(stream)), "sq_unpack")


def sq_export(pool: Pool, layer0, n_layers, batch, slots, codes, r, c, stream=None):
    import torch
    n = n_layers * batch * pool.H
    _check(_lib.load().sq_export(pool.handle, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
                                 _dev(codes, torch.int16, n * pool.d_k * pool.d_v, "codes"),
                                 _dev(r, torch.int16, n * pool.d_k, "r"), _dev(c, torch.int16, n * pool.d_v, "c"),
                                 _stream(stream)), "sq_export")


def sq_import(pool: Pool, layer0, n_layers, batch, slots, codes, r, c, stream=None):
    import torch
    n = n_layers * batch * pool.H
    _check(_lib.load().sq_import(pool.handle, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
                                 _dev(codes, torch.int16, n * pool.d_k * pool.d_v, "codes"),
                                 _dev(r, torch.int16, n * pool.d_k, "r"), _dev(c, torch.int16, n * pool.d_v, "c"),
                                 _stream(stream)), "sq_import")


def sq_int8_step(form, n_heads, d_k, d_v, n_slots, layer0, n_layers, batch, slots, codes, scales,
                 q, k, v, gate, beta, y, stream=None):
    import torch
    n = n_layers * batch * n_heads
    n_states = (layer0 + n_layers) * n_slots * n_heads
    f = torch.float32
    _check(_lib.load().sq_int8_step(
        form, n_heads, d_k, d_v, n_slots, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
        _dev(codes, torch.int8, n_states * d_k * d_v, "codes"), _dev(scales, f, n_states * d_k, "scales"),
        _dev(q, f, n * d_k, "q"), _dev(k, f, n * d_k, "k"), _dev(v, f, n * d_v, "v"),
        _dev(gate, f, n * (d_k if form == SQ_FORM_KDA else 1), "gate"), _dev(beta, f, n, "beta"),
        _dev(y, f, n * d_v, "y"), _stream(stream)), "sq_int8_step")


def sq_fp32_step(form, n_heads, d_k, d_v, n_slots, layer0, n_layers, batch, slots, S, q, k, v, gate, beta, y,
                 stream=None):
    import torch
    n = n_layers * batch * n_heads
    n_states = (layer0 + n_layers) * n_slots * n_heads
    f = torch.float32
    _check(_lib.load().sq_fp32_step(
        form, n_heads, d_k, d_v, n_slots, layer0, n_layers, batch, _dev(slots, torch.int32, batch, "slots"),
        _dev(S, f, n_states * d_k * d_v, "S"), _dev(q, f, n * d_k, "q"), _dev(k, f, n * d_k, "k"),
        _dev(v, f, n * d_v, "v"), _dev(gate, f, n * (d_k if form == SQ_FORM_KDA else 1), "gate"),
        _dev(beta, f, n, "beta"), _dev(y, f, n * d_v, "y"), _stream(stream)), "sq_fp32_step")


def sq_copy(src, dst, n_bytes=None, stream=None):
    import torch
    nb = src.numel() * src.element_size() if n_bytes is None else int(n_bytes)
    if src.numel() * src.element_size() < nb or dst.numel() * dst.element_size() < nb:
        raise ValueError("copy larger than the tensors")
    _check(_lib.load().sq_copy(c_void_p(src.data_ptr()), c_void_p(dst.data_ptr()), nb, _stream(stream)), "sq_copy")


def sq_valu_probe(waves_per_simd, out, stream=None):
    """Launch the FMA issue-rate probe over out.numel() // 256 workgroups (out: float32 on the GPU).
    Returns (wave-level FMA instructions issued, workgroups resident per CU)."""
    import torch
    n_blocks = out.numel() // 256
    if out.dtype != torch.float32 or not out.is_cuda or n_blocks < 1:
        raise ValueError("out must be a float32 GPU tensor of at least 256 elements")
    n = c_uint64(0)
    fit = c_int32(0)
    _check(_lib.load().sq_valu_probe(int(waves_per_simd), n_blocks, c_void_p(out.data_ptr()), byref(n), byref(fit),
                                     _stream(stream)), "sq_valu_probe")
    return n.value, fit.value


# ---------------------------------------------------------------- scan and norms

_DTYPES = {}                 # torch's element types to SQ_DTYPE_*


def _types() -> dict:
    import torch
    _DTYPES.update({torch.float32: SQ_DTYPE_F32, torch.bfloat16: SQ_DTYPE_BF16, torch.float16: SQ_DTYPE_F16})
    return _DTYPES


def _dtype_code(dtype) -> int:
    code = (_DTYPES or _types()).get(dtype)
    if code is None:
        raise TypeError(f"element type {dtype}: float32, bfloat16 or float16")
    return code


def _fits(*numbers):
    """Refuses what a 32-bit field of a configuration does not hold (ctypes would keep its low bits: another, smaller call)."""
    if max(numbers) > 0x7fffffff or min(numbers) < -0x80000000:
        raise ValueError(f"{[n for n in numbers if not -0x80000000 <= n <= 0x7fffffff][0]}: sizes are numbers of 32 bits")


_raw_stream = None           # (device index) -> handle of its current stream, and the current device's index


def _stream_calls():
    """torch's own lookups behind torch.cuda.current_stream and current_device, without the objects they build (2 us a call); the public
    calls in a torch that has none of these names."""
    global _raw_stream
    import torch
    torch.cuda.current_stream()                          # initialises torch's side
    raw, current = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    _raw_stream = (raw or (lambda index: torch.cuda.current_stream(index).cuda_stream), current or torch.cuda.current_device)
    return _raw_stream


def _call(fn, name, device, stream, *args):
    """fn(*args, stream handle) with `device` current (None: the device's current stream)."""
    raw, current = _raw_stream or _stream_calls()
    if stream is None:
        handle = raw(device.index)
    elif getattr(stream, "device", device) != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if current() == device.index:
        status = fn(*args, handle)
    else:
        import torch
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != 0:
        _check(status, name)


def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace, checked, or a new one that belongs to the stream of the call."""
    import torch
    if workspace is not None:
        _on(workspace, device, "workspace")
        return _dev(workspace, torch.uint8, nbytes, "workspace"), workspace.numel(), workspace
    if stream is None:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        owner = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(owner):
            buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return buf.data_ptr(), nbytes, buf


def _on(t, device, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _row_array(t, shape, dtype, device, name):
    """sq_rows of a tensor [tokens, heads, d] (or [rows, d]) whose heads lie side by side (any stride between tokens)."""
    if getattr(t, "device", None) != device:
        _on(t, device, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    T, d = shape[0], shape[-1]
    H = shape[1] if len(shape) == 3 else 1
    if ((d > 1 and st[-1] != 1) or (H > 1 and st[1] != d)) and t.numel():
        raise ValueError(f"{name}: the elements and heads of a token must be contiguous")
    return _lib.SqRows(t.data_ptr(), st[0] if T > 1 else H * d)


def _plain(t, shape, device, name):
    """Pointer of a contiguous float32 tensor of exactly this shape (None stays NULL)."""
    if t is None:
        return None
    if getattr(t, "device", None) != device:
        _on(t, device, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if (_DTYPES or _types()).get(t.dtype) != SQ_DTYPE_F32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _scan_cfg(form, q, v, seq_start):
    import torch
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dim() != 3:
            raise ValueError(f"{name} must be [tokens, heads, d]")
    T, Hk, dk = q.shape
    H, dv = v.shape[1:]
    n_seq, start = 1, None
    if seq_start is not None:
        _on(seq_start, q.device, "seq_start")
        if seq_start.dim() != 1 or seq_start.numel() < 1:
            raise ValueError("seq_start must hold n_seq + 1 offsets")
        n_seq = seq_start.numel() - 1
        start = _dev(seq_start, torch.int32, n_seq + 1, "seq_start")
    _fits(form, H, Hk, dk, dv, n_seq)
    return _lib.SqScanCfg(int(form), _dtype_code(q.dtype), H, Hk, dk, dv, n_seq, T, start)


def sq_delta_scan_bytes(form, dtype, n_heads, n_heads_k, d_k, d_v, n_seq, n_tokens, backward=False) -> int:
    """Workspace bytes of sq_delta_scan (or of sq_delta_scan_bwd) for arrays of these sizes."""
    _fits(form, n_heads, n_heads_k, d_k, d_v, n_seq)
    cfg = _lib.SqScanCfg(int(form), _dtype_code(dtype), n_heads, n_heads_k, d_k, d_v, n_seq, n_tokens, None)
    n = c_size_t(0)
    _check(_lib.load().sq_delta_scan_bytes(byref(cfg), int(backward), byref(n)), "sq_delta_scan_bytes")
    return n.value


def _scan_bytes(cfg, backward):
    n = c_size_t(0)
    _check(_lib.load().sq_delta_scan_bytes(byref(cfg), backward, byref(n)), "sq_delta_scan_bytes")
    return n.value


def sq_delta_scan(form, q, k, v, gate, beta, y, seq_start=None, s0=None, s1=None, workspace=None, stream=None):
    """The recurrence over packed sequences: writes y and, if given, the final states s1.

    q, k [tokens, heads_k, d_k], v, y [tokens, heads, d_v] (one type; any token stride); gate [tokens, heads] or
    [tokens, heads, d_k], beta [tokens, heads], s0, s1 [n_seq, heads, d_k, d_v] float32; seq_start int32 [n_seq + 1].
    """
    cfg = _scan_cfg(form, q, v, seq_start)
    T, H, Hk, dk, dv, dev = cfg.n_tokens, cfg.n_heads, cfg.n_heads_k, cfg.d_k, cfg.d_v, q.device
    st = (cfg.n_seq, H, dk, dv)
    rows = lambda t, h, d, name: byref(_row_array(t, (T, h, d), q.dtype, dev, name))  # noqa: E731
    args = [rows(q, Hk, dk, "q"), rows(k, Hk, dk, "k"), rows(v, H, dv, "v"),
            _plain(gate, (T, H, dk) if form == SQ_FORM_KDA else (T, H), dev, "gate"), _plain(beta, (T, H), dev, "beta"),
            _plain(s0, st, dev, "s0"), rows(y, H, dv, "y"), _plain(s1, st, dev, "s1")]
    work, nbytes, keep = _workspace(workspace, _scan_bytes(cfg, 0), dev, stream)
    _call(_lib.load().sq_delta_scan, "sq_delta_scan", dev, stream, byref(cfg), *args, work, nbytes)
    del keep


def sq_delta_scan_bwd(form, q, k, v, gate, beta, dy, dq, dk, dv, dgate, dbeta, seq_start=None, s0=None, ds1=None,
                      ds0=None, workspace=None, stream=None):
    """Gradients of sq_delta_scan, from dy and (optional) ds1, into dq, dk, dv, dgate, dbeta and (optional) ds0."""
    cfg = _scan_cfg(form, q, v, seq_start)
    T, H, Hk, nk, nv, dev = cfg.n_tokens, cfg.n_heads, cfg.n_heads_k, cfg.d_k, cfg.d_v, q.device
    st, gs = (cfg.n_seq, H, nk, nv), ((T, H, nk) if form == SQ_FORM_KDA else (T, H))
    rows = lambda t, h, d, name: byref(_row_array(t, (T, h, d), q.dtype, dev, name))  # noqa: E731
    args = [rows(q, Hk, nk, "q"), rows(k, Hk, nk, "k"), rows(v, H, nv, "v"), _plain(gate, gs, dev, "gate"),
            _plain(beta, (T, H), dev, "beta"), _plain(s0, st, dev, "s0"), rows(dy, H, nv, "dy"), _plain(ds1, st, dev, "ds1"),
            rows(dq, Hk, nk, "dq"), rows(dk, Hk, nk, "dk"), rows(dv, H, nv, "dv"), _plain(dgate, gs, dev, "dgate"),
            _plain(dbeta, (T, H), dev, "dbeta"), _plain(ds0, st, dev, "ds0")]
    work, nbytes, keep = _workspace(workspace, _scan_bytes(cfg, 1), dev, stream)
    _call(_lib.load().sq_delta_scan_bwd, "sq_delta_scan_bwd", dev, stream, byref(cfg), *args, work, nbytes)
    del keep


class _NormCall:
    """The configuration and row arrays of one norm call; `first` fixes the shape: [rows, d] or [tokens, heads, d]."""

    def __init__(self, first, name):
        import torch
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        self.shape, self.device = first.shape, first.device
        n = len(self.shape)
        if n != 2 and n != 3:
            raise ValueError(f"{name} must be [rows, d] or [tokens, heads, d]")
        self.outer, self.d = self.shape[0], self.shape[-1]
        self.inner = self.shape[1] if n == 3 else 1

    def rows(self, t, dtype, name):
        return None if t is None else byref(_row_array(t, self.shape, dtype, self.device, name))

    def vec(self, t, name):
        return None if t is None else _plain(t, (self.d,), self.device, name)

    def cfg(self, dtype, dtype_out, kind, act, eps, res_scale, out_scale):
        _fits(kind, act, self.inner, self.d)
        return byref(_lib.SqNormCfg(_dtype_code(dtype), _dtype_code(dtype_out), kind, act, self.outer,
                                    self.inner, self.d, eps, res_scale, out_scale))

    def work(self, workspace, stream, wanted):
        if not wanted:
            return None, 0, None
        return _workspace(workspace, sq_norm_bytes(self.outer * self.inner, self.d), self.device, stream)


def sq_norm_bytes(n_rows, d) -> int:
    """Workspace bytes of the norms' backward passes over n_rows rows of d elements."""
    _fits(d)
    n = c_size_t(0)
    _check(_lib.load().sq_norm_bytes(int(n_rows), int(d), byref(n)), "sq_norm_bytes")
    return n.value


def sq_norm_in(x, n, weight=None, r=None, h=None, chan_scale=None, res_scale=1.0, kind=SQ_NORM_RMS, eps=1e-6,
               out_scale=1.0, stream=None):
    """h = x + res_scale chan_scale r (written if given);  n = out_scale weight h / sqrt(mean or sum of h^2 + eps)."""
    c = _NormCall(x, "x")
    args = [c.rows(x, x.dtype, "x"), c.rows(r, x.dtype, "r"), c.vec(weight, "weight"), c.vec(chan_scale, "chan_scale"),
            c.rows(h, x.dtype, "h"), c.rows(n, n.dtype, "n")]
    _call(_lib.load().sq_norm_in, "sq_norm_in", c.device, stream, c.cfg(x.dtype, n.dtype, kind, 0, eps, res_scale, out_scale), *args)


def sq_norm_in_bwd(h, dn, dx, weight=None, r=None, dh=None, dr=None, chan_scale=None, res_scale=1.0, dweight=None,
                   dchan_scale=None, kind=SQ_NORM_RMS, eps=1e-6, out_scale=1.0, workspace=None, stream=None):
    """Gradients of sq_norm_in from h, dn and (optional) dh: dx and, if given, dr, dweight, dchan_scale (needs r)."""
    c = _NormCall(h, "h")
    args = [c.rows(h, h.dtype, "h"), c.rows(dn, dn.dtype, "dn"), c.rows(dh, h.dtype, "dh"), c.rows(r, h.dtype, "r"),
            c.vec(weight, "weight"), c.vec(chan_scale, "chan_scale"), c.rows(dx, h.dtype, "dx"), c.rows(dr, h.dtype, "dr"),
            c.vec(dweight, "dweight"), c.vec(dchan_scale, "dchan_scale")]
    work, nbytes, keep = c.work(workspace, stream, dweight is not None or dchan_scale is not None)
    _call(_lib.load().sq_norm_in_bwd, "sq_norm_in_bwd", c.device, stream, c.cfg(h.dtype, dn.dtype, kind, 0, eps, res_scale, out_scale), *args, work, nbytes)
    del keep


def sq_norm_out(y, o, weight=None, z=None, act=SQ_ACT_SILU, x=None, chan_scale=None, res_scale=1.0, eps=1e-6,
                kind=SQ_NORM_RMS, stream=None):
    """o = x + res_scale chan_scale (weight y / sqrt(mean y^2 + eps) act(z)); x and z may be left out."""
    c = _NormCall(y, "y")
    args = [c.rows(y, y.dtype, "y"), c.rows(z, o.dtype, "z"), c.rows(x, o.dtype, "x"), c.vec(weight, "weight"),
            c.vec(chan_scale, "chan_scale"), c.rows(o, o.dtype, "o")]
    _call(_lib.load().sq_norm_out, "sq_norm_out", c.device, stream, c.cfg(y.dtype, o.dtype, kind, act, eps, res_scale, 1.0), *args)


def sq_norm_out_bwd(y, do, dy, weight=None, z=None, dz=None, act=SQ_ACT_SILU, chan_scale=None, res_scale=1.0,
                    dweight=None, dchan_scale=None, eps=1e-6, kind=SQ_NORM_RMS, workspace=None, stream=None):
    """Gradients of sq_norm_out from y, z and do: dy and, if given, dz, dweight, dchan_scale (that of x is do)."""
    c = _NormCall(y, "y")
    args = [c.rows(y, y.dtype, "y"), c.rows(z, do.dtype, "z"), c.rows(do, do.dtype, "do"), c.vec(weight, "weight"),
            c.vec(chan_scale, "chan_scale"), c.rows(dy, y.dtype, "dy"), c.rows(dz, do.dtype, "dz"),
            c.vec(dweight, "dweight"), c.vec(dchan_scale, "dchan_scale")]
    work, nbytes, keep = c.work(workspace, stream, dweight is not None or dchan_scale is not None)
    _call(_lib.load().sq_norm_out_bwd, "sq_norm_out_bwd", c.device, stream, c.cfg(y.dtype, do.dtype, kind, act, eps, res_scale, 1.0), *args, work, nbytes)
    del keep


# ---------------------------------------------------------------- convolution, selective scan, row cache

def _first(t, n, what, name):
    """The device of the tensor that fixes a call's sizes."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    if len(t.shape) != n:
        raise ValueError(f"{name} must be {what}")
    return t.device


def _seqs(seq_start, device):
    """n_seq and the address of the offsets (one sequence of all tokens if there are none)."""
    import torch
    if seq_start is None:
        return 1, None
    _on(seq_start, device, "seq_start")
    if seq_start.dim() != 1 or seq_start.numel() < 1:
        raise ValueError("seq_start must hold n_seq + 1 offsets")
    return seq_start.numel() - 1, _dev(seq_start, torch.int32, seq_start.numel(), "seq_start")


def _typed(t, shape, dtype, device, name):
    """Pointer of a contiguous tensor of exactly this shape and type (None stays NULL)."""
    if t is None:
        return None
    if getattr(t, "device", None) != device:
        _on(t, device, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _slots(slots, n, device):
    import torch
    return _typed(slots, (n,), torch.int32, device, "slots")


def _conv_cfg(x, weight, act, n_seq, start):
    dev = _first(x, 2, "[tokens, channels]", "x")
    _first(weight, 2, "[channels, width]", "weight")
    (T, C), W = x.shape, weight.shape[1]
    _fits(act, C, W, n_seq)
    return _lib.SqConvCfg(_dtype_code(x.dtype), int(act), C, W, n_seq, T, start), dev


def sq_conv_bytes(dtype, channels, width, n_seq, n_tokens) -> int:
    """Workspace bytes of sq_conv_bwd for arrays of these sizes."""
    _fits(channels, width, n_seq)
    cfg = _lib.SqConvCfg(_dtype_code(dtype), SQ_ACT_NONE, channels, width, n_seq, n_tokens, None)
    n = c_size_t(0)
    _check(_lib.load().sq_conv_bytes(byref(cfg), byref(n)), "sq_conv_bytes")
    return n.value


def sq_conv(x, weight, y, bias=None, act=SQ_ACT_SILU, seq_start=None, s0=None, s1=None, stream=None):
    """The causal convolution of packed sequences: writes y and, if given, each sequence's last inputs s1.

    x, y [tokens, channels] (one type; any token stride); weight [channels, width], bias [channels] float32; s0, s1
    [n_seq, width - 1, channels] of x's type; seq_start int32 [n_seq + 1].
    """
    dev = _first(x, 2, "[tokens, channels]", "x")
    n_seq, start = _seqs(seq_start, dev)
    cfg, _ = _conv_cfg(x, weight, act, n_seq, start)
    C, W = weight.shape
    st = (n_seq, W - 1, x.shape[1])
    args = [byref(_row_array(x, x.shape, x.dtype, dev, "x")), _plain(weight, (x.shape[1], W), dev, "weight"), _plain(bias, (C,), dev, "bias"),
            _typed(s0, st, x.dtype, dev, "s0"), byref(_row_array(y, x.shape, x.dtype, dev, "y")), _typed(s1, st, x.dtype, dev, "s1")]
    _call(_lib.load().sq_conv, "sq_conv", dev, stream, byref(cfg), *args)


def sq_conv_bwd(x, weight, dy, dx, dweight=None, bias=None, dbias=None, act=SQ_ACT_SILU, seq_start=None, s0=None, ds1=None,
                ds0=None, workspace=None, stream=None):
    """Gradients of sq_conv, from dy and (optional) ds1, into dx and, if given, dweight, dbias and ds0."""
    dev = _first(x, 2, "[tokens, channels]", "x")
    n_seq, start = _seqs(seq_start, dev)
    cfg, _ = _conv_cfg(x, weight, act, n_seq, start)
    W, C = weight.shape[1], x.shape[1]
    st = (n_seq, W - 1, C)
    rows = lambda t, name: byref(_row_array(t, x.shape, x.dtype, dev, name))  # noqa: E731
    args = [rows(x, "x"), _plain(weight, (C, W), dev, "weight"), _plain(bias, (C,), dev, "bias"), _typed(s0, st, x.dtype, dev, "s0"),
            rows(dy, "dy"), _typed(ds1, st, x.dtype, dev, "ds1"), rows(dx, "dx"), _plain(dweight, (C, W), dev, "dweight"),
            _plain(dbias, (C,), dev, "dbias"), _typed(ds0, st, x.dtype, dev, "ds0")]
    work, nbytes, keep = None, 0, None
    if dweight is not None or dbias is not None:
        n = c_size_t(0)
        _check(_lib.load().sq_conv_bytes(byref(cfg), byref(n)), "sq_conv_bytes")
        work, nbytes, keep = _workspace(workspace, n.value, dev, stream)
    _call(_lib.load().sq_conv_bwd, "sq_conv_bwd", dev, stream, byref(cfg), *args, work, nbytes)
    del keep


def sq_conv_step(x, weight, window, y, slots=None, bias=None, act=SQ_ACT_SILU, stream=None):
    """One token of each request: x, y [batch, channels]; window [n_slots, width - 1, channels] of x's type, updated in place."""
    cfg, dev = _conv_cfg(x, weight, act, 0, None)
    _first(window, 3, "[n_slots, width - 1, channels]", "window")
    (T, C), W = x.shape, weight.shape[1]
    args = [byref(_row_array(x, x.shape, x.dtype, dev, "x")), _plain(weight, (C, W), dev, "weight"), _plain(bias, (C,), dev, "bias"),
            _slots(slots, T, dev), window.shape[0], _typed(window, (window.shape[0], W - 1, C), x.dtype, dev, "window"),
            byref(_row_array(y, x.shape, x.dtype, dev, "y"))]
    _call(_lib.load().sq_conv_step, "sq_conv_step", dev, stream, byref(cfg), *args)


class _SsmCall:
    """The configuration and inputs of one call of the selective scan; u, a and b fix its sizes."""

    def __init__(self, u, dt, a, b, c, d, dt_bias, z, softplus, seq_start=None, step=False):
        self.dev = dev = _first(u, 2, "[tokens, channels]", "u")
        _first(a, 2, "[channels, d_state]", "a")
        _first(b, 3, "[tokens, groups, d_state]", "b")
        self.T, self.C = T, C = u.shape
        self.N, self.G = N, G = a.shape[1], b.shape[1]
        self.dtype = u.dtype
        self.n_seq, start = (0, None) if step else _seqs(seq_start, dev)
        _fits(C, N, G, self.n_seq)
        self.cfg = _lib.SqSsmCfg(_dtype_code(u.dtype), C, N, G, int(bool(softplus)), self.n_seq, T, start)
        self.inputs = _lib.SqSsmIn(self.rows(u, "u"), self.rows(dt, "dt"), self.bc(b, "b"), self.bc(c, "c"), self.rows(z, "z"),
                                   self.vec(a, (C, N), "a"), self.vec(d, (C,), "d"), self.vec(dt_bias, (C,), "dt_bias"))
        self.states = (self.n_seq, C, N)

    def _ptr(self, t, shape, name):
        if t is None:
            return None
        return ctypes.pointer(_row_array(t, shape, self.dtype, self.dev, name))     # the structure it goes into keeps it

    def rows(self, t, name):
        return self._ptr(t, (self.T, self.C), name)

    def bc(self, t, name):
        return self._ptr(t, (self.T, self.G, self.N), name)

    def vec(self, t, shape, name):
        return _plain(t, shape, self.dev, name)

    def work(self, workspace, backward, stream):
        n = c_size_t(0)
        _check(_lib.load().sq_ssm_scan_bytes(byref(self.cfg), backward, byref(n)), "sq_ssm_scan_bytes")
        return _workspace(workspace, n.value, self.dev, stream) if n.value else (None, 0, None)


def sq_ssm_scan_bytes(dtype, channels, d_state, n_groups, n_seq, n_tokens, backward=False) -> int:
    """Workspace bytes of sq_ssm_scan (or of sq_ssm_scan_bwd) for arrays of these sizes."""
    _fits(channels, d_state, n_groups, n_seq)
    cfg = _lib.SqSsmCfg(_dtype_code(dtype), channels, d_state, n_groups, 1, n_seq, n_tokens, None)
    n = c_size_t(0)
    _check(_lib.load().sq_ssm_scan_bytes(byref(cfg), int(backward), byref(n)), "sq_ssm_scan_bytes")
    return n.value


def sq_ssm_scan(u, dt, a, b, c, y, d=None, dt_bias=None, z=None, softplus=True, seq_start=None, s0=None, s1=None, workspace=None,
                stream=None):
    """The selective scan over packed sequences: writes y and, if given, the final states s1.

    u, dt, z, y [tokens, channels], b, c [tokens, groups, d_state] (one type; any token stride); a [channels, d_state], d,
    dt_bias [channels], s0, s1 [n_seq, channels, d_state] float32; seq_start int32 [n_seq + 1].
    """
    call = _SsmCall(u, dt, a, b, c, d, dt_bias, z, softplus, seq_start)
    args = [call.vec(s0, call.states, "s0"), call.rows(y, "y"), call.vec(s1, call.states, "s1")]
    work, nbytes, keep = call.work(workspace, 0, stream)
    _call(_lib.load().sq_ssm_scan, "sq_ssm_scan", call.dev, stream, byref(call.cfg), byref(call.inputs), *args, work, nbytes)
    del keep


def sq_ssm_scan_bwd(u, dt, a, b, c, dy, du, ddt, da, db, dc, d=None, dt_bias=None, z=None, dz=None, dd=None, ddt_bias=None, softplus=True,
                    seq_start=None, s0=None, ds1=None, ds0=None, workspace=None, stream=None):
    """Gradients of sq_ssm_scan, from dy and (optional) ds1: du, ddt, db, dc and, where not None, da, dz, dd, ddt_bias and ds0."""
    call = _SsmCall(u, dt, a, b, c, d, dt_bias, z, softplus, seq_start)
    C, N = call.C, call.N
    grads = _lib.SqSsmGrads(call.rows(du, "du"), call.rows(ddt, "ddt"), call.bc(db, "db"), call.bc(dc, "dc"), call.rows(dz, "dz"),
                            call.vec(da, (C, N), "da"), call.vec(dd, (C,), "dd"), call.vec(ddt_bias, (C,), "ddt_bias"))
    args = [call.vec(s0, call.states, "s0"), call.rows(dy, "dy"), call.vec(ds1, call.states, "ds1"), byref(grads), call.vec(ds0, call.states, "ds0")]
    work, nbytes, keep = call.work(workspace, 1, stream)
    _call(_lib.load().sq_ssm_scan_bwd, "sq_ssm_scan_bwd", call.dev, stream, byref(call.cfg), byref(call.inputs), *args, work, nbytes)
    del keep


def sq_ssm_step(u, dt, a, b, c, state, y, slots=None, d=None, dt_bias=None, z=None, softplus=True, stream=None):
    """One token of each request: u, dt, z, y [batch, channels], b, c [batch, groups, d_state]; state [n_slots, channels,
    d_state] float32, updated in place."""
    call = _SsmCall(u, dt, a, b, c, d, dt_bias, z, softplus, step=True)
    _first(state, 3, "[n_slots, channels, d_state]", "state")
    n = state.shape[0]
    args = [_slots(slots, call.T, call.dev), n, call.vec(state, (n, call.C, call.N), "state"), call.rows(y, "y")]
    _call(_lib.load().sq_ssm_step, "sq_ssm_step", call.dev, stream, byref(call.cfg), byref(call.inputs), *args)


def _cache_call(rows, codes, scales, slots, format, name):
    import torch
    dev = _first(rows, 2, "[rows, d]", name)
    _first(codes, 2, "[n_slots, bytes of a row]", "codes")
    _first(scales, 2, "[n_slots, d / group]", "scales")
    R, d = rows.shape
    S, groups = scales.shape
    if groups < 1 or d % groups:
        raise ValueError(f"scales: {groups} a row of {d} elements")
    _fits(format, d)
    cfg = _lib.SqCacheCfg(_dtype_code(rows.dtype), int(format), d, d // groups, R, S)
    if codes.dtype not in (torch.uint8, torch.int8):
        raise TypeError(f"codes must be uint8 or int8, got {codes.dtype}")
    held = (S, d // 2 if format == SQ_CACHE_INT4 else d)
    return (dev, byref(cfg), byref(_row_array(rows, rows.shape, rows.dtype, dev, name)), _slots(slots, R, dev),
            _typed(codes, held, codes.dtype, dev, "codes"), _plain(scales, (S, groups), dev, "scales"))


def sq_cache_write(x, codes, scales, slots=None, format=SQ_CACHE_INT8, stream=None):
    """Quantises rows x [rows, d] into slots of a cache: codes [n_slots, d] (4-bit codes: d / 2) bytes, scales [n_slots, d / group]
    float32; slots int32 [rows] (None: row i is slot i)."""
    dev, cfg, rows, at, held, scale = _cache_call(x, codes, scales, slots, format, "x")
    _call(_lib.load().sq_cache_write, "sq_cache_write", dev, stream, cfg, rows, at, held, scale)


def sq_cache_read(codes, scales, out, slots=None, format=SQ_CACHE_INT8, stream=None):
    """Reads slots of a cache back into rows out [rows, d]."""
    dev, cfg, rows, at, held, scale = _cache_call(out, codes, scales, slots, format, "out")
    _call(_lib.load().sq_cache_read, "sq_cache_read", dev, stream, cfg, held, scale, at, rows)
