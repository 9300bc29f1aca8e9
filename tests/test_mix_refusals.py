"""What the convolution, the selective scan and the row cache refuse, on the CPU: every check comes before any device call, so the
addresses here are never followed."""
import ctypes
from ctypes import byref, c_size_t

import pytest

import quantized_delta_rule_02_amd as sq
from quantized_delta_rule_02_amd import _lib

ARG, SHAPE, UNSUPPORTED = -1, -2, -3
BASE = 1 << 20           # an aligned address that nothing reads
LIB = _lib.load


def R(ptr=BASE, stride=256):
    return _lib.SqRows(ptr, stride)


def make(cls, base, kw):
    d = dict(base)
    d.update(kw)
    return cls(*[d[n] for n, _ in cls._fields_])


def ptr(r):
    return byref(r) if isinstance(r, ctypes.Structure) else r


# ---------------------------------------------------------------- convolution

CONV = dict(dtype=1, act=0, channels=256, width=4, n_seq=2, n_tokens=40, d_seq_start=BASE)


def conv(fn, cfg, **kw):
    a = dict(x=R(), w=BASE, b=BASE, s0=None, y=R(), s1=None, dy=R(), ds1=None, dx=R(), dw=BASE, db=BASE, ds0=None, work=BASE, nbytes=1 << 40, slots=BASE,
             n_slots=50, window=BASE)
    a.update(kw)
    names = {"sq_conv": ["x", "w", "b", "s0", "y", "s1"], "sq_conv_bwd": ["x", "w", "b", "s0", "dy", "ds1", "dx", "dw", "db", "ds0", "work", "nbytes"],
             "sq_conv_step": ["x", "w", "b", "slots", "n_slots", "window", "y"]}[fn]
    return getattr(LIB(), fn)(ptr(cfg), *[ptr(a[n]) for n in names], None)


@pytest.mark.parametrize("fn", ("sq_conv", "sq_conv_bwd", "sq_conv_step"))
def test_conv(fn):
    cfg = lambda **kw: make(_lib.SqConvCfg, CONV, kw)  # noqa: E731
    assert conv(fn, None) == ARG
    for kw, st in ((dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(act=1), ARG), (dict(act=3), ARG), (dict(channels=0), ARG),
                   (dict(channels=(1 << 24) + 1), ARG), (dict(width=1), UNSUPPORTED), (dict(width=9), UNSUPPORTED), (dict(n_seq=-1), ARG),
                   (dict(n_tokens=-1), ARG), (dict(n_tokens=1 << 31), ARG), (dict(channels=1 << 24, n_tokens=1 << 20), ARG), (dict(d_seq_start=BASE + 2), ARG)):
        assert conv(fn, cfg(**kw)) == st, kw
        assert LIB().sq_last_error().decode()
    rows = {"sq_conv": ("x", "y"), "sq_conv_bwd": ("x", "dy", "dx"), "sq_conv_step": ("x", "y")}[fn]
    for n in rows:
        assert conv(fn, cfg(), **{n: None}) == ARG
        assert conv(fn, cfg(), **{n: R(None)}) == ARG
        assert conv(fn, cfg(), **{n: R(stride=255)}) == SHAPE
        assert conv(fn, cfg(), **{n: R(stride=1 << 41)}) == SHAPE
        assert conv(fn, cfg(), **{n: R(ptr=BASE + 1)}) == ARG
    assert conv(fn, cfg(), w=None) == ARG
    for n in {"sq_conv": ("w", "b"), "sq_conv_bwd": ("w", "b", "dw", "db"), "sq_conv_step": ("w", "b", "slots")}[fn]:
        assert conv(fn, cfg(), **{n: BASE + 2}) == ARG
    for n in {"sq_conv": ("s0", "s1"), "sq_conv_bwd": ("s0", "ds1", "ds0"), "sq_conv_step": ("window",)}[fn]:
        assert conv(fn, cfg(), **{n: BASE + 1}) == ARG
    if fn != "sq_conv_step":
        assert conv(fn, cfg(d_seq_start=None)) == ARG
    else:
        assert conv(fn, cfg(), window=None) == ARG and conv(fn, cfg(), n_slots=-1) == ARG and conv(fn, cfg(), n_slots=1 << 31) == ARG


def test_conv_workspace():
    cfg, n = make(_lib.SqConvCfg, CONV, {}), c_size_t(0)
    assert LIB().sq_conv_bytes(byref(cfg), byref(n)) == 0 and n.value == 2 * 5 * 256 * 4       # (40 >> 6) + 2 rows of (4 + 1) x 256 sums
    assert conv("sq_conv_bwd", cfg, nbytes=n.value - 1) == SHAPE
    assert conv("sq_conv_bwd", cfg, work=None) == ARG and conv("sq_conv_bwd", cfg, work=BASE + 128) == ARG
    assert LIB().sq_conv_bytes(byref(cfg), None) == ARG and LIB().sq_conv_bytes(None, byref(n)) == ARG
    assert sq.sq_conv_bytes(__import__("torch").bfloat16, 256, 4, 2, 40) == 2 * 5 * 256 * 4


# ---------------------------------------------------------------- selective scan

SSM = dict(dtype=1, channels=256, d_state=16, n_groups=2, softplus=1, n_seq=2, n_tokens=40, d_seq_start=BASE)


def ssm(fn, cfg, **kw):
    a = {n: R() for n in ("u", "dt", "z", "y", "dy", "du", "ddt", "dz")}
    a.update({n: R(stride=32) for n in ("b", "c", "db", "dc")})
    a.update(a=BASE, d=BASE, bias=BASE, s0=None, s1=None, ds1=None, ds0=None, da=BASE, dd=BASE, dbias=BASE, work=BASE, nbytes=1 << 40, slots=BASE, n_slots=50,
             state=BASE, ins=True, grads=True)
    a.update(kw)
    p = lambda n: ctypes.pointer(a[n]) if a[n] is not None else None  # noqa: E731
    ins = _lib.SqSsmIn(p("u"), p("dt"), p("b"), p("c"), p("z"), a["a"], a["d"], a["bias"])
    grads = _lib.SqSsmGrads(p("du"), p("ddt"), p("db"), p("dc"), p("dz"), a["da"], a["dd"], a["dbias"])
    i = byref(ins) if a["ins"] else None
    rest = {"sq_ssm_scan": (a["s0"], ptr(a["y"]), a["s1"], a["work"], a["nbytes"]),
            "sq_ssm_scan_bwd": (a["s0"], ptr(a["dy"]), a["ds1"], byref(grads) if a["grads"] else None, a["ds0"], a["work"], a["nbytes"]),
            "sq_ssm_step": (a["slots"], a["n_slots"], a["state"], ptr(a["y"]))}[fn]
    return getattr(LIB(), fn)(ptr(cfg), i, *rest, None)


@pytest.mark.parametrize("fn", ("sq_ssm_scan", "sq_ssm_scan_bwd", "sq_ssm_step"))
def test_ssm(fn):
    cfg = lambda **kw: make(_lib.SqSsmCfg, SSM, kw)  # noqa: E731
    assert ssm(fn, None) == ARG
    for kw, st in ((dict(dtype=3), ARG), (dict(channels=0), ARG), (dict(channels=(1 << 20) + 2), ARG), (dict(n_groups=3), ARG), (dict(n_groups=0), ARG),
                   (dict(d_state=24), UNSUPPORTED), (dict(d_state=4), UNSUPPORTED), (dict(d_state=256), UNSUPPORTED), (dict(softplus=2), ARG),
                   (dict(n_seq=-1), ARG), (dict(n_tokens=-1), ARG), (dict(n_tokens=1 << 31), ARG), (dict(channels=1 << 20, n_tokens=1 << 30), ARG),
                   (dict(d_seq_start=BASE + 2), ARG)):
        assert ssm(fn, cfg(**kw)) == st, kw
        assert LIB().sq_last_error().decode()
    assert ssm(fn, cfg(), ins=False) == ARG
    rows = ["u", "dt", "b", "c"] + {"sq_ssm_scan": ["y"], "sq_ssm_scan_bwd": ["dy", "du", "ddt", "db", "dc"], "sq_ssm_step": ["y"]}[fn]
    for n in rows:
        assert ssm(fn, cfg(), **{n: None}) == ARG, n
        assert ssm(fn, cfg(), **{n: R(None)}) == ARG, n
    for n in rows + ["z"] + (["dz"] if fn == "sq_ssm_scan_bwd" else []):
        assert ssm(fn, cfg(), **{n: R(stride=31)}) == SHAPE, n
        assert ssm(fn, cfg(), **{n: R(ptr=BASE + 1)}) == ARG, n
    assert ssm(fn, cfg(), a=None) == ARG and ssm(fn, cfg(), a=BASE + 4) == ARG
    for n in ("d", "bias"):
        assert ssm(fn, cfg(), **{n: BASE + 2}) == ARG
    for n in {"sq_ssm_scan": ("s0", "s1"), "sq_ssm_scan_bwd": ("s0", "ds1", "ds0"), "sq_ssm_step": ("state",)}[fn]:
        assert ssm(fn, cfg(), **{n: BASE + 4}) == ARG, n
    if fn == "sq_ssm_step":
        assert ssm(fn, cfg(), state=None) == ARG and ssm(fn, cfg(), n_slots=-1) == ARG and ssm(fn, cfg(), slots=BASE + 2) == ARG
        return
    assert ssm(fn, cfg(d_seq_start=None)) == ARG
    if fn == "sq_ssm_scan_bwd":
        assert ssm(fn, cfg(), grads=False) == ARG and ssm(fn, cfg(), z=None) == ARG              # dz without z
        for n in ("da", "dd", "dbias"):
            assert ssm(fn, cfg(), **{n: BASE + 2}) == ARG


@pytest.mark.parametrize("backward", (0, 1))
def test_ssm_workspace(backward):
    fn = "sq_ssm_scan_bwd" if backward else "sq_ssm_scan"
    cfg, n = make(_lib.SqSsmCfg, SSM, dict(n_tokens=4000)), c_size_t(0)
    assert LIB().sq_ssm_scan_bytes(byref(cfg), backward, byref(n)) == 0 and n.value > 0
    assert ssm(fn, cfg, nbytes=n.value - 1) == SHAPE
    assert ssm(fn, cfg, work=None, nbytes=n.value) == ARG and ssm(fn, cfg, work=BASE + 128, nbytes=n.value) == ARG
    assert LIB().sq_ssm_scan_bytes(byref(cfg), backward, None) == ARG
    assert sq.sq_ssm_scan_bytes(__import__("torch").bfloat16, 256, 16, 2, 2, 4000, backward=backward) == n.value


# ---------------------------------------------------------------- cache

CACHE = dict(dtype=1, format=0, d=256, group=64, n_rows=8, n_slots=20)


def cache(fn, cfg, x=R(), slots=BASE, codes=BASE, scales=BASE):
    args = (ptr(x), slots, codes, scales) if fn == "sq_cache_write" else (codes, scales, slots, ptr(x))
    return getattr(LIB(), fn)(ptr(cfg), *args, None)


@pytest.mark.parametrize("fn", ("sq_cache_write", "sq_cache_read"))
def test_cache(fn):
    cfg = lambda **kw: make(_lib.SqCacheCfg, CACHE, kw)  # noqa: E731
    assert cache(fn, None) == ARG
    for kw, st in ((dict(dtype=3), ARG), (dict(format=3), ARG), (dict(format=-1), ARG), (dict(group=0), UNSUPPORTED), (dict(group=1025, d=1025), UNSUPPORTED),
                   (dict(format=1, group=1), UNSUPPORTED), (dict(format=1, d=15, group=15), UNSUPPORTED), (dict(group=100), SHAPE), (dict(d=0), SHAPE),
                   (dict(n_rows=-1), ARG), (dict(n_slots=-1), ARG), (dict(n_slots=1 << 31), ARG), (dict(n_rows=1 << 31), SHAPE), (dict(n_rows=1 << 25), SHAPE)):
        assert cache(fn, cfg(**kw)) == st, kw
        assert LIB().sq_last_error().decode()
    assert cache(fn, cfg(), x=None) == ARG and cache(fn, cfg(), x=R(None)) == ARG
    assert cache(fn, cfg(), x=R(stride=255)) == SHAPE and cache(fn, cfg(), x=R(ptr=BASE + 1)) == ARG
    assert cache(fn, cfg(), codes=None) == ARG and cache(fn, cfg(), scales=None) == ARG
    assert cache(fn, cfg(), scales=BASE + 2) == ARG and cache(fn, cfg(), slots=BASE + 2) == ARG
    assert cache(fn, cfg(n_rows=0), x=None, codes=None, scales=None) == 0


def test_nothing_to_do():
    assert conv("sq_conv", make(_lib.SqConvCfg, CONV, dict(n_seq=0)), x=None, y=None, w=None) == 0
    assert conv("sq_conv_step", make(_lib.SqConvCfg, CONV, dict(n_tokens=0)), x=None, y=None, w=None, window=None) == 0
    assert conv("sq_conv_step", make(_lib.SqConvCfg, CONV, {}), n_slots=0, window=None) == 0           # every slot is outside
    assert ssm("sq_ssm_step", make(_lib.SqSsmCfg, SSM, {}), n_slots=0, state=None) == 0
    assert cache("sq_cache_write", make(_lib.SqCacheCfg, CACHE, dict(n_slots=0)), codes=None, scales=None) == 0
    assert ssm("sq_ssm_scan", make(_lib.SqSsmCfg, SSM, dict(n_seq=0)), u=None, y=None, a=None, work=None, nbytes=0) == 0
    assert ssm("sq_ssm_step", make(_lib.SqSsmCfg, SSM, dict(n_tokens=0)), u=None, y=None, a=None, state=None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    t, b = torch.zeros(4, 64), torch.zeros(4, 1, 16)
    for call in (lambda: sq.sq_conv(t, torch.zeros(64, 4), t), lambda: sq.sq_conv_bwd(t, torch.zeros(64, 4), t, t), lambda: sq.sq_conv_step(t, torch.zeros(64, 4), t, t),
                 lambda: sq.sq_ssm_scan(t, t, torch.zeros(64, 16), b, b, t), lambda: sq.sq_ssm_step(t, t, torch.zeros(64, 16), b, b, t, t),
                 lambda: sq.sq_cache_write(t, t, t), lambda: sq.sq_cache_read(t, t, t), lambda: sq.sq_conv_bytes(torch.float64, 64, 4, 1, 4),
                 lambda: sq.sq_ssm_scan_bytes(torch.int8, 64, 16, 1, 1, 4)):
        with pytest.raises(TypeError):
            call()
    assert [ctypes.sizeof(c) for c in (_lib.SqConvCfg, _lib.SqSsmCfg, _lib.SqCacheCfg, _lib.SqSsmIn)] == [40, 40, 32, 64]
