"""What the scan and the norms refuse, on the CPU: every check comes before any device call, so the addresses here are
never followed."""
import ctypes
from ctypes import byref, c_size_t

import pytest

import quantized_delta_rule_02_amd as sq
from quantized_delta_rule_02_amd import _lib

ARG, SHAPE, UNSUPPORTED = -1, -2, -3
BASE = 1 << 20           # an aligned address that nothing reads


def R(ptr=BASE, stride=512):
    return _lib.SqRows(ptr, stride)


def scan_cfg(**kw):
    d = dict(form=0, dtype=1, n_heads=4, n_heads_k=2, d_k=128, d_v=128, n_seq=2, n_tokens=40, d_seq_start=BASE)
    d.update(kw)
    return _lib.SqScanCfg(*[d[n] for n, _ in _lib.SqScanCfg._fields_])


def scan(cfg, backward=False, nbytes=1 << 40, work=BASE, **kw):
    a = dict(q=R(stride=256), k=R(stride=256), v=R(), gate=BASE, beta=BASE, s0=None, y=R(), s1=None, dy=R(), ds1=None,
             dq=R(stride=256), dk=R(stride=256), dv=R(), dgate=BASE, dbeta=BASE, ds0=None)
    a.update(kw)
    names = (["q", "k", "v", "gate", "beta", "s0", "y", "s1"] if not backward else
             ["q", "k", "v", "gate", "beta", "s0", "dy", "ds1", "dq", "dk", "dv", "dgate", "dbeta", "ds0"])
    args = [byref(a[n]) if isinstance(a[n], _lib.SqRows) else a[n] for n in names]
    fn = _lib.load().sq_delta_scan_bwd if backward else _lib.load().sq_delta_scan
    return fn(byref(cfg) if cfg is not None else None, *args, work, nbytes, None)


BAD_CFG = [(dict(form=2), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(n_heads=0), ARG), (dict(n_heads_k=3), ARG),
           (dict(n_heads_k=0), ARG), (dict(n_heads=4097, n_heads_k=4097), ARG), (dict(d_k=96), UNSUPPORTED),
           (dict(d_k=64, d_v=128), UNSUPPORTED), (dict(n_seq=-1), ARG), (dict(n_tokens=-1), ARG), (dict(n_tokens=1 << 31), ARG),
           (dict(n_heads=4096, n_heads_k=4096, n_seq=1 << 20), ARG), (dict(d_seq_start=None), ARG),
           (dict(n_heads=64, n_heads_k=64, n_seq=90000, n_tokens=0), ARG)]


@pytest.mark.parametrize("kw,st", BAD_CFG, ids=[str(b[0]) for b in BAD_CFG])
@pytest.mark.parametrize("backward", (False, True))
def test_scan_configurations(kw, st, backward):
    assert scan(scan_cfg(**kw), backward) == st
    assert _lib.load().sq_last_error().decode()


def test_scan_arrays():
    c = scan_cfg()
    assert scan(None) == ARG
    for bwd, names in ((False, ("q", "k", "v", "y")), (True, ("q", "k", "v", "dy", "dq", "dk", "dv"))):
        for n in names:
            assert scan(c, bwd, **{n: None}) == ARG
            assert scan(c, bwd, **{n: R(None)}) == ARG
            assert scan(c, bwd, **{n: R(stride=255)}) == SHAPE
            assert scan(c, bwd, **{n: R(ptr=BASE + 1, stride=512)}) == ARG
        for n in ("gate", "beta") + (("dgate", "dbeta") if bwd else ()):
            assert scan(c, bwd, **{n: None}) == ARG
            assert scan(c, bwd, **{n: BASE + 2}) == ARG
    for n in ("q", "k"):
        assert scan(c, **{n: R(ptr=BASE + 8, stride=256)}) == ARG       # read 16 bytes at a time
        assert scan(c, **{n: R(stride=260)}) == ARG
    assert scan(c, True, dy=R(stride=516)) == ARG
    for bwd, names in ((False, ("s0", "s1")), (True, ("s0", "ds1", "ds0"))):
        for n in names:
            assert scan(c, bwd, **{n: BASE + 2}) == ARG
    assert scan(scan_cfg(form=1), gate=BASE + 4) == ARG


@pytest.mark.parametrize("backward", (False, True))
def test_scan_workspace(backward):
    c = scan_cfg()
    n = c_size_t(0)
    assert _lib.load().sq_delta_scan_bytes(byref(c), int(backward), byref(n)) == 0 and n.value > 0
    assert scan(c, backward, nbytes=n.value - 1) == SHAPE
    assert scan(c, backward, work=None, nbytes=n.value) == ARG
    assert scan(c, backward, work=BASE + 128, nbytes=n.value) == ARG
    assert _lib.load().sq_delta_scan_bytes(byref(c), 0, None) == ARG
    assert sq.sq_delta_scan_bytes(0, __import__("torch").bfloat16, 4, 2, 128, 128, 2, 40, backward=backward) == n.value


def test_nothing_to_do():
    assert scan(scan_cfg(n_seq=0), q=None, k=None, v=None, y=None, work=None, nbytes=0) == 0
    assert norm("sq_norm_in", norm_cfg(n_outer=0), x=None, n=None) == 0
    assert norm("sq_norm_out", norm_cfg(n_outer=0), y=None, o=None) == 0


def norm_cfg(**kw):
    d = dict(dtype=1, dtype_out=0, kind=0, act=0, n_outer=6, n_inner=2, d=64, eps=1e-6, res_scale=1.0, out_scale=1.0)
    d.update(kw)
    return _lib.SqNormCfg(*[d[n] for n, _ in _lib.SqNormCfg._fields_])


NORM_ARGS = {"sq_norm_in": ["x", "r", "weight", "chan", "h", "n"],
             "sq_norm_in_bwd": ["h", "dn", "dh", "r", "weight", "chan", "dx", "dr", "dw", "dc", "work", "nbytes"],
             "sq_norm_out": ["y", "z", "x", "weight", "chan", "o"],
             "sq_norm_out_bwd": ["y", "z", "do", "weight", "chan", "dy", "dz", "dw", "dc", "work", "nbytes"]}
NEEDED = {"sq_norm_in": ["x", "n"], "sq_norm_in_bwd": ["h", "dn", "dx"], "sq_norm_out": ["y", "o"],
          "sq_norm_out_bwd": ["y", "do", "dy"]}
ARRAYS = {"x", "r", "h", "n", "dn", "dh", "dx", "dr", "y", "z", "o", "do", "dy", "dz"}


def norm(fn, cfg, **kw):
    a = {n: R(stride=128) for n in ARRAYS}
    a.update(weight=BASE, chan=BASE, dw=BASE, dc=BASE, work=BASE, nbytes=1 << 40)
    a.update(kw)
    args = [byref(a[n]) if isinstance(a[n], _lib.SqRows) else a[n] for n in NORM_ARGS[fn]]
    return getattr(_lib.load(), fn)(byref(cfg) if cfg is not None else None, *args, None)


@pytest.mark.parametrize("fn", list(NORM_ARGS))
def test_norm_refusals(fn):
    assert norm(fn, None) == ARG
    for kw, st in ((dict(dtype=5), ARG), (dict(dtype_out=-1), ARG), (dict(kind=2), ARG), (dict(d=0), UNSUPPORTED),
                   (dict(d=16385), UNSUPPORTED), (dict(n_outer=-1), SHAPE), (dict(n_inner=0), SHAPE),
                   (dict(n_outer=1 << 31), SHAPE), (dict(n_outer=1 << 30, n_inner=2), SHAPE),
                   (dict(n_inner=1 << 20, d=16384), SHAPE), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
                   (dict(eps=float("inf")), ARG), (dict(res_scale=float("inf")), ARG), (dict(out_scale=float("nan")), ARG)):
        assert norm(fn, norm_cfg(**kw)) == st, kw
    for n in NEEDED[fn]:
        assert norm(fn, norm_cfg(), **{n: None}) == ARG
    for n in set(NORM_ARGS[fn]) & ARRAYS:
        assert norm(fn, norm_cfg(), **{n: R(stride=127)}) == SHAPE, n
        assert norm(fn, norm_cfg(), **{n: R(ptr=BASE + 1, stride=128)}) == ARG, n
    assert norm(fn, norm_cfg(), weight=BASE + 2) == ARG
    assert norm(fn, norm_cfg(), chan=BASE + 2) == ARG
    if fn.endswith("bwd"):
        assert norm(fn, norm_cfg(), nbytes=100) == SHAPE
        assert norm(fn, norm_cfg(), work=None) == ARG
        assert norm(fn, norm_cfg(), work=BASE + 64) == ARG
    if fn.startswith("sq_norm_out"):
        assert norm(fn, norm_cfg(act=2)) == ARG
    if fn == "sq_norm_in_bwd":
        assert norm(fn, norm_cfg(), r=None) == ARG            # dchan_scale needs r
    if fn == "sq_norm_out_bwd":
        assert norm(fn, norm_cfg(), z=None) == ARG            # dz without z


def test_norm_bytes():
    n = c_size_t(0)
    lib = _lib.load()
    assert lib.sq_norm_bytes(0, 128, byref(n)) == 0 and n.value == 0
    assert lib.sq_norm_bytes(1, 128, byref(n)) == 0 and n.value == 2 * 128 * 4
    for rows, d in ((-1, 128), (1 << 31, 128), (10, 0), (10, 16385)):
        assert lib.sq_norm_bytes(rows, d, byref(n)) == ARG
    assert lib.sq_norm_bytes(1, 128, None) == ARG
    assert sq.sq_norm_bytes(1 << 20, 16384) == 2 * 256 * 16384 * 4


def test_chunk_slots_are_distinct():
    """Chunk c of sequence b has the slot (start_b >> 5) + b + c: distinct, in order, and below (n_tokens >> 5) + n_seq."""
    import random
    r = random.Random(4)
    for _ in range(300):
        lens = [r.choice([0, 0, 1, 31, 32, 33, r.randrange(200)]) for _ in range(r.randrange(1, 12))]
        lead = r.randrange(70)
        at, seen = lead, []
        for b, n in enumerate(lens):
            seen += [(at >> 5) + b + c for c in range((n + 31) // 32)]
            at += n
        assert seen == sorted(set(seen)) and (not seen or seen[-1] < ((at + r.randrange(3)) >> 5) + len(lens))


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 2, 64)
    with pytest.raises(TypeError):
        sq.sq_delta_scan(0, t, t, t, t, t, t)
    with pytest.raises(TypeError):
        sq.sq_norm_in(t, t)
    with pytest.raises(TypeError):
        sq.sq_delta_scan_bytes(0, torch.float64, 2, 2, 64, 64, 1, 4)
    assert ctypes.sizeof(_lib.SqScanCfg) == 48 and ctypes.sizeof(_lib.SqNormCfg) == 48
