"""Calls of the convolution and the selective scan where their tiles, segments and alignments end, on the GPU against float64.

The tolerances are those of test_gpu_conv.py and test_gpu_ssm.py (derived there) unless a test derives its own.
"""
import pytest
import torch

import _mix_ref as ref
import quantized_delta_rule_02_amd as sq
import test_gpu_conv as conv
import test_gpu_ssm as ssm

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = {F32: "f32", BF16: "bf16", F16: "f16"}


@pytest.mark.parametrize("lead", (0, 3, 5))
@pytest.mark.parametrize("N", (16, 128))
def test_scan_gradients_of_many_short_sequences(N, lead, dev):
    """Tiles of 8 tokens and segments of 32 that begin anywhere in the packed rows, each with states of its own before it."""
    lens = [1, 9, 7, 8, 15, 16, 17, 0, 23, 25, 33, 31, 2, 41, 9, 0, 0, 65, 10, 11, 12, 13, 14] * 2
    ssm.check(20, N, 1, lens, F32, dev, lead=lead, behind=2)
    ssm.check(20, N, 1, lens, BF16, dev, lead=lead, seed=9)


def test_scan_gradients_stay_in_their_workspace(dev):
    """Exactly the bytes that the library asks for, fenced; what was there before does not matter."""
    C, N, lens = 40, 16, [9, 1, 17, 0, 8, 33, 40, 2, 16, 25] * 20
    T, n = sum(lens), len(lens)
    g, start = ssm.put(ref.ssm_inputs(C, N, 1, lens, 5, F32), dev), ref.starts(lens).to(dev)
    size = sq.sq_ssm_scan_bytes(F32, C, N, 1, n, T, backward=True)
    outs = []
    for fill in (0, 0x7f):
        buf = torch.full((size + 2 * 4096,), fill, dtype=torch.uint8, device=dev)
        o = {k: torch.empty_like(g[s]) for k, s in (("du", "u"), ("ddt", "dt"), ("da", "a"), ("db", "b"), ("dc", "c"), ("dz", "z"), ("dd", "d"),
                                                    ("ddt_bias", "dt_bias"), ("ds0", "s0"))}
        sq.sq_ssm_scan_bwd(g["u"], g["dt"], g["a"], g["b"], g["c"], g["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], d=g["d"], dt_bias=g["dt_bias"],
                           z=g["z"], dz=o["dz"], dd=o["dd"], ddt_bias=o["ddt_bias"], seq_start=start, s0=g["s0"], ds1=g["ds1"], ds0=o["ds0"],
                           workspace=buf[4096:4096 + size])
        torch.cuda.synchronize()
        assert bool((buf[:4096] == fill).all()) and bool((buf[4096 + size:] == fill).all())
        outs.append(o)
    for k in outs[0]:
        assert torch.equal(outs[0][k], outs[1][k]), k


@pytest.mark.parametrize("N", (8, 16, 32, 64, 128))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_scan_of_64_tokens_and_more_in_one_piece(N, dtype, dev):
    """Too short for segments, long enough for the larger tiles: two whole blocks of channels and a part of a third, in fours and in ones."""
    per = 1024 // N                                            # channels of a workgroup
    for C, lens in ((2 * per + 4, [100, 64, 91, 127, 66]), (2 * per + 3, [65, 63, 128, 1, 96, 70])):
        assert 64 * len(lens) <= sum(lens) < 128 * len(lens)
        assert sq.sq_ssm_scan_bytes(dtype, C, N, 1, len(lens), sum(lens)) == 0
        ssm.check(C, N, 1, lens, dtype, dev, grads=False, lead=2, behind=1)


@pytest.mark.parametrize("n_seq", (30, 44))
@pytest.mark.parametrize("N,C", ((8, 1536), (16, 768), (128, 96)))
def test_scan_of_many_long_sequences(N, C, n_seq, dev):
    """Enough workgroups to go without segments; 360 of them are staged 64 tokens at a time where their LDS allows it, 528 are not (nor with 8 states)."""
    assert n_seq * (C * N // 1024) in (360, 528)
    lens = [70 + 37 * i % 130 for i in range(n_seq)]
    assert sum(lens) >= 128 * n_seq and sq.sq_ssm_scan_bytes(BF16, C, N, 1, n_seq, sum(lens)) == 0
    ssm.check(C, N, 1, lens, BF16, dev, grads=False)


# A gate's 1 / (1 + e^-z), |z| <= 64, in units of 2^-24 of its value: the hardware's 2^x and reciprocal 2 each, the exponent's remainder 3 (64 times the
# 2^-28.4 by which float32's ln 2 is off, and its sum), two roundings.  So z s(z) is off by at most 11 units of itself; s (1 + z (1 - s)), with
# products, sums and 1 - s (10 units of one), by at most 24 of s (1 + |z|).  One token, so no sums over tokens.
UNIT = 2.0 ** -24


@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_conv_gradients_in_float32_carry_float32_gates(dtype, dev):
    """dweight and dbias are float32 for rows of 16 bits too: the gate's exponent is not rounded to less."""
    C = 4096
    p = torch.linspace(-64.0, 64.0, C)                          # exactly the sum before the activation
    one = torch.ones(1, C, dtype=dtype, device=dev)
    weight, bias = torch.zeros(C, 2, device=dev), p.to(dev)
    dw, db, dx = torch.empty_like(weight), torch.empty_like(bias), torch.empty_like(one)
    sq.sq_conv_bwd(1.5 * one, weight, one, dx, dweight=dw, bias=bias, dbias=db)
    z = p.double()
    s = z.sigmoid()
    want, size = s * (1 + z * (1 - s)), s * (1 + z.abs())
    assert bool(((db.double().cpu() - want).abs() <= 24 * UNIT * size).all())
    assert bool(((dw[:, 1].double().cpu() - 1.5 * want).abs() <= 25 * UNIT * 1.5 * size).all()) and not dw[:, 0].any()


@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_scan_gradients_in_float32_carry_float32_gates(dtype, dev):
    """The same of dd: dy z s(z) u."""
    C, N = 4096, 16
    z = torch.linspace(-64.0, 64.0, C)[None].to(dtype)
    g = ssm.put(dict(ref.ssm_inputs(C, N, 1, [1], 5, dtype), z=z), dev)
    one = torch.ones_like(g["u"])
    o = {k: torch.empty_like(g[s]) for k, s in (("du", "u"), ("ddt", "dt"), ("da", "a"), ("db", "b"), ("dc", "c"), ("dz", "z"), ("dd", "d"))}
    sq.sq_ssm_scan_bwd(g["u"], g["dt"], g["a"], g["b"], g["c"], one, o["du"], o["ddt"], o["da"], o["db"], o["dc"], d=g["d"], dt_bias=g["dt_bias"], z=g["z"],
                       dz=o["dz"], dd=o["dd"])
    want = (z.double() * z.double().sigmoid() * g["u"].double().cpu())[0]
    assert bool(((o["dd"].double().cpu() - want).abs() <= 12 * UNIT * want.abs()).all())          # 11 and the product with u


@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_gates_of_all_sizes_are_finite(dtype, dev):
    """Sums before the activation where its exponential is infinite, zero or next to either.  Below 2^-126 a sigmoid may be lost: 88 x 2^-126 of a product."""
    p = torch.tensor([float(s) * x for x in (0.0, 1.0, 20.0, 87.0, 88.0, 88.7, 88.8, 89.0, 100.0, 103.0, 104.0, 127.0, 128.0, 150.0, 200.0, 1e4, 1e30, 3e38)
                      for s in (1, -1)])
    C = p.numel()
    one = torch.ones(1, C, dtype=dtype, device=dev)
    weight, bias = torch.zeros(C, 2, device=dev), p.to(dev)
    y, dx, db = torch.empty_like(one), torch.empty_like(one), torch.empty_like(bias)
    sq.sq_conv(one, weight, y, bias=bias)
    sq.sq_conv_bwd(one, weight, one, dx, bias=bias, dbias=db)
    z, most = p.double(), torch.finfo(dtype).max
    want = z * z.sigmoid()
    fits = want.abs() <= most
    half = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == F16 else 88 * 2.0 ** -126
    assert bool(((y[0].double().cpu() - want).abs() <= (half + 12 * UNIT) * want.abs() + tiny)[fits].all())
    want = z.sigmoid() * (1 + z * (1 - z.sigmoid()))
    assert bool(((db.double().cpu() - want).abs() <= 24 * UNIT * z.sigmoid() * (1 + z.abs().clamp(max=20)) + 88 * 2.0 ** -126).all())
    step, state = torch.zeros(1, 1, C, dtype=dtype, device=dev), torch.empty_like(y)
    sq.sq_conv_step(one, weight, step, state, bias=bias)
    assert torch.equal(state, y)


@pytest.mark.parametrize("C", (2, 4, 6, 12, 258, 2052, 4100))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_conv_channels_that_are_no_multiple_of_16_bytes(C, dtype, dev):
    conv.check(C, 4, [3, 40, 0, 1], dtype, dev)


@pytest.mark.parametrize("pad,shift", ((4, 0), (4, 4), (2, 0), (2, 2), (6, 4), (10, 2), (1, 0)))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_conv_rows_of_wider_arrays_at_4_and_8_bytes(pad, shift, dtype, dev):
    conv.check(52, 4, [5, 37], dtype, dev, pad=pad, shift=shift)


@pytest.mark.parametrize("shift", (1, 2, 4))
def test_conv_states_that_are_aligned_less_than_the_rows(shift, dev):
    C, W, lens = 16, 4, [20, 2]
    x = ref.conv_inputs(C, W, lens, 3, BF16)
    g, start = {k: v.to(dev) for k, v in x.items()}, ref.starts(lens).to(dev)

    def moved(t):
        flat = torch.full((t.numel() + 2 * 8,), 7.0, dtype=t.dtype, device=dev)
        flat[shift:shift + t.numel()] = t.reshape(-1)
        return flat[shift:shift + t.numel()].view(t.shape), flat

    def run(place):
        s0, s1, ds1, ds0 = (place(g[k])[0] for k in ("s0", "s0", "ds1", "ds1"))
        y, dx, dw = torch.empty_like(g["x"]), torch.empty_like(g["x"]), torch.empty_like(g["weight"])
        sq.sq_conv(g["x"], g["weight"], y, bias=g["bias"], seq_start=start, s0=s0, s1=s1)
        sq.sq_conv_bwd(g["x"], g["weight"], g["dy"], dx, dweight=dw, bias=g["bias"], seq_start=start, s0=s0, ds1=ds1, ds0=ds0)
        window, step = place(g["s0"])[0], torch.empty_like(g["x"][:2])
        sq.sq_conv_step(g["x"][:2], g["weight"], window, step, bias=g["bias"])
        return [t.clone() for t in (y, s1, dx, dw, ds0, window, step)]

    for a, b in zip(run(lambda t: (t.clone(), None)), run(moved)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("C", (1, 2, 6, 257, 514, 4098))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_conv_step_of_few_and_odd_channels(C, dtype, dev):
    conv.test_step(3, C, dtype, dev)
    conv.test_step(8, C, dtype, dev)


@pytest.mark.parametrize("C,N,lens", ((8, 16, [175]), (8, 16, [173]), (40, 128, [190, 178, 0, 400]), (40, 128, [190, 178, 0, 353]), (24, 64, [130] * 9 + [900])), ids=str)
def test_scan_at_the_border_of_segments(C, N, lens, dev):
    """Mean lengths on both sides of where whole sequences go in one piece, and a long one among short ones."""
    g = len(lens) * -(-C // (1024 // N))                       # workgroups of whole sequences
    cut = sum(lens) // len(lens) * (288 - g) >= 50000
    assert (sq.sq_ssm_scan_bytes(F32, C, N, 1, len(lens), sum(lens)) > 0) == cut
    ssm.check(C, N, 1, lens, F32, dev, grads=False)
    ssm.check(C, N, 1, lens, BF16, dev, grads=False, seed=4)


@pytest.mark.parametrize("lens", ([300, 290], [20, 90]), ids=str)
def test_scan_with_decays_above_one(lens, dev, monkeypatch):
    """Rates of both signs up to 0.2.  A channel's steps average at most 0.37, so an exponent grows by 0.074 a token, and a step's error of 32 units
    makes 2.4 units of the whole a token: the tolerance has 6."""
    made = ref.ssm_inputs

    def inputs(C, N, *args, **kw):
        return dict(made(C, N, *args, **kw), a=(0.2 * (ref.rnd(C, N, seed=77)).clamp(-1, 1)).float())

    monkeypatch.setattr(ref, "ssm_inputs", inputs)
    ssm.check(24, 16, 1, lens, F32, dev)
    ssm.check(24, 64, 2, lens, BF16, dev, seed=3)
