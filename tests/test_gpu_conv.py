"""The causal convolution, its gradients and its single-token form on the GPU against float64.

Tolerance.  p is at most nine float32 products and sums: 10 roundings of 2^-24 of the terms' magnitudes.  The activation carries an
exponential, a reciprocal and products of 2^-23 each (16 bits: an exponent's rounding, up to 2^-17 of a value at an exponent of
88), its derivative twice that.  2^-19 of the magnitudes covers them in float32, 2^-16 in 16 bits.  Sums over n tokens add in runs of 64 and
then run by run: (64 + n / 64 / 16 + 16 + 10) roundings, below 2^-16 of their magnitudes.  An output in t adds half a step of t.
"""
import pytest
import torch

import _mix_ref as ref
import quantized_delta_rule_02_amd as sq

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = {F32: "f32", BF16: "bf16", F16: "f16"}


def near(got, want, size, what, tol=None):
    t = got.dtype
    tol = tol or (2.0 ** -19 if t == F32 else 2.0 ** -16)
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    half = 0.0 if t == F32 else torch.finfo(t).eps / 2
    tiny = 2.0 ** -25 if t == F16 else 0.0
    off = (got - want).abs() - half * want.abs() - tiny - tol * size
    assert not want.numel() or off.max() <= 0, f"{what}: off by {(got - want).abs().max():.3e}"


def put(x, dev, pad=0, shift=0):
    """On the GPU as rows of a wider array: `pad` elements more a row, starting `shift` elements in."""
    if not pad and not shift:
        return x.to(dev)
    wide = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device=dev)
    wide[:, shift:shift + x.shape[1]] = x.to(dev)
    return wide[:, shift:shift + x.shape[1]]


def check(C, W, lens, dtype, dev, silu=True, s0=True, bias=True, lead=0, behind=0, pad=0, shift=0, ds1=True, seed=1):
    x = ref.conv_inputs(C, W, lens, seed, dtype, extra=lead + behind)
    act = sq.SQ_ACT_SILU if silu else sq.SQ_ACT_NONE
    g = {k: (put(v, dev, pad, shift) if k in ("x", "dy") else v.to(dev)) for k, v in x.items()}
    start = ref.starts(lens, lead).to(dev)
    kw = dict(lead=lead, silu=silu, s0=s0, bias=bias)
    common = dict(bias=g["bias"] if bias else None, act=act, seq_start=start, s0=g["s0"] if s0 else None)
    want, size = ref.conv_ref(x, lens, **kw), ref.conv_ref(x, lens, size=True, **kw)
    y, s1 = put(torch.full_like(x["x"], 3.0), dev, pad, shift), torch.empty_like(g["s0"])
    sq.sq_conv(g["x"], g["weight"], y, s1=s1, **common)
    inside = slice(lead, lead + sum(lens))
    near(y[inside], want["y"][inside], size["y"][inside], "y")
    assert torch.equal(s1.double().cpu(), want["s1"])
    assert bool((y[:lead] == 3).all()) and bool((y[lead + sum(lens):] == 3).all())
    if pad:                                             # nothing beside the rows was written
        wide = y.as_strided((x["x"].shape[0], C + pad), (C + pad, 1), 0)
        assert bool((wide[:, :shift] == 7).all()) and bool((wide[:, shift + C:] == 7).all())
    # in place: the states' own array
    both = g["s0"].clone()
    y2 = torch.empty_like(y)
    sq.sq_conv(g["x"], g["weight"], y2, s1=both, **dict(common, s0=both if s0 else None))
    assert torch.equal(both, s1) and torch.equal(y2[inside], y[inside])
    # gradients
    want, size = (ref.conv_ref(x, lens, grads=True, ds1=ds1, size=z, **kw) for z in (False, True))
    dx, ds0 = put(torch.full_like(x["x"], 3.0), dev, pad, shift), torch.empty_like(g["s0"])
    dw, db = torch.empty_like(g["weight"]), torch.empty_like(g["bias"])
    sq.sq_conv_bwd(g["x"], g["weight"], g["dy"], dx, dweight=dw, dbias=db, ds1=g["ds1"] if ds1 else None, ds0=ds0, **common)
    near(dx[inside], want["dx"][inside], size["dx"][inside], "dx")
    near(ds0, want["ds0"], size["ds0"], "ds0")
    near(dw, want["dweight"], size["dweight"], "dweight", 2.0 ** -16)
    near(db, want["dbias"], size["dbias"], "dbias", 2.0 ** -16)
    assert bool((dx[:lead] == 3).all()) and bool((dx[lead + sum(lens):] == 3).all())
    dx2 = torch.empty_like(dx)
    sq.sq_conv_bwd(g["x"], g["weight"], g["dy"], dx2, ds1=g["ds1"] if ds1 else None, **common)       # nothing but dx wanted
    assert torch.equal(dx2[inside], dx[inside])


@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_widths_and_types(W, dtype, dev):
    check(64, W, [1, 0, 2, 70, 5, 33], dtype, dev)


@pytest.mark.parametrize("C", (1, 3, 8, 20, 257, 2056, 4100))
@pytest.mark.parametrize("dtype", (F32, BF16), ids=NAMES.get)
def test_channels(C, dtype, dev):
    check(C, 4, [3, 40, 1], dtype, dev)


@pytest.mark.parametrize("lens", ([1], [0], [0, 0, 0], [31], [32], [33], [64], [65], [3], [128, 129, 127], [1] * 130, [200, 0, 0, 1, 2, 3, 4]),
                         ids=lambda v: "-".join(map(str, v[:8])))
def test_lengths(lens, dev):
    check(24, 4, lens, BF16, dev)
    check(24, 8, lens, F32, dev, seed=5)


def test_no_activation_no_bias_no_states(dev):
    for dtype in (F32, F16):
        check(40, 4, [9, 70, 2], dtype, dev, silu=False)
        check(40, 3, [9, 70, 2], dtype, dev, bias=False, s0=False, ds1=False)


@pytest.mark.parametrize("pad,shift", ((8, 0), (16, 8), (3, 0), (5, 2), (8, 1)))
def test_rows_of_wider_arrays(pad, shift, dev):
    check(48, 4, [5, 37], BF16, dev, pad=pad, shift=shift)
    check(48, 4, [5, 37], F32, dev, pad=pad, shift=shift)


def test_tokens_outside_the_sequences(dev):
    check(16, 4, [5, 0, 37], BF16, dev, lead=9, behind=6)
    check(16, 4, [0, 0], F32, dev, lead=70, behind=100)


def test_one_sequence_without_offsets(dev):
    x = ref.conv_inputs(32, 4, [77], 3, F32)
    g = {k: v.to(dev) for k, v in x.items()}
    y = torch.empty_like(g["x"])
    sq.sq_conv(g["x"], g["weight"], y, bias=g["bias"], s0=g["s0"])
    near(y, ref.conv_ref(x, [77])["y"], ref.conv_ref(x, [77], size=True)["y"], "y")


@pytest.mark.parametrize("W", (2, 4, 8))
@pytest.mark.parametrize("C", (8, 19, 2064))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_step(W, C, dtype, dev):
    batch, S = 37, 50
    x = ref.conv_inputs(C, W, [1] * batch, 11, dtype)
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(2))[:batch].to(torch.int32)
    slots[5], slots[20] = -1, S                                         # skipped
    live = [i for i in range(batch) if 0 <= slots[i] < S]
    pool = ref.rnd(S, W - 1, C, seed=8).to(dtype)
    pool[slots[live].long()] = x["s0"][live]
    g, window = {k: v.to(dev) for k, v in x.items()}, pool.to(dev)
    y = torch.full((batch, C), 3.0, dtype=dtype, device=dev)
    sq.sq_conv_step(g["x"], g["weight"], window, y, slots=slots.to(dev), bias=g["bias"])
    want, size = ref.conv_ref(x, [1] * batch), ref.conv_ref(x, [1] * batch, size=True)
    near(y[live], want["y"][live], size["y"][live], "y")
    assert bool((y[5] == 3).all()) and bool((y[20] == 3).all())
    after = pool.clone()
    after[slots[live].long()] = want["s1"][live].to(dtype)
    assert torch.equal(window.cpu(), after)
    # x's own array, no slot list
    w2, xy = x["s0"].to(dev), g["x"].clone()
    sq.sq_conv_step(xy, g["weight"], w2, xy, bias=g["bias"])
    near(xy, want["y"], size["y"], "y")
    assert torch.equal(w2.double().cpu(), want["s1"])


def test_tokens_one_by_one_are_the_sequence(dev):
    """A prompt, then its next tokens by single steps: the same as the whole sequence at once, bit for bit in float32."""
    C, W, n, m = 72, 4, 41, 6
    x = ref.conv_inputs(C, W, [n + m], 13, F32)
    g = {k: v.to(dev) for k, v in x.items()}
    whole, y = torch.empty_like(g["x"]), torch.empty_like(g["x"])
    sq.sq_conv(g["x"], g["weight"], whole, bias=g["bias"], s0=g["s0"])
    window = g["s0"].clone()
    sq.sq_conv(g["x"][:n], g["weight"], y[:n], bias=g["bias"], s0=window, s1=window)
    for t in range(n, n + m):
        sq.sq_conv_step(g["x"][t:t + 1], g["weight"], window, y[t:t + 1], bias=g["bias"])
    assert torch.equal(y, whole)


def test_values_that_are_not_finite_stay_in_their_channel_and_reach(dev):
    C, W, lens = 40, 4, [50, 30]
    x = ref.conv_inputs(C, W, lens, 17, F32)
    g = {k: v.to(dev) for k, v in x.items()}
    start, run = ref.starts(lens).to(dev), lambda z: (torch.empty_like(z), torch.empty_like(g["s0"]))  # noqa: E731
    clean, bad = run(g["x"]), run(g["x"])
    z = g["x"].clone()
    z[20, 3], z[49, 5], z[60, 7] = float("nan"), float("inf"), -float("inf")
    for src, (y, s1) in ((g["x"], clean), (z, bad)):
        sq.sq_conv(src, g["weight"], y, bias=g["bias"], seq_start=start, s0=g["s0"], s1=s1)
    same = torch.ones(80, C, dtype=torch.bool, device=dev)
    same[20:24, 3] = same[49:50, 5] = same[60:64, 7] = False
    assert torch.equal(clean[0][same], bad[0][same]) and bool((~torch.isfinite(bad[0])[20:24, 3]).all())
    assert float(bad[1][0, 2, 5]) == float("inf")


def test_graphs_streams_and_calls_at_once(dev):
    """Two captured calls with workspaces of their own, replayed with other lengths and inputs; another stream; the same bits."""
    C, W = 136, 4
    x = [ref.conv_inputs(C, W, [60, 40], 21 + i, BF16) for i in range(2)]
    g = [{k: v.to(dev) for k, v in z.items()} for z in x]
    start = [ref.starts([60, 40]).to(dev) for _ in range(2)]
    out = [{k: torch.empty_like(z[s]) for k, s in (("y", "x"), ("dx", "x"), ("s1", "s0"), ("ds0", "s0"), ("dw", "weight"), ("db", "bias"))} for z in g]
    work = [torch.empty(sq.sq_conv_bytes(BF16, C, W, 2, 100), dtype=torch.uint8, device=dev) for _ in range(2)]

    def call(i, o, w, stream=None):
        z = g[i]
        sq.sq_conv(z["x"], z["weight"], o["y"], bias=z["bias"], seq_start=start[i], s0=z["s0"], s1=o["s1"], stream=stream)
        sq.sq_conv_bwd(z["x"], z["weight"], z["dy"], o["dx"], dweight=o["dw"], dbias=o["db"], bias=z["bias"], seq_start=start[i], s0=z["s0"],
                       ds1=z["ds1"], ds0=o["ds0"], workspace=w, stream=stream)

    for i in range(2):
        call(i, out[i], work[i])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(i, out[i], work[i])
        graphs.append(graph)
    side = torch.cuda.Stream()
    for lens in ([60, 40], [1, 99], [100, 0], [3, 2]):
        for s in start:
            s.copy_(ref.starts(lens))
        torch.cuda.synchronize()
        eager = [{k: torch.zeros_like(v) for k, v in o.items()} for o in out]
        for i in range(2):
            for v in out[i].values():
                v.zero_()
            call(i, eager[i], torch.empty_like(work[i]))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for k in out[i]:
                assert torch.equal(out[i][k], eager[i][k]), (lens, k)
        other = {k: torch.zeros_like(v) for k, v in out[0].items()}
        torch.cuda.synchronize()
        call(0, other, None, stream=side)
        side.synchronize()
        for k in other:
            assert torch.equal(other[k], eager[0][k]), k


def test_thousands_of_sequences(dev):
    """More sequences than two rounds of the search for a run's sequence cover (64 x 64)."""
    check(8, 4, [(i * 5) % 4 for i in range(5000)], F32, dev)


def test_offsets_that_break_the_rules_touch_nothing_else(dev):
    C, W, T, n = 40, 4, 100, 4
    x = ref.conv_inputs(C, W, [25] * n, 71, BF16)
    g = {k: v.to(dev) for k, v in x.items()}

    def fenced(shape, dtype):
        size = 1
        for s in shape:
            size *= s
        buf = torch.full((size + 2 * 4096,), 3.0, dtype=dtype, device=dev)
        return buf, buf[4096:4096 + size].view(shape)

    for at in ([0, 60, 20, 90, 100], [-50, 10, 20, 30, 4000], [100, 80, 60, 40, 20], [2 ** 31 - 1, -2 ** 31, 5, 2 ** 30, -7]):
        start = torch.tensor(at, dtype=torch.int32, device=dev)
        outs = {k: fenced(s, d) for k, s, d in (("y", (T, C), BF16), ("s1", (n, W - 1, C), BF16), ("dx", (T, C), BF16), ("ds0", (n, W - 1, C), BF16),
                                                ("dw", (C, W), F32), ("db", (C,), F32))}
        nbytes = sq.sq_conv_bytes(BF16, C, W, n, T)
        buf = torch.full((nbytes + 2 * 4096,), 7, dtype=torch.uint8, device=dev)
        v = {k: o[1] for k, o in outs.items()}
        sq.sq_conv(g["x"], g["weight"], v["y"], bias=g["bias"], seq_start=start, s0=g["s0"], s1=v["s1"])
        sq.sq_conv_bwd(g["x"], g["weight"], g["dy"], v["dx"], dweight=v["dw"], dbias=v["db"], bias=g["bias"], seq_start=start, s0=g["s0"], ds1=g["ds1"],
                       ds0=v["ds0"], workspace=buf[4096:4096 + nbytes])
        torch.cuda.synchronize()
        for k, (b, _) in outs.items():
            assert bool((b[:4096] == 3).all()) and bool((b[-4096:] == 3).all()), (at, k)
        assert bool((buf[:4096] == 7).all()) and bool((buf[4096 + nbytes:] == 7).all()), at


def test_no_sequences_and_no_tokens(dev):
    C, W = 24, 4
    w, b = torch.randn(C, W, device=dev), torch.randn(C, device=dev)
    x = torch.zeros(10, C, device=dev)
    y, dx = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
    none = torch.zeros(1, dtype=torch.int32, device=dev)
    sq.sq_conv(x, w, y, seq_start=none)
    dw, db = torch.full_like(w, 3.0), torch.full_like(b, 3.0)
    sq.sq_conv_bwd(x, w, x, dx, dweight=dw, dbias=db, seq_start=none)
    assert bool((y == 3).all()) and bool((dx == 3).all()) and not dw.any() and not db.any()
    e = torch.zeros(0, C, device=dev)
    s0 = torch.randn(2, W - 1, C, device=dev)
    s1, ds0 = torch.empty_like(s0), torch.empty_like(s0)
    start = torch.zeros(3, dtype=torch.int32, device=dev)
    sq.sq_conv(e, w, e, seq_start=start, s0=s0, s1=s1)
    sq.sq_conv_bwd(e, w, e, e, dweight=dw, dbias=db, seq_start=start, s0=s0, ds1=s1, ds0=ds0)
    assert torch.equal(s1, s0) and torch.equal(ds0, s0) and not dw.any() and not db.any()
    sq.sq_conv_step(e, w, s0, e)


def test_beyond_32_bit_offsets(dev):
    """Rows 2^31 elements and more from the array's start, and a window pool of that size."""
    C, W, T, stride = 64, 4, 6, 1 << 29
    base = torch.zeros((T - 1) * stride + C, dtype=BF16, device=dev)
    x = ref.conv_inputs(C, W, [T], 31, BF16)
    rows = base.as_strided((T, C), (stride, 1))
    rows[:] = x["x"].to(dev)
    y = torch.empty(T, C, dtype=BF16, device=dev)
    sq.sq_conv(rows, x["weight"].to(dev), y, bias=x["bias"].to(dev), s0=x["s0"].to(dev))
    near(y, ref.conv_ref(x, [T])["y"], ref.conv_ref(x, [T], size=True)["y"], "y")
    del base, rows
    S = (1 << 32) // (3 * 1024) + 5                                      # slots of 3 x 1024 elements: above 2^32 in all
    pool = torch.zeros(S, W - 1, 1024, dtype=BF16, device=dev)
    z = ref.conv_inputs(1024, W, [1, 1], 33, BF16)
    slots = torch.tensor([S - 1, 0], dtype=torch.int32, device=dev)
    pool[slots.long()] = z["s0"].to(dev)
    y = torch.empty(2, 1024, dtype=BF16, device=dev)
    sq.sq_conv_step(z["x"].to(dev), z["weight"].to(dev), pool, y, slots=slots, bias=z["bias"].to(dev))
    near(y, ref.conv_ref(z, [1, 1])["y"], ref.conv_ref(z, [1, 1], size=True)["y"], "y")
    assert torch.equal(pool[slots.long()].double().cpu(), ref.conv_ref(z, [1, 1])["s1"])
