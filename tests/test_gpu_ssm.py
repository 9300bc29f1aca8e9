"""The selective scan, its gradients and its single-token form on the GPU against float64.

Tolerance.  Every token multiplies a state by one decay (an exponential and its argument's roundings: 2^-22) and adds a product (two
roundings of 2^-24), so after L tokens a state is off by at most (6 L + 32) 2^-24 of its terms' magnitudes, the 32 for the step
itself (softplus: an exponential, a reciprocal and ten products).  A step's relative error e = 32 2^-24 makes a decay exp(-v) of all
tokens between off by e v exp(-v), and v exp(-v) <= (2 / 2.718) exp(-v / 2): 24 2^-24 of the terms' magnitudes with decays of half
the exponent.  The gradient's recurrence runs over as many tokens again, its inputs are such states, and sums over a group's C channels or over the
tokens add their own roundings, at most one for every 64 terms and 64 more: (12 L + 64 + C / 64 + 64) 2^-24.  16-bit rows put up to
2^-17 into a gate (its exponent's rounding).  An output in t adds half a step of t.
"""
import pytest
import torch

import _mix_ref as ref
import quantized_delta_rule_02_amd as sq

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = {F32: "f32", BF16: "bf16", F16: "f16"}
ROWS, BC = ("u", "dt", "z", "dy"), ("b", "c")


STEP = 24 * 2.0 ** -24


def sizes(x, lens, tol, **kw):
    """What float32 may be off by, for every result (see above)."""
    whole, half = ref.ssm_ref(x, lens, size=True, **kw), ref.ssm_ref(x, lens, size=True, rate=0.5, **kw)
    return {k: whole[k] + half[k] * (STEP / tol) for k in whole}


def near(got, want, size, what, tol):
    t = got.dtype
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    half = 0.0 if t == F32 else torch.finfo(t).eps / 2
    tiny = 2.0 ** -25 if t == F16 else 1e-37
    off = (got - want).abs() - half * want.abs() - tiny - (tol + (0.0 if t == F32 else 2.0 ** -16)) * size
    assert not want.numel() or off.max() <= 0, f"{what}: off by {(got - want).abs().max():.3e}, {off.max():.3e} too much"


def wide(x, dev, pad, shift):
    """Rows of a wider array."""
    if not pad and not shift:
        return x.to(dev)
    w = torch.full((x.shape[0], x[0].numel() + pad), 7.0, dtype=x.dtype, device=dev)
    v = w[:, shift:shift + x[0].numel()].unflatten(1, tuple(x.shape[1:]))
    v[:] = x.to(dev)
    return v


def put(x, dev, pad=0, shift=0):
    return {k: wide(v, dev, pad, shift) if k in ROWS + BC else v.to(dev) for k, v in x.items()}


def check(C, N, G, lens, dtype, dev, z=True, d=True, bias=True, softplus=True, s0=True, ds1=True, lead=0, behind=0, pad=0, shift=0, seed=1,
          steps="usual", grads=True, positive=False):
    x = ref.ssm_inputs(C, N, G, lens, seed, dtype, extra=lead + behind, steps=steps)
    if positive:                                        # without softplus the steps are the inputs themselves
        x["dt"], x["dt_bias"] = (x["dt"].float().abs() * 0.1).to(dtype), x["dt_bias"].abs() * 0.01
    g, start = put(x, dev, pad, shift), ref.starts(lens, lead).to(dev)
    kw = dict(lead=lead, z=z, d=d, bias=bias, softplus=softplus, s0=s0)
    opt = dict(d=g["d"] if d else None, dt_bias=g["dt_bias"] if bias else None, z=g["z"] if z else None, softplus=softplus, seq_start=start,
               s0=g["s0"] if s0 else None)
    ins = [g[k] for k in ("u", "dt", "a", "b", "c")]
    L = max(lens, default=0)
    tol = (6 * L + 32) * 2.0 ** -24
    want, size = ref.ssm_ref(x, lens, **kw), sizes(x, lens, tol, **kw)
    y, s1 = wide(torch.full_like(x["u"], 3.0), dev, pad, shift), torch.empty_like(g["s0"])
    sq.sq_ssm_scan(*ins, y, s1=s1, **opt)
    inside = slice(lead, lead + sum(lens))
    near(y[inside], want["y"][inside], size["y"][inside], "y", tol)
    near(s1, want["s1"], size["s1"], "s1", tol)
    out = torch.ones(x["u"].shape[0], dtype=torch.bool)
    out[inside] = False
    assert bool((y[out.to(dev)] == 3).all())
    both = g["s0"].clone()                              # in place
    y2 = torch.empty_like(y)
    sq.sq_ssm_scan(*ins, y2, s1=both, **dict(opt, s0=both if s0 else None))
    assert torch.equal(both, s1) and torch.equal(y2[inside], y[inside])
    if not grads:
        return
    tol = (12 * L + 128 + C / 64) * 2.0 ** -24
    want, size = ref.ssm_ref(x, lens, grads=True, ds1=ds1, **kw), sizes(x, lens, tol, grads=True, ds1=ds1, **kw)
    new = lambda k: wide(torch.full_like(x[k], 3.0), dev, pad, shift)  # noqa: E731
    got = {"du": new("u"), "ddt": new("dt"), "db": new("b"), "dc": new("c"), "dz": new("z") if z else None, "da": torch.empty_like(g["a"]),
           "dd": torch.empty_like(g["d"]), "ddt_bias": torch.empty_like(g["dt_bias"]), "ds0": torch.empty_like(g["s0"])}

    def run(o, grad_in):
        sq.sq_ssm_scan_bwd(*ins, g["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], dz=o["dz"], dd=o["dd"], ddt_bias=o["ddt_bias"], ds1=grad_in,
                           ds0=o["ds0"], **opt)

    run(got, g["ds1"] if ds1 else None)
    for k, v in got.items():
        if v is None:
            continue
        rows = k in ("du", "ddt", "db", "dc", "dz")
        near(v[inside] if rows else v, want[k][inside] if rows else want[k], size[k][inside] if rows else size[k], k, tol)
        if rows:
            assert bool((v[out.to(dev)] == 3).all()), k
            if pad:
                flat = v.as_strided((v.shape[0], v[0].numel() + pad), (v.stride(0), 1), v.storage_offset() - shift)
                assert bool((flat[:, :shift] == 7).all()) and bool((flat[:, shift + v[0].numel():] == 7).all()), k
    # the same bits again, with nothing optional and the states' gradient in place
    more = {k: None if v is None else torch.empty_like(v) for k, v in got.items()}
    if ds1:
        more["ds0"] = g["ds1"].clone()
    run(dict(more, da=None, dd=None, ddt_bias=None, dz=None), more["ds0"] if ds1 else None)
    for k in ("du", "ddt", "db", "dc"):
        assert torch.equal(more[k][inside], got[k][inside]), k
    assert torch.equal(more["ds0"], got["ds0"])


@pytest.mark.parametrize("N", (8, 16, 32, 64, 128))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_states_and_types(N, dtype, dev):
    check(24, N, 2, [5, 0, 40, 1], dtype, dev)


@pytest.mark.parametrize("C,G", ((1, 1), (3, 1), (64, 1), (65, 1), (130, 2), (260, 4), (12, 12), (200, 1)))
@pytest.mark.parametrize("N", (8, 16, 128))
def test_channels_and_groups(C, G, N, dev):
    check(C, N, G, [33, 7], F32, dev)
    check(C, N, G, [9], BF16, dev, seed=3)


@pytest.mark.parametrize("lens", ([1], [0], [0, 0], [2], [8], [9], [31], [32], [33], [63], [64], [65], [128], [7, 64, 1, 66], [1] * 70, [200, 0, 0, 3]),
                         ids=lambda v: "-".join(map(str, v[:8])))
def test_lengths(lens, dev):
    check(20, 16, 1, lens, F32, dev)
    check(20, 16, 1, lens, BF16, dev, seed=7)


@pytest.mark.parametrize("what", (dict(z=False), dict(d=False), dict(bias=False), dict(s0=False), dict(ds1=False), dict(softplus=False, positive=True),
                                  dict(z=False, d=False, bias=False, s0=False, ds1=False)), ids=str)
def test_parts_left_out(what, dev):
    for N in (16, 64):
        check(36, N, 1, [40, 3], F32, dev, **what)


@pytest.mark.parametrize("pad,shift", ((8, 0), (16, 8), (3, 0), (5, 2)))
def test_rows_of_wider_arrays(pad, shift, dev):
    check(32, 16, 2, [5, 70], BF16, dev, pad=pad, shift=shift)
    check(32, 16, 2, [5, 70], F32, dev, pad=pad, shift=shift)


def test_tokens_outside_the_sequences(dev):
    check(16, 16, 1, [5, 0, 90], BF16, dev, lead=9, behind=6)
    check(16, 8, 1, [0, 0], F32, dev, lead=70, behind=100)
    check(16, 8, 1, [150], F32, dev, lead=70, behind=100)


@pytest.mark.parametrize("N", (16, 64))
def test_steps_of_all_sizes(N, dev):
    check(20, N, 1, [70, 20], F32, dev, steps="spread")
    check(20, N, 1, [70, 20], F16, dev, steps="spread")


@pytest.mark.parametrize("lens,C,N", (([700], 8, 16), ([300, 500], 40, 8), ([257, 0, 260, 800], 16, 64)), ids=str)
def test_segments(lens, C, N, dev):
    """Few long sequences, which the forward call cuts into segments."""
    assert sq.sq_ssm_scan_bytes(F32, C, N, 1, len(lens), sum(lens)) > 0
    check(C, N, 1, lens, F32, dev, grads=False)
    check(C, N, 1, lens, BF16, dev, grads=False, seed=5, lead=3)
    check(C, N, 1, lens, F32, dev, s0=False, seed=6)


def test_segments_of_64_tokens_of_the_gradients(dev):
    """The calls of the other tests are small enough for segments of 32 tokens; this one is above the border."""
    C, N, lens = 376, 128, [460, 1, 250]
    assert (sum(lens) >> 6) * (C // 8) >= 512                  # workgroups of segments of 64
    check(C, N, 1, lens, BF16, dev)


def test_long_and_short_segments_of_the_gradients(dev):
    """A call that is large enough for segments of 128 tokens against its channels in four calls, whose segments have 64."""
    C, N, lens, parts = 2048, 16, [5000, 1, 3300], 4
    T = sum(lens)
    rn = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    gen = torch.Generator(device=dev).manual_seed(3)
    u, dt, z, dy, b, c = rn(T, C), 0.5 * rn(T, C) - 3.0, rn(T, C), rn(T, C), rn(T, 1, N), rn(T, 1, N)
    a, d = -(1.0 + torch.arange(N, device=dev)) * (1 + 0.1 * rn(C, N)).clamp(0.5, 2), rn(C)
    s0, ds1, start = rn(3, C, N), rn(3, C, N), ref.starts(lens).to(dev)

    def run(k):
        at = lambda t: t[:, k].contiguous()  # noqa: E731
        v = {n: at(t) for n, t in (("u", u), ("dt", dt), ("z", z), ("dy", dy))}
        o = {n: torch.empty_like(t) for n, t in (("du", v["u"]), ("ddt", v["u"]), ("dz", v["u"]), ("da", a[k].contiguous()), ("db", b), ("dc", c),
                                                ("dd", d[k].contiguous()), ("ds0", at(s0)))}
        sq.sq_ssm_scan_bwd(v["u"], v["dt"], a[k].contiguous(), b, c, v["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], d=d[k].contiguous(), z=v["z"],
                           dz=o["dz"], dd=o["dd"], seq_start=start, s0=at(s0), ds1=at(ds1), ds0=o["ds0"])
        return o

    whole = run(slice(0, C))
    some = [run(slice(i * C // parts, (i + 1) * C // parts)) for i in range(parts)]
    assert (T >> 7) * 32 >= 2048 > (T >> 7) * 8                # workgroups of segments of 128
    rel = lambda x, y: float((x.double() - y.double()).norm() / y.double().norm())  # noqa: E731
    # both are float32 sums of the same terms in other orders: a few roundings of 2^-24 for each of some hundred tokens that last
    for n, dim in (("du", 1), ("ddt", 1), ("dz", 1), ("da", 0), ("dd", 0), ("ds0", 1)):
        assert rel(whole[n], torch.cat([s[n] for s in some], dim)) < 300 * 2.0 ** -24, n
    for n in ("db", "dc"):
        assert rel(whole[n], sum(s[n].double() for s in some)) < 300 * 2.0 ** -24, n


@pytest.mark.parametrize("N,C,G", ((8, 130, 1), (16, 72, 2), (64, 21, 1), (128, 16, 4)))
@pytest.mark.parametrize("dtype", (F32, BF16, F16), ids=NAMES.get)
def test_step(N, C, G, dtype, dev):
    batch, S = 13, 20
    x = ref.ssm_inputs(C, N, G, [1] * batch, 11, dtype)
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(2))[:batch].to(torch.int32)
    slots[2], slots[9] = -1, S
    live = [i for i in range(batch) if 0 <= slots[i] < S]
    pool = ref.rnd(S, C, N, seed=5).float()
    pool[slots[live].long()] = x["s0"][live]
    g, state = put(x, dev), pool.to(dev)
    y = torch.full((batch, C), 3.0, dtype=dtype, device=dev)
    kw = dict(d=g["d"], dt_bias=g["dt_bias"], z=g["z"])
    sq.sq_ssm_step(*[g[k] for k in ("u", "dt", "a", "b", "c")], state, y, slots=slots.to(dev), **kw)
    tol = (6 + 32) * 2.0 ** -24
    want, size = ref.ssm_ref(x, [1] * batch), sizes(x, [1] * batch, tol)
    near(y[live], want["y"][live], size["y"][live], "y", tol)
    near(state[slots[live].long()], want["s1"][live], size["s1"][live], "state", tol)
    rest = torch.ones(S, dtype=torch.bool)
    rest[slots[live].long()] = False
    assert torch.equal(state.cpu()[rest], pool[rest]) and bool((y[2] == 3).all()) and bool((y[9] == 3).all())
    st2, y2 = g["s0"].clone(), torch.empty_like(y)              # no slot list, nothing optional
    sq.sq_ssm_step(*[g[k] for k in ("u", "dt", "a", "b", "c")], st2, y2)
    kw = dict(z=False, d=False, bias=False)
    near(y2, ref.ssm_ref(x, [1] * batch, **kw)["y"], sizes(x, [1] * batch, tol, **kw)["y"], "y", tol)


def test_many_sequences_and_channels(dev):
    """More workgroups than the GPU holds at once; every sequence its own result."""
    C, N, n = 1024, 16, 300
    lens = [1 + (i * 7) % 5 for i in range(n)]
    x = ref.ssm_inputs(C, N, 1, lens, 31, BF16)
    g, start = put(x, dev), ref.starts(lens).to(dev)
    y, s1 = torch.empty_like(g["u"]), torch.empty_like(g["s0"])
    ins = [g[k] for k in ("u", "dt", "a", "b", "c")]
    kw = dict(d=g["d"], dt_bias=g["dt_bias"], z=g["z"])
    sq.sq_ssm_scan(*ins, y, seq_start=start, s0=g["s0"], s1=s1, **kw)
    tol = (6 * 5 + 32) * 2.0 ** -24
    want, size = ref.ssm_ref(x, lens), sizes(x, lens, tol)
    near(y, want["y"], size["y"], "y", tol)
    near(s1, want["s1"], size["s1"], "s1", tol)


def test_tokens_one_by_one_are_the_sequence(dev):
    """A prompt, then its next tokens by single steps against the whole sequence at once; the state set aside in 8 bits between."""
    C, N, n, m = 72, 16, 41, 6
    x = ref.ssm_inputs(C, N, 1, [n + m], 13, F32)
    g = put(x, dev)
    at = lambda s: [g[k][s] if k != "a" else g[k] for k in ("u", "dt", "a", "b", "c")]  # noqa: E731
    kw = lambda s: dict(d=g["d"], dt_bias=g["dt_bias"], z=g["z"][s])  # noqa: E731
    y, state = torch.empty_like(g["u"]), g["s0"].clone()
    sq.sq_ssm_scan(*at(slice(0, n)), y[:n], s0=state, s1=state, **kw(slice(0, n)))
    aside = state.clone()
    for t in range(n, n + m):
        s = slice(t, t + 1)
        sq.sq_ssm_step(*at(s), state, y[s], **kw(s))
    tol = (6 * (n + m) + 32) * 2.0 ** -24
    want, size = ref.ssm_ref(x, [n + m]), sizes(x, [n + m], tol)
    near(y, want["y"], size["y"], "y", tol)
    near(state, want["s1"], size["s1"], "state", tol)
    # set aside in slot 2 of a cache, brought back, and on
    codes, scales = torch.zeros(4, C * N, dtype=torch.uint8, device=dev), torch.zeros(4, C * N // 64, device=dev)
    slot = torch.tensor([2], dtype=torch.int32, device=dev)
    sq.sq_cache_write(aside.view(1, -1), codes, scales, slots=slot)
    back = torch.empty_like(aside)
    sq.sq_cache_read(codes, scales, back.view(1, -1), slots=slot)
    # half a step of the largest value of 64 among 127, and the scale's own rounding
    most = aside.view(-1, 64).abs().amax(1, keepdim=True).expand(-1, 64).reshape(aside.shape)
    assert bool(((back - aside).abs() <= most * (0.5 / 127 + 2.0 ** -20)).all())
    y2 = torch.empty_like(y[n:])
    sq.sq_ssm_scan(*at(slice(n, n + m)), y2, s0=back, s1=back, **kw(slice(n, n + m)))
    err = (0.5 / 127 + 2.0 ** -20) * most.cpu().double()        # decays below one never enlarge it
    assert bool(((y2.cpu().double() - want["y"][n:]).abs() <=
                 ((err * x["c"][n:].double().abs()).sum(-1) * (x["z"][n:].double() * x["z"][n:].double().sigmoid()).abs()) + tol * size["y"][n:]).all())


def test_values_that_are_not_finite_stay_in_their_channel(dev):
    C, N, lens = 80, 16, [100, 30]
    x = ref.ssm_inputs(C, N, 1, lens, 17, F32)
    g, start = put(x, dev), ref.starts(lens).to(dev)

    def run(u, dt):
        y, s1 = torch.empty_like(u), torch.empty_like(g["s0"])
        sq.sq_ssm_scan(u, dt, g["a"], g["b"], g["c"], y, d=g["d"], dt_bias=g["dt_bias"], z=g["z"], seq_start=start, s0=g["s0"], s1=s1)
        o = {k: torch.empty_like(g[s]) for k, s in (("du", "u"), ("ddt", "dt"), ("da", "a"), ("db", "b"), ("dc", "c"), ("dz", "z"), ("ds0", "s0"))}
        sq.sq_ssm_scan_bwd(u, dt, g["a"], g["b"], g["c"], g["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], d=g["d"], dt_bias=g["dt_bias"],
                           z=g["z"], dz=o["dz"], seq_start=start, s0=g["s0"], ds1=g["ds1"], ds0=o["ds0"])
        return dict(o, y=y, s1=s1)

    clean = run(g["u"], g["dt"])
    u, dt = g["u"].clone(), g["dt"].clone()
    u[20, 3], dt[70, 9] = float("inf"), float("nan")
    bad = run(u, dt)
    cols = torch.ones(C, dtype=torch.bool, device=dev)
    cols[3] = cols[9] = False
    for k in ("y", "du", "ddt", "dz"):
        assert torch.equal(clean[k][:, cols], bad[k][:, cols]) and torch.equal(clean[k][100:], bad[k][100:]), k
    for k in ("s1", "ds0"):
        assert torch.equal(clean[k][:, cols], bad[k][:, cols]) and torch.equal(clean[k][1], bad[k][1]), k
    assert torch.equal(clean["da"][cols], bad["da"][cols])
    assert torch.equal(clean["db"][100:], bad["db"][100:]) and torch.equal(clean["dc"][100:], bad["dc"][100:])
    assert torch.equal(clean["y"][:20], bad["y"][:20]) and not bool(torch.isfinite(bad["y"][20:100, 3]).any())
    assert bool(torch.isnan(bad["y"][70:100, 9]).all()) and bool(torch.isnan(bad["s1"][0, 9]).all())


@pytest.mark.parametrize("lens", ([300, 211], [60, 40]), ids=str)
def test_graphs_streams_and_calls_at_once(lens, dev):
    C, N, T = 40, 16, sum(lens)
    g = [put(ref.ssm_inputs(C, N, 1, lens, 21 + i, BF16), dev) for i in range(2)]
    start = [ref.starts(lens).to(dev) for _ in range(2)]
    names = {"y": "u", "s1": "s0", "du": "u", "ddt": "dt", "da": "a", "db": "b", "dc": "c", "dz": "z", "dd": "d", "ddt_bias": "dt_bias", "ds0": "s0"}
    out = [{k: torch.empty_like(z[s]) for k, s in names.items()} for z in g]
    size = [sq.sq_ssm_scan_bytes(BF16, C, N, 1, 2, T, backward=b) for b in (False, True)]
    space = lambda: [torch.empty(max(n, 1), dtype=torch.uint8, device=dev) for n in size]  # noqa: E731
    work = [space() for _ in range(2)]

    def call(i, o, w, stream=None):
        z = g[i]
        ins = [z[k] for k in ("u", "dt", "a", "b", "c")]
        kw = dict(d=z["d"], dt_bias=z["dt_bias"], z=z["z"], seq_start=start[i], s0=z["s0"], stream=stream)
        sq.sq_ssm_scan(*ins, o["y"], s1=o["s1"], workspace=w and w[0], **kw)
        sq.sq_ssm_scan_bwd(*ins, z["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], dz=o["dz"], dd=o["dd"], ddt_bias=o["ddt_bias"], ds1=z["ds1"],
                           ds0=o["ds0"], workspace=w and w[1], **kw)

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
    for now in (lens, [1, T - 1], [T, 0], [3, 2]):
        for s in start:
            s.copy_(ref.starts(now))
        eager = [{k: torch.zeros_like(v) for k, v in o.items()} for o in out]
        for i in range(2):
            for v in out[i].values():
                v.zero_()
            call(i, eager[i], space())
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for k in out[i]:
                assert torch.equal(out[i][k], eager[i][k]), (now, k)
        other = {k: torch.zeros_like(v) for k, v in out[0].items()}
        torch.cuda.synchronize()
        call(0, other, None, stream=side)
        side.synchronize()
        for k in other:
            assert torch.equal(other[k], eager[0][k]), k


def test_offsets_that_break_the_rules_touch_nothing_else(dev):
    C, N, n, T = 24, 16, 3, 900
    x = ref.ssm_inputs(C, N, 1, [300] * n, 71, F32)
    g = put(x, dev)
    names = {"y": "u", "s1": "s0", "du": "u", "ddt": "dt", "da": "a", "db": "b", "dc": "c", "dz": "z", "dd": "d", "ddt_bias": "dt_bias", "ds0": "s0"}
    size = [sq.sq_ssm_scan_bytes(F32, C, N, 1, n, T, backward=b) for b in (False, True)]
    assert size[0] > 0                                  # goes by segments
    for at in ([0, 600, 100, 900], [-50, 10, 20, 4000], [900, 800, 600, 40], [2 ** 31 - 1, -2 ** 31, 5, 2 ** 30]):
        start = torch.tensor(at, dtype=torch.int32, device=dev)
        bufs, o = {}, {}
        for k, s in names.items():
            bufs[k] = torch.full((g[s].numel() + 2 * 4096,), 3.0, device=dev)
            o[k] = bufs[k][4096:4096 + g[s].numel()].view(g[s].shape)
        work = [torch.full((b + 2 * 4096,), 7, dtype=torch.uint8, device=dev) for b in size]
        ins = [g[k] for k in ("u", "dt", "a", "b", "c")]
        kw = dict(d=g["d"], dt_bias=g["dt_bias"], z=g["z"], seq_start=start, s0=g["s0"])
        sq.sq_ssm_scan(*ins, o["y"], s1=o["s1"], workspace=work[0][4096:4096 + size[0]], **kw)
        sq.sq_ssm_scan_bwd(*ins, g["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], dz=o["dz"], dd=o["dd"], ddt_bias=o["ddt_bias"], ds1=g["ds1"],
                           ds0=o["ds0"], workspace=work[1][4096:4096 + size[1]], **kw)
        torch.cuda.synchronize()
        for k, b in bufs.items():
            assert bool((b[:4096] == 3).all()) and bool((b[-4096:] == 3).all()), (at, k)
        for b, w in zip(size, work):
            assert bool((w[:4096] == 7).all()) and bool((w[4096 + b:] == 7).all()), at


def test_no_sequences_and_no_tokens(dev):
    C, N = 24, 16
    x = ref.ssm_inputs(C, N, 1, [10], 3, F32)
    g = put(x, dev)
    none = torch.zeros(1, dtype=torch.int32, device=dev)
    ins = [g[k] for k in ("u", "dt", "a", "b", "c")]
    y = torch.full_like(g["u"], 3.0)
    sq.sq_ssm_scan(*ins, y, seq_start=none)
    o = {k: torch.full_like(g[s], 3.0) for k, s in (("du", "u"), ("ddt", "dt"), ("da", "a"), ("db", "b"), ("dc", "c"), ("dd", "d"), ("dt", "dt_bias"))}
    sq.sq_ssm_scan_bwd(*ins, g["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], dd=o["dd"], ddt_bias=o["dt"], seq_start=none)
    assert bool((y == 3).all()) and all(bool((o[k] == 3).all()) for k in ("du", "ddt", "db", "dc"))
    assert not o["da"].any() and not o["dd"].any() and not o["dt"].any()
    e, eb = torch.zeros(0, C, device=dev), torch.zeros(0, 1, N, device=dev)
    s0, start = torch.randn(2, C, N, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    s1, ds0 = torch.empty_like(s0), torch.empty_like(s0)
    sq.sq_ssm_scan(e, e, g["a"], eb, eb, e, seq_start=start, s0=s0, s1=s1)
    sq.sq_ssm_scan_bwd(e, e, g["a"], eb, eb, e, e, e, o["da"], eb, eb, seq_start=start, s0=s0, ds1=s1, ds0=ds0)
    assert torch.equal(s1, s0) and torch.equal(ds0, s0) and not o["da"].any()
    sq.sq_ssm_step(e, e, g["a"], eb, eb, s0, e)


def test_beyond_32_bit_offsets(dev):
    """A pool of states above 2^32 bytes and 2^31 elements, its first and last slot."""
    C, N = 4096, 128
    S = (1 << 31) // (C * N) + 3
    pool = torch.zeros(S, C, N, device=dev)
    x = ref.ssm_inputs(C, N, 1, [1, 1], 41, BF16)
    g = put(x, dev)
    slots = torch.tensor([S - 1, 0], dtype=torch.int32, device=dev)
    pool[slots.long()] = g["s0"]
    y = torch.empty_like(g["u"])
    sq.sq_ssm_step(*[g[k] for k in ("u", "dt", "a", "b", "c")], pool, y, slots=slots, d=g["d"], dt_bias=g["dt_bias"], z=g["z"])
    want, size = ref.ssm_ref(x, [1, 1]), sizes(x, [1, 1], 38 * 2.0 ** -24)
    near(y, want["y"], size["y"], "y", 38 * 2.0 ** -24)
    near(pool[slots.long()], want["s1"], size["s1"], "state", 38 * 2.0 ** -24)


def test_conv_then_scan_is_a_layer(dev):
    """Convolution, scan and gated output of a layer over a ragged batch, its gradients chained back to the convolution's input,
    against float64 of the whole."""
    C, N, W, lens = 48, 16, 4, [70, 5, 33]
    x = ref.ssm_inputs(C, N, 1, lens, 51, F32)
    v = ref.conv_inputs(C, W, lens, 61, F32)
    g, k, start = put(x, dev), {n: t.to(dev) for n, t in v.items()}, ref.starts(lens).to(dev)
    u, y = torch.empty_like(g["u"]), torch.empty_like(g["u"])
    sq.sq_conv(k["x"], k["weight"], u, bias=k["bias"], seq_start=start)
    opt = dict(d=g["d"], dt_bias=g["dt_bias"], z=g["z"], seq_start=start)
    ins = (g["dt"], g["a"], g["b"], g["c"])
    sq.sq_ssm_scan(u, *ins, y, **opt)
    o = {n: torch.empty_like(g[s]) for n, s in (("du", "u"), ("ddt", "dt"), ("da", "a"), ("db", "b"), ("dc", "c"), ("dz", "z"))}
    sq.sq_ssm_scan_bwd(u, *ins, g["dy"], o["du"], o["ddt"], o["da"], o["db"], o["dc"], dz=o["dz"], **opt)
    dx, dw, db = torch.empty_like(u), torch.empty_like(k["weight"]), torch.empty_like(k["bias"])
    sq.sq_conv_bwd(k["x"], k["weight"], o["du"], dx, dweight=dw, dbias=db, bias=k["bias"], seq_start=start)
    mid = ref.conv_ref(v, lens, s0=False)["y"]
    x64 = {n: t.double() for n, t in x.items()}
    x64["u"] = mid
    want = ref.ssm_ref(x64, lens, s0=False)["y"]
    back = ref.ssm_ref(x64, lens, s0=False, ds1=False, grads=True)
    last = ref.conv_ref(dict(v, dy=back["du"]), lens, s0=False, ds1=False, grads=True)
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    # float32 all the way: 70 tokens there and back of 2^-24 each at most (12 x 70 + 128) 2^-24 = 5.8e-5 in the worst order of signs
    for a, b in ((y, want), (o["du"], back["du"]), (o["db"], back["db"]), (dx, last["dx"]), (dw, last["dweight"]), (db, last["dbias"])):
        assert rel(a, b) < 5.8e-5
