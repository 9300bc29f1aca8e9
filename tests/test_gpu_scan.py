"""The gated delta scan and its gradients on the GPU against float64 references, token by token.

Tolerance.  Products split every float32 operand exactly into three bfloat16 parts (8 bits each, rounded to nearest: what one
leaves is at most 2^-8 of the value, what two leave 2^-16) and leave out two terms of at most 2^-8 * 2^-16 = 2^-24 of |a||b|;
float32 accumulation adds some 2^-24 per term, over at most 24 products of matrix instructions a result.  TOL holds an output's
largest error against its largest value: a result passes through at most five such products within a chunk (state, That, P,
update; one more for gradients), 5 * 26 * 2^-24 = 7.7e-6 of the terms if all roundings agree.  L2 and L2_GRAD hold the relative error of a
whole array, where roundings add up in quadrature: see test_every_part_counts.  An output in t adds half a step:
torch.finfo(t).eps / 2 of its value.
"""
import numpy as np
import pytest
import torch

import quantized_delta_rule_02_amd as sq
from _ops_ref import scan_grad_ref, scan_inputs, scan_ref

pytestmark = pytest.mark.gpu

TOL = 1e-5
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
GRADS = ("dq", "dk", "dv", "dgate", "dbeta", "ds0")


def say(*a):
    print(*a, flush=True)


def starts(lens, dev, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(lens)]), dtype=torch.int32, device=dev)


def near(got, ref, what, tol=TOL):
    t = got.dtype
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    if not ref.numel():
        return
    half = 0.0 if t == F32 else torch.finfo(t).eps / 2
    off = (got - ref).abs() - half * ref.abs() - tol * ref.abs().max()
    assert off.max() <= 0, f"{what}: off by {(got - ref).abs().max():.3e}, largest {ref.abs().max():.3e}"


def forward(form, x, lens, dev, s0=True, **kw):
    d = {n: t.to(dev) for n, t in x.items()}
    y, s1 = torch.zeros_like(d["v"]), torch.zeros_like(d["s0"])
    sq.sq_delta_scan(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], y, seq_start=starts(lens, dev),
                     s0=d["s0"] if s0 else None, s1=s1, **kw)
    return y, s1


def backward(form, x, lens, dev, s0=True, ds1=True, **kw):
    d = {n: t.to(dev) for n, t in x.items()}
    g = {"d" + n: torch.zeros_like(d[n]) for n in ("q", "k", "v", "gate", "beta", "s0")}
    sq.sq_delta_scan_bwd(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], d["dy"], g["dq"], g["dk"], g["dv"],
                         g["dgate"], g["dbeta"], seq_start=starts(lens, dev), s0=d["s0"] if s0 else None,
                         ds1=d["ds1"] if ds1 else None, ds0=g["ds0"], **kw)
    return g


# form, dtype, heads, q/k heads, d_k, d_v, lengths, gates
CASES = [
    (0, F32, 2, 2, 16, 16, [5], "usual"),
    (0, F32, 2, 1, 16, 16, [1, 0, 33], "strong"),
    (1, F32, 2, 2, 16, 16, [40, 1], "usual"),
    (0, F32, 2, 1, 64, 64, [1, 16, 0, 70], "usual"),
    (1, F32, 2, 2, 64, 64, [31, 32, 33], "strong"),
    (0, BF16, 4, 2, 128, 128, [65, 1, 97], "usual"),
    (0, F16, 2, 2, 128, 128, [17, 64], "resets"),
    (0, F32, 3, 1, 128, 128, [50, 15], "resets"),
    (1, BF16, 4, 2, 128, 128, [65, 0, 30], "usual"),
    (1, F16, 2, 1, 128, 128, [33], "resets"),
    (1, F32, 1, 1, 128, 256, [47], "usual"),
    (0, BF16, 2, 1, 128, 256, [64, 2], "one"),
    (1, BF16, 2, 2, 64, 64, [96], "one"),
]
IDS = [f"{'kda' if c[0] else 'gdn'}-{str(c[1])[6:]}-{c[2]}h{c[3]}-{c[4]}x{c[5]}-{'_'.join(map(str, c[6]))}-{c[7]}" for c in CASES]


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_forward(c, dev):
    form, dt, H, Hk, dk, dv, lens, gate = c
    say("scan", c)
    x = scan_inputs(form, H, Hk, dk, dv, lens, 11, dt, gate)
    for s0 in (True, False):
        y, s1 = forward(form, x, lens, dev, s0)
        yr, sr = scan_ref(x, lens, s0)
        near(y, yr, "y")
        near(s1, sr, "s1")


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_backward(c, dev):
    form, dt, H, Hk, dk, dv, lens, gate = c
    say("scan bwd", c)
    x = scan_inputs(form, H, Hk, dk, dv, lens, 23, dt, gate)
    for states in (True, False):
        g = backward(form, x, lens, dev, states, states)
        r = scan_grad_ref(x, lens, states, states)
        for n in GRADS:
            if n == "ds0" and not states:
                continue                    # the reference has no first state to differentiate by
            near(g[n], r[n], n)


@pytest.mark.parametrize("dt", (BF16, F16, F32), ids=("bfloat16", "float16", "float32"))
@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_many_states(form, dt, dev):
    """More workgroups than CUs: eight computing waves to a workgroup instead of four (both directions)."""
    H, Hk, dk, dv, lens = 32, 16, 128, 128, [33, 1, 0, 4, 2]
    x = scan_inputs(form, H, Hk, dk, dv, lens, 71, dt)
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    for n in GRADS:
        near(g[n], r[n], n)


@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_many_wide_states(form, dev):
    H, dk, dv, lens = 32, 128, 256, [5, 33, 1]
    x = scan_inputs(form, H, H, dk, dv, lens, 72, BF16)
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")


SHORT = [(0, BF16, 4, 2, 128, 128), (0, F16, 2, 2, 128, 256), (0, F32, 3, 1, 64, 64), (0, F32, 2, 1, 128, 128),
         (1, BF16, 4, 4, 128, 128), (1, F16, 3, 1, 64, 64), (1, F32, 2, 2, 128, 256), (0, BF16, 2, 1, 16, 16), (1, F32, 2, 2, 16, 16)]


@pytest.mark.parametrize("gate", ("usual", "strong"))
@pytest.mark.parametrize("c", SHORT, ids=[f"{'kda' if c[0] else 'gdn'}-{str(c[1])[6:]}-{c[2]}h{c[3]}-{c[4]}x{c[5]}" for c in SHORT])
def test_short_sequences(c, gate, dev):
    """Few tokens a sequence, and one of 17 and one of 40 among them: the sequences of up to 16 go token by token."""
    form, dt, H, Hk, dk, dv = c
    lens = [1, 0, 8, 2, 9, 3, 40, 4, 1, 5, 10, 6, 0, 7, 16, 17, 1, 2]
    assert sum(lens) <= 12 * len(lens)
    x = scan_inputs(form, H, Hk, dk, dv, lens, 61, dt, gate)
    for s0 in (True, False):
        y, s1 = forward(form, x, lens, dev, s0)
        yr, sr = scan_ref(x, lens, s0)
        near(y, yr, "y")
        near(s1, sr, "s1")
    for few in ([3], [0, 16], [1] * 5):              # no sequence can be longer: nothing else runs
        x = scan_inputs(form, H, Hk, dk, dv, few, 62, dt, gate)
        y, s1 = forward(form, x, few, dev)
        yr, sr = scan_ref(x, few)
        near(y, yr, "y")
        near(s1, sr, "s1")


def test_short_sequences_in_wider_arrays_in_place_and_captured(dev):
    """Parts of wider arrays with NaN around them, tokens of no sequence, the states replaced in place; the captured call
    replayed gives what the eager calls give."""
    form, H, Hk, dk, dv, lens, lead, tail = 1, 4, 2, 128, 128, [1, 5, 20, 0, 8], 2, 3
    x = scan_inputs(form, H, Hk, dk, dv, lens, 63, BF16)
    T = sum(lens)
    assert lead + T + tail <= 12 * len(lens)
    nan = lambda *s, dt=BF16: torch.full(s, float("nan"), dtype=dt, device=dev)  # noqa: E731
    N, wide = lead + T + tail, nan(lead + T + tail, 2 * Hk * dk + H * dv + 8)
    q, k = (wide[:, i * Hk * dk:(i + 1) * Hk * dk].unflatten(1, (Hk, dk)) for i in (0, 1))
    v = wide[:, 2 * Hk * dk:2 * Hk * dk + H * dv].unflatten(1, (H, dv))
    gate, beta = nan(N, H, dk, dt=F32), nan(N, H, dt=F32)
    for a, n in ((q, "q"), (k, "k"), (v, "v"), (gate, "gate"), (beta, "beta")):
        a[lead:lead + T] = x[n].to(dev)
    out = torch.full((N, H * dv + 8), 7.0, dtype=BF16, device=dev)
    y, st, at = out[:, :H * dv].unflatten(1, (H, dv)), x["s0"].to(dev), starts(lens, dev, lead)
    work = torch.empty(sq.sq_delta_scan_bytes(form, BF16, H, Hk, dk, dv, len(lens), N), dtype=torch.uint8, device=dev)
    call = lambda: sq.sq_delta_scan(form, q, k, v, gate, beta, y, seq_start=at, s0=st, s1=st, workspace=work)  # noqa: E731
    call()
    yr, sr = scan_ref(x, lens)
    near(y[lead:lead + T], yr, "y")
    near(st, sr, "s1")
    assert (out[:lead] == 7).all() and (out[lead + T:] == 7).all() and (out[:, H * dv:] == 7).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        before = st.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), st.clone()
        st.copy_(before)
        call()
        assert torch.equal(got[1], st) and torch.equal(got[0][lead:lead + T], y[lead:lead + T])


@pytest.mark.parametrize("N", (40, 16), ids=("chunks", "tokens"))
def test_offsets_that_break_the_rules_stay_inside(N, dev):
    """Offsets below zero, beyond the arrays or decreasing: results are unspecified, the rows around the arrays stay."""
    H, dk, dv = 2, 64, 64
    for at in ([-7, 50, 20], [30, 10, 400], [0, 2 ** 31 - 1, 5], [-2 ** 31, 0, 40]):
        pad = torch.full((N + 16, H * dv), 7.0, device=dev)
        y = pad[8:8 + N].view(N, H, dv)
        z = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
        sq.sq_delta_scan(0, z(N, H, dk), z(N, H, dk), z(N, H, dv), torch.ones(N, H, device=dev), z(N, H), y,
                         seq_start=torch.tensor(at, dtype=torch.int32, device=dev), s1=z(2, H, dk, dv))
        torch.cuda.synchronize()
        assert (pad[:8] == 7).all() and (pad[8 + N:] == 7).all(), at


@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_equal_keys_and_extreme_beta(form, dev):
    """One key for all tokens, no decay, beta 1 or 0: (I + A)^-1 has rows that sum large terms; beta = 0 divides nowhere."""
    lens, H, dk, dv = [64, 7], 2, 64, 64
    x = scan_inputs(form, H, H, dk, dv, lens, 5, F32, "one")
    x["k"] = x["k"][:1].expand_as(x["k"]).contiguous()
    x["beta"] = torch.ones_like(x["beta"])
    x["beta"][3::5] = 0.0
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    for n in GRADS:
        near(g[n], r[n], n)
    x["beta"].zero_()
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    for n in GRADS:
        near(g[n], r[n], n)
    assert not g["dv"].any()


@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_gates_of_zero(form, dev):
    """A zero gate forgets the state; its gradient stays that of the formula (no quotient by it)."""
    lens, H, dk, dv = [70], 2, 64, 64
    x = scan_inputs(form, H, H, dk, dv, lens, 8, F32, "usual")
    x["gate"][::9] = 0.0
    x["gate"][40] = 1e-38
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    for n in GRADS:
        near(g[n], r[n], n)
    near(g["dgate"][::9], r["dgate"][::9], "dgate of the zero gates")


def test_gradients_against_differences(dev):
    """Central differences of the forward call itself, along random directions of each input, in float32."""
    form, lens, H, dk, dv = 1, [45, 3], 2, 64, 64
    x = scan_inputs(form, H, 1, dk, dv, lens, 31, F32)
    g = backward(form, x, lens, dev)

    def loss(z):
        y, s1 = forward(form, z, lens, dev)
        return ((y.double().cpu() * x["dy"].double()).sum() + (s1.double().cpu() * x["ds1"].double()).sum()).item()

    step = 1e-2
    for i, n in enumerate(("q", "k", "v", "gate", "beta", "s0")):
        d = torch.randn(x[n].shape, generator=torch.Generator().manual_seed(50 + i))
        d = (d / d.norm()).float() * (0.05 if n == "gate" else 1.0)
        hi, lo = dict(x), dict(x)
        hi[n], lo[n] = x[n] + step * d, x[n] - step * d
        d64 = (hi[n].double() - lo[n].double()) / (2 * step)
        num = (loss(hi) - loss(lo)) / (2 * step)
        ana = (g["d" + n].double().cpu() * d64).sum().item()
        scale = g["d" + n].double().norm().item() * d64.norm().item()
        # float32 losses of size |loss| carry 1e-5 |loss| / step; the third derivative adds step^2 of the gradient's size
        assert abs(num - ana) <= 1e-5 * abs(loss(x)) / step + 4 * step ** 2 * scale + 1e-5 * scale, (n, num, ana, scale)


def test_cut_sequence_equals_whole(dev):
    """A sequence in pieces of odd lengths, states handed on in place, gives the whole sequence's outputs."""
    form, H, dk, dv, T = 0, 4, 128, 128, 150
    x = scan_inputs(form, H, 2, dk, dv, [T], 3, BF16)
    d = {n: t.to(dev) for n, t in x.items()}
    yr, sr = scan_ref(x, [T])
    st, y, t0 = d["s0"].clone(), torch.zeros_like(d["v"]), 0
    for n in (1, 40, 32, 0, 70, 7):
        s = slice(t0, t0 + n)
        sq.sq_delta_scan(form, d["q"][s], d["k"][s], d["v"][s], d["gate"][s], d["beta"][s], y[s], s0=st, s1=st)
        t0 += n
    near(y, yr, "y")
    near(st, sr, "s1")


def test_one_token_is_the_decode_step(dev):
    """One token per request is what sq_fp32_step computes (float32 inputs, same state)."""
    H, dk, dv, B = 4, 128, 128, 9
    x = scan_inputs(1, H, H, dk, dv, [1] * B, 17, F32)
    d = {n: t.to(dev) for n, t in x.items()}
    y, s1 = forward(1, x, [1] * B, dev)
    S, y2 = d["s0"].clone(), torch.zeros(B * H * dv, device=dev)
    slots = torch.arange(B, dtype=torch.int32, device=dev)
    sq.sq_fp32_step(1, H, dk, dv, B, 0, 1, B, slots, S, d["q"], d["k"], d["v"], d["gate"], d["beta"], y2)
    near(y.view(-1), y2.cpu(), "y")
    near(s1, S.cpu(), "state")


def test_parts_of_wider_arrays_and_rows_outside(dev):
    """q, k, v, y and their gradients as parts of wider arrays; tokens before, between and behind stay untouched."""
    form, H, Hk, dk, dv, lens = 0, 4, 2, 128, 128, [33, 20]
    lead, tail = 3, 5
    x = scan_inputs(form, H, Hk, dk, dv, lens, 41, BF16)
    T = sum(lens)
    N = lead + T + tail
    wide = torch.full((N, 2 * Hk * dk + H * dv + 8), float("nan"), dtype=BF16, device=dev)
    part = lambda a, at, h, w: a[:, at:at + h * w].unflatten(1, (h, w))  # noqa: E731
    cut = lambda a: (part(a, 0, Hk, dk), part(a, Hk * dk, Hk, dk), part(a, 2 * Hk * dk, H, dv))  # noqa: E731
    for a, n in zip(cut(wide), ("q", "k", "v")):
        a[lead:lead + T] = x[n].to(dev)
    pad = lambda t: torch.cat([torch.full((lead, *t.shape[1:]), float("nan")), t.float(),  # noqa: E731
                               torch.full((tail, *t.shape[1:]), float("nan"))]).to(dev)
    gate, beta = pad(x["gate"]), pad(x["beta"])
    out = torch.full((N, H * dv + 8), 7.0, dtype=BF16, device=dev)
    y, s1 = part(out, 0, H, dv), torch.zeros(2, H, dk, dv, device=dev)
    q, k, v = cut(wide)
    sq.sq_delta_scan(form, q, k, v, gate, beta, y, seq_start=starts(lens, dev, lead), s0=x["s0"].to(dev), s1=s1)
    yr, sr = scan_ref(x, lens)
    near(y[lead:lead + T], yr, "y")
    near(s1, sr, "s1")
    assert (out[:lead] == 7).all() and (out[lead + T:] == 7).all() and (out[:, H * dv:] == 7).all()
    gw = torch.full_like(wide, 7.0)
    dq, dk_, dv_ = cut(gw)
    dgate, dbeta = torch.full_like(gate, 7.0), torch.full_like(beta, 7.0)
    dy = pad(x["dy"]).to(BF16)
    sq.sq_delta_scan_bwd(form, q, k, v, gate, beta, dy, dq, dk_, dv_, dgate, dbeta, seq_start=starts(lens, dev, lead),
                         s0=x["s0"].to(dev))
    r = scan_grad_ref(x, lens, True, False)
    for n, t in (("dq", dq), ("dk", dk_), ("dv", dv_), ("dgate", dgate), ("dbeta", dbeta)):
        near(t[lead:lead + T], r[n], n)
        assert (t[:lead] == 7).all() and (t[lead + T:] == 7).all(), n
    assert (gw[:, -8:] == 7).all()


def test_empty_sequences_only(dev):
    s0 = torch.randn(3, 2, 64, 64, device=dev)
    e = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    s1 = e(3, 2, 64, 64)
    sq.sq_delta_scan(0, e(0, 2, 64), e(0, 2, 64), e(0, 2, 64), e(0, 2), e(0, 2), e(0, 2, 64),
                     seq_start=starts([0, 0, 0], dev), s0=s0, s1=s1)
    assert torch.equal(s0, s1)
    ds0 = e(3, 2, 64, 64)
    sq.sq_delta_scan_bwd(0, e(0, 2, 64), e(0, 2, 64), e(0, 2, 64), e(0, 2), e(0, 2), e(0, 2, 64), e(0, 2, 64), e(0, 2, 64),
                         e(0, 2, 64), e(0, 2), e(0, 2), seq_start=starts([0, 0, 0], dev), ds1=s0, ds0=ds0)
    assert torch.equal(s0, ds0)
    sq.sq_delta_scan(0, e(0, 2, 64), e(0, 2, 64), e(0, 2, 64), e(0, 2), e(0, 2), e(0, 2, 64), seq_start=starts([], dev))


def test_runs_are_bitwise_equal_and_streams_are_kept(dev):
    """Repeated calls, one on another stream with its own workspace, give the same bits."""
    form, H, dk, dv, lens = 1, 4, 128, 128, [90, 33]
    x = scan_inputs(form, H, 2, dk, dv, lens, 77, BF16)
    a = (*forward(form, x, lens, dev), *backward(form, x, lens, dev).values())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d = {n: t.to(dev) for n, t in x.items()}
    torch.cuda.synchronize()
    y, s1 = torch.zeros_like(d["v"]), torch.zeros_like(d["s0"])
    g = {"d" + n: torch.zeros_like(d[n]) for n in ("q", "k", "v", "gate", "beta", "s0")}
    at = starts(lens, dev)
    torch.cuda.synchronize()
    sq.sq_delta_scan(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], y, seq_start=at, s0=d["s0"], s1=s1, stream=side)
    sq.sq_delta_scan_bwd(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], d["dy"], g["dq"], g["dk"], g["dv"], g["dgate"],
                         g["dbeta"], seq_start=at, s0=d["s0"], ds1=d["ds1"], ds0=g["ds0"], stream=side)
    torch.cuda.synchronize()
    for u, w in zip(a, (y, s1, *g.values())):
        assert torch.equal(u, w)


def test_two_calls_at_once(dev):
    """A forward and a backward call on two streams, each with its own workspace, and calls on a third in between."""
    form, H, dk, dv, lens = 0, 16, 128, 128, [500, 33, 700]
    x = scan_inputs(form, H, 8, dk, dv, lens, 78, BF16)
    d = {n: t.to(dev) for n, t in x.items()}
    at = starts(lens, dev)
    ya, sa = forward(form, x, lens, dev)
    ga = backward(form, x, lens, dev)
    y, s1 = torch.zeros_like(d["v"]), torch.zeros_like(d["s0"])
    y2, s2 = torch.zeros_like(y), torch.zeros_like(s1)
    g = {"d" + n: torch.zeros_like(d[n]) for n in ("q", "k", "v", "gate", "beta", "s0")}
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    for _ in range(3):
        sq.sq_delta_scan_bwd(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], d["dy"], g["dq"], g["dk"], g["dv"], g["dgate"],
                             g["dbeta"], seq_start=at, s0=d["s0"], ds1=d["ds1"], ds0=g["ds0"], stream=a)
        sq.sq_delta_scan(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], y, seq_start=at, s0=d["s0"], s1=s1, stream=b)
        sq.sq_delta_scan(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], y2, seq_start=at, s0=d["s0"], s1=s2, stream=c)
    torch.cuda.synchronize()
    for u, w in zip((ya, sa, ya, sa, *ga.values()), (y, s1, y2, s2, *g.values())):
        assert torch.equal(u, w)


def test_arrays_beyond_32_bits(dev):
    """One sequence whose gates pass 4 GiB and whose q rows lie 64 KiB apart: its last piece (a whole number of chunks in)
    equals a call for that piece from the state before it, bit for bit."""
    form, H, Hk, dk, dv, T, cut = 1, 32, 2, 128, 128, 280001, 279936
    r = lambda *s: torch.randn(*s, device=dev)  # noqa: E731
    wide = torch.zeros(T, 1 << 15, dtype=BF16, device=dev)
    q, k = wide[:, 512:512 + Hk * dk].unflatten(1, (Hk, dk)), (r(T, Hk, dk) * dk ** -0.5).to(BF16)
    q.copy_(r(T, Hk, dk))
    v, y = r(T, H, dv).to(BF16), torch.empty(T, H, dv, dtype=BF16, device=dev)
    gate, beta = torch.rand(T, H, dk, device=dev).mul_(0.1).add_(0.9), torch.rand(T, H, device=dev)
    assert gate.numel() * 4 > 1 << 32 and wide.numel() * 2 > 1 << 32
    s1, sc, s2 = (torch.empty(1, H, dk, dv, device=dev) for _ in range(3))
    sq.sq_delta_scan(form, q, k, v, gate, beta, y, s1=s1)
    say("whole sequence queued")
    y2 = torch.empty_like(y[cut:])
    sq.sq_delta_scan(form, q[:cut], k[:cut], v[:cut], gate[:cut], beta[:cut], torch.empty_like(y[:cut]), s1=sc)
    sq.sq_delta_scan(form, q[cut:], k[cut:], v[cut:], gate[cut:], beta[cut:], y2, s0=sc, s1=s2)
    assert torch.isfinite(y).all() and torch.equal(y[cut:], y2) and torch.equal(s1, s2)


def test_gradients_with_states_beyond_32_bits(dev):
    """States and their gradients of more than 2^31 elements each in the workspace: the last piece's gradients equal a
    call for that piece from the state before it."""
    form, H, Hk, dk, dv, T, cut = 0, 32, 8, 128, 128, 140001, 139936
    assert (cut // 32) * H * dk * dv > 1 << 31 and cut % 32 == 0
    r = lambda *s: torch.randn(*s, device=dev)  # noqa: E731
    q, k, v, dy = r(T, Hk, dk).to(BF16), (r(T, Hk, dk) * dk ** -0.5).to(BF16), r(T, H, dv).to(BF16), r(T, H, dv).to(BF16)
    gate, beta = torch.rand(T, H, device=dev).mul_(0.1).add_(0.9), torch.rand(T, H, device=dev)
    sc = torch.empty(1, H, dk, dv, device=dev)
    sq.sq_delta_scan(form, q[:cut], k[:cut], v[:cut], gate[:cut], beta[:cut], torch.empty_like(v[:cut]), s1=sc)
    out = lambda s: [torch.empty_like(t[s]) for t in (q, k, v, gate, beta)]  # noqa: E731
    whole, last = out(slice(0, T)), out(slice(cut, T))
    sq.sq_delta_scan_bwd(form, q, k, v, gate, beta, dy, *whole)
    say("whole sequence queued")
    sq.sq_delta_scan_bwd(form, q[cut:], k[cut:], v[cut:], gate[cut:], beta[cut:], dy[cut:], *last, s0=sc)
    for a, b, n in zip(whole, last, GRADS):
        assert torch.isfinite(a).all(), n
        near(a[cut:], b.double().cpu(), n, 2 * TOL + (0.0 if a.dtype == F32 else torch.finfo(a.dtype).eps / 2))    # both round


def test_captured_and_replayed(dev):
    """Scan and gradients captured into one graph; replays with changed inputs equal the eager calls."""
    form, H, dk, dv, lens = 0, 4, 128, 128, [70, 5]
    x = scan_inputs(form, H, 2, dk, dv, lens, 91, BF16)
    d = {n: t.to(dev) for n, t in x.items()}
    at = starts(lens, dev)
    y, s1 = torch.zeros_like(d["v"]), torch.zeros_like(d["s0"])
    g = {"d" + n: torch.zeros_like(d[n]) for n in ("q", "k", "v", "gate", "beta", "s0")}
    nb = sq.sq_delta_scan_bytes(form, BF16, H, 2, dk, dv, 2, sum(lens), backward=True)
    work = torch.empty(nb, dtype=torch.uint8, device=dev)

    def both():
        sq.sq_delta_scan(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], y, seq_start=at, s0=d["s0"], s1=s1, workspace=work)
        sq.sq_delta_scan_bwd(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], d["dy"], g["dq"], g["dk"], g["dv"], g["dgate"],
                             g["dbeta"], seq_start=at, s0=d["s0"], ds1=d["ds1"], ds0=g["ds0"], workspace=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(3):
        z = scan_inputs(form, H, 2, dk, dv, lens, 200 + i, BF16)
        for n in d:
            d[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, s1, *g.values())]
        ey, es = forward(form, z, lens, dev)
        for u, w in zip(got, (ey, es, *backward(form, z, lens, dev).values())):
            assert torch.equal(u, w)


@pytest.mark.parametrize("n,dk,form", ((65, 64, 1), (150, 64, 0), (4200, 16, 0)))
def test_many_sequences(n, dk, form, dev):
    """More sequences than a wave has lanes, empty ones and longer ones among them."""
    lens = [int(i) for i in np.random.default_rng(n).choice([0, 1, 2, 20, 35], size=n, p=[0.3, 0.4, 0.25, 0.03, 0.02])]
    lens[-1], lens[n // 2] = 33, 40
    x = scan_inputs(form, 1, 1, dk, dk, lens, 97, F32)
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    for i in GRADS:
        near(g[i], r[i], i)


@pytest.mark.parametrize("sizes", ([[1, 3, 0, 20, 2], [16, 17, 1, 0, 5], [0, 0, 39, 0, 0], [8] * 5], [[70, 30, 1], [0, 101, 0], [33, 32, 36]]),
                         ids=("short", "long"))
def test_captured_then_other_lengths(sizes, dev):
    """The offsets live on the device: a captured call replayed with other lengths takes those."""
    form, H, Hk, dk, dv = 0, 4, 2, 128, 128
    N, n = max(map(sum, sizes)), len(sizes[0])
    x = scan_inputs(form, H, Hk, dk, dv, [N], 95, BF16)
    d = {i: t.to(dev) for i, t in x.items()}
    s0 = 0.3 * torch.randn(n, H, dk, dv, device=dev)
    y, s1, at = torch.zeros_like(d["v"]), torch.zeros_like(s0), starts(sizes[0], dev)
    work = torch.empty(sq.sq_delta_scan_bytes(form, BF16, H, Hk, dk, dv, n, N), dtype=torch.uint8, device=dev)
    call = lambda: sq.sq_delta_scan(form, d["q"], d["k"], d["v"], d["gate"], d["beta"], y, seq_start=at, s0=s0, s1=s1,  # noqa: E731
                                    workspace=work)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in sizes[1:] + sizes[:1]:
        at.copy_(starts(lens, dev))
        y.zero_(), s1.zero_()
        graph.replay()
        torch.cuda.synchronize()
        T = sum(lens)
        yr, sr = scan_ref({**{i: t[:T] for i, t in x.items()}, "s0": s0.cpu()}, lens)
        near(y[:T], yr, "y")
        near(s1, sr, "s1")
        assert not y[T:].any()


def test_prompt_then_packed_decode(dev):
    """The whole path: unit-norm rows, scan of a prompt, sq_pack, decode steps, sq_unpack, scan again, gated norm."""
    H, dk, dv, T = 2, 64, 64, 75
    raw = torch.randn(T, 2, H, dk, device=dev)
    q, k = torch.empty(T, H, dk, device=dev), torch.empty(T, H, dk, device=dev)
    sq.sq_norm_in(raw[:, 0], q, kind=sq.SQ_NORM_L2)
    sq.sq_norm_in(raw[:, 1], k, kind=sq.SQ_NORM_L2)
    x = scan_inputs(0, H, H, dk, dv, [T], 61, F32)
    x["q"], x["k"] = q.cpu(), k.cpu()
    d = {n: t.to(dev) for n, t in x.items()}
    y, s1 = forward(0, x, [T], dev, s0=False)
    near(y, scan_ref(x, [T], False)[0], "prompt")
    plan = sq.sq_plan_create(form=0, unit=0, n_layers=1, n_heads=H, d_k=dk, d_v=dv, widths=(8,), budget_milli=8000,
                             pivot_ppm=0, grid=(1.0, 0.875), gate=np.full((1, H), 0.95, np.float32),
                             impact=np.ones((1, H, dk), np.float32), unit_bits=np.full(H, 8, np.int32))
    mem = torch.zeros(sq.sq_pool_bytes(plan, 1), dtype=torch.uint8, device=dev)
    pool = sq.sq_pool_create(plan, mem, 1)
    slot = torch.zeros(1, dtype=torch.int32, device=dev)
    sq.sq_pack(pool, 0, 1, 1, slot, s1)
    back = torch.empty_like(s1)
    sq.sq_unpack(pool, 0, 1, 1, slot, back)
    z = scan_inputs(0, H, H, dk, dv, [1], 62, F32)
    z["s0"] = back.cpu()
    ys = torch.zeros(H * dv, device=dev)
    sq.sq_state_step(pool, 0, 1, 1, slot, *(z[n].to(dev) for n in ("q", "k", "v", "gate", "beta")), ys)
    y1, _ = forward(0, z, [1], dev)
    near(y1.view(-1), ys.cpu(), "decode step against a scan from the unpacked state")
    assert (back - s1).norm() < 0.02 * s1.norm()          # 8-bit codes: 1/254 of a row-and-column scale each
    o = torch.empty(1, H, dv, dtype=BF16, device=dev)
    gate = torch.randn(1, H, dv, device=dev).to(BF16)
    sq.sq_norm_out(ys.view(1, H, dv), o, z=gate)
    yd = ys.double().cpu().view(1, H, dv)
    near(o, yd / (yd.square().mean(-1, keepdim=True) + 1e-6).sqrt() * torch.nn.functional.silu(gate.double().cpu()), "gated norm")
    pool.close()
    plan.close()


@pytest.mark.parametrize("workload", ("gdn-decode-32h-64", "kda-decode-32h-64"))
def test_block_experiment_runs(workload, dev, capsys):
    import argparse
    import json

    import experiments
    experiments.block(argparse.Namespace(workload=workload, prompt=40, batch=3, steps=2))
    got = json.loads(capsys.readouterr().out.strip().splitlines()[-1])
    assert got["experiment"] == "block" and got["requests"] == 3 and np.isfinite(got["output_rel_mean"])


@pytest.mark.parametrize("lens", ([40, 70], [9, 3, 1]), ids=("chunks", "tokens"))
@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_a_nan_gate_is_not_a_reset(form, lens, dev):
    """One gate of NaN: its head's outputs from there to the sequence's end, its last state and the gradients that hold it are
    NaN; the other heads' and sequences' are what they are without it."""
    H, dk, dv, h = 3, 64, 64, 1
    x = scan_inputs(form, H, H, dk, dv, lens, 83, BF16)
    at = lens[0] - 5
    bad = dict(x, gate=x["gate"].clone())
    bad["gate"][(at, h, 7) if form else (at, h)] = float("nan")
    y, s1 = forward(form, bad, lens, dev)
    assert torch.isnan(y[at:lens[0], h]).all() and torch.isnan(s1[0, h]).all()
    g = backward(form, bad, lens, dev)
    assert torch.isnan(g["dq"][at:lens[0], h]).all() and torch.isnan(g["ds0"][0, h]).any()
    ok, rest = forward(form, x, lens, dev), backward(form, x, lens, dev)
    others = [i for i in range(H) if i != h]
    for a, b in ((y, ok[0]), *((g[n], rest[n]) for n in GRADS if n != "ds0")):
        assert torch.equal(a[:, others], b[:, others]) and torch.equal(a[lens[0]:], b[lens[0]:])
    for a, b in ((s1, ok[1]), (g["ds0"], rest["ds0"])):
        assert torch.equal(a[0, others], b[0, others]) and torch.equal(a[1:], b[1:])


@pytest.mark.parametrize("H", (2, 130), ids=("few", "many"))
@pytest.mark.parametrize("dk", (64, 128))
@pytest.mark.parametrize("dt", (BF16, F16, F32), ids=("bfloat16", "float16", "float32"))
@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_outputs_small_against_their_terms(form, dt, dk, H, dev):
    """y = 2^-14 as the difference of two terms of 32 and more that are the same but for a last part of 2^-20: in the state, in
    the updates, in the gates' products of a chunk and (a gate per key row) in those from the state.  A float32 holds each term
    exactly (21 bits), so do three parts of 8 bits, and every partial sum is a multiple of 2^-14 below 2^9; two parts lose y."""
    T, n = 64, 4
    hi, lo, one = 0.5 + 2.0 ** -10 + 2.0 ** -20, 0.5 + 2.0 ** -10, 64.0
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    q, k, v, beta, s0 = z(n * T, H, dk), z(n * T, H, dk), torch.full((n * T, H, dk), one), z(n * T, H), z(n, H, dk, dk)
    gate = torch.ones(n * T, H, dk if form else 1, dtype=torch.float64)
    t, even, odd = torch.arange(T), torch.arange(0, T, 2), torch.arange(1, T, 2)
    # 0: the state holds both terms
    q[t, :, 2 * t % dk], q[t, :, (2 * t + 1) % dk] = 1.0, -1.0
    s0[0, :, 0::2], s0[0, :, 1::2] = one * hi, one * lo
    # 1: a token's update against the one before it
    for b in (1, 2):
        k[b * T + t, :, t] = 1.0
        q[b * T + odd, :, even], q[b * T + odd, :, odd] = 1.0, -1.0
    beta[T + even], beta[T + odd] = hi, lo
    # 2: the update before, times a gate, against the token's own
    beta[2 * T + even], beta[2 * T + odd] = 1.0, lo
    gate[2 * T + odd] = hi
    # 3: the state times a gate per key row (a gate per head: the state itself), the first token of each chunk
    q[3 * T::32, :, 0::2], q[3 * T::32, :, 1::2] = 2.0 / dk, -2.0 / dk
    if form:
        gate[3 * T, :, 0::2] = hi
        s0[3, :, 0::2], s0[3, :, 1::2] = one, one * lo
    else:
        s0[3, :, 0::2], s0[3, :, 1::2] = one * hi, one * lo
    x = {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "gate": (gate if form else gate[..., 0]).float(), "beta": beta.float(), "s0": s0.float()}
    y, s1 = forward(form, x, [T] * n, dev)
    yr, sr = scan_ref(x, [T] * n)
    assert (yr[T + odd] == 2.0 ** -14).all() and (yr[2 * T + odd] == 2.0 ** -14).all() and (yr[:T] == 2.0 ** -14).all()
    assert (yr[3 * T::32] == 2.0 ** -14).all() and not yr[T + even].any()
    near(y, yr, "y")
    near(s1, sr, "s1")


L2, L2_GRAD = 1e-6, 1.5e-6


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_every_part_counts(c, dev):
    """The relative L2 error of the float32 outputs.  A rounding to float32 is off by 2^-24 / sqrt(3) = 3.4e-8 of a partial sum,
    24 of them (six products of parts for each 32 of 128 key rows) in quadrature by 1.7e-7; the terms left out, 2^-24 at most, are
    some 2^-27 in the mean square.  Outputs and states pass through five products (3.7e-7), gradients through twelve (5.9e-7); states hand errors on, damped by the gates;
    terms that cancel, a factor of 2, and for gradients 2.5: 1e-6 and 1.5e-6.  One product of parts lost (say the first with the
    third of two operands) makes 2.6e-6 to 4e-6 of y and the states, which 1e-5 of the largest value does not show."""
    form, dt, H, Hk, dk, dv, lens, gate = c
    x = scan_inputs(form, H, Hk, dk, dv, lens, 29, dt, gate)
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    off = {}
    for n, a, b in [("y", y, yr), ("s1", s1, sr)] + [(n, g[n], r[n]) for n in GRADS]:
        if a.dtype == F32:
            off[n] = ((a.double().cpu() - b).norm() / b.norm()).item(), L2 if n in ("y", "s1") else L2_GRAD
    say({n: f"{e:.2e}" for n, (e, _) in off.items()})
    for n, (e, tol) in off.items():
        assert e <= tol, (n, e)


@pytest.mark.parametrize("value", (float("nan"), float("inf")), ids=("nan", "inf"))
@pytest.mark.parametrize("what", ("q", "k", "v", "beta", "s0"))
@pytest.mark.parametrize("lens", ([90, 40], [16, 3, 1]), ids=("chunks", "tokens"))
@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_a_value_that_is_not_finite_stays_in_its_head(form, lens, what, value, dev):
    """What it reaches is not finite; chunks before it, other heads and sequences keep their bits."""
    H, dk, dv, h = 3, 64, 64, 1
    x = scan_inputs(form, H, H, dk, dv, lens, 84, F32)
    at = 0 if what == "s0" else lens[0] - 10
    bad = dict(x, **{what: x[what].clone()})
    bad[what][{"q": (at, h, 3), "k": (at, h, 3), "v": (at, h), "beta": (at, h), "s0": (0, h)}[what]] = value
    y, s1 = forward(form, bad, lens, dev)
    oy, os_ = forward(form, x, lens, dev)
    end = at + 1 if what == "q" else lens[0]
    assert not torch.isfinite(y[at:end, h]).any()
    assert torch.isfinite(s1[0, h]).any() == (what == "q")
    others, before = [i for i in range(H) if i != h], at // 32 * 32
    assert torch.equal(y[:, others], oy[:, others]) and torch.equal(s1[:, others], os_[:, others])
    assert torch.equal(y[lens[0]:], oy[lens[0]:]) and torch.equal(s1[1:], os_[1:])
    assert torch.equal(y[:before], oy[:before])


@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_one_query_head_for_many_value_heads(form, dev):
    """Sixteen value heads share q and k: dq and dk are sums over all of them."""
    H, dk, dv, lens = 16, 64, 64, [37, 5]
    x = scan_inputs(form, H, 1, dk, dv, lens, 85, F32)
    y, s1 = forward(form, x, lens, dev)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")
    g, r = backward(form, x, lens, dev), scan_grad_ref(x, lens)
    for n in GRADS:
        near(g[n], r[n], n)


@pytest.mark.parametrize("lens", ([40], [6, 3]), ids=("chunks", "tokens"))
@pytest.mark.parametrize("form", (0, 1), ids=("gdn", "kda"))
def test_the_widest_strides(form, lens, dev):
    """float32 rows just below 2^24 elements apart: a chunk of them spans 2 GiB, the arrays more than 4 GiB in between."""
    H, dk, dv, T, stride = 2, 64, 64, sum(lens), (1 << 24) - 4
    x = scan_inputs(form, H, H, dk, dv, lens, 86, F32)
    d = {n: t.to(dev) for n, t in x.items()}
    buf = torch.empty(T, 2, stride // 2, device=dev).view(T, stride)     # parts of one array, far enough apart
    at = iter(range(0, stride, stride // 8 // 4 * 4))
    part = lambda w: buf[:, (i := next(at)):i + H * w].unflatten(1, (H, w))  # noqa: E731
    q, k, v, y, dq, dk_, dv_, dy = (part(w) for w in (dk, dk, dv, dv, dk, dk, dv, dv))
    for a, n in ((q, "q"), (k, "k"), (v, "v"), (dy, "dy")):
        a.copy_(d[n])
    s1, ds0 = torch.zeros_like(d["s0"]), torch.zeros_like(d["s0"])
    dgate, dbeta = torch.zeros_like(d["gate"]), torch.zeros_like(d["beta"])
    sq.sq_delta_scan(form, q, k, v, d["gate"], d["beta"], y, seq_start=starts(lens, dev), s0=d["s0"], s1=s1)
    sq.sq_delta_scan_bwd(form, q, k, v, d["gate"], d["beta"], dy, dq, dk_, dv_, dgate, dbeta, seq_start=starts(lens, dev),
                         s0=d["s0"], ds1=d["ds1"], ds0=ds0)
    yr, sr = scan_ref(x, lens)
    near(y, yr, "y")
    near(s1, sr, "s1")
    r = scan_grad_ref(x, lens)
    for n, t in zip(GRADS, (dq, dk_, dv_, dgate, dbeta, ds0)):
        near(t, r[n], n)
